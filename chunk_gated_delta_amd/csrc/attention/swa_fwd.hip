// Forward pass of sliding-window attention with sinks.
//
// One pass over the visible keys with a running maximum and sum: for the tokens t of a tile
//   s_tj = scale q_t . k_j,  m = max,  l = sum exp(s - m),  o_t = sum exp(s - m) v_j / l,
//   lse_t = m + log l,
// key tiles taken in the order sinks, then window.  Workgroup = 128 tokens of one query
// head (32 a wave); S^T = K Q^T and O^T = V^T P^T, so a lane owns one token and the
// weights stay in its registers between the two products.
#include <algorithm>

#include "attn_device.h"

namespace carve {

constexpr int kFwdQ = 128, kFwdK = 64;

template <typename T, int D>
__global__ __launch_bounds__(256) void swa_fwd_kernel(SwaArgs a) {
  using St = RowStage<T, kFwdK, D, 256>;
  constexpr int LD = St::LD;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Ks = reinterpret_cast<T*>(smem);
  T* Vs = Ks + kFwdK * LD;
  const int G = a.Hq / a.Hkv, NQ = (a.T + kFwdQ - 1) / kFwdQ;
  const int unit = xcd_unit(a.B * a.Hq * NQ);
  const int g = unit % G, qt = NQ - 1 - (unit / G) % NQ, bk = unit / (G * NQ);   // bk = b * Hkv + key head
  const int b = bk / a.Hkv, hq = (bk % a.Hkv) * G + g;
  const int n = seq_len(a.lens, b, a.T);
  const int lane = lane_id(), wave = wave_id(), half = lane >> 5;
  const int t0 = qt * kFwdQ, tw = t0 + 32 * wave, t = tw + (lane & 31);
  const size_t row = (size_t)(b * a.Hq + hq) * a.T;
  const T* qb = reinterpret_cast<const T*>(a.q) + row * D;
  T* ob = reinterpret_cast<T*>(a.o) + row * D;
  const T* kb = reinterpret_cast<const T*>(a.k) + (size_t)bk * a.T * D;
  const T* vb = reinterpret_cast<const T*>(a.v) + (size_t)bk * a.T * D;

  f32x16 O[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) O[dt] = zero16();
  float m = kNegBig, l = 0.f;
  if (t0 < n) {
    Frag<T> Q[D / 16];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) Q[kk] = load_frag(qb + (size_t)min(t, n - 1) * D + 16 * kk + 8 * half);
    const float c = a.scale * kLog2e;
    const int hi = min(t0 + kFwdQ, n);                          // keys 0 .. hi - 1 at most
    const int kt_lo = max(0, t0 - a.window + 1) / kFwdK, kt_hi = (hi - 1) / kFwdK;
    const int nsink = min((min(a.sinks, hi) + kFwdK - 1) / kFwdK, kt_lo);
    const int ntile = nsink + kt_hi - kt_lo + 1;
    auto tile = [&](int i) { return (i < nsink ? i : kt_lo + i - nsink) * kFwdK; };
    St kst, vst;
    kst.load(kb, tile(0), n);
    vst.load(vb, tile(0), n);
    for (int i = 0; i < ntile; ++i) {
      const int s0 = tile(i);
      __syncthreads();
      kst.store(Ks);
      vst.store(Vs);
      __syncthreads();
      if (i + 1 < ntile) {
        kst.load(kb, tile(i + 1), n);
        vst.load(vb, tile(i + 1), n);
      }
#pragma unroll
      for (int u = 0; u < kFwdK / 32; ++u) {
        const int su = s0 + 32 * u;
        // no token of this wave sees a key of these 32
        if (su > tw + 31 || (su >= a.sinks && tw - (su + 31) >= a.window)) continue;
        f32x16 S = zero16();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) mma32(S, frag_rows32(Ks, LD, 32 * u, 16 * kk), Q[kk]);
        const bool full = su + 31 <= tw && (tw + 31 - su < a.window || su + 32 <= a.sinks);
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          S[r] *= c;
          if (!full) {
            const int s = su + acc_row(r, half);
            if (!(s <= t && (t - s < a.window || s < a.sinks))) S[r] = -INFINITY;
          }
          mx = fmaxf(mx, S[r]);
        }
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float mn = fmaxf(m, mx), alpha = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) O[dt] *= alpha;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          S[r] = __builtin_amdgcn_exp2f(S[r] - m);
          l += S[r];
        }
        // the weights are rounded to the operand type for the product with v (the sum l is not)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Frag<T> P;
          acc_frag(S, x, P);
#pragma unroll
          for (int dt = 0; dt < D / 32; ++dt) mma32(O[dt], frag_cols32(Vs, LD, 32 * dt, 32 * u + 16 * x), P);
        }
      }
    }
    l += __shfl_xor(l, 32);
  }
  if (t < a.T) {
    const bool live = t < n && l > 0.f;
    if (!live) {
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) O[dt] = zero16();
    }
    store_column<T, D>(ob + (size_t)t * D, O, live ? 1.f / l : 0.f);
    if (a.lse && half == 0) a.lse[row + t] = live ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
  }
}

template <typename T, int D>
static hipError_t launch(const SwaArgs& a, hipStream_t st) {
  constexpr size_t lds = sizeof(T) * 2 * kFwdK * RowStage<T, kFwdK, D, 256>::LD;
  return launch_kernel<lds>(swa_fwd_kernel<T, D>, dim3(a.B * a.Hq * ((a.T + kFwdQ - 1) / kFwdQ)), 256, a, st);
}

hipError_t launch_swa_fwd(const SwaArgs& a, hipStream_t st) {
  if (a.dtype) return a.D == 128 ? launch<bf16, 128>(a, st) : launch<bf16, 64>(a, st);
  return a.D == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
}

}  // namespace carve
