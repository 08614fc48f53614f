// Backward pass of sliding-window attention with sinks.
//
// With p_ts = exp(scale q_t . k_s - lse_t) and delta_t = dO_t . o_t:
//   ds_ts = p_ts (dO_t . v_s - delta_t)
//   dq_t = scale sum_s ds_ts k_s,   dk_s = scale sum_t ds_ts q_t,   dv_s = sum_t p_ts dO_t,
// the last two also summed over the query heads that share the key head.  Two passes, each
// with its sums in registers in a fixed order, and no atomics: one over the keys of a tile
// of tokens (dq, and delta for the other pass), one over the tokens of a tile of keys.
// That is seven products of a visible pair where one pass with shared sums has five.
#include <algorithm>

#include "attn_device.h"

namespace carve {

constexpr int kDqQ = 128, kDqK = 64;

// ------------------------------------------------------------------ dq
// Workgroup = 128 tokens of one query head, as in the forward pass.
template <typename T, int D>
__global__ __launch_bounds__(256) void swa_dq_kernel(SwaArgs a) {
  using St = RowStage<T, kDqK, D, 256>;
  constexpr int LD = St::LD;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Ks = reinterpret_cast<T*>(smem);
  T* Vs = Ks + kDqK * LD;
  const int G = a.Hq / a.Hkv, NQ = (a.T + kDqQ - 1) / kDqQ;
  const int unit = xcd_unit(a.B * a.Hq * NQ);
  const int g = unit % G, qt = NQ - 1 - (unit / G) % NQ, bk = unit / (G * NQ);
  const int b = bk / a.Hkv, hq = (bk % a.Hkv) * G + g;
  const int n = seq_len(a.lens, b, a.T);
  const int lane = lane_id(), wave = wave_id(), half = lane >> 5;
  const int t0 = qt * kDqQ, tw = t0 + 32 * wave, t = tw + (lane & 31);
  const size_t row = (size_t)(b * a.Hq + hq) * a.T;
  const T* kb = reinterpret_cast<const T*>(a.k) + (size_t)bk * a.T * D;
  const T* vb = reinterpret_cast<const T*>(a.v) + (size_t)bk * a.T * D;

  f32x16 dQ[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) dQ[dt] = zero16();
  if (t0 < n) {
    Frag<T> Q[D / 16], dO[D / 16];
    const size_t at = (row + min(t, n - 1)) * D + 8 * half;
    // delta_t from the product of the rows of o with dO, formed as dO . v is below: a token
    // that sees one key has o = v, and its ds is zero to the last bit
    f32x16 od = zero16();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      Q[kk] = load_frag(reinterpret_cast<const T*>(a.q) + at + 16 * kk);
      dO[kk] = load_frag(reinterpret_cast<const T*>(a.dO) + at + 16 * kk);
      mma32(od, load_frag(reinterpret_cast<const T*>(a.o) + at + 16 * kk), dO[kk]);
    }
    float delta = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) delta = acc_row(r, half) == (lane & 31) ? od[r] : delta;
    const float other = __shfl_xor(delta, 32);
    if (((lane >> 2) & 1) != half) delta = other;
    if (half == 0 && t < n) a.delta[row + t] = delta;
    const float c = a.scale * kLog2e;
    const float lse = a.lse[row + min(t, n - 1)];
    const float lse2 = lse == -INFINITY ? INFINITY : lse * kLog2e;    // no visible weight: p = 0
    const int hi = min(t0 + kDqQ, n);
    const int kt_lo = max(0, t0 - a.window + 1) / kDqK, kt_hi = (hi - 1) / kDqK;
    const int nsink = min((min(a.sinks, hi) + kDqK - 1) / kDqK, kt_lo);
    const int ntile = nsink + kt_hi - kt_lo + 1;
    auto tile = [&](int i) { return (i < nsink ? i : kt_lo + i - nsink) * kDqK; };
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
      for (int u = 0; u < kDqK / 32; ++u) {
        const int su = s0 + 32 * u;
        if (su > tw + 31 || (su >= a.sinks && tw - (su + 31) >= a.window)) continue;
        f32x16 S = zero16(), dP = zero16();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          mma32(S, frag_rows32(Ks, LD, 32 * u, 16 * kk), Q[kk]);
          mma32(dP, frag_rows32(Vs, LD, 32 * u, 16 * kk), dO[kk]);
        }
        const bool full = su + 31 <= tw && (tw + 31 - su < a.window || su + 32 <= a.sinks);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float p = __builtin_amdgcn_exp2f(S[r] * c - lse2);
          if (!full) {
            const int s = su + acc_row(r, half);
            if (!(s <= t && (t - s < a.window || s < a.sinks))) p = 0.f;
          }
          S[r] = p == 0.f ? 0.f : p * (dP[r] - delta);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Frag<T> F;
          acc_frag(S, x, F);       // ds rounded to the operand type for its product with k
#pragma unroll
          for (int dt = 0; dt < D / 32; ++dt) mma32(dQ[dt], frag_cols32(Ks, LD, 32 * dt, 32 * u + 16 * x), F);
        }
      }
    }
  }
  if (t < a.T) {
    if (t >= n) {
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) dQ[dt] = zero16();
    }
    store_column<T, D>(reinterpret_cast<T*>(a.dq) + (row + t) * D, dQ, a.scale);
  }
}

// ------------------------------------------------------------------ dk, dv
// Workgroup = 128 keys of one key head (32 a wave, a lane owns one key), over the tokens that
// see them inside the window and all heads of the group.  The tokens behind the window of a
// tile that holds sinks see only the sinks: they are cut into n_far ranges with workgroups of
// their own, whose sums, like the tile's, go to `part` and are added by swa_sink_kernel.
constexpr int kDkQ = 32;

template <typename T, int D>
__global__ __launch_bounds__(256) void swa_dkdv_kernel(SwaArgs a) {
  using St = RowStage<T, kDkQ, D, 256>;
  constexpr int LD = St::LD, KT = kSwaKeyTile;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Qs = reinterpret_cast<T*>(smem);
  T* Gs = Qs + kDkQ * LD;                                  // dO
  float* Ls = reinterpret_cast<float*>(Gs + kDkQ * LD);    // lse in the log2 domain, delta
  const int G = a.Hq / a.Hkv, NK = (a.T + KT - 1) / KT;
  const int per = NK + a.n_sink_tiles * a.n_far;           // units of one key head
  const int unit = xcd_unit(a.B * a.Hkv * per);
  const int bk = unit / per, w = unit % per;
  const bool far = w >= NK;
  const int kt = far ? (w - NK) / a.n_far : w, fi = far ? (w - NK) % a.n_far : 0;
  const int b = bk / a.Hkv;
  const int n = seq_len(a.lens, b, a.T);
  const int lane = lane_id(), wave = wave_id(), half = lane >> 5;
  const int s0 = kt * KT, sw = s0 + 32 * wave, s = sw + (lane & 31);
  // tokens of this unit
  const long long band = (long long)s0 + KT - 1 + a.window;          // first token that sees no key of the tile
  int t_lo, t_hi;
  if (!far) {
    t_lo = s0;
    t_hi = (int)min((long long)n, band);
  } else {
    const long long f = band + (long long)fi * a.far_len;
    t_lo = (int)min((long long)n, f);
    t_hi = (int)min((long long)n, f + a.far_len);
  }
  f32x16 dK[D / 32], dV[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) {
    dK[dt] = zero16();
    dV[dt] = zero16();
  }
  if (t_lo < t_hi && s0 < n) {
    Frag<T> K[D / 16], V[D / 16];
    const size_t at = ((size_t)bk * a.T + min(s, n - 1)) * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      K[kk] = load_frag(reinterpret_cast<const T*>(a.k) + at + 16 * kk);
      V[kk] = load_frag(reinterpret_cast<const T*>(a.v) + at + 16 * kk);
    }
    const float c = a.scale * kLog2e;
    const int nt = (t_hi - t_lo + kDkQ - 1) / kDkQ, total = nt * G;
    St qst, gst;
    float lst = 0.f, dst = 0.f;
    auto load = [&](int i) {
      const int hq = (bk % a.Hkv) * G + i / nt, tt = t_lo + (i % nt) * kDkQ;
      const size_t row = (size_t)(b * a.Hq + hq) * a.T;
      qst.load(reinterpret_cast<const T*>(a.q) + row * D, tt, t_hi);
      gst.load(reinterpret_cast<const T*>(a.dO) + row * D, tt, t_hi);
      if (threadIdx.x < kDkQ) {
        const int t = tt + threadIdx.x;
        // past the end, or no visible weight: p = exp2(. - inf) = 0
        const float lse = t < t_hi ? a.lse[row + t] : -INFINITY;
        lst = lse == -INFINITY ? INFINITY : lse * kLog2e;
        dst = t < t_hi ? a.delta[row + t] : 0.f;
      }
    };
    load(0);
    for (int i = 0; i < total; ++i) {
      const int tt = t_lo + (i % nt) * kDkQ;
      __syncthreads();
      qst.store(Qs);
      gst.store(Gs);
      if (threadIdx.x < kDkQ) {
        Ls[threadIdx.x] = lst;
        Ls[kDkQ + threadIdx.x] = dst;
      }
      __syncthreads();
      if (i + 1 < total) load(i + 1);
      if (sw > tt + 31 || (sw >= a.sinks && tt - (sw + 31) >= a.window)) continue;
      f32x16 S = zero16(), dP = zero16();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        mma32(S, frag_rows32(Qs, LD, 0, 16 * kk), K[kk]);
        mma32(dP, frag_rows32(Gs, LD, 0, 16 * kk), V[kk]);
      }
      const bool full = sw + 31 <= tt && (tt + 31 - sw < a.window || sw + 32 <= a.sinks);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 ls = *reinterpret_cast<const f32x4*>(Ls + 8 * q + 4 * half);
        const f32x4 de = *reinterpret_cast<const f32x4*>(Ls + kDkQ + 8 * q + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * q + e;
          float p = __builtin_amdgcn_exp2f(S[r] * c - ls[e]);
          if (!full) {
            const int t = tt + acc_row(r, half);
            if (!(s <= t && (t - s < a.window || s < a.sinks))) p = 0.f;
          }
          S[r] = p;
          dP[r] = p == 0.f ? 0.f : p * (dP[r] - de[e]);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Frag<T> P, F;              // p and ds rounded to the operand type for the products
        acc_frag(S, x, P);
        acc_frag(dP, x, F);
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) {
          mma32(dV[dt], frag_cols32(Gs, LD, 32 * dt, 16 * x), P);
          mma32(dK[dt], frag_cols32(Qs, LD, 32 * dt, 16 * x), F);
        }
      }
    }
  }
  if (kt < a.n_sink_tiles && a.n_far > 0) {
    float* dst = a.part + ((((size_t)bk * a.n_sink_tiles + kt) * (1 + a.n_far) + (far ? 1 + fi : 0)) * 2 * KT +
                           32 * wave + (lane & 31)) * D;
    store_column<float, D>(dst, dK, a.scale);
    store_column<float, D>(dst + (size_t)KT * D, dV, 1.f);
  } else if (s < a.T) {
    if (s >= n) {
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) {
        dK[dt] = zero16();
        dV[dt] = zero16();
      }
    }
    const size_t row = ((size_t)bk * a.T + s) * D;
    store_column<T, D>(reinterpret_cast<T*>(a.dk) + row, dK, a.scale);
    store_column<T, D>(reinterpret_cast<T*>(a.dv) + row, dV, 1.f);
  }
}

// dk, dv of the tiles that hold sinks: the sums of the tile's window and far ranges, in order.
template <typename T, int D>
__global__ __launch_bounds__(256) void swa_sink_kernel(SwaArgs a) {
  constexpr int KT = kSwaKeyTile, PR = D / 4;
  const int kt = blockIdx.x % a.n_sink_tiles, bk = blockIdx.x / a.n_sink_tiles;
  const int n = seq_len(a.lens, bk / a.Hkv, a.T);
  const float* src = a.part + ((size_t)bk * a.n_sink_tiles + kt) * (1 + a.n_far) * 2 * KT * D;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < 2 * KT * PR; i += 256 * gridDim.y) {
    const int which = i / (KT * PR), r = (i / PR) % KT, s = kt * KT + r;
    if (s >= a.T) continue;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    if (s < n)
      for (int f = 0; f <= a.n_far; ++f) x += load4f(src + (size_t)f * 2 * KT * D + (size_t)i * 4);
    T* dst = reinterpret_cast<T*>(which ? a.dv : a.dk);
    store4(dst + ((size_t)bk * a.T + s) * D + 4 * (i % PR), x);
  }
}

template <typename T, int D>
static hipError_t launch(const SwaArgs& a, hipStream_t st) {
  constexpr size_t lds_q = sizeof(T) * 2 * kDqK * RowStage<T, kDqK, D, 256>::LD;
  constexpr size_t lds_k = sizeof(T) * 2 * kDkQ * RowStage<T, kDkQ, D, 256>::LD + sizeof(float) * 2 * kDkQ;
  hipError_t e =
      launch_kernel<lds_q>(swa_dq_kernel<T, D>, dim3(a.B * a.Hq * ((a.T + kDqQ - 1) / kDqQ)), 256, a, st);
  if (e != hipSuccess) return e;
  const int per = (a.T + kSwaKeyTile - 1) / kSwaKeyTile + a.n_sink_tiles * a.n_far;
  e = launch_kernel<lds_k>(swa_dkdv_kernel<T, D>, dim3(a.B * a.Hkv * per), 256, a, st);
  if (e != hipSuccess || a.n_sink_tiles * a.n_far == 0) return e;
  return launch_kernel<0>(swa_sink_kernel<T, D>, dim3(a.B * a.Hkv * a.n_sink_tiles, 8), 256, a, st);
}

hipError_t launch_swa_bwd(const SwaArgs& a, hipStream_t st) {
  if (a.dtype) return a.D == 128 ? launch<bf16, 128>(a, st) : launch<bf16, 64>(a, st);
  return a.D == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
}

}  // namespace carve
