// Forward pass of sliding-window attention with sinks.
//
// One pass over the visible keys with a running maximum and sum: for the tokens t of a tile
//   s_tj = scale q_t . k_j,  m = max,  l = sum exp(s - m),  o_t = sum exp(s - m) v_j / l,
//   lse_t = m + log l,
// key tiles taken in the order sinks, then window.  S^T = K Q^T and O^T = V^T P^T, so a lane
// owns one token and its weights stay in registers between the two products.
#include <algorithm>

#include "attn_device.h"

namespace carve {

struct FwdUnit {
  int b, bk, hq, t0, n;
};
// unit of work -> (sequence, key head, query head, first token): the heads of a group and the
// tiles of a key head next to each other, late tokens (which see the most keys) first
__device__ __forceinline__ FwdUnit fwd_unit(const SwaArgs& a, int QT) {
  const int G = a.Hq / a.Hkv, NQ = (a.T + QT - 1) / QT;
  const int unit = attn_unit(a.B * a.Hq * NQ, G, a.window, a.T);
  FwdUnit u;
  u.bk = uniform(unit / (G * NQ));
  u.t0 = uniform((NQ - 1 - (unit / G) % NQ) * QT);
  u.b = uniform(u.bk / a.Hkv);
  u.hq = uniform((u.bk % a.Hkv) * G + unit % G);
  u.n = seq_len(a.lens, u.b, a.T);
  return u;
}

template <typename T, int D>
__device__ __forceinline__ void fwd_store(const SwaArgs& a, const FwdUnit& u, int t, f32x16 (&O)[D / 32], float m, float l) {
  if (t >= a.T) return;
  const size_t row = (size_t)(u.b * a.Hq + u.hq) * a.T + t;
  const bool live = t < u.n && l != 0.f;        // (a sum that is not a number stays one)
  if (!live) {
#pragma unroll
    for (int dt = 0; dt < D / 32; ++dt) O[dt] = zero16();
  }
  store_column<T, D>(reinterpret_cast<T*>(a.o) + row * D, O, live ? 1.f / l : 0.f);
  if (a.lse && (lane_id() >> 5) == 0) a.lse[row] = live ? (m + __builtin_amdgcn_logf(l)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------------ bf16
// Workgroup = 4 waves x 32 NQ tokens of one query head, key tiles of 64 rows in two pairs of LDS
// buffers: the next tile's loads go straight to LDS while this one is worked on, one barrier a tile.
// The accumulators are rescaled only when a token's maximum grows by more than 2^8 (weights
// up to 2^8 keep their relative precision in bf16 and fp32).
constexpr int kFwdK = 64, kFwdKeys = 32;

template <int D, int NQ>
__global__ __launch_bounds__(256, 3) void swa_fwd_bf16_kernel(SwaArgs a) {
  using Tile = SwzTile<D, kFwdKeys>;
  constexpr int QW = 32 * NQ, QT = 4 * QW, KK = D / 16, DT = D / 32;
  __shared__ __align__(16) unsigned char K0[Tile::bytes], K1[Tile::bytes];
  __shared__ __align__(16) unsigned char V0[Tile::bytes], V1[Tile::bytes];
  const FwdUnit un = fwd_unit(a, QT);
  const int n = un.n, t0 = un.t0, lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int tw = t0 + QW * wave;
  const bf16* kb = reinterpret_cast<const bf16*>(a.k) + (size_t)un.bk * a.T * D;
  const bf16* vb = reinterpret_cast<const bf16*>(a.v) + (size_t)un.bk * a.T * D;

  f32x16 O[NQ][DT];
  float m[NQ], l[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) O[q][dt] = zero16();
    m[q] = kNegBig;
    l[q] = 0.f;
  }
  if (t0 < n) {
    const KeyTiles<kFwdKeys> kt(t0, min(t0 + QT, n), a.window, a.sinks);
    Tile::template load<4>(K0, kb, kt[0], n, wave);
    Tile::template load<4>(V0, vb, kt[0], n, wave);
    Frag<bf16> Q[NQ][KK];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const bf16* qr = reinterpret_cast<const bf16*>(a.q) +
                       ((size_t)(un.b * a.Hq + un.hq) * a.T + min(tw + 32 * q + (lane & 31), n - 1)) * D + 8 * half;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) Q[q][kk] = load_frag(qr + 16 * kk);
    }
    const float c = a.scale * kLog2e;
    const int rb = Tile::row_base(), cb = Tile::col_base();

    // one tile of 64 keys from s0 against the wave's 32 tokens from ts
    auto block = [&](const unsigned char* Ks, const unsigned char* Vs, int s0, int ts, bool masked, const Frag<bf16>(&Qf)[KK],
                     f32x16(&Of)[DT], float& mf, float& lf) {
      f32x16 S[kFwdKeys / 32];
#pragma unroll
      for (int u = 0; u < kFwdKeys / 32; ++u) {
        S[u] = zero16();
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) mma32(S[u], Tile::row_frag(Ks, rb, 32 * u, kk), Qf[kk]);
      }
      if (masked) {
        const int t = ts + (lane & 31);
#pragma unroll
        for (int u = 0; u < kFwdKeys / 32; ++u)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int s = s0 + 32 * u + acc_row(r, half);
            const bool see = (s <= t) & ((t - s < a.window) | (s < a.sinks));
            S[u][r] = see ? S[u][r] : -INFINITY;
          }
      }
      float mx = S[0][0];
#pragma unroll
      for (int u = 0; u < kFwdKeys / 32; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, S[u][r]);
      mx = fmaxf(mx, other_half(mx)) * c;
      if (__any(mx > mf + 8.f)) {
        const float mn = fmaxf(mf, mx), alpha = __builtin_amdgcn_exp2f(mf - mn);
        mf = mn;
        lf *= alpha;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) Of[dt] *= alpha;
      }
#pragma unroll
      for (int u = 0; u < kFwdKeys / 32; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          S[u][r] = __builtin_amdgcn_exp2f(S[u][r] * c - mf);
          lf += S[u][r];
        }
      // the weights are rounded to bf16 for the product with v (their sum is not)
#pragma unroll
      for (int u = 0; u < kFwdKeys / 32; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Frag<bf16> P;
          acc_frag(S[u], x, P);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) mma32(Of[dt], Tile::col_frag(Vs, cb, dt, 32 * u + 16 * x), P);
        }
    };
    auto step = [&](const unsigned char* Ks, const unsigned char* Vs, int s0) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int ts = tw + 32 * q;
        // nothing of the tile is seen / all of it is seen by all of the 32 tokens
        if (s0 > ts + 31 || (s0 >= a.sinks && ts - (s0 + kFwdKeys - 1) >= a.window)) continue;
        const bool full = s0 + kFwdKeys - 1 <= ts && (ts + 31 - s0 < a.window || s0 + kFwdKeys <= a.sinks);
        block(Ks, Vs, s0, ts, !full, Q[q], O[q], m[q], l[q]);
      }
    };
    for (int i = 0; i < kt.count; i += 2) {
      loads_and_barrier();
      if (i + 1 < kt.count) {
        Tile::template load<4>(K1, kb, kt[i + 1], n, wave);
        Tile::template load<4>(V1, vb, kt[i + 1], n, wave);
      }
      step(K0, V0, kt[i]);
      loads_and_barrier();
      if (i + 2 < kt.count) {
        Tile::template load<4>(K0, kb, kt[i + 2], n, wave);
        Tile::template load<4>(V0, vb, kt[i + 2], n, wave);
      }
      if (i + 1 < kt.count) step(K1, V1, kt[i + 1]);
    }
  }
#pragma unroll
  for (int q = 0; q < NQ; ++q)
    fwd_store<bf16, D>(a, un, tw + 32 * q + (lane & 31), O[q], m[q], l[q] + other_half(l[q]));
}

// ------------------------------------------------------------------ fp32
// As above with one tile in LDS (padded rows, staged through registers) and a product per 32 keys.
constexpr int kFwdQ = 128;

template <int D>
__global__ __launch_bounds__(256) void swa_fwd_f32_kernel(SwaArgs a) {
  using T = float;
  using St = RowStage<T, kFwdK, D, 256>;
  constexpr int LD = St::LD;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Ks = reinterpret_cast<T*>(smem);
  T* Vs = Ks + kFwdK * LD;
  const FwdUnit un = fwd_unit(a, kFwdQ);
  const int n = un.n, t0 = un.t0, lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int tw = t0 + 32 * wave, t = tw + (lane & 31);
  const T* qb = reinterpret_cast<const T*>(a.q) + (size_t)(un.b * a.Hq + un.hq) * a.T * D;
  const T* kb = reinterpret_cast<const T*>(a.k) + (size_t)un.bk * a.T * D;
  const T* vb = reinterpret_cast<const T*>(a.v) + (size_t)un.bk * a.T * D;

  f32x16 O[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) O[dt] = zero16();
  float m = kNegBig, l = 0.f;
  if (t0 < n) {
    Frag<T> Q[D / 16];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) Q[kk] = load_frag(qb + (size_t)min(t, n - 1) * D + 16 * kk + 8 * half);
    const float c = a.scale * kLog2e;
    const KeyTiles<kFwdK> tile(t0, min(t0 + kFwdQ, n), a.window, a.sinks);
    St kst, vst;
    kst.load(kb, tile[0], n);
    vst.load(vb, tile[0], n);
    for (int i = 0; i < tile.count; ++i) {
      const int s0 = tile[i];
      __syncthreads();
      kst.store(Ks);
      vst.store(Vs);
      __syncthreads();
      if (i + 1 < tile.count) {
        kst.load(kb, tile[i + 1], n);
        vst.load(vb, tile[i + 1], n);
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
  fwd_store<T, D>(a, un, t, O, m, l);
}

template <int D, int NQ>
static hipError_t launch_bf16(const SwaArgs& a, hipStream_t st) {
  return launch_kernel<0>(swa_fwd_bf16_kernel<D, NQ>, dim3(a.B * a.Hq * ((a.T + 128 * NQ - 1) / (128 * NQ))), 256, a, st);
}
template <int D>
static hipError_t launch_f32(const SwaArgs& a, hipStream_t st) {
  constexpr size_t lds = sizeof(float) * 2 * kFwdK * RowStage<float, kFwdK, D, 256>::LD;
  return launch_kernel<lds>(swa_fwd_f32_kernel<D>, dim3(a.B * a.Hq * ((a.T + kFwdQ - 1) / kFwdQ)), 256, a, st);
}

hipError_t launch_swa_fwd(const SwaArgs& a, hipStream_t st) {
  if (a.dtype) return a.D == 128 ? launch_bf16<128, 1>(a, st) : launch_bf16<64, 1>(a, st);
  return a.D == 128 ? launch_f32<128>(a, st) : launch_f32<64>(a, st);
}

}  // namespace carve
