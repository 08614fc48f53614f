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
  const int total = a.B * a.Hq * NQ, unit = attn_unit(total, G, a.window, a.T, a.B * a.Hkv, total > 3 * 256 ? 4 : 2);
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
// Workgroup = 4 waves x 32 tokens of one query head, key tiles of 32 rows in two pairs of LDS
// buffers: the next tile's loads go straight to LDS while this one is worked on, one barrier a
// tile.  The accumulators are rescaled only when a token's maximum grows by more than 2^8 (weights
// up to 2^8 keep their relative precision in bf16 and fp32).
// Its time is that of the products and the vector work one after the other (counters: matrix cores
// busy 0.54, vector units 0.52; per 32 x 32 scores at D = 128: 16 products of 32 cycles, 16
// exponentials of 16, some 60 other vector instructions of 4).  32 tokens a wave
// and 32 keys a tile keep it at 162 registers, three waves a SIMD: tiles of 64 keys (two waves)
// took 580 us where this took 531, 64 tokens a wave spilled (1,261 us), and the next tile's
// scores formed among this one's exponentials in one wave gained nothing over a second wave.
// B1, 16 heads on 4, T = 32,768, window 2,048, 4 sinks, D = 128: 530 to 565 us from card to card, 0.94
// to 1.01 PFLOP/s of visible pairs (a library product of 8,192^3 reaches 1.20).
constexpr int kFwdQ = 128, kFwdKeys = 32;

template <int D>
__global__ __launch_bounds__(256, 3) void swa_fwd_bf16_kernel(SwaArgs a) {
  using Tile = SwzTile<D, kFwdKeys>;
  constexpr int KK = D / 16, DT = D / 32;
  __shared__ __align__(16) unsigned char K0[Tile::bytes], K1[Tile::bytes];
  __shared__ __align__(16) unsigned char V0[Tile::bytes], V1[Tile::bytes];
  const FwdUnit un = fwd_unit(a, kFwdQ);
  const int n = un.n, t0 = un.t0, lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int tw = t0 + 32 * wave, t = tw + (lane & 31);
  const bf16* kb = reinterpret_cast<const bf16*>(a.k) + (size_t)un.bk * a.T * D;
  const bf16* vb = reinterpret_cast<const bf16*>(a.v) + (size_t)un.bk * a.T * D;

  f32x16 O[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) O[dt] = zero16();
  float m = kNegBig, l = 0.f;
  if (t0 < n) {
    const KeyTiles<kFwdKeys> kt(t0, min(t0 + kFwdQ, n), a.window, a.sinks);
    auto load = [&](unsigned char* Ks, unsigned char* Vs, int i) {
      if (i < kt.count) {
        Tile::template load<4>(Ks, kb, kt[i], kt.rows(i, n), wave);
        Tile::template load<4>(Vs, vb, kt[i], kt.rows(i, n), wave);
      }
    };
    load(K0, V0, 0);
    Frag<bf16> Q[KK];
    const bf16* qr = reinterpret_cast<const bf16*>(a.q) +
                     ((size_t)(un.b * a.Hq + un.hq) * a.T + min(t, n - 1)) * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) Q[kk] = load_frag(qr + 16 * kk);
    const float c = a.scale * kLog2e;
    const int rb = Tile::row_base(), cb = Tile::col_base();

    auto step = [&](const unsigned char* Ks, const unsigned char* Vs, int s0) {
      // nothing of the tile is seen by any of the wave's tokens
      if (s0 > tw + 31 || (s0 >= a.sinks && tw - (s0 + kFwdKeys - 1) >= a.window)) return;
      f32x16 S = zero16();
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) mma32(S, Tile::row_frag(Ks, rb, 0, kk), Q[kk]);
      const bool full = s0 + kFwdKeys - 1 <= tw && (tw + 31 - s0 < a.window || s0 + kFwdKeys <= a.sinks);
      if (!full) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int s = s0 + acc_row(r, half);
          const bool see = (s <= t) & ((t - s < a.window) | (s < a.sinks));
          S[r] = see ? S[r] : -INFINITY;
        }
      }
      float mx = S[0];
#pragma unroll
      for (int r = 1; r < 16; ++r) mx = fmaxf(mx, S[r]);
      mx = fmaxf(mx, other_half(mx)) * c;
      if (__any(mx > m + 8.f)) {
        const float mn = fmaxf(m, mx), alpha = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= alpha;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) O[dt] *= alpha;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        S[r] = __builtin_amdgcn_exp2f(S[r] * c - m);
        l += S[r];
      }
      // the weights are rounded to bf16 for the product with v (their sum is not)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Frag<bf16> P;
        acc_frag(S, x, P);
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) mma32(O[dt], Tile::col_frag(Vs, cb, dt, 16 * x), P);
      }
    };
    for (int i = 0; i < kt.count; i += 2) {
      loads_and_barrier();
      load(K1, V1, i + 1);
      step(K0, V0, kt[i]);
      loads_and_barrier();
      load(K0, V0, i + 2);
      if (i + 1 < kt.count) step(K1, V1, kt[i + 1]);
    }
  }
  fwd_store<bf16, D>(a, un, t, O, m, l + other_half(l));
}

// ------------------------------------------------------------------ fp32
// As above with one tile of 64 keys in LDS (padded rows, staged through registers).  Bound by the fp32
// products, a sixteenth of the bf16 rate.
constexpr int kFwdK = 64;

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
    kst.load(kb, tile[0], tile.rows(0, n));
    vst.load(vb, tile[0], tile.rows(0, n));
    for (int i = 0; i < tile.count; ++i) {
      const int s0 = tile[i];
      __syncthreads();
      kst.store(Ks);
      vst.store(Vs);
      __syncthreads();
      if (i + 1 < tile.count) {
        kst.load(kb, tile[i + 1], tile.rows(i + 1, n));
        vst.load(vb, tile[i + 1], tile.rows(i + 1, n));
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

template <int D>
static hipError_t launch_bf16(const SwaArgs& a, hipStream_t st) {
  return launch_kernel<0>(swa_fwd_bf16_kernel<D>, dim3(a.B * a.Hq * ((a.T + kFwdQ - 1) / kFwdQ)), 256, a, st);
}
template <int D>
static hipError_t launch_f32(const SwaArgs& a, hipStream_t st) {
  constexpr size_t lds = sizeof(float) * 2 * kFwdK * RowStage<float, kFwdK, D, 256>::LD;
  return launch_kernel<lds>(swa_fwd_f32_kernel<D>, dim3(a.B * a.Hq * ((a.T + kFwdQ - 1) / kFwdQ)), 256, a, st);
}

hipError_t launch_swa_fwd(const SwaArgs& a, hipStream_t st) {
  if (a.dtype) return a.D == 128 ? launch_bf16<128>(a, st) : launch_bf16<64>(a, st);
  return a.D == 128 ? launch_f32<128>(a, st) : launch_f32<64>(a, st);
}

}  // namespace carve
