// Attention weight that every key receives: w_s = sum over the tokens that see s and the query
// heads that share its key head of p_ts = exp(scale q_t . k_s - lse_t).
//
// Workgroup = 128 keys of one key head (32 a wave, a lane owns one key, k in registers) and a
// range of tokens; S = Q K^T puts the keys on the columns, so a key's weights are added up
// in its lane.  The sums of the token ranges are added in order by weight_sum_kernel.
#include "attn_device.h"

namespace carve {

constexpr int kWtK = 128;

// A unit of work: keys s0 .. + 127 of a key head, the tokens t_lo .. t_hi - 1 (a range that may see
// them; t_lo >= t_hi: none) and the heads h_lo .. h_hi - 1 of the group.
struct WeightUnit {
  int b, bk, n, part, s0, t_lo, t_hi, h_lo, h_hi;
};
__device__ __forceinline__ WeightUnit weight_unit(const WeightArgs& a) {
  const int NK = (a.T + kWtK - 1) / kWtK;
  const int parts = a.n_chunk * a.n_head;
  const int unit = attn_unit(a.B * a.Hkv * NK * parts, 1, a.window, a.T, a.B * a.Hkv, 4);
  WeightUnit u;
  u.s0 = uniform(unit % NK) * kWtK;
  u.part = uniform((unit / NK) % parts);
  u.bk = uniform(unit / (NK * parts));
  const int ch = u.part / a.n_head, G = a.Hq / a.Hkv, per = (G + a.n_head - 1) / a.n_head;
  u.h_lo = uniform(u.part % a.n_head * per);
  u.h_hi = min(G, u.h_lo + per);
  u.b = uniform(u.bk / a.Hkv);
  u.n = seq_len(a.lens, u.b, a.T);
  u.t_lo = uniform(max(ch * a.chunk, u.s0));
  u.t_hi = uniform((int)min((long long)u.n, (long long)(ch + 1) * a.chunk));
  // behind the window of the tile only sinks are seen
  if (u.s0 >= a.sinks) u.t_hi = uniform((int)min((long long)u.t_hi, (long long)u.s0 + kWtK - 1 + a.window));
  return u;
}
__device__ __forceinline__ void weight_store(const WeightArgs& a, const WeightUnit& u, int s, float sum) {
  sum += __shfl_xor(sum, 32);
  if ((lane_id() >> 5) == 0 && s < a.T) {
    float* dst = a.n_chunk * a.n_head > 1 ? a.part + ((size_t)u.part * a.B * a.Hkv + u.bk) * a.T : a.out + (size_t)u.bk * a.T;
    dst[s] = s < u.n ? sum : 0.f;
  }
}

// ------------------------------------------------------------------ bf16
// Tiles of 64 tokens in two swizzled LDS buffers filled by direct loads; their lse goes through a
// register one tile ahead.  Little state a wave (k and one sum): four waves a SIMD.  Its time is that of
// the vector work and the products one after the other (vector units 0.58, matrix cores 0.47; per 32 x
// 32 scores at D = 128: 16 exponentials of 16 cycles, 32 vector instructions of 4, 8 products of
// 32).  B1, 16 heads on 4, T = 8,192: 174 us, 0.79 PFLOP/s of visible pairs.  With a window, the
// tiles of sinks walk every token of their range for the sinks alone: T = 32,768, window 2,048, 340 us
// without sinks and 955 with four.
constexpr int kWtRows = 64;

template <int D>
__global__ __launch_bounds__(256, 4) void weight_bf16_kernel(WeightArgs a) {
  using Tile = SwzTile<D, kWtRows>;
  constexpr int KK = D / 16;
  __shared__ __align__(16) unsigned char Q0[Tile::bytes], Q1[Tile::bytes];
  __shared__ __align__(16) float L0[kWtRows], L1[kWtRows];
  const WeightUnit un = weight_unit(a);
  const int G = a.Hq / a.Hkv, n = un.n, t_lo = un.t_lo, t_hi = un.t_hi;
  const int lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int sw = un.s0 + 32 * wave, s = sw + (lane & 31);
  float sum = 0.f;
  if (t_lo < t_hi && un.h_lo < un.h_hi) {
    Frag<bf16> K[KK];
    const size_t at = ((size_t)un.bk * a.T + min(s, n - 1)) * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) K[kk] = load_frag(reinterpret_cast<const bf16*>(a.k) + at + 16 * kk);
    const float c = a.scale * kLog2e;
    const int nt = (t_hi - t_lo + kWtRows - 1) / kWtRows, total = nt * (un.h_hi - un.h_lo), rb = Tile::row_base();
    const int row0 = un.b * a.Hq + (un.bk % a.Hkv) * G;
    int lg = un.h_lo, lt = 0;              // head and tile of the next load
    float lse = 0.f;
    auto load = [&](unsigned char* Qs) {
      if (lg >= un.h_hi) return;
      const size_t row = (size_t)(row0 + lg) * a.T;
      const int tt = t_lo + lt * kWtRows;
      if (wave == 0) {
        // past the end, or no visible weight: p = exp2(. - inf) = 0
        const float x = tt + lane < t_hi ? a.lse[row + tt + lane] : -INFINITY;
        lse = x == -INFINITY ? INFINITY : x * kLog2e;
      }
      Tile::template load<4>(Qs, reinterpret_cast<const bf16*>(a.q) + row * D, tt, t_hi, wave);
      if (++lt == nt) {
        lt = 0;
        ++lg;
      }
    };
    auto step = [&](const unsigned char* Qs, const float* Ls, int tile0) {
#pragma unroll
      for (int u = 0; u < kWtRows / 32; ++u) {
        const int tt = tile0 + 32 * u;
        if (!(sw > tt + 31 || (sw >= a.sinks && tt - (sw + 31) >= a.window))) {
          f32x16 S = zero16();
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) mma32(S, Tile::row_frag(Qs, rb, 32 * u, kk), K[kk]);
          const bool full = sw + 31 <= tt && (tt + 31 - sw < a.window || sw + 32 <= a.sinks);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f32x4 ls = *reinterpret_cast<const f32x4*>(Ls + 32 * u + 8 * q + 4 * half);
#pragma unroll
            for (int e = 0; e < 4; ++e) S[4 * q + e] = S[4 * q + e] * c - ls[e];
          }
          // masked after the lse is taken off: one that is not a number stays with the keys that are seen
          if (!full) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int t = tt + acc_row(r, half);
              const bool see = (s <= t) & ((t - s < a.window) | (s < a.sinks));
              S[r] = see ? S[r] : -INFINITY;
            }
          }
#pragma unroll
          for (int r = 0; r < 16; ++r) sum += __builtin_amdgcn_exp2f(S[r]);
        }
      }
    };
    load(Q0);
    if (wave == 0) L0[lane] = lse;
    int ct = 0;                            // tile of the next step
    for (int i = 0; i < total; i += 2) {
      loads_and_barrier();
      load(Q1);
      step(Q0, L0, t_lo + ct * kWtRows);
      if (wave == 0) L1[lane] = lse;
      ct = ct + 1 == nt ? 0 : ct + 1;
      loads_and_barrier();
      load(Q0);
      if (i + 1 < total) step(Q1, L1, t_lo + ct * kWtRows);
      if (wave == 0) L0[lane] = lse;
      ct = ct + 1 == nt ? 0 : ct + 1;
    }
  }
  weight_store(a, un, s, sum);
}

// ------------------------------------------------------------------ fp32
constexpr int kWtQ = 32;

template <int D>
__global__ __launch_bounds__(256) void weight_f32_kernel(WeightArgs a) {
  using T = float;
  using St = RowStage<T, kWtQ, D, 256>;
  constexpr int LD = St::LD;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Qs = reinterpret_cast<T*>(smem);
  float* Ls = reinterpret_cast<float*>(Qs + kWtQ * LD);
  const WeightUnit un = weight_unit(a);
  const int G = a.Hq / a.Hkv, n = un.n, t_lo = un.t_lo, t_hi = un.t_hi, b = un.b, bk = un.bk;
  const int lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int sw = un.s0 + 32 * wave, s = sw + (lane & 31);
  float sum = 0.f;
  if (t_lo < t_hi && un.h_lo < un.h_hi) {
    Frag<T> K[D / 16];
    const size_t at = ((size_t)bk * a.T + min(s, n - 1)) * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) K[kk] = load_frag(reinterpret_cast<const T*>(a.k) + at + 16 * kk);
    const float c = a.scale * kLog2e;
    const int nt = (t_hi - t_lo + kWtQ - 1) / kWtQ, total = nt * (un.h_hi - un.h_lo);
    St qst;
    float lst = 0.f;
    auto load = [&](int i) {
      const int hq = (bk % a.Hkv) * G + un.h_lo + i / nt, tt = t_lo + (i % nt) * kWtQ;
      const size_t row = (size_t)(b * a.Hq + hq) * a.T;
      qst.load(reinterpret_cast<const T*>(a.q) + row * D, tt, t_hi);
      if (threadIdx.x < kWtQ) {
        const int t = tt + threadIdx.x;
        const float lse = t < t_hi ? a.lse[row + t] : -INFINITY;
        lst = lse == -INFINITY ? INFINITY : lse * kLog2e;
      }
    };
    load(0);
    for (int i = 0; i < total; ++i) {
      const int tt = t_lo + (i % nt) * kWtQ;
      __syncthreads();
      qst.store(Qs);
      if (threadIdx.x < kWtQ) Ls[threadIdx.x] = lst;
      __syncthreads();
      if (i + 1 < total) load(i + 1);
      if (sw > tt + 31 || (sw >= a.sinks && tt - (sw + 31) >= a.window)) continue;
      f32x16 S = zero16();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) mma32(S, frag_rows32(Qs, LD, 0, 16 * kk), K[kk]);
      const bool full = sw + 31 <= tt && (tt + 31 - sw < a.window || sw + 32 <= a.sinks);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 ls = *reinterpret_cast<const f32x4*>(Ls + 8 * q + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float p = __builtin_amdgcn_exp2f(S[4 * q + e] * c - ls[e]);
          if (!full) {
            const int t = tt + acc_row(4 * q + e, half);
            if (!(s <= t && (t - s < a.window || s < a.sinks))) p = 0.f;
          }
          sum += p;
        }
      }
    }
  }
  weight_store(a, un, s, sum);
}

__global__ __launch_bounds__(256) void weight_sum_kernel(WeightArgs a) {
  const size_t N = (size_t)a.B * a.Hkv * a.T;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= N) return;
  const int parts = a.n_chunk * a.n_head;
  constexpr int U = 8;                           // loads in flight together, added in order
  float x = 0.f;
  for (int c0 = 0; c0 < parts; c0 += U) {
    float y[U];
#pragma unroll
    for (int u = 0; u < U; ++u) y[u] = a.part[min(c0 + u, parts - 1) * N + i];
#pragma unroll
    for (int u = 0; u < U; ++u) x += c0 + u < parts ? y[u] : 0.f;
  }
  a.out[i] = x;
}

template <typename T, int D>
static hipError_t launch(const WeightArgs& a, hipStream_t st) {
  const dim3 grid(a.B * a.Hkv * ((a.T + kWtK - 1) / kWtK) * a.n_chunk * a.n_head);
  hipError_t e;
  if constexpr (sizeof(T) == 2) {
    e = launch_kernel<0>(weight_bf16_kernel<D>, grid, 256, a, st);
  } else {
    constexpr size_t lds = sizeof(T) * kWtQ * RowStage<T, kWtQ, D, 256>::LD + sizeof(float) * kWtQ;
    e = launch_kernel<lds>(weight_f32_kernel<D>, grid, 256, a, st);
  }
  if (e != hipSuccess || a.n_chunk * a.n_head == 1) return e;
  const size_t N = (size_t)a.B * a.Hkv * a.T;
  return launch_kernel<0>(weight_sum_kernel, dim3((unsigned)((N + 255) / 256)), 256, a, st);
}

hipError_t launch_weights(const WeightArgs& a, hipStream_t st) {
  if (a.dtype) return a.D == 128 ? launch<bf16, 128>(a, st) : launch<bf16, 64>(a, st);
  return a.D == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
}

}  // namespace carve
