// Pieces of a decode step that caches of rows as they are and of rows in codes share: the new token's
// slot, the weights it adds, and the join of several workgroups' slot ranges.
#pragma once
#include "attn_device.h"

namespace carve {

constexpr int kDecThreads = 256;
// Running maximum before the first live slot, at or below every finite score.  Ranges and waves without one have it as theirs:
// the factor that joins them in is then 0, or 1 of a sum of 0.
constexpr float kLeast = -__FLT_MAX__;

// Slot of the new token in a cache kept by weight, by the least (class, weight, slot):
// class 0 the slot that holds this position already (a repeated call), 1 an empty one, 2 one
// that is neither first nor recent, 3 any other.  NaN counts as the largest weight.
__device__ __forceinline__ unsigned weight_order(float w) {
  const unsigned u = __builtin_bit_cast(unsigned, w + 0.f);
  return w != w ? 0xffffffffu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
template <int NW>
__device__ __forceinline__ int pick_slot(const CacheArgs& a, int bk, int p, unsigned long long* red) {
  const float* w = a.cache_w + (size_t)bk * a.C;
  const int* held = a.cache_pos + (size_t)bk * a.C;
  unsigned long long best = ~0ull;
  constexpr int U = 4;                           // slots a thread takes at a time, their loads in flight together
  for (int j0 = threadIdx.x; j0 < a.C; j0 += U * 64 * NW) {
    int h[U];
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u * 64 * NW, a.C - 1);        // (the last slot again, behind it)
      h[u] = held[j];
      x[u] = w[j];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u * 64 * NW, a.C - 1);
      const int cls = h[u] == p ? 0 : h[u] < 0 ? 1 : (h[u] >= a.sinks && h[u] <= p - a.recent) ? 2 : 3;
      const unsigned o = cls < 2 ? 0u : weight_order(x[u]);
      const unsigned long long key = ((unsigned long long)cls << 62) | ((unsigned long long)o << 30) | (unsigned)j;
      best = key < best ? key : best;
    }
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const unsigned long long x = __shfl_xor(best, o);
    best = x < best ? x : best;
  }
  if (lane_id() == 0) red[wave_id()] = best;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NW; ++i) best = red[i] < best ? red[i] : best;
  return (int)(best & ((1u << 30) - 1));
}

__device__ __forceinline__ int ring_slot(const CacheArgs& a, int p) {
  return p < a.sinks ? p : a.sinks + (p - a.sinks) % a.window;
}

// Slots a thread takes at a time, their positions and weights in flight together; a kernel may ask for the
// first of them (from `lo` on) early.
template <int NW>
struct WeightBatch {
  static constexpr int STEP = 64 * NW, U = 4;
  int held[U];
  float w[U];
  __device__ __forceinline__ void load(const CacheArgs& a, int bk, int j0, int hi) {
    const size_t row = (size_t)bk * a.C;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u * STEP, hi - 1);
      held[u] = a.cache_pos[row + j];
      w[u] = a.cache_w[row + j];
    }
  }
};
// Adds the token's weights to the cache's: slots lo .. hi - 1, with max and sum of every head
// (log2 domain) in st[head] = {m, 1 / l}, scores [G][score_row(C)] of the key head in `score`; b: the first batch.
template <int NW>
__device__ __forceinline__ void add_weights(const CacheArgs& a, int bk, int p, int at, int lo, int hi, const float* st,
                                            const float* score, WeightBatch<NW> b) {
  const int G = a.Hq / a.Hkv;
  const size_t row = (size_t)bk * a.C;
  constexpr int STEP = WeightBatch<NW>::STEP, U = WeightBatch<NW>::U;
  for (int j0 = lo + threadIdx.x; j0 < hi; j0 += U * STEP) {
    float x[U] = {};
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] += __builtin_amdgcn_exp2f(score[(size_t)g * score_row(a.C) + min(j0 + u * STEP, hi - 1)] - st[2 * g]) *
                st[2 * g + 1];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * STEP;
      if (j < hi && (j == at || b.held[u] >= 0)) a.cache_w[row + j] = j == at ? x[u] : b.w[u] + x[u];
      if (j < hi && j == at) a.cache_pos[row + j] = p;
    }
    if (j0 + U * STEP < hi) b.load(a, bk, j0 + U * STEP, hi);
  }
}
template <int NW>
__device__ __forceinline__ void add_weights(const CacheArgs& a, int bk, int p, int at, int lo, int hi, const float* st,
                                            const float* score) {
  WeightBatch<NW> b;
  b.load(a, bk, lo + threadIdx.x, hi);
  add_weights<NW>(a, bk, p, at, lo, hi, st, score, b);
}

// Joins the ranges of one key head: the output (a workgroup per head of the group, its ranges'
// partial sums read at once), and for a cache kept by weight the weights, a range of slots a workgroup.
// The token sees itself, so a head's sum is 1 or more unless all its scores are -inf, as an infinite query
// makes them: then it is zero, and its output and weights 0 / 0, not a number.
constexpr int kMaxSplit = 64;
template <typename T, int D, bool BUDGET>
__global__ __launch_bounds__(kDecThreads) void cache_join_kernel(CacheArgs a) {
  __shared__ float st[64][2];
  __shared__ float f[kMaxSplit];
  const int G = a.Hq / a.Hkv, per = BUDGET ? G + a.n_split : G;
  const int w = blockIdx.x % per, bk = blockIdx.x / per, p = a.pos[bk / a.Hkv];
  if (p < 0) return;
  const float* part = a.part + (size_t)bk * a.n_split * G * (D + 4);
  auto stats = [&](int g) {                      // lanes of a wave: max and sum of head g over the ranges
    const int lane = lane_id();
    const float* q = part + ((size_t)min(lane, a.n_split - 1) * G + g) * (D + 4);
    const float m = lane < a.n_split ? q[0] : kLeast;
    float M = m;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) M = fmaxf(M, __shfl_xor(M, o));
    const float x = __builtin_amdgcn_exp2f(m - M);
    float L = lane < a.n_split ? x * q[1] : 0.f;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) L += __shfl_xor(L, o);
    if (lane == 0) {
      st[g][0] = M;
      st[g][1] = 1.f / L;
    }
    return x;
  };
  if (w < G) {
    if (threadIdx.x < 64) f[threadIdx.x] = stats(w);
    __syncthreads();
    const int d = threadIdx.x;
    if (d < D) {
      float x = 0.f;
      const float* q = part + (size_t)w * (D + 4) + 4 + d;
#pragma unroll 8
      for (int s = 0; s < a.n_split; ++s) x += q[(size_t)s * G * (D + 4)] * f[s];
      reinterpret_cast<T*>(a.o)[((size_t)bk * G + w) * D + d] = to<T>(x * st[w][1]);
    }
  } else if constexpr (BUDGET) {
    for (int g = wave_uid(); g < G; g += kDecThreads / 64) (void)stats(g);
    __syncthreads();
    const int lo = (w - G) * a.split_len, hi = min(lo + a.split_len, a.C);
    add_weights<4>(a, bk, p, a.slot[bk], lo, hi, &st[0][0], a.score + (size_t)bk * G * score_row(a.C));
  }
}

}  // namespace carve
