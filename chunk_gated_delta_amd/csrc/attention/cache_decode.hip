// One new token per sequence against a cache of C slots: the ring cache of windowed attention,
// and the cache whose slots are given up by accumulated attention weight.
//
// Workgroup = a range of slots of one key head, for all query heads that share it (16 a tile on
// the columns of v_mfma_f32_16x16x32): every cached row is read once.  S^T = K Q^T and
// O^T = V^T P^T per 32 slots of a wave, running maximum and sum per head; the four waves
// and then the ranges are joined by rescaling.  The new token's k, v are taken from the call
// and written by the workgroup whose range holds their slot, so no other workgroup reads it.
#include <algorithm>

#include "attn_device.h"

namespace carve {

constexpr int kDecThreads = 256;

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
  for (int j = threadIdx.x; j < a.C; j += 64 * NW) {
    const int h = held[j];
    const int cls = h == p ? 0 : h < 0 ? 1 : (h >= a.sinks && h <= p - a.recent) ? 2 : 3;
    const unsigned o = cls < 2 ? 0u : weight_order(w[j]);
    const unsigned long long key = ((unsigned long long)cls << 62) | ((unsigned long long)o << 30) | (unsigned)j;
    best = key < best ? key : best;
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

// Adds the token's weights to the cache's: slots lo .. hi - 1, with max and sum of every head
// (log2 domain) in st[head] = {m, 1 / l}, scores [G][score_row(C)] of the key head in `score`.
template <int NW>
__device__ __forceinline__ void add_weights(const CacheArgs& a, int bk, int p, int at, int lo, int hi, const float* st,
                                            const float* score) {
  const int G = a.Hq / a.Hkv;
  const size_t row = (size_t)bk * a.C;
  constexpr int STEP = 64 * NW, U = 4;           // slots a thread takes at a time, their loads in flight together
  for (int j0 = lo + threadIdx.x; j0 < hi; j0 += U * STEP) {
    float x[U], w[U];
    int held[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(j0 + u * STEP, hi - 1);
      held[u] = a.cache_pos[row + j];
      w[u] = a.cache_w[row + j];
      x[u] = 0.f;
    }
    for (int g = 0; g < G; ++g) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        x[u] += __builtin_amdgcn_exp2f(score[(size_t)g * score_row(a.C) + min(j0 + u * STEP, hi - 1)] - st[2 * g]) *
                st[2 * g + 1];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = j0 + u * STEP;
      if (j < hi && (j == at || held[u] >= 0)) a.cache_w[row + j] = j == at ? x[u] : w[u] + x[u];
      if (j < hi && j == at) a.cache_pos[row + j] = p;
    }
  }
}

// ------------------------------------------------------------------ fp32
// 32 slots of a wave at a time through registers, the v rows on into LDS of the wave's own.
template <int D, int NT, bool BUDGET>
__global__ __launch_bounds__(kDecThreads) void cache_decode_f32_kernel(CacheArgs a) {
  using T = float;
  constexpr int LD = D + Pad<T>::v, PR = D / 8, NV = 32 * PR / 64, LDM = D + 4;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ unsigned long long red[kDecThreads / 64];
  __shared__ float ml[4][16][2];
  __shared__ float st[16 * NT][2];
  const int G = a.Hq / a.Hkv;
  const int split = blockIdx.x % a.n_split, bk = blockIdx.x / a.n_split, b = bk / a.Hkv;
  const int lane = lane_id(), wave = wave_id(), lr = lane & 15, lg = lane >> 4;
  const int p = a.pos[b];
  T* ob = reinterpret_cast<T*>(a.o) + (size_t)bk * G * D;
  if (p < 0) {                                   // no token: the cache stays as it is
    if (split == 0) {
      for (int i = threadIdx.x; i < G * D; i += kDecThreads) ob[i] = to<T>(0.f);
      if (BUDGET && threadIdx.x == 0) a.slot[bk] = -1;
    }
    return;
  }
  const int at = BUDGET ? pick_slot<4>(a, bk, p, red) : ring_slot(a, p);
  if (BUDGET && split == 0 && threadIdx.x == 0) a.slot[bk] = at;
  const int count = BUDGET ? a.C : min(p, a.C - 1) + 1;          // a ring holds its tokens from slot 0 up
  const int lo = split * a.split_len, hi = min(min(lo + a.split_len, a.C), count);
  T* ck = reinterpret_cast<T*>(a.cache_k) + (size_t)bk * a.C * D;
  T* cv = reinterpret_cast<T*>(a.cache_v) + (size_t)bk * a.C * D;
  const T* kn = reinterpret_cast<const T*>(a.k) + (size_t)bk * D;
  const T* vn = reinterpret_cast<const T*>(a.v) + (size_t)bk * D;
  const int* held = BUDGET ? a.cache_pos + (size_t)bk * a.C : nullptr;

  Frag<T> Q[NT][D / 32];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int g = min(16 * nt + lr, G - 1);
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk)
      Q[nt][kk] = load_frag(reinterpret_cast<const T*>(a.q) + ((size_t)bk * G + g) * D + 32 * kk + 8 * lg);
  }
  const float c = a.scale * kLog2e;
  f32x4 O[NT][D / 16];
  float m[NT], l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = kNegBig;
    l[nt] = 0.f;
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) O[nt][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  T* Vs = reinterpret_cast<T*>(smem) + wave * 32 * LD;
  for (int j0 = lo + 32 * wave; j0 < hi; j0 += 128) {
    // live slots of the 32, one bit each
    const int jl = j0 + (lane & 31);
    bool on = jl < hi;
    if (BUDGET) on = on && (jl == at || held[min(jl, a.C - 1)] >= 0);
    const unsigned live = (unsigned)__ballot(on);
    Frag<T> K[2][D / 32], V[NV];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = min(j0 + 16 * u + lr, hi - 1);
      const T* row = j == at ? kn : ck + (size_t)j * D;
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) K[u][kk] = load_frag(row + 32 * kk + 8 * lg);
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int pc = lane + 64 * u, r = pc / PR, j = min(j0 + r, hi - 1);
      const T* row = j == at ? vn : cv + (size_t)j * D;
      V[u] = load_frag(row + 8 * (pc % PR));
      if (!((live >> r) & 1)) V[u] = zero_frag(T());
    }
#pragma unroll
    for (int u = 0; u < NV; ++u) {
      const int pc = lane + 64 * u;
      *reinterpret_cast<Frag<T>*>(Vs + (pc / PR) * LD + 8 * (pc % PR)) = V[u];
    }
    __builtin_amdgcn_wave_barrier();             // the wave's own tile: written, then read across its lanes
    Frag<T> P[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      f32x4 S[2];
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        S[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) mma(S[u], K[u][kk], Q[nt][kk]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * u + 4 * lg + i;
          S[u][i] = ((live >> r) & 1) ? S[u][i] * c : -INFINITY;
          if (BUDGET && 16 * nt + lr < G && j0 + r < hi)
            a.score[((size_t)bk * G + 16 * nt + lr) * score_row(a.C) + j0 + r] = S[u][i];
          mx = fmaxf(mx, S[u][i]);
        }
      }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float mn = fmaxf(m[nt], mx), alpha = __builtin_amdgcn_exp2f(m[nt] - mn);
      m[nt] = mn;
      l[nt] *= alpha;
#pragma unroll
      for (int dt = 0; dt < D / 16; ++dt) O[nt][dt] *= alpha;
      float x[8];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[4 * u + i] = __builtin_amdgcn_exp2f(S[u][i] - mn);
          l[nt] += x[4 * u + i];
        }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        P[nt].lo[j] = x[j];
        P[nt].hi[j] = x[4 + j];
      }
    }
    // V^T operand, its contraction in the order of P: slots 4 lg + j, then 16 + 4 lg + j
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      Frag<T> F;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        F.lo[j] = Vs[(4 * lg + j) * LD + 16 * dt + lr];
        F.hi[j] = Vs[(16 + 4 * lg + j) * LD + 16 * dt + lr];
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma(O[nt][dt], F, P[nt]);
    }
    __builtin_amdgcn_wave_barrier();
  }
  // the new rows, by the workgroup that owns their slot
  if (at >= lo && at < hi && threadIdx.x < 2 * PR) {
    const int i = 8 * (threadIdx.x % PR);
    if (threadIdx.x < PR) *reinterpret_cast<Frag<T>*>(ck + (size_t)at * D + i) = load_frag(kn + i);
    else *reinterpret_cast<Frag<T>*>(cv + (size_t)at * D + i) = load_frag(vn + i);
  }
  // join the waves, 16 heads at a time
  float* mg = reinterpret_cast<float*>(smem);                      // [4][16][LDM]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (16 * nt >= G) break;
    float lt = l[nt] + __shfl_xor(l[nt], 16);
    lt += __shfl_xor(lt, 32);
    __syncthreads();
    if (lg == 0) {
      ml[wave][lr][0] = m[nt];
      ml[wave][lr][1] = lt;
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) store4(mg + (wave * 16 + lr) * LDM + 16 * dt + 4 * lg, O[nt][dt]);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * D / 4; i += kDecThreads) {
      const int h = i / (D / 4), d = 4 * (i % (D / 4)), g = 16 * nt + h;
      if (g >= G) continue;
      float M = kNegBig, L = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, ml[w][h][0]);
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[w][h][0] - M);
        L += f * ml[w][h][1];
        x += load4f(mg + (w * 16 + h) * LDM + d) * f;
      }
      if (a.n_split == 1) {
        const float f = L != 0.f ? 1.f / L : 0.f;
        store4(ob + (size_t)g * D + d, x * f);
        if (d == 0) {
          st[g][0] = M;
          st[g][1] = f;
        }
      } else {
        float* dst = a.part + (((size_t)bk * a.n_split + split) * G + g) * (D + 4);
        store4(dst + 4 + d, x);
        if (d == 0) {
          dst[0] = M;
          dst[1] = L;
        }
      }
    }
  }
  if (BUDGET && a.n_split == 1) {
    __syncthreads();                             // scores of all waves, and st
    add_weights<4>(a, bk, p, at, 0, a.C, &st[0][0], a.score + (size_t)bk * G * score_row(a.C));
  }
}

// ------------------------------------------------------------------ bf16
// A wave's 32 slots at a time, brought to LDS by buffer loads that write it directly: the k rows of the
// next slots are on their way while these are worked on, and so are its v rows, each wave in
// buffers of its own and without barriers.  Rows of slots that are not live lie past the
// buffer's end and read as zero.  Layout: blocks of 32 columns, [32][64 bytes], piece c of a row at
// c ^ f(row), f = row bits 2 and 3 swapped, which spreads 16 rows at one piece and 8 rows at 2 pieces
// over the banks (counted in all: 0.28 conflicts an active LDS cycle, with LDS active for 0.06 of
// the time).  Bound by the cache's read: 256 sequences, 16 heads on 4, window 4,096, D = 128 in
// 342 us, 6.2 TB/s (rows through registers, two launches more often: 405 us); 64 sequences at 2,048
// slots with weights 60 us, 4.6 TB/s (one workgroup a compute unit: the slot's search at its start
// and the weights at its end overlap no reads); one sequence at window 1,024 9 us, latency.
template <int D>
struct WaveRows {
  static constexpr int RB = 2 * D, BLOCK = 2048, bytes = 32 * RB, kLoads = bytes / 1024;   // instructions of a load
  static __device__ __forceinline__ int swz(int r) { return ((r >> 1) & 2) | ((r >> 3) & 1); }
  // rows j0 .. j0 + 31 of base, those whose bit of `live` is set (one descriptor: 32 rows)
  static __device__ __forceinline__ void load(unsigned char* dst, const bf16* base, int j0, unsigned live) {
    const int lane = lane_id(), rl = lane >> 2;
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16*>(base) + (size_t)j0 * D, 0, bytes, 0x00020000);
    const int voff = rl * RB + (((lane & 3) ^ swz(rl)) << 4);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int v = (live >> (16 * h + rl)) & 1 ? voff : bytes;      // (past the end)
#pragma unroll
      for (int blk = 0; blk < D / 32; ++blk)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(dst + blk * BLOCK + 1024 * h), 16, v,
                                                 blk * 64 + 16 * h * RB, 0, 0);
    }
  }
  // rows 16 u .. + 15 as A operand, 32-deep block kk
  static __device__ __forceinline__ Frag<bf16> row_frag(const unsigned char* src, int u, int kk) {
    const int lane = lane_id(), r = lane & 15;
    Frag<bf16> f;
    f.v = *(lds_bf16x8*)(src + kk * BLOCK + 1024 * u + r * 64 + (((lane >> 4) ^ swz(r)) << 4));
    return f;
  }
  // columns 16 dt .. + 15 as rows of an A operand, contraction over rows 4 g + j, then 16 + 4 g + j
  static __device__ __forceinline__ Frag<bf16> col_frag(const unsigned char* src, int dt) {
    const int lane = lane_id(), s = lane & 15, r = 4 * (lane >> 4) + (s >> 2);
    const unsigned char* p = src + (dt >> 1) * BLOCK + r * 64 +
                             (((2 * (dt & 1) + ((s & 3) >> 1)) ^ swz(r)) << 4) + 8 * (s & 1);
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 1024));
    Frag<bf16> f;
    f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    return f;
  }
};

// NEAR: this step's scores of a cache kept by weight stay in LDS (the caller's rule: where that keeps no
// second workgroup off the compute unit).
template <int D, int NT, int NW, bool BUDGET, bool NEAR>
__global__ __launch_bounds__(64 * NW, NT == 1 ? 2 : 1) void cache_decode_bf16_kernel(CacheArgs a) {
  using Rows = WaveRows<D>;
  constexpr int STEP = 32 * NW;
  __shared__ __align__(16) unsigned char Ks[NW * Rows::bytes], Vs[NW * Rows::bytes];
  __shared__ unsigned long long red[NW];
  __shared__ float ml[NW][16][2];
  __shared__ float st[16 * NT][2];
  __shared__ __align__(16) float near_score[NEAR ? kNearScores : 4];
  const int G = a.Hq / a.Hkv;
  const int split = uniform(blockIdx.x % a.n_split), bk = uniform(blockIdx.x / a.n_split), b = uniform(bk / a.Hkv);
  const int lane = lane_id(), wave = wave_uid(), lr = lane & 15, lg = lane >> 4;
  const int p = uniform(a.pos[b]);
  bf16* ob = reinterpret_cast<bf16*>(a.o) + (size_t)bk * G * D;
  if (p < 0) {                                   // no token: the cache stays as it is
    if (split == 0) {
      for (int i = threadIdx.x; i < G * D; i += 64 * NW) ob[i] = (bf16)0.f;
      if (BUDGET && threadIdx.x == 0) a.slot[bk] = -1;
    }
    return;
  }
  const int count = BUDGET ? a.C : min(p, a.C - 1) + 1;          // a ring holds its tokens from slot 0 up
  const int lo = split * a.split_len, hi = min(min(lo + a.split_len, a.C), count);
  bf16* ck = reinterpret_cast<bf16*>(a.cache_k) + (size_t)bk * a.C * D;
  bf16* cv = reinterpret_cast<bf16*>(a.cache_v) + (size_t)bk * a.C * D;
  const int* held = BUDGET ? a.cache_pos + (size_t)bk * a.C : nullptr;
  unsigned char* kw = Ks + wave * Rows::bytes;
  unsigned char* vw = Vs + wave * Rows::bytes;
  const int first = lo + 32 * wave;
  // live slots of the 32 from j0, one bit each (`at`: the new token's, live whatever it held)
  auto live_of = [&](int j0, int at) -> unsigned {
    const int j = j0 + (lane & 31);
    bool on = j < hi;
    if (BUDGET) on = on && (j == at || held[min(j, a.C - 1)] >= 0);
    return (unsigned)__ballot(on);
  };
  unsigned live = 0;
  auto fetch_first = [&](int at) {
    live = live_of(first, at);
    Rows::load(kw, ck, first, live);
    Rows::load(vw, cv, first, live);
  };
  if (BUDGET && first < hi) fetch_first(-1);     // on their way while the slot is looked for
  const int at = uniform(BUDGET ? pick_slot<NW>(a, bk, p, red) : ring_slot(a, p));
  if (BUDGET && split == 0 && threadIdx.x == 0) a.slot[bk] = at;
  // the new rows go to the cache first, by the workgroup that owns their slot and alone reads it
  if (at >= lo && at < hi) {
    if (threadIdx.x < D / 4) {
      const int i = 8 * (threadIdx.x % (D / 8));
      const bool is_v = threadIdx.x >= D / 8;
      const bf16* src = reinterpret_cast<const bf16*>(is_v ? a.v : a.k) + (size_t)bk * D + i;
      *reinterpret_cast<bf16x8*>((is_v ? cv : ck) + (size_t)at * D + i) = *reinterpret_cast<const bf16x8*>(src);
    }
    __syncthreads();
  }
  if (first < hi && (!BUDGET || (at >= first && at < first + 32))) fetch_first(at);
  Frag<bf16> Q[NT][D / 32];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int g = min(16 * nt + lr, G - 1);
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk)
      Q[nt][kk] = load_frag(reinterpret_cast<const bf16*>(a.q) + ((size_t)bk * G + g) * D + 32 * kk + 8 * lg);
  }
  const float c = a.scale * kLog2e;
  f32x4 O[NT][D / 16];
  float m[NT], l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = kNegBig;
    l[nt] = 0.f;
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) O[nt][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // the positions of the slots after next, asked for a step early: waiting for them at their use
  // would also wait for the rows that were asked for before them
  auto position = [&](int j0) { return BUDGET ? held[min(j0 + (lane & 31), a.C - 1)] : 0; };
  int ahead = position(first + STEP);
  for (int j0 = first; j0 < hi; j0 += STEP) {
    const int jn = j0 + STEP + (lane & 31);
    const unsigned next = (unsigned)__ballot(jn < hi && (!BUDGET || jn == at || ahead >= 0));
    ahead = position(j0 + 2 * STEP);
    wait_loads<Rows::kLoads>();                  // this k has arrived (its v, issued after it, may not have)
    f32x4 X[NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Frag<bf16> K[D / 32];
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) K[kk] = Rows::row_frag(kw, u, kk);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        X[nt][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk) mma(X[nt][u], K[kk], Q[nt][kk]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    Rows::load(kw, ck, j0 + STEP, next);         // (behind the last slots: no rows)
    Frag<bf16> P[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 16 * u + 4 * lg + i;
          const float x = ((live >> r) & 1) ? X[nt][u][i] * c : -INFINITY;
          X[nt][u][i] = x;
          mx = fmaxf(mx, x);
        }
      // four slots of a head at a time (past the last slot into the row's padding)
      if (BUDGET && 16 * nt + lr < G) {
        const size_t row = (size_t)(16 * nt + lr) * score_row(a.C) + j0 + 4 * lg;
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (j0 + 16 * u + 4 * lg < hi) {
            if (NEAR) store4(near_score + row + 16 * u, X[nt][u]);
            else store4(a.score + (size_t)bk * G * score_row(a.C) + row + 16 * u, X[nt][u]);
          }
      }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      if (__any(mx > m[nt] + 8.f)) {             // rescale only when a maximum grows by 2^8
        const float mn = fmaxf(m[nt], mx), alpha = __builtin_amdgcn_exp2f(m[nt] - mn);
        m[nt] = mn;
        l[nt] *= alpha;
#pragma unroll
        for (int dt = 0; dt < D / 16; ++dt) O[nt][dt] *= alpha;
      }
      // the weights are rounded to bf16 for the product with v (the sum l is not)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = __builtin_amdgcn_exp2f(X[nt][u][i] - m[nt]);
          l[nt] += x;
          P[nt].v[4 * u + i] = (bf16)x;
        }
    }
    wait_loads<Rows::kLoads>();                  // this v has arrived (the next k, issued after it, may not have)
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      const Frag<bf16> F = Rows::col_frag(vw, dt);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma(O[nt][dt], F, P[nt]);
    }
    __builtin_amdgcn_sched_barrier(0);
    Rows::load(vw, cv, j0 + STEP, next);
    live = next;
  }
  wait_loads<0>();                               // nothing writes LDS any more
  // join the waves, 16 heads at a time (4-float pieces of a row swizzled by the head)
  float* mg = reinterpret_cast<float*>(Ks);                        // [NW][16][D]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if (16 * nt >= G) break;
    float lt = l[nt] + __shfl_xor(l[nt], 16);
    lt += __shfl_xor(lt, 32);
    __syncthreads();
    if (lg == 0) {
      ml[wave][lr][0] = m[nt];
      ml[wave][lr][1] = lt;
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt)
      store4(mg + (wave * 16 + lr) * D + (((4 * dt + lg) ^ lr) << 2), O[nt][dt]);
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * D / 4; i += 64 * NW) {
      const int h = i / (D / 4), c4 = i % (D / 4), g = 16 * nt + h;
      if (g >= G) continue;
      float M = kNegBig, L = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[w][h][0]);
      f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[w][h][0] - M);
        L += f * ml[w][h][1];
        x += load4f(mg + (w * 16 + h) * D + ((c4 ^ h) << 2)) * f;
      }
      if (a.n_split == 1) {
        const float f = L != 0.f ? 1.f / L : 0.f;
        store4(ob + (size_t)g * D + 4 * c4, x * f);
        if (c4 == 0) {
          st[g][0] = M;
          st[g][1] = f;
        }
      } else {
        float* dst = a.part + (((size_t)bk * a.n_split + split) * G + g) * (D + 4);
        store4(dst + 4 + 4 * c4, x);
        if (c4 == 0) {
          dst[0] = M;
          dst[1] = L;
        }
      }
    }
  }
  if (BUDGET && a.n_split == 1) {
    __syncthreads();                             // scores of all waves, and st
    if (NEAR) add_weights<NW>(a, bk, p, at, 0, a.C, &st[0][0], near_score);
    else add_weights<NW>(a, bk, p, at, 0, a.C, &st[0][0], a.score + (size_t)bk * G * score_row(a.C));
  }
}

// Joins the ranges of one key head: the output (a workgroup per head of the group, its ranges'
// partial sums read at once), and for a cache kept by weight the weights, a range of slots a workgroup.
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
    const float m = lane < a.n_split ? q[0] : kNegBig;
    float M = m;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) M = fmaxf(M, __shfl_xor(M, o));
    const float x = __builtin_amdgcn_exp2f(m - M);
    float L = lane < a.n_split ? x * q[1] : 0.f;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) L += __shfl_xor(L, o);
    if (lane == 0) {
      st[g][0] = M;
      st[g][1] = L != 0.f ? 1.f / L : 0.f;
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

template <typename T, int D, int NT, bool BUDGET>
static hipError_t launch_nt(const CacheArgs& a, hipStream_t st) {
  const int units = a.B * a.Hkv, G = a.Hq / a.Hkv;
  hipError_t e;
  if constexpr (sizeof(T) == 2) {
    const dim3 grid(units * a.n_split);
    if (NT == 1 && a.waves == 8 && BUDGET && !a.score)
      e = launch_kernel<0>(cache_decode_bf16_kernel<D, 1, 8, BUDGET, BUDGET>, grid, 512, a, st);
    else if (NT == 1 && a.waves == 8)
      e = launch_kernel<0>(cache_decode_bf16_kernel<D, 1, 8, BUDGET, false>, grid, 512, a, st);
    else
      e = launch_kernel<0>(cache_decode_bf16_kernel<D, NT, 4, BUDGET, false>, grid, kDecThreads, a, st);
  } else {
    constexpr size_t lds = std::max(sizeof(T) * 4 * 32 * (D + Pad<T>::v), sizeof(float) * 4 * 16 * (D + 4));
    e = launch_kernel<lds>(cache_decode_f32_kernel<D, NT, BUDGET>, dim3(units * a.n_split), kDecThreads, a, st);
  }
  if (e != hipSuccess || a.n_split == 1) return e;
  return launch_kernel<0>(cache_join_kernel<T, D, BUDGET>, dim3(units * (BUDGET ? G + a.n_split : G)), kDecThreads, a, st);
}
template <typename T, int D, bool BUDGET>
static hipError_t launch_g(const CacheArgs& a, hipStream_t st) {
  const int G = a.Hq / a.Hkv;
  if (G <= 16) return launch_nt<T, D, 1, BUDGET>(a, st);
  if (G <= 32) return launch_nt<T, D, 2, BUDGET>(a, st);
  return launch_nt<T, D, 4, BUDGET>(a, st);
}
template <typename T, int D>
static hipError_t launch(const CacheArgs& a, hipStream_t st) {
  return a.cache_w ? launch_g<T, D, true>(a, st) : launch_g<T, D, false>(a, st);
}
hipError_t launch_cache_decode(const CacheArgs& a, hipStream_t st) {
  if (a.dtype) return a.D == 128 ? launch<bf16, 128>(a, st) : launch<bf16, 64>(a, st);
  return a.D == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
}

}  // namespace carve
