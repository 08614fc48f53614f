// One new token per sequence against a cache held in codes of 4 or 8 bits (mx_device.h): the ring cache
// and the cache kept by attention weight, with the split, the softmax and the joins of cache_decode.hip.
//
// What codes stand for is a bf16 exactly, so both products run on bf16 operands; where q is float32, q
// and the weights go in as three bf16 parts each, which hold all their bits.  Cached rows go from
// memory to registers without LDS: a lane's contraction elements of S^T = K Q^T may come in any order
// that q's have too, so it takes D / 4 neighbouring elements of its key, with one scale; for O^T = V^T P^T it
// takes D / 16 neighbouring elements of each of its eight slots and pairs the slots up as it converts.
// The token's own row goes into the registers of the wave that holds its slot as well as
// to the cache, so no wave waits for a store.
#include <algorithm>

#include "cache_step.h"
#include "mx_device.h"

namespace carve {

// x as N bf16 parts that add up to it (N = 1: rounded; 3: all bits of a float)
template <int N>
__device__ __forceinline__ void bf16_parts(const float (&x)[8], Frag<bf16> (&f)[N]) {
  if constexpr (N == 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[0].v[j] = (bf16)x[j];
  } else {
    u32 w[N][4];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float a = x[j], b = x[j + 1];
#pragma unroll
      for (int n = 0; n < N; ++n) {               // the upper half of a float is a bf16; the rest is exact
        const u32 ua = __builtin_bit_cast(u32, a), ub = __builtin_bit_cast(u32, b);
        w[n][j / 2] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        a -= __builtin_bit_cast(float, ua & 0xffff0000u);
        b -= __builtin_bit_cast(float, ub & 0xffff0000u);
      }
    }
#pragma unroll
    for (int n = 0; n < N; ++n) f[n].v = __builtin_bit_cast(bf16x8, u32x4{w[n][0], w[n][1], w[n][2], w[n][3]});
  }
}

// 32 slots of a wave as they come from memory.  Lane (lr, lg): elements lg D / 4 .. of the keys of slots lr
// and 16 + lr; elements lr D / 16 .. of the values of slots 16 u + 4 lg + i, i < 4; scales of all
// blocks of these slots.
template <int BITS, int D>
struct MxStep {
  static constexpr int RB = D * BITS / 8, SB = D / 32;         // bytes of a row, of its scales
  static constexpr int KW = RB / 16, VB = RB / 16, VW = VB < 4 ? 1 : VB / 4;   // words a lane and key; bytes, words a slot
  u32 k[2][KW], v[8][VW], ks[2], vs[2][SB];

  // n rows from slot j0 on (a read behind them gives zero)
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const void* base, size_t j0, int n, int row_bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((char*)base + j0 * row_bytes, 0, n * row_bytes, 0x00020000);
  }
  // (constant parts of an offset are the scalar operand: one address register for all slots)
  template <int N>
  static __device__ __forceinline__ void words(__amdgpu_buffer_rsrc_t r, int off, int more, u32* w) {
    if constexpr (N == 1) {
      w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, more, 0);
    } else if constexpr (N == 2) {
      const u32x2 x = __builtin_amdgcn_raw_buffer_load_b64(r, off, more, 0);
      w[0] = x[0];
      w[1] = x[1];
    } else {
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(r, off, more + 16 * h, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * h + i] = x[i];
      }
    }
  }
  __device__ __forceinline__ void load_k(const void* codes, const void* scales, size_t j0, int n) {
    const int lane = lane_id(), lr = lane & 15, lg = lane >> 4;
    const auto c = rows(codes, j0, n, RB), s = rows(scales, j0, n, SB);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      words<KW>(c, lr * RB + lg * KW * 4, 16 * u * RB, k[u]);
      ks[u] = (unsigned char)__builtin_amdgcn_raw_buffer_load_b8(s, lr * SB + lg * SB / 4, 16 * u * SB, 0);
    }
  }
  __device__ __forceinline__ void load_v(const void* codes, const void* scales, size_t j0, int n) {
    const int lane = lane_id(), lr = lane & 15, lg = lane >> 4;
    const auto c = rows(codes, j0, n, RB), s = rows(scales, j0, n, SB);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int more = 16 * (j >> 2) + (j & 3), off = 4 * lg * RB + lr * VB;
      if constexpr (VB == 2) v[j][0] = (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(c, off, more * RB, 0);
      else words<VW>(c, off, more * RB, v[j]);
    }
    if (n == 32) {                               // four slots at a time, where all four are there
#pragma unroll
      for (int u = 0; u < 2; ++u) words<SB>(s, 4 * lg * SB, 16 * u * SB, vs[u]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int u = j >> 2, i = j & 3, more = (16 * u + i) * SB;
        if constexpr (SB == 4) {
          vs[u][i] = __builtin_amdgcn_raw_buffer_load_b32(s, 4 * lg * SB, more, 0);
        } else {
          const u32 x = (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(s, 4 * lg * SB, more, 0);
          vs[u][i >> 1] = (i & 1) ? vs[u][i >> 1] | x << 16 : x;
        }
      }
    }
  }
  // scale of this lane's values of its slot j
  __device__ __forceinline__ u32 v_scale(int j) const {
    const int lr = lane_id() & 15, blk = lr * SB / 16;
    const int i = j & 3;
    if constexpr (SB == 4) return (vs[j >> 2][i] >> (8 * blk)) & 255u;
    else return (vs[j >> 2][i >> 1] >> (8 * (blk + 2 * (i & 1)))) & 255u;
  }
};

// the largest x of the four lanes l, l ^ 16, l ^ 32, l ^ 48
__device__ __forceinline__ float group_max(float x) {
  const u32 u = __builtin_bit_cast(u32, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float y = fmaxf(__builtin_bit_cast(float, (u32)r[0]), __builtin_bit_cast(float, (u32)r[1]));
  const u32 w = __builtin_bit_cast(u32, y);
  const auto s = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__builtin_bit_cast(float, (u32)s[0]), __builtin_bit_cast(float, (u32)s[1]));
}

template <typename T, int BITS, int D, int NT, int NW, bool BUDGET, bool NEAR>
__global__ __launch_bounds__(64 * NW, NT == 1 ? 2 : 1) void mx_decode_kernel(CacheArgs a) {
  using Step = MxStep<BITS, D>;
  constexpr int STEP = 32 * NW, N = sizeof(T) == 2 ? 1 : 3, KK = D / 32, DT = D / 16;
  constexpr int RB = Step::RB, SB = Step::SB;
  __shared__ __align__(16) float mg[NW * 16 * D];
  __shared__ unsigned long long red[NW];
  __shared__ float ml[NW][16][2];
  __shared__ float st[16 * NT][2];
  __shared__ __align__(16) u32 fresh[2][RB / 4];                 // the token's k and v
  __shared__ unsigned char fresh_scale[2][SB];
  __shared__ __align__(16) float near_score[NEAR ? kNearScores : 4];
  const int G = a.Hq / a.Hkv;
  const int split = uniform(blockIdx.x % a.n_split), bk = uniform(blockIdx.x / a.n_split), b = uniform(bk / a.Hkv);
  const int lane = lane_id(), wave = wave_uid(), lr = lane & 15, lg = lane >> 4;
  const int p = uniform(a.pos[b]);
  T* ob = reinterpret_cast<T*>(a.o) + (size_t)bk * G * D;
  if (p < 0) {                                   // no token: the cache stays as it is
    if (split == 0) {
      for (int i = threadIdx.x; i < G * D; i += 64 * NW) ob[i] = to<T>(0.f);
      if (BUDGET && threadIdx.x == 0) a.slot[bk] = -1;
    }
    return;
  }
  const int count = BUDGET ? a.C : min(p, a.C - 1) + 1;          // a ring holds its tokens from slot 0 up
  const int lo = split * a.split_len, hi = min(min(lo + a.split_len, a.C), count);
  char* ck = reinterpret_cast<char*>(a.cache_k) + (size_t)bk * a.C * RB;
  char* cv = reinterpret_cast<char*>(a.cache_v) + (size_t)bk * a.C * RB;
  unsigned char* sk = a.k_scales + (size_t)bk * a.C * SB;
  unsigned char* sv = a.v_scales + (size_t)bk * a.C * SB;
  const int* held = BUDGET ? a.cache_pos + (size_t)bk * a.C : nullptr;
  const int first = lo + 32 * wave;
  // slots of the 32 from j0 that hold a token, one bit each
  auto position = [&](int j0) { return BUDGET ? held[min(j0 + (lane & 31), a.C - 1)] : 0; };
  auto live_of = [&](int j0, int pos) {
    const int j = j0 + (lane & 31);
    return (unsigned)__ballot(j < hi && (!BUDGET || pos >= 0));
  };
  // (q before the rows: loads arrive in order, so what waits for rows has q)
  Frag<bf16> Q[NT][KK][N];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int g = min(16 * nt + lr, G - 1);
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      const Frag<T> f = load_frag(reinterpret_cast<const T*>(a.q) + ((size_t)bk * G + g) * D + lg * (D / 4) + 8 * kk);
      if constexpr (N == 1) {
        Q[nt][kk][0] = f;
      } else {
        float y[8];
        to_floats(f, y);
        bf16_parts<N>(y, Q[nt][kk]);
      }
    }
  }
  // rows of the 32 to read: up to the last that holds a token
  auto rows_of = [&](unsigned live) { return uniform(32 - __clz((int)live)); };
  Step x;
  unsigned live = 0;
  if (first < hi) {
    live = live_of(first, position(first));
    x.load_k(ck, sk, first, rows_of(live));
    x.load_v(cv, sv, first, rows_of(live));
  }
  const int at = uniform(BUDGET ? pick_slot<NW>(a, bk, p, red) : ring_slot(a, p));
  if (BUDGET && split == 0 && threadIdx.x == 0) a.slot[bk] = at;
  // the wave that holds the slot writes the token's rows
  if (at >= lo && at < hi && (at - lo) / 32 % NW == wave) {
    if (lane < D / 4) {
      const int piece = lane % (D / 8), is_v = lane / (D / 8);
      u32 scale;
      const Eight<BITS> c =
          write_block<BITS>(load_frag(reinterpret_cast<const T*>(is_v ? a.v : a.k) + (size_t)bk * D + 8 * piece), scale);
      reinterpret_cast<Eight<BITS>*>(fresh[is_v])[piece] = c;
      reinterpret_cast<Eight<BITS>*>((is_v ? cv : ck) + (size_t)at * RB)[piece] = c;
      if ((piece & 3) == 0) {
        fresh_scale[is_v][piece >> 2] = (unsigned char)scale;
        (is_v ? sv : sk)[(size_t)at * SB + (piece >> 2)] = (unsigned char)scale;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");       // written and read by this wave alone
    __builtin_amdgcn_wave_barrier();
  }
  const float c = a.scale * kLog2e;
  f32x4 O[NT][DT];
  float m[NT], l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = kNegBig;
    l[nt] = 0.f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) O[nt][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  int ahead = position(first + STEP);            // positions are asked for a step before the rows
  for (int j0 = first; j0 < hi; j0 += STEP) {
    const unsigned next = live_of(j0 + STEP, ahead);
    ahead = position(j0 + 2 * STEP);
    const int own = at - j0;                     // the token's slot, if of these
    if (own >= 0 && own < 32) {
      live |= 1u << own;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (own == 16 * u + lr) {
#pragma unroll
          for (int i = 0; i < Step::KW; ++i) x.k[u][i] = fresh[0][lg * Step::KW + i];
          x.ks[u] = fresh_scale[0][lg * SB / 4];
        }
    }
    f32x4 X[NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Frag<bf16> K[KK];
      const float s = scale_value(x.ks[u]);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        Eight<BITS> e;
        if constexpr (BITS == 4) e.w = x.k[u][kk];
        else e.w = u32x2{x.k[u][2 * kk], x.k[u][2 * kk + 1]};
        K[kk] = read_eight<BITS>(e, s);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        X[nt][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = N - 1; n >= 0; --n)         // the smallest parts first
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) mma(X[nt][u], K[kk], Q[nt][kk][n]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    x.load_k(ck, sk, (size_t)j0 + STEP, rows_of(next));   // (behind the last slots: no rows)
    Frag<bf16> P[NT][N];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int u = 0; u < 2; ++u) X[nt][u] *= c;
      if (live != ~0u) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!((live >> (16 * (j >> 2) + 4 * lg + (j & 3))) & 1)) X[nt][j >> 2][j & 3] = -INFINITY;
      }
      float mx = X[nt][0][0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mx = fmaxf(mx, X[nt][j >> 2][j & 3]);
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
      mx = group_max(mx);
      if (__any(mx > m[nt] + 8.f)) {             // rescale only when a maximum grows by 2^8
        const float mn = fmaxf(m[nt], mx), alpha = __builtin_amdgcn_exp2f(m[nt] - mn);
        m[nt] = mn;
        l[nt] *= alpha;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) O[nt][dt] *= alpha;
      }
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = __builtin_amdgcn_exp2f(X[nt][j >> 2][j & 3] - m[nt]);
        l[nt] += y[j];
      }
      bf16_parts<N>(y, P[nt]);                   // (bf16: rounded for the product with v, the sum l is not)
    }
    if (own >= 0 && own < 32) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = j & 3, u = j >> 2;
        if (own == 16 * u + 4 * lg + i) {
          if constexpr (Step::VB == 2) x.v[j][0] = reinterpret_cast<const unsigned short*>(fresh[1])[lr];
          else
#pragma unroll
            for (int w = 0; w < Step::VW; ++w) x.v[j][w] = fresh[1][lr * Step::VW + w];
          if constexpr (SB == 4) x.vs[u][i] = *reinterpret_cast<const u32*>(fresh_scale[1]);
          else {
            const u32 s = *reinterpret_cast<const unsigned short*>(fresh_scale[1]);
            x.vs[u][i >> 1] = (i & 1) ? (x.vs[u][i >> 1] & 0xffffu) | s << 16 : (x.vs[u][i >> 1] & 0xffff0000u) | s;
          }
        }
      }
    }
    // V^T operands, two rows d of it at a time: two values of each of the eight slots, paired up by slot
    float vscale[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) vscale[j] = scale_value(x.v_scale(j));
    if (BUDGET && live != ~0u) {                 // what stands in empty slots reaches nothing
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!((live >> (16 * (j >> 2) + 4 * lg + (j & 3))) & 1)) {
          vscale[j] = 0.f;
#pragma unroll
          for (int w = 0; w < Step::VW; ++w) x.v[j][w] = 0;
        }
    }
    auto pair_of_rows = [&](auto xx) {
      constexpr int X2 = decltype(xx)::value, W = BITS == 4 ? X2 / 4 : X2 / 2, S = BITS == 4 ? X2 % 4 : X2 % 2;
      u32x4 even, odd;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const u32 y = read_pair<BITS, S>(x.v[j][W], vscale[j]), z = read_pair<BITS, S>(x.v[j + 1][W], vscale[j + 1]);
        even[j / 2] = __builtin_amdgcn_perm(z, y, 0x05040100u);
        odd[j / 2] = __builtin_amdgcn_perm(z, y, 0x07060302u);
      }
      Frag<bf16> F0, F1;
      F0.v = __builtin_bit_cast(bf16x8, even);
      F1.v = __builtin_bit_cast(bf16x8, odd);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n = N - 1; n >= 0; --n) {
          mma(O[nt][2 * X2], F0, P[nt][n]);
          mma(O[nt][2 * X2 + 1], F1, P[nt][n]);
        }
    };
    pair_of_rows(std::integral_constant<int, 0>());
    pair_of_rows(std::integral_constant<int, 1>());
    if constexpr (D == 128) {
      pair_of_rows(std::integral_constant<int, 2>());
      pair_of_rows(std::integral_constant<int, 3>());
    }
    __builtin_amdgcn_sched_barrier(0);
    x.load_v(cv, sv, (size_t)j0 + STEP, rows_of(next));
    live = next;
  }
  // join the waves, 16 heads at a time (4-float pieces of a row swizzled by the head); row 4 lg + i of tile
  // dt of an accumulator is element (4 lg + i) D / 16 + dt
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
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int h = 0; h < DT / 4; ++h)
        store4(mg + (wave * 16 + lr) * D + ((((4 * lg + i) * (DT / 4) + h) ^ lr) << 2),
               f32x4{O[nt][4 * h][i], O[nt][4 * h + 1][i], O[nt][4 * h + 2][i], O[nt][4 * h + 3][i]});
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * D / 4; i += 64 * NW) {
      const int h = i / (D / 4), c4 = i % (D / 4), g = 16 * nt + h;
      if (g >= G) continue;
      float M = kNegBig, L = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, ml[w][h][0]);
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float f = __builtin_amdgcn_exp2f(ml[w][h][0] - M);
        L += f * ml[w][h][1];
        y += load4f(mg + (w * 16 + h) * D + ((c4 ^ h) << 2)) * f;
      }
      if (a.n_split == 1) {
        const float f = L != 0.f ? 1.f / L : 0.f;
        store4(ob + (size_t)g * D + 4 * c4, y * f);
        if (c4 == 0) {
          st[g][0] = M;
          st[g][1] = f;
        }
      } else {
        float* dst = a.part + (((size_t)bk * a.n_split + split) * G + g) * (D + 4);
        store4(dst + 4 + 4 * c4, y);
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

template <typename T, int BITS, int D, int NT, bool BUDGET>
static hipError_t launch_nt(const CacheArgs& a, hipStream_t st) {
  const int units = a.B * a.Hkv, G = a.Hq / a.Hkv;
  const dim3 grid(units * a.n_split);
  hipError_t e;
  if (NT == 1 && a.waves == 8 && BUDGET && !a.score)
    e = launch_kernel<0>(mx_decode_kernel<T, BITS, D, 1, 8, BUDGET, BUDGET>, grid, 512, a, st);
  else if (NT == 1 && a.waves == 8)
    e = launch_kernel<0>(mx_decode_kernel<T, BITS, D, 1, 8, BUDGET, false>, grid, 512, a, st);
  else
    e = launch_kernel<0>(mx_decode_kernel<T, BITS, D, NT, 4, BUDGET, false>, grid, kDecThreads, a, st);
  if (e != hipSuccess || a.n_split == 1) return e;
  return launch_kernel<0>(cache_join_kernel<T, D, BUDGET>, dim3(units * (BUDGET ? G + a.n_split : G)), kDecThreads, a, st);
}
template <typename T, int BITS, int D, bool BUDGET>
static hipError_t launch_g(const CacheArgs& a, hipStream_t st) {
  const int G = a.Hq / a.Hkv;
  if (G <= 16) return launch_nt<T, BITS, D, 1, BUDGET>(a, st);
  if (G <= 32) return launch_nt<T, BITS, D, 2, BUDGET>(a, st);
  return launch_nt<T, BITS, D, 4, BUDGET>(a, st);
}
template <typename T, int BITS, int D>
static hipError_t launch(const CacheArgs& a, hipStream_t st) {
  return a.cache_w ? launch_g<T, BITS, D, true>(a, st) : launch_g<T, BITS, D, false>(a, st);
}
template <typename T, int BITS>
static hipError_t launch_d(const CacheArgs& a, hipStream_t st) {
  return a.D == 128 ? launch<T, BITS, 128>(a, st) : launch<T, BITS, 64>(a, st);
}
hipError_t launch_mx_decode(const CacheArgs& a, hipStream_t st) {
  if (a.bits == 4) return a.dtype ? launch_d<bf16, 4>(a, st) : launch_d<float, 4>(a, st);
  return a.dtype ? launch_d<bf16, 8>(a, st) : launch_d<float, 8>(a, st);
}

}  // namespace carve
