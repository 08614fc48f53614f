// One new token per sequence against a cache held in codes of 4 or 8 bits (mx_device.h): the ring cache
// and the cache kept by attention weight, with the split, the softmax and the joins of cache_decode.hip.
//
// What codes stand for is a bf16 exactly, so both products run on bf16 operands; where q is float32, q
// and the weights go in as three bf16 parts each, which hold all their bits (256 sequences, 16 heads on 4, window 4,096,
// 4 bits: 130 us, bf16 111).  With bf16 queries the weights are two parts: rounded to one, the largest weight of a row would be
// off by as much as the output's own rounding (error against 64 bits 2.0e-3 to 2.5e-3; two parts 1.5e-3 to 1.6e-3, the
// rounding of the output alone).  One part: 108 us; 4 key heads of 1,028 slots 8.6 us, two parts 9.1; 64 heads on one,
// 2,048 slots 39 and 45.
// Codes reach LDS by loads that write it directly; a lane converts what it reads from there.
// The contraction of S^T = K Q^T may run over a key's elements in any order that q's have too, so a lane takes D / 4
// neighbouring ones, with one scale; for O^T = V^T P^T it takes D / 16 neighbouring elements of each of its eight
// slots and pairs the slots up as it converts.  The token's own row is written over its place in LDS by the wave that
// holds its slot, as well as to the cache, so no wave waits for a store.
//
// Bound by the cache's read where a compute unit has several key heads: 256 sequences as above, some still
// filling (about 540 MB), in 91 to 106 us, 5.1 to 5.9 TB/s; a plain read of as much takes 88.  The vector units are then busy for
// 0.71 of the time (conversions, their pairing, exponentials), the matrix units for 0.28 (one part of the weights: 0.58 and
// 0.15; then the time was the same without the value products, and without exponentials).  With few key heads it is latency:
// 4 of 1,028 slots 9.1 us, about 5 of them before and after the slots, 1.05 a step of 256 slots.  With weights 64
// sequences of 2,048 slots 22 us (the slot's search before, the weights after the steps); 256 of 4,096 slots 140 us:
// the scores' way to memory and back, 134 MB, beside 570 MB of rows and 50 of positions and weights.  More than 32 heads on a
// key head take 64 columns of registers, one wave a SIMD (80 heads on 2, 256 sequences of 4,096 slots: 153 us, read in 50),
// and spill in float32 with D = 128 (64 heads on one, 2,048 slots: 138 us, bf16 45).
#include <algorithm>

#include "cache_step.h"
#include "mx_device.h"

namespace carve {

// x as N bf16 parts that add up to it (N = 2: but for 2^-15 of it, the second part's rounding; 3: all bits of a float)
template <int N>
__device__ __forceinline__ void bf16_parts(const float (&x)[8], Frag<bf16> (&f)[N]) {
  u32 w[N][4];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float a = x[j], b = x[j + 1];
#pragma unroll
    for (int n = 0; n < N; ++n) {                 // the upper half of a float is a bf16; the rest is exact
      if (N == 2 && n == 1) {
        w[n][j / 2] = __builtin_bit_cast(u32, bf16x2{(bf16)a, (bf16)b});
        break;
      }
      const u32 ua = __builtin_bit_cast(u32, a), ub = __builtin_bit_cast(u32, b);
      w[n][j / 2] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
      a -= __builtin_bit_cast(float, ua & 0xffff0000u);
      b -= __builtin_bit_cast(float, ub & 0xffff0000u);
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) f[n].v = __builtin_bit_cast(bf16x8, u32x4{w[n][0], w[n][1], w[n][2], w[n][3]});
}

// 32 slots of a wave in LDS, where buffer loads that write it directly put them (the scales come through a
// register each).  Such loads fill LDS in lane order, 16 bytes a lane; which row they come from is free.
// Keys stand row by row, the 16-byte pieces of a row swizzled: lane (lr, lg) reads elements lg D / 4 .. of slots lr and
// 16 + lr, sixteen rows at one piece.  Of each 16 values, rows 4 lg + i stand at places 4 i + lg: lanes
// (lr, lg) read elements lr D / 16 .. of slots 4 lg + i, one i at a time, which are then neighbours.
template <int BITS, int D>
struct MxTile {
  static constexpr int RB = D * BITS / 8, SB = D / 32;                  // bytes of a row, of its scales
  static constexpr int KW = RB / 16, VB = RB / 16, VW = VB < 4 ? 1 : VB / 4;   // words a lane and key; bytes, words a slot
  static constexpr int kRows = 32 * RB, kBytes = 2 * kRows, kLoads = kRows / 1024;   // a side; both; instructions a side
  static constexpr int kScales = 64 * SB;

  // n rows of a cache from slot j0 on (a read behind them gives zero)
  static __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(const void* base, size_t j0, int n, int row_bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((char*)base + j0 * row_bytes, 0, n * row_bytes, 0x00020000);
  }
  // place of a key row's piece of 16 bytes within the row: ^ this
  static __device__ __forceinline__ int swz(int row) { return RB == 32 ? 0 : RB == 64 ? (row >> 2) & 3 : (row >> 1) & 7; }
  // 16 bytes a lane to LDS, marked as not used again (2): codes are read once a step, and a load that takes no place in
  // the caches need not move out what others wrote there.  256 / 64 sequences, 16 heads on 4, window 4,096, 4 bits: 111 /
  // 30 us again and again, 134 / 44 after other work has filled the caches; without the mark 124 / 27 and 178 / 66.
  // (The scales, 128 bytes of a line at a time, are left their places: marked too, 4 us more of the 107 at the time.)
  static __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, unsigned char* dst, int off, int more) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)dst, 16, off, more, 0, 2);
  }
  static __device__ __forceinline__ void load_k(unsigned char* dst, const void* codes, size_t j0, int n) {
    const auto r = rows(codes, j0, n, RB);
    const int lane = lane_id(), row = lane * 16 / RB;
    const int off = 16 * (lane ^ swz(row));
#pragma unroll
    for (int h = 0; h < kLoads; ++h)             // (8 bits, D = 128: eight rows a load; the swizzle of rows 8 .. 15 is ^ 4)
      load(r, dst + 1024 * h, RB == 128 && (h & 1) ? off ^ 64 : off, 1024 * h);
  }
  static __device__ __forceinline__ void load_v(unsigned char* dst, const void* codes, size_t j0, int n) {
    const int lane = lane_id(), place = lane * 16 / RB;
    const auto r = rows(codes, j0, n, RB);
    const int off = (16 * (place >> 4) + 4 * (place & 3) + ((place & 15) >> 2)) * RB + lane * 16 % RB;
#pragma unroll
    for (int h = 0; h < kLoads; ++h)
      load(r, dst + kRows + 1024 * h, off, (RB == 128 ? (h >> 1) * 16 + (h & 1) * 2 : h * 16) * RB);
  }
  // the scales of slot lane % 32, of its key and its value
  static __device__ __forceinline__ u32x2 load_scales(const void* sk, const void* sv, size_t j0, int n) {
    const int slot = lane_id() & 31;
    const auto rk = rows(sk, j0, n, SB), rv = rows(sv, j0, n, SB);
    u32 x, y;
    if constexpr (SB == 4) {
      x = __builtin_amdgcn_raw_buffer_load_b32(rk, slot * SB, 0, 0);
      y = __builtin_amdgcn_raw_buffer_load_b32(rv, slot * SB, 0, 0);
    } else {
      x = (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(rk, slot * SB, 0, 0);
      y = (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(rv, slot * SB, 0, 0);
    }
    return u32x2{x, y};
  }
  // to LDS: all keys', then all values'
  static __device__ __forceinline__ void put_scales(unsigned char* s, u32x2 f) {
    const u32 x = lane_id() < 32 ? f[0] : f[1];
    if constexpr (SB == 4) reinterpret_cast<u32*>(s)[lane_id()] = x;
    else reinterpret_cast<unsigned short*>(s)[lane_id()] = (unsigned short)x;
  }
  // Reads of what direct loads brought are written out, each with its own wait: before a read that the
  // compiler makes it waits for every direct load, those of the next steps too.
  static __device__ __forceinline__ u32 address(const unsigned char* p) {
    return (u32)(uintptr_t)(__attribute__((address_space(3))) const unsigned char*)p;
  }
  // the lane's key elements of slots lr and 16 + lr, and their scales
  static __device__ __forceinline__ void read_k(const unsigned char* src, const unsigned char* s, u32 (&w)[2][KW], float (&f)[2]) {
    const int lane = lane_id(), lr = lane & 15, lg = lane >> 4;
    const u32 at = address(src) + (KW == 2 ? 32 * lr + 8 * lg : KW == 4 ? 64 * lr + 16 * (lg ^ swz(lr)) : 128 * lr + 16 * ((2 * lg) ^ swz(lr))), st = address(s) + lr * SB + lg * SB / 4;
    u32 sc[2];
    if constexpr (KW == 2) {
      u32x2 x, y;
      asm volatile("ds_read_b64 %0, %4\n\tds_read_b64 %1, %4 offset:512\n\tds_read_u8 %2, %5\n\tds_read_u8 %3, %5 offset:%6\n\t"
                   "s_waitcnt lgkmcnt(0)" : "=&v"(x), "=&v"(y), "=&v"(sc[0]), "=&v"(sc[1]) : "v"(at), "v"(st), "n"(16 * SB) : "memory");
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[0][i] = x[i];
        w[1][i] = y[i];
      }
    } else if constexpr (KW == 4) {
      u32x4 x, y;
      asm volatile("ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:1024\n\tds_read_u8 %2, %5\n\tds_read_u8 %3, %5 offset:%6\n\t"
                   "s_waitcnt lgkmcnt(0)" : "=&v"(x), "=&v"(y), "=&v"(sc[0]), "=&v"(sc[1]) : "v"(at), "v"(st), "n"(16 * SB) : "memory");
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[0][i] = x[i];
        w[1][i] = y[i];
      }
    } else {
      u32x4 x[4];
      asm volatile("ds_read_b128 %0, %6\n\tds_read_b128 %1, %7\n\tds_read_b128 %2, %6 offset:2048\n\t"
                   "ds_read_b128 %3, %7 offset:2048\n\tds_read_u8 %4, %8\n\tds_read_u8 %5, %8 offset:%9\n\ts_waitcnt lgkmcnt(0)"
                   : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(sc[0]), "=&v"(sc[1])
                   : "v"(at), "v"(at ^ 16), "v"(st), "n"(16 * SB) : "memory");
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[0][i] = x[i >> 2][i & 3];
        w[1][i] = x[2 + (i >> 2)][i & 3];
      }
    }
    f[0] = scale_value(sc[0]);
    f[1] = scale_value(sc[1]);
  }
  // the lane's value elements of slots 16 u + 4 lg + i, j = 4 u + i, and their scales: the byte of the block
  // turned to where a float has its exponent (the conversions look at nothing else of it)
  static __device__ __forceinline__ void read_v(const unsigned char* src, const unsigned char* s, u32 (&w)[8][VW], float (&f)[8]) {
    const int lane = lane_id(), blk = (lane & 15) * SB / 16;
    const u32 at = address(src + kRows) + lane * VB, st = address(s) + (32 + 4 * (lane >> 4)) * SB;
    u32 sc[2][SB];
    if constexpr (VB == 2) {
      u32x2 p, q;
      asm volatile("ds_read_u16 %0, %10\n\tds_read_u16 %1, %10 offset:128\n\tds_read_u16 %2, %10 offset:256\n\t"
                   "ds_read_u16 %3, %10 offset:384\n\tds_read_u16 %4, %10 offset:512\n\tds_read_u16 %5, %10 offset:640\n\t"
                   "ds_read_u16 %6, %10 offset:768\n\tds_read_u16 %7, %10 offset:896\n\t"
                   "ds_read_b64 %8, %11\n\tds_read_b64 %9, %11 offset:32\n\ts_waitcnt lgkmcnt(0)"
                   : "=&v"(w[0][0]), "=&v"(w[1][0]), "=&v"(w[2][0]), "=&v"(w[3][0]), "=&v"(w[4][0]), "=&v"(w[5][0]),
                     "=&v"(w[6][0]), "=&v"(w[7][0]), "=&v"(p), "=&v"(q) : "v"(at), "v"(st) : "memory");
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[0][i] = p[i];
        sc[1][i] = q[i];
      }
    } else if constexpr (VB == 4) {
      u32x2 x[4];
      if constexpr (SB == 4) {
        u32x4 p, q;
        asm volatile("ds_read2st64_b32 %0, %6 offset1:1\n\tds_read2st64_b32 %1, %6 offset0:2 offset1:3\n\t"
                     "ds_read2st64_b32 %2, %6 offset0:4 offset1:5\n\tds_read2st64_b32 %3, %6 offset0:6 offset1:7\n\t"
                     "ds_read_b128 %4, %7\n\tds_read_b128 %5, %7 offset:64\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(p), "=&v"(q) : "v"(at), "v"(st) : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[0][i] = p[i];
          sc[1][i] = q[i];
        }
      } else {
        u32x2 p, q;
        asm volatile("ds_read2st64_b32 %0, %6 offset1:1\n\tds_read2st64_b32 %1, %6 offset0:2 offset1:3\n\t"
                     "ds_read2st64_b32 %2, %6 offset0:4 offset1:5\n\tds_read2st64_b32 %3, %6 offset0:6 offset1:7\n\t"
                     "ds_read_b64 %4, %7\n\tds_read_b64 %5, %7 offset:32\n\ts_waitcnt lgkmcnt(0)"
                     : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(p), "=&v"(q) : "v"(at), "v"(st) : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sc[0][i] = p[i];
          sc[1][i] = q[i];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j][0] = x[j >> 1][j & 1];
    } else {
      u32x4 x[4], p, q;
      asm volatile("ds_read2st64_b64 %0, %6 offset1:1\n\tds_read2st64_b64 %1, %6 offset0:2 offset1:3\n\t"
                   "ds_read2st64_b64 %2, %6 offset0:4 offset1:5\n\tds_read2st64_b64 %3, %6 offset0:6 offset1:7\n\t"
                   "ds_read_b128 %4, %7\n\tds_read_b128 %5, %7 offset:64\n\ts_waitcnt lgkmcnt(0)"
                   : "=&v"(x[0]), "=&v"(x[1]), "=&v"(x[2]), "=&v"(x[3]), "=&v"(p), "=&v"(q) : "v"(at), "v"(st) : "memory");
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) w[j][i] = x[j >> 1][2 * (j & 1) + i];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[0][i] = p[i];
        sc[1][i] = q[i];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = j & 3;
      const u32 y = sc[j >> 2][i * SB / 4];
      f[j] = __builtin_bit_cast(float, __builtin_amdgcn_alignbit(y, y, (8 * (blk + (SB == 4 ? 0 : 2 * (i & 1))) + 9) & 31));
    }
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
__global__ __launch_bounds__(64 * NW, NT == 1 ? (sizeof(T) == 2 ? 4 : 2) : 1) void mx_decode_kernel(CacheArgs a) {
  using Tile = MxTile<BITS, D>;
  constexpr int STEP = 32 * NW, N = sizeof(T) == 2 ? 1 : 3, NP = sizeof(T) == 2 ? 2 : 3, KK = D / 32, DT = D / 16;
  constexpr int RB = Tile::RB, SB = Tile::SB;
  constexpr int AHEAD = 2;                                       // steps whose rows are on their way or in use
  constexpr int BUFFERS = NW * AHEAD * Tile::kBytes, MERGE = NW * 16 * D * 4;
  __shared__ __align__(16) unsigned char smem[BUFFERS > MERGE ? BUFFERS : MERGE];
  __shared__ __align__(16) unsigned char scales[NW][Tile::kScales];
  __shared__ unsigned long long red[NW];
  __shared__ float ml[NW][16][2];
  __shared__ float st[16 * NT][2];
  __shared__ __align__(16) u32 fresh[2][RB / 4];                 // the token's k and v
  __shared__ unsigned char fresh_scale[2][SB];
  __shared__ __align__(16) float near_score[NEAR ? mx_near_scores(BITS, D, NW) : 4];
  const int G = a.Hq / a.Hkv;
  const int split = uniform(blockIdx.x % a.n_split), bk = uniform(blockIdx.x / a.n_split), b = uniform(bk / a.Hkv);
  const int lane = lane_id(), wave = wave_uid(), lr = lane & 15, lg = lane >> 4;
  const int lo = split * a.split_len, end = min(lo + a.split_len, a.C), first = lo + 32 * wave;
  char* ck = reinterpret_cast<char*>(a.cache_k) + (size_t)bk * a.C * RB;
  char* cv = reinterpret_cast<char*>(a.cache_v) + (size_t)bk * a.C * RB;
  unsigned char* sk = a.k_scales + (size_t)bk * a.C * SB;
  unsigned char* sv = a.v_scales + (size_t)bk * a.C * SB;
  const int* held = BUDGET ? a.cache_pos + (size_t)bk * a.C : nullptr;
  auto position = [&](int j0) { return BUDGET ? held[min(j0 + (lane & 31), a.C - 1)] : 0; };
  // What does not depend on the position is asked for before it is known: q, a piece a lane of the token's k and v, the
  // first steps' rows.  In this order, since loads arrive in order.
  const int pos_b = a.pos[b];
  const int piece = lane % (D / 8), is_v = lane / (D / 8) & 1;
  const Frag<T> token = load_frag(reinterpret_cast<const T*>(is_v ? a.v : a.k) + (size_t)bk * D + 8 * piece);
  Frag<T> q[NT][KK];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
      q[nt][kk] = load_frag(reinterpret_cast<const T*>(a.q) + ((size_t)bk * G + min(16 * nt + lr, G - 1)) * D + lg * (D / 4) + 8 * kk);
  int pos[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) pos[i] = position(first + i * STEP);
  unsigned char* buf = smem + wave * AHEAD * Tile::kBytes;
  unsigned char* sc = scales[wave];
  u32x2 scale_ahead[AHEAD];
  auto fetch_k = [&](int stage, int j0, int n) {
    Tile::load_k(buf + stage * Tile::kBytes, ck, j0, n);
    scale_ahead[stage] = Tile::load_scales(sk, sv, j0, n);
  };
  auto fetch_v = [&](int stage, int j0, int n) { Tile::load_v(buf + stage * Tile::kBytes, cv, j0, n); };
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    const int j0 = first + i * STEP, n = uniform(max(0, min(end - j0, 32)));
    fetch_k(i, j0, n);
    __builtin_amdgcn_sched_barrier(0);           // the waits below count on this order
    fetch_v(i, j0, n);
    __builtin_amdgcn_sched_barrier(0);
  }
  const int p = uniform(pos_b);
  T* ob = reinterpret_cast<T*>(a.o) + (size_t)bk * G * D;
  if (p < 0) {                                   // no token: the cache stays as it is
    if (split == 0) {
      for (int i = threadIdx.x; i < G * D; i += 64 * NW) ob[i] = to<T>(0.f);
      if (BUDGET && threadIdx.x == 0) a.slot[bk] = -1;
    }
    wait_loads<0>();                             // (they write LDS that the next workgroup may have)
    return;
  }
  const int count = BUDGET ? a.C : min(p, a.C - 1) + 1;          // a ring holds its tokens from slot 0 up
  const int hi = min(end, count);
  // slots of the 32 from j0 that hold a token, one bit each; rows to read: up to the last of them
  auto live_of = [&](int j0, int held_pos) {
    const int j = j0 + (lane & 31);
    return (unsigned)__ballot(j < hi && (!BUDGET || held_pos >= 0));
  };
  auto rows_of = [&](unsigned live) { return uniform(32 - __clz((int)live)); };
  unsigned live[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) live[i] = live_of(first + i * STEP, pos[i]);
  const int at = uniform(BUDGET ? pick_slot<NW>(a, bk, p, red) : ring_slot(a, p));
  if (BUDGET && split == 0 && threadIdx.x == 0) a.slot[bk] = at;
  // the wave that holds the slot writes the token's rows
  if (at >= lo && at < hi && (at - lo) / 32 % NW == wave) {
    if (lane < D / 4) {
      u32 scale;
      const Eight<BITS> c = write_block<BITS>(token, scale);
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
  auto put_token = [&](unsigned char* rows, unsigned char* s, int own) {
    const int u = own >> 4, r = own & 15;
    const u32* k = fresh[0];
    const u32* v = fresh[1];
    if (lane < RB / 4) {                         // a word of k and of v
      const int place = own * (RB / 4) + (lane ^ 4 * Tile::swz(r));
      reinterpret_cast<u32*>(rows)[place] = k[lane];
      reinterpret_cast<u32*>(rows + Tile::kRows)[(16 * u + 4 * (r & 3) + (r >> 2)) * (RB / 4) + lane] = v[lane];
    }
    if (lane < SB) {
      s[own * SB + lane] = fresh_scale[0][lane];
      s[(32 + own) * SB + lane] = fresh_scale[1][lane];
    }
  };
  Frag<bf16> Q[NT][KK][N];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      if constexpr (N == 1) {
        Q[nt][kk][0] = q[nt][kk];
      } else {
        float y[8];
        to_floats(q[nt][kk], y);
        bf16_parts<N>(y, Q[nt][kk]);
      }
    }
  const float c = a.scale * kLog2e;
  f32x4 O[NT][DT];
  float m[NT], l[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt] = kLeast;
    l[nt] = 0.f;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) O[nt][dt] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // instructions of a step's loads in the order they are issued: k, scales (two), v, and one for positions; waiting
  // for k (v) leaves those that were issued after it on their way
  constexpr int kStep = 2 * Tile::kLoads + 2 + BUDGET;
  constexpr int kAfterK = Tile::kLoads + (AHEAD - 1) * kStep, kAfterV = (AHEAD - 1) * kStep + Tile::kLoads + 2;
  int ahead = position(first + AHEAD * STEP);    // asked for a step before the rows
  auto step = [&](auto stage_, int j0) {
    constexpr int stage = decltype(stage_)::value;
    unsigned char* rows = buf + stage * Tile::kBytes;
    const unsigned next = live_of(j0 + AHEAD * STEP, ahead);
    ahead = position(j0 + (AHEAD + 1) * STEP);
    const int own = at - j0;                     // the token's slot, if of these
    wait_loads<kAfterK>();
    Tile::put_scales(sc, scale_ahead[stage]);
    if (own >= 0 && own < 32) {                  // its rows as codes, over what was there
      live[stage] |= 1u << own;
      wait_loads<0>();
      put_token(rows, sc, own);
    }
    const unsigned on = live[stage];
    u32 kw[2][Tile::KW];
    float kscale[2];
    Tile::read_k(rows, sc, kw, kscale);
    f32x4 X[NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Frag<bf16> K[KK];
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        Eight<BITS> e;
        if constexpr (BITS == 4) e.w = kw[u][kk];
        else e.w = u32x2{kw[u][2 * kk], kw[u][2 * kk + 1]};
        K[kk] = read_eight<BITS>(e, kscale[u]);
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
    live[stage] = next;
    __builtin_amdgcn_sched_barrier(0);
    fetch_k(stage, j0 + AHEAD * STEP, rows_of(next));            // (behind the last slots: no rows)
    Frag<bf16> P[NT][NP];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int u = 0; u < 2; ++u) X[nt][u] *= c;
      if (on != ~0u) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!((on >> (16 * (j >> 2) + 4 * lg + (j & 3))) & 1)) X[nt][j >> 2][j & 3] = -INFINITY;
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
      bf16_parts<NP>(y, P[nt]);
    }
    // V^T operands, two rows d of it at a time: two values of each of the eight slots, paired up by slot
    u32 v[8][Tile::VW];
    float vscale[8];
    wait_loads<kAfterV>();
    Tile::read_v(rows, sc, v, vscale);
    if (on != ~0u) {                             // what stands in empty slots reaches nothing
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!((on >> (16 * (j >> 2) + 4 * lg + (j & 3))) & 1)) {
          vscale[j] = 0.f;
#pragma unroll
          for (int w = 0; w < Tile::VW; ++w) v[j][w] = 0;
        }
    }
    auto pair_of_rows = [&](auto xx) {
      constexpr int X2 = decltype(xx)::value, W = BITS == 4 ? X2 / 4 : X2 / 2, S = BITS == 4 ? X2 % 4 : X2 % 2;
      u32x4 even, odd;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const u32 y = read_pair<BITS, S>(v[j][W], vscale[j]), z = read_pair<BITS, S>(v[j + 1][W], vscale[j + 1]);
        even[j / 2] = __builtin_amdgcn_perm(z, y, 0x05040100u);
        odd[j / 2] = __builtin_amdgcn_perm(z, y, 0x07060302u);
      }
      Frag<bf16> F0, F1;
      F0.v = __builtin_bit_cast(bf16x8, even);
      F1.v = __builtin_bit_cast(bf16x8, odd);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) {
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
    fetch_v(stage, j0 + AHEAD * STEP, rows_of(next));
  };
  if (first < hi) {
    for (int j0 = first;;) {
      step(std::integral_constant<int, 0>(), j0);
      j0 += STEP;
      if (j0 >= hi) break;
      step(std::integral_constant<int, 1>(), j0);
      j0 += STEP;
      if (j0 >= hi) break;
    }
  }
  wait_loads<0>();                               // nothing writes LDS any more
  float* mg = reinterpret_cast<float*>(smem);
  WeightBatch<NW> before;                        // on their way while the waves are joined
  if (BUDGET && a.n_split == 1) before.load(a, bk, threadIdx.x, a.C);
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
      float M = kLeast, L = 0.f;
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
        const float f = 1.f / L;                 // (where that is zero: see cache_join_kernel)
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
    add_weights<NW>(a, bk, p, at, 0, a.C, &st[0][0], NEAR ? near_score : a.score + (size_t)bk * G * score_row(a.C), before);
  }
}

template <typename T, int BITS, int D, int NT, bool BUDGET>
static hipError_t launch_nt(const CacheArgs& a, hipStream_t st) {
  const int units = a.B * a.Hkv, G = a.Hq / a.Hkv;
  const dim3 grid(units * a.n_split);
  hipError_t e;
  constexpr int N8 = NT == 4 ? 2 : NT;           // (more than 32 heads: 4 waves only, registers)
  if (NT < 4 && a.waves == 8 && BUDGET && !a.score)
    e = launch_kernel<0>(mx_decode_kernel<T, BITS, D, N8, 8, BUDGET, BUDGET>, grid, 512, a, st);
  else if (NT < 4 && a.waves == 8)
    e = launch_kernel<0>(mx_decode_kernel<T, BITS, D, N8, 8, BUDGET, false>, grid, 512, a, st);
  else if (NT == 1 && BUDGET && !a.score)
    e = launch_kernel<0>(mx_decode_kernel<T, BITS, D, 1, 4, BUDGET, BUDGET>, grid, kDecThreads, a, st);
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
