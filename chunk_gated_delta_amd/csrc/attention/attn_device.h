// Building blocks of the attention kernels: 32x32 MFMA tiles and staging of token rows.
//
// A score tile is always formed with the tokens that own the softmax statistics on its
// columns, so that a lane holds values of ONE token: v_mfma_f32_32x32x16_bf16 returns
//   C (32 x 32): lane l holds C[8 (i / 4) + 4 (l / 32) + i % 4][l % 32], i = 0..15,
// of operands A (32 x 16): lane l holds A[l % 32][8 (l / 32) + j], and B (16 x 32): lane l
// holds B[8 (l / 32) + j][l % 32], j = 0..7 (fp32: eight v_mfma_f32_32x32x2 steps over
// the same lane values).  Registers 8 x .. 8 x + 7 of C are, rounded, a B operand whose
// contraction index runs over the rows 16 x + 8 (j / 4) + 4 (l / 32) + j % 4 of C, so
// weights go from the score tile into the next product without leaving their lane; the
// other operand of that product is read with its rows in the same order (frag_cols32, col_frag).
#pragma once
#include "../carve_device.h"
#include "attn_internal.h"

namespace carve {

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegBig = -1.0e30f;     // running maximum before any visible score (whole sequences)

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}
__device__ __forceinline__ void mma32(f32x16& c, const Frag<bf16>& a, const Frag<bf16>& b) {
  c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ void mma32(f32x16& c, const Frag<float>& a, const Frag<float>& b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.lo[j], b.lo[j], c, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.hi[j], b.hi[j], c, 0, 0, 0);
}
// row of register i of a 32 x 32 accumulator tile
__device__ __forceinline__ int acc_row(int i, int half) { return 8 * (i >> 2) + 4 * half + (i & 3); }

// Rows r0 .. r0 + 31 of a row-major LDS matrix, 16-deep block at column k0 (A operand).
template <typename T>
__device__ __forceinline__ Frag<T> frag_rows32(const T* m, int ld, int r0, int k0) {
  const int lane = lane_id();
  return load_frag(m + (r0 + (lane & 31)) * ld + k0 + 8 * (lane >> 5));
}
// Columns c0 .. c0 + 31 of a row-major LDS matrix as the 32 rows of an A operand, its 16-deep
// contraction over rows k0 + 8 (j / 4) + 4 (l / 32) + j % 4 (fp32; bf16 tiles: SwzTile::col_frag).
__device__ __forceinline__ Frag<float> frag_cols32(const float* m, int ld, int c0, int k0) {
  const int lane = lane_id();
  const float* p = m + (k0 + 4 * (lane >> 5)) * ld + c0 + (lane & 31);
  Frag<float> f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.lo[j] = p[j * ld];
    f.hi[j] = p[(j + 8) * ld];
  }
  return f;
}
// registers 8 x .. 8 x + 7 of an accumulator tile as a B operand (rounded for bf16)
__device__ __forceinline__ void acc_frag(const f32x16& c, int x, Frag<bf16>& f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f.v[j] = (bf16)c[8 * x + j];
}
__device__ __forceinline__ void acc_frag(const f32x16& c, int x, Frag<float>& f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f.lo[j] = c[8 * x + j];
    f.hi[j] = c[8 * x + 4 + j];
  }
}

// ROWS token rows of a [n][D] matrix, moved through registers into a padded LDS tile by
// NT threads in pieces of 8 elements; rows at or past n become zero, so that nothing
// behind a sequence's end (not a number, say) reaches a product.
template <typename T, int ROWS, int D, int NT>
struct RowStage {
  static constexpr int PR = D / 8, NP = ROWS * PR, NST = NP / NT;
  static_assert(NP % NT == 0, "whole pieces per thread");
  static constexpr int LD = D + Pad<T>::v;
  Frag<T> x[NST];
  __device__ __forceinline__ void load(const T* base, int r0, int n) {
#pragma unroll
    for (int u = 0; u < NST; ++u) {
      const int p = threadIdx.x + NT * u, r = r0 + p / PR;
      x[u] = load_frag(base + (size_t)(r < n ? r : n - 1) * D + 8 * (p % PR));
      if (r >= n) x[u] = zero_frag(T());
    }
  }
  __device__ __forceinline__ void store(T* tile) const {
#pragma unroll
    for (int u = 0; u < NST; ++u) {
      const int p = threadIdx.x + NT * u;
      *reinterpret_cast<Frag<T>*>(tile + (p / PR) * LD + 8 * (p % PR)) = x[u];
    }
  }
};

// A value every lane of the wave has, as a scalar: branches on it are uniform, and buffer
// descriptors made of it need no loop over the lanes.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int wave_uid() { return uniform(threadIdx.x >> 6); }

// ROWS bf16 token rows of width D in LDS, brought there by buffer loads that write LDS directly
// (16 bytes a lane, 1 KB a wave and instruction, no registers on the way; rows past a sequence's
// end lie past the buffer's end and read as zero).  Such loads fill LDS in lane order, so rows
// cannot be padded.  The tile is D / 64 blocks of [ROWS][128 bytes], whole cache lines of a row, and
// the 16-byte piece c of a row's eight stands at piece c ^ swz(row), swz = bits 1, 3, 2 of the row
// from the top: neither read pattern has bank conflicts (32 rows at one piece for the row
// operand, 4 rows at 4 neighbouring pieces a 16 lanes for the transpose read), and blocks and rows
// are reached by constant offsets from two addresses a pattern.
// The compiler does not always wait for such loads before the LDS they fill is read: every reader
// waits itself (wait_loads<N>: all but the N youngest vector memory operations of the wave are
// done, loads among themselves in order), then, where other waves read, the barrier.
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) const bf16x8 lds_bf16x8;
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
  __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void loads_and_barrier() {
  wait_loads<0>();
  __syncthreads();
}

template <int D, int ROWS>
struct SwzTile {
  static constexpr int RB = 2 * D, BLOCK = 128 * ROWS, bytes = ROWS * RB;
  static __device__ __forceinline__ int swz(int r) { return (((r >> 1) & 1) << 2) | ((r >> 2) & 3); }
  // rows r0 .. r0 + ROWS - 1 of base [n][D] by NW waves
  template <int NW>
  static __device__ __forceinline__ void load(unsigned char* tile, const bf16* base, int r0, int n, int wave) {
    constexpr int INS = bytes / 1024, PER = INS / NW, IPB = BLOCK / 1024;   // instructions: all, a wave's, a block's
    static_assert(PER * NW == INS && IPB % PER == 0, "a wave's instructions lie in one block");
    const int lane = lane_id(), rows = uniform(max(0, min(n - r0, ROWS)));
    const __amdgpu_buffer_rsrc_t rsrc =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16*>(base) + (size_t)r0 * D, 0, rows * RB, 0x00020000);
    const int rl = lane >> 3, blk = wave * PER / IPB, row0 = wave * PER % IPB * 8;
    const int voff = rl * RB + (((lane & 7) ^ swz(rl)) << 4), odd = row0 & 8;
#pragma unroll
    for (int u = 0; u < PER; ++u)            // (swz of rows 8 .. 15: ^ 2)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(tile + blk * BLOCK + (row0 + 8 * u) * 128), 16,
                                               voff ^ (((u & 1) ^ (odd ? 1 : 0)) << 5), blk * 128 + (row0 + 8 * u) * RB, 0, 0);
  }
  // byte offset of the lane's row operand (contraction block kk: ^ (kk % 4) * 32)
  static __device__ __forceinline__ int row_base() {
    const int lane = lane_id(), r = lane & 31;
    return r * 128 + (((lane >> 5) ^ swz(r)) << 4);
  }
  // rows r0 .. r0 + 31, 16-deep block kk
  static __device__ __forceinline__ Frag<bf16> row_frag(const unsigned char* tile, int base, int r0, int kk) {
    Frag<bf16> f;
    f.v = *(lds_bf16x8*)(tile + (kk >> 2) * BLOCK + r0 * 128 + (base ^ ((kk & 3) << 5)));
    return f;
  }
  // byte offset of the lane's transpose read (columns 32 dt: ^ (dt % 2) * 64; rows + 8: ^ 32, + 1024)
  static __device__ __forceinline__ int col_base() {
    const int lane = lane_id(), s = lane & 15, g = lane >> 4, r = 4 * (g >> 1) + (s >> 2);
    return r * 128 + (((2 * (g & 1) + ((s & 3) >> 1)) ^ swz(r)) << 4) + 8 * (s & 1);
  }
  // columns 32 dt .. + 31 as rows of an A operand, contraction over rows k0 + 8 (j / 4) + 4 (l / 32) + j % 4
  // (k0 a multiple of 16)
  static __device__ __forceinline__ Frag<bf16> col_frag(const unsigned char* tile, int base, int dt, int k0) {
    const unsigned char* p = tile + (dt >> 1) * BLOCK + k0 * 128;
    const int b = base ^ ((dt & 1) << 6);
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + b));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 1024 + (b ^ 32)));
    Frag<bf16> f;
    f.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    return f;
  }
};

// x of the lane 32 away
__device__ __forceinline__ float other_half(float x) {
  typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const u32x2 r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (lane_id() & 32) ? r[0] : r[1]);
}

// Key tiles that a tile of tokens t0 .. t1 - 1 sees, in the order sinks, then window.  Of the tiles
// before the window only the sinks are read (rows(i): the keys that tile i is cut off at): what stands
// beside them is not seen, and a product of its weight 0 with a value that is not finite would be.
template <int KT>
struct KeyTiles {
  int lo, nsink, count, n_sinks;
  __device__ __forceinline__ KeyTiles(int t0, int t1, int window, int sinks) {
    lo = max(0, t0 - window + 1) / KT;
    n_sinks = min(sinks, t1);
    nsink = min((n_sinks + KT - 1) / KT, lo);
    count = nsink + (t1 - 1) / KT - lo + 1;
  }
  __device__ __forceinline__ int operator[](int i) const { return (i < nsink ? i : lo + i - nsink) * KT; }
  __device__ __forceinline__ int rows(int i, int n) const { return i < nsink ? n_sinks : n; }
};

// tokens of sequence b, the same for every lane of the wave
__device__ __forceinline__ int seq_len(const int* lens, int b, int T) {
  return uniform(lens ? min(max(lens[b], 0), T) : T);
}

// The token of a prompt whose last is `last` that slot j of a ring cache holds (the last of its residue
// behind the sinks), -1 if none.
__device__ __forceinline__ int ring_token(const FillArgs& a, int j, int last) {
  if (j < a.sinks) return j <= last ? j : -1;
  const int back = last >= a.sinks ? ((last - a.sinks) % a.window - (j - a.sinks) + a.window) % a.window : last + 1;
  const int p = last - back;
  return p < a.sinks ? -1 : p;
}

// Workgroups are dispatched round-robin over the 8 XCDs, each with its own L2.  Consecutive units share
// keys, so they go to one XCD, an eighth of all units each.  Where the window covers half the
// sequence or more, the units of a key head go from long to short; with few key heads an
// eighth is then all long or all short, and an XCD takes every eighth group of units instead.
// Time of every eighth group over an eighth in one, D = 128, window = T, 4 heads on 1:
//   key heads                1     2     3     4     6     8    16
//   forward  T 4,096       1.02  1.01  1.13  1.20  1.25  1.44  1.26
//            T 16,384      0.78  0.74  0.84  0.92  0.95  1.08
//   backward T 4,096       0.99  0.98  1.04  1.05  1.08  1.22  1.40
//            T 16,384      0.91  0.89  0.78  1.01  1.02  1.20
//   weights  T 4,096       0.92  0.89  0.96  1.07  1.15  1.25  1.28
//            T 16,384      0.61  0.70  0.84  0.93  0.99  1.08
// (window T / 4, T = 16,384: forward 0.96, 1.02, 0.96, 0.99, 0.98, 1.05.)  So `few` is 3 in the backward;
// 4 in the weight pass, where less is read again; in the forward 4 where more units than the chip
// holds at once (three a compute unit) leave a short eighth idle early, else 2.
__device__ __forceinline__ int xcd_unit(int total) {
  const int id = blockIdx.x, per = total / 8;
  return id < 8 * per ? (id % 8) * per + id / 8 : id;
}
__device__ __forceinline__ int xcd_unit_spread(int total, int group) {
  const int id = blockIdx.x, even = total / (8 * group) * (8 * group);
  return id < even ? ((id / 8) / group * 8 + id % 8) * group + (id / 8) % group : id;
}
__device__ __forceinline__ int attn_unit(int total, int group, int window, int T, int key_heads, int few) {
  return window >= T / 2 && key_heads <= few ? xcd_unit_spread(total, group) : xcd_unit(total);
}

// Launch with `lds` bytes of dynamic LDS (above 64 KB the limit has to be raised first).
template <size_t LDS, typename Args>
static hipError_t launch_kernel(void (*kern)(Args), dim3 grid, int threads, const Args& a, hipStream_t st) {
  if constexpr (LDS > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)LDS);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, grid, dim3(threads), LDS, st, a);
  return hipGetLastError();
}

// One token's accumulator column, d = 32 dt + acc_row(i), written to its row times f.
template <typename T, int D>
__device__ __forceinline__ void store_column(T* row, const f32x16 (&c)[D / 32], float f) {
  const int half = lane_id() >> 5;
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt)
#pragma unroll
    for (int m = 0; m < 4; ++m)
      store4(row + 32 * dt + 8 * m + 4 * half,
             f32x4{c[dt][4 * m] * f, c[dt][4 * m + 1] * f, c[dt][4 * m + 2] * f, c[dt][4 * m + 3] * f});
}

}  // namespace carve
