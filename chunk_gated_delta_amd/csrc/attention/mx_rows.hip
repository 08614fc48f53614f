// Rows written in codes and scales and read back, and the caches of a prompt written that way.
//
// A lane holds eight values, a quarter of a block, so a block's largest value needs two exchanges
// between neighbouring lanes; loads are 16 bytes a lane (bf16), stores of codes 4 or 8, and lanes of one
// instruction touch neighbouring bytes.  Bound by the bytes moved.  Plain rows are read and written once, by
// loads and stores marked so; codes, which the next kernel reads, keep their places in the caches:
// 67 M values to 8 bits and back 63 us (73 after other work has filled the caches; unmarked 69 and 98), the
// ring of 32 sequences of 8,192 tokens, 4 key heads, window 4,096, 4 bits, written and read back 110 us
// (122; unmarked 136 and 160; codes marked too 120 and 129).  Both move 400 and 680 MB, at 5.9 TB/s, a copy's rate, in 69
// and 115 us: part of the codes is read back from the last-level cache.
#include <algorithm>

#include "mx_device.h"

namespace carve {

constexpr int kRowThreads = 256, kRowUnroll = 4;

// Eight values that are read, or written, once.  (float32: unmarked, since a lane's 32 bytes are two accesses to one
// line: 67 M values to 4 bits and back 130 us, marked 165.)
__device__ __forceinline__ Frag<bf16> load_once(const bf16* p) {
  Frag<bf16> f;
  f.v = __builtin_nontemporal_load(reinterpret_cast<const bf16x8*>(p));
  return f;
}
__device__ __forceinline__ Frag<float> load_once(const float* p) { return load_frag(p); }
__device__ __forceinline__ void store_once(bf16* p, const Frag<bf16>& f) {
  __builtin_nontemporal_store(f.v, reinterpret_cast<bf16x8*>(p));
}
__device__ __forceinline__ void store_once(float* p, f32x4 lo, f32x4 hi) {
  *reinterpret_cast<f32x4*>(p) = lo;
  *reinterpret_cast<f32x4*>(p + 4) = hi;
}

// Pieces of eight values; a thread takes kRowUnroll of them, a workgroup's width apart, all loads first.
template <typename T, int BITS>
__global__ __launch_bounds__(kRowThreads) void mx_quant_kernel(MxRowArgs a) {
  const T* x = reinterpret_cast<const T*>(a.x);
  for (size_t p0 = (size_t)blockIdx.x * kRowUnroll * kRowThreads + threadIdx.x; p0 < a.pieces;
       p0 += (size_t)gridDim.x * kRowUnroll * kRowThreads) {
    Frag<T> f[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const size_t p = p0 + u * kRowThreads;
      f[u] = p < a.pieces ? load_once(x + 8 * p) : zero_frag(T());
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const size_t p = p0 + u * kRowThreads;
      u32 scale;
      const Eight<BITS> c = write_block<BITS>(f[u], scale);
      if (p < a.pieces) {
        reinterpret_cast<Eight<BITS>*>(a.codes)[p] = c;
        if ((p & 3) == 0) reinterpret_cast<unsigned char*>(a.scales)[p >> 2] = (unsigned char)scale;
      }
    }
  }
}

__device__ __forceinline__ void store_eight(bf16* x, const Eight<4>& c, float s) {
  store_once(x, read_eight<4>(c, s));
}
__device__ __forceinline__ void store_eight(bf16* x, const Eight<8>& c, float s) {
  store_once(x, read_eight<8>(c, s));
}
__device__ __forceinline__ void store_eight(float* x, const Eight<4>& c, float s) {
  const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.w, s, 0), q = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.w, s, 1);
  const f32x2 r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.w, s, 2), t = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c.w, s, 3);
  store_once(x, f32x4{p[0], p[1], q[0], q[1]}, f32x4{r[0], r[1], t[0], t[1]});
}
__device__ __forceinline__ void store_eight(float* x, const Eight<8>& c, float s) {
  f32x4 y[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.w[h], s, false), q = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c.w[h], s, true);
    y[h] = f32x4{p[0], p[1], q[0], q[1]};
  }
  store_once(x, y[0], y[1]);
}
template <typename T, int BITS>
__global__ __launch_bounds__(kRowThreads) void mx_dequant_kernel(MxRowArgs a) {
  T* x = reinterpret_cast<T*>(a.x);
  for (size_t p0 = (size_t)blockIdx.x * kRowUnroll * kRowThreads + threadIdx.x; p0 < a.pieces;
       p0 += (size_t)gridDim.x * kRowUnroll * kRowThreads) {
    Eight<BITS> c[kRowUnroll];
    u32 s[kRowUnroll];
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const size_t p = std::min(p0 + u * kRowThreads, a.pieces - 1);
      c[u] = reinterpret_cast<const Eight<BITS>*>(a.codes)[p];
      s[u] = reinterpret_cast<const unsigned char*>(a.scales)[p >> 2];
    }
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const size_t p = p0 + u * kRowThreads;
      if (p < a.pieces) store_eight(x + 8 * p, c[u], scale_value(s[u]));
    }
  }
}

// The cache of a prompt: blockIdx.y is the key head, a thread takes a piece of eight values of k and of v of one
// slot (two or four slots a thread: 136, 139 us of the 131 then).  Which token a slot holds as in
// fill_rows_kernel; rows of slots that hold none stay as they were.
template <typename T, int BITS, int D, bool BUDGET>
__global__ __launch_bounds__(kRowThreads) void mx_fill_kernel(FillArgs a) {
  constexpr int PR = D / 8, ROWS = kRowThreads / PR;       // pieces of a row, rows of a workgroup
  const size_t bk = blockIdx.y;
  const int piece = threadIdx.x % PR, last = seq_len(a.lens, (int)(bk / a.Hkv), a.T) - 1;
  for (long long j = (long long)blockIdx.x * ROWS + threadIdx.x / PR; j < a.C; j += (long long)gridDim.x * ROWS) {
    const size_t row = bk * a.C + j, at = row * PR + piece;      // (whole rows of lanes, whole blocks)
    const int p = BUDGET ? a.cache_pos[row] : ring_token(a, (int)j, last);
    if (BUDGET && piece == 0) a.cache_w[row] = p < 0 ? 0.f : a.weights[bk * a.T + p];
    if (p < 0) continue;
    const size_t src = (bk * a.T + p) * D + 8 * piece;
    const Frag<T> k = load_once(reinterpret_cast<const T*>(a.k) + src), v = load_once(reinterpret_cast<const T*>(a.v) + src);
    u32 ks, vs;
    reinterpret_cast<Eight<BITS>*>(a.cache_k)[at] = write_block<BITS>(k, ks);
    reinterpret_cast<Eight<BITS>*>(a.cache_v)[at] = write_block<BITS>(v, vs);
    if ((piece & 3) == 0) {
      reinterpret_cast<unsigned char*>(a.k_scales)[at >> 2] = (unsigned char)ks;
      reinterpret_cast<unsigned char*>(a.v_scales)[at >> 2] = (unsigned char)vs;
    }
  }
}

template <bool QUANT, int BITS>
static hipError_t launch_rows(const MxRowArgs& a, hipStream_t st) {
  const size_t per = kRowUnroll * kRowThreads;
  const dim3 grid((unsigned)std::min<size_t>((a.pieces + per - 1) / per, 1u << 16));
  if (QUANT)
    return a.dtype ? launch_kernel<0>(mx_quant_kernel<bf16, BITS>, grid, kRowThreads, a, st)
                   : launch_kernel<0>(mx_quant_kernel<float, BITS>, grid, kRowThreads, a, st);
  return a.dtype ? launch_kernel<0>(mx_dequant_kernel<bf16, BITS>, grid, kRowThreads, a, st)
                 : launch_kernel<0>(mx_dequant_kernel<float, BITS>, grid, kRowThreads, a, st);
}
hipError_t launch_mx_quant(const MxRowArgs& a, hipStream_t st) {
  return a.bits == 4 ? launch_rows<true, 4>(a, st) : launch_rows<true, 8>(a, st);
}
hipError_t launch_mx_dequant(const MxRowArgs& a, hipStream_t st) {
  return a.bits == 4 ? launch_rows<false, 4>(a, st) : launch_rows<false, 8>(a, st);
}

template <typename T, int BITS, int D>
static hipError_t launch_fill(const FillArgs& a, hipStream_t st) {
  constexpr int rows = kRowThreads / (D / 8);
  const dim3 grid(std::min((a.C + rows - 1) / rows, 1 << 16), a.B * a.Hkv);
  return a.cache_w ? launch_kernel<0>(mx_fill_kernel<T, BITS, D, true>, grid, kRowThreads, a, st)
                   : launch_kernel<0>(mx_fill_kernel<T, BITS, D, false>, grid, kRowThreads, a, st);
}
template <typename T, int BITS>
static hipError_t launch_fill_d(const FillArgs& a, hipStream_t st) {
  return a.D == 128 ? launch_fill<T, BITS, 128>(a, st) : launch_fill<T, BITS, 64>(a, st);
}
hipError_t launch_mx_fill(const FillArgs& a, hipStream_t st) {
  if (a.bits == 4) return a.dtype ? launch_fill_d<bf16, 4>(a, st) : launch_fill_d<float, 4>(a, st);
  return a.dtype ? launch_fill_d<bf16, 8>(a, st) : launch_fill_d<float, 8>(a, st);
}

}  // namespace carve
