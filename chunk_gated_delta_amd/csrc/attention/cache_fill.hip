// Caches made from a prompt: the ring cache of windowed attention, and the cache of C slots that
// keeps the first tokens, the recent ones and the heaviest of the others.
#include <algorithm>

#include "attn_device.h"

namespace carve {

constexpr int kSelThreads = 1024;

__device__ __forceinline__ unsigned heavy_order(float w) {
  const unsigned u = __builtin_bit_cast(unsigned, w + 0.f);
  return w != w ? 0xffffffffu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Inclusive sum over the workgroup's threads (red: one int per wave), and the total.
__device__ __forceinline__ int block_scan(int x, int* red, int& total) {
  const int lane = lane_id(), wave = wave_id();
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 63) red[wave] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 64; ++w) {
    before += w < wave ? red[w] : 0;
    total += red[w];
  }
  return x + before;
}

// Positions kept of one (sequence, key head): a workgroup.  Tokens 0 .. lo - 1 and hi .. n - 1
// stay; of lo .. hi - 1 the m heaviest, the lowest positions of equal weights.  The m-th largest
// weight is found by digits of its ordered bits (11, 11, 10) with a histogram each, then
// the positions are written in order by a running count.
__global__ __launch_bounds__(kSelThreads) void keep_select_kernel(FillArgs a) {
  __shared__ int hist[2048];
  __shared__ int red[kSelThreads / 64];
  __shared__ unsigned found[2];
  const int bk = blockIdx.x, tid = threadIdx.x;
  const int n = seq_len(a.lens, bk / a.Hkv, a.T);
  const float* w = a.weights + (size_t)bk * a.T;
  float* cw = a.cache_w + (size_t)bk * a.C;
  int* cp = a.cache_pos + (size_t)bk * a.C;
  const int lo = min(a.sinks, n), hi = max(lo, n - a.recent);
  const int cand = hi - lo, m = min(cand, a.C - (lo + n - hi));
  unsigned prefix = 0, mask = 0;
  int need = m;                            // of the weights equal to the digits so far
  if (m < cand && m > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      hist[tid] = 0;
      hist[tid + 1024] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kSelThreads) {
        const unsigned key = heavy_order(w[j]);
        if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
      }
      __syncthreads();
      // bins from the top: thread t has bins - 1 - 2 t and the one below
      const int b1 = bins - 1 - 2 * tid, h1 = b1 >= 0 ? hist[b1] : 0, h0 = b1 >= 1 ? hist[b1 - 1] : 0;
      int total;
      const int upto = block_scan(h1 + h0, red, total), above = upto - h1 - h0;
      if (above < need && need <= upto) {
        const bool top = need <= above + h1;
        found[0] = (unsigned)(top ? b1 : b1 - 1);
        found[1] = (unsigned)(need - (top ? above : above + h1));
      }
      __syncthreads();
      prefix |= found[0] << shift;
      mask |= (unsigned)(bins - 1) << shift;
      need = (int)found[1];
      __syncthreads();
    }
  }
  // need = how many weights equal to the threshold `prefix` stay
  int kept = 0, ties = 0;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + tid;
    bool keep = false, tie = false;
    float x = 0.f;
    if (j < n) {
      x = w[j];
      if (j < lo || j >= hi || m == cand) {
        keep = true;
      } else if (m > 0) {
        const unsigned key = heavy_order(x);
        keep = key > prefix;
        tie = key == prefix;
      }
    }
    int total;
    const int sum = block_scan((keep ? 1 : 0) | (tie ? 1 << 16 : 0), red, total);
    const int tied = ties + (sum >> 16);                        // ties up to and with this token
    const int at = kept + (sum & 0xffff) + min(tied, need) - 1;
    if ((keep || (tie && tied <= need)) && at < a.C) {
      cp[at] = j;
      cw[at] = x;
    }
    kept += total & 0xffff;
    ties += total >> 16;
  }
  const int end = m == cand ? kept : kept + min(ties, need);
  for (int j = end + tid; j < a.C; j += kSelThreads) {
    cp[j] = -1;
    cw[j] = 0.f;
  }
}

// Copies the kept rows: 16 bytes a thread.  A slot of the ring holds the last token of its
// residue; a slot that holds no token is left as it was.
template <int ROW16, bool BUDGET>
__global__ __launch_bounds__(256) void fill_rows_kernel(FillArgs a) {
  const size_t rows = (size_t)a.B * a.Hkv * a.C, total = rows * ROW16;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
    const size_t row = i / ROW16;
    const int j = (int)(row % a.C);
    const size_t bk = row / a.C;
    int p;
    if (BUDGET) {
      p = a.cache_pos[row];
    } else {
      const int last = (a.lens ? min(max(a.lens[bk / a.Hkv], 0), a.T) : a.T) - 1;   // (lanes of several rows)
      if (j < a.sinks) {
        p = j <= last ? j : -1;
      } else {
        const int back = last >= a.sinks ? ((last - a.sinks) % a.window - (j - a.sinks) + a.window) % a.window : last + 1;
        p = last - back;
        if (p < a.sinks) p = -1;
      }
    }
    if (p < 0) continue;
    const size_t src = (bk * a.T + p) * ROW16 + i % ROW16;
    const f32x4 x = reinterpret_cast<const f32x4*>(a.k)[src], y = reinterpret_cast<const f32x4*>(a.v)[src];
    reinterpret_cast<f32x4*>(a.cache_k)[i] = x;
    reinterpret_cast<f32x4*>(a.cache_v)[i] = y;
  }
}

hipError_t launch_keep_select(const FillArgs& a, hipStream_t st) {
  return launch_kernel<0>(keep_select_kernel, dim3(a.B * a.Hkv), kSelThreads, a, st);
}

template <int ROW16>
static hipError_t fill_rows(const FillArgs& a, hipStream_t st) {
  const size_t total = (size_t)a.B * a.Hkv * a.C * ROW16;
  const unsigned grid = (unsigned)std::min<size_t>((total + 255) / 256, 1u << 14);
  return a.weights ? launch_kernel<0>(fill_rows_kernel<ROW16, true>, dim3(grid), 256, a, st)
                   : launch_kernel<0>(fill_rows_kernel<ROW16, false>, dim3(grid), 256, a, st);
}
hipError_t launch_fill_rows(const FillArgs& a, hipStream_t st) {
  switch (a.D * (a.dtype ? 2 : 4) / 16) {
    case 8: return fill_rows<8>(a, st);
    case 16: return fill_rows<16>(a, st);
    default: return fill_rows<32>(a, st);
  }
}

}  // namespace carve
