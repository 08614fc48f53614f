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

// lanes below this one whose bit is set
__device__ __forceinline__ int bits_below(unsigned long long b) {
  return __builtin_amdgcn_mbcnt_hi((unsigned)(b >> 32), __builtin_amdgcn_mbcnt_lo((unsigned)b, 0));
}

// Positions kept of one (sequence, key head): a workgroup of 16 waves.  Tokens 0 .. lo - 1 and
// hi .. n - 1 stay; of lo .. hi - 1 the m heaviest, the lowest positions of equal weights.  The
// m-th largest weight is found by digits of its ordered bits (11, 11, 10) with a histogram each;
// then every wave counts what stays of its stretch of tokens, and writes it behind the waves
// before it.  A wave's stretch is kept in registers as ordered bits, VPT a lane (VPT = 0: sequences
// past 64 x 1024 tokens, read again in every pass).  The one compute unit's instruction rate
// bounds it, so tokens that are not candidates carry the key 0, below every weight's, and are told
// apart by nothing else.  32 key heads of 32,768 tokens: 17 us (55 us with the weights read again in
// every pass and a scan across the workgroup for every 1,024 of them).  Of it the loads take 2.8 us,
// the digits 3.7, 1.8 and 1.8, the counts 1.4, the positions 3.1.
template <int VPT>
__global__ __launch_bounds__(kSelThreads) void keep_select_kernel(FillArgs a) {
  constexpr int NW = kSelThreads / 64;
  // the first digit's histogram in four copies, a quarter of the lanes each: weights crowd into few
  // bins, and lanes that add to one address take turns (one copy 1.3 us more, eight 0.6 us more to
  // clear and add up); the later digits are of few weights
  __shared__ __align__(16) int hist[4 * 2048];
  __shared__ int red[NW];
  __shared__ int count[NW][2];
  __shared__ unsigned found[3];
  const int bk = blockIdx.x, tid = threadIdx.x, lane = lane_id(), wave = wave_uid();
  const int n = seq_len(a.lens, bk / a.Hkv, a.T);
  const float* w = a.weights + (size_t)bk * a.T;
  int* cp = a.cache_pos + (size_t)bk * a.C;
  const int lo = min(a.sinks, n), hi = max(lo, n - a.recent);
  const int cand = hi - lo, m = min(cand, a.C - (lo + n - hi));
  const int steps = (n + kSelThreads - 1) / kSelThreads;         // of 64 tokens a wave
  const int j_wave = wave * steps * 64 + lane;                   // token of step i: + 64 i
  auto key_of = [&](int j, float v) { return j >= lo && j < hi ? heavy_order(v) : 0u; };
  unsigned x[VPT > 0 ? VPT : 1];
  if constexpr (VPT > 0) {
    // loads without branches, all in flight together; past the last token they give zero
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(w), 0, n * 4, 0x00020000);
    unsigned v[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      v[i] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, j_wave * 4 + (i % 16) * 256, (i / 16) * 4096, 0);
    const int j0 = wave * steps * 64;
    if (steps == VPT && j0 >= lo && j0 + 64 * VPT <= hi) {       // candidates alone
#pragma unroll
      for (int i = 0; i < VPT; ++i) x[i] = heavy_order(__builtin_bit_cast(float, v[i]));
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) x[i] = i < steps ? key_of(j_wave + 64 * i, __builtin_bit_cast(float, v[i])) : 0u;
    }
  }
  // fn(token, key) over the wave's tokens, in order
  auto each = [&](auto&& fn) {
    if constexpr (VPT > 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) fn(j_wave + 64 * i, x[i]);
    } else {
      for (int i = 0; i < steps; ++i) {
        const int j = j_wave + 64 * i;
        fn(j, key_of(j, w[min(j, n - 1)]));
      }
    }
  };
  // the threshold: keys above it stay; of those equal to it the first `need`, and if that is all of
  // them it is lowered by one step, so that nothing more asks for equal keys
  unsigned limit = m == cand ? 0u : 0xffffffffu;
  int need = 0;
  if (m < cand && m > 0) {
    unsigned prefix = 0;
    int same = 0;
    need = m;
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    // The digit of `BITS` bits above the lowest SHIFT of the keys that agree with prefix above it.
    // Keys 0 share no first digit with a candidate (-inf, the lowest, has the key 0x007fffff).
    auto digit = [&](auto shift_c, auto bits_c, auto copies_c) {
      constexpr int SHIFT = decltype(shift_c)::value, BITS = decltype(bits_c)::value, bins = 1 << BITS;
      constexpr int COPIES = decltype(copies_c)::value;
      for (int i = tid; i < bins * COPIES / 4; i += kSelThreads) reinterpret_cast<i32x4*>(hist)[i] = i32x4{0, 0, 0, 0};
      __syncthreads();
      each([&](int, unsigned key) {
        const unsigned rest = key ^ prefix;
        if (SHIFT + BITS == 32 ? key != 0u : rest < 1u << ((SHIFT + BITS) & 31))
          atomicAdd(&hist[(rest >> SHIFT) * COPIES + lane % COPIES], 1);
      });
      __syncthreads();
      // bins from the top: thread t has two, the upper one first
      int h1 = 0, h0 = 0;
      const int b1 = bins - 1 - 2 * tid;
      if (b1 > 0) {
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          h0 += hist[(b1 - 1) * COPIES + i];
          h1 += hist[b1 * COPIES + i];
        }
      }
      int total;
      const int upto = block_scan(h1 + h0, red, total), above = upto - h1 - h0;
      if (above < need && need <= upto) {
        const bool top = need <= above + h1;
        found[0] = (unsigned)(top ? b1 : b1 - 1);
        found[1] = (unsigned)(need - (top ? above : above + h1));
        found[2] = (unsigned)(top ? h1 : h0);
      }
      __syncthreads();
      prefix |= uniform(found[0]) << SHIFT;
      need = uniform((int)found[1]);
      same = uniform((int)found[2]);
    };
    digit(std::integral_constant<int, 21>{}, std::integral_constant<int, 11>{}, std::integral_constant<int, 4>{});
    digit(std::integral_constant<int, 10>{}, std::integral_constant<int, 11>{}, std::integral_constant<int, 1>{});
    digit(std::integral_constant<int, 0>{}, std::integral_constant<int, 10>{}, std::integral_constant<int, 1>{});
    limit = prefix;
    if (need == same) {
      limit = prefix - 1;
      need = 0;
    }
  }
  int kept = 0, ties = 0;
  each([&](int, unsigned key) { kept += __popcll(__ballot(key > limit)); });
  if (need > 0) each([&](int, unsigned key) { ties += __popcll(__ballot(key == limit)); });
  if (lane == 0) {
    count[wave][0] = kept;
    count[wave][1] = ties;
  }
  __syncthreads();
  int base = lo, tied = 0, end = lo + need;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    base += i < wave ? count[i][0] : 0;
    tied += i < wave ? count[i][1] : 0;
    end += count[i][0];
  }
  base = uniform(base);
  tied = uniform(tied);
  if (need == 0) {
    each([&](int j, unsigned key) {
      const unsigned long long keeps = __ballot(key > limit);
      if (key > limit) cp[base + bits_below(keeps)] = j;
      base += __popcll(keeps);
    });
  } else if (kept + ties > 0) {
    each([&](int j, unsigned key) {
      const unsigned long long keeps = __ballot(key > limit), equal = __ballot(key == limit);
      const int t = tied + bits_below(equal);                    // equal weights before this one
      if (key > limit || (key == limit && t < need)) cp[base + bits_below(keeps) + min(t, need)] = j;
      base += __popcll(keeps);
      tied += __popcll(equal);
    });
  }
  // the first and the recent tokens, and the empty slots
  for (int j = tid; j < lo; j += kSelThreads) cp[j] = j;
  for (int j = hi + tid; j < n; j += kSelThreads) cp[end + j - hi] = j;
  for (int j = end + n - hi + tid; j < a.C; j += kSelThreads) cp[j] = -1;
}

// Copies the kept rows, 16 bytes a thread, and their weights: 32 key heads x 4,096 rows in 23 us, 5.8
// TB/s.  A slot of the ring holds the last token of its residue (128 key heads x 4,100 slots of
// sequences of 8,192 tokens in 99 us, 5.4 TB/s); the row of a slot that holds no token is left as it was.
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
      if (i % ROW16 == 0) a.cache_w[row] = p < 0 ? 0.f : a.weights[bk * a.T + p];
    } else {
      const int last = (a.lens ? min(max(a.lens[bk / a.Hkv], 0), a.T) : a.T) - 1;   // (lanes of several rows)
      p = ring_token(a, j, last);
    }
    if (p < 0) continue;
    const size_t src = (bk * a.T + p) * ROW16 + i % ROW16;
    const f32x4 x = reinterpret_cast<const f32x4*>(a.k)[src], y = reinterpret_cast<const f32x4*>(a.v)[src];
    reinterpret_cast<f32x4*>(a.cache_k)[i] = x;
    reinterpret_cast<f32x4*>(a.cache_v)[i] = y;
  }
}

// Weights stay in registers as far as they go, 64 a lane (of its 128 registers 32 spill there); longer
// prompts read them again for every digit and count.  Both launches of a cache, 32 key heads and 64
// slots: 32,768 tokens 18 us; 65,536 tokens 30 us in registers and 70 read again.  With 4,096 slots at
// D = 64: 27, 41 and 90 us; 131,072 tokens 161 us and 262,144 tokens 330 us, read again.
hipError_t launch_keep_select(const FillArgs& a, hipStream_t st) {
  const dim3 grid(a.B * a.Hkv);
  if (a.T <= 4 * kSelThreads) return launch_kernel<0>(keep_select_kernel<4>, grid, kSelThreads, a, st);
  if (a.T <= 12 * kSelThreads) return launch_kernel<0>(keep_select_kernel<12>, grid, kSelThreads, a, st);
  if (a.T <= 32 * kSelThreads) return launch_kernel<0>(keep_select_kernel<32>, grid, kSelThreads, a, st);
  if (a.T <= 64 * kSelThreads) return launch_kernel<0>(keep_select_kernel<64>, grid, kSelThreads, a, st);
  return launch_kernel<0>(keep_select_kernel<0>, grid, kSelThreads, a, st);
}

template <int ROW16>
static hipError_t fill_rows(const FillArgs& a, hipStream_t st) {
  const size_t total = (size_t)a.B * a.Hkv * a.C * ROW16;
  const unsigned grid = (unsigned)std::min<size_t>((total + 255) / 256, 1u << 14);
  return a.cache_w ? launch_kernel<0>(fill_rows_kernel<ROW16, true>, dim3(grid), 256, a, st)
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
