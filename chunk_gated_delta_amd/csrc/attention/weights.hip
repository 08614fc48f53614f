// Attention weight that every key receives: w_s = sum over the tokens that see s and the query
// heads that share its key head of p_ts = exp(scale q_t . k_s - lse_t).
//
// Workgroup = 128 keys of one key head (32 a wave, a lane owns one key, k in registers) and a
// range of tokens; S = Q K^T puts the keys on the columns, so a key's weights are added up
// in its lane.  The sums of the token ranges are added in order by weight_sum_kernel.
#include "attn_device.h"

namespace carve {

constexpr int kWtK = 128, kWtQ = 32;

template <typename T, int D>
__global__ __launch_bounds__(256) void weight_kernel(WeightArgs a) {
  using St = RowStage<T, kWtQ, D, 256>;
  constexpr int LD = St::LD;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Qs = reinterpret_cast<T*>(smem);
  float* Ls = reinterpret_cast<float*>(Qs + kWtQ * LD);
  const int G = a.Hq / a.Hkv, NK = (a.T + kWtK - 1) / kWtK;
  const int unit = xcd_unit(a.B * a.Hkv * NK * a.n_chunk);
  const int kt = unit % NK, ch = (unit / NK) % a.n_chunk, bk = unit / (NK * a.n_chunk);
  const int b = bk / a.Hkv;
  const int n = seq_len(a.lens, b, a.T);
  const int lane = lane_id(), wave = wave_id(), half = lane >> 5;
  const int s0 = kt * kWtK, sw = s0 + 32 * wave, s = sw + (lane & 31);
  const int t_lo = max(ch * a.chunk, s0) / kWtQ * kWtQ;
  int t_hi = (int)min((long long)n, (long long)(ch + 1) * a.chunk);
  // behind the window of the tile only sinks are seen
  if (s0 >= a.sinks) t_hi = (int)min((long long)t_hi, (long long)s0 + kWtK - 1 + a.window);
  float sum = 0.f;
  if (t_lo < t_hi) {
    Frag<T> K[D / 16];
    const size_t at = ((size_t)bk * a.T + min(s, n - 1)) * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) K[kk] = load_frag(reinterpret_cast<const T*>(a.k) + at + 16 * kk);
    const float c = a.scale * kLog2e;
    const int nt = (t_hi - t_lo + kWtQ - 1) / kWtQ, total = nt * G;
    St qst;
    float lst = 0.f;
    auto load = [&](int i) {
      const int hq = (bk % a.Hkv) * G + i / nt, tt = t_lo + (i % nt) * kWtQ;
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
  sum += __shfl_xor(sum, 32);
  if (half == 0 && s < a.T) {
    float* dst = a.n_chunk > 1 ? a.part + ((size_t)ch * a.B * a.Hkv + bk) * a.T : a.out + (size_t)bk * a.T;
    dst[s] = s < n ? sum : 0.f;
  }
}

__global__ __launch_bounds__(256) void weight_sum_kernel(WeightArgs a) {
  const size_t N = (size_t)a.B * a.Hkv * a.T;
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= N) return;
  float x = 0.f;
  for (int c = 0; c < a.n_chunk; ++c) x += a.part[c * N + i];
  a.out[i] = x;
}

template <typename T, int D>
static hipError_t launch(const WeightArgs& a, hipStream_t st) {
  constexpr size_t lds = sizeof(T) * kWtQ * RowStage<T, kWtQ, D, 256>::LD + sizeof(float) * kWtQ;
  const int NK = (a.T + kWtK - 1) / kWtK;
  hipError_t e = launch_kernel<lds>(weight_kernel<T, D>, dim3(a.B * a.Hkv * NK * a.n_chunk), 256, a, st);
  if (e != hipSuccess || a.n_chunk == 1) return e;
  const size_t N = (size_t)a.B * a.Hkv * a.T;
  return launch_kernel<0>(weight_sum_kernel, dim3((unsigned)((N + 255) / 256)), 256, a, st);
}

hipError_t launch_weights(const WeightArgs& a, hipStream_t st) {
  if (a.dtype) return a.D == 128 ? launch<bf16, 128>(a, st) : launch<bf16, 64>(a, st);
  return a.D == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
}

}  // namespace carve
