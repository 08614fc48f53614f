// Launch interface between the C ABI (attn_api.cpp) and the kernels of the attention
// operators whose memory per sequence is fixed.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

namespace carve {

// Sliding-window attention with sinks over whole sequences: token t of a sequence of n
// tokens sees s <= t with t - s < window or s < sinks.
struct SwaArgs {
  int B, Hq, Hkv, T, D;
  int window, sinks;          // window >= 1; sinks = 0 when the window covers the sequence
  int dtype;                  // 0 f32, 1 bf16
  float scale;
  const void* q;              // [B,Hq,T,D]
  const void* k;              // [B,Hkv,T,D]
  const void* v;              // [B,Hkv,T,D]
  const int* lens;            // [B] or null (= T)
  void* o;                    // [B,Hq,T,D]
  float* lse;                 // [B,Hq,T], may be null (forward)
  // backward
  const void* dO;
  void* dq;
  void* dk;
  void* dv;
  float* delta;               // [B,Hq,T] dO . o
  float* lse2;                // [B,Hq,T] lse in the log2 domain (+inf: no visible weight)
  // tokens far behind the window of the sink tiles: partial dk, dv of the first n_sink_tiles
  // key tiles, [B*Hkv][n_sink_tiles][1 + n_far][2][kSwaKeyTile][D] fp32
  float* part;
  int n_sink_tiles, n_far, far_len;
  // few key tiles: the heads of a group in n_head_part parts, [B*Hkv][tiles][n_head_part][2][kSwaKeyTile][D]
  float* head_part;
  int n_head_part;
};
constexpr int kSwaKeyTile = 64;        // keys of a workgroup of the dk / dv pass

// Accumulated attention weight of every key.
struct WeightArgs {
  int B, Hq, Hkv, T, D;
  int window, sinks;
  int dtype;
  float scale;
  const void* q;
  const void* k;
  const float* lse;           // [B,Hq,T]
  const int* lens;
  float* out;                 // [B,Hkv,T]
  float* part;                // [n_chunk * n_head][B*Hkv][T] (more than one)
  int n_chunk, chunk;         // query tokens of a workgroup
  int n_head;                 // parts of a group's heads
};

// One new token per sequence against a cache of C slots.
struct CacheArgs {
  int B, Hq, Hkv, D, C;
  int window, sinks, recent;
  int dtype;
  float scale;
  const void* q;              // [B,Hq,D]
  const void* k;              // [B,Hkv,D]
  const void* v;              // [B,Hkv,D]
  void* cache_k;              // [B,Hkv,C,D]
  void* cache_v;
  int bits;                   // of a code; 0: the cache holds rows of dtype
  unsigned char* k_scales;    // [B,Hkv,C,D/32], rows of codes only (cache_k, cache_v: [B,Hkv,C,D*bits/8])
  unsigned char* v_scales;
  float* cache_w;             // [B,Hkv,C]  accumulated weights (null: ring cache)
  int* cache_pos;             // [B,Hkv,C]  position of every slot, < 0 = empty
  const int* pos;             // [B] tokens before this one, < 0 = no token for this sequence
  void* o;                    // [B,Hq,D]
  int* slot;                  // [B,Hkv]
  int n_split, split_len;     // slots of a workgroup
  int waves;                  // of a workgroup, 4 or 8 (rows: bf16 and at most 16 heads a group; codes: at most 32)
  float* part;                // [B*Hkv][n_split][G][4 + D]: max, sum, two unused, sum of p v
  float* score;               // [B*Hkv][G][score_row(C)] scores (log2 domain), budget cache only;
                              // null: they stay in LDS
};
__host__ __device__ constexpr int score_row(int C) { return (C + 3) & ~3; }
constexpr int kNearScores = 4096;      // most scores of a key head that stay in LDS (bf16, one workgroup of 8 waves)

// The same for rows of codes: what a compute unit's 160 KB of LDS leave beside one workgroup of 8 waves, or two of 4.
// Such a workgroup holds two steps of 32 slots a wave (k and v; later, in the same place, its 16 heads' sums in float),
// a step's scales, 136 bytes of sums a wave, 32 heads' maxima and sums, and the token's row (1 KB for these two).
__host__ __device__ constexpr int mx_near_scores(int bits, int D, int waves) {
  const int rows = waves * 128 * (D * bits / 8), sums = waves * 64 * D;
  return ((160 << 10) / (waves == 8 ? 1 : 2) - (rows > sums ? rows : sums) - waves * (2 * D + 136) - 1024) / 16 * 4;
}

// Rows of k and v copied into a cache.
struct FillArgs {
  int B, Hkv, T, D, C;
  int window, sinks, recent;
  int dtype;
  const void* k;              // [B,Hkv,T,D]
  const void* v;
  const float* weights;       // [B,Hkv,T]
  const int* lens;
  void* cache_k;
  void* cache_v;
  int bits;                   // as in CacheArgs
  unsigned char* k_scales;
  unsigned char* v_scales;
  float* cache_w;             // null: ring cache
  int* cache_pos;
};

// Rows written in codes and scales, and read back.
struct MxRowArgs {
  size_t pieces;              // of eight values
  int dtype, bits;
  void* x;                    // written by the read back
  void* codes;
  void* scales;
};

hipError_t launch_swa_fwd(const SwaArgs& a, hipStream_t st);
hipError_t launch_swa_bwd(const SwaArgs& a, hipStream_t st);
hipError_t launch_weights(const WeightArgs& a, hipStream_t st);
hipError_t launch_cache_decode(const CacheArgs& a, hipStream_t st);
hipError_t launch_keep_select(const FillArgs& a, hipStream_t st);
hipError_t launch_fill_rows(const FillArgs& a, hipStream_t st);
hipError_t launch_mx_quant(const MxRowArgs& a, hipStream_t st);
hipError_t launch_mx_dequant(const MxRowArgs& a, hipStream_t st);
hipError_t launch_mx_fill(const FillArgs& a, hipStream_t st);
hipError_t launch_mx_decode(const CacheArgs& a, hipStream_t st);

}  // namespace carve
