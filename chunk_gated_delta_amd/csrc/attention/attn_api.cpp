// C ABI of the attention operators whose memory per sequence is fixed: argument checks,
// workspace sizing and dispatch.  Checks run on the host before any launch.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <initializer_list>

#include <hip/hip_runtime.h>

#include "../../../include/carve.h"
#include "attn_internal.h"

namespace {

constexpr int kMaxTokens = 1 << 30;
constexpr int kMaxGroup = 64;             // query heads of one key head (decode: four tiles of 16)
constexpr long long kMaxUnits = 1ll << 30;   // workgroups of a launch

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool all_given(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!p) return false;
  return true;
}
bool all_aligned(std::initializer_list<const void*> ptrs, unsigned n) {
  for (const void* p : ptrs)
    if (p && !aligned(p, n)) return false;
  return true;
}
carve_status hip_status(hipError_t e) { return e == hipSuccess ? CARVE_OK : CARVE_ERR_HIP; }
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

carve_status check_heads(int B, int Hq, int Hkv, int T, int D, carve_dtype dtype, float scale) {
  if (B < 0 || Hq < 0 || Hkv < 0 || T < 0) return CARVE_ERR_INVALID_ARG;
  if (dtype != CARVE_F32 && dtype != CARVE_BF16) return CARVE_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return CARVE_ERR_INVALID_ARG;
  if ((Hkv == 0) != (Hq == 0) || (Hkv > 0 && Hq % Hkv != 0)) return CARVE_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return CARVE_ERR_UNSUPPORTED;
  if ((long long)B * Hq > 65535 || T > kMaxTokens) return CARVE_ERR_UNSUPPORTED;
  return CARVE_OK;
}
carve_status check_swa(const carve_swa_shape* s) {
  if (!s) return CARVE_ERR_INVALID_ARG;
  if (s->window < 1 || s->sinks < 0) return CARVE_ERR_INVALID_ARG;
  const carve_status st = check_heads(s->B, s->Hq, s->Hkv, s->T, s->D, s->dtype, s->scale);
  if (st != CARVE_OK) return st;
  if ((long long)s->window + s->sinks > kMaxTokens) return CARVE_ERR_UNSUPPORTED;
  return CARVE_OK;
}
bool empty(const carve_swa_shape* s) { return s->B == 0 || s->Hq == 0 || s->T == 0; }

// The same mask with the window cut to the sequence, and no sinks where the window (or the
// sinks themselves) let every token see all before it.
void mask_of(const carve_swa_shape* s, int* window, int* sinks) {
  const bool whole = s->window >= s->T || s->sinks >= s->T;
  *window = whole ? std::max(s->T, 1) : s->window;
  *sinks = whole ? 0 : s->sinks;
}

// Parts of a group's heads, at most `most` and none without heads.
int head_parts(const carve_swa_shape* s, long long most) {
  const int G = s->Hq / s->Hkv, n = (int)std::max(1ll, std::min<long long>(G, most));
  return ceil_div(G, ceil_div(G, n));
}

// Backward: ranges of the tokens behind the window of the first key tile, so that a tile with
// sinks is not one workgroup's walk over the whole sequence; at most about 64 (tile, range)
// pairs a key head, of 256 tokens or more (64 in fp32): short, so that they fill the gaps of the
// last round.  While key tiles are fewer than the 256 compute units, the heads that share a key
// head are also taken apart.
struct SwaPlan {
  int window, sinks, n_sink_tiles, n_far, far_len, n_head_part;
  size_t delta_bytes, part_bytes, head_bytes;
  size_t bytes() const { return 2 * delta_bytes + part_bytes + head_bytes + 256; }
};
SwaPlan swa_plan(const carve_swa_shape* s) {
  SwaPlan p;
  mask_of(s, &p.window, &p.sinks);
  p.n_sink_tiles = p.n_far = p.far_len = 0;
  const long long far = (long long)s->T - (carve::kSwaKeyTile - 1 + (long long)p.window);
  if (p.sinks > 0 && far > 0) {
    p.n_sink_tiles = ceil_div(p.sinks, carve::kSwaKeyTile);
    const int most = std::max(1, 64 / p.n_sink_tiles);
    const int want = std::min(most, ceil_div(far, s->dtype == CARVE_F32 ? 64 : 256));
    p.far_len = ceil_div(ceil_div(far, want), 32) * 32;
    p.n_far = ceil_div(far, p.far_len);
  }
  p.delta_bytes = up256((size_t)s->B * s->Hq * s->T * sizeof(float));
  const size_t one = 2 * carve::kSwaKeyTile * s->D * sizeof(float);
  p.part_bytes = up256((size_t)s->B * s->Hkv * p.n_sink_tiles * (p.n_far ? 1 + p.n_far : 0) * one);
  const long long tiles = (long long)s->B * s->Hkv * ceil_div(s->T, carve::kSwaKeyTile);
  p.n_head_part = head_parts(s, 256 / tiles);
  p.head_bytes = p.n_head_part > 1 ? (size_t)tiles * p.n_head_part * one : 0;
  return p;
}

carve::SwaArgs swa_args(const carve_swa_shape* s, const void* q, const void* k, const void* v, const int* lens) {
  carve::SwaArgs a;
  memset(&a, 0, sizeof(a));
  a.B = s->B;
  a.Hq = s->Hq;
  a.Hkv = s->Hkv;
  a.T = s->T;
  a.D = s->D;
  mask_of(s, &a.window, &a.sinks);
  a.dtype = s->dtype == CARVE_BF16;
  a.scale = s->scale;
  a.q = q;
  a.k = k;
  a.v = v;
  a.lens = lens;
  return a;
}

// Token ranges of the weight pass: enough workgroups to fill the chip several times over (the
// later keys are seen by few tokens, so the ranges are uneven), of at least 128 tokens.  In fp32,
// whose products take sixteen times as long, ranges from 64 tokens and, up to four workgroups a
// compute unit, the heads of a group apart (4 rows of 11 tokens, 32 heads on 4: 28 -> 13 us, where
// the sum's launch costs 3; in bf16 it would cost more than it gives), into no more than 48 parts
// with the ranges (one row of 1,999 tokens, 3 heads on 1: 26 us of 32 parts, 29 of 64).
struct WeightPlan {
  int n_chunk, chunk, n_head;
};
WeightPlan weight_plan(const carve_swa_shape* s) {
  const bool f32 = s->dtype == CARVE_F32;
  const long long units = (long long)s->B * s->Hkv * ceil_div(s->T, 128);
  const int want = (int)std::max(1ll, std::min<long long>(4096 / std::max(1ll, units), ceil_div(s->T, f32 ? 64 : 128)));
  WeightPlan p;
  p.chunk = ceil_div(ceil_div(s->T, want), 32) * 32;
  p.n_chunk = ceil_div(s->T, p.chunk);
  p.n_head = f32 ? head_parts(s, std::min(1024 / (units * p.n_chunk), 48ll / p.n_chunk)) : 1;
  return p;
}

int row_bytes(int D, carve_dtype dtype) { return D * (dtype == CARVE_BF16 ? 2 : 4); }

// Slot ranges of a decode call and waves of a workgroup.  From 512 key heads on, a workgroup of 4
// waves each (two a compute unit); from 256 on, and where a key head's rows are few enough that
// one compute unit reads them in less time than the second launch that joins ranges takes,
// a workgroup of 8.  Else ranges of whole 128-slot steps, for two workgroups a compute unit.
constexpr size_t kOneUnitBytes = 640 << 10;
void split_plan(int units, int C, int row_bytes, int* n_split, int* split_len, int* waves) {
  int n = 1;
  *waves = units < 512 ? 8 : 4;
  if (units < 256 && (size_t)C * 2 * row_bytes > kOneUnitBytes) {
    n = std::min({ceil_div(512, units), ceil_div(C, 128), 64});
    *waves = 4;
  }
  *split_len = ceil_div(ceil_div(C, n), 128) * 128;
  *n_split = ceil_div(C, *split_len);
}
// The same for rows of codes, which are read sooner than a step of 128 slots is computed.  Up to 256 key heads one
// workgroup of 8 waves each, above of 4 (400 of 512 slots with weights: 14.5 us of 4 waves, 20.0 of 8, without 10.8 and
// 11.1; 256: 10.6 and 10.6, 8.4 and 7.9; of 2,048 slots with weights 28.1 and 22.3).  Up to 128 key heads, half a chip of
// workgroups, are cut into ranges where that saves more than the launch that joins them.  In one workgroup / in ranges,
// D = 128, 4 heads on one, bf16, 4 bits, us:
//   key heads            4          64          68          96         128        160         240
//   ring    1,024     9.1/7.9
//           1,536               11.7/11.7   11.7/11.7
//           2,048    13.4/8.2   14.2/12.7   14.3/13.0   14.3/14.9   14.6/15.6
//           4,096    22.2/9.0   22.9/15.6   23.0/16.3   23.7/20.6   24.3/21.5   25.3/27.2   28.5/33.3
//   weights 1,024    12.0/10.3
//           1,536               16.4/15.5
//           2,048    17.2/11.1  19.3/16.6   19.1/18.3   19.7/20.8
//           4,096               -           31.4/26.6   32.2/31.0   33.0/32.4               (192: 34.5/44.7)
//           8,192               -           54.0/39.0   55.2/47.8   56.9/53.7               74.9/82.9
// 8 bits, D = 64, float32 and 16 heads on one cross over at the same lengths or a little below (128 key heads of 2,999 slots
// in 8 bits 27.5/25.3, d64 14.6/13.6, fp32 24.0/20.1; 160 of 8,192 in 8 bits 71.7/73.1, d64 32.2/29.4, fp32 55/49, with
// weights 90/99, 51/50, 73/70).  A caller that launches each step anew pays the second launch's 4 us too, so few
// key heads of up to 1,536 slots stay in one.
void mx_split_plan(int units, int C, bool weights, int* n_split, int* split_len, int* waves) {
  const int most = units <= 64 ? 1536 : weights ? 4096 : 3000;      // slots of one workgroup
  int n = 1;
  *waves = units <= 256 ? 8 : 4;
  if (units <= 128 && C > most) {
    n = std::min({ceil_div(512, units), ceil_div(C, 128), 64});
    *waves = 4;
  }
  *split_len = ceil_div(ceil_div(C, n), 128) * 128;
  *n_split = ceil_div(C, *split_len);
}
size_t part_bytes(int units, int G, int D, int n_split) {
  return n_split > 1 ? up256((size_t)units * n_split * G * (D + 4) * sizeof(float)) : 0;
}

carve_status check_rows(const carve_mx_rows* r) {
  if (!r) return CARVE_ERR_INVALID_ARG;
  if (r->bits != 4 && r->bits != 8) return CARVE_ERR_UNSUPPORTED;
  if (!all_given({r->k_codes, r->k_scales, r->v_codes, r->v_scales}) || !all_aligned({r->k_codes, r->v_codes}, 16) ||
      !all_aligned({r->k_scales, r->v_scales}, 4))
    return CARVE_ERR_INVALID_ARG;
  return CARVE_OK;
}

carve_status check_budget(const carve_budget_shape* s) {
  if (!s) return CARVE_ERR_INVALID_ARG;
  if (s->sinks < 0 || s->recent < 1 || s->C < 1) return CARVE_ERR_INVALID_ARG;
  const carve_status st = check_heads(s->B, s->Hq, s->Hkv, s->T, s->D, s->dtype, s->scale);
  if (st != CARVE_OK) return st;
  // a full cache always has a slot to give up: the first and the recent tokens leave one
  if ((long long)s->sinks + s->recent > s->C) return CARVE_ERR_INVALID_ARG;
  if (s->C > kMaxTokens) return CARVE_ERR_UNSUPPORTED;
  return CARVE_OK;
}

// Whether a budget cache's scores of this step stay in LDS: where its workgroup of 8 waves is its
// compute unit's only one anyway, up to one a unit or by the LDS that its rows take at D = 128.  At D = 64
// two fit, and the scores' 16 KB would keep the second off: 300 key heads of 1,024 slots 26.5 us with
// them in LDS, 22.0 without, 480 of 512 slots 20.5 and 16.6 (one sequence of four heads 13.4 and 14.9).
bool plain_near_scores(const carve_budget_shape* s, int n_split, int waves) {
  const long long G = s->Hq / s->Hkv;
  return s->dtype == CARVE_BF16 && n_split == 1 && waves == 8 && (s->D == 128 || s->B * s->Hkv <= 256) && G <= 16 &&
         G * carve::score_row(s->C) <= carve::kNearScores;
}
// The same for rows of codes: workgroups of 8 waves are one a compute unit at most; of 4, up to two are that few
// (64 / 128 sequences of 2,048 slots, 16 heads on 4: 22 / 38 us in LDS, 25 / 42 without; 129: 57 in LDS, 50 without).
bool near_scores(const carve_budget_shape* s, int bits, int n_split, int waves) {
  if (!bits) return plain_near_scores(s, n_split, waves);
  const long long G = s->Hq / s->Hkv;
  return n_split == 1 && (waves == 8 || s->B * s->Hkv <= 512) && G <= (waves == 8 ? 32 : 16) &&
         G * carve::score_row(s->C) <= carve::mx_near_scores(bits, s->D, waves);
}

// A cache as the calls give it: rows of the call's dtype, or codes and scales.
struct CacheRows {
  int bits;                                 // 0: rows of dtype
  void *k, *v;
  unsigned char *k_scales, *v_scales;
};
CacheRows plain_rows(void* k, void* v) { return {0, k, v, nullptr, nullptr}; }
CacheRows mx_rows(const carve_mx_rows* r) {
  return {r->bits, r->k_codes, r->v_codes, (unsigned char*)r->k_scales, (unsigned char*)r->v_scales};
}
template <typename Args>
void set_rows(Args& a, const CacheRows& r) {
  a.cache_k = r.k;
  a.cache_v = r.v;
  a.bits = r.bits;
  a.k_scales = r.k_scales;
  a.v_scales = r.v_scales;
}
void plan(int units, int C, int D, carve_dtype dtype, int bits, bool weights, int* n_split, int* split_len, int* waves) {
  if (bits) mx_split_plan(units, C, weights, n_split, split_len, waves);
  else split_plan(units, C, row_bytes(D, dtype), n_split, split_len, waves);
}
hipError_t fill(const carve::FillArgs& a, hipStream_t st) {
  return a.bits ? carve::launch_mx_fill(a, st) : carve::launch_fill_rows(a, st);
}
hipError_t decode(const carve::CacheArgs& a, hipStream_t st) {
  return a.bits ? carve::launch_mx_decode(a, st) : carve::launch_cache_decode(a, st);
}

carve_status swa_fill(const carve_swa_shape* s, const void* k, const void* v, const int* lens, const CacheRows& rows,
                      void* stream) {
  carve::FillArgs a;
  memset(&a, 0, sizeof(a));
  a.B = s->B;
  a.Hkv = s->Hkv;
  a.T = s->T;
  a.D = s->D;
  a.C = s->window + s->sinks;
  a.window = s->window;
  a.sinks = s->sinks;
  a.dtype = s->dtype == CARVE_BF16;
  a.k = k;
  a.v = v;
  a.lens = lens;
  set_rows(a, rows);
  return hip_status(fill(a, (hipStream_t)stream));
}

size_t swa_decode_bytes(const carve_swa_shape* s, int bits) {
  if (check_swa(s) != CARVE_OK || s->T != 1 || empty(s) || s->Hq / s->Hkv > kMaxGroup) return 0;
  int n, len, waves;
  plan(s->B * s->Hkv, s->window + s->sinks, s->D, s->dtype, bits, false, &n, &len, &waves);
  const size_t bytes = part_bytes(s->B * s->Hkv, s->Hq / s->Hkv, s->D, n);
  return bytes ? bytes + 256 : 0;
}

carve_status swa_decode(const carve_swa_shape* s, const void* q, const void* k, const void* v, const CacheRows& rows,
                        const int* pos, void* o, void* workspace, size_t workspace_bytes, void* stream) {
  carve::CacheArgs a;
  memset(&a, 0, sizeof(a));
  a.B = s->B;
  a.Hq = s->Hq;
  a.Hkv = s->Hkv;
  a.D = s->D;
  a.C = s->window + s->sinks;
  a.window = s->window;
  a.sinks = s->sinks;
  a.dtype = s->dtype == CARVE_BF16;
  a.scale = s->scale;
  a.q = q;
  a.k = k;
  a.v = v;
  set_rows(a, rows);
  a.pos = pos;
  a.o = o;
  plan(a.B * a.Hkv, a.C, a.D, s->dtype, rows.bits, false, &a.n_split, &a.split_len, &a.waves);
  const size_t need = swa_decode_bytes(s, rows.bits);
  if (need && (!workspace || workspace_bytes < need)) return CARVE_ERR_WORKSPACE;
  a.part = reinterpret_cast<float*>(up256(reinterpret_cast<uintptr_t>(workspace)));
  return hip_status(decode(a, (hipStream_t)stream));
}

carve_status budget_keep(const carve_budget_shape* s, const void* k, const void* v, const float* weights, const int* lens,
                         const CacheRows& rows, float* cache_w, int* cache_pos, void* stream) {
  carve::FillArgs a;
  memset(&a, 0, sizeof(a));
  a.B = s->B;
  a.Hkv = s->Hkv;
  a.T = s->T;
  a.D = s->D;
  a.C = s->C;
  a.sinks = s->sinks;
  a.recent = s->recent;
  a.dtype = s->dtype == CARVE_BF16;
  a.k = k;
  a.v = v;
  a.weights = weights;
  a.lens = lens;
  set_rows(a, rows);
  a.cache_w = cache_w;
  a.cache_pos = cache_pos;
  const hipError_t e = carve::launch_keep_select(a, (hipStream_t)stream);
  if (e != hipSuccess) return hip_status(e);
  return hip_status(fill(a, (hipStream_t)stream));
}

size_t budget_decode_bytes(const carve_budget_shape* s, int bits) {
  if (check_budget(s) != CARVE_OK || s->T != 1 || s->B == 0 || s->Hq == 0 || s->Hq / s->Hkv > kMaxGroup) return 0;
  int n, len, waves;
  plan(s->B * s->Hkv, s->C, s->D, s->dtype, bits, true, &n, &len, &waves);
  const size_t bytes = part_bytes(s->B * s->Hkv, s->Hq / s->Hkv, s->D, n) +
                       (near_scores(s, bits, n, waves) ? 0 : (size_t)s->B * s->Hq * carve::score_row(s->C) * sizeof(float));
  return bytes ? bytes + 256 : 0;
}

carve_status budget_decode(const carve_budget_shape* s, const void* q, const void* k, const void* v,
                           const CacheRows& rows, float* cache_w, int* cache_pos, const int* pos, void* o, int* slot,
                           void* workspace, size_t workspace_bytes, void* stream) {
  carve::CacheArgs a;
  memset(&a, 0, sizeof(a));
  a.B = s->B;
  a.Hq = s->Hq;
  a.Hkv = s->Hkv;
  a.D = s->D;
  a.C = s->C;
  a.sinks = s->sinks;
  a.recent = s->recent;
  a.dtype = s->dtype == CARVE_BF16;
  a.scale = s->scale;
  a.q = q;
  a.k = k;
  a.v = v;
  set_rows(a, rows);
  a.cache_w = cache_w;
  a.cache_pos = cache_pos;
  a.pos = pos;
  a.o = o;
  a.slot = slot;
  plan(a.B * a.Hkv, a.C, a.D, s->dtype, rows.bits, true, &a.n_split, &a.split_len, &a.waves);
  const size_t need = budget_decode_bytes(s, rows.bits);
  if (need && (!workspace || workspace_bytes < need)) return CARVE_ERR_WORKSPACE;
  char* ws = reinterpret_cast<char*>(up256(reinterpret_cast<uintptr_t>(workspace)));
  a.part = reinterpret_cast<float*>(ws);
  a.score = near_scores(s, rows.bits, a.n_split, a.waves)
                ? nullptr
                : reinterpret_cast<float*>(ws + part_bytes(a.B * a.Hkv, a.Hq / a.Hkv, a.D, a.n_split));
  return hip_status(decode(a, (hipStream_t)stream));
}

}  // namespace

extern "C" {

carve_status carve_swa_fwd(const carve_swa_shape* s, const void* q, const void* k, const void* v, const int* lens,
                           void* o, float* lse, void* stream) {
  const carve_status st = check_swa(s);
  if (st != CARVE_OK) return st;
  if (empty(s)) return CARVE_OK;
  if (!all_given({q, k, v, o}) || !all_aligned({q, k, v, o}, 16) || !all_aligned({lens, lse}, 4))
    return CARVE_ERR_INVALID_ARG;
  if ((long long)s->B * s->Hq * ceil_div(s->T, 128) > kMaxUnits) return CARVE_ERR_UNSUPPORTED;
  carve::SwaArgs a = swa_args(s, q, k, v, lens);
  a.o = o;
  a.lse = lse;
  return hip_status(carve::launch_swa_fwd(a, (hipStream_t)stream));
}

size_t carve_swa_bwd_workspace_size(const carve_swa_shape* s) {
  if (check_swa(s) != CARVE_OK || empty(s)) return 0;
  const SwaPlan p = swa_plan(s);
  return p.bytes();
}

carve_status carve_swa_bwd(const carve_swa_shape* s, const void* q, const void* k, const void* v, const int* lens,
                           const void* o, const float* lse, const void* dO, void* dq, void* dk, void* dv,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const carve_status st = check_swa(s);
  if (st != CARVE_OK) return st;
  if (empty(s)) return CARVE_OK;
  if (!all_given({q, k, v, o, lse, dO, dq, dk, dv}) || !all_aligned({q, k, v, o, dO, dq, dk, dv}, 16) ||
      !all_aligned({lens, lse}, 4))
    return CARVE_ERR_INVALID_ARG;
  const SwaPlan p = swa_plan(s);
  const long long per = (long long)ceil_div(s->T, carve::kSwaKeyTile) * p.n_head_part + (long long)p.n_sink_tiles * p.n_far;
  if ((long long)s->B * s->Hq * per > kMaxUnits)
    return CARVE_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < p.bytes()) return CARVE_ERR_WORKSPACE;
  carve::SwaArgs a = swa_args(s, q, k, v, lens);
  a.o = const_cast<void*>(o);
  a.lse = const_cast<float*>(lse);
  a.dO = dO;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  char* ws = reinterpret_cast<char*>(up256(reinterpret_cast<uintptr_t>(workspace)));
  a.delta = reinterpret_cast<float*>(ws);
  a.lse2 = reinterpret_cast<float*>(ws + p.delta_bytes);
  a.part = reinterpret_cast<float*>(ws + 2 * p.delta_bytes);
  a.head_part = reinterpret_cast<float*>(ws + 2 * p.delta_bytes + p.part_bytes);
  a.n_head_part = p.n_head_part;
  a.n_sink_tiles = p.n_sink_tiles;
  a.n_far = p.n_far;
  a.far_len = p.far_len;
  return hip_status(carve::launch_swa_bwd(a, (hipStream_t)stream));
}

// (a cache in codes: the same checks, of its rows last)
static carve_status fill_call(const carve_swa_shape* s, const void* k, const void* v, const int* lens) {
  const carve_status st = check_swa(s);
  if (st != CARVE_OK || empty(s)) return st;
  if (!all_given({k, v}) || !all_aligned({k, v}, 16) || !aligned(lens, 4)) return CARVE_ERR_INVALID_ARG;
  return CARVE_OK;
}
static carve_status decode_call(const carve_swa_shape* s, const void* q, const void* k, const void* v, const int* pos,
                                const void* o) {
  const carve_status st = check_swa(s);
  if (st != CARVE_OK) return st;
  if (s->T != 1) return CARVE_ERR_INVALID_ARG;
  if (empty(s)) return CARVE_OK;
  if (s->Hq / s->Hkv > kMaxGroup) return CARVE_ERR_UNSUPPORTED;
  if (!all_given({q, k, v, pos, o}) || !all_aligned({q, k, v, o}, 16) || !aligned(pos, 4)) return CARVE_ERR_INVALID_ARG;
  return CARVE_OK;
}

carve_status carve_swa_fill(const carve_swa_shape* s, const void* k, const void* v, const int* lens, void* cache_k,
                            void* cache_v, void* stream) {
  const carve_status st = fill_call(s, k, v, lens);
  if (st != CARVE_OK || empty(s)) return st;
  if (!all_given({cache_k, cache_v}) || !all_aligned({cache_k, cache_v}, 16)) return CARVE_ERR_INVALID_ARG;
  return swa_fill(s, k, v, lens, plain_rows(cache_k, cache_v), stream);
}

carve_status carve_swa_fill_mx(const carve_swa_shape* s, const void* k, const void* v, const int* lens,
                               const carve_mx_rows* cache, void* stream) {
  carve_status st = fill_call(s, k, v, lens);
  if (st != CARVE_OK || empty(s)) return st;
  st = check_rows(cache);
  if (st != CARVE_OK) return st;
  return swa_fill(s, k, v, lens, mx_rows(cache), stream);
}

size_t carve_swa_decode_workspace_size(const carve_swa_shape* s) { return swa_decode_bytes(s, 0); }

carve_status carve_swa_decode(const carve_swa_shape* s, const void* q, const void* k, const void* v, void* cache_k,
                              void* cache_v, const int* pos, void* o, void* workspace, size_t workspace_bytes,
                              void* stream) {
  const carve_status st = decode_call(s, q, k, v, pos, o);
  if (st != CARVE_OK || empty(s)) return st;
  if (!all_given({cache_k, cache_v}) || !all_aligned({cache_k, cache_v}, 16)) return CARVE_ERR_INVALID_ARG;
  return swa_decode(s, q, k, v, plain_rows(cache_k, cache_v), pos, o, workspace, workspace_bytes, stream);
}

size_t carve_swa_decode_mx_workspace_size(const carve_swa_shape* s, int bits) {
  return bits == 4 || bits == 8 ? swa_decode_bytes(s, bits) : 0;
}

carve_status carve_swa_decode_mx(const carve_swa_shape* s, const void* q, const void* k, const void* v,
                                 const carve_mx_rows* cache, const int* pos, void* o, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  carve_status st = decode_call(s, q, k, v, pos, o);
  if (st != CARVE_OK || empty(s)) return st;
  st = check_rows(cache);
  if (st != CARVE_OK) return st;
  return swa_decode(s, q, k, v, mx_rows(cache), pos, o, workspace, workspace_bytes, stream);
}

size_t carve_budget_weights_workspace_size(const carve_swa_shape* s) {
  if (check_swa(s) != CARVE_OK || empty(s)) return 0;
  const WeightPlan p = weight_plan(s);
  const int n = p.n_chunk * p.n_head;
  return n > 1 ? (size_t)n * s->B * s->Hkv * s->T * sizeof(float) + 256 : 0;
}

carve_status carve_budget_weights(const carve_swa_shape* s, const void* q, const void* k, const float* lse,
                                  const int* lens, float* weights, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  const carve_status st = check_swa(s);
  if (st != CARVE_OK) return st;
  if (empty(s)) return CARVE_OK;
  if (!all_given({q, k, lse, weights}) || !all_aligned({q, k}, 16) || !all_aligned({lse, lens, weights}, 4))
    return CARVE_ERR_INVALID_ARG;
  carve::WeightArgs a;
  memset(&a, 0, sizeof(a));
  a.B = s->B;
  a.Hq = s->Hq;
  a.Hkv = s->Hkv;
  a.T = s->T;
  a.D = s->D;
  mask_of(s, &a.window, &a.sinks);
  a.dtype = s->dtype == CARVE_BF16;
  a.scale = s->scale;
  a.q = q;
  a.k = k;
  a.lse = lse;
  a.lens = lens;
  a.out = weights;
  const WeightPlan p = weight_plan(s);
  a.n_chunk = p.n_chunk;
  a.chunk = p.chunk;
  a.n_head = p.n_head;
  if ((long long)a.B * a.Hkv * ceil_div(a.T, 128) * a.n_chunk * a.n_head > kMaxUnits) return CARVE_ERR_UNSUPPORTED;
  const size_t need = carve_budget_weights_workspace_size(s);
  if (need && (!workspace || workspace_bytes < need)) return CARVE_ERR_WORKSPACE;
  a.part = reinterpret_cast<float*>(up256(reinterpret_cast<uintptr_t>(workspace)));
  return hip_status(carve::launch_weights(a, (hipStream_t)stream));
}

static carve_status keep_call(const carve_budget_shape* s, const void* k, const void* v, const float* weights,
                              const int* lens, const float* cache_w, const int* cache_pos) {
  const carve_status st = check_budget(s);
  if (st != CARVE_OK || s->B == 0 || s->Hkv == 0) return st;
  if (!all_given({cache_w, cache_pos}) || (s->T > 0 && !all_given({k, v, weights})) || !all_aligned({k, v}, 16) ||
      !all_aligned({weights, lens, cache_w, cache_pos}, 4))
    return CARVE_ERR_INVALID_ARG;
  return CARVE_OK;
}
static carve_status evict_call(const carve_budget_shape* s, const void* q, const void* k, const void* v,
                               const float* cache_w, const int* cache_pos, const int* pos, const void* o, const int* slot) {
  const carve_status st = check_budget(s);
  if (st != CARVE_OK) return st;
  if (s->T != 1) return CARVE_ERR_INVALID_ARG;
  if (s->B == 0 || s->Hq == 0) return CARVE_OK;
  if (s->Hq / s->Hkv > kMaxGroup) return CARVE_ERR_UNSUPPORTED;
  if (!all_given({q, k, v, cache_w, cache_pos, pos, o, slot}) || !all_aligned({q, k, v, o}, 16) ||
      !all_aligned({cache_w, cache_pos, pos, slot}, 4))
    return CARVE_ERR_INVALID_ARG;
  return CARVE_OK;
}

carve_status carve_budget_keep(const carve_budget_shape* s, const void* k, const void* v, const float* weights,
                               const int* lens, void* cache_k, void* cache_v, float* cache_w, int* cache_pos,
                               void* stream) {
  const carve_status st = keep_call(s, k, v, weights, lens, cache_w, cache_pos);
  if (st != CARVE_OK || s->B == 0 || s->Hkv == 0) return st;
  if (!all_given({cache_k, cache_v}) || !all_aligned({cache_k, cache_v}, 16)) return CARVE_ERR_INVALID_ARG;
  return budget_keep(s, k, v, weights, lens, plain_rows(cache_k, cache_v), cache_w, cache_pos, stream);
}

carve_status carve_budget_keep_mx(const carve_budget_shape* s, const void* k, const void* v, const float* weights,
                                  const int* lens, const carve_mx_rows* cache, float* cache_w, int* cache_pos,
                                  void* stream) {
  carve_status st = keep_call(s, k, v, weights, lens, cache_w, cache_pos);
  if (st != CARVE_OK || s->B == 0 || s->Hkv == 0) return st;
  st = check_rows(cache);
  if (st != CARVE_OK) return st;
  return budget_keep(s, k, v, weights, lens, mx_rows(cache), cache_w, cache_pos, stream);
}

size_t carve_budget_decode_workspace_size(const carve_budget_shape* s) { return budget_decode_bytes(s, 0); }

carve_status carve_budget_decode(const carve_budget_shape* s, const void* q, const void* k, const void* v,
                                 void* cache_k, void* cache_v, float* cache_w, int* cache_pos, const int* pos, void* o,
                                 int* slot, void* workspace, size_t workspace_bytes, void* stream) {
  const carve_status st = evict_call(s, q, k, v, cache_w, cache_pos, pos, o, slot);
  if (st != CARVE_OK || s->B == 0 || s->Hq == 0) return st;
  if (!all_given({cache_k, cache_v}) || !all_aligned({cache_k, cache_v}, 16)) return CARVE_ERR_INVALID_ARG;
  return budget_decode(s, q, k, v, plain_rows(cache_k, cache_v), cache_w, cache_pos, pos, o, slot, workspace,
                       workspace_bytes, stream);
}

size_t carve_budget_decode_mx_workspace_size(const carve_budget_shape* s, int bits) {
  return bits == 4 || bits == 8 ? budget_decode_bytes(s, bits) : 0;
}

carve_status carve_budget_decode_mx(const carve_budget_shape* s, const void* q, const void* k, const void* v,
                                    const carve_mx_rows* cache, float* cache_w, int* cache_pos, const int* pos, void* o,
                                    int* slot, void* workspace, size_t workspace_bytes, void* stream) {
  carve_status st = evict_call(s, q, k, v, cache_w, cache_pos, pos, o, slot);
  if (st != CARVE_OK || s->B == 0 || s->Hq == 0) return st;
  st = check_rows(cache);
  if (st != CARVE_OK) return st;
  return budget_decode(s, q, k, v, mx_rows(cache), cache_w, cache_pos, pos, o, slot, workspace, workspace_bytes, stream);
}

// Values in pieces of eight; both directions check alike.
static carve_status row_call(size_t n, carve_dtype dtype, int bits, const void* x, const void* codes, const void* scales) {
  if (dtype != CARVE_F32 && dtype != CARVE_BF16) return CARVE_ERR_INVALID_ARG;
  if (n % 32 != 0) return CARVE_ERR_INVALID_ARG;
  if (bits != 4 && bits != 8) return CARVE_ERR_UNSUPPORTED;
  if (n == 0) return CARVE_OK;
  if (!all_given({x, codes, scales}) || !all_aligned({x, codes}, 16)) return CARVE_ERR_INVALID_ARG;
  return CARVE_OK;
}

carve_status carve_mx_quant(size_t n, carve_dtype dtype, int bits, const void* x, void* codes, void* scales, void* stream) {
  const carve_status st = row_call(n, dtype, bits, x, codes, scales);
  if (st != CARVE_OK || n == 0) return st;
  const carve::MxRowArgs a = {n / 8, dtype == CARVE_BF16, bits, const_cast<void*>(x), codes, scales};
  return hip_status(carve::launch_mx_quant(a, (hipStream_t)stream));
}

carve_status carve_mx_dequant(size_t n, carve_dtype dtype, int bits, const void* codes, const void* scales, void* x,
                              void* stream) {
  const carve_status st = row_call(n, dtype, bits, x, codes, scales);
  if (st != CARVE_OK || n == 0) return st;
  const carve::MxRowArgs a = {n / 8, dtype == CARVE_BF16, bits, x, const_cast<void*>(codes), const_cast<void*>(scales)};
  return hip_status(carve::launch_mx_dequant(a, (hipStream_t)stream));
}

}  // extern "C"
