// Backward pass of sliding-window attention with sinks.
//
// With p_ts = exp(scale q_t . k_s - lse_t) and delta_t = dO_t . o_t:
//   ds_ts = p_ts (dO_t . v_s - delta_t)
//   dq_t = scale sum_s ds_ts k_s,   dk_s = scale sum_t ds_ts q_t,   dv_s = sum_t p_ts dO_t,
// the last two also summed over the query heads that share the key head.  Two passes, each
// with its sums in registers in a fixed order, and no atomics: one over the keys of a tile
// of tokens (dq, and delta for the other pass), one over the tokens of a tile of keys.
// That is seven products of a visible pair where one pass with shared sums has five.
// Bound by the products and the vector work beside them, and in the second pass by waits that its
// 256 registers a wave leave uncovered (matrix cores busy 0.48, vector units 0.37 and 0.30).
// B4, 16 heads on 4, T = 4,096, window 1,024, 4 sinks, D = 128: dq 224 us, dk/dv 285 us, sinks 5 us
// (0.60 to 0.65 ms from card to card with the forward pass, 0.65 to 0.70 PFLOP/s of 14 D flops a visible
// pair).
#include <algorithm>

#include "attn_device.h"

namespace carve {

constexpr int kDqQ = 128, kDqK = 64;

struct DqUnit {
  int b, bk, hq, t0, n;
};
__device__ __forceinline__ DqUnit dq_unit(const SwaArgs& a, int QT) {
  const int G = a.Hq / a.Hkv, NQ = (a.T + QT - 1) / QT;
  const int unit = attn_unit(a.B * a.Hq * NQ, G, a.window, a.T, a.B * a.Hkv, 3);
  DqUnit u;
  u.bk = uniform(unit / (G * NQ));
  u.t0 = uniform((NQ - 1 - (unit / G) % NQ) * QT);
  u.b = uniform(u.bk / a.Hkv);
  u.hq = uniform((u.bk % a.Hkv) * G + unit % G);
  u.n = seq_len(a.lens, u.b, a.T);
  return u;
}
// the lane's element of the diagonal of a 32 x 32 accumulator tile (both halves of the wave)
__device__ __forceinline__ float diagonal(const f32x16& c) {
  const int lane = lane_id(), half = lane >> 5;
  float x = 0.f;
#pragma unroll
  for (int r = 0; r < 16; ++r) x = acc_row(r, half) == (lane & 31) ? c[r] : x;
  const float other = __shfl_xor(x, 32);
  return ((lane >> 2) & 1) == half ? x : other;
}
// p x, and zero where p is zero whatever x is (v_mul_legacy_f32; clang has no builtin for it, so the
// compiler's intrinsic is named): a key that a token does not see gets no part of a delta or
// product that is not finite.  A select on ds beside that on p costs 4 % of the training step (634
// against 608 us), this nothing.
extern "C" __device__ float weighted(float p, float x) __asm("llvm.amdgcn.fmul.legacy");
// no visible weight (lse = -inf): every p is exp2(. - inf) = 0
__device__ __forceinline__ float log2_lse(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// A workgroup of the dk / dv pass: kSwaKeyTile keys of one key head (a lane owns one key), over the
// tokens t_lo .. t_hi - 1 that see them inside the window and all heads of the group.  The tokens
// behind the window of a tile that holds sinks see only the sinks: they are cut into n_far ranges
// with workgroups of their own, whose sums, like the tile's, go to `part` and are added by
// swa_sink_kernel.
// Where tiles are few (a.n_head_part > 1), the heads of a group are cut into parts as well; then every
// tile's sums go to `head_part`, and the same kernel adds them.
struct KeyUnit {
  int b, bk, n, kt, s0, t_lo, t_hi, h_lo, h_hi;
  bool far;
  float* part;                                // partial sums [2][kSwaKeyTile][D], null = final
};
__device__ __forceinline__ KeyUnit key_unit(const SwaArgs& a) {
  constexpr int KT = kSwaKeyTile;
  const int NK = (a.T + KT - 1) / KT, HP = a.n_head_part, G = a.Hq / a.Hkv, per = NK * HP + a.n_sink_tiles * a.n_far;
  const int unit = attn_unit(a.B * a.Hkv * per, 1, a.window, a.T, a.B * a.Hkv, 3);
  KeyUnit u;
  u.bk = uniform(unit / per);
  u.b = uniform(u.bk / a.Hkv);
  u.n = seq_len(a.lens, u.b, a.T);
  const int w = uniform(unit % per);
  u.far = w >= NK * HP;
  u.kt = uniform(u.far ? (w - NK * HP) / a.n_far : w / HP);
  const int fi = uniform(u.far ? (w - NK * HP) % a.n_far : 0), hp = uniform(u.far ? 0 : w % HP);
  const int heads = (G + HP - 1) / HP;
  u.h_lo = u.far ? 0 : hp * heads;
  u.h_hi = u.far ? G : min(G, u.h_lo + heads);
  u.s0 = u.kt * KT;
  const long long band = (long long)u.s0 + KT - 1 + a.window;     // first token that sees no key of the tile
  const long long lo = u.far ? band + (long long)fi * a.far_len : u.s0, hi = u.far ? lo + a.far_len : band;
  u.t_lo = uniform((int)min((long long)u.n, lo));
  u.t_hi = uniform((int)min((long long)u.n, hi));
  u.part = nullptr;
  constexpr size_t one = 2 * KT;
  if (u.far || (HP == 1 && u.kt < a.n_sink_tiles && a.n_far > 0))
    u.part = a.part + (((size_t)u.bk * a.n_sink_tiles + u.kt) * (1 + a.n_far) + (u.far ? 1 + fi : 0)) * one * a.D;
  else if (HP > 1)
    u.part = a.head_part + (((size_t)u.bk * NK + u.kt) * HP + hp) * one * a.D;
  return u;
}
template <typename T, int D>
__device__ __forceinline__ void store_key_grads(const SwaArgs& a, const KeyUnit& u, int s, int kb, f32x16 (&dK)[D / 32],
                                                f32x16 (&dV)[D / 32]) {
  constexpr int KT = kSwaKeyTile;
  if (u.part) {
    float* dst = u.part + (32 * kb + (lane_id() & 31)) * D;
    if (!u.far || s < a.sinks) {              // (a far range adds to sinks only)
      store_column<float, D>(dst, dK, a.scale);
      store_column<float, D>(dst + (size_t)KT * D, dV, 1.f);
    }
  } else if (s < a.T) {
    if (s >= u.n) {
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) {
        dK[dt] = zero16();
        dV[dt] = zero16();
      }
    }
    const size_t row = ((size_t)u.bk * a.T + s) * D;
    store_column<T, D>(reinterpret_cast<T*>(a.dk) + row, dK, a.scale);
    store_column<T, D>(reinterpret_cast<T*>(a.dv) + row, dV, 1.f);
  }
}

// x of the waves th = 1 added to that of the waves th = 0, through 128 D bytes of LDS a pair
template <int D>
__device__ __forceinline__ void join_halves(float* park, int th, f32x16 (&x)[D / 32]) {
  const int lane = lane_id();
  __syncthreads();
  if (th) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      store4(park + (i * 64 + lane) * 4, f32x4{x[i / 4][4 * (i & 3)], x[i / 4][4 * (i & 3) + 1], x[i / 4][4 * (i & 3) + 2],
                                               x[i / 4][4 * (i & 3) + 3]});
  }
  __syncthreads();
  if (!th) {
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const f32x4 y = load4f(park + (i * 64 + lane) * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i / 4][4 * (i & 3) + e] += y[e];
    }
  }
}

// ------------------------------------------------------------------ bf16: dq
// Workgroup = 128 tokens of one query head (32 a wave, a lane owns one), tiles of 64 keys in two
// pairs of swizzled LDS buffers as in the forward pass.  delta comes from the rounded o where many
// keys share it.  Where few are seen (at most kExactKeys, or the sequence's first tile) its rounding,
// half a step of o, would be as large as that of ds itself: there a first sweep forms
// delta_t = sum_s p_ts (dO_t . v_s).  (Error of dq against 64 bits at window 3: 3.3e-3 -> 2.3e-3.)
constexpr int kExactKeys = 64;

template <int D>
__global__ __launch_bounds__(256, 2) void swa_dq_bf16_kernel(SwaArgs a) {
  using Tile = SwzTile<D, kDqK>;
  constexpr int KK = D / 16, DT = D / 32;
  __shared__ __align__(16) unsigned char K0[Tile::bytes], K1[Tile::bytes];
  __shared__ __align__(16) unsigned char V0[Tile::bytes], V1[Tile::bytes];
  const DqUnit un = dq_unit(a, kDqQ);
  const int n = un.n, t0 = un.t0, lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int tw = t0 + 32 * wave, t = tw + (lane & 31);
  const size_t row = (size_t)(un.b * a.Hq + un.hq) * a.T;
  const bf16* kb = reinterpret_cast<const bf16*>(a.k) + (size_t)un.bk * a.T * D;
  const bf16* vb = reinterpret_cast<const bf16*>(a.v) + (size_t)un.bk * a.T * D;

  f32x16 dQ[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) dQ[dt] = zero16();
  if (t0 < n) {
    const KeyTiles<kDqK> kt(t0, min(t0 + kDqQ, n), a.window, a.sinks);
    Frag<bf16> Q[KK], dO[KK];
    const size_t at = (row + min(t, n - 1)) * D + 8 * half;
    // delta_t = dO_t . o_t as the diagonal of a product formed as dO . v is below: a token that
    // sees one key has o = v, and its ds is zero to the last bit
    f32x16 od = zero16();
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      Q[kk] = load_frag(reinterpret_cast<const bf16*>(a.q) + at + 16 * kk);
      dO[kk] = load_frag(reinterpret_cast<const bf16*>(a.dO) + at + 16 * kk);
      mma32(od, load_frag(reinterpret_cast<const bf16*>(a.o) + at + 16 * kk), dO[kk]);
    }
    float delta = diagonal(od);
    const float c = a.scale * kLog2e;
    const float lse2 = log2_lse(a.lse[row + min(t, n - 1)]);
    const int rb = Tile::row_base(), cb = Tile::col_base();

    // weights p and dp = dO . v of 32 keys; what is not seen has p = 0.  That is decided before the
    // products, so that they and the exponentials stand in one stretch of code without branches.
    auto scores = [&](const unsigned char* Ks, const unsigned char* Vs, int u, const bool(&see)[16], f32x16& S, f32x16& dP) {
      S = zero16();
      dP = zero16();
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) mma32(S, Tile::row_frag(Ks, rb, 32 * u, kk), Q[kk]);
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) mma32(dP, Tile::row_frag(Vs, rb, 32 * u, kk), dO[kk]);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float p = __builtin_amdgcn_exp2f(S[r] * c - lse2);
        S[r] = see[r] ? p : 0.f;
      }
    };
    auto sight = [&](int su, bool(&see)[16]) {
      const bool full = su + 31 <= tw && (tw + 31 - su < a.window || su + 32 <= a.sinks);
#pragma unroll
      for (int r = 0; r < 16; ++r) see[r] = true;
      if (!full) {
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int s = su + acc_row(r, half);
          see[r] = (s <= t) & ((t - s < a.window) | (s < a.sinks));
        }
      }
    };
    auto seen = [&](int s0) {
      return !(s0 > tw + 31 || (s0 >= a.sinks && tw - (s0 + kDqK - 1) >= a.window));
    };
    auto load = [&](unsigned char* Ks, unsigned char* Vs, int i) {
      if (i < kt.count) {
        Tile::template load<4>(Ks, kb, kt[i], kt.rows(i, n), wave);
        Tile::template load<4>(Vs, vb, kt[i], kt.rows(i, n), wave);
      }
    };
    auto sweep = [&](auto&& step) {
      load(K0, V0, 0);
      for (int i = 0; i < kt.count; i += 2) {
        loads_and_barrier();
        load(K1, V1, i + 1);
        if (seen(kt[i])) step(K0, V0, kt[i]);
        loads_and_barrier();
        load(K0, V0, i + 2);
        if (i + 1 < kt.count && seen(kt[i + 1])) step(K1, V1, kt[i + 1]);
      }
    };
    if (t0 == 0 || a.window + a.sinks <= kExactKeys) {
      float sum = 0.f;
      sweep([&](const unsigned char* Ks, const unsigned char* Vs, int s0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          bool see[16];
          f32x16 S, dP;
          sight(s0 + 32 * u, see);
          scores(Ks, Vs, u, see, S, dP);
#pragma unroll
          for (int r = 0; r < 16; ++r) sum += S[r] * (dP[r] - delta);   // a correction of the rounded one
        }
      });
      delta += sum + __shfl_xor(sum, 32);
      __syncthreads();                               // the second sweep loads over the last tile
    }
    if (half == 0 && t < n) {
      a.delta[row + t] = delta;
      a.lse2[row + t] = lse2;
    }
    sweep([&](const unsigned char* Ks, const unsigned char* Vs, int s0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        bool see[16];
        f32x16 S, dP;
        sight(s0 + 32 * u, see);
        scores(Ks, Vs, u, see, S, dP);
        // ds rounded to bf16 for its product with k
#pragma unroll
        for (int r = 0; r < 16; ++r) S[r] = weighted(S[r], dP[r] - delta);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Frag<bf16> F;
          acc_frag(S, x, F);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) mma32(dQ[dt], Tile::col_frag(Ks, cb, dt, 32 * u + 16 * x), F);
        }
      }
    });
  }
  if (t < a.T) {
    if (t >= n) {
#pragma unroll
      for (int dt = 0; dt < DT; ++dt) dQ[dt] = zero16();
    }
    store_column<bf16, D>(reinterpret_cast<bf16*>(a.dq) + (row + t) * D, dQ, a.scale);
  }
}

// ------------------------------------------------------------------ bf16: dk, dv
// Workgroup = 64 keys: waves 0, 1 take 32 keys each with the first 32 tokens of every tile, waves 2,
// 3 the same keys with the last 32 (their sums are added at the end), so that a unit of work is
// half as long as with 128 keys: two rounds of units at the size above, not two and a short third (when
// they were halved, before the masks were decided ahead of the products, 695 -> 374 us; 285 now).
// Tiles of 64 tokens (q, dO, lse, delta) in two sets of LDS buffers.  Rows at and past t_hi read as
// zero throughout: p = 1 there, but dO = 0 and ds = 1 (0 - 0), so they add nothing.
constexpr int kDkRows = 64;

template <int D>
__global__ __launch_bounds__(256, 2) void swa_dkdv_bf16_kernel(SwaArgs a) {
  using Tile = SwzTile<D, kDkRows>;
  constexpr int KK = D / 16, DT = D / 32;
  __shared__ __align__(16) unsigned char Q0[Tile::bytes], Q1[Tile::bytes];
  __shared__ __align__(16) unsigned char G0[Tile::bytes], G1[Tile::bytes];
  __shared__ __align__(16) float L0[2 * kDkRows], L1[2 * kDkRows];     // lse (log2), delta
  const KeyUnit un = key_unit(a);
  const int G = a.Hq / a.Hkv, n = un.n, s0 = un.s0, t_lo = un.t_lo, t_hi = un.t_hi;
  const int lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int kb = wave & 1, th = wave >> 1;
  const int sw = s0 + 32 * kb, s = sw + (lane & 31);
  f32x16 dK[DT], dV[DT];
#pragma unroll
  for (int dt = 0; dt < DT; ++dt) {
    dK[dt] = zero16();
    dV[dt] = zero16();
  }
  if (t_lo < t_hi && s0 < n && un.h_lo < un.h_hi) {
    Frag<bf16> K[KK], V[KK];
    const size_t at = ((size_t)un.bk * a.T + min(s, n - 1)) * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) {
      K[kk] = load_frag(reinterpret_cast<const bf16*>(a.k) + at + 16 * kk);
      V[kk] = load_frag(reinterpret_cast<const bf16*>(a.v) + at + 16 * kk);
    }
    const float c = a.scale * kLog2e;
    const int nt = (t_hi - t_lo + kDkRows - 1) / kDkRows, total = nt * (un.h_hi - un.h_lo);
    const int rt = Tile::row_base() + 4096 * th, ct0 = Tile::col_base() + 4096 * th;   // (32 rows of a block)
    const int row0 = (un.b * a.Hq + (un.bk % a.Hkv) * G);
    int lg = un.h_lo, lt = 0;              // head and tile of the next load
    auto load = [&](unsigned char* Qs, unsigned char* Gs, float* Ls) {
      if (lg >= un.h_hi) return;
      const size_t row = (size_t)(row0 + lg) * a.T;
      const int tt = t_lo + lt * kDkRows;
      Tile::template load<4>(Qs, reinterpret_cast<const bf16*>(a.q) + row * D, tt, t_hi, wave);
      Tile::template load<4>(Gs, reinterpret_cast<const bf16*>(a.dO) + row * D, tt, t_hi, wave);
      if (wave < 2) {
        const float* src = (wave ? a.delta : a.lse2) + row + tt;
        const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<float*>(src), 0, uniform(min(t_hi - tt, kDkRows)) * 4, 0x00020000);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(Ls + kDkRows * wave), 4, 4 * lane, 0, 0, 0);
      }
      if (++lt == nt) {
        lt = 0;
        ++lg;
      }
    };
    auto step = [&](const unsigned char* Qs, const unsigned char* Gs, const float* Ls, int tile0) {
      const int tt = tile0 + 32 * th;
      if (!(sw > tt + 31 || (sw >= a.sinks && tt - (sw + 31) >= a.window))) {
        // what is seen, decided before the products: they and the exponentials then stand in one
        // stretch of code without branches, where the products run beside the vector work
        const bool full = sw + 31 <= tt && (tt + 31 - sw < a.window || sw + 32 <= a.sinks);
        bool see[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) see[r] = true;
        if (!full) {
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int t = tt + acc_row(r, half);
            see[r] = (s <= t) & ((t - s < a.window) | (s < a.sinks));
          }
        }
        f32x16 S = zero16(), dP = zero16();
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) mma32(S, Tile::row_frag(Qs, rt, 0, kk), K[kk]);
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) mma32(dP, Tile::row_frag(Gs, rt, 0, kk), V[kk]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 ls = *reinterpret_cast<const f32x4*>(Ls + 32 * th + 8 * q + 4 * half);
          const f32x4 de = *reinterpret_cast<const f32x4*>(Ls + kDkRows + 32 * th + 8 * q + 4 * half);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = __builtin_amdgcn_exp2f(S[4 * q + e] * c - ls[e]);
            S[4 * q + e] = see[4 * q + e] ? p : 0.f;
            dP[4 * q + e] = weighted(S[4 * q + e], dP[4 * q + e] - de[e]);
          }
        }
        // p and ds rounded to bf16 for their products with dO and q
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Frag<bf16> P, F;
          acc_frag(S, x, P);
          acc_frag(dP, x, F);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) mma32(dV[dt], Tile::col_frag(Gs, ct0, dt, 16 * x), P);
#pragma unroll
          for (int dt = 0; dt < DT; ++dt) mma32(dK[dt], Tile::col_frag(Qs, ct0, dt, 16 * x), F);
        }
      }
    };
    load(Q0, G0, L0);
    int ct = 0;                            // tile of the next step
    for (int i = 0; i < total; i += 2) {
      loads_and_barrier();
      load(Q1, G1, L1);
      step(Q0, G0, L0, t_lo + ct * kDkRows);
      ct = ct + 1 == nt ? 0 : ct + 1;
      loads_and_barrier();
      load(Q0, G0, L0);
      if (i + 1 < total) step(Q1, G1, L1, t_lo + ct * kDkRows);
      ct = ct + 1 == nt ? 0 : ct + 1;
    }
  }
  // add the sums of the two token halves, dK and then dV, through the tiles' memory
  float* park = reinterpret_cast<float*>(kb ? G0 : Q0);
  join_halves<D>(park, th, dK);
  join_halves<D>(park, th, dV);
  if (!th) store_key_grads<bf16, D>(a, un, s, kb, dK, dV);
}

// ------------------------------------------------------------------ fp32
// The same two passes with one tile in LDS (padded rows, staged through registers).
template <int D>
__global__ __launch_bounds__(256) void swa_dq_f32_kernel(SwaArgs a) {
  using T = float;
  using St = RowStage<T, kDqK, D, 256>;
  constexpr int LD = St::LD;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Ks = reinterpret_cast<T*>(smem);
  T* Vs = Ks + kDqK * LD;
  const DqUnit un = dq_unit(a, kDqQ);
  const int n = un.n, t0 = un.t0, lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int tw = t0 + 32 * wave, t = tw + (lane & 31);
  const size_t row = (size_t)(un.b * a.Hq + un.hq) * a.T;
  const T* kb = reinterpret_cast<const T*>(a.k) + (size_t)un.bk * a.T * D;
  const T* vb = reinterpret_cast<const T*>(a.v) + (size_t)un.bk * a.T * D;

  f32x16 dQ[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) dQ[dt] = zero16();
  if (t0 < n) {
    Frag<T> Q[D / 16], dO[D / 16];
    const size_t at = (row + min(t, n - 1)) * D + 8 * half;
    f32x16 od = zero16();
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      Q[kk] = load_frag(reinterpret_cast<const T*>(a.q) + at + 16 * kk);
      dO[kk] = load_frag(reinterpret_cast<const T*>(a.dO) + at + 16 * kk);
      mma32(od, load_frag(reinterpret_cast<const T*>(a.o) + at + 16 * kk), dO[kk]);
    }
    const float delta = diagonal(od);
    const float lse2 = log2_lse(a.lse[row + min(t, n - 1)]);
    if (half == 0 && t < n) {
      a.delta[row + t] = delta;
      a.lse2[row + t] = lse2;
    }
    const float c = a.scale * kLog2e;
    const KeyTiles<kDqK> tile(t0, min(t0 + kDqQ, n), a.window, a.sinks);
    St kst, vst;
    kst.load(kb, tile[0], tile.rows(0, n));
    vst.load(vb, tile[0], tile.rows(0, n));
    for (int i = 0; i < tile.count; ++i) {
      const int s0 = tile[i];
      __syncthreads();
      kst.store(Ks);
      vst.store(Vs);
      __syncthreads();
      if (i + 1 < tile.count) {
        kst.load(kb, tile[i + 1], tile.rows(i + 1, n));
        vst.load(vb, tile[i + 1], tile.rows(i + 1, n));
      }
#pragma unroll
      for (int u = 0; u < kDqK / 32; ++u) {
        const int su = s0 + 32 * u;
        if (su > tw + 31 || (su >= a.sinks && tw - (su + 31) >= a.window)) continue;
        f32x16 S = zero16(), dP = zero16();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          mma32(S, frag_rows32(Ks, LD, 32 * u, 16 * kk), Q[kk]);
          mma32(dP, frag_rows32(Vs, LD, 32 * u, 16 * kk), dO[kk]);
        }
        const bool full = su + 31 <= tw && (tw + 31 - su < a.window || su + 32 <= a.sinks);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float p = __builtin_amdgcn_exp2f(S[r] * c - lse2);
          if (!full) {
            const int s = su + acc_row(r, half);
            if (!(s <= t && (t - s < a.window || s < a.sinks))) p = 0.f;
          }
          S[r] = p == 0.f ? 0.f : p * (dP[r] - delta);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          Frag<T> F;
          acc_frag(S, x, F);       // ds rounded to the operand type for its product with k
#pragma unroll
          for (int dt = 0; dt < D / 32; ++dt) mma32(dQ[dt], frag_cols32(Ks, LD, 32 * dt, 32 * u + 16 * x), F);
        }
      }
    }
  }
  if (t < a.T) {
    if (t >= n) {
#pragma unroll
      for (int dt = 0; dt < D / 32; ++dt) dQ[dt] = zero16();
    }
    store_column<T, D>(reinterpret_cast<T*>(a.dq) + (row + t) * D, dQ, a.scale);
  }
}

constexpr int kDkQ = 64;

template <int D>
__global__ __launch_bounds__(256) void swa_dkdv_f32_kernel(SwaArgs a) {
  using T = float;
  using St = RowStage<T, kDkQ, D, 256>;
  constexpr int LD = St::LD;
  extern __shared__ __align__(16) unsigned char smem[];
  T* Qs = reinterpret_cast<T*>(smem);
  T* Gs = Qs + kDkQ * LD;                                  // dO
  float* Ls = reinterpret_cast<float*>(Gs + kDkQ * LD);    // lse in the log2 domain, delta
  const KeyUnit un = key_unit(a);
  const int G = a.Hq / a.Hkv, bk = un.bk, b = un.b, n = un.n, s0 = un.s0, t_lo = un.t_lo, t_hi = un.t_hi;
  const int lane = lane_id(), wave = wave_uid(), half = lane >> 5;
  const int kb = wave & 1, th = wave >> 1, sw = s0 + 32 * kb, s = sw + (lane & 31);
  f32x16 dK[D / 32], dV[D / 32];
#pragma unroll
  for (int dt = 0; dt < D / 32; ++dt) {
    dK[dt] = zero16();
    dV[dt] = zero16();
  }
  if (t_lo < t_hi && s0 < n && un.h_lo < un.h_hi) {
    Frag<T> K[D / 16], V[D / 16];
    const size_t at = ((size_t)bk * a.T + min(s, n - 1)) * D + 8 * half;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      K[kk] = load_frag(reinterpret_cast<const T*>(a.k) + at + 16 * kk);
      V[kk] = load_frag(reinterpret_cast<const T*>(a.v) + at + 16 * kk);
    }
    const float c = a.scale * kLog2e;
    const int nt = (t_hi - t_lo + kDkQ - 1) / kDkQ, total = nt * (un.h_hi - un.h_lo);
    St qst, gst;
    float lst = 0.f, dst = 0.f;
    auto load = [&](int i) {
      const int hq = (bk % a.Hkv) * G + un.h_lo + i / nt, tt = t_lo + (i % nt) * kDkQ;
      const size_t row = (size_t)(b * a.Hq + hq) * a.T;
      qst.load(reinterpret_cast<const T*>(a.q) + row * D, tt, t_hi);
      gst.load(reinterpret_cast<const T*>(a.dO) + row * D, tt, t_hi);
      if (threadIdx.x < kDkQ) {
        const int t = tt + threadIdx.x;
        // (past the end: p = exp2(. - inf) = 0)
        lst = t < t_hi ? a.lse2[row + t] : INFINITY;
        dst = t < t_hi ? a.delta[row + t] : 0.f;
      }
    };
    load(0);
    for (int i = 0; i < total; ++i) {
      const int tt = t_lo + (i % nt) * kDkQ + 32 * th;
      __syncthreads();
      qst.store(Qs);
      gst.store(Gs);
      if (threadIdx.x < kDkQ) {
        Ls[threadIdx.x] = lst;
        Ls[kDkQ + threadIdx.x] = dst;
      }
      __syncthreads();
      if (i + 1 < total) load(i + 1);
      if (sw > tt + 31 || (sw >= a.sinks && tt - (sw + 31) >= a.window)) continue;
      f32x16 S = zero16(), dP = zero16();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        mma32(S, frag_rows32(Qs, LD, 32 * th, 16 * kk), K[kk]);
        mma32(dP, frag_rows32(Gs, LD, 32 * th, 16 * kk), V[kk]);
      }
      const bool full = sw + 31 <= tt && (tt + 31 - sw < a.window || sw + 32 <= a.sinks);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 ls = *reinterpret_cast<const f32x4*>(Ls + 32 * th + 8 * q + 4 * half);
        const f32x4 de = *reinterpret_cast<const f32x4*>(Ls + kDkQ + 32 * th + 8 * q + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * q + e;
          float p = __builtin_amdgcn_exp2f(S[r] * c - ls[e]);
          if (!full) {
            const int t = tt + acc_row(r, half);
            if (!(s <= t && (t - s < a.window || s < a.sinks))) p = 0.f;
          }
          S[r] = p;
          dP[r] = p == 0.f ? 0.f : p * (dP[r] - de[e]);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Frag<T> P, F;              // p and ds rounded to the operand type for the products
        acc_frag(S, x, P);
        acc_frag(dP, x, F);
#pragma unroll
        for (int dt = 0; dt < D / 32; ++dt) {
          mma32(dV[dt], frag_cols32(Gs, LD, 32 * dt, 32 * th + 16 * x), P);
          mma32(dK[dt], frag_cols32(Qs, LD, 32 * dt, 32 * th + 16 * x), F);
        }
      }
    }
  }
  T* park = kb ? Gs : Qs;
  join_halves<D>(park, th, dK);
  join_halves<D>(park, th, dV);
  if (!th) store_key_grads<T, D>(a, un, s, kb, dK, dV);
}

// dk, dv of the tiles whose sums are in parts, added in order: the parts of the heads (or the tile's one
// sum), then, for sinks, the far ranges.  `tiles` of a key head, from the first.
template <typename T, int D>
__global__ __launch_bounds__(256) void swa_sink_kernel(SwaArgs a) {
  constexpr int KT = kSwaKeyTile, PR = D / 4;
  constexpr size_t one = 2 * KT * D;
  const int NK = (a.T + KT - 1) / KT, HP = a.n_head_part, tiles = HP > 1 ? NK : a.n_sink_tiles;
  const int kt = blockIdx.x % tiles, bk = blockIdx.x / tiles;
  const int n = seq_len(a.lens, bk / a.Hkv, a.T);
  const bool sink = kt < a.n_sink_tiles && a.n_far > 0;
  const float* far = a.part + ((size_t)bk * a.n_sink_tiles + kt) * (1 + a.n_far) * one;
  const float* src = HP > 1 ? a.head_part + ((size_t)bk * NK + kt) * HP * one : far;
  for (int i = blockIdx.y * 256 + threadIdx.x; i < 2 * KT * PR; i += 256 * gridDim.y) {
    const int which = i / (KT * PR), r = (i / PR) % KT, s = kt * KT + r;
    if (s >= a.T) continue;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
    const int last = sink && s < a.sinks ? a.n_far : 0;
    if (s < n) {
#pragma unroll 4
      for (int f = 0; f < HP; ++f) x += load4f(src + (size_t)f * one + (size_t)i * 4);
#pragma unroll 4
      for (int f = 1; f <= last; ++f) x += load4f(far + (size_t)f * one + (size_t)i * 4);
    }
    T* dst = reinterpret_cast<T*>(which ? a.dv : a.dk);
    store4(dst + ((size_t)bk * a.T + s) * D + 4 * (i % PR), x);
  }
}

template <typename T, int D>
static hipError_t launch(const SwaArgs& a, hipStream_t st) {
  const dim3 grid_q(a.B * a.Hq * ((a.T + kDqQ - 1) / kDqQ));
  const int NK = (a.T + kSwaKeyTile - 1) / kSwaKeyTile;
  const dim3 grid_k(a.B * a.Hkv * (NK * a.n_head_part + a.n_sink_tiles * a.n_far));
  hipError_t e;
  if constexpr (sizeof(T) == 2) {
    e = launch_kernel<0>(swa_dq_bf16_kernel<D>, grid_q, 256, a, st);
    if (e == hipSuccess) e = launch_kernel<0>(swa_dkdv_bf16_kernel<D>, grid_k, 256, a, st);
  } else {
    constexpr size_t lds_q = sizeof(T) * 2 * kDqK * RowStage<T, kDqK, D, 256>::LD;
    constexpr size_t lds_k = sizeof(T) * 2 * kDkQ * RowStage<T, kDkQ, D, 256>::LD + sizeof(float) * 2 * kDkQ;
    e = launch_kernel<lds_q>(swa_dq_f32_kernel<D>, grid_q, 256, a, st);
    if (e == hipSuccess) e = launch_kernel<lds_k>(swa_dkdv_f32_kernel<D>, grid_k, 256, a, st);
  }
  const int tiles = a.n_head_part > 1 ? NK : a.n_sink_tiles * (a.n_far > 0);
  if (e != hipSuccess || tiles == 0) return e;
  return launch_kernel<0>(swa_sink_kernel<T, D>, dim3(a.B * a.Hkv * tiles, 8), 256, a, st);
}

hipError_t launch_swa_bwd(const SwaArgs& a, hipStream_t st) {
  if (a.dtype) return a.D == 128 ? launch<bf16, 128>(a, st) : launch<bf16, 64>(a, st);
  return a.D == 128 ? launch<float, 128>(a, st) : launch<float, 64>(a, st);
}

}  // namespace carve
