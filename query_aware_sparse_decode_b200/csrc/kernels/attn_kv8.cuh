// Attention and soft-vote logits over 8-bit K/V caches (kv8.cuh): the
// formulas of attn.cuh and softvote.cuh with
//
//   K[t] = ks[t/16] * kcode[t],   V[t] = vs[t/16] * vcode[t].
//
// The scales enter after the dot product (logit = (q . kcode) ks) and in the
// weight of the value row (p vs), so no row is expanded in memory.
#pragma once

#include "attn.cuh"
#include "kv8.cuh"
#include "softvote.cuh"

namespace tb {

struct AttnKv8Params : AttnParams {
  const float* k_scale;  // one per 16 cache rows
  const float* v_scale;
};

constexpr int kKv8ListBytes = ((kAttnMaxChunk + kAttnTile) * 5 + 15) / 16 * 16;
template <int D, int GS>
constexpr int attn_kv8_f32_smem() { return kKv8ListBytes + kAttnWarps * GS * (D + 2) * 4; }

// The gather list of a sub-chunk, page ids checked: a token whose page is not
// one of the pool's is listed without a head (nothing reads its codes as a
// selected row) and flags TB_DEV_ERR_INDEX.
template <int GS>
__device__ __forceinline__ int build_union_list_kv8(const AttnKv8Params& p, int b, int g, int t0, int t1,
                                                    int32_t* list_idx, uint8_t* list_hb, uint32_t* scan_sm) {
  return build_union<GS>(p, b, g, t0, t1, scan_sm, [&](int pos, int t, uint32_t hb) {
    uint32_t row;
    if (!kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t, &row)) {
      atomicOr(p.status, TB_DEV_ERR_INDEX);
      hb = 0u;
    }
    list_idx[pos] = (int32_t)row;
    list_hb[pos] = (uint8_t)hb;
  });
}

// fp32 queries, fp32 FMA: one warp per token at a time, lane owns D/32 consecutive dims.
template <int FMT, int D, int GS>
__global__ void __launch_bounds__(kAttnThreads) attn_kv8_f32_kernel(const AttnKv8Params p) {
  pdl_wait();
  pdl_trigger();
  constexpr int DPL = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  int32_t* list_idx = reinterpret_cast<int32_t*>(smem);
  uint8_t* list_hb = reinterpret_cast<uint8_t*>(list_idx + kAttnMaxChunk + kAttnTile);
  float* wm = reinterpret_cast<float*>(smem + kKv8ListBytes);
  float* wl = wm + kAttnWarps * GS;
  float* wo = wl + kAttnWarps * GS;
  __shared__ uint32_t scan_sm[32];
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = p.lens[b];
  const int t0 = split * p.chunk;
  if (t0 >= L) return;
  const int t1 = min(t0 + p.chunk, L);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint8_t* Kb = reinterpret_cast<const uint8_t*>(p.k_cache) + lane * DPL;
  const uint8_t* Vb = reinterpret_cast<const uint8_t*>(p.v_cache) + lane * DPL;
  float q[GS][DPL], o[GS][DPL], m[GS], l[GS];
#pragma unroll
  for (int hh = 0; hh < GS; ++hh) {
    m[hh] = kNegInf;
    l[hh] = 0.f;
#pragma unroll
    for (int j = 0; j < DPL; ++j) {
      q[hh][j] = reinterpret_cast<const float*>(p.q)[((size_t)b * p.Hq + g * GS + hh) * D + lane * DPL + j];
      o[hh][j] = 0.f;
    }
  }
  for (int sc0 = t0; sc0 < t1; sc0 += kAttnMaxChunk) {
    const int n = build_union_list_kv8<GS>(p, b, g, sc0, min(sc0 + kAttnMaxChunk, t1), list_idx, list_hb, scan_sm);
    for (int i = warp; i < n; i += kAttnWarps) {
      const uint32_t row = (uint32_t)list_idx[i];
      const uint32_t hb = list_hb[i];
      const float ks = p.k_scale[row >> 4] * p.scale_log2, vs = p.v_scale[row >> 4];
      float kv[DPL], vv[DPL];
#pragma unroll
      for (int j = 0; j < DPL; ++j) {
        kv[j] = kv8_decode<FMT>(Kb[(size_t)row * D + j]);
        vv[j] = kv8_decode<FMT>(Vb[(size_t)row * D + j]) * vs;
      }
#pragma unroll
      for (int hh = 0; hh < GS; ++hh) {
        if (!((hb >> hh) & 1u)) continue;
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < DPL; ++j) dot = fmaf(q[hh][j], kv[j], dot);
#pragma unroll
        for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        const float s = dot * ks;
        const float mn = fmaxf(m[hh], s);
        const float alpha = exp2f(m[hh] - mn), pw = exp2f(s - mn);
        l[hh] = l[hh] * alpha + pw;
#pragma unroll
        for (int j = 0; j < DPL; ++j) o[hh][j] = o[hh][j] * alpha + pw * vv[j];
        m[hh] = mn;
      }
    }
    __syncthreads();  // the gather list is free for the next sub-chunk
  }
#pragma unroll
  for (int hh = 0; hh < GS; ++hh) {
    if (lane == 0) {
      wm[warp * GS + hh] = m[hh];
      wl[warp * GS + hh] = l[hh];
    }
#pragma unroll
    for (int j = 0; j < DPL; ++j) wo[(warp * GS + hh) * D + lane * DPL + j] = o[hh][j];
  }
  __syncthreads();
  write_partial<D, GS>(p, b, g, split, wm, wl, wo);
}

// ---------------------------------------------------------------- tensor cores
// D(16x8, f32) += A(16x16, f16, row) * B(16x8, f16, col)
__device__ __forceinline__ void mma_16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// The four codes of a word as two fp16 pairs (exact): e4m3 by conversion;
// int8 by placing code + 128 in the low mantissa bits of 1024 and
// subtracting 1152.
template <int FMT>
__device__ __forceinline__ void kv8_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == kFmtE4m3) {
    lo = e4m3x2_to_f16x2((uint16_t)(w & 0xFFFFu));
    hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), c = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(c), "r"(0x64806480u));
  }
}
// cache codes: read once, straight from L2 into registers
__device__ __forceinline__ uint4 ld_codes16(const uint8_t* p) {
  uint4 v;
  asm("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_codes8(const uint8_t* p) {
  uint2 v;
  asm("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// The bf16 queries of a group as fp16 B fragments of S^T = K Q^T.  Lane
// (grp, tq) of head grp holds dims 64i + 16tq + 4j + {0,1 | 2,3} in
// fragment 4i + j: the dims of the 16-byte pieces it loads of a K row (the
// order of the k indices of a product is free as long as both sides share it).
// Each head's row is scaled by a power of two that brings its largest
// magnitude to [2^14, 2^15): products with the codes are then exact in the
// fp32 accumulator's inputs (a bf16 has 8 significant bits, and only
// elements 2^-28 below the row's largest lose any).  qs[e] is the inverse
// scale of head 2tq + e, whose logits the lane receives.
template <int D, int GS>
__device__ __forceinline__ void load_q_f16(const void* q, size_t head0, int grp, int tq, uint32_t (&qb)[D / 16][2],
                                           float (&qs)[2]) {
  float x[D / 16][4];
  float amax = 0.f;
  const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(q) + (head0 + (grp < GS ? grp : 0)) * D;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint2 w = *reinterpret_cast<const uint2*>(row + 64 * (kk / 4) + 16 * tq + 4 * (kk % 4));
    x[kk][0] = __uint_as_float(w.x << 16);
    x[kk][1] = __uint_as_float(w.x & 0xFFFF0000u);
    x[kk][2] = __uint_as_float(w.y << 16);
    x[kk][3] = __uint_as_float(w.y & 0xFFFF0000u);
#pragma unroll
    for (int u = 0; u < 4; ++u) amax = fmaxf(amax, fabsf(x[kk][u]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int ex = (int)(__float_as_uint(amax) >> 23) - 127;
  const int up = min(14 - ex, 126);  // the exponent added to the row
  const float f = grp < GS ? kv8_pow2(up) : 0.f;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    qb[kk][0] = grp < GS ? pack_f16(x[kk][0] * f, x[kk][1] * f) : 0u;
    qb[kk][1] = grp < GS ? pack_f16(x[kk][2] * f, x[kk][3] * f) : 0u;
  }
  qs[0] = kv8_pow2(-__shfl_sync(0xffffffffu, up, (8 * tq) & 31));
  qs[1] = kv8_pow2(-__shfl_sync(0xffffffffu, up, (8 * tq + 4) & 31));
}

template <int D, int GS>
constexpr int attn_kv8_smem() {
  constexpr int list = (kAttnMaxChunk + kAttnTile) * 6 + (kAttnMaxChunk / kKv8Block) * 8;
  constexpr int merge = kAttnWarps * GS * (D + 2) * 4;
  return list > merge ? list : merge;
}

// bf16 queries over 8-bit codes.  As in attn_bf16_kernel a warp takes 16
// listed tokens at a time as the M rows of S^T = K Q^T and the K dimension of
// O^T = V^T P^T, on mma.sync m16n8k16 with fp16 operands (both formats' codes
// are exact in fp16) and fp32 accumulators.  The codes go from global memory
// straight into the registers of the A fragments:
//  - K: lane (grp, tq) loads 16-byte pieces of rows grp and grp + 8; a word
//    (4 dims) is one k-step's share of a lane, so no shuffle or shared memory;
//  - V: it loads D/8 bytes (dims grp D/8 ..) of token rows 2tq, 2tq+1, 2tq+8,
//    2tq+9; byte permutes pair the tokens of a dim, and m-tile mt takes dims
//    grp D/8 + 2mt and + 2mt + 1 as its rows grp and grp + 8.
// The next tile's K is requested when S is done, its V when O is done.
//
// Softmax (log2 domain, fp32): l sums p = 2^(x - m); the weights of the V
// codes are w = 2^(x + log2 vs - r + 7) with their own running exponent r, so
// that fp16 holds them whatever the blocks' scales are.  m and r need
// not be the exact maxima: they are raised only when a logit passes them by
// 8 (p <= 2^8, w <= 2^15), which after the first tiles is rare, and saves the
// cross-lane maximum of every tile.  Weights keep fp16's 11 bits down to
// 2^-21 of the largest one.
template <int FMT, int D, int GS>
__global__ void __launch_bounds__(kAttnThreads, 4) attn_kv8_kernel(const AttnKv8Params p) {
  pdl_wait();
  pdl_trigger();
  static_assert(D == 64 || D == 128, "head dim");
  constexpr int KSTEPS = D / 16, MT = D / 16;
  constexpr int KLD = D / 64;  // 16-byte loads of a K row per lane
  constexpr int VW = D / 32;   // words of a V row per lane
  extern __shared__ __align__(128) uint8_t smem[];
  int32_t* list_idx = reinterpret_cast<int32_t*>(smem);
  float2* tab = reinterpret_cast<float2*>(list_idx + kAttnMaxChunk + kAttnTile);  // per block: ks log2e/sqrt(D), log2 vs
  uint16_t* list_hb = reinterpret_cast<uint16_t*>(tab + kAttnMaxChunk / kKv8Block);
  __shared__ uint32_t scan_sm[32];
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = p.lens[b];
  const int t0 = split * p.chunk;
  if (t0 >= L) return;
  const int t1 = min(t0 + p.chunk, L);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tq = lane & 3;
  const uint8_t* Kb = reinterpret_cast<const uint8_t*>(p.k_cache) + 16 * tq;
  const uint8_t* Vb = reinterpret_cast<const uint8_t*>(p.v_cache) + grp * (D / 8);

  uint32_t qb[KSTEPS][2];
  float qs[2];
  load_q_f16<D, GS>(p.q, (size_t)b * p.Hq + g * GS, grp, tq, qb, qs);
  const uint32_t head_bits = ((1u << GS) - 1u) >> (2 * tq) & 3u;

  float o[MT][4];  // dims grp D/8 + 2mt (+1), heads 2tq + {0,1}
#pragma unroll
  for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m_run[2] = {kNegInf, kNegInf}, r_run[2] = {kNegInf, kNegInf}, l_run[2] = {0.f, 0.f};

  for (int sc0 = t0; sc0 < t1; sc0 += kAttnMaxChunk) {
    const int sc1 = min(sc0 + kAttnMaxChunk, t1);
    {  // the sub-chunk's block scales: at most one block per thread
      const int t = sc0 + tid * kKv8Block;
      uint32_t row;
      if (t < sc1 && kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t, &row))
        tab[tid] = make_float2(p.k_scale[row >> 4] * p.scale_log2, __log2f(p.v_scale[row >> 4]));
    }
    const int n = build_union<GS>(p, b, g, sc0, sc1, scan_sm, [&](int pos, int t, uint32_t hb) {
      uint32_t row;
      if (!kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t, &row)) {
        atomicOr(p.status, TB_DEV_ERR_INDEX);
        hb = 0u;
      }
      list_idx[pos] = (int32_t)row;
      list_hb[pos] = (uint16_t)(hb | (uint32_t)(t - sc0) / kKv8Block << 8);
    });
    const int ntiles = (n + kAttnTile - 1) / kAttnTile;
    uint4 kc[2][KLD];
    uint32_t vc[4][VW];
    auto load_k = [&](int tile) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* src = Kb + (size_t)(uint32_t)list_idx[tile * kAttnTile + grp + 8 * r] * D;
#pragma unroll
        for (int i = 0; i < KLD; ++i) kc[r][i] = ld_codes16(src + 64 * i);
      }
    };
    auto load_v = [&](int tile) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int2 rows = *reinterpret_cast<const int2*>(list_idx + tile * kAttnTile + 2 * tq + 8 * r);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint8_t* src = Vb + (size_t)(uint32_t)(e ? rows.y : rows.x) * D;
          if constexpr (VW == 4) {
            const uint4 v = ld_codes16(src);
            vc[2 * r + e][0] = v.x;
            vc[2 * r + e][1] = v.y;
            vc[2 * r + e][2] = v.z;
            vc[2 * r + e][3] = v.w;
          } else {
            const uint2 v = ld_codes8(src);
            vc[2 * r + e][0] = v.x;
            vc[2 * r + e][1] = v.y;
          }
        }
      }
    };
    if (warp < ntiles) {
      load_k(warp);
      load_v(warp);
    }
    for (int tile = warp; tile < ntiles; tile += kAttnWarps) {
      const bool more = tile + kAttnWarps < ntiles;
      // ---- S^T = K Q^T: s[0..1] = token grp, s[2..3] = token grp + 8; heads 2tq + {0,1}
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KLD; ++i) {
        const uint32_t wa[4] = {kc[0][i].x, kc[0][i].y, kc[0][i].z, kc[0][i].w};
        const uint32_t wb[4] = {kc[1][i].x, kc[1][i].y, kc[1][i].z, kc[1][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          kv8_to_f16<FMT>(wa[j], a0, a2);
          kv8_to_f16<FMT>(wb[j], a1, a3);
          mma_16816_f16(s, a0, a1, a2, a3, qb[4 * i + j][0], qb[4 * i + j][1]);
        }
      }
      if (more) load_k(tile + kAttnWarps);
      const uint32_t e0 = list_hb[tile * kAttnTile + grp], e1 = list_hb[tile * kAttnTile + grp + 8];
      const float2 c0 = tab[e0 >> 8], c1 = tab[e1 >> 8];
      const uint32_t hb0 = (e0 & 0xFFu) >> (2 * tq) & head_bits, hb1 = (e1 & 0xFFu) >> (2 * tq) & head_bits;
      float x[4];
      x[0] = (hb0 & 1u) ? s[0] * qs[0] * c0.x : kNegInf;
      x[1] = (hb0 & 2u) ? s[1] * qs[1] * c0.x : kNegInf;
      x[2] = (hb1 & 1u) ? s[2] * qs[0] * c1.x : kNegInf;
      x[3] = (hb1 & 2u) ? s[3] * qs[1] * c1.x : kNegInf;
      const float y[4] = {x[0] + c0.y, x[1] + c0.y, x[2] + c1.y, x[3] + c1.y};
      float mt[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
      float rt[2] = {fmaxf(y[0], y[2]), fmaxf(y[1], y[3])};
      const bool over = mt[0] > m_run[0] + 8.f || mt[1] > m_run[1] + 8.f || rt[0] > r_run[0] + 8.f ||
                        rt[1] > r_run[1] + 8.f;
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) {
            mt[e] = fmaxf(mt[e], __shfl_xor_sync(0xffffffffu, mt[e], sh));
            rt[e] = fmaxf(rt[e], __shfl_xor_sync(0xffffffffu, rt[e], sh));
          }
          const float mn = fmaxf(m_run[e], mt[e]), rn = fmaxf(r_run[e], rt[e]);
          // a head with no token so far has l = 0 and o = 0: any factor serves
          l_run[e] *= m_run[e] == mn ? 1.f : fast_exp2(m_run[e] - mn);
          const float al = r_run[e] == rn ? 1.f : fast_exp2(r_run[e] - rn);
          m_run[e] = mn;
          r_run[e] = rn;
#pragma unroll
          for (int j = 0; j < MT; ++j) {
            o[j][e] *= al;
            o[j][2 + e] *= al;
          }
        }
      }
      // a head with no kept token so far subtracts 0: every exponent is -inf
      const float mu0 = m_run[0] == kNegInf ? 0.f : m_run[0], mu1 = m_run[1] == kNegInf ? 0.f : m_run[1];
      const float ru0 = r_run[0] == kNegInf ? 0.f : r_run[0] - 7.f, ru1 = r_run[1] == kNegInf ? 0.f : r_run[1] - 7.f;
      l_run[0] += fast_exp2(x[0] - mu0) + fast_exp2(x[2] - mu0);
      l_run[1] += fast_exp2(x[1] - mu1) + fast_exp2(x[3] - mu1);
      const uint32_t pb0 = movmatrix_trans(pack_f16(fast_exp2(y[0] - ru0), fast_exp2(y[1] - ru1)));
      const uint32_t pb1 = movmatrix_trans(pack_f16(fast_exp2(y[2] - ru0), fast_exp2(y[3] - ru1)));
      // ---- O^T += V^T P^T
#pragma unroll
      for (int j = 0; j < VW; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // bytes 2h and 2h + 1 of the word: m-tile 2j + h
          const uint32_t sel = h ? 0x7362 : 0x5140;
          uint32_t a0, a1, a2, a3;
          kv8_to_f16<FMT>(__byte_perm(vc[0][j], vc[1][j], sel), a0, a1);
          kv8_to_f16<FMT>(__byte_perm(vc[2][j], vc[3][j], sel), a2, a3);
          mma_16816_f16(o[2 * j + h], a0, a1, a2, a3, pb0, pb1);
        }
      }
      if (more) load_v(tile + kAttnWarps);
    }
    __syncthreads();  // the gather list is free for the next sub-chunk
  }

  // ---- merge the four warps through shared memory (the list's)
  float* wm = reinterpret_cast<float*>(smem);
  float* wl = wm + kAttnWarps * GS;
  float* wo = wl + kAttnWarps * GS;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], sh);
    const int h = 2 * tq + e;
    if (h < GS) {
      if (grp == 0) {
        wm[warp * GS + h] = m_run[e];
        wl[warp * GS + h] = l_run[e];
      }
      // back from the weights' exponent to m's
      const float f = r_run[e] == kNegInf ? 0.f : exp2f(r_run[e] - 7.f - m_run[e]);
      float* dst = wo + (warp * GS + h) * D + grp * (D / 8);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        dst[2 * j] = o[j][e] * f;
        dst[2 * j + 1] = o[j][2 + e] * f;
      }
    }
  }
  __syncthreads();
  write_partial<D, GS>(p, b, g, split, wm, wl, wo);
}

struct VoteKv8Params : VoteParams {
  const float* k_scale;
  uint32_t* status;
};

// Soft-vote logits (log2 domain) and per-chunk (max, sum) pairs over 8-bit
// keys; softvote_reduce_kernel follows.  S^T = K Q^T as in attn_kv8_kernel, over
// consecutive tokens: a tile of 16 is one block of the cache, so it has one
// scale and one row lookup.  A warp keeps the next kVoteKv8Ahead tiles' codes
// in flight in registers.
constexpr int kVoteKv8Ahead = 2;
template <int FMT, int D, int GS>
__global__ void __launch_bounds__(kVoteThreads, 4) softvote_kv8_logits_kernel(const VoteKv8Params p) {
  pdl_wait();
  pdl_trigger();
  constexpr int KLD = D / 64;
  constexpr int AHEAD = kVoteKv8Ahead;
  __shared__ float wm[kVoteWarps * GS], wl[kVoteWarps * GS];
  const int chunk = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = p.lens[b];
  const int t0 = chunk * p.chunk;
  if (t0 >= L) return;
  const int t1 = min(t0 + p.chunk, L);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tq = lane & 3;
  const uint8_t* Kb = reinterpret_cast<const uint8_t*>(p.k_cache) + 16 * tq;
  uint32_t qb[D / 16][2];
  float qs[2];
  load_q_f16<D, GS>(p.q, (size_t)b * p.Hq + g * GS, grp, tq, qb, qs);
  const int hp = 2 * tq;
  const bool real[2] = {hp < GS, hp + 1 < GS};
  float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};  // over the lane's tokens
  float* lrow[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    lrow[e] = p.logits + ((size_t)b * p.Hq + g * GS + (real[e] ? hp + e : 0)) * p.max_len;

  uint4 kc[AHEAD][2][KLD];
  float ks[AHEAD];
  // tile tt: rows of one block; rows past the chunk's end repeat its last one; a
  // page outside the pool leaves scale NaN, which marks the tile
  auto load = [&](int slot, int tt) {
    uint32_t row;
    const bool ok = kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, tt, &row);
    if (!ok && lane == 0) atomicOr(p.status, TB_DEV_ERR_INDEX);
    const int last = ok ? t1 - 1 - tt : 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t* src = Kb + (size_t)(row + min(grp + 8 * r, last)) * D;
#pragma unroll
      for (int i = 0; i < KLD; ++i) kc[slot][r][i] = ld_codes16(src + 64 * i);
    }
    ks[slot] = ok ? p.k_scale[row >> 4] * p.scale_log2 : __int_as_float(0x7fffffff);
  };
  const int stride = kVoteWarps * kAttnTile;
  int tt = t0 + warp * kAttnTile;
#pragma unroll
  for (int u = 0; u < AHEAD; ++u)
    if (tt + u * stride < t1) load(u, tt + u * stride);
  for (; tt < t1; tt += AHEAD * stride) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int tc = tt + u * stride;
      if (tc >= t1) break;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KLD; ++i) {
        const uint32_t wa[4] = {kc[u][0][i].x, kc[u][0][i].y, kc[u][0][i].z, kc[u][0][i].w};
        const uint32_t wb[4] = {kc[u][1][i].x, kc[u][1][i].y, kc[u][1][i].z, kc[u][1][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          kv8_to_f16<FMT>(wa[j], a0, a2);
          kv8_to_f16<FMT>(wb[j], a1, a3);
          mma_16816_f16(s, a0, a1, a2, a3, qb[4 * i + j][0], qb[4 * i + j][1]);
        }
      }
      const float sc = ks[u];
      if (tc + AHEAD * stride < t1) load(u, tc + AHEAD * stride);
      const bool in[2] = {tc + grp < t1 && sc == sc, tc + grp + 8 < t1 && sc == sc};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float xa = in[0] ? s[e] * qs[e] * sc : kNegInf, xb = in[1] ? s[2 + e] * qs[e] * sc : kNegInf;
        if (real[e]) {
          if (tc + grp < t1) lrow[e][tc + grp] = xa;
          if (tc + grp + 8 < t1) lrow[e][tc + grp + 8] = xb;
        }
        const float mn = fmaxf(m[e], fmaxf(xa, xb));
        if (mn != kNegInf) {
          l[e] = l[e] * fast_exp2(m[e] - mn) + fast_exp2(xa - mn) + fast_exp2(xb - mn);
          m[e] = mn;
        }
      }
    }
  }
  // merge the lanes' pairs of each head (the 8 lanes with the same tq)
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m[e], sh), l2 = __shfl_xor_sync(0xffffffffu, l[e], sh);
      const float mn = fmaxf(m[e], m2);
      if (mn != kNegInf) {
        l[e] = (m[e] == kNegInf ? 0.f : l[e] * exp2f(m[e] - mn)) + (m2 == kNegInf ? 0.f : l2 * exp2f(m2 - mn));
        m[e] = mn;
      }
    }
    if (grp == 0 && real[e]) {
      wm[warp * GS + hp + e] = m[e];
      wl[warp * GS + hp + e] = l[e];
    }
  }
  __syncthreads();
  if (tid < GS) {
    float M = kNegInf;
    for (int w = 0; w < kVoteWarps; ++w) M = fmaxf(M, wm[w * GS + tid]);
    float sum = 0.f;
    if (M != kNegInf)
      for (int w = 0; w < kVoteWarps; ++w)
        if (wm[w * GS + tid] != kNegInf) sum += wl[w * GS + tid] * exp2f(wm[w * GS + tid] - M);
    const size_t ph = (((size_t)b * p.Hq + g * GS + tid) * p.nchunk + chunk) * 2;
    p.stats[ph] = M;
    p.stats[ph + 1] = sum;
  }
}

}  // namespace tb
