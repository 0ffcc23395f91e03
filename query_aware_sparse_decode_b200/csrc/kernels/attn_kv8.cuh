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

// Split of the 8-bit attention (host side): the shortest chunks (whole mask
// words) that keep all of the call's CTAs in one wave of kKv8CtasPerSm per SM,
// counting the tokens that each sequence has.
constexpr int kKv8CtasPerSm = 4;
constexpr int kKv8MinChunk = 128;
inline void attn_split_kv8(int num_sms, int kv_heads, const int* lens, int batch, int max_splits, int* chunk_out,
                           int* nsplit_out) {
  long long total = 0;
  int longest = 1;
  for (int b = 0; b < batch; ++b) {
    total += lens[b];
    longest = lens[b] > longest ? lens[b] : longest;
  }
  const long long slots = (long long)kKv8CtasPerSm * num_sms;
  long long chunk = (total * kv_heads + slots - 1) / slots;
  const long long least = (longest + max_splits - 1) / max_splits;
  chunk = chunk < least ? least : chunk;
  chunk = chunk < kKv8MinChunk ? kKv8MinChunk : (chunk + 31) / 32 * 32;
  for (;;) {
    long long n = 0, next = longest + 31;  // the CTAs, and the next chunk that has fewer
    for (int b = 0; b < batch; ++b) {
      const long long ns = (lens[b] + chunk - 1) / chunk;
      n += ns;
      if (ns > 1) {
        const long long c = ((lens[b] + ns - 2) / (ns - 1) + 31) / 32 * 32;
        next = c < next ? c : next;
      }
    }
    if (n * kv_heads <= slots || chunk >= longest) break;
    chunk = next > chunk ? next : chunk + 32;
  }
  *chunk_out = (int)chunk;
  *nsplit_out = (int)((longest + chunk - 1) / chunk);
}

constexpr int kKv8ListBytes = ((kAttnMaxChunk + kAttnTile) * 5 + 15) / 16 * 16;
template <int D, int GS>
constexpr int attn_kv8_f32_smem() { return kKv8ListBytes + kAttnWarps * GS * (D + 2) * 4; }

// The gather list of a sub-chunk, page ids checked: a token whose page is not
// one of the pool's is listed without a head (nothing reads its codes as a
// selected row) and flags TB_DEV_ERR_INDEX.
template <int GS>
__device__ __forceinline__ int build_union_list_kv8(const AttnKv8Params& p, int b, int g, int t0, int t1,
                                                    int32_t* list_idx, uint8_t* list_hb, uint32_t* scan_sm) {
  return build_union<GS, kAttnMaxChunk, kAttnTile>(p, b, g, t0, t1, scan_sm, [&](int pos, int t, uint32_t hb) {
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

// Ring of one warp: kKv8Stages stages of 32 tokens.
constexpr int kKv8Stages = 3;
constexpr int kKv8Tok = 16;       // tokens of an iteration
constexpr int kKv8MaxList = 1024; // tokens per gather list
template <int D>
constexpr int kv8_stage_bytes() { return 2 * kKv8Tok * D; }
template <int D, int GS, bool DENSE>
constexpr int attn_kv8_smem() {
  constexpr int ring = kAttnWarps * kKv8Stages * (kv8_stage_bytes<D>() + (DENSE ? kKv8Tok / 2 : 0));
  constexpr int list = DENSE ? 0 : (kKv8MaxList + kKv8Tok) * 6 + (kKv8MaxList / kKv8Block) * 8;
  constexpr int merge = kAttnWarps * GS * (D + 2) * 4;
  return ring + list > merge ? ring + list : merge;
}
// 16-byte pieces of a cached row are stored at piece ^ swizzle(row), so that the
// lanes of a shared-memory phase touch different banks: for K two rows' pieces
// tq, for V rows 0, 2, 4, 6 (+ 1) of two neighbouring pieces.
template <int D>
__device__ __forceinline__ int kv8_swizzle_k(int row) { return D == 128 ? (row & 1) << 2 : 0; }
template <int D>
__device__ __forceinline__ int kv8_swizzle_v(int row) { return D == 128 ? row & 6 : (row >> 1) & 3; }
__device__ __forceinline__ void cp_async_4(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_16u(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// bf16 queries over 8-bit codes.  As in attn_bf16_kernel a warp takes 16
// tokens at a time as the M rows of S^T = K Q^T and the K dimension of
// O^T = V^T P^T, on mma.sync m16n8k16 with fp16 operands (both formats' codes
// are exact in fp16) and fp32 accumulators.  The codes reach the A fragments
// without ldmatrix or shuffles:
//  - K: lane (grp, tq) takes 16-byte pieces of rows grp and grp + 8; a word
//    (4 dims) is one k-step's share of a lane;
//  - V: it takes D/8 bytes (dims grp D/8 ..) of token rows 2tq, 2tq+1, 2tq+8,
//    2tq+9; byte permutes pair the tokens of a dim, and m-tile mt takes dims
//    grp D/8 + 2mt and + 2mt + 1 as its rows grp and grp + 8.
// Two tiles an iteration: their products and conversions are independent, which
// a warp needs more than bytes in flight (one tile at a time was a chain of about
// 2100 cycles).  A ring of kKv8Stages iterations per warp holds the loads.  Rows
// are copied whole (eight lanes a 128-byte row: four lanes that took a sector each of
// four rows made L2 send half as much again).
//
// DENSE takes every token of the chunk: tiles are blocks of the cache, so one
// row lookup and one scale pair serve a tile and there is no gather list.
// Otherwise the union of the group's masks is listed as in attn_bf16_kernel,
// with each token's block in the sub-chunk beside its head bits.
//
// Softmax (log2 domain, fp32): l sums p = 2^(x - m); the weights of the V
// codes are w = 2^(x + log2 vs - r + 7) with their own running exponent r, so
// that fp16 holds them whatever the blocks' scales are.  m and r need
// not be the exact maxima: they are raised only when a logit passes them by
// 8 (p <= 2^8, w <= 2^15), which after the first tiles is rare, and saves the
// cross-lane maximum of every tile.  Weights keep fp16's 11 bits down to
// 2^-21 of the largest one.
template <int FMT, int D, int GS, bool DENSE>
__global__ void __launch_bounds__(kAttnThreads, kKv8CtasPerSm) attn_kv8_kernel(const AttnKv8Params p) {
  pdl_wait();
  pdl_trigger();
  static_assert(D == 64 || D == 128, "head dim");
  constexpr int KSTEPS = D / 16, MT = D / 16;
  constexpr int KLD = D / 64;                   // 16-byte pieces of a K row per lane
  constexpr int VW = D / 32, VB = D / 8;        // words and bytes of a V row per lane
  constexpr int U = kKv8Tok / 16;               // mma tiles of an iteration
  constexpr int VOFF = kKv8Tok * D;             // V slots of a stage
  constexpr int STAGE = kv8_stage_bytes<D>();
  extern __shared__ __align__(128) uint8_t smem[];
  int32_t* list_idx = reinterpret_cast<int32_t*>(smem + kAttnWarps * kKv8Stages * STAGE);
  float2* tab = reinterpret_cast<float2*>(list_idx + kKv8MaxList + kKv8Tok);  // per block: ks log2e/sqrt(D), log2 vs
  uint16_t* list_hb = reinterpret_cast<uint16_t*>(tab + kKv8MaxList / kKv8Block);
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = p.lens[b];
  const int t0 = split * p.chunk;
  if (t0 >= L) return;
  const int t1 = min(t0 + p.chunk, L);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tq = lane & 3;
  // copies: whole rows, NPC 16-byte pieces each, CR rows per request; reads: K
  // pieces tq + 4i of rows grp and grp + 8, V bytes grp VB .. of rows 2tq, + 1, + 8, + 9
  constexpr int NPC = D / 16, CR = 32 / NPC;
  const int c_row = lane / NPC, c_part = lane % NPC;
  const uint8_t* Kb = reinterpret_cast<const uint8_t*>(p.k_cache) + 16 * c_part;
  const uint8_t* Vb = reinterpret_cast<const uint8_t*>(p.v_cache) + 16 * c_part;
  const uint32_t ring = smem_u32(smem) + warp * kKv8Stages * STAGE;
  const uint32_t c_dst = ring + c_row * D, k_src = ring + grp * D, v_src = ring + VOFF + 2 * tq * D + grp * VB % 16;
  // DENSE: per stage, the (ks, vs) pairs of its two blocks
  const uint32_t scales = smem_u32(smem) + kAttnWarps * kKv8Stages * STAGE + warp * kKv8Stages * 8 * U;

  uint32_t qb[KSTEPS][2];
  float qs[2];
  const uint32_t head_bits = ((1u << GS) - 1u) >> (2 * tq) & 3u;
  float o[MT][4];  // dims grp D/8 + 2mt (+1), heads 2tq + {0,1}
#pragma unroll
  for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m_run[2] = {kNegInf, kNegInf}, r_run[2] = {kNegInf, kNegInf}, l_run[2] = {0.f, 0.f};

  for (int sc0 = t0, sc1; sc0 < t1; sc0 = sc1) {
    sc1 = DENSE ? t1 : min(sc0 + kKv8MaxList, t1);  // one gather list each
    int n = sc1 - sc0;
    if constexpr (!DENSE) {
      __shared__ uint32_t scan_sm[32];
      // the sub-chunk's block scales: at most one block per thread
      const int t = sc0 + tid * kKv8Block;
      uint32_t row;
      if (t < sc1 && kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t, &row))
        tab[tid] = make_float2(p.k_scale[row >> 4] * p.scale_log2, __log2f(p.v_scale[row >> 4]));
      n = build_union<GS, kKv8MaxList, kKv8Tok>(p, b, g, sc0, sc1, scan_sm, [&](int pos, int tt, uint32_t hb) {
        uint32_t rr;
        if (!kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, tt, &rr)) {
          atomicOr(p.status, TB_DEV_ERR_INDEX);
          hb = 0u;
        }
        list_idx[pos] = (int32_t)rr;
        list_hb[pos] = (uint16_t)(hb | (uint32_t)(tt - sc0) / kKv8Block << 8);
      });
    }
    const int niter = (n + kKv8Tok - 1) / kKv8Tok;
    const int my_n = niter > warp ? (niter - warp + kAttnWarps - 1) / kAttnWarps : 0;
    auto issue = [&](int it) {
      const int base = (warp + it * kAttnWarps) * kKv8Tok;
      const uint32_t off = (uint32_t)(it % kKv8Stages) * STAGE;
      uint32_t rows[kKv8Tok / CR];
      if constexpr (DENSE) {
        uint32_t row[U];
        int last[U];  // rows past the end repeat the last one
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int tt = sc0 + base + 16 * u;
          const bool in = tt < sc1;
          const bool ok = kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, in ? tt : sc0 + base, &row[u]);
          last[u] = ok && in ? sc1 - 1 - tt : 0;
          const uint32_t dst = scales + (it % kKv8Stages) * 8 * U + 8 * u;
          if (ok) {
            if (lane == 0) cp_async_4(dst, p.k_scale + (row[u] >> 4));
            if (lane == 1) cp_async_4(dst + 4, p.v_scale + (row[u] >> 4));
          } else if (lane == 0) {  // a page outside the pool: the block's scale is NaN
            atomicOr(p.status, TB_DEV_ERR_INDEX);
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst), "r"(0x7fffffff) : "memory");
          }
        }
#pragma unroll
        for (int r = 0; r < kKv8Tok / CR; ++r) {
          const int u = r * CR / 16;
          rows[r] = row[u] + min(c_row + CR * r - 16 * u, last[u]);
        }
      } else {
#pragma unroll
        for (int r = 0; r < kKv8Tok / CR; ++r) rows[r] = (uint32_t)list_idx[base + c_row + CR * r];
      }
#pragma unroll
      for (int r = 0; r < kKv8Tok / CR; ++r) {
        const size_t src = (size_t)rows[r] * D;
        const uint32_t dst = c_dst + off + r * CR * D;
        cp_async_16u(dst + ((c_part ^ kv8_swizzle_k<D>(c_row + CR * r)) << 4), Kb + src);
        cp_async_16u(dst + VOFF + ((c_part ^ kv8_swizzle_v<D>(c_row + CR * r)) << 4), Vb + src);
      }
    };
#pragma unroll
    for (int s = 0; s < kKv8Stages - 1; ++s) {
      if (s < my_n) issue(s);
      cp_async_commit();
    }
    if (sc0 == t0) load_q_f16<D, GS>(p.q, (size_t)b * p.Hq + g * GS, grp, tq, qb, qs);
    for (int it = 0; it < my_n; ++it) {
      __syncwarp();  // the stage refilled now has been read by every lane
      if (it + kKv8Stages - 1 < my_n) issue(it + kKv8Stages - 1);
      cp_async_commit();
      cp_async_wait<kKv8Stages - 1>();
      __syncwarp();  // the pieces come from other lanes
      const uint32_t off = (uint32_t)(it % kKv8Stages) * STAGE;
      const int base = (warp + it * kAttnWarps) * kKv8Tok;
      // ---- S^T = K Q^T: s[u][0..1] = token 16u + grp, s[u][2..3] = 16u + grp + 8; heads 2tq + {0,1}
      float s[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) s[u][0] = s[u][1] = s[u][2] = s[u][3] = 0.f;
#pragma unroll
      for (int i = 0; i < KLD; ++i) {
        uint32_t w[U][2][4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t at = k_src + off + 16 * u * D + (((tq + 4 * i) ^ kv8_swizzle_k<D>(grp)) << 4);
          const uint4 ka = lds16(at), kb = lds16(at + 8 * D);  // rows grp, grp + 8
          w[u][0][0] = ka.x; w[u][0][1] = ka.y; w[u][0][2] = ka.z; w[u][0][3] = ka.w;
          w[u][1][0] = kb.x; w[u][1][1] = kb.y; w[u][1][2] = kb.z; w[u][1][3] = kb.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            uint32_t a0, a1, a2, a3;
            kv8_to_f16<FMT>(w[u][0][j], a0, a2);
            kv8_to_f16<FMT>(w[u][1][j], a1, a3);
            mma_16816_f16(s[u], a0, a1, a2, a3, qb[4 * i + j][0], qb[4 * i + j][1]);
          }
      }
      float x[U][4], y[U][4];
      float mt[2] = {kNegInf, kNegInf}, rt[2] = {kNegInf, kNegInf};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float2 c[2];     // of tokens grp and grp + 8
        uint32_t hb[2];  // the lane's two heads
        if constexpr (DENSE) {
          const uint2 sc = lds8(scales + (it % kKv8Stages) * 8 * U + 8 * u);
          const float ks = __uint_as_float(sc.x);
          c[0] = c[1] = make_float2(ks * p.scale_log2, __log2f(__uint_as_float(sc.y)));
          const int left = ks == ks ? n - base - 16 * u : 0;
          hb[0] = grp < left ? head_bits : 0u;
          hb[1] = grp + 8 < left ? head_bits : 0u;
        } else {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t e = list_hb[base + 16 * u + grp + 8 * r];
            c[r] = tab[e >> 8];
            hb[r] = (e & 0xFFu) >> (2 * tq) & head_bits;
          }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // a masked token's weight is zero whatever its block's scale says
            const bool in = hb[r] >> e & 1u;
            x[u][2 * r + e] = in ? s[u][2 * r + e] * qs[e] * c[r].x : kNegInf;
            y[u][2 * r + e] = in ? x[u][2 * r + e] + c[r].y : kNegInf;
            mt[e] = fmaxf(mt[e], x[u][2 * r + e]);
            rt[e] = fmaxf(rt[e], y[u][2 * r + e]);
          }
      }
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
      float mu[2], ru[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mu[e] = m_run[e] == kNegInf ? 0.f : m_run[e];
        ru[e] = r_run[e] == kNegInf ? 0.f : r_run[e] - 7.f;
#pragma unroll
        for (int u = 0; u < U; ++u) l_run[e] += fast_exp2(x[u][e] - mu[e]) + fast_exp2(x[u][2 + e] - mu[e]);
      }
      uint32_t pb[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          pb[u][r] = movmatrix_trans(pack_f16(fast_exp2(y[u][2 * r] - ru[0]), fast_exp2(y[u][2 * r + 1] - ru[1])));
      // ---- O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t vc[4][VW];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = (r & 1) + 8 * (r >> 1);  // + 2tq
          const uint32_t at = v_src + off + (16 * u + row) * D + (((grp * VB >> 4) ^ kv8_swizzle_v<D>(2 * tq + row)) << 4);
          if constexpr (VW == 4) {
            const uint4 v = lds16(at);
            vc[r][0] = v.x;
            vc[r][1] = v.y;
            vc[r][2] = v.z;
            vc[r][3] = v.w;
          } else {
            const uint2 v = lds8(at);
            vc[r][0] = v.x;
            vc[r][1] = v.y;
          }
        }
#pragma unroll
        for (int j = 0; j < VW; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // bytes 2h and 2h + 1 of the word: m-tile 2j + h
            const uint32_t sel = h ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            kv8_to_f16<FMT>(__byte_perm(vc[0][j], vc[1][j], sel), a0, a1);
            kv8_to_f16<FMT>(__byte_perm(vc[2][j], vc[3][j], sel), a2, a3);
            mma_16816_f16(o[2 * j + h], a0, a1, a2, a3, pb[u][0], pb[u][1]);
          }
        }
      }
    }
    cp_async_wait<0>();
    if (!DENSE) __syncthreads();  // the gather list is free for the next sub-chunk
  }

  // ---- merge the four warps through shared memory (reuses the ring)
  __syncthreads();
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
