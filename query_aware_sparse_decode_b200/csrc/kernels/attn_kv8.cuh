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
  // calls of one split: the output itself (bf16 or fp32) and its lse, no combine (out null: partials)
  void* out;             // [B][Hq][D]
  float* lse;            // [B][Hq] or null
  int out_bf16;
};

// The heads' outputs from the CTA's per-warp states in shared memory (wm null: a
// sequence without tokens): what write_partial and the combine kernel make of a single
// split, without their traffic and launch (128 sequences, dense: of 512 tokens 41.5 -> 29.9
// us, of 100 24.6 -> 12.7 us).
template <int D, int GS>
__device__ __forceinline__ void write_output(const AttnKv8Params& p, int b, int g, const float* wm, const float* wl,
                                             const float* wo) {
  for (int e = threadIdx.x; e < GS * D; e += kAttnThreads) {
    const int hh = e / D, d = e % D;
    float M = kNegInf, o = 0.f, l = 0.f;
    if (wm != nullptr) {
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) M = fmaxf(M, wm[w * GS + hh]);
    }
    if (M != kNegInf) {
#pragma unroll
      for (int w = 0; w < kAttnWarps; ++w) {
        const float m = wm[w * GS + hh];
        const float f = m == kNegInf ? 0.f : exp2f(m - M);
        o += f * wo[(w * GS + hh) * D + d];
        l += f * wl[w * GS + hh];
      }
      o *= 1.f / l;
    }
    const size_t row = (size_t)b * p.Hq + g * GS + hh;
    if (p.out_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[row * D + d] = __float2bfloat16_rn(o);
    else reinterpret_cast<float*>(p.out)[row * D + d] = o;
    if (p.lse != nullptr && d == 0) p.lse[row] = M == kNegInf ? kNegInf : (M + log2f(l)) * 0.69314718055994531f;
  }
}

// Split of the 8-bit attention (host side), counting the tokens that each
// sequence has: the shortest chunks (whole mask words) that keep the call's CTAs
// within one wave of kKv8CtasPerSm per SM, or, where these would be longer than
// `long_chunk`, within as many waves as bring them down to it.  A batch with more
// (sequence, KV head) pairs than these waves have CTAs takes chunks of long_chunk, whatever
// its lengths are: a long sequence among many short ones is then on few CTAs (8 KV heads, 127
// sequences of 100 tokens and one of 32768: dense 66 us, one set per KV group 75 us; the long
// one alone 17 and 14 us).
//  - Every token: 2048 (B = 4, L = 131072: 163 us, 203 us in one wave of 7296, 173 us with 512).
//  - Lists: 8192, since a CTA's first tile waits for a chain of mask, row and scale
//    loads and a sparse chunk has few tiles (the same lengths, one set per KV group with
//    10 % / 30 % of the tokens: 32.6 / 61.5 us, with 2048 39.9 / 71.0 us; 30 % per head 132
//    against 141 us).  From 4096 on, chunks are multiples of the four warps' segments.
constexpr int kKv8CtasPerSm = 4;
constexpr int kKv8Seg = 256;  // tokens of a warp's gather list
struct Kv8Split {
  int min_chunk, long_chunk;
};
constexpr Kv8Split kKv8SplitDense{128, 2048};  // 128: a tile or two a warp
constexpr Kv8Split kKv8SplitList{128, 8192};
// soft votes: by the tokens that are there (lengths 16383, 1, 1000, 4097: 13.6 us, 17.1 us
// split by the longest alone), B = 4, L = 131072: 109 us, in one wave 125 us
constexpr Kv8Split kKv8SplitVotes{kVoteMinChunk, 2048};
constexpr Kv8Split kKv8SplitF32{32, 2048};     // tokens one by one (B = 2, L = 512: 16.4 us with 128, 9.6 us with 32)
inline long long kv8_round_chunk(long long chunk, const Kv8Split& how) {
  const long long unit = how.long_chunk > 4096 && chunk >= 4096 ? kAttnWarps * kKv8Seg : 32;
  return (chunk + unit - 1) / unit * unit;
}
inline void attn_split_kv8(int num_sms, int kv_heads, const int* lens, int batch, int max_splits, const Kv8Split& how,
                           int* chunk_out, int* nsplit_out) {
  long long total = 0, longest = 1, used = 0;
  for (int b = 0; b < batch; ++b) {
    total += lens[b];
    longest = lens[b] > longest ? lens[b] : longest;
    used += lens[b] > 0;
  }
  const long long wave = (long long)kKv8CtasPerSm * num_sms;
  const long long one = (total * kv_heads + wave - 1) / wave;  // the chunk of one wave
  const long long waves = one > how.long_chunk ? (one + how.long_chunk - 1) / how.long_chunk : 1;
  const long long slots = wave * waves;
  const bool fits = used * kv_heads <= slots;
  long long chunk = fits ? (total * kv_heads + slots - 1) / slots : how.long_chunk;
  const long long least = (longest + max_splits - 1) / max_splits;
  chunk = chunk < least ? least : chunk;
  chunk = kv8_round_chunk(chunk < how.min_chunk ? how.min_chunk : chunk, how);
  while (fits && chunk < longest) {
    long long n = 0, next = longest;  // the CTAs, and the next chunk that has fewer
    for (int b = 0; b < batch; ++b) {
      const long long ns = (lens[b] + chunk - 1) / chunk;
      n += ns;
      if (ns > 1) {
        const long long c = (lens[b] + ns - 2) / (ns - 1);
        next = c < next ? c : next;
      }
    }
    if (n * kv_heads <= slots) break;
    chunk = kv8_round_chunk(next, how);  // > chunk: at least one sequence has a split less
  }
  *chunk_out = (int)chunk;
  *nsplit_out = (int)((longest + chunk - 1) / chunk);
}

constexpr int kKv8ListBytes = ((kAttnMaxChunk + kAttnTile) * 5 + 15) / 16 * 16;
template <int D, int GS>
constexpr int attn_kv8_f32_smem() { return kKv8ListBytes + kAttnWarps * GS * (D + 2) * 4; }

// The gather list of a sub-chunk, page ids checked: a token whose page is not
// one of the pool's is listed without a head (nothing reads its codes as a
// selected row) and flags TB_DEV_ERR_INDEX.  The list's padding (no head either)
// flags nothing: its token need not be one of the union's.
template <int GS>
__device__ __forceinline__ int build_union_list_kv8(const AttnKv8Params& p, int b, int g, int t0, int t1,
                                                    int32_t* list_idx, uint8_t* list_hb, uint32_t* scan_sm) {
  return build_union<GS>(p, b, g, t0, t1, scan_sm, [&](int pos, int t, uint32_t hb) {
    uint32_t row;
    if (!kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t, &row)) {
      if (hb) atomicOr(p.status, TB_DEV_ERR_INDEX);
      hb = 0u;
    }
    list_idx[pos] = (int32_t)row;
    list_hb[pos] = (uint8_t)hb;
  });
}

__device__ __forceinline__ void load_codes(uint8_t (&c)[4], const uint8_t* p) {
  const uchar4 v = *reinterpret_cast<const uchar4*>(p);
  c[0] = v.x;
  c[1] = v.y;
  c[2] = v.z;
  c[3] = v.w;
}
__device__ __forceinline__ void load_codes(uint8_t (&c)[2], const uint8_t* p) {
  const uchar2 v = *reinterpret_cast<const uchar2*>(p);
  c[0] = v.x;
  c[1] = v.y;
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
  if (t0 >= L) {
    if (p.out != nullptr) write_output<D, GS>(p, b, g, nullptr, nullptr, nullptr);
    return;
  }
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
    constexpr int AHEAD = 4;  // tokens whose rows and scales are requested together
    for (int i0 = warp; i0 < n; i0 += AHEAD * kAttnWarps) {
      uint8_t kc[AHEAD][DPL], vc[AHEAD][DPL];
      float ks[AHEAD], vs[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const uint32_t row = (uint32_t)list_idx[min(i0 + u * kAttnWarps, n - 1)];
        load_codes(kc[u], Kb + (size_t)row * D);
        load_codes(vc[u], Vb + (size_t)row * D);
        ks[u] = p.k_scale[row >> 4] * p.scale_log2;
        vs[u] = p.v_scale[row >> 4];
      }
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = i0 + u * kAttnWarps;
        const uint32_t hb = i < n ? list_hb[i] : 0u;
#pragma unroll
        for (int hh = 0; hh < GS; ++hh) {
          if (!((hb >> hh) & 1u)) continue;
          float dot = 0.f;
#pragma unroll
          for (int j = 0; j < DPL; ++j) dot = fmaf(q[hh][j], kv8_decode<FMT>(kc[u][j]), dot);
#pragma unroll
          for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
          const float s = dot * ks[u];
          const float mn = fmaxf(m[hh], s);
          const float alpha = exp2f(m[hh] - mn), pw = exp2f(s - mn);
          l[hh] = l[hh] * alpha + pw;
#pragma unroll
          for (int j = 0; j < DPL; ++j) o[hh][j] = o[hh][j] * alpha + pw * (kv8_decode<FMT>(vc[u][j]) * vs[u]);
          m[hh] = mn;
        }
      }
    }
    __syncthreads();  // the gather list is free for the next sub-chunk
  }
#pragma unroll
  for (int hh = 0; hh < GS; ++hh) {
    if (lane == 0) {
      wm[warp * GS + hh] = l[hh] != l[hh] ? 0.f : m[hh];  // (a NaN logit moves no maximum)
      wl[warp * GS + hh] = l[hh];
    }
#pragma unroll
    for (int j = 0; j < DPL; ++j) wo[(warp * GS + hh) * D + lane * DPL + j] = o[hh][j];
  }
  __syncthreads();
  if (p.out != nullptr) write_output<D, GS>(p, b, g, wm, wl, wo);
  else write_partial<D, GS>(p, b, g, split, wm, wl, wo);
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

// S^T of one tile: ka[i], kb[i] are pieces tq + 4i of rows grp and grp + 8;
// s[0..1] = row grp, s[2..3] = row grp + 8, heads 2tq + {0,1}, over qs.
template <int FMT, int D>
__device__ __forceinline__ void kv8_scores(const uint4 (&ka)[D / 64], const uint4 (&kb)[D / 64],
                                           const uint32_t (&qb)[D / 16][2], float (&s)[4]) {
  float s1[4] = {0.f, 0.f, 0.f, 0.f};  // two chains of products: each waits 20 cycles for its last
  s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const uint32_t wa[4] = {ka[i].x, ka[i].y, ka[i].z, ka[i].w}, wb[4] = {kb[i].x, kb[i].y, kb[i].z, kb[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t a0, a1, a2, a3;
      kv8_to_f16<FMT>(wa[j], a0, a2);
      kv8_to_f16<FMT>(wb[j], a1, a3);
      mma_16816_f16(j & 1 ? s1 : s, a0, a1, a2, a3, qb[4 * i + j][0], qb[4 * i + j][1]);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s[j] += s1[j];
}

// Ring of one warp, in tiles of 16 K and V rows (three are as fast for lists and slower
// for dense calls, a step over 16 x 8192 tokens 56.5 us against 54.4; four leave three
// CTAs an SM and lose everywhere).
constexpr int kKv8Stages = 2;
template <int D>
constexpr int kv8_stage_bytes() { return 2 * kAttnTile * D; }
// per warp: the ring, per stage the tokens' (ks, log2 vs, head bits), and for a
// list its entries and the segment's blocks
template <int D, bool DENSE>
constexpr int attn_kv8_warp_bytes() {
  return kKv8Stages * (kv8_stage_bytes<D>() + kAttnTile * 16) + (DENSE ? 0 : kKv8Seg * 2 + kKv8Seg / kKv8Block * 16);
}
template <int D, int GS, bool DENSE>
constexpr int attn_kv8_smem() {
  constexpr int work = kAttnWarps * attn_kv8_warp_bytes<D, DENSE>();
  constexpr int merge = kAttnWarps * GS * (D + 2) * 4;
  return work > merge ? work : merge;
}
// log2 of a V scale, in [-200, 200], which holds every positive finite one; a scale of zero (a
// block never written) weighs 2^-200
__device__ __forceinline__ float kv8_log2_scale(float vs) { return fminf(fmaxf(__log2f(vs), -200.f), 200.f); }
// 16-byte pieces of a cached row are stored at piece ^ swizzle(row), so that the
// lanes of a shared-memory phase touch different banks: for K two rows' pieces
// tq, for V rows 0, 2, 4, 6 (+ 1) of two neighbouring pieces.  Both are linear over
// xor in rows without common bits, so that a lane's share is a constant.
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
// the same for data that is read once: its lines are the first to leave L2
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async_16_once(uint32_t smem, const void* gmem, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;\n" ::"r"(smem), "l"(gmem), "l"(policy)
               : "memory");
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
//    (4 dims) is one k-step's share of a lane (fp8 mma.sync would take the codes as they
//    are, but sm_100a expands it into the same conversions: in this kernel's form of that
//    time 557 instructions a tile instead of 398);
//  - V: it takes D/8 bytes (dims grp D/8 ..) of token rows 2tq, 2tq+1, 2tq+8,
//    2tq+9; byte permutes pair the tokens of a dim, and m-tile mt takes dims
//    grp D/8 + 2mt and + 2mt + 1 as its rows grp and grp + 8.
// A ring of kKv8Stages tiles per warp holds the loads.  Rows are copied whole
// (eight lanes a 128-byte row: requests that took one sector of each of four rows
// made L2 send half as much again).
//
// DENSE takes every token of the chunk, tiles in turn over the warps: a tile is
// one block of the cache, so one row lookup and one scale pair serve it.
// Otherwise each warp walks its quarter of the chunk in segments of kKv8Seg
// tokens: it lists the union of the group's masks (8 tokens a lane), with the
// next segment's words, rows and scales already requested, and cuts the list
// into tiles; tokens that do not fill a tile wait in registers for the next
// segment's.  No barrier joins the warps, and the ring does not drain between
// segments (a CTA-wide list cost 40 % of the stalls).
//
// Softmax (log2 domain, fp32): l sums p = 2^(x - T); the weights of the V codes
// are w = 2^(x + log2 vs - R + 15) with a reference of their own, so that fp16
// holds them whatever the blocks' scales are.  T and R are not the exact maxima
// but 4 above one: they move only when a logit passes them (p <= 1, w <= 2^15),
// which after the first tiles is rare, and saves the cross-lane maximum of every
// tile.  Weights keep fp16's 11 bits down to 2^-25 of the largest one.
// References and exponents come from one rounded x, and R is held as its distance
// from T: however large the logits are, x - T is exact where it matters and not above
// 0, and log2 vs is added to it and not to x.  (From the unrounded product a weight
// passed fp16 above |x| = 2^26 or so, where the step of x exceeds the 4.)
//
// Measured with the combine (32 / 8 heads, D = 128, e4m3, L = 131072, B = 4): every
// token 167 us, 6.5 TB/s, the copy peak; 30 % per head 133 us, 6.2 TB/s (gathered 128-byte
// rows); one set of 30 % per KV group 65 us, 5.0 TB/s.  int8 takes 2 % longer for every token
// and 10 to 17 % for sets (434 instructions a tile against 340: its widening has no
// instruction of its own).
template <int FMT, int D, int GS, bool DENSE>
__global__ void __launch_bounds__(kAttnThreads, kKv8CtasPerSm) attn_kv8_kernel(const AttnKv8Params p) {
  pdl_wait();
  pdl_trigger();
  static_assert(D == 64 || D == 128, "head dim");
  constexpr int MT = D / 16;
  constexpr int KLD = D / 64;                   // 16-byte pieces of a K row per lane
  constexpr int VW = D / 32, VB = D / 8;        // words and bytes of a V row per lane
  constexpr int VOFF = kAttnTile * D;           // V rows of a stage
  constexpr int STAGE = kv8_stage_bytes<D>();
  extern __shared__ __align__(128) uint8_t smem[];
  const int split = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = p.lens[b];
  const int t0 = split * p.chunk;
  if (t0 >= L) {
    if (p.out != nullptr) write_output<D, GS>(p, b, g, nullptr, nullptr, nullptr);
    return;
  }
  const int t1 = min(t0 + p.chunk, L);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tq = lane & 3;
  // copies: whole rows, NPC 16-byte pieces each, CR rows per request; reads: K
  // pieces tq + 4i of rows grp and grp + 8, V bytes grp VB .. of rows 2tq, + 1, + 8, + 9
  constexpr int NPC = D / 16, CR = 32 / NPC;
  const int c_row = lane / NPC, c_part = lane % NPC;
  const uint8_t* Kb = reinterpret_cast<const uint8_t*>(p.k_cache) + 16 * c_part;
  const uint8_t* Vb = reinterpret_cast<const uint8_t*>(p.v_cache) + 16 * c_part;
  uint8_t* mine = smem + warp * attn_kv8_warp_bytes<D, DENSE>();
  const uint32_t ring = smem_u32(mine);
  // (a tile's rows differ from the lane's first by multiples of CR, 8 or 1, which
  // share no bits with it)
  const uint32_t ck_dst = ring + c_row * D + ((c_part ^ kv8_swizzle_k<D>(c_row)) << 4);
  const uint32_t cv_dst = ring + VOFF + c_row * D + ((c_part ^ kv8_swizzle_v<D>(c_row)) << 4);
  const uint32_t k_src = ring + grp * D + ((tq ^ kv8_swizzle_k<D>(grp)) << 4);
  const uint32_t v_src = ring + VOFF + 2 * tq * D + (((grp * VB >> 4) ^ kv8_swizzle_v<D>(2 * tq)) << 4) + grp * VB % 16;
  // per stage: DENSE: the block's (ks, vs); else the 16 tokens' (ks log2e/sqrt(D), log2 vs, head bits)
  const uint32_t meta = ring + kKv8Stages * STAGE;

  const uint32_t group_bits = (1u << GS) - 1u;
  const uint32_t head_bit[2] = {(1u << 2 * tq) & group_bits, (2u << 2 * tq) & group_bits};
  float o[MT][4];  // dims grp D/8 + 2mt (+1), heads 2tq + {0,1}
#pragma unroll
  for (int j = 0; j < MT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  // of heads 2tq + {0,1}: the reference T (kLowest: no token yet), T - R + 15, the lane's part of l
  constexpr float kLowest = -3.402823466e38f, kHead = 4.f;
  float ref[2] = {kLowest, kLowest}, lift[2] = {15.f, 15.f}, l_run[2] = {0.f, 0.f};

  // copies of a tile's 16 rows (of cache rows rows[r] = that of token c_row + CR r)
  auto copy_rows = [&](uint32_t off, const uint32_t (&rows)[kAttnTile / CR]) {
#pragma unroll
    for (int r = 0; r < kAttnTile / CR; ++r) {
      const size_t src = (size_t)rows[r] * D;
      cp_async_16u((ck_dst ^ kv8_swizzle_k<D>(CR * r) << 4) + (off + r * CR * D), Kb + src);
      cp_async_16u((cv_dst ^ kv8_swizzle_v<D>(CR * r) << 4) + (off + r * CR * D), Vb + src);
    }
  };

  // ---- the warp's tiles: issue(it, stage) starts the copies of tile `it`, false when there is none
  const int dense_tiles = (t1 - t0 + kAttnTile - 1) / kAttnTile;
  // list state: the segment being cut (list entries [pos, cnt)), the waiting tokens
  // (lanes 0 .. wait_n - 1), the next segment [seg, seg_end) and what is requested of it
  uint16_t* list = reinterpret_cast<uint16_t*>(mine + kKv8Stages * (STAGE + kAttnTile * 16));
  uint4* blocks = reinterpret_cast<uint4*>(list + kKv8Seg);  // (row, ks log2e/sqrt(D), log2 vs) of a segment's blocks
  constexpr int MW = (GS * (kKv8Seg / 32) + 31) / 32;        // mask words a lane requests
  const int quarter = ((t1 - t0 + kAttnWarps - 1) / kAttnWarps + 31) / 32 * 32;
  int seg = min(t0 + warp * quarter, t1);
  const int seg_end = min(seg + quarter, t1);
  int pos = 0, cnt = 0, wait_n = 0;
  uint32_t w_row = 0, w_hb = 0, n_word[MW], n_row = 0;
  float w_ks = 0.f, w_ev = 0.f, n_scale = 0.f;
  bool n_ok = true;
  const bool per_head = p.mask_mode == TB_MASK_PER_HEAD;
  auto request = [&]() {  // segment [seg, ..): its mask words, and lane l's block l % 16 (row; ks below lane 16, vs above)
#pragma unroll
    for (int i = 0; i < MW; ++i) {
      const int e = lane + 32 * i, h = e / (kKv8Seg / 32), w = e % (kKv8Seg / 32);
      n_word[i] = 0u;
      if (seg + 32 * w < seg_end && (per_head ? h < GS : h == 0)) {
        const size_t row = per_head ? (size_t)b * p.Hq + g * GS + h
                                    : p.mask_mode == TB_MASK_GROUP ? (size_t)b * p.Hkv + g : (size_t)b;
        n_word[i] = p.mask[row * p.mask_words + (seg >> 5) + w];
      }
    }
    const int t = seg + (lane & 15) * kKv8Block;
    n_ok = true;
    if (t < seg_end) {
      n_ok = kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t, &n_row);
      n_scale = (lane < 16 ? p.k_scale : p.v_scale)[n_row >> 4];
    }
  };
  auto build = [&]() {  // lists the requested segment and requests the next one
    __syncwarp();       // the previous list has been read
    const int w = lane >> 2, sh = 8 * (lane & 3);
    uint32_t byte[GS], u = 0;  // per head, the mask bits of the lane's 8 tokens
#pragma unroll
    for (int h = 0; h < GS; ++h) {
      const int e = (per_head ? h : 0) * (kKv8Seg / 32) + w;
      uint32_t v = __shfl_sync(0xffffffffu, n_word[0], e & 31);
      if (MW > 1) {
        const uint32_t v1 = __shfl_sync(0xffffffffu, n_word[MW - 1], e & 31);
        v = e < 32 ? v : v1;
      }
      byte[h] = v >> sh & 0xFFu;
      u |= byte[h];
    }
    const int valid = seg_end - (seg + 8 * lane);
    if (valid < 8) u &= valid > 0 ? (1u << valid) - 1u : 0u;
    const bool ok = __shfl_sync(0xffffffffu, n_ok, lane >> 1);
    if (!ok && u) {
      atomicOr(p.status, TB_DEV_ERR_INDEX);
      u = 0u;
    }
    const uint32_t c = __popc(u);
    uint32_t incl = c;
#pragma unroll
    for (int o2 = 1; o2 < 32; o2 <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o2);
      if (lane >= o2) incl += y;
    }
    uint16_t* at = list + (incl - c);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (u >> j & 1u) {
        uint32_t hb = 0;
#pragma unroll
        for (int h = 0; h < GS; ++h) hb |= (byte[h] >> j & 1u) << h;
        *at++ = (uint16_t)((8 * lane + j) | hb << 8);
      }
    }
    const float vs = __shfl_sync(0xffffffffu, n_scale, (lane & 15) + 16);
    if (lane < 16)
      blocks[lane] = make_uint4(n_row, __float_as_uint(n_scale * p.scale_log2), __float_as_uint(kv8_log2_scale(vs)), 0u);
    cnt = (int)__shfl_sync(0xffffffffu, incl, 31);
    pos = 0;
    seg += kKv8Seg;
    if (seg < seg_end) request();
    __syncwarp();
  };
  // lane's token of the list, entry i
  auto entry = [&](int i, uint32_t& row, float& ks, float& ev, uint32_t& hb) {
    const uint32_t v = list[i];
    const uint4 blk = blocks[(v & 0xFFu) >> 4];
    row = blk.x + (v & 15u);
    ks = __uint_as_float(blk.y);
    ev = __uint_as_float(blk.z);
    hb = v >> 8;
  };
  auto issue = [&](int it, uint32_t stage) -> bool {
    uint32_t rows[kAttnTile / CR];
    if constexpr (DENSE) {
      const int tile = warp + it * kAttnWarps;
      if (tile >= dense_tiles) return false;
      const int tt = t0 + tile * kAttnTile;
      uint32_t row;
      const bool ok = kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, tt, &row);
      const int last = ok ? t1 - 1 - tt : 0;  // rows past the end repeat the last one
      const uint32_t dst = meta + stage * (kAttnTile * 16);
      if (ok) {  // one lane per scale: a request fetches a sector for each active lane
        if (lane == 0) cp_async_4(dst, p.k_scale + (row >> 4));
        if (lane == 1) cp_async_4(dst + 4, p.v_scale + (row >> 4));
      } else if (lane == 0) {  // a page outside the pool: the block's scale is NaN
        atomicOr(p.status, TB_DEV_ERR_INDEX);
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(dst), "r"(0x7fffffff), "r"(0x3f800000) : "memory");
      }
#pragma unroll
      for (int r = 0; r < kAttnTile / CR; ++r) rows[r] = row + min(c_row + CR * r, last);
    } else {
      const int l16 = lane & 15;
      uint32_t row, hb;
      float ks, ev;
      if (wait_n == 0 && cnt - pos >= kAttnTile) {  // most tiles: 16 entries of the list
        entry(pos + l16, row, ks, ev, hb);
        pos += kAttnTile;
      } else {
        while (wait_n + cnt - pos < kAttnTile && seg < seg_end) {
          if (l16 >= wait_n && l16 < wait_n + cnt - pos) entry(pos + l16 - wait_n, w_row, w_ks, w_ev, w_hb);
          wait_n += cnt - pos;
          build();
        }
        const int n = min(wait_n + cnt - pos, kAttnTile);
        if (n == 0) return false;
        row = w_row;
        hb = w_hb;
        ks = w_ks;
        ev = w_ev;
        if (l16 >= wait_n && l16 < n) entry(pos + l16 - wait_n, row, ks, ev, hb);
        pos += n - wait_n;
        wait_n = 0;
        const uint32_t first = __shfl_sync(0xffffffffu, row, 0);
        if (l16 >= n) {  // past the last token: its row again, for no head
          row = first;
          ks = ev = 0.f;
          hb = 0u;
        }
      }
      if (lane < 16)
        *reinterpret_cast<uint4*>(mine + kKv8Stages * STAGE + (stage * kAttnTile + lane) * 16) =
            make_uint4(__float_as_uint(ks), __float_as_uint(ev), hb, 0u);
#pragma unroll
      for (int r = 0; r < kAttnTile / CR; ++r) rows[r] = __shfl_sync(0xffffffffu, row, c_row + CR * r);
    }
    copy_rows(stage * STAGE, rows);
    return true;
  };

  if (!DENSE && seg < seg_end) request();
  int queued = 0;  // tiles whose copies have started
#pragma unroll
  for (int s = 0; s < kKv8Stages - 1; ++s) {
    if (issue(s, s)) ++queued;
    cp_async_commit();
  }
  uint32_t qb[D / 16][2];
  float qs[2];
  load_q_f16<D, GS>(p.q, (size_t)b * p.Hq + g * GS, grp, tq, qb, qs);
  uint32_t stage = 0;
  for (int it = 0; it < queued; ++it, stage = stage == kKv8Stages - 1 ? 0 : stage + 1) {
    __syncwarp();  // the stage refilled now has been read by every lane
    if (queued == it + kKv8Stages - 1 && issue(queued, stage == 0 ? kKv8Stages - 1 : stage - 1)) ++queued;
    cp_async_commit();
    cp_async_wait<kKv8Stages - 1>();
    __syncwarp();  // the pieces come from other lanes
    const uint32_t off = stage * STAGE;
    // ---- S^T = K Q^T: s[0..1] = token grp, s[2..3] = grp + 8; heads 2tq + {0,1}
    float s[4];
    {
      uint4 ka[KLD], kb[KLD];  // rows grp, grp + 8
#pragma unroll
      for (int i = 0; i < KLD; ++i) {
        const uint32_t at = (k_src ^ i << 6) + off;
        ka[i] = lds16(at);
        kb[i] = lds16(at + 8 * D);
      }
      kv8_scores<FMT, D>(ka, kb, qb, s);
    }
    // x = (s qs) f, rounded once (s qs is exact above 2^-102, and in range where qs f need not be); d = x - T;
    // z = d + log2 vs + T - R + 15
    float f[2], ev[2];
    uint32_t hb[2];  // tokens grp and grp + 8: their heads
    bool masked = true;
    if constexpr (DENSE) {
      const uint2 sc = lds8(meta + stage * (kAttnTile * 16));
      const float ks = __uint_as_float(sc.x);
      ev[0] = ev[1] = kv8_log2_scale(__uint_as_float(sc.y));
      f[0] = f[1] = ks * p.scale_log2;
      const int left = ks == ks ? t1 - t0 - (warp + it * kAttnWarps) * kAttnTile : 0;
      masked = left < kAttnTile;
      hb[0] = grp < left ? ~0u : 0u;
      hb[1] = grp + 8 < left ? ~0u : 0u;
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint4 e = lds16(meta + (stage * kAttnTile + grp + 8 * r) * 16);
        ev[r] = __uint_as_float(e.y);
        f[r] = __uint_as_float(e.x);
        hb[r] = e.z;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = __fmul_rn(s[j] * qs[j & 1], f[j >> 1]);  // x (never fused into d)
    float d[4], z[4];
    auto exponents = [&]() {
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = 2 * r + e;
          d[j] = s[j] - ref[e];
          if (masked && !(hb[r] & head_bit[e])) d[j] = kNegInf;
          z[j] = d[j] + (ev[r] + lift[e]);
        }
    };
    exponents();
    const float dm = fmaxf(fmaxf(d[0], d[1]), fmaxf(d[2], d[3])), zm = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    if (__any_sync(0xffffffffu, dm > 0.f || zm > 15.f)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mt = kNegInf, rt = kNegInf;  // the head's largest x, and x - T + log2 vs, of the tile
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (!masked || (hb[r] & head_bit[e])) mt = fmaxf(mt, s[2 * r + e]);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, sh));
        const float t_old = ref[e], t_new = mt > t_old ? mt + kHead : t_old;
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (!masked || (hb[r] & head_bit[e])) rt = fmaxf(rt, (s[2 * r + e] - t_new) + ev[r]);
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) rt = fmaxf(rt, __shfl_xor_sync(0xffffffffu, rt, sh));
        // R - T, before and after (a head with no token so far has l = 0 and o = 0: any factor serves)
        const float r_old = (15.f - lift[e]) - (t_new - t_old), r_new = rt > r_old ? rt + kHead : r_old;
        if (t_new != t_old) l_run[e] *= fast_exp2(t_old - t_new);
        const float al = r_new != r_old ? fast_exp2(r_old - r_new) : 1.f;
        ref[e] = t_new;
        lift[e] = 15.f - r_new;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          o[j][e] *= al;
          o[j][2 + e] *= al;
        }
      }
      exponents();
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) l_run[e] += fast_exp2(d[e]) + fast_exp2(d[2 + e]);
    const uint32_t pb0 = movmatrix_trans(pack_f16(fast_exp2(z[0]), fast_exp2(z[1])));
    const uint32_t pb1 = movmatrix_trans(pack_f16(fast_exp2(z[2]), fast_exp2(z[3])));
    // ---- O^T += V^T P^T
    uint32_t vc[4][VW];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t at = v_src + off + ((r & 1) + 8 * (r >> 1)) * D;  // row 2tq + {0, 1, 8, 9}
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
        mma_16816_f16(o[2 * j + h], a0, a1, a2, a3, pb0, pb1);
      }
    }
  }
  cp_async_wait<0>();

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
        wm[warp * GS + h] = l_run[e] == 0.f ? kNegInf : ref[e];  // no token (a NaN logit moves no reference)
        wl[warp * GS + h] = l_run[e];
      }
      const float f = exp2f(-lift[e]);  // back from the weights' reference to T
      float* dst = wo + (warp * GS + h) * D + grp * (D / 8);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        dst[2 * j] = o[j][e] * f;
        dst[2 * j + 1] = o[j][2 + e] * f;
      }
    }
  }
  __syncthreads();
  if (p.out != nullptr) write_output<D, GS>(p, b, g, wm, wl, wo);
  else write_partial<D, GS>(p, b, g, split, wm, wl, wo);
}

struct VoteKv8Params : VoteParams {
  const float* k_scale;
  uint32_t* status;
};

// Soft-vote logits (log2 domain) and per-chunk (max, sum) pairs over 8-bit
// keys; softvote_reduce_kernel follows.  S^T = K Q^T as in attn_kv8_kernel, over
// consecutive tokens: a tile of 16 is one block of the cache, so it has one
// scale and one row lookup.  A ring of kVoteKv8Stages tiles per warp.  Measured (B = 1, L =
// 131072): 25 us of the call's 34 us, 5.3 TB/s; no unit is full (cold, 27 us: 58 % of the
// issue slots, ALU 47 %, DRAM cycles 63 %).
constexpr int kVoteKv8Stages = 3;
template <int D>
constexpr int vote_kv8_smem() { return kVoteWarps * kVoteKv8Stages * (kAttnTile * D + 16); }
template <int FMT, int D, int GS>
__global__ void __launch_bounds__(kVoteThreads, 4) softvote_kv8_logits_kernel(const VoteKv8Params p) {
  pdl_wait();
  pdl_trigger();
  constexpr int KLD = D / 64, NPC = D / 16, CR = 32 / NPC, STAGE = kAttnTile * D;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float wm[kVoteWarps * GS], wl[kVoteWarps * GS];
  const int chunk = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = p.lens[b];
  const int t0 = chunk * p.chunk;
  if (t0 >= L) return;
  const int t1 = min(t0 + p.chunk, L);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tq = lane & 3;
  const int c_row = lane / NPC, c_part = lane % NPC;
  const uint8_t* Kb = reinterpret_cast<const uint8_t*>(p.k_cache) + 16 * c_part;
  const uint32_t ring = smem_u32(smem) + warp * kVoteKv8Stages * STAGE;
  const uint32_t scales = smem_u32(smem) + kVoteWarps * kVoteKv8Stages * STAGE + warp * kVoteKv8Stages * 16;
  const uint64_t policy = evict_first_policy();  // the logits stay in L2 for the reduce pass
  const int my_n = (t1 - t0 - warp * kAttnTile + kVoteWarps * kAttnTile - 1) / (kVoteWarps * kAttnTile);  // may be <= 0
  auto issue = [&](int it) {
    const int tt = t0 + (warp + it * kVoteWarps) * kAttnTile;
    const uint32_t stage = (uint32_t)(it % kVoteKv8Stages);
    uint32_t row;
    const bool ok = kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, tt, &row);
    const int last = ok ? t1 - 1 - tt : 0;  // rows past the end repeat the last one
    if (lane == 0) {
      if (ok) {
        cp_async_4(scales + 16 * stage, p.k_scale + (row >> 4));
      } else {  // a page outside the pool: the block's scale is NaN
        atomicOr(p.status, TB_DEV_ERR_INDEX);
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(scales + 16 * stage), "r"(0x7fffffff) : "memory");
      }
    }
#pragma unroll
    for (int r = 0; r < kAttnTile / CR; ++r) {
      const int rr = c_row + CR * r;
      cp_async_16_once(ring + stage * STAGE + rr * D + ((c_part ^ kv8_swizzle_k<D>(rr)) << 4),
                       Kb + (size_t)(row + min(rr, last)) * D, policy);
    }
  };
#pragma unroll
  for (int s = 0; s < kVoteKv8Stages - 1; ++s) {
    if (s < my_n) issue(s);
    cp_async_commit();
  }
  uint32_t qb[D / 16][2];
  float qs[2];
  load_q_f16<D, GS>(p.q, (size_t)b * p.Hq + g * GS, grp, tq, qb, qs);
  const int hp = 2 * tq;
  const bool real[2] = {hp < GS, hp + 1 < GS};
  // per lane and head: a reference (8 above a logit that passed the last one) and the sum of 2^(x - it)
  constexpr float kLowest = -3.402823466e38f;
  float m[2] = {kLowest, kLowest}, l[2] = {0.f, 0.f};
  float* lrow[2];
#pragma unroll
  for (int e = 0; e < 2; ++e)
    lrow[e] = p.logits + ((size_t)b * p.Hq + g * GS + (real[e] ? hp + e : 0)) * p.max_len + t0 + warp * kAttnTile + grp;
  for (int it = 0; it < my_n; ++it) {
    __syncwarp();  // the stage refilled now has been read by every lane
    if (it + kVoteKv8Stages - 1 < my_n) issue(it + kVoteKv8Stages - 1);
    cp_async_commit();
    cp_async_wait<kVoteKv8Stages - 1>();
    __syncwarp();  // the pieces come from other lanes
    const uint32_t stage = (uint32_t)(it % kVoteKv8Stages);
    uint4 ka[KLD], kb[KLD];
#pragma unroll
    for (int i = 0; i < KLD; ++i) {
      const uint32_t at = ring + stage * STAGE + grp * D + (((tq + 4 * i) ^ kv8_swizzle_k<D>(grp)) << 4);
      ka[i] = lds16(at);
      kb[i] = lds16(at + 8 * D);
    }
    float s[4];
    kv8_scores<FMT, D>(ka, kb, qb, s);
    const float ks = __uint_as_float(lds8(scales + 16 * stage).x);
    const int left = t1 - t0 - (warp + it * kVoteWarps) * kAttnTile;
    const float f = ks * p.scale_log2;
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __fmul_rn(s[j] * qs[j & 1], f);  // rounded once: the reduce pass reads these logits
    const bool in[2] = {grp < left, grp + 8 < left};
    if (left < kAttnTile || !(ks == ks)) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!in[j >> 1] || !(ks == ks)) x[j] = kNegInf;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (real[e] && in[0]) lrow[e][0] = x[e];
      if (real[e] && in[1]) lrow[e][8] = x[2 + e];
      lrow[e] += kVoteWarps * kAttnTile;
      const float top = fmaxf(x[e], x[2 + e]);
      if (top > m[e]) {
        l[e] *= fast_exp2(m[e] - (top + 8.f));
        m[e] = top + 8.f;
      }
      l[e] += fast_exp2(x[e] - m[e]) + fast_exp2(x[2 + e] - m[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (l[e] == 0.f) m[e] = kNegInf;  // no token
  cp_async_wait<0>();
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
    // A chunk whose pages are all outside the pool counts as one token of the lowest logit: nothing
    // beside other chunks, and a sum to divide by where there are none (its logits of -inf vote 0).
    const bool none = M == kNegInf;
    const size_t ph = (((size_t)b * p.Hq + g * GS + tid) * p.nchunk + chunk) * 2;
    p.stats[ph] = none ? kLowest : M;
    p.stats[ph + 1] = none ? 1.f : sum;
  }
}

}  // namespace tb
