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
constexpr int attn_kv8_fma_smem() { return kKv8ListBytes + kAttnWarps * GS * (D + 2) * 4; }

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

// fp32 FMA: one warp per token at a time, lane owns D/32 consecutive dims.
template <typename T, int FMT, int D, int GS>
__global__ void __launch_bounds__(kAttnThreads) attn_kv8_fma_kernel(const AttnKv8Params p) {
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
      q[hh][j] = to_f32(reinterpret_cast<const T*>(p.q)[((size_t)b * p.Hq + g * GS + hh) * D + lane * DPL + j]);
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

struct VoteKv8Params : VoteParams {
  const float* k_scale;
  uint32_t* status;
};

// Soft-vote logits (log2 domain) and per-chunk (max, sum) pairs over 8-bit
// keys: one warp per token at a time.  softvote_reduce_kernel follows.
template <int FMT, int D, int GS>
__global__ void __launch_bounds__(kVoteThreads) softvote_kv8_logits_kernel(const VoteKv8Params p) {
  pdl_wait();
  pdl_trigger();
  constexpr int DPL = D / 32;
  __shared__ float wm[kVoteWarps * GS], wl[kVoteWarps * GS];
  const int chunk = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int L = p.lens[b];
  const int t0 = chunk * p.chunk;
  if (t0 >= L) return;
  const int t1 = min(t0 + p.chunk, L);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint8_t* Kb = reinterpret_cast<const uint8_t*>(p.k_cache) + lane * DPL;
  float q[GS][DPL], m[GS], l[GS];
#pragma unroll
  for (int hh = 0; hh < GS; ++hh) {
    m[hh] = kNegInf;
    l[hh] = 0.f;
#pragma unroll
    for (int j = 0; j < DPL; ++j)
      q[hh][j] = to_f32(
          reinterpret_cast<const __nv_bfloat16*>(p.q)[((size_t)b * p.Hq + g * GS + hh) * D + lane * DPL + j]);
  }
  for (int t = t0 + warp; t < t1; t += kVoteWarps) {
    uint32_t row;
    const bool ok = kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t, &row);
    if (!ok && lane == 0) atomicOr(p.status, TB_DEV_ERR_INDEX);
    const float ks = p.k_scale[row >> 4] * p.scale_log2;
    float kv[DPL];
#pragma unroll
    for (int j = 0; j < DPL; ++j) kv[j] = kv8_decode<FMT>(Kb[(size_t)row * D + j]);
#pragma unroll
    for (int hh = 0; hh < GS; ++hh) {
      float dot = 0.f;
#pragma unroll
      for (int j = 0; j < DPL; ++j) dot = fmaf(q[hh][j], kv[j], dot);
#pragma unroll
      for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      const float s = ok ? dot * ks : kNegInf;
      if (lane == 0) p.logits[((size_t)b * p.Hq + g * GS + hh) * p.max_len + t] = s;
      const float mn = fmaxf(m[hh], s);
      if (mn != kNegInf) {
        l[hh] = l[hh] * exp2f(m[hh] - mn) + exp2f(s - mn);
        m[hh] = mn;
      }
    }
  }
#pragma unroll
  for (int hh = 0; hh < GS; ++hh)
    if (lane == 0) {
      wm[warp * GS + hh] = m[hh];
      wl[warp * GS + hh] = l[hh];
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
