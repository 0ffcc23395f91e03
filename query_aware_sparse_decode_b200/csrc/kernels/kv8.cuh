// 8-bit K/V caches: the formats, quantising rows as they are written, reading
// them back and projecting K_imp from them.
//
// A cache row (one token of one (b, KV head)) holds D codes of one byte; the
// 16 tokens of an aligned block share one fp32 scale.  With F the largest code
// value (e4m3: 448, int8: 127) and amax the block's largest finite magnitude
//
//   e = smallest integer with amax <= F 2^e, in [-100, 119] (int8: 121),  scale = 2^e,
//   code = x 2^-e rounded to the format's nearest value, ties to even.
//
// A power of two makes the scaling exact: a code differs from x only by its own
// rounding (e4m3: at most 2^-4 relative, or 2^-10 scale for small values; int8:
// half a scale), the result does not depend on the order of operations, and a
// block whose scale grows when a token joins it re-rounds its older codes by a
// power of two (e4m3 codes then change only where they become subnormal; int8
// codes lose at most half a step of each scale passed, under one final step in
// all).  It costs up to one bit of the int8 range.  The upper limit keeps F 2^e
// finite: the few values above it (2.98e38, int8 3.38e38) are stored as it.  Blocks of 16 tokens never
// cross a page (pages hold a power of two >= 16 tokens), so the scale of cache
// row r is scale[r / 16] in dense and paged caches.
#pragma once

#include "common.cuh"

namespace tb {

constexpr int kKv8Block = TB_KV8_BLOCK;
constexpr int kKv8MinExp = -100;
template <int FMT>
constexpr int kKv8MaxExp = FMT == TB_KV8_E4M3 ? 119 : 121;
constexpr int kFmtE4m3 = TB_KV8_E4M3;
constexpr int kFmtInt8 = TB_KV8_INT8;

// ------------------------------------------------------------ codes
// exponent e of the rule above from amax >= 0 (finite), by its bits: F is
// 1.75 * 2^8 (e4m3) or 1.984375 * 2^6 (int8)
template <int FMT>
__device__ __forceinline__ int kv8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int ex = (int)(u >> 23) - 127;
  const uint32_t mant = u & 0x7FFFFFu;
  const int e = FMT == kFmtE4m3 ? ex - 8 + (mant > 0x600000u) : ex - 6 + (mant > 0x7E0000u);
  return e < kKv8MinExp ? kKv8MinExp : e > kKv8MaxExp<FMT> ? kKv8MaxExp<FMT> : e;
}
// 2^e, -126 <= e <= 127
__device__ __forceinline__ float kv8_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// magnitude that counts towards amax: infinities and NaN do not
__device__ __forceinline__ float kv8_mag(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
__device__ __forceinline__ bool kv8_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// code of x * inv (inv = 1 / scale, a power of two): rounded to nearest even,
// infinities and values above the largest code to it, NaN to zero
template <int FMT>
__device__ __forceinline__ uint8_t kv8_encode(float y) {
  if (y != y) y = 0.f;
  if constexpr (FMT == kFmtE4m3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(y));
    return (uint8_t)(r & 0xFFu);
  } else {
    y = fminf(fmaxf(y, -127.f), 127.f);
    return (uint8_t)(int8_t)__float2int_rn(y);
  }
}
// e4m3 pair -> two fp16 values (exact), low byte in the low half
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ float f16_bits_to_f32(uint16_t v) {
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"(v));
  return f;
}
template <int FMT>
__device__ __forceinline__ float kv8_decode(uint8_t c) {
  if constexpr (FMT == kFmtE4m3)
    return f16_bits_to_f32((uint16_t)(e4m3x2_to_f16x2(c) & 0xFFFFu));
  else
    return (float)(int8_t)c;
}
// the four codes of a word as fp32 values
template <int FMT>
__device__ __forceinline__ void kv8_decode4(uint32_t w, float (&x)[4]) {
  if constexpr (FMT == kFmtE4m3) {
    const uint32_t a = e4m3x2_to_f16x2((uint16_t)(w & 0xFFFFu)), c = e4m3x2_to_f16x2((uint16_t)(w >> 16));
    x[0] = f16_bits_to_f32((uint16_t)(a & 0xFFFFu));
    x[1] = f16_bits_to_f32((uint16_t)(a >> 16));
    x[2] = f16_bits_to_f32((uint16_t)(c & 0xFFFFu));
    x[3] = f16_bits_to_f32((uint16_t)(c >> 16));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
  }
}

// ------------------------------------------------------------ writing rows
struct Kv8WriteParams {
  const void* src[2];        // K and V rows: element (b, g, i, d) at b*sb + g*sh + i*st + d
  long long sb[2], sh[2], st[2];
  uint8_t* codes[2];         // [B][Hkv][max_len][D], or page pools
  float* scale[2];           // one per 16 cache rows
  void* kimp;                // [B][Hkv][max_len/256][d'][256] (kimp_index)
  const void* w_k;           // [D][d']
  uint32_t* status;
  KvLayout kl;
  int Hkv, dimp, max_len, kimp_bf16;
  int pos[kMaxBatch];        // first row written of sequence b (its length before)
  int cnt[kMaxBatch];        // rows written
};

// fp32 rows: one CTA per touched block of 16 tokens of a (b, g): grid (blocks,
// Hkv, B), 128 threads.  Both tensors' new rows are staged in shared memory as fp32; the
// block's amax gives the scale; rows of the block that were cached before are
// re-rounded when the scale grows.  Rows behind the last written one keep their
// codes.  K_imp of the new rows comes from the unrounded values.
constexpr int kKv8WriteThreads = 128;
template <int FMT, int D>
__global__ void __launch_bounds__(kKv8WriteThreads) kv8_write_f32_kernel(const Kv8WriteParams p) {
  using T = float;
  pdl_wait();
  pdl_trigger();
  constexpr int NT = kKv8WriteThreads;
  __shared__ float x[kKv8Block][D];
  __shared__ float wsm[D * 32];
  __shared__ float s_max[NT / 32];
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int pos = p.pos[b], end = pos + p.cnt[b];
  const int t_lo = (pos / kKv8Block + blockIdx.x) * kKv8Block;
  if (p.cnt[b] == 0 || t_lo >= end) return;
  const int r0 = max(pos - t_lo, 0), r1 = min(end - t_lo, kKv8Block);  // the block's new rows
  uint32_t row0;
  if (!kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t_lo, &row0)) {
    if (tid == 0) atomicOr(p.status, TB_DEV_ERR_INDEX);
    return;
  }
  const T* W = reinterpret_cast<const T*>(p.w_k);
  for (int e = tid; e < D * p.dimp; e += NT) wsm[e] = to_f32(W[e]);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const T* src = reinterpret_cast<const T*>(p.src[kv]) + b * p.sb[kv] + g * p.sh[kv] +
                   (long long)(t_lo - pos) * p.st[kv];
    float amax = 0.f;
    bool odd = false;
    for (int e = tid; e < (r1 - r0) * D; e += NT) {
      const int r = r0 + e / D, d = e % D;
      const float v = to_f32(src[r * p.st[kv] + d]);
      x[r][d] = v;
      amax = fmaxf(amax, kv8_mag(v));
      odd = odd || !kv8_finite(v);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    if (__syncthreads_or(odd) && tid == 0) atomicOr(p.status, TB_DEV_ERR_VALUE);
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) amax = fmaxf(amax, s_max[w]);
    float sc = kv8_pow2(kv8_exponent<FMT>(amax));
    float* scale = p.scale[kv] + (row0 >> 4);
    uint8_t* codes = p.codes[kv] + (size_t)row0 * D;
    if (r0 > 0) {
      const float old = *scale;
      if (old >= sc) {
        sc = old;
      } else {
        const float ratio = old * (1.f / sc);
        for (int e = tid; e < r0 * D; e += NT) codes[e] = kv8_encode<FMT>(kv8_decode<FMT>(codes[e]) * ratio);
      }
    }
    const float inv = 1.f / sc;
    for (int e = r0 * D + tid; e < r1 * D; e += NT) codes[e] = kv8_encode<FMT>(x[e / D][e % D] * inv);
    if (kv == 0) {  // K_imp[j] = sum_d K[d] W_K[d][j], four interleaved chains
      const int j = tid % p.dimp;
      for (int r = r0 + tid / p.dimp; r < r1; r += NT / p.dimp) {
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        for (int d = 0; d < D; d += 4)
#pragma unroll
          for (int u = 0; u < 4; ++u) a[u] = fmaf(x[r][d + u], wsm[(d + u) * p.dimp + j], a[u]);
        store_kimp(p.kimp, kimp_index((size_t)b * p.Hkv + g, j, t_lo + r, p.dimp, p.max_len),
                   (a[0] + a[1]) + (a[2] + a[3]), p.kimp_bf16);
      }
    }
    __syncthreads();  // every thread has read the old scale and its staged rows
    if (tid == 0) *scale = sc;
  }
}

// bf16 rows: one warp per touched block, everything in registers.  Lane (grp,
// tq) loads 16-byte pieces (dims 32i + 8tq ..) of rows grp and grp + 8 of K and
// of V: 16 rows of both are in flight at once.  The same registers are the A
// fragments of K_imp = K W_K on mma.sync m16n8k16 (the k indices of step
// 2i + h are dims 32i + 8tq + 4h + {0,1 | 2,3}), the input of the block's amax
// (one warp maximum) and of the codes, stored 8 bytes a lane in whole
// 32-byte sectors.  W_K's B fragments are staged once per CTA, in lane order.
// A warp's blocks are gridDim.x apart, so few blocks spread over the CTAs; the next
// block's V is requested when V's registers are free, its K when K's are.  Measured:
// 32768 tokens of 8 heads (D = 128, d' = 32) 44 us, 235 MB, 5.3 TB/s of mixed reads and writes.
struct Kv8WriteBf16Params : Kv8WriteParams {
  int first[kMaxBatch + 1];  // units (block, head) before sequence b's; [B]: all of them
  int batch;
};

// largest |x| pattern of a bf16 pair; NaN patterns exceed infinity's
__device__ __forceinline__ uint32_t bf16x2_absmax(uint32_t m, uint32_t w) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7FFF7FFFu));
  return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// codes of x0..x3 (finite, |x| inv <= F) in a word
template <int FMT>
__device__ __forceinline__ uint32_t kv8_encode4(float x0, float x1, float x2, float x3, float inv) {
  if constexpr (FMT == kFmtE4m3) {
    uint16_t a, c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x1 * inv), "f"(x0 * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x3 * inv), "f"(x2 * inv));
    return (uint32_t)a | (uint32_t)c << 16;
  } else {
    // adding 1.5 * 2^23 rounds to an integer (ties to even) in the low mantissa bits
    const float magic = 12582912.f;
    const uint32_t a = __byte_perm(__float_as_uint(fmaf(x0, inv, magic)), __float_as_uint(fmaf(x1, inv, magic)), 0x0040);
    const uint32_t c = __byte_perm(__float_as_uint(fmaf(x2, inv, magic)), __float_as_uint(fmaf(x3, inv, magic)), 0x0040);
    return __byte_perm(a, c, 0x5410);
  }
}
template <int FMT>
__device__ __forceinline__ uint32_t kv8_encode4_any(float x0, float x1, float x2, float x3, float inv) {
  return (uint32_t)kv8_encode<FMT>(x0 * inv) | (uint32_t)kv8_encode<FMT>(x1 * inv) << 8 |
         (uint32_t)kv8_encode<FMT>(x2 * inv) << 16 | (uint32_t)kv8_encode<FMT>(x3 * inv) << 24;
}

// A unit of the write: one block of one (b, g).
struct Kv8Unit {
  int b, g, t_lo, r0, r1;  // its first token, and the block's new rows [r0, r1)
  uint32_t row0;           // its first cache row
  bool ok;                 // false: no page of the pool
};
__device__ __forceinline__ Kv8Unit kv8_unit(const Kv8WriteBf16Params& p, int u) {
  Kv8Unit r;
  r.b = 0;
  for (int hi = p.batch; hi - r.b > 1;) {
    const int mid = (r.b + hi) >> 1;
    if (p.first[mid] <= u) r.b = mid;
    else hi = mid;
  }
  const int pos = p.pos[r.b], end = pos + p.cnt[r.b];
  const int per_head = (p.first[r.b + 1] - p.first[r.b]) / p.Hkv;
  r.g = (u - p.first[r.b]) / per_head;
  r.t_lo = (pos / kKv8Block + (u - p.first[r.b]) % per_head) * kKv8Block;
  r.r0 = max(pos - r.t_lo, 0);
  r.r1 = min(end - r.t_lo, kKv8Block);
  r.ok = kv_row_checked(p.kl, r.b, r.g, p.Hkv, p.max_len, r.t_lo, &r.row0);
  return r;
}
// The lane's pieces of the unit's new rows (zeros in the others) and the block's old scale.
template <int D>
__device__ __forceinline__ void kv8_load_rows(const Kv8WriteBf16Params& p, int kv, const Kv8Unit& u, int grp, int tq,
                                              uint4 (&x)[2][D / 32], float& old) {
  const uint16_t* src = reinterpret_cast<const uint16_t*>(p.src[kv]) + u.b * p.sb[kv] + u.g * p.sh[kv] +
                        (long long)(u.t_lo - p.pos[u.b]) * p.st[kv] + 8 * tq;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = grp + 8 * h;
    const bool fresh = r >= u.r0 && r < u.r1;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      x[h][i] = fresh ? __ldcs(reinterpret_cast<const uint4*>(src + r * p.st[kv] + 32 * i)) : make_uint4(0u, 0u, 0u, 0u);
  }
  old = u.r0 > 0 ? p.scale[kv][u.row0 >> 4] : 0.f;
}
// Codes and scale of the unit's rows of one tensor.
template <int FMT, int D>
__device__ __forceinline__ void kv8_store_rows(const Kv8WriteBf16Params& p, int kv, const Kv8Unit& u, int lane,
                                               const uint4 (&x)[2][D / 32], float old) {
  constexpr int NP = D / 32;
  const int grp = lane >> 2, tq = lane & 3;
  uint32_t m2 = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint4 w = x[h][i];
      m2 = bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(m2, w.x), w.y), w.z), w.w);
    }
  uint32_t top = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
  const bool odd = top >= 0x7F80u;  // an infinity or a NaN
  const bool clamp = top > (FMT == kFmtE4m3 ? 0x7F60u : 0x7F7Eu);  // these, or a value above F 2^e
  if (odd) {
    float a = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint32_t w[4] = {x[h][i].x, x[h][i].y, x[h][i].z, x[h][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) a = fmaxf(a, fmaxf(kv8_mag(bf16_lo(w[j])), kv8_mag(bf16_hi(w[j]))));
      }
    top = __reduce_max_sync(0xffffffffu, __float_as_uint(a) >> 16);
    if (lane == 0) atomicOr(p.status, TB_DEV_ERR_VALUE);
  }
  float sc = kv8_pow2(kv8_exponent<FMT>(__uint_as_float(top << 16)));
  float ratio = 1.f;  // of the old scale to the new one, for the block's older rows
  if (u.r0 > 0) {
    if (old >= sc) sc = old;
    else ratio = old * (1.f / sc);
  }
  const float inv = 1.f / sc;
  uint8_t* dst = p.codes[kv] + (size_t)u.row0 * D + 8 * tq;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = grp + 8 * h;
    if (r >= u.r0 && r < u.r1) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint4 w = x[h][i];
        uint2 c;
        if (!clamp) {
          c.x = kv8_encode4<FMT>(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), inv);
          c.y = kv8_encode4<FMT>(bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w), inv);
        } else {
          c.x = kv8_encode4_any<FMT>(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y), inv);
          c.y = kv8_encode4_any<FMT>(bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w), inv);
        }
        *reinterpret_cast<uint2*>(dst + r * D + 32 * i) = c;
      }
    } else if (r < u.r0 && ratio != 1.f) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint2* at = reinterpret_cast<uint2*>(dst + r * D + 32 * i);
        float y[4], z[4];
        kv8_decode4<FMT>(at->x, y);
        kv8_decode4<FMT>(at->y, z);
        *at = make_uint2(kv8_encode4_any<FMT>(y[0], y[1], y[2], y[3], ratio),
                         kv8_encode4_any<FMT>(z[0], z[1], z[2], z[3], ratio));
      }
    }
  }
  if (lane == 0) p.scale[kv][u.row0 >> 4] = sc;
}

template <int FMT, int D, int DIMP>
__global__ void __launch_bounds__(kKv8WriteThreads, 4) kv8_write_bf16_kernel(const Kv8WriteBf16Params p) {
  pdl_wait();
  pdl_trigger();
  constexpr int KST = D / 16, NT = DIMP / 8, NP = D / 32;
  __shared__ uint2 wf[KST * NT * 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = lane >> 2, tq = lane & 3;
  const int units = p.first[p.batch], step = gridDim.x * (kKv8WriteThreads / 32);
  int u = blockIdx.x + warp * gridDim.x;
  Kv8Unit cur{};
  uint4 xk[2][NP], xv[2][NP];
  float old_k = 0.f, old_v = 0.f;
  if (u < units) {  // the first unit's rows are on their way while W_K is staged
    cur = kv8_unit(p, u);
    kv8_load_rows<D>(p, 1, cur, grp, tq, xv, old_v);
    kv8_load_rows<D>(p, 0, cur, grp, tq, xk, old_k);
  }
  {
    const uint16_t* W = reinterpret_cast<const uint16_t*>(p.w_k);
#pragma unroll
    for (int e = tid; e < KST * NT * 32; e += kKv8WriteThreads) {
      const int ln = e & 31, nt = (e >> 5) % NT, kk = (e >> 5) / NT;
      const uint16_t* w = W + (32 * (kk >> 1) + 8 * (ln & 3) + 4 * (kk & 1)) * DIMP + 8 * nt + (ln >> 2);
      wf[e] = make_uint2((uint32_t)w[0] | (uint32_t)w[DIMP] << 16, (uint32_t)w[2 * DIMP] | (uint32_t)w[3 * DIMP] << 16);
    }
  }
  __syncthreads();
  while (u < units) {
    u += step;
    Kv8Unit next{};
    if (u < units) next = kv8_unit(p, u);
    if (!cur.ok && lane == 0) atomicOr(p.status, TB_DEV_ERR_INDEX);
    if (cur.ok) kv8_store_rows<FMT, D>(p, 1, cur, lane, xv, old_v);
    if (u < units) kv8_load_rows<D>(p, 1, next, grp, tq, xv, old_v);
    if (cur.ok) {
      kv8_store_rows<FMT, D>(p, 0, cur, lane, xk, old_k);
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint4 w0 = xk[0][i], w1 = xk[1][i];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 f0 = wf[(2 * i * NT + nt) * 32 + lane], f1 = wf[((2 * i + 1) * NT + nt) * 32 + lane];
          mma_16816(acc[nt], w0.x, w1.x, w0.y, w1.y, f0.x, f0.y);
          mma_16816(acc[nt], w0.z, w1.z, w0.w, w1.w, f1.x, f1.y);
        }
      }
      const size_t slab = (size_t)cur.b * p.Hkv + cur.g;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = grp + 8 * h;
        if (r < cur.r0 || r >= cur.r1) continue;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            store_kimp(p.kimp, kimp_index(slab, 8 * nt + 2 * tq + e, cur.t_lo + r, DIMP, p.max_len), acc[nt][2 * h + e],
                       p.kimp_bf16);
      }
    }
    if (u < units) kv8_load_rows<D>(p, 0, next, grp, tq, xk, old_k);
    cur = next;
  }
}

// ------------------------------------------------------------ reading rows
struct Kv8ReadParams {
  const uint8_t* codes[2];
  const float* scale[2];
  void* out[2];              // [B][Hkv][count][D], or null
  uint32_t* status;
  KvLayout kl;
  int Hkv, max_len, start, count;
  int lens[kMaxBatch];
};

// out[b][g][t - start] = code * scale for t < len[b]; rows past the length are
// left alone.  A thread turns codes into 16 bytes of output, kKv8ReadPieces
// times, so that loads and stores of a warp are contiguous and several are
// in flight; grid (ceil(count * pieces / (256 kKv8ReadPieces)), Hkv, B).  Measured: 32768
// tokens of 8 heads (D = 128, bf16) 30 us, 6.6 TB/s.
constexpr int kKv8ReadPieces = 4;
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(256) kv8_read_kernel(const Kv8ReadParams p) {
  pdl_wait();
  pdl_trigger();
  constexpr int CW = 4 / sizeof(T);   // words of codes per piece: 2 (bf16) or 1 (fp32)
  constexpr int NP = D / (4 * CW);    // pieces per row
  const int g = blockIdx.y, b = blockIdx.z;
  const int n = min(p.count, p.lens[b] - p.start);
  const long long e0 = (long long)blockIdx.x * (256 * kKv8ReadPieces) + threadIdx.x;
  uint32_t c[2][kKv8ReadPieces][CW];
  float s[2][kKv8ReadPieces];
#pragma unroll
  for (int u = 0; u < kKv8ReadPieces; ++u) {
    const int i = (int)((e0 + u * 256) / NP), part = (int)((e0 + u * 256) % NP);
    uint32_t row = 0;
    bool ok = i < n;
    if (ok && !kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, p.start + i, &row)) {
      atomicOr(p.status, TB_DEV_ERR_INDEX);
      ok = false;
    }
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      s[kv][u] = -1.f;  // nothing to write
      if (!ok || p.out[kv] == nullptr) continue;
      s[kv][u] = p.scale[kv][row >> 4];
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.codes[kv] + (size_t)row * D) + part * CW;
      if constexpr (CW == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        c[kv][u][0] = w.x;
        c[kv][u][1] = w.y;
      } else {
        c[kv][u][0] = *src;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kKv8ReadPieces; ++u) {
    const long long e = e0 + u * 256;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float f = s[kv][u];
      if (f < 0.f) continue;
      uint8_t* out = reinterpret_cast<uint8_t*>(p.out[kv]) +
                     (((size_t)b * p.Hkv + g) * p.count * NP + (size_t)e) * 16;
      float x[4], y[4];
      kv8_decode4<FMT>(c[kv][u][0], x);
      if constexpr (CW == 2) {
        kv8_decode4<FMT>(c[kv][u][CW - 1], y);
        __stcs(reinterpret_cast<uint4*>(out), make_uint4(pack_bf16(x[0] * f, x[1] * f), pack_bf16(x[2] * f, x[3] * f),
                                                         pack_bf16(y[0] * f, y[1] * f), pack_bf16(y[2] * f, y[3] * f)));
      } else {
        __stcs(reinterpret_cast<float4*>(out), make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f));
      }
    }
  }
}

// ------------------------------------------------------------ K_imp from codes
struct Kv8ProjectParams {
  const uint8_t* codes;
  const float* scale;
  void* kimp;
  const void* w_k;
  uint32_t* status;
  KvLayout kl;
  int Hkv, max_len, start, count, kimp_bf16;
  int lens[kMaxBatch];
};

// K_imp of rows [start, start + count) from the cached (rounded) keys, fp32
// FMA: grid (ceil(count/32), Hkv, B), 256 threads, 32 rows x d' outputs.  A row without
// a page projects to zero; it is missed (TB_DEV_ERR_INDEX) only below its sequence's length.
template <typename T, int FMT, int D, int DIMP>
__global__ void __launch_bounds__(256) kv8_project_kernel(const Kv8ProjectParams p) {
  constexpr int ROWS = 32;
  constexpr int OPT = ROWS * DIMP / 256;  // outputs per thread
  __shared__ float ks[ROWS][D + 1];
  __shared__ float ws[D][DIMP];
  __shared__ uint32_t krow[ROWS];
  __shared__ float kscale[ROWS];
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int t0 = p.start + blockIdx.x * ROWS;
  const int n = min(ROWS, p.start + p.count - t0);
  const T* W = reinterpret_cast<const T*>(p.w_k);
  for (int i = tid; i < D * DIMP; i += 256) ws[i / DIMP][i % DIMP] = to_f32(W[i]);
  bool missed = false;
  if (tid < ROWS) {
    uint32_t row = 0;
    float s = 0.f;
    if (tid < n) {
      const bool ok = kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t0 + tid, &row);
      s = ok ? p.scale[row >> 4] : 0.f;
      missed = !ok && t0 + tid < p.lens[b];
    }
    krow[tid] = row;
    kscale[tid] = s;
  }
  if (__syncthreads_or(missed) && tid == 0) atomicOr(p.status, TB_DEV_ERR_INDEX);
  for (int i = tid; i < ROWS * D / 4; i += 256) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    float x[4];
    kv8_decode4<FMT>(*reinterpret_cast<const uint32_t*>(p.codes + (size_t)krow[r] * D + d), x);
#pragma unroll
    for (int u = 0; u < 4; ++u) ks[r][d + u] = x[u] * kscale[r];
  }
  __syncthreads();
  const int r = tid / (256 / ROWS), j0 = tid % (256 / ROWS) * OPT;
  float acc[OPT];
#pragma unroll
  for (int j = 0; j < OPT; ++j) acc[j] = 0.f;
  for (int d = 0; d < D; ++d) {
    const float kv = ks[r][d];
#pragma unroll
    for (int j = 0; j < OPT; ++j) acc[j] = fmaf(kv, ws[d][j0 + j], acc[j]);
  }
  if (r < n)
#pragma unroll
    for (int j = 0; j < OPT; ++j)
      store_kimp(p.kimp, kimp_index((size_t)b * p.Hkv + g, j0 + j, t0 + r, DIMP, p.max_len), acc[j], p.kimp_bf16);
}

}  // namespace tb
