// 8-bit K/V caches: the formats, quantising rows as they are written, reading
// them back and projecting K_imp from them.
//
// A cache row (one token of one (b, KV head)) holds D codes of one byte; the
// 16 tokens of an aligned block share one fp32 scale.  With F the largest code
// value (e4m3: 448, int8: 127) and amax the block's largest finite magnitude
//
//   e = max(-100, smallest integer with amax <= F 2^e),  scale = 2^e,
//   code = x 2^-e rounded to the format's nearest value, ties to even.
//
// A power of two makes the scaling exact: a code differs from x only by its own
// rounding (e4m3: at most 2^-4 relative, or 2^-10 scale for small values; int8:
// half a scale), the result does not depend on the order of operations, and a
// block whose scale grows when a token joins it re-rounds its older codes by a
// power of two (e4m3 codes then change only where they become subnormal; int8
// codes lose at most half a step of each scale passed, under one final step in
// all).  It costs up to one bit of the int8 range.  Blocks of 16 tokens never
// cross a page (pages hold a power of two >= 16 tokens), so the scale of cache
// row r is scale[r / 16] in dense and paged caches.
#pragma once

#include "common.cuh"

namespace tb {

constexpr int kKv8Block = TB_KV8_BLOCK;
constexpr int kKv8MinExp = -100;
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
  return e < kKv8MinExp ? kKv8MinExp : e;
}
__device__ __forceinline__ float kv8_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// magnitude that counts towards amax: infinities and NaN do not
__device__ __forceinline__ float kv8_mag(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
__device__ __forceinline__ bool kv8_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// code of x * inv (inv = 1 / scale, a power of two): rounded to nearest even,
// infinities to the largest code value, NaN to zero
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

// One CTA per touched block of 16 tokens of a (b, g): grid (blocks, Hkv, B),
// 128 threads.  Both tensors' new rows are staged in shared memory as fp32; the
// block's amax gives the scale; rows of the block that were cached before are
// re-rounded when the scale grows.  Rows behind the last written one keep their
// codes.  K_imp of the new rows comes from the unrounded values.
constexpr int kKv8WriteThreads = 128;
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(kKv8WriteThreads) kv8_write_kernel(const Kv8WriteParams p) {
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
// left alone.  A thread decodes 16 codes (one 16-byte load); grid
// (ceil(count * D/16 / 256), Hkv, B).
template <typename T, int FMT, int D>
__global__ void __launch_bounds__(256) kv8_read_kernel(const Kv8ReadParams p) {
  pdl_wait();
  pdl_trigger();
  constexpr int NP = D / 16;
  const int g = blockIdx.y, b = blockIdx.z;
  const int e = blockIdx.x * 256 + threadIdx.x;
  const int i = e / NP, part = e % NP, t = p.start + i;
  if (i >= p.count || t >= p.lens[b]) return;
  uint32_t row;
  if (!kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t, &row)) {
    atomicOr(p.status, TB_DEV_ERR_INDEX);
    return;
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    if (p.out[kv] == nullptr) continue;
    const uint4 c = *reinterpret_cast<const uint4*>(p.codes[kv] + (size_t)row * D + part * 16);
    const float s = p.scale[kv][row >> 4];
    T* out = reinterpret_cast<T*>(p.out[kv]) + (((size_t)b * p.Hkv + g) * p.count + i) * D + part * 16;
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float x[4];
      kv8_decode4<FMT>(w[q], x);
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint2*>(out + 4 * q) = make_uint2(pack_bf16(x[0] * s, x[1] * s), pack_bf16(x[2] * s, x[3] * s));
      } else {
        *reinterpret_cast<float4*>(out + 4 * q) = make_float4(x[0] * s, x[1] * s, x[2] * s, x[3] * s);
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
};

// K_imp of rows [start, start + count) from the cached (rounded) keys, fp32
// FMA: grid (ceil(count/32), Hkv, B), 256 threads, 32 rows x d' outputs.
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
  bool bad = false;
  if (tid < ROWS) {
    uint32_t row = 0;
    float s = 0.f;
    if (tid < n) {
      bad = !kv_row_checked(p.kl, b, g, p.Hkv, p.max_len, t0 + tid, &row);
      s = bad ? 0.f : p.scale[row >> 4];  // a row without a page projects to zero
    }
    krow[tid] = row;
    kscale[tid] = s;
  }
  if (__syncthreads_or(bad) && tid == 0) atomicOr(p.status, TB_DEV_ERR_INDEX);
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
