// rows.cuh -- what the norms share: rows held as they lie in memory by lanes of a warp or a block,
// their sums and maxima, the 8-bit output's scales, a row's copy to shared memory.
#pragma once
#include <cuda_fp8.h>

#include "ops_common.cuh"

namespace atlas {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxMin = 1e-30f;

// The scale of a group whose largest magnitude is m, and what multiplies its elements: 1 / scale to
// nearest.  The approximate reciprocal alone is off by its last bit, which puts some elements of every
// few rows on the wrong side of a tie.  One step of Newton's iteration squares its error, 2^-23, with an
// exact residual; the built-in rounded reciprocal has a call for subnormal arguments, for whose sake the
// compiler keeps registers free (32768 x 2048 to e4m3: 83.5 us with it, 81.8 so).
__device__ __forceinline__ float scale_of(float m) { return fmaxf(m, kAmaxMin) * (1.f / kE4m3Max); }
__device__ __forceinline__ float inverse(float scale) {
  const float i = rcp(scale);  // 0 for an infinite scale, and so the result
  return fmaf(fmaf(-fminf(scale, 3.4e38f), i, 1.f), i, i);
}

// The threads that share a row: TPR lanes of a warp (TPR <= 32), or the whole block.
struct RowGroup {
  int tpr, lane, tid;  // threads per row, lane within them
  int first = 0;       // (layer norm: what a thread's columns go by)
};

// Sum and maximum over a row's threads.  A block's warps meet in red[0 .. 31], of which the
// words past their number are zero; the next use of the same words has to be another
// reduction's barrier away.
template <typename F>
__device__ __forceinline__ float row_reduce(float v, const RowGroup& g, float* red, F f) {
  if (g.tpr >= 32) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
  } else {
    for (int m = g.tpr >> 1; m; m >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
  }
  if (g.tpr > 32) {
    if ((g.tid & 31) == 0) red[g.tid >> 5] = v;
    __syncthreads();
    const float4* q = reinterpret_cast<const float4*>(red);
    v = 0.f;
    for (int i = 0; i < (g.tpr + 127) / 128; ++i) {
      const float4 t = q[i];
      v = f(v, f(f(t.x, t.y), f(t.z, t.w)));
    }
  }
  return v;
}
__device__ __forceinline__ float row_sum(float v, const RowGroup& g, float* red) {
  return row_reduce(v, g, red, [](float x, float y) { return x + y; });
}
// NaN stays out of a maximum (fmaxf), as it does of its scale; the element itself stays NaN.
__device__ __forceinline__ float row_max(float v, const RowGroup& g, float* red) {
  return row_reduce(v, g, red, [](float x, float y) { return fmaxf(x, y); });
}
// The words that reductions meet in, before their first use.
__device__ __forceinline__ void clear_red(float* red, int n) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) red[i] = 0.f;
  __syncthreads();
}

// One element as it lies in memory: BYTES (0: none), so that all of a row's loads can be
// issued before the first conversion.
template <int BYTES>
__device__ __forceinline__ uint32_t ld_raw(const void* p, long i) {
  if (BYTES == 2) return reinterpret_cast<const uint16_t*>(p)[i];
  if (BYTES == 4) return reinterpret_cast<const uint32_t*>(p)[i];
  return 0;
}
template <int BYTES>
__device__ __forceinline__ float raw_float(uint32_t v, int dtype) {
  if (BYTES == 4) return __uint_as_float(v);
  if (dtype == ATLAS_BF16) return __uint_as_float(v << 16);
  return __half2float(__ushort_as_half((unsigned short)v));
}
__device__ __forceinline__ void st_elem(void* p, long i, int dtype, float v) {
  if (dtype == ATLAS_F32)
    reinterpret_cast<float*>(p)[i] = v;
  else if (dtype == ATLAS_BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else if (dtype == ATLAS_F16)
    reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
  else  // e4m3, to nearest even; the values are within +-448 by their scale
    reinterpret_cast<__nv_fp8_storage_t*>(p)[i] = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

// ------------------------------------------------------- aligned rows

// Eight elements as they lie in memory: BYTES each (0: none).
template <int BYTES>
struct Raw8 {
  uint4 q[BYTES == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, long i) {
    if (BYTES == 0) return;
    const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + i * BYTES);
    q[0] = __ldcs(v);
    if (BYTES == 4) q[BYTES == 4] = __ldcs(v + 1);
  }
  __device__ __forceinline__ void load_kept(const void* p, long i) {  // read again by other rows
    if (BYTES == 0) return;
    const uint4* v = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + i * BYTES);
    q[0] = v[0];
    if (BYTES == 4) q[BYTES == 4] = v[1];
  }
  __device__ __forceinline__ void zero() { q[0] = q[BYTES == 4] = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void floats(int dtype, float* v) const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(q);
    if (BYTES == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[BYTES == 4 ? i : 0]);
    } else if (BYTES == 2) {
      if (dtype == ATLAS_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
      }
    }
  }
};

// Eight values to an element type of 4, 2 or 1 bytes (e4m3: within +-448 by their scale).
__device__ __forceinline__ void st8(void* p, long i, int dtype, const float* v) {
  if (dtype == ATLAS_F32) {
    float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    __stcs(o, make_float4(v[0], v[1], v[2], v[3]));
    __stcs(o + 1, make_float4(v[4], v[5], v[6], v[7]));
  } else if (dtype == ATLAS_E4M3) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[k] = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k], v[4 * k + 1]), __NV_SATFINITE, __NV_E4M3) |
             (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2], v[4 * k + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
    __stcs(reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(p) + i), make_uint2(w[0], w[1]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (dtype == ATLAS_BF16) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&t);
      } else {
        const __half2 t = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
    __stcs(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i), make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// A row of n bytes (a multiple of 16) from p to shared memory by `threads` threads, neighbouring
// lanes taking neighbouring 16 bytes (a lane that took its own eight 32-bit elements would
// have each 32-byte sector asked for twice).
// Q pieces a thread.
template <int Q>
__device__ __forceinline__ void copy_row(char* s, const void* p, long at, int n, bool live, int lane, int threads) {
  const char* q = reinterpret_cast<const char*>(p) + (live ? at : 0);
#pragma unroll
  for (int k = 0; k < Q; ++k) {
    const int i = (k * threads + lane) * 16;
    if (i < n) cp_async<16>(s + i, live ? q + i : q, live);
  }
}

// Threads per row, vectors per thread and threads per block for rows of d channels in
// vectors of V.
struct RowPlan {
  int tpr, k, block;
};
inline RowPlan elem_plan(int d) {
  RowPlan p;
  p.k = d <= 8192 ? 8 : 32;
  if (d <= 256) {
    p.tpr = d <= 64 ? 8 : d <= 128 ? 16 : 32;
    p.block = 256;
  } else {
    p.tpr = ((d + p.k - 1) / p.k + 31) / 32 * 32;
    p.block = p.tpr;
  }
  return p;
}
// Up to `lanes_k` vectors a lane, a row belongs to lanes of a warp; else to a block of at most
// 512 threads.
inline RowPlan rows_plan(int d, int lanes_k) {
  const int nv = (d + 7) / 8;
  RowPlan p;
  if (nv <= 32 * lanes_k) {
    p.tpr = nv <= 8 ? 8 : nv <= 16 ? 16 : 32;
    p.k = (nv + p.tpr - 1) / p.tpr;
    p.block = 128;
  } else {
    p.k = 1;
    while ((nv + p.k - 1) / p.k > 512) p.k *= 2;
    p.tpr = ((nv + p.k - 1) / p.k + 31) / 32 * 32;
    p.block = p.tpr;
  }
  p.k = p.k <= 1 ? 1 : p.k <= 2 ? 2 : p.k <= 4 ? 4 : 8;
  return p;
}

// Blocks an SM for a kernel that needs `smem` bytes a block, at most `most`.
inline int resident(size_t smem, int most) {
  const int n = (int)((size_t)224 * 1024 / (smem + 1024));
  return n < 1 ? 1 : n < most ? n : most;
}

}  // namespace atlas
