// norm.cu -- residual addition and root-mean-square norm, with an output in 32, 16 or
// 8 bits, and its backward pass.
//
//   h = x + r,  y = h rstd w,  rstd = 1 / sqrt(mean(h^2) + eps)
//   dx = rstd (w dy - hat mean(w dy hat)) + dh,  dw = sum over rows of dy hat,  hat = h rstd
//
// Both passes are bound by memory, so what counts is how many loads are under way and that
// instructions do not get in their way.  Aligned rows are held as they lie in memory, eight
// elements a load (the element's type is known at run time, its size at compile time).  A row
// of up to 256 channels belongs to 8, 16 or 32 lanes of a warp, four rows under way; a longer
// one to a block, which walks rows with the next two on their way through shared memory (a few
// rows: a block each).  Rows of odd widths or addresses take the element-wise kernels.  Sums
// run in 32 bits; the only roundings are those of the outputs to their types.
//
// Measured (copy rate 6.78 TB/s): 32768 x 2048 bf16 + residual to e4m3 with scales of 128: 82 us,
// 85% (a warp a row, loads in its turn: 123 us; divisions and a loop over the warps' sums: 96);
// 524288 x 128 bf16: 51 us, 77%; backward, 16384 x 2560, 32-bit stream: 99 us, 88% (one row's
// loads ahead in registers: 134); 20000 x 1371 bf16 element by element: 123 and 330 us.
#include <cuda_fp8.h>

#include <limits>

#include "ops_common.cuh"

namespace atlas {
namespace {

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

// 1 / sqrt(mean of squares + eps).  eps = 0 and a row of zeros: the outputs are zeros, and so is the
// norm's part of the gradients.  Forward the launch takes the least number for eps = 0, so that 0 rstd is 0
// without a word for it in the kernels (a select cost the rows of 128 channels 2%).
__device__ __forceinline__ float rstd_of(float sum, const NormArgs& a) { return rsqrtf(sum * a.inv_d + a.eps); }
__device__ __forceinline__ float back_rstd_of(float sum, const NormArgs& a) {
  const float v = sum * a.inv_d + a.eps;
  return v == 0.f ? 0.f : rsqrtf(v);
}

// The threads that share a row: TPR lanes of a warp (TPR <= 32), or the whole block.
struct RowGroup {
  int tpr, lane, tid;  // threads per row, lane within them
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

// Rows of any width and alignment, K elements a thread.
template <int XB, int RB, int K>
__global__ void __launch_bounds__(1024) norm_forward_elem(NormArgs a, int tpr) {
  extern __shared__ __align__(16) float sm[];  // 64 floats, then the groups' maxima of an 8-bit output
  float* red = sm;
  clear_red(red, 64);
  const RowGroup g{tpr, (int)threadIdx.x % tpr, (int)threadIdx.x};
  const int rpb = blockDim.x / tpr;
  const long row = (long)blockIdx.x * rpb + threadIdx.x / tpr;
  const bool live = row < a.rows;
  uint32_t x[K], r[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * tpr + g.lane;
    const bool in = live && c < a.d;
    x[k] = in ? ld_raw<XB>(a.x, row * a.sx + c) : 0u;
    r[k] = RB && in ? ld_raw<RB>(a.r, row * a.sr + c) : 0u;
  }
  float h[K], ss = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * tpr + g.lane;
    h[k] = raw_float<XB>(x[k], a.dt) + (RB ? raw_float<RB>(r[k], a.rt) : 0.f);
    if (a.r_out && live && c < a.d) st_elem(a.r_out, row * a.sr + c, a.rt, h[k]);
    ss += h[k] * h[k];
  }
  const float rstd = rstd_of(row_sum(ss, g, red), a);
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * tpr + g.lane;
    if (c < a.d) {
      h[k] *= rstd;
      if (a.w) h[k] *= ld_any(a.w, c, a.wt);
      amax = fmaxf(amax, fabsf(h[k]));
      if (live && a.ot != ATLAS_E4M3) st_elem(a.y, row * a.sy + c, a.ot, h[k]);
    }
  }
  if (a.ot != ATLAS_E4M3) return;
  if (a.group == 0) {
    const float scale = scale_of(row_max(amax, g, red + 32)), inv = inverse(scale);
    if (live && g.lane == 0) a.scale[row] = scale;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * tpr + g.lane;
      if (live && c < a.d) st_elem(a.y, row * a.sy + c, a.ot, h[k] * inv);
    }
    return;
  }
  // groups of channels: maxima of non-negative floats order like their bits, so integer
  // maxima in shared memory give the same result in any order
  const int ng = a.ng;
  unsigned* gm = reinterpret_cast<unsigned*>(sm + 64) + (threadIdx.x / tpr) * ng;
  for (int i = g.lane; i < ng; i += tpr) gm[i] = 0u;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * tpr + g.lane;
    if (c < a.d) atomicMax(&gm[c / a.group], __float_as_uint(fmaxf(0.f, fabsf(h[k]))));
  }
  __syncthreads();
  for (int i = g.lane; i < ng; i += tpr) {
    const float scale = scale_of(__uint_as_float(gm[i]));
    if (live) a.scale[row * ng + i] = scale;
    gm[i] = __float_as_uint(inverse(scale));
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = k * tpr + g.lane;
    if (live && c < a.d) st_elem(a.y, row * a.sy + c, a.ot, h[k] * __uint_as_float(gm[c / a.group]));
  }
}

// A block walks the rows blockIdx.x * rpb + .., step gridDim.x * rpb, the next row's loads under
// way; each thread keeps the sums of dy hat of its columns over its rows, and the block writes
// one row of partial sums.
template <int HB, int DB, int K>
__global__ void __launch_bounds__(1024) norm_backward_elem(NormArgs a, int tpr) {
  extern __shared__ __align__(16) float sm[];
  float* red = sm;
  clear_red(red, 64);
  const RowGroup g{tpr, (int)threadIdx.x % tpr, (int)threadIdx.x};
  const int rpb = blockDim.x / tpr, mine = threadIdx.x / tpr;
  float dw[K];
  uint32_t h[K], dy[K];
  auto fetch = [&](long row) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * tpr + g.lane;
      const bool in = row < a.rows && c < a.d;
      h[k] = in ? ld_raw<HB>(a.x, row * a.sr + c) : 0u;
      dy[k] = in ? ld_raw<DB>(a.dy, row * a.sy + c) : 0u;
    }
  };
#pragma unroll
  for (int k = 0; k < K; ++k) dw[k] = 0.f;
  long row = (long)blockIdx.x * rpb + mine;
  fetch(row);
  for (; row - mine < a.rows; row += (long)gridDim.x * rpb) {
    const bool live = row < a.rows;
    float hv[K], dv[K], ss = 0.f, dot = 0.f;
    uint32_t up[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * tpr + g.lane;
      hv[k] = raw_float<HB>(h[k], a.rt);
      dv[k] = raw_float<DB>(dy[k], a.dt);
      up[k] = a.r && live && c < a.d ? ld_raw<HB>(a.r, row * a.sr + c) : 0u;
    }
    fetch(row + (long)gridDim.x * rpb);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * tpr + g.lane;
      ss += hv[k] * hv[k];
      dot += hv[k] * (a.w && c < a.d ? ld_any(a.w, c, a.wt) * dv[k] : dv[k]);
    }
    ss = row_sum(ss, g, red);  // the other sum's barrier lies between two uses of the same words
    dot = row_sum(dot, g, red + 32);
    const float rstd = back_rstd_of(ss, a);
    const float mean = dot * rstd * a.inv_d;  // mean(w dy hat)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = k * tpr + g.lane;
      if (live && c < a.d) {
        const float hat = hv[k] * rstd, wdy = a.w ? ld_any(a.w, c, a.wt) * dv[k] : dv[k];
        dw[k] += dv[k] * hat;
        st_elem(a.y, row * a.sr + c, a.rt, rstd * (wdy - hat * mean) + raw_float<HB>(up[k], a.rt));
      }
    }
  }
  if (!a.dw) return;
  float* acc = sm + 64;
  for (int r = 0; r < rpb; ++r) {  // rows of one block in a fixed order
    __syncthreads();
    if (r == mine) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = k * tpr + g.lane;
        if (c < a.d) {
          const float s = (r == 0 ? 0.f : acc[c]) + dw[k];
          if (r == rpb - 1)
            a.part[(long)blockIdx.x * a.d + c] = s;
          else
            acc[c] = s;
        }
      }
    }
  }
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

// This thread's weights: K vectors of eight, ones without a weight.
template <int K>
__device__ __forceinline__ void load_weights(const NormArgs& a, int tpr, int lane, float (*w)[8]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * tpr + lane) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[k][i] = 1.f;
    if (a.w && c < a.d) {
      if (a.wt == ATLAS_F32) {
        Raw8<4> q;
        q.load_kept(a.w, c);
        q.floats(a.wt, w[k]);
      } else {
        Raw8<2> q;
        q.load_kept(a.w, c);
        q.floats(a.wt, w[k]);
      }
    }
  }
}

// One row from its vectors and weights: K of eight a thread.  red: 64 words, of which the next row of the
// same threads takes another 64.
template <int XB, int RB, int K>
__device__ __forceinline__ void forward_row(const NormArgs& a, const RowGroup& g, float* red, long row,
                                            bool live, const Raw8<XB>* x, const Raw8<RB>* r,
                                            const float (*w)[8]) {
  float h[K][8], ss = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * g.tpr + g.lane) * 8;
    x[k].floats(a.dt, h[k]);
    if (RB) {
      float v[8];
      r[k].floats(a.rt, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] += v[i];
    }
    if (a.r_out && live && c < a.d) st8(a.r_out, row * a.sr + c, a.rt, h[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += h[k][i] * h[k][i];
  }
  const float rstd = rstd_of(row_sum(ss, g, red), a);
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * g.tpr + g.lane) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[k][i] = h[k][i] * rstd * w[k][i];
    if (a.ot != ATLAS_E4M3) {
      if (live && c < a.d) st8(a.y, row * a.sy + c, a.ot, h[k]);
      continue;
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(h[k][i]));
    if (a.group == 0) {
      amax = fmaxf(amax, m);
      continue;
    }
    // the group's lanes are neighbours: group / 8 of them, a power of two
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (8 * o < a.group) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float scale = scale_of(m), inv = inverse(scale);
    if (live && c < a.d) {
      if ((c & (a.group - 1)) == 0) a.scale[row * a.ng + (c >> a.gshift)] = scale;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] *= inv;
      st8(a.y, row * a.sy + c, a.ot, h[k]);
    }
  }
  if (a.ot == ATLAS_E4M3 && a.group == 0) {
    const float scale = scale_of(row_max(amax, g, red + 32)), inv = inverse(scale);
    if (live && g.lane == 0) a.scale[row] = scale;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * g.tpr + g.lane) * 8;
      if (live && c < a.d) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] *= inv;
        st8(a.y, row * a.sy + c, a.ot, h[k]);
      }
    }
  }
}

// R rows at a time.  tpr threads a row: 8, 16 or 32 lanes, or the whole block (R = 1).
template <int XB, int RB, int K, int R>
__global__ void __launch_bounds__(512) norm_forward_rows(NormArgs a, int tpr) {
  extern __shared__ __align__(16) float sm[];
  if (tpr > 32) clear_red(sm, 64);
  const RowGroup g{tpr, (int)threadIdx.x % tpr, (int)threadIdx.x};
  const int rpb = blockDim.x / tpr;
  const long row0 = (long)blockIdx.x * rpb * R + threadIdx.x / tpr;
  Raw8<XB> x[R][K];
  Raw8<RB> r[R][K];
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long row = row0 + j * rpb;
      const int c = (k * tpr + g.lane) * 8;
      x[j][k].zero();
      r[j][k].zero();
      if (row < a.rows && c < a.d) {
        x[j][k].load(a.x, row * a.sx + c);
        if (RB) r[j][k].load(a.r, row * a.sr + c);
      }
    }
  float w[K][8];
  load_weights<K>(a, tpr, g.lane, w);
#pragma unroll
  for (int j = 0; j < R; ++j)
    forward_row<XB, RB, K>(a, g, sm, row0 + j * rpb, row0 + j * rpb < a.rows, x[j], r[j], w);
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

// Many rows of a block each: a block walks rows and copies the next kStages - 1 to shared
// memory while it computes one, so that loads are always under way.  The lanes that copy 16-bit
// elements are those that read them; with 32-bit elements the barrier in a row's reduction also
// hands over the next row, whose copies have been waited for before it.
constexpr int kStages = 3;
template <int XB, int RB, int K>
__global__ void __launch_bounds__(512) norm_forward_ring(NormArgs a) {
  extern __shared__ __align__(16) float sm[];  // [2][64] for the reductions, then [stage]: x, r
  constexpr bool kOwn = XB == 2 && RB != 4;
  clear_red(sm, 128);
  const RowGroup g{(int)blockDim.x, (int)threadIdx.x, (int)threadIdx.x};
  const int bytes = a.d * (XB + RB);
  char* ring = reinterpret_cast<char*>(sm + 128);
  auto fetch = [&](long row, int stage) {
    char* s = ring + stage * bytes;
    copy_row<K * XB / 2>(s, a.x, row * a.sx * XB, a.d * XB, row < a.rows, g.lane, g.tpr);
    if (RB) copy_row<K * RB / 2>(s + a.d * XB, a.r, row * a.sr * RB, a.d * RB, row < a.rows, g.lane, g.tpr);
    cp_commit();
  };
  float w[K][8];
  if (K <= 2) load_weights<K>(a, g.tpr, g.lane, w);
  long row = blockIdx.x;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(row + (long)i * gridDim.x, i);
  cp_wait<kStages - 2>();
  __syncthreads();
  int stage = 0;
  for (int odd = 0; row < a.rows; row += gridDim.x, odd ^= 64) {
    fetch(row + (long)(kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);
    if (kOwn) cp_wait<kStages - 1>();
    Raw8<XB> x[K];
    Raw8<RB> r[K];
    const char* s = ring + stage * bytes;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * g.tpr + g.lane) * 8;
      x[k].zero();
      r[k].zero();
      if (c < a.d) {
        x[k].load_kept(s, c);
        if (RB) r[k].load_kept(s + a.d * XB, c);
      }
    }
    if (!kOwn) cp_wait<kStages - 2>();  // the next row's
    if (K > 2) load_weights<K>(a, g.tpr, g.lane, w);  // (long rows: again for each, from L2)
    forward_row<XB, RB, K>(a, g, sm + odd, row, true, x, r, w);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_wait<0>();
}

// Backward: tpr threads a row as above; block b takes the rows b * rpb + .., step
// gridDim.x * rpb.  Both sums of a row are reduced together.
// MT: most threads; up to 320 (2560 channels), two blocks an SM without a register in memory.
template <int HB, int DB, int GB, int K, int MT>  // bytes of h, dy, dh (0: none)
__global__ void __launch_bounds__(MT, MT == 320 ? 2 : 1) norm_backward_rows(NormArgs a, int tpr) {
  extern __shared__ __align__(16) float sm[];
  float2* red = reinterpret_cast<float2*>(sm);  // [2][16], then the rows' ring
  const int lane = threadIdx.x % tpr, rpb = blockDim.x / tpr, mine = threadIdx.x / tpr;
  const int nw = tpr >> 5;
  clear_red(sm, 64);
  float dw[K][8], w[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.f;
  load_weights<K>(a, tpr, lane, w);
  // [stage][row of the block]: h, dy, dh
  const int bytes = a.d * (HB + DB + GB);
  char* ring = reinterpret_cast<char*>(sm + 64) + mine * bytes;
  const long step = (long)gridDim.x * rpb;
  auto fetch = [&](long row, int stage) {
    char* s = ring + stage * rpb * bytes;
    copy_row<K * HB / 2>(s, a.x, row * a.sr * HB, a.d * HB, row < a.rows, lane, tpr);
    copy_row<K * DB / 2>(s + a.d * HB, a.dy, row * a.sy * DB, a.d * DB, row < a.rows, lane, tpr);
    if (GB) copy_row<K * GB / 2>(s + a.d * (HB + DB), a.r, row * a.sr * GB, a.d * GB, row < a.rows, lane, tpr);
    cp_commit();
  };
  long row = (long)blockIdx.x * rpb + mine;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(row + i * step, i);
  cp_wait<kStages - 2>();
  __syncthreads();
  int stage = 0;
  for (int odd = 0; row - mine < a.rows; row += step, odd ^= 1) {
    fetch(row + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
    float hv[K][8], dv[K][8], gv[K][8], ss = 0.f, dot = 0.f;
    const char* s = ring + stage * rpb * bytes;
    stage = stage + 1 == kStages ? 0 : stage + 1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * tpr + lane) * 8;
      Raw8<HB> h;
      Raw8<DB> dy;
      Raw8<GB> dh;
      h.zero(), dy.zero(), dh.zero();
      if (c < a.d) {
        h.load_kept(s, c);
        dy.load_kept(s + a.d * HB, c);
        if (GB) dh.load_kept(s + a.d * (HB + DB), c);
      }
      h.floats(a.rt, hv[k]);
      dy.floats(a.dt, dv[k]);
      if (GB) dh.floats(a.rt, gv[k]);
    }
    cp_wait<kStages - 2>();  // the next row's copies, handed over by the barrier below
    if (nw <= 1) __syncwarp();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss += hv[k][i] * hv[k][i];
        dot += hv[k][i] * (w[k][i] * dv[k][i]);
      }
    for (int m = min(tpr, 32) >> 1; m; m >>= 1) {
      ss += __shfl_xor_sync(0xFFFFFFFFu, ss, m);
      dot += __shfl_xor_sync(0xFFFFFFFFu, dot, m);
    }
    if (nw > 1) {  // one row a block; two buffers, so that one barrier a row is enough
      if ((threadIdx.x & 31) == 0) red[odd * 16 + (threadIdx.x >> 5)] = make_float2(ss, dot);
      __syncthreads();
      ss = dot = 0.f;
      for (int i = 0; i < (nw + 1) / 2; ++i) {
        const float4 v = reinterpret_cast<const float4*>(red + odd * 16)[i];
        ss += v.x + v.z;
        dot += v.y + v.w;
      }
    }
    const float rstd = back_rstd_of(ss, a);  // (a place of the block without a row holds zeros)
    const float mean = dot * rstd * a.inv_d;  // mean(w dy hat)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * tpr + lane) * 8;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float hat = hv[k][i] * rstd;
        dw[k][i] += dv[k][i] * hat;
        o[i] = rstd * (w[k][i] * dv[k][i] - hat * mean) + (GB ? gv[k][i] : 0.f);
      }
      if (row < a.rows && c < a.d) st8(a.y, row * a.sr + c, a.rt, o);
    }
  }
  cp_wait<0>();
  if (!a.dw) return;
  float* acc = sm + 64;  // over the rows' ring
  for (int r = 0; r < rpb; ++r) {  // rows of one block in a fixed order
    __syncthreads();
    if (r == mine) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * tpr + lane) * 8;
        if (c < a.d) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float s = (r == 0 ? 0.f : acc[c + i]) + dw[k][i];
            if (r == rpb - 1)
              a.part[(long)blockIdx.x * a.d + c + i] = s;
            else
              acc[c + i] = s;
          }
        }
      }
    }
  }
}

// dw[c] = sum over the blocks' partial sums; 32 columns a block, 8 threads a column.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* part, float* dw, int nblk, int d) {
  __shared__ float s[8][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float v = 0.f;
  if (c < d)
    for (int r = ry; r < nblk; r += 8) v += part[(long)r * d + c];
  s[ry][cx] = v;
  __syncthreads();
  if (ry == 0 && c < d) {
#pragma unroll
    for (int r = 1; r < 8; ++r) v += s[r][cx];
    dw[c] = v;
  }
}

// Threads per row, vectors per thread and threads per block for rows of d channels in
// vectors of V.
struct RowPlan {
  int tpr, k, block;
};
RowPlan elem_plan(int d) {
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
RowPlan rows_plan(int d, int lanes_k) {
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

int back_blocks(const NormArgs& a, const RowPlan& p) {
  const long rpb = p.block / p.tpr;
  const long need = (a.rows + rpb - 1) / rpb;
  const long most = (long)kSMs * (1536 / (p.block < 256 ? 256 : p.block));
  return (int)(need < most ? need : most);
}

// Blocks an SM for a kernel that needs `smem` bytes a block, at most `most`.
int resident(size_t smem, int most) {
  const int n = (int)((size_t)224 * 1024 / (smem + 1024));
  return n < 1 ? 1 : n < most ? n : most;
}

template <int XB, int RB, int K>
int forward_ring(const NormArgs& a, int threads, size_t smem, cudaStream_t st) {
  auto* f = norm_forward_ring<XB, RB, K>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATLAS_ERR_CUDA;
  const long most = (long)kSMs * resident(smem, 8 * 256 / threads);
  f<<<(unsigned)(a.rows < most ? a.rows : most), threads, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <int XB, int RB>
int forward_rows(const NormArgs& a, cudaStream_t st) {
  // rows of up to 256 channels: lanes of a warp; longer ones: a block
  const bool few = a.rows <= kSMs * 8;
  const RowPlan p = rows_plan(a.d, 1);
  const size_t ring = 512 + (size_t)kStages * a.d * (XB + RB);
  if (!few && p.tpr > 32 && ring <= 200 * 1024) {
    if (p.k == 1) return forward_ring<XB, RB, 1>(a, p.block, ring, st);
    if (p.k == 2) return forward_ring<XB, RB, 2>(a, p.block, ring, st);
    if (p.k == 4) return forward_ring<XB, RB, 4>(a, p.block, ring, st);
    return forward_ring<XB, RB, 8>(a, p.block, ring, st);
  }
  const int rpb = p.block / p.tpr;
  const int R = p.k == 1 && p.tpr <= 32 && !few ? 4 : 1;  // short rows: four under way
  const long blocks = (a.rows + (long)rpb * R - 1) / ((long)rpb * R);
  if (blocks > 0x7FFFFFFFL) return ATLAS_ERR_UNSUPPORTED;
  const size_t smem = 64 * 4;
  if (p.k == 1 && R == 4)
    norm_forward_rows<XB, RB, 1, 4><<<(unsigned)blocks, p.block, smem, st>>>(a, p.tpr);
  else if (p.k == 1)
    norm_forward_rows<XB, RB, 1, 1><<<(unsigned)blocks, p.block, smem, st>>>(a, p.tpr);
  else if (p.k == 2)
    norm_forward_rows<XB, RB, 2, 1><<<(unsigned)blocks, p.block, smem, st>>>(a, p.tpr);
  else if (p.k == 4)
    norm_forward_rows<XB, RB, 4, 1><<<(unsigned)blocks, p.block, smem, st>>>(a, p.tpr);
  else
    norm_forward_rows<XB, RB, 8, 1><<<(unsigned)blocks, p.block, smem, st>>>(a, p.tpr);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <int HB, int DB, int GB, int K, int MT>
int backward_rows(const NormArgs& a, const RowPlan& p, int& blocks, cudaStream_t st) {
  const size_t ring = (size_t)kStages * (p.block / p.tpr) * a.d * (HB + DB + GB), sums = (size_t)a.d * 4;
  const size_t smem = 256 + (ring > sums ? ring : sums);
  auto* f = norm_backward_rows<HB, DB, GB, K, MT>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATLAS_ERR_CUDA;
  // no more blocks than run at once
  const int most = kSMs * resident(smem, (MT == 320 ? 640 : 512) / p.block);
  blocks = blocks < most ? blocks : most;
  f<<<blocks, p.block, smem, st>>>(a, p.tpr);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}
template <int HB, int DB, int GB>
int backward_rows(const NormArgs& a, const RowPlan& p, int& blocks, cudaStream_t st) {
  if (p.k == 1 && p.block <= 320) return backward_rows<HB, DB, GB, 1, 320>(a, p, blocks, st);
  if (p.k == 1) return backward_rows<HB, DB, GB, 1, 512>(a, p, blocks, st);
  return backward_rows<HB, DB, GB, 2, 512>(a, p, blocks, st);
}

// Rows whose registers and ring the backward kernel can hold: three rows of h, dy and dh.
bool back_wide(const NormArgs& a) {
  const int hb = a.rt == ATLAS_F32 ? 4 : 2, db = a.dt == ATLAS_F32 ? 4 : 2;
  return a.wide && a.d <= 8192 && (size_t)kStages * a.d * (2 * hb + db) <= 200 * 1024;
}

}  // namespace

int norm_forward_launch(const NormArgs& args, cudaStream_t st) {
  // a group of an 8-bit output in neighbouring lanes of one warp: a power of two from 8 to 256
  NormArgs a = args;
  a.inv_d = 1.f / a.d;
  if (a.eps == 0.f) a.eps = std::numeric_limits<float>::denorm_min();  // 2^-149, nothing beside a row's own mean
  a.ng = a.group ? (a.d + a.group - 1) / a.group : 1;
  for (a.gshift = 0; (1 << a.gshift) < a.group;) ++a.gshift;
  const bool lanes = a.group == 0 || (a.group >= 8 && a.group <= 256 && (a.group & (a.group - 1)) == 0);
  if (a.wide && lanes) {
    const int xb = a.dt == ATLAS_F32 ? 4 : 2, rb = !a.r ? 0 : a.rt == ATLAS_F32 ? 4 : 2;
    if (xb == 2) return rb == 0 ? forward_rows<2, 0>(a, st) : rb == 2 ? forward_rows<2, 2>(a, st) : forward_rows<2, 4>(a, st);
    return rb == 0 ? forward_rows<4, 0>(a, st) : rb == 2 ? forward_rows<4, 2>(a, st) : forward_rows<4, 4>(a, st);
  }
  const RowPlan p = elem_plan(a.d);
  const int rpb = p.block / p.tpr;
  const long blocks = (a.rows + rpb - 1) / rpb;
  if (blocks > 0x7FFFFFFFL) return ATLAS_ERR_UNSUPPORTED;
  const int ng = a.group ? (a.d + a.group - 1) / a.group : 0;
  const size_t smem = (64 + (size_t)rpb * ng) * 4;
  const int xb = a.dt == ATLAS_F32 ? 4 : 2, rb = !a.r ? 0 : a.rt == ATLAS_F32 ? 4 : 2;
  auto pick = [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (xb == 2) return rb == 0 ? norm_forward_elem<2, 0, K> : rb == 2 ? norm_forward_elem<2, 2, K> : norm_forward_elem<2, 4, K>;
    return rb == 0 ? norm_forward_elem<4, 0, K> : rb == 2 ? norm_forward_elem<4, 2, K> : norm_forward_elem<4, 4, K>;
  };
  auto* f = p.k == 8 ? pick(std::integral_constant<int, 8>()) : pick(std::integral_constant<int, 32>());
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATLAS_ERR_CUDA;
  f<<<(unsigned)blocks, p.block, smem, st>>>(a, p.tpr);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

size_t norm_backward_workspace(const NormArgs& a) {
  const int n1 = back_blocks(a, elem_plan(a.d)), n8 = back_blocks(a, rows_plan(a.d, 1));
  return (size_t)(n1 > n8 ? n1 : n8) * a.d * 4;
}

int norm_backward_launch(const NormArgs& args, cudaStream_t st) {
  NormArgs a = args;
  a.inv_d = 1.f / a.d;
  const bool wide = back_wide(a);
  const RowPlan p = wide ? rows_plan(a.d, 1) : elem_plan(a.d);
  int blocks = back_blocks(a, p);
  if (blocks > 0 && wide) {
    const int hb = a.rt == ATLAS_F32 ? 4 : 2, db = a.dt == ATLAS_F32 ? 4 : 2;
    int rc;
    if (hb == 2 && db == 2)
      rc = a.r ? backward_rows<2, 2, 2>(a, p, blocks, st) : backward_rows<2, 2, 0>(a, p, blocks, st);
    else if (hb == 2)
      rc = a.r ? backward_rows<2, 4, 2>(a, p, blocks, st) : backward_rows<2, 4, 0>(a, p, blocks, st);
    else if (db == 2)
      rc = a.r ? backward_rows<4, 2, 4>(a, p, blocks, st) : backward_rows<4, 2, 0>(a, p, blocks, st);
    else
      rc = a.r ? backward_rows<4, 4, 4>(a, p, blocks, st) : backward_rows<4, 4, 0>(a, p, blocks, st);
    if (rc != ATLAS_OK) return rc;
  } else if (blocks > 0) {
    const size_t smem = (64 + (size_t)(p.block > p.tpr ? a.d : 0)) * 4;
    const int hb = a.rt == ATLAS_F32 ? 4 : 2, db = a.dt == ATLAS_F32 ? 4 : 2;
    auto pick = [&](auto k) {
      constexpr int K = decltype(k)::value;
      if (hb == 2) return db == 2 ? norm_backward_elem<2, 2, K> : norm_backward_elem<2, 4, K>;
      return db == 2 ? norm_backward_elem<4, 2, K> : norm_backward_elem<4, 4, K>;
    };
    auto* f = p.k == 8 ? pick(std::integral_constant<int, 8>()) : pick(std::integral_constant<int, 32>());
    f<<<blocks, p.block, smem, st>>>(a, p.tpr);
  }
  if (a.dw) norm_dw_kernel<<<(a.d + 31) / 32, 256, 0, st>>>(a.part, a.dw, blocks, a.d);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // namespace atlas
