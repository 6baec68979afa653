// norm.cu -- residual addition and root-mean-square norm, with an output in 32, 16 or
// 8 bits, and its backward pass.
//
//   h = x + r,  y = h rstd w,  rstd = 1 / sqrt(mean(h^2) + eps)
//   dx = rstd (w dy - hat mean(w dy hat)) + dh,  dw = sum over rows of dy hat,  hat = h rstd
//
// Both passes are bound by memory: a row is read once into registers, reduced, and
// written once.  A row of at most 1024 channels belongs to 8, 16 or 32 lanes of a warp
// (keys and queries: one row is one head), a longer one to a block.  Sums run in 32
// bits; the only roundings are those of the outputs to their types.
#include <cuda_fp8.h>

#include "ops_common.cuh"

namespace atlas {
namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kAmaxMin = 1e-30f;

// V consecutive elements (1 or 8) of a type known at run time.
template <int V>
__device__ __forceinline__ void ld_row(const void* p, long i, int dtype, float* v) {
  if (V == 1) {
    v[0] = ld_any(p, i, dtype);
    return;
  }
  if (dtype == ATLAS_F32) {
    const auto* q = reinterpret_cast<const float*>(p) + i;
    const auto a = ld_pack<float, 4>(q), b = ld_pack<float, 4>(q + 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = a.e[k], v[4 + k] = b.e[k];
  } else if (dtype == ATLAS_BF16) {
    const auto a = ld_pack<__nv_bfloat16, 8>(reinterpret_cast<const __nv_bfloat16*>(p) + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = a.get(k);
  } else {
    const auto a = ld_pack<__half, 8>(reinterpret_cast<const __half*>(p) + i);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = a.get(k);
  }
}

template <typename T, int V>
__device__ __forceinline__ void st_as(void* p, long i, const float* v) {
  Pack<T, V> a;
#pragma unroll
  for (int k = 0; k < V; ++k) a.set(k, v[k]);
  st_pack<T, V>(reinterpret_cast<T*>(p) + i, a);
}

template <int V>
__device__ __forceinline__ void st_row(void* p, long i, int dtype, const float* v) {
  if (dtype == ATLAS_F32) {
    if (V == 1) {
      reinterpret_cast<float*>(p)[i] = v[0];
    } else {
      st_as<float, 4>(p, i, v);
      st_as<float, 4>(p, i + 4, v + 4);
    }
  } else if (dtype == ATLAS_BF16) {
    st_as<__nv_bfloat16, V>(p, i, v);
  } else if (dtype == ATLAS_F16) {
    st_as<__half, V>(p, i, v);
  } else {  // e4m3, to nearest even; the values are within +-448 by their scale
    alignas(8) __nv_fp8_storage_t q[V];
#pragma unroll
    for (int k = 0; k < V; ++k) q[k] = __nv_cvt_float_to_fp8(v[k], __NV_SATFINITE, __NV_E4M3);
    auto* o = reinterpret_cast<__nv_fp8_storage_t*>(p) + i;
    if (V == 8)
      *reinterpret_cast<uint2*>(o) = *reinterpret_cast<const uint2*>(q);
    else
      o[0] = q[0];
  }
}

// The threads that share a row: TPR lanes of a warp (TPR <= 32), or the whole block.
struct RowGroup {
  int tpr, lane, tid;  // threads per row, lane within them
};

__device__ __forceinline__ float row_sum(float v, const RowGroup& g, float* red) {
  for (int m = min(g.tpr, 32) >> 1; m; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  if (g.tpr > 32) {
    const int nw = g.tpr >> 5;
    __syncthreads();
    if ((g.tid & 31) == 0) red[g.tid >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < nw; ++i) v += red[i];
  }
  return v;
}
// NaN stays out of a maximum (fmaxf), as it does of its scale; the element itself stays NaN.
__device__ __forceinline__ float row_max(float v, const RowGroup& g, float* red) {
  for (int m = min(g.tpr, 32) >> 1; m; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, m));
  if (g.tpr > 32) {
    const int nw = g.tpr >> 5;
    __syncthreads();
    if ((g.tid & 31) == 0) red[g.tid >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < nw; ++i) v = fmaxf(v, red[i]);
  }
  return v;
}

template <int V, int K>
__global__ void __launch_bounds__(V == 8 ? 512 : 1024) norm_forward_kernel(NormArgs a, int tpr) {
  extern __shared__ float sm[];  // 32 floats, then (8-bit groups that cross lanes) the groups' maxima
  float* red = sm;
  const RowGroup g{tpr, (int)threadIdx.x % tpr, (int)threadIdx.x};
  const int rpb = blockDim.x / tpr;
  const long row = (long)blockIdx.x * rpb + threadIdx.x / tpr;
  const bool live = row < a.rows;
  float h[K][V];
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * tpr + g.lane) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) h[k][j] = 0.f;
    if (live && c < a.d) {
      ld_row<V>(a.x, row * a.sx + c, a.dt, h[k]);
      if (a.r) {
        float r[V];
        ld_row<V>(a.r, row * a.sr + c, a.rt, r);
#pragma unroll
        for (int j = 0; j < V; ++j) h[k][j] += r[j];
      }
      if (a.r_out) st_row<V>(a.r_out, row * a.sr + c, a.rt, h[k]);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) ss += h[k][j] * h[k][j];
  }
  const float rstd = rsqrtf(row_sum(ss, g, red) / a.d + a.eps);
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * tpr + g.lane) * V;
    if (c < a.d) {
      float w[V];
      if (a.w) ld_row<V>(a.w, c, a.wt, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        h[k][j] *= rstd;
        if (a.w) h[k][j] *= w[j];
        amax = fmaxf(amax, fabsf(h[k][j]));
      }
      if (live && a.ot != ATLAS_E4M3) st_row<V>(a.y, row * a.sy + c, a.ot, h[k]);
    }
  }
  if (a.ot != ATLAS_E4M3) return;
  if (a.group == 0) {
    const float scale = fmaxf(row_max(amax, g, red), kAmaxMin) * (1.f / kE4m3Max);
    const float inv = 1.f / scale;
    if (live && g.lane == 0) a.scale[row] = scale;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * tpr + g.lane) * V;
      if (live && c < a.d) {
#pragma unroll
        for (int j = 0; j < V; ++j) h[k][j] *= inv;
        st_row<V>(a.y, row * a.sy + c, a.ot, h[k]);
      }
    }
    return;
  }
  // groups of channels: maxima of non-negative floats order like their bits, so integer
  // maxima in shared memory give the same result in any order
  const int ng = (a.d + a.group - 1) / a.group;
  unsigned* gm = reinterpret_cast<unsigned*>(sm + 32) + (threadIdx.x / tpr) * ng;
  for (int i = g.lane; i < ng; i += tpr) gm[i] = 0u;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * tpr + g.lane) * V;
    if (c < a.d) {
      if (V == 1 || a.group % V == 0) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) m = fmaxf(m, fabsf(h[k][j]));
        atomicMax(&gm[c / a.group], __float_as_uint(m));
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          atomicMax(&gm[(c + j) / a.group], __float_as_uint(fmaxf(0.f, fabsf(h[k][j]))));
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * tpr + g.lane) * V;
    if (live && c < a.d) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        h[k][j] *= 1.f / (fmaxf(__uint_as_float(gm[(c + j) / a.group]), kAmaxMin) * (1.f / kE4m3Max));
      st_row<V>(a.y, row * a.sy + c, a.ot, h[k]);
    }
  }
  if (live)
    for (int i = g.lane; i < ng; i += tpr)
      a.scale[row * ng + i] = fmaxf(__uint_as_float(gm[i]), kAmaxMin) * (1.f / kE4m3Max);
}

// A block walks the rows blockIdx.x * rpb + .., step gridDim.x * rpb; each thread keeps the
// sums of dy hat of its columns over its rows, and the block writes one row of partial sums.
template <int V, int K>
__global__ void __launch_bounds__(V == 8 ? 512 : 1024) norm_backward_kernel(NormArgs a, int tpr) {
  extern __shared__ float sm[];
  float* red = sm;
  const RowGroup g{tpr, (int)threadIdx.x % tpr, (int)threadIdx.x};
  const int rpb = blockDim.x / tpr;
  float dw[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) dw[k][j] = 0.f;
  for (long row0 = (long)blockIdx.x * rpb; row0 < a.rows; row0 += (long)gridDim.x * rpb) {
    const long row = row0 + threadIdx.x / tpr;
    const bool live = row < a.rows;
    float h[K][V], dy[K][V], ss = 0.f, dot = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * tpr + g.lane) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) h[k][j] = dy[k][j] = 0.f;
      if (live && c < a.d) {
        ld_row<V>(a.x, row * a.sr + c, a.rt, h[k]);
        ld_row<V>(a.dy, row * a.sy + c, a.dt, dy[k]);
        float w[V];
        if (a.w) ld_row<V>(a.w, c, a.wt, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          ss += h[k][j] * h[k][j];
          dot += h[k][j] * (a.w ? w[j] * dy[k][j] : dy[k][j]);
        }
      }
    }
    ss = row_sum(ss, g, red);
    dot = row_sum(dot, g, red);
    const float rstd = rsqrtf(ss / a.d + a.eps);
    const float mean = dot * rstd / a.d;  // mean(w dy hat)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * tpr + g.lane) * V;
      if (live && c < a.d) {
        float w[V], o[V];
        if (a.w) ld_row<V>(a.w, c, a.wt, w);
        if (a.r) ld_row<V>(a.r, row * a.sr + c, a.rt, o);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float hat = h[k][j] * rstd;
          const float wdy = a.w ? w[j] * dy[k][j] : dy[k][j];
          dw[k][j] += dy[k][j] * hat;
          o[j] = rstd * (wdy - hat * mean) + (a.r ? o[j] : 0.f);
        }
        st_row<V>(a.y, row * a.sr + c, a.rt, o);
      }
    }
  }
  if (!a.dw) return;
  // rows of one block are added in a fixed order
  float* acc = sm + 32;
  const int mine = threadIdx.x / tpr;
  for (int r = 0; r < rpb; ++r) {
    __syncthreads();
    if (r == mine) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (k * tpr + g.lane) * V;
        if (c < a.d) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float s = (r == 0 ? 0.f : acc[c + j]) + dw[k][j];
            if (r == rpb - 1)
              a.part[(long)blockIdx.x * a.d + c + j] = s;
            else
              acc[c + j] = s;
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
// vectors of V.  Rows up to 32 x 4 vectors: lanes of a warp; longer: a block with at most
// `most` vectors a thread.
struct RowPlan {
  int tpr, k, block;
};
RowPlan row_plan(int d, int V, int most) {
  const int nv = (d + V - 1) / V;
  RowPlan p;
  if (nv <= 128) {
    p.tpr = nv <= 8 ? 8 : nv <= 16 ? 16 : 32;
    p.k = (nv + p.tpr - 1) / p.tpr;
    p.block = 256;
  } else {
    p.k = most;
    while (p.k < 32 && (nv + p.k - 1) / p.k > (V == 8 ? 512 : 1024)) p.k *= 2;
    p.tpr = ((nv + p.k - 1) / p.k + 31) / 32 * 32;
    p.block = p.tpr;
  }
  p.k = p.k <= 1 ? 1 : p.k <= 2 ? 2 : p.k <= 4 ? 4 : p.k <= 8 ? 8 : 32;
  return p;
}

int back_blocks(const NormArgs& a, const RowPlan& p) {
  const long rpb = p.block / p.tpr;
  const long need = (a.rows + rpb - 1) / rpb;
  const long most = 152L * (2048 / (p.block < 256 ? 256 : p.block)) / 2;
  return (int)(need < most ? need : most);
}

}  // namespace

int norm_forward_launch(const NormArgs& a, cudaStream_t st) {
  const int V = a.wide ? 8 : 1;
  const RowPlan p = row_plan(a.d, V, 2);
  const int rpb = p.block / p.tpr;
  const long blocks = (a.rows + rpb - 1) / rpb;
  if (blocks > 0x7FFFFFFFL) return ATLAS_ERR_UNSUPPORTED;
  const int ng = a.group ? (a.d + a.group - 1) / a.group : 0;
  const size_t smem = (32 + (size_t)rpb * ng) * 4;
#define ATLAS_RUN(VV, KK)                                                                      \
  do {                                                                                         \
    if (smem > 48 * 1024 &&                                                                    \
        cudaFuncSetAttribute(norm_forward_kernel<VV, KK>,                                      \
                             cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=        \
            cudaSuccess)                                                                       \
      return ATLAS_ERR_CUDA;                                                                   \
    norm_forward_kernel<VV, KK><<<(unsigned)blocks, p.block, smem, st>>>(a, p.tpr);            \
  } while (0)
  if (V == 8) {
    if (p.k == 1) ATLAS_RUN(8, 1);
    else if (p.k == 2) ATLAS_RUN(8, 2);
    else if (p.k == 4) ATLAS_RUN(8, 4);
    else ATLAS_RUN(8, 8);
  } else {
    if (p.k <= 4) ATLAS_RUN(1, 4); else ATLAS_RUN(1, 32);
  }
#undef ATLAS_RUN
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

size_t norm_backward_workspace(const NormArgs& a) {
  const RowPlan p1 = row_plan(a.d, 1, 4), p8 = row_plan(a.d, 8, 2);
  const int n1 = back_blocks(a, p1), n8 = back_blocks(a, p8);
  return (size_t)(n1 > n8 ? n1 : n8) * a.d * 4;
}

int norm_backward_launch(const NormArgs& a, cudaStream_t st) {
  const int V = a.wide ? 8 : 1;
  const RowPlan p = row_plan(a.d, V, V == 8 ? 2 : 4);
  const int blocks = back_blocks(a, p);
  const size_t smem = (32 + (size_t)(p.block > p.tpr ? a.d : 0)) * 4;
  if (blocks > 0) {
    if (V == 8) {
      if (p.k == 1) norm_backward_kernel<8, 1><<<blocks, p.block, smem, st>>>(a, p.tpr);
      else if (p.k == 2) norm_backward_kernel<8, 2><<<blocks, p.block, smem, st>>>(a, p.tpr);
      else if (p.k == 4) norm_backward_kernel<8, 4><<<blocks, p.block, smem, st>>>(a, p.tpr);
      else norm_backward_kernel<8, 8><<<blocks, p.block, smem, st>>>(a, p.tpr);
    } else {
      if (p.k <= 4) norm_backward_kernel<1, 4><<<blocks, p.block, smem, st>>>(a, p.tpr);
      else norm_backward_kernel<1, 32><<<blocks, p.block, smem, st>>>(a, p.tpr);
    }
  }
  if (a.dw) norm_dw_kernel<<<(a.d + 31) / 32, 256, 0, st>>>(a.part, a.dw, blocks, a.d);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // namespace atlas
