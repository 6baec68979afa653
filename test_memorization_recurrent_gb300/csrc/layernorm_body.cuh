// layernorm_body.cuh -- residual addition and layer norm, with an output in 32, 16 or 8 bits.
//
//   h = x + r,  mu = mean h,  v = mean (h - mu)^2,  y = (h - mu) / sqrt(v + eps) w + b
//
// A row stays in registers from its load to its output, so the variance is taken of the deviations
// themselves: a sum, then the sums of (h - m) and (h - m)^2 about the rounded mean m.  The first of
// the two is what m's rounding left out, and enters mu and v: rows whose mean is large beside their
// deviations lose nothing by the sum's roundings.
//
// Rows of up to 256 channels belong to lanes of a warp, four rows under way; longer ones to a block,
// which walks rows with the next two on their way through shared memory (a few rows: a block each).
// A thread has K times eight elements: eight neighbours of an aligned row, every tpr-th one of a row
// that starts anywhere.  Such rows come to shared memory in whole pieces of 16 bytes too, from the
// boundary in front of the row on, and keep their distance from it there; neighbouring lanes then
// read and store neighbouring elements.
#pragma once
#include "rows.cuh"

namespace atlas {
namespace layernorm {

typedef LayerNormArgs Args;

constexpr int kStages = 3;
constexpr int kRed = 64;  // floats that a block's sums meet in: 16 sums, 16 pairs, 16 maxima

// Column of element i of vector k.
template <bool AL>
__device__ __forceinline__ int col(int k, int i, int tpr, int lane) {
  return AL ? (k * tpr + lane) * 8 + i : (k * 8 + i) * tpr + lane;
}

// Two sums over a row's threads, as row_reduce; words past the last warp's pair are zero.
__device__ __forceinline__ void row_sums2(float& x, float& y, const RowGroup& g, float* red) {
  for (int m = min(g.tpr, 32) >> 1; m; m >>= 1) {
    x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
    y += __shfl_xor_sync(0xFFFFFFFFu, y, m);
  }
  if (g.tpr > 32) {
    if ((g.tid & 31) == 0) *reinterpret_cast<float2*>(red + (g.tid >> 5) * 2) = make_float2(x, y);
    __syncthreads();
    x = y = 0.f;
    for (int i = 0; i < (g.tpr + 63) / 64; ++i) {
      const float4 t = reinterpret_cast<const float4*>(red)[i];
      x += t.x + t.z;
      y += t.y + t.w;
    }
  }
}

// Parameters of vector k: eight of a type, `none` without a tensor.
template <bool AL>
__device__ __forceinline__ void load_params(const void* p, int type, float none, int k, int d, int tpr, int lane, float* w) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = none;
  if (!p) return;
  if (AL) {
    const int c = col<AL>(k, 0, tpr, lane);
    if (c >= d) return;
    if (type == ATLAS_F32) {
      Raw8<4> q;
      q.load_kept(p, c);
      q.floats(type, w);
    } else {
      Raw8<2> q;
      q.load_kept(p, c);
      q.floats(type, w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col<AL>(k, i, tpr, lane);
      if (c < d) w[i] = ld_any(p, c, type);
    }
  }
}

// A thread's weights and biases: kept in registers, or, of long rows (more than two vectors a thread), read
// again for each row.
template <int K, bool AL>
struct Params {
  static constexpr bool kKept = K <= 2;
  float w[kKept ? K : 1][8], b[kKept ? K : 1][8];
  __device__ __forceinline__ void load(const Args& a, int tpr, int lane) {
    if constexpr (kKept) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        load_params<AL>(a.w, a.wt, 1.f, k, a.d, tpr, lane, w[k]);
        load_params<AL>(a.b, a.wt, 0.f, k, a.d, tpr, lane, b[k]);
      }
    }
  }
  __device__ __forceinline__ void apply(const Args& a, int k, int tpr, int lane, float* h) {
    if constexpr (!kKept) {
      load_params<AL>(a.w, a.wt, 1.f, k, a.d, tpr, lane, w[0]);
      load_params<AL>(a.b, a.wt, 0.f, k, a.d, tpr, lane, b[0]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = fmaf(h[i], w[kKept ? k : 0][i], b[kKept ? k : 0][i]);
  }
};

// Eight elements of a row that lies at p (`live` and inside the row), aligned or not; zeros elsewhere.
template <int BYTES, bool AL>
struct Raw {
  Raw8<BYTES> v;
  __device__ __forceinline__ void load(const void* p, long at, int k, int d, int tpr, int lane, bool live) {
    v.zero();
    if (BYTES == 0) return;
    if (AL) {
      const int c = col<AL>(k, 0, tpr, lane);
      if (live && c < d) v.load(p, at + c);
    }
  }
  __device__ __forceinline__ void floats(int type, float* f) const { v.floats(type, f); }
};
template <int BYTES>
struct Raw<BYTES, false> {
  uint32_t v[8];
  __device__ __forceinline__ void load(const void* p, long at, int k, int d, int tpr, int lane, bool live) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col<false>(k, i, tpr, lane);
      v[i] = BYTES && live && c < d ? ld_raw<BYTES>(p, at + c) : 0u;
    }
  }
  __device__ __forceinline__ void floats(int type, float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = BYTES ? raw_float<BYTES>(v[i], type) : 0.f;
  }
};

// Eight outputs of vector k.
template <bool AL>
__device__ __forceinline__ void store(void* p, long at, int type, int k, int d, int tpr, int lane, const float* v) {
  if (AL) {
    const int c = col<AL>(k, 0, tpr, lane);
    if (c < d) st8(p, at + c, type, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col<AL>(k, i, tpr, lane);
      if (c < d) st_elem(p, at + c, type, v[i]);
    }
  }
}

// One row from its elements h (zeros past its end).  red: kRed words; gm: this row's a.ng words for the
// maxima of groups that are not neighbouring lanes' (every thread of the block comes here then).
template <int K, bool AL>
__device__ __forceinline__ void forward_row(const Args& a, const RowGroup& g, float* red, unsigned* gm, long row,
                                            bool live, float (*h)[8], Params<K, AL>& par) {
  const auto in = [&](int k, int i) { return col<AL>(k, AL ? 0 : i, g.tpr, g.lane) < a.d; };
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (a.r_out && live) store<AL>(a.r_out, row * a.sr, a.rt, k, a.d, g.tpr, g.lane, h[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += h[k][i];
  }
  const float mean = row_sum(sum, g, red) * a.inv_d;
  float rest = 0.f, ss = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      h[k][i] = in(k, i) ? h[k][i] - mean : 0.f;
      rest += h[k][i];
      ss = fmaf(h[k][i], h[k][i], ss);
    }
  row_sums2(rest, ss, g, red + 16);
  rest *= a.inv_d;
  const float rstd = rsqrtf(fmaxf(fmaf(ss, a.inv_d, -rest * rest), 0.f) + a.eps), off = -rest * rstd;
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[k][i] = fmaf(h[k][i], rstd, off);
    par.apply(a, k, g.tpr, g.lane, h[k]);
    if (a.ot != ATLAS_E4M3) {
      if (live) store<AL>(a.y, row * a.sy, a.ot, k, a.d, g.tpr, g.lane, h[k]);
      continue;
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (in(k, i)) m = fmaxf(m, fabsf(h[k][i]));
    if (a.group == 0 || !a.lanes) {
      amax = fmaxf(amax, m);
      continue;
    }
    // the group's lanes are neighbours: group / 8 of them, a power of two
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (8 * o < a.group) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float scale = scale_of(m), inv = inverse(scale);
    const int c = col<AL>(k, 0, g.tpr, g.lane);
    if (live && c < a.d) {
      if ((c & (a.group - 1)) == 0) a.scale[row * a.ng + (c >> a.gshift)] = scale;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] *= inv;
      st8(a.y, row * a.sy + c, a.ot, h[k]);
    }
  }
  if (a.ot != ATLAS_E4M3 || (a.group && a.lanes)) return;
  float inv = 0.f;
  if (a.group == 0) {
    const float scale = scale_of(row_max(amax, g, red + 48));
    inv = inverse(scale);
    if (live && g.lane == 0) a.scale[row] = scale;
  } else {
    // maxima of non-negative floats order like their bits, so integer maxima in shared memory
    // give the same result in any order
    for (int i = g.lane; i < a.ng; i += g.tpr) gm[i] = 0u;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = col<AL>(k, i, g.tpr, g.lane);
        if (c < a.d) atomicMax(&gm[c / a.group], __float_as_uint(fmaxf(0.f, fabsf(h[k][i]))));
      }
    __syncthreads();
    for (int i = g.lane; i < a.ng; i += g.tpr) {
      const float scale = scale_of(__uint_as_float(gm[i]));
      if (live) a.scale[row * a.ng + i] = scale;
      gm[i] = __float_as_uint(inverse(scale));
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col<AL>(k, i, g.tpr, g.lane);
      h[k][i] *= a.group == 0 ? inv : c < a.d ? __uint_as_float(gm[c / a.group]) : 0.f;
    }
    if (live) store<AL>(a.y, row * a.sy, a.ot, k, a.d, g.tpr, g.lane, h[k]);
  }
}

// R rows at a time, straight from memory.  tpr threads a row: up to 32 lanes, or the whole block (R = 1).
template <int XB, int RB, int K, int R, bool AL>
__global__ void __launch_bounds__(512) forward_rows(Args a, int tpr) {
  extern __shared__ __align__(16) float sm[];
  if (tpr > 32) clear_red(sm, kRed);
  const RowGroup g{tpr, (int)threadIdx.x % tpr, (int)threadIdx.x};
  const int rpb = blockDim.x / tpr, mine = threadIdx.x / tpr;
  const long row0 = (long)blockIdx.x * rpb * R + mine;
  Raw<XB, AL> x[R][K];
  Raw<RB, AL> r[R][K];
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long row = row0 + j * rpb;
      x[j][k].load(a.x, row * a.sx, k, a.d, tpr, g.lane, row < a.rows);
      r[j][k].load(a.r, row * a.sr, k, a.d, tpr, g.lane, row < a.rows);
    }
  Params<K, AL> par;
  par.load(a, tpr, g.lane);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    float h[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[j][k].floats(a.dt, h[k]);
      if (RB) {
        float v[8];
        r[j][k].floats(a.rt, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] += v[i];
      }
    }
    forward_row<K, AL>(a, g, sm, reinterpret_cast<unsigned*>(sm + kRed) + mine * a.ng, row0 + j * rpb,
                       row0 + j * rpb < a.rows, h, par);
  }
}

// ------------------------------------------------------- rows through shared memory

// A tensor of rows and what of it may be read.
struct Rows {
  const char *lo, *hi;  // its first byte, the byte behind its last row
  long stride;          // bytes from row to row
};
template <int E>
__device__ __forceinline__ Rows rows_of(const void* p, long stride, long rows, int d) {
  const char* lo = reinterpret_cast<const char*>(p);
  return Rows{lo, lo + ((rows - 1) * stride + d) * E, stride * E};
}

// Bytes that a row of d elements takes in shared memory.
template <int E, bool AL>
__host__ __device__ __forceinline__ int slot_bytes(int d) {
  return AL || E == 0 ? d * E : (d * E + 30) / 16 * 16;
}

// Distance of a row's first byte from the boundary of 16 in front of it.
__device__ __forceinline__ int ahead(const Rows& t, long row) {
  return (int)(reinterpret_cast<uintptr_t>(t.lo + row * t.stride) & 15);
}

// One row to shared memory; Q pieces of 16 bytes a thread cover an aligned one.  The pieces at the ends of a row that starts
// anywhere hold bytes of its neighbours or of the gaps between rows, which nothing uses; those that reach
// beyond the tensor's ends come element by element.
template <int E, int Q, bool AL>
__device__ __forceinline__ void fetch_row(char* s, const Rows& t, long row, long rows, int d, int lane, int threads) {
  if (E == 0) return;
  if (AL) {
    copy_row<Q>(s, t.lo, row * t.stride, d * E, row < rows, lane, threads);
    return;
  }
  if (row >= rows) return;
  const int shift = ahead(t, row), n = shift + d * E;
  const char* p = t.lo + row * t.stride - shift;
#pragma unroll
  for (int k = 0; k <= Q; ++k) {
    const int i = (k * threads + lane) * 16;
    if (i >= n) continue;
    if (p + i >= t.lo && p + i + 16 <= t.hi) {
      cp_async<16>(s + i, p + i, true);
    } else {
      for (int j = i; j < i + 16; j += E > 0 ? E : 1)
        if (p + j >= t.lo && p + j < t.hi) {
          if (E == 2) *reinterpret_cast<uint16_t*>(s + j) = *reinterpret_cast<const uint16_t*>(p + j);
          if (E == 4) *reinterpret_cast<uint32_t*>(s + j) = *reinterpret_cast<const uint32_t*>(p + j);
        }
    }
  }
}

// Vector k of a row in shared memory, zeros past its end.
template <int E, bool AL>
__device__ __forceinline__ void slot_floats(const char* s, int shift, int type, int k, int d, int tpr, int lane, float* f) {
  if (AL) {
    Raw8<E> q;
    q.zero();
    const int c = col<AL>(k, 0, tpr, lane);
    if (c < d) q.load_kept(s, c);
    q.floats(type, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col<AL>(k, i, tpr, lane);
      f[i] = c < d ? raw_float<E>(ld_raw<E>(s + shift, c), type) : 0.f;
    }
  }
}

template <int XB, int RB, int K, bool AL>
__global__ void __launch_bounds__(512) forward_ring(Args a) {
  extern __shared__ __align__(16) float sm[];  // [kRed], [stage]: x, r, then the groups' maxima
  clear_red(sm, kRed);
  const RowGroup g{(int)blockDim.x, (int)threadIdx.x, (int)threadIdx.x};
  const int xs = slot_bytes<XB, AL>(a.d), bytes = xs + slot_bytes<RB, AL>(a.d);
  char* ring = reinterpret_cast<char*>(sm + kRed);
  unsigned* gm = reinterpret_cast<unsigned*>(ring + kStages * bytes);
  const Rows tx = rows_of<XB>(a.x, a.sx, a.rows, a.d), tr = rows_of<RB>(a.r, a.sr, a.rows, a.d);
  auto fetch = [&](long row, int stage) {
    char* s = ring + stage * bytes;
    fetch_row<XB, K * XB / 2, AL>(s, tx, row, a.rows, a.d, g.lane, g.tpr);
    fetch_row<RB, K * RB / 2, AL>(s + xs, tr, row, a.rows, a.d, g.lane, g.tpr);
    cp_commit();
  };
  Params<K, AL> par;
  par.load(a, g.tpr, g.lane);
  long row = blockIdx.x;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(row + (long)i * gridDim.x, i);
  cp_wait<kStages - 2>();
  __syncthreads();
  int stage = 0;
  for (; row < a.rows; row += gridDim.x) {
    fetch(row + (long)(kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);
    const char* s = ring + stage * bytes;
    float h[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      slot_floats<XB, AL>(s, AL ? 0 : ahead(tx, row), a.dt, k, a.d, g.tpr, g.lane, h[k]);
      if constexpr (RB > 0) {
        float v[8];
        slot_floats<RB, AL>(s + xs, AL ? 0 : ahead(tr, row), a.rt, k, a.d, g.tpr, g.lane, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] += v[i];
      }
    }
    cp_wait<kStages - 2>();  // the next row's copies, handed over by the barriers of this one's sums
    forward_row<K, AL>(a, g, sm, gm, row, true, h, par);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_wait<0>();
}

// ------------------------------------------------------------------ launches

// Rows of up to 256 channels by the lanes that their vectors fill; longer ones by a block.
inline RowPlan forward_plan(int d) {
  RowPlan p = rows_plan(d, 1);
  if (p.tpr <= 32) {
    const int nv = (d + 7) / 8;
    for (p.tpr = 1; p.tpr < nv;) p.tpr *= 2;
  }
  return p;
}

inline int status() { return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA; }

template <typename F>
int shared(F* f, size_t smem) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATLAS_ERR_CUDA;
  return ATLAS_OK;
}

template <int XB, int RB, int K, bool AL>
int run_ring(const Args& a, int threads, size_t smem, cudaStream_t st) {
  auto* f = forward_ring<XB, RB, K, AL>;
  if (const int rc = shared(f, smem)) return rc;
  const long most = (long)kSMs * resident(smem, 8 * 256 / threads);
  f<<<(unsigned)(a.rows < most ? a.rows : most), threads, smem, st>>>(a);
  return status();
}

template <int XB, int RB, int K, int R, bool AL>
int run_rows(const Args& a, const RowPlan& p, cudaStream_t st) {
  const long rpb = p.block / p.tpr, blocks = (a.rows + rpb * R - 1) / (rpb * R);
  if (blocks > 0x7FFFFFFFL) return ATLAS_ERR_UNSUPPORTED;
  const size_t smem = (kRed + (a.lanes ? 0 : (size_t)rpb * a.ng)) * 4;
  auto* f = forward_rows<XB, RB, K, R, AL>;
  if (const int rc = shared(f, smem)) return rc;
  f<<<(unsigned)blocks, p.block, smem, st>>>(a, p.tpr);
  return status();
}

template <int XB, int RB, bool AL>
int forward(const Args& args, cudaStream_t st) {
  Args a = args;
  // a group of an 8-bit output in neighbouring lanes of one warp: a power of two from 8 to 256
  a.lanes = a.ot != ATLAS_E4M3 || a.group == 0 || (AL && a.group >= 8 && a.group <= 256 && (a.group & (a.group - 1)) == 0);
  const RowPlan p = forward_plan(a.d);
  const bool few = a.rows <= kSMs * 8;
  const size_t ring = kRed * 4 + (size_t)kStages * (slot_bytes<XB, AL>(a.d) + slot_bytes<RB, AL>(a.d)) + (a.lanes ? 0 : (size_t)a.ng * 4);
  if (!few && p.tpr > 32 && p.k <= 2 && ring <= 200 * 1024)
    return p.k == 1 ? run_ring<XB, RB, 1, AL>(a, p.block, ring, st) : run_ring<XB, RB, 2, AL>(a, p.block, ring, st);
  if (p.tpr <= 32) return few ? run_rows<XB, RB, 1, 1, AL>(a, p, st) : run_rows<XB, RB, 1, 4, AL>(a, p, st);
  if (p.k == 1) return run_rows<XB, RB, 1, 1, AL>(a, p, st);
  if (p.k == 2) return run_rows<XB, RB, 2, 1, AL>(a, p, st);
  if (p.k == 4) return run_rows<XB, RB, 4, 1, AL>(a, p, st);
  return run_rows<XB, RB, 8, 1, AL>(a, p, st);
}
template <int XB>
int forward(const Args& a, cudaStream_t st) {
  const int rb = !a.r ? 0 : a.rt == ATLAS_F32 ? 4 : 2;
  if (a.wide) return rb == 0 ? forward<XB, 0, true>(a, st) : rb == 2 ? forward<XB, 2, true>(a, st) : forward<XB, 4, true>(a, st);
  return rb == 0 ? forward<XB, 0, false>(a, st) : rb == 2 ? forward<XB, 2, false>(a, st) : forward<XB, 4, false>(a, st);
}

}  // namespace layernorm
}  // namespace atlas
