// layernorm_body.cuh -- residual addition and layer norm, with an output in 32, 16 or 8 bits.
//
//   h = x + r,  mu = mean h,  v = mean (h - mu)^2,  y = (h - mu) / sqrt(v + eps) w + b
//
// A row stays in registers from its load to its output.  Its sums are those of t = h - c, c a number near the row's own:
// mu = c + mean t, v = mean t^2 - (mean t)^2.  A large mean thus enters no sum.  What the difference cancels goes by
// (mean t)^2 / v; where that is above a bound, or t^2 leaves the 32-bit range, the row takes a second round of sums, about
// mu.  So one round, and one barrier of a block, is enough but for few rows of ordinary numbers.
//   An output in 32 bits shows the last places, one in 8 bits has to be what those round to, and gradients are sums of many:
// PRECISE, c is the mean of the first eight elements and the bound 1 (a row of two hundred of ordinary numbers is above).  The
// scaling takes t, and after a second round h less the new c: aligned rows that are still in shared memory are read again there
// (32768 x 2048 bf16 to e4m3: 90 us, so held 94); others are held as h, and mu, as two numbers (c + mean t rounded, and
// what that lost), is taken from h before the scaling.  The rms error is then at most 1.3 times that of two passes, whichever
// elements come first.
//   Outputs in 16 bits of the kernels that walk rows of up to 8192 channels, whose rounding is a thousand times what is lost: c is
// the first element and the bound 16 (some rows of ten thousand), and the row is held as t.  Its error is 2.4 times that of two
// passes in 32 bits, and 17 times with a first element 3.9 deviations from the mean.  (As the others: 524288 x 128 fp32 to bf16 72 us, so 67; 500000 x 40 bf16 + residual 43, so 39.)
//
// Rows of up to 256 channels belong to lanes of a warp; longer ones to a block,
// which walks rows with the next two on their way through shared memory (up to 1216 rows, eight an SM: a block each, straight
// from memory: 8 rows of 2048 in 5.9 us a call, which is the launch).
// A thread has K times eight elements: eight neighbours of an aligned row, every tpr-th one of a row
// that starts anywhere.  Such rows come to shared memory in whole pieces of 16 bytes too, from the
// boundary in front of the row on, and keep their distance from it there; neighbouring lanes then
// read and store neighbouring elements, in 16 bits by pairs where the tensors' rows begin alike.
//
// Bound by memory, and next to it by instructions.  Measured (copy rate 6.79 TB/s): 32768 x 2048 bf16 + residual to e4m3 with
// scales of 128: 90 us, 77% (about the first element: 88; when that was so, a round of sums for the mean and one about it: 119, one
// vector a thread: 115, a warp a row: 135); 524288 x 128 fp32 to bf16: 67 us, 89%; 20000 x 1371 fp16 + residual: 57 us, 56% (one by
// one: 85).
#pragma once
#include <initializer_list>

#include "rows.cuh"

namespace atlas {
namespace layernorm {

typedef LayerNormArgs Args;

constexpr int kStages = 3;
constexpr int kRed = 160;  // floats that a block's sums meet in: twice 16 pairs (rows take turns), 16 pairs, 16 maxima twice

// AL, how a thread's elements lie: 1: eight neighbours; 2: pairs of neighbours, of rows in 16 bits that begin anywhere (four bytes an
// access; a block's rows all begin on the same side of four); 0: one by one.
// Column of element i of vector k.  lane: the thread's place in its row, of pairs (AL == 2) twice that, less one where the
// rows begin between two words.
template <int AL>
__device__ __forceinline__ int col(int k, int i, int tpr, int lane) {
  if (AL == 2) return (k * 4 + i / 2) * 2 * tpr + lane + (i & 1);
  return AL == 1 ? (k * tpr + lane) * 8 + i : (k * 8 + i) * tpr + lane;
}
__device__ __forceinline__ bool inside(int c, int d) { return (unsigned)c < (unsigned)d; }

// Two sums over a row's threads.  A block's warps meet in red: pairs, of which those past the last warp's are
// zero; the next use of the same words has to be another reduction's barrier away.
__device__ __forceinline__ void row_sums2(float& x, float& y, const RowGroup& g, float* red) {
  if (g.tpr >= 32) {
#pragma unroll
    for (int m = 16; m; m >>= 1) {
      x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
      y += __shfl_xor_sync(0xFFFFFFFFu, y, m);
    }
  } else {
    for (int m = g.tpr >> 1; m; m >>= 1) {
      x += __shfl_xor_sync(0xFFFFFFFFu, x, m);
      y += __shfl_xor_sync(0xFFFFFFFFu, y, m);
    }
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
template <int AL>
__device__ __forceinline__ void load_params(const void* p, int type, float none, int k, int d, int tpr, int lane, float* w) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = none;
  if (!p) return;
  if (AL == 1) {
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
    const auto each = [&](auto* q) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = col<AL>(k, i, tpr, lane);
        if (inside(c, d)) w[i] = to_f(q[c]);
      }
    };
    if (type == ATLAS_F32)
      each(reinterpret_cast<const float*>(p));
    else if (type == ATLAS_BF16)
      each(reinterpret_cast<const __nv_bfloat16*>(p));
    else
      each(reinterpret_cast<const __half*>(p));
  }
}

__device__ __forceinline__ void add8(float* h, const float* v) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) unpair(pair_add(pair(h[i], h[i + 1]), pair(v[i], v[i + 1])), h[i], h[i + 1]);
}

// Eight elements of a row that lies at p (`live` and inside the row), aligned or not; zeros elsewhere.
template <int BYTES, int AL>
struct Raw {
  Raw8<BYTES> v;
  __device__ __forceinline__ void load(const void* p, long at, int k, int d, int tpr, int lane, bool live) {
    v.zero();
    if (BYTES == 0) return;
    if (AL == 1) {
      const int c = col<AL>(k, 0, tpr, lane);
      if (live && c < d) v.load(p, at + c);
    }
  }
  __device__ __forceinline__ void floats(int type, float* f) const { v.floats(type, f); }
};
template <int BYTES>
struct Raw<BYTES, 0> {
  uint32_t v[8];
  __device__ __forceinline__ void load(const void* p, long at, int k, int d, int tpr, int lane, bool live) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col<0>(k, i, tpr, lane);
      v[i] = BYTES && live && c < d ? ld_raw<BYTES>(p, at + c) : 0u;
    }
  }
  __device__ __forceinline__ void floats(int type, float* f) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = BYTES ? raw_float<BYTES>(v[i], type) : 0.f;
  }
};

// Eight outputs of vector k.
template <int AL>
__device__ __forceinline__ void store(void* p, long at, int type, int k, int d, int tpr, int lane, const float* v) {
  if (AL == 1) {
    const int c = col<AL>(k, 0, tpr, lane);
    if (c < d) st8(p, at + c, type, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col<AL>(k, i, tpr, lane);
      if (inside(c, d)) st_elem(p, at + c, type, v[i]);
    }
  }
}

// A row's outputs in a type of 32 or 16 bits.  The type is looked at once: its branch around each element would
// be most of an unaligned row's code.
template <int K, int AL>
__device__ __forceinline__ void store_row(void* p, long at, int type, int d, int tpr, int lane, const float (*h)[8]) {
  if (AL == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) store<AL>(p, at, type, k, d, tpr, lane, h[k]);
    return;
  }
  const auto each = [&](auto* q) {
    typedef std::remove_pointer_t<decltype(q)> T;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const int c = col<AL>(k, i, tpr, lane), c1 = col<AL>(k, i + 1, tpr, lane);
        if (AL == 2 && sizeof(T) == 2 && inside(c, d) && inside(c1, d)) {
          Pack<T, 2> two;
          two.set2(0, h[k][i], h[k][i + 1]);
          st_pack<T, 2>(q + c, two);
        } else {
          if (inside(c, d)) q[c] = from_f<T>(h[k][i]);
          if (inside(c1, d)) q[c1] = from_f<T>(h[k][i + 1]);
        }
      }
  };
  if (type == ATLAS_F32)
    each(reinterpret_cast<float*>(p) + at);
  else if (type == ATLAS_BF16)
    each(reinterpret_cast<__nv_bfloat16*>(p) + at);
  else
    each(reinterpret_cast<__half*>(p) + at);
}
// And in 8 bits.
template <int K, int AL>
__device__ __forceinline__ void store_row8(void* p, long at, int d, int tpr, int lane, const float (*h)[8]) {
#pragma unroll
  for (int k = 0; k < K; ++k) store<AL>(p, at, ATLAS_E4M3, k, d, tpr, lane, h[k]);
}

// A thread's weights and biases: kept in registers, or, of long rows (more than two vectors a thread), read
// again for each row.
template <int K, int AL>
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
  // y of vector k: (h - less) rstd + off, through weight and bias (LESS: otherwise that is none)
  template <bool LESS>
  __device__ __forceinline__ void apply(const Args& a, int k, int tpr, int lane, float less, float rstd, float off, float* h) {
    if constexpr (!kKept) {
      load_params<AL>(a.w, a.wt, 1.f, k, a.d, tpr, lane, w[0]);
      load_params<AL>(a.b, a.wt, 0.f, k, a.d, tpr, lane, b[0]);
    }
    const float *pw = w[kKept ? k : 0], *pb = b[kKept ? k : 0];
    const pair32 less2 = pair(-less, -less), rstd2 = pair(rstd, rstd), off2 = pair(off, off);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const pair32 t = LESS ? pair_add(pair(h[i], h[i + 1]), less2) : pair(h[i], h[i + 1]);
      unpair(pair_fma(pair_fma(t, rstd2, off2), pair(pw[i], pw[i + 1]), pair(pb[i], pb[i + 1])), h[i], h[i + 1]);
    }
  }
};

// Whether sums about c are not enough: its distance to the mean, or squares that leave the 32-bit range (and a row that is not
// finite).
template <bool PRECISE>
__device__ __forceinline__ bool far(float mean, float var) {
  return !(mean * mean <= (PRECISE ? 1.f : 16.f) * var && var < 3e38f);
}
// The mean of eight neighbouring lanes' numbers.
__device__ __forceinline__ float mean8(float v) {
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v * 0.125f;
}
// The mean of those of a row's lanes' first one's eight elements h (of the first vector) that there are, zeros elsewhere.
// base: that lane.  Equal numbers may be off by a rounding here if there are not eight: they take the second round.
template <int AL>
__device__ __forceinline__ float mean_first(const float* h, int d, int tpr, int base) {
  const int n = AL == 1 ? 8 : min(8, (d - 1) / tpr + 1);
  return __shfl_sync(0xFFFFFFFFu, pair_sum(pair_add(pair_add(pair(h[0], h[1]), pair(h[2], h[3])), pair_add(pair(h[4], h[5]), pair(h[6], h[7])))), base) *
         (n == 8 ? 0.125f : 1.f / n);
}
// c, or 0 if an element less c could leave the 32-bit range: differences are finite where the elements are.
__device__ __forceinline__ float within(float c) { return fabsf(c) < 1e30f ? c : 0.f; }
// The second round.  If the first one's mean is a number, so is every element, and the differences from it are summed.  Else
// the elements times 0 are: 0 of a finite row, whose sum alone has left the range and whose squares do all the more, or NaN.
__device__ __forceinline__ bool summed(float mean) { return fabsf(mean) < 3.4e38f; }
// The variance from sums about the mean: infinite where their squares are, and the row then its bias.
__device__ __forceinline__ float var_of(float mean, float squares, float inv_d) {
  return squares < 3e38f ? fmaf(squares, inv_d, -mean * mean) : squares;
}

// A row that is not read again: in the second round a precise one has its elements (HELD, its outputs subtract mu).
struct NoReload {
  __device__ __forceinline__ void operator()(float (*)[8]) const {}
};
// One row from its elements h (zeros past its end) and c, a number near its mean.  red: kRed words, odd: every other row of a
// block; gm: this row's a.ng words for the maxima of groups that are not neighbouring lanes' (every thread of the
// block comes here then); reload: reads h again, of rows that hold t.
template <int K, int AL, bool PRECISE, typename R = NoReload>
__device__ __forceinline__ void forward_row(const Args& a, const RowGroup& g, float* red, int odd, unsigned* gm,
                                            long row, bool live, float c, float (*h)[8], Params<K, AL>& par, const R& reload = R()) {
  constexpr bool AGAIN = !std::is_same_v<R, NoReload>, HELD = PRECISE && !AGAIN;
  const int lane = AL == 2 ? g.first : g.lane;
  const auto in = [&](int k, int i) { return inside(col<AL>(k, AL == 1 ? 0 : i, g.tpr, lane), a.d); };
  // the sums of the elements less v and of their squares, what is past the row's end left out; keep: the differences, to h
  const auto less = [&](float v, float times, bool keep, float& s1, float& s2) {
    const pair32 minus = pair(-v, -v);
    s1 = s2 = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      pair32 p1 = pair(0.f, 0.f), p2 = p1;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float t0, t1;
        unpair(pair_add(pair(h[k][i], h[k][i + 1]), minus), t0, t1);
        if (AL != 1) t0 = in(k, i) ? t0 : 0.f, t1 = in(k, i + 1) ? t1 : 0.f;
        const pair32 t = pair(t0 * times, t1 * times);
        p1 = pair_add(p1, t);
        p2 = pair_fma(t, t, p2);
        if (keep) h[k][i] = t0, h[k][i + 1] = t1;
      }
      const bool some = AL != 1 || in(k, 0);
      s1 += some ? pair_sum(p1) : 0.f;
      s2 += some ? pair_sum(p2) : 0.f;
    }
  };
  if (a.r_out && live) store_row<K, AL>(a.r_out, row * a.sr, a.rt, a.d, g.tpr, lane, h);
  float s1, s2;
  c = within(c);
  less(c, 1.f, !HELD, s1, s2);
  row_sums2(s1, s2, g, red + odd * 32);
  float mean = s1 * a.inv_d, var = fmaf(s2, a.inv_d, -mean * mean);
  const bool again = far<PRECISE>(mean, var);
  if (g.tpr > 32 ? again : __any_sync(0xFFFFFFFFu, again)) {
    const bool sum = summed(mean);
    if (AGAIN) reload(h);
    less(!sum ? 0.f : PRECISE ? c + mean : mean, sum ? 1.f : 0.f, false, s1, s2);
    row_sums2(s1, s2, g, red + 64);
    if (again) {
      s1 *= a.inv_d;
      var = var_of(s1, s2, a.inv_d);
      c += mean;
      mean = PRECISE ? s1 : mean + s1;
      if (!sum || !(var < 3e38f)) {
        c = 0.f, mean = sum ? 0.f : s1, var = __int_as_float(0x7F800000);
      } else if (AGAIN) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) h[k][i] -= c;
      }
    }
    if (g.tpr > 32)
      __syncthreads();  // (the next row may come here too)
    else if (AGAIN)
      __syncwarp();  // (the row's place is filled again when all lanes have read it)
  }
  const float rstd = rsqrtf(fmaxf(var, 0.f) + a.eps), mu = c + mean, off = (HELD ? (mu - c) - mean : -mean) * rstd;
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    par.template apply<HELD>(a, k, g.tpr, lane, mu, rstd, off, h[k]);
    if (!PRECISE || a.ot != ATLAS_E4M3) continue;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (AL == 1 || in(k, i)) m = fmaxf(m, fabsf(h[k][i]));
    if (AL == 1 && !in(k, 0)) m = 0.f;
    if (a.group == 0 || !a.lanes) {
      amax = fmaxf(amax, m);
      continue;
    }
    // the group's lanes are neighbours: group / 8 of them, a power of two
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
      if (8 * o < a.group) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float scale = scale_of(m), inv = inverse(scale);
    const int c = col<AL>(k, 0, g.tpr, lane);
    if (live && c < a.d) {
      if ((c & (a.group - 1)) == 0) a.scale[row * a.ng + (c >> a.gshift)] = scale;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[k][i] *= inv;
      st8(a.y, row * a.sy + c, a.ot, h[k]);
    }
  }
  if (!PRECISE || a.ot != ATLAS_E4M3) {
    if (live) store_row<K, AL>(a.y, row * a.sy, a.ot, a.d, g.tpr, lane, h);
    return;
  }
  if (a.group && a.lanes) return;
  float inv = 0.f;
  if (a.group == 0) {
    const float scale = scale_of(row_max(amax, g, red + 96 + odd * 32));
    inv = inverse(scale);
    if (live && g.lane == 0) a.scale[row] = scale;
  } else {
    // maxima of non-negative floats order like their bits, so integer maxima in shared memory
    // give the same result in any order
    if (g.tpr <= 32) __syncwarp();  // (the row before has read them)
    for (int i = g.lane; i < a.ng; i += g.tpr) gm[i] = 0u;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = col<AL>(k, i, g.tpr, lane);
        if (inside(c, a.d)) atomicMax(&gm[c / a.group], __float_as_uint(fmaxf(0.f, fabsf(h[k][i]))));
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
      const int c = col<AL>(k, i, g.tpr, lane);
      h[k][i] *= a.group == 0 ? inv : inside(c, a.d) ? __uint_as_float(gm[c / a.group]) : 0.f;
    }
  }
  if (live) store_row8<K, AL>(a.y, row * a.sy, a.d, g.tpr, lane, h);
}

template <typename XT>
constexpr int code_of() {
  return std::is_same_v<XT, float> ? ATLAS_F32 : std::is_same_v<XT, __half> ? ATLAS_F16 : ATLAS_BF16;
}
// The residual's type: of 16 bits it is x's where that has 16 bits, but for elements one by one (the launch sees to it).
template <typename XT, int RB, int AL>
__device__ __forceinline__ int r_code(const Args& a) {
  return RB == 4 ? ATLAS_F32 : AL != 0 && sizeof(XT) == 2 ? code_of<XT>() : a.rt;
}

// The two tensors' elements as they lie in memory, to h.
template <typename XT, int RB, int K, int AL>
struct RawRow {
  Raw<sizeof(XT), AL> x[K];
  Raw<RB, AL> r[K];
  __device__ __forceinline__ void load(const Args& a, long row, int tpr, int lane) {
    const bool live = row < a.rows;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k].load(a.x, row * a.sx, k, a.d, tpr, lane, live);
      r[k].load(a.r, row * a.sr, k, a.d, tpr, lane, live);
    }
  }
  __device__ __forceinline__ void floats(const Args& a, float (*h)[8]) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      x[k].floats(code_of<XT>(), h[k]);
      if (RB) {
        float v[8];
        r[k].floats(r_code<XT, RB, AL>(a), v);
        add8(h[k], v);
      }
    }
  }
};


// A row's element i.
template <typename XT, int RB>
__device__ __forceinline__ float element_of(const Args& a, long row, int i) {
  float v = to_f(reinterpret_cast<const XT*>(a.x)[row * a.sx + i]);
  if (RB) v += ld_any(a.r, row * a.sr + i, a.rt);
  return v;
}

// A block a row, straight from memory.
template <typename XT, int RB, int K, int AL>
__global__ void __launch_bounds__(512) forward_rows(Args a) {
  extern __shared__ __align__(16) float sm[];
  const int tpr = blockDim.x;
  const RowGroup g{tpr, (int)threadIdx.x, (int)threadIdx.x};
  const long row = blockIdx.x;
  RawRow<XT, RB, K, AL> raw;
  raw.load(a, row, tpr, g.lane);
  const float first = element_of<XT, RB>(a, row, g.lane & 7);
  Params<K, AL> par;
  par.load(a, tpr, g.lane);
  clear_red(sm, kRed);
  float h[K][8];
  raw.floats(a, h);
  forward_row<K, AL, true>(a, g, sm, 0, reinterpret_cast<unsigned*>(sm + kRed), row, true, mean8(first), h, par);
}

// Rows of up to 256 channels: tpr lanes of a warp each.  Warps walk rows, the next two of their lanes' under way
// while they compute two.
template <typename XT, int RB, int AL, bool PRECISE>
__global__ void __launch_bounds__(128, 5) forward_lanes(Args a, int tpr) {
  extern __shared__ __align__(16) float sm[];
  constexpr int R = 2;
  const RowGroup g{tpr, (int)threadIdx.x % tpr, (int)threadIdx.x};
  const int rpb = blockDim.x / tpr, mine = threadIdx.x / tpr;
  RawRow<XT, RB, 1, AL> raw[R];
  const long step = (long)gridDim.x * rpb;
  long row = (long)blockIdx.x * rpb + mine;
#pragma unroll
  for (int j = 0; j < R; ++j) raw[j].load(a, row + j * step, tpr, g.lane);
  Params<1, AL> par;
  par.load(a, tpr, g.lane);
  for (; row - mine < a.rows; row += R * step) {  // (the same turns for a block's threads)
    float h[R][1][8];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      raw[j].floats(a, h[j]);
      raw[j].load(a, row + (j + R) * step, tpr, g.lane);
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int base = (threadIdx.x & 31) - g.lane;
      const float c = PRECISE ? mean_first<AL>(h[j][0], a.d, tpr, base) : __shfl_sync(0xFFFFFFFFu, h[j][0][0], base);
      forward_row<1, AL, PRECISE>(a, g, sm, 0, reinterpret_cast<unsigned*>(sm) + mine * a.ng, row + j * step, row + j * step < a.rows, c, h[j], par);
    }
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
template <int E, int AL>
__host__ __device__ __forceinline__ int slot_bytes(int d) {
  return AL == 1 || E == 0 ? d * E : (d * E + 30) / 16 * 16;
}

// Distance of a row's first byte from the boundary of 16 in front of it.
__device__ __forceinline__ int ahead(const Rows& t, long row) {
  return (int)(reinterpret_cast<uintptr_t>(t.lo + row * t.stride) & 15);
}

// One row to shared memory; Q pieces of 16 bytes a thread cover an aligned one.  The pieces at the ends of a row that starts
// anywhere hold bytes of its neighbours or of the gaps between rows, which nothing uses; those that reach
// beyond the tensor's ends come element by element.
template <int E, int Q, int AL>
__device__ __forceinline__ void fetch_row(char* s, const Rows& t, long row, long rows, int d, int lane, int threads) {
  if (E == 0 || row >= rows) return;
  if (AL == 1) {
    const char* p = t.lo + row * t.stride + lane * 16;
#pragma unroll
    for (int k = 0; k < Q; ++k)
      if ((k * threads + lane) * 16 < d * E) cp_async<16>(s + (k * threads + lane) * 16, p + k * threads * 16, true);
    return;
  }
  const int shift = ahead(t, row), n = shift + d * E;
  const char* p = t.lo + row * t.stride - shift;
  if (p >= t.lo && p + (n + 15) / 16 * 16 <= t.hi) {
#pragma unroll
    for (int k = 0; k <= Q; ++k) {
      const int i = (k * threads + lane) * 16;
      if (i < n) cp_async<16>(s + i, p + i, true);
    }
    return;
  }
#pragma unroll 1
  for (int i = lane * 16; i < n; i += threads * 16) {
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
template <int E, int AL>
__device__ __forceinline__ void slot_floats(const char* s, int shift, int type, int k, int d, int tpr, int lane, float* f) {
  if (AL == 1) {
    Raw8<E> q;
    q.zero();
    const int c = col<AL>(k, 0, tpr, lane);
    if (c < d) q.load_kept(s, c);
    q.floats(type, f);
    return;
  }
  const auto each = [&](auto code) {  // (the type looked at once, not for each element)
    constexpr int kType = decltype(code)::value;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const int c = col<AL>(k, i, tpr, lane), c1 = col<AL>(k, i + 1, tpr, lane);
      if (AL == 2 && E == 2) {  // (the slot has room for a pair's other element)
        const uint32_t two = c < d ? *reinterpret_cast<const uint32_t*>(s + shift + c * 2) : 0u;
        f[i] = inside(c, d) ? raw_float<E>(two & 0xFFFFu, kType) : 0.f;
        f[i + 1] = inside(c1, d) ? raw_float<E>(two >> 16, kType) : 0.f;
      } else {
        f[i] = inside(c, d) ? raw_float<E>(ld_raw<E>(s + shift, c), kType) : 0.f;
        f[i + 1] = inside(c1, d) ? raw_float<E>(ld_raw<E>(s + shift, c1), kType) : 0.f;
      }
    }
  };
  if (E == 4 || type == ATLAS_BF16)
    each(std::integral_constant<int, ATLAS_BF16>());
  else
    each(std::integral_constant<int, ATLAS_F16>());
}

// About the mean of a row's first eight elements, for sums to be taken about: any number would do, so 16-bit elements
// are added in their type.  Every thread reads them: what is handed on between lanes waits behind all copies and reads of
// the others (backward 16384 x 2560 with a 32-bit stream: 120 us with three exchanges, so 111).  Of rows that begin anywhere
// eight lanes read one each all the same: eight reads of a thread cost more (20000 x 1371 fp32 + residual: 113 us and 82).
template <int E, int AL>
__device__ __forceinline__ float near_mean(const char* s, int type, int d) {
  if (E == 4) {
    float f[8];
    if (AL == 1) {
      ld_vec<8>(reinterpret_cast<const float*>(s), f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = reinterpret_cast<const float*>(s)[min(i, d - 1)];
    }
    pair32 v = pair(f[0], f[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) v = pair_add(v, pair(f[i], f[i + 1]));
    return pair_sum(v) * 0.125f;
  }
  if (AL != 1 && d <= 8) return raw_float<E>(ld_raw<E>(s, 0), type);
  uint32_t w[4];
  if (AL == 1) {
    *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(s);
  } else {
    // (a row that begins between two words: from its second element on)
    const uint32_t* p = reinterpret_cast<const uint32_t*>((reinterpret_cast<uintptr_t>(s) + 2) & ~(uintptr_t)3);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p[i];
  }
  if (type == ATLAS_BF16) {
    const auto h = [&](int i) { return *reinterpret_cast<const __nv_bfloat162*>(&w[i]); };
    const __nv_bfloat162 v = __hadd2(__hadd2(h(0), h(1)), __hadd2(h(2), h(3)));
    return (__low2float(v) + __high2float(v)) * 0.125f;
  }
  // an eighth of each, whose sum stays in the range
  const auto h = [&](int i) { return *reinterpret_cast<const __half2*>(&w[i]); };
  const __half2 part = __float2half2_rn(0.125f);
  const __half2 v = __hfma2(h(0), part, __hfma2(h(1), part, __hfma2(h(2), part, __hmul2(h(3), part))));
  return __low2float(v) + __high2float(v);
}

// Many rows of a block each (long ones, unaligned: more than there are SMs): a block walks rows and copies the next kStages - 1 to shared memory while it computes
// one.  The barrier in a row's sums also hands over the next row, whose copies have been waited for before it, and this
// row's place; a block of one warp (rows of 257 to 512 channels) has no barrier there, and takes one of its own.
// Registers: 80 (32768 x 2048 bf16 + residual to e4m3, at the step that chose it: 92 us; 64: 108, 72: 100, 88: 94), 72 of
// aligned rows of two 32-bit tensors, whose stages leave room for four blocks of an SM anyway (20000 x 2048: 109 us, 80: 122; x 4096:
// 213 and 228).
template <typename XT, int RB, int K, int AL, bool PRECISE>
__global__ void __maxnreg__(K > 2 ? 128 : AL == 1 && RB == 4 && sizeof(XT) == 4 ? 72 : 80) forward_ring(Args a) {
  extern __shared__ __align__(16) float sm[];  // [kRed], [stage]: x, r, then the groups' maxima
  constexpr int XB = sizeof(XT);
  clear_red(sm, kRed);
  RowGroup g{(int)blockDim.x, (int)threadIdx.x, (int)threadIdx.x};
  // (the grid is even, so a block's rows begin alike)
  if (AL == 2) g.first = 2 * g.lane - (int)((reinterpret_cast<uintptr_t>(a.x) / 2 + blockIdx.x * a.sx) & 1);
  const int lane = AL == 2 ? g.first : g.lane;
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
  par.load(a, g.tpr, lane);
  long row = blockIdx.x;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(row + (long)i * gridDim.x, i);
  cp_wait<kStages - 2>();
  __syncthreads();
  int stage = 0;
  for (int odd = 0; row < a.rows; row += gridDim.x, odd ^= 1) {
    fetch(row + (long)(kStages - 1) * gridDim.x, stage == 0 ? kStages - 1 : stage - 1);
    const char* s = ring + stage * bytes;
    const int ax = AL == 1 ? 0 : ahead(tx, row), ar = AL == 1 || RB == 0 ? 0 : ahead(tr, row);
    float c;
    if (PRECISE && AL == 1) {
      c = near_mean<XB, AL>(s, code_of<XT>(), a.d);
      if constexpr (RB > 0) c += near_mean<RB, AL>(s + xs, a.rt, a.d);
    } else {
      const int at = PRECISE ? g.lane & 7 : 0;
      c = to_f(reinterpret_cast<const XT*>(s + ax)[at]);
      if constexpr (RB > 0) c += raw_float<RB>(ld_raw<RB>(s + xs + ar, at), a.rt);
      if (PRECISE) c = mean8(c);
    }
    const auto load = [&](float (*h)[8]) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        slot_floats<XB, AL>(s, ax, code_of<XT>(), k, a.d, g.tpr, lane, h[k]);
        if constexpr (RB > 0) {
          float v[8];
          slot_floats<RB, AL>(s + xs, ar, r_code<XT, RB, AL>(a), k, a.d, g.tpr, lane, v);
          add8(h[k], v);
        }
      }
    };
    float h[K][8];
    load(h);
    cp_wait<kStages - 2>();  // the next row's
    if (g.tpr <= 32) __syncwarp();
    // (rows that begin anywhere stay held: read again 109 us for 82, 20000 x 1371 fp32 + residual)
    if constexpr (PRECISE && AL == 1)
      forward_row<K, AL, true>(a, g, sm, odd, gm, row, true, c, h, par, load);
    else
      forward_row<K, AL, PRECISE>(a, g, sm, odd, gm, row, true, c, h, par);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  cp_wait<0>();
}

// ------------------------------------------------------------------ launches

// Rows of up to 256 channels by the lanes that their vectors fill; longer ones by a block of at most 512 threads, of
// one vector each while that is enough (`two`: two: what a row costs a thread besides its elements is then
// shared by sixteen).
inline RowPlan forward_plan(int d, bool two) {
  RowPlan p = rows_plan(d, 1);
  const int nv = (d + 7) / 8;
  if (p.tpr <= 32) {
    for (p.tpr = 1; p.tpr < nv;) p.tpr *= 2;
  } else if (two && p.k == 1) {
    p = RowPlan{(nv + 63) / 64 * 32, 2, (nv + 63) / 64 * 32};
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

// Blocks of a kernel that an SM holds by its registers, as many as run at once: rows are dealt to them in equal shares, and
// a second wave of blocks for the rest would take as long as the first.
template <auto F>
int by_registers(int threads) {
  static const int regs = [] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, F) == cudaSuccess && at.numRegs > 0 ? (at.numRegs + 7) / 8 * 8 : 128;
  }();
  const int n = 65536 / (regs * threads), most = 2048 / threads;
  return n < 1 ? 1 : n < most ? n : most;
}

template <typename XT, int RB, int K, int AL, bool PRECISE>
int run_ring(const Args& a, int threads, size_t smem, cudaStream_t st) {
  auto* f = forward_ring<XT, RB, K, AL, PRECISE>;
  if (const int rc = shared(f, smem)) return rc;
  const long most = (long)kSMs * resident(smem, by_registers<forward_ring<XT, RB, K, AL, PRECISE>>(threads));  // (even)
  f<<<(unsigned)(a.rows < most ? a.rows & ~1L : most), threads, smem, st>>>(a);
  return status();
}

template <typename XT, int RB, int K, int AL>
int run_rows(const Args& a, int threads, cudaStream_t st) {
  if (a.rows > 0x7FFFFFFFL) return ATLAS_ERR_UNSUPPORTED;
  const size_t smem = (kRed + (a.lanes ? 0 : (size_t)a.ng)) * 4;
  auto* f = forward_rows<XT, RB, K, AL>;
  if (const int rc = shared(f, smem)) return rc;
  f<<<(unsigned)a.rows, threads, smem, st>>>(a);
  return status();
}

// Whether the 16-bit tensors' rows all begin on the same side of four bytes, row by row, and the plan's threads reach
// one column further.
struct Begins {
  const void* p;
  long stride;
  int type;
};
inline bool pairs(const Args& a, std::initializer_list<Begins> tensors, const RowPlan& p) {
  int base = -1, step = 0;
  for (const Begins& t : tensors) {
    if (!t.p || (t.type != ATLAS_BF16 && t.type != ATLAS_F16)) continue;
    const int b = (int)(reinterpret_cast<uintptr_t>(t.p) / 2 & 1), s = (int)(t.stride & 1);
    if (base >= 0 && (b != base || s != step)) return false;
    base = b, step = s;
  }
  return base >= 0 && p.tpr * 8 * p.k > a.d;
}

// The precise kernels of a type, which are compiled by themselves.
template <typename XT>
int precise(const Args& a, cudaStream_t st);

template <typename XT, int RB, int AL, bool PRECISE>
int forward(const Args& args, cudaStream_t st) {
  Args a = args;
  // a group of an 8-bit output in neighbouring lanes of one warp: a power of two from 8 to 256
  a.lanes = a.ot != ATLAS_E4M3 || a.group == 0 || (AL == 1 && a.group >= 8 && a.group <= 256 && (a.group & (a.group - 1)) == 0);
  const bool many = a.rows > kSMs * 8;
  const RowPlan p = forward_plan(a.d, many);
  // (rows straight from memory and those of more than 8192 channels: the precise way, whatever the output)
  if constexpr (!PRECISE)
    if (a.d > 256 && !(p.k == 2 && many)) return precise<XT>(args, st);
  if (a.d <= 256) {
    const int rpb = p.block / p.tpr;
    const size_t smem = a.lanes ? 0 : (size_t)rpb * a.ng * 4;
    auto* f = forward_lanes<XT, RB, AL, PRECISE>;
    if (const int rc = shared(f, smem)) return rc;
    const long need = (a.rows + rpb - 1) / rpb, most = 5L * kSMs;
    f<<<(unsigned)(need < most ? need : most), p.block, smem, st>>>(a, p.tpr);
    return status();
  }
  const size_t ring = kRed * 4 + (size_t)kStages * (slot_bytes<sizeof(XT), AL>(a.d) + slot_bytes<RB, AL>(a.d)) + (a.lanes ? 0 : (size_t)a.ng * 4);
  // (rows of more than 8192 channels: only of those that start anywhere; 2000 x 9001 bf16: 125 us straight from memory, 58
  // so, x 32767: 558 and 168; aligned 2000 x 9000: 27 and, when it was chosen, 34, x 32768: 88 and 95)
  if ((p.k == 2 ? many : AL != 1 && p.k > 2 && a.rows > kSMs) && ring <= 200 * 1024) {
    const auto run = [&](auto k) -> int {
      constexpr int K = decltype(k)::value;
      if constexpr (AL == 0 && sizeof(XT) == 2)
        if ((RB != 2 || a.rt == a.dt) && pairs(a, {{a.x, a.sx, a.dt}, {a.r, a.sr, a.rt}, {a.r_out, a.sr, a.rt}, {a.y, a.sy, a.ot}}, p)) return run_ring<XT, RB, K, 2, PRECISE>(a, p.block, ring, st);
      return run_ring<XT, RB, K, AL, PRECISE>(a, p.block, ring, st);
    };
    if constexpr (PRECISE && AL != 1) {
      if (p.k == 4) return run(std::integral_constant<int, 4>());
      if (p.k == 8) return run(std::integral_constant<int, 8>());
    }
    return run(std::integral_constant<int, 2>());
  }
  if constexpr (PRECISE) {
    if (p.k == 1) return run_rows<XT, RB, 1, AL>(a, p.block, st);
    if (p.k == 2) return run_rows<XT, RB, 2, AL>(a, p.block, st);
    if (p.k == 4) return run_rows<XT, RB, 4, AL>(a, p.block, st);
    return run_rows<XT, RB, 8, AL>(a, p.block, st);
  } else {
    return precise<XT>(args, st);
  }
}
template <typename XT, bool PRECISE>
int forward(const Args& a, cudaStream_t st) {
  const int rb = !a.r ? 0 : a.rt == ATLAS_F32 ? 4 : 2;
  const bool mixed = rb == 2 && sizeof(XT) == 2 && a.rt != a.dt;  // bf16 and fp16: element by element
  if (a.wide && !mixed)
    return rb == 0 ? forward<XT, 0, 1, PRECISE>(a, st) : rb == 2 ? forward<XT, 2, 1, PRECISE>(a, st) : forward<XT, 4, 1, PRECISE>(a, st);
  return rb == 0 ? forward<XT, 0, 0, PRECISE>(a, st) : rb == 2 ? forward<XT, 2, 0, PRECISE>(a, st) : forward<XT, 4, 0, PRECISE>(a, st);
}

}  // namespace layernorm
}  // namespace atlas
