// ops_common.cuh -- helpers of the layer operators (norm, conv, scan): elements of
// a type known at run or compile time, the tiling of (packed) sequences, and
// reductions over groups of lanes.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "atlas_ops.h"
#include "common.cuh"
#include "ops.h"

namespace atlas {

// ------------------------------------------------------------------ elements

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// V consecutive elements as one aligned block of registers.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T e[V];
  __device__ __forceinline__ float get(int i) const { return to_f(e[i]); }
  __device__ __forceinline__ void set(int i, float v) { e[i] = from_f<T>(v); }
  // elements i, i + 1 (i even) at once: one conversion instruction for both where there is one
  __device__ __forceinline__ void get2(int i, float& lo, float& hi) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(e)[i / 2];
      if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        lo = f.x;
        hi = f.y;
      }
    } else {
      lo = to_f(e[i]);
      hi = to_f(e[i + 1]);
    }
  }
  __device__ __forceinline__ void set2(int i, float lo, float hi) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
      reinterpret_cast<uint32_t*>(e)[i / 2] = *reinterpret_cast<const uint32_t*>(&w);
    } else if constexpr (std::is_same_v<T, __half>) {
      const __half2 w = __floats2half2_rn(lo, hi);
      reinterpret_cast<uint32_t*>(e)[i / 2] = *reinterpret_cast<const uint32_t*>(&w);
    } else {
      set(i, lo);
      set(i + 1, hi);
    }
  }
  __device__ __forceinline__ void unpack(float* v) const {
    if constexpr (V == 1) {
      v[0] = get(0);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) get2(i, v[i], v[i + 1]);
    }
  }
  __device__ __forceinline__ void pack(const float* v) {
    if constexpr (V == 1) {
      set(0, v[0]);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) set2(i, v[i], v[i + 1]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f<T>(0.f);
  }
};

// V elements from p; aligned to V elements when V > 1.  Inputs that are read once go
// past L1.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> ld_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void st_pack(T* p, const Pack<T, V>& v) {
  *reinterpret_cast<Pack<T, V>*>(p) = v;
}

// V neighbouring 32-bit numbers, aligned to V (at most four at a time).
template <int V>
__device__ __forceinline__ void ld_vec(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < V; i += (V < 4 ? V : 4)) {
    const auto q = ld_pack<float, (V < 4 ? V : 4)>(p + i);
#pragma unroll
    for (int j = 0; j < (V < 4 ? V : 4); ++j) v[i + j] = q.e[j];
  }
}
template <int V>
__device__ __forceinline__ void st_vec(float* p, const float* v) {
#pragma unroll
  for (int i = 0; i < V; i += (V < 4 ? V : 4)) {
    Pack<float, (V < 4 ? V : 4)> q;
#pragma unroll
    for (int j = 0; j < (V < 4 ? V : 4); ++j) q.e[j] = v[i + j];
    st_pack<float, (V < 4 ? V : 4)>(p + i, q);
  }
}

// Element of a type known at run time (parameters, read once per block).
__device__ __forceinline__ float ld_any(const void* p, long i, int dtype) {
  if (dtype == ATLAS_BF16) return to_f(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == ATLAS_F16) return to_f(reinterpret_cast<const __half*>(p)[i]);
  return reinterpret_cast<const float*>(p)[i];
}

// Asynchronous copy of BYTES (4, 8 or 16) to shared memory, zeros when !some; done for this
// thread when cp_wait leaves at most `n` later groups open.
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src, bool some) {
  const unsigned d = static_cast<unsigned>(__cvta_generic_to_shared(dst));
  const int n = some ? BYTES : 0;
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(d), "l"(src), "n"(BYTES), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------ functions

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
#define ATLAS_LOG2E 1.4426950408889634f
// 1 / (1 + exp(-x)); for x < -88 the exponential is infinite and the result 0.
__device__ __forceinline__ float sigmoidf(float x) { return rcp(1.f + ex2(-ATLAS_LOG2E * x)); }
// x / (1 + exp(-x)); NaN at -infinity, as the formula gives.
__device__ __forceinline__ float siluf(float x) { return x * sigmoidf(x); }
// d/dx (x sigmoid(x)) given s = sigmoid(x).
__device__ __forceinline__ float silu_slope(float x, float s) { return s * (1.f + x * (1.f - s)); }

// Two 32-bit numbers as one 64-bit register: an instruction on a pair takes the arithmetic
// pipe as long as two single ones, but one issue slot.
typedef unsigned long long pair32;
__device__ __forceinline__ pair32 pair(float lo, float hi) {
  pair32 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(pair32 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ pair32 pair_mul(pair32 a, pair32 b) {
  pair32 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair32 pair_add(pair32 a, pair32 b) {
  pair32 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ pair32 pair_fma(pair32 a, pair32 b, pair32 c) {
  pair32 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ pair32 pair_ex2(pair32 a) {
  float x, y;
  unpair(a, x, y);
  return pair(ex2(x), ex2(y));
}
__device__ __forceinline__ float pair_sum(pair32 a) {
  float x, y;
  unpair(a, x, y);
  return x + y;
}

// log(1 + exp(x)) = max(x, 0) + log(1 + e), e = exp(-|x|) in [0, 1].  log(1 + e) = e P(e):
// P fitted to log(1 + e) / e on [0, 1] by reweighted least squares at Chebyshev nodes
// (relative error 5e-9; 1.5e-7 with the roundings of its evaluation).
__device__ __forceinline__ float softplusf(float x) {
  constexpr float k[10] = {1.f, -0.49999902f, 0.33329964f, -0.24954133f, 0.19675931f,
                           -0.1530557f, 0.10603617f, -0.05695916f, 0.019851262f, -0.0032439807f};
  const float e = ex2(-ATLAS_LOG2E * fabsf(x));
  float p = k[9];
#pragma unroll
  for (int i = 8; i >= 0; --i) p = fmaf(p, e, k[i]);
  return fmaf(p, e, fmaxf(x, 0.f));
}
// ------------------------------------------------------------------ sequences

// Tiles of TT tokens.  With seq_start, tile numbers are handed out so that a tile
// belongs to one sequence without a prefix sum over lengths: sequence b has the numbers
// start[b] / TT + b .. start[b + 1] / TT + b, at least as many as its ceil(len / TT)
// tiles and at least one; L / TT + B numbers in all.
struct SeqTile {
  int b;      // sequence
  int t0;     // the tile's first token in the sequence
  int len;    // the sequence's tokens
  int first;  // row of the sequence's first token (packed), 0 otherwise
  int slot;   // its state
  bool carry; // whether it starts from its state
};

// (lengths may be next to 2^31: sums with a tile's do not fit)
inline __host__ __device__ int seq_tiles_of(int L, int TT) { return L > TT ? (L - 1) / TT + 1 : 1; }
__device__ __forceinline__ int seq_tile_end(const SeqTile& t, int TT) { return (int)min((unsigned)t.t0 + TT, (unsigned)t.len); }

// Number of tile numbers for a description.
inline __host__ __device__ long seq_tiles(const SeqArgs& a, int TT) {
  if (a.B == 0) return 0;
  return a.start ? (long)a.L / TT + a.B : (long)a.B * seq_tiles_of(a.L, TT);
}

// How many sequences lie in front of the first fall of seq_start: the search below needs starts that
// rise, and behind a fall rows would belong to two sequences.  Called by all threads of a block, once.  (It has
// no shared memory of its own: with a word of it the scan's pass of kept states took 126 us, without 119.)
__device__ __forceinline__ int seq_rising(const SeqArgs& a) {
  if (!a.start) return a.B;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, n = blockDim.x * blockDim.y;
  bool falls = false;
#pragma unroll 4
  for (int b = tid; b < a.B; b += n) falls |= a.start[b + 1] < a.start[b];
  if (!__syncthreads_or(falls)) return a.B;
  int first = 0;
  while (first < a.B && a.start[first + 1] >= a.start[first]) ++first;
  return first;
}

// The last sequence whose first tile number is not above i, of the first `rising` (0: the first sequence
// falls, and the search ends there).  32 candidates at a time, by a whole warp.  Sequence b's first number is clamp(start[b]) / TT + b * each.
__device__ __forceinline__ int seq_search(const SeqArgs& a, int rising, long i, int TT, int each) {
  int lo = 0, n = a.B;  // (not `rising`, whose load may be under way)
  const int lane = threadIdx.x & 31;
  while (n > 1) {
    const int step = (n + 31) / 32, j = lane * step;
    bool le = false;
    if (j < n) {
      const int s = min(max(a.start[lo + j], 0), a.L);
      le = j == 0 || (lo + j < rising && (long)s / TT + (long)(lo + j) * each <= i);
    }
    const unsigned m = __ballot_sync(0xFFFFFFFFu, le);
    const int last = 31 - __clz((int)m);  // of the candidates not above i (the first always counts)
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// The state of sequence t.b; false when it has none of its own and is left out.  By a whole warp.
__device__ __forceinline__ bool seq_state(const SeqArgs& a, SeqTile& t) {
  t.slot = t.b;
  if (a.slot) {
    t.slot = a.slot[t.b];
    const int lane = threadIdx.x & 31;  // (of the warp's lanes, each looks at some)
    bool bad = t.slot < 0 || t.slot >= a.n_slots;
    for (int j = lane; j < t.b; j += 32) bad |= a.slot[j] == t.slot;
    if (__any_sync(0xFFFFFFFFu, bad)) {
      if (a.status && t.slot >= 0 && t.t0 == 0 && lane == 0) *a.status = ATLAS_ERR_INVALID;
      return false;
    }
  }
  t.carry = a.carry ? a.carry[t.b] != 0 : true;
  return true;
}

// Which tile number `i` is; false when it is none (or its sequence is left out).  Called by whole
// warps with the same i.
__device__ __forceinline__ bool seq_tile(const SeqArgs& a, int rising, long i, int TT, SeqTile& t) {
  if (a.start) {
    const int lo = seq_search(a, rising, i, TT, 1);
    const int s = a.start[lo], e = a.start[lo + 1];
    if (s < 0 || e < s || e > a.L) return false;  // reported by seq_check
    t.b = lo;
    t.first = s;
    t.len = e - s;
    const long k = i - ((long)s / TT + lo);
    if (k < 0 || (k > 0 && k * TT >= t.len)) return false;
    t.t0 = (int)k * TT;
  } else {
    const int n = seq_tiles_of(a.L, TT);
    t.b = (int)(i / n);
    t.t0 = (int)(i % n) * TT;
    t.first = 0;
    t.len = a.L;
  }
  return seq_state(a, t);
}

// Rows dealt to workers in equal shares, whatever the sequences' lengths.  Sequence b has the units from
// clamp(start[b]) + b kStart on: kStart for its start (what a worker needs to begin with a sequence takes
// about as long as that many rows) and one a row; worker w takes the units w * share .., and walks
// what they hold of one sequence after the other.  A cut among a sequence's first kLead rows moves to the
// nearer end of them, so a piece that begins later has no state in its reach (moved to the start, and
// from 16 rows, they made some workers half as long again).
constexpr int kStart = 16, kLead = 8;
static_assert(ATLAS_CONV_MAX_W - 1 <= kLead, "a state reaches kLead rows");
inline long seq_units(const SeqArgs& a) {
  return a.B == 0 ? 0 : (a.start ? (long)a.L : (long)a.B * a.L) + (long)a.B * kStart;
}
// Units a worker for at most n workers, 16 at least; short sequences (single tokens) have a worker each
// for up to `rounds` times n of them.
inline long seq_share(const SeqArgs& a, long n, int rounds) {
  if (a.B < 1) return 1;
  const long u = seq_units(a), B = a.B, one = (u + B - 1) / B;
  if (one <= kStart + 16 && B <= rounds * n) return one;
  const long even = (u + n - 1) / n;
  return even > 16 ? even : 16;
}

struct SeqWalk {
  int b, end;  // the next sequence to look at, the number of sequences
};

// A worker's walk; rising as above.  Called by whole warps.
__device__ __forceinline__ SeqWalk seq_walk(const SeqArgs& a, int rising, long worker, long share) {
  const long u0 = worker * share;
  if (a.start) return SeqWalk{seq_search(a, rising, u0, 1, kStart), rising};
  const unsigned each = (unsigned)a.L + kStart;
  return SeqWalk{(int)min(u0 >> 32 ? u0 / each : (long)((unsigned)u0 / each), (long)a.B), a.B};
}

// The next piece: tokens t.t0 .. t1 of a sequence (none of an empty one), its start and state with it when
// t0 is 0.  False behind the last.
__device__ __forceinline__ bool seq_piece(const SeqArgs& a, SeqWalk& w, long worker, long share, SeqTile& t,
                                          int& t1) {
  const long u0 = worker * share, u1 = u0 + share;
  while (w.b < w.end) {
    t.b = w.b++;
    long unit;
    bool ok = true;
    if (a.start) {
      const int s = a.start[t.b], e = a.start[t.b + 1];
      unit = (long)min(max(s, 0), a.L) + (long)t.b * kStart;
      t.first = s;
      t.len = e - s;
      ok = s >= 0 && e <= a.L;  // else reported by seq_check
    } else {
      unit = t.b * ((long)a.L + kStart);
      t.first = 0;
      t.len = a.L;
    }
    if (unit >= u1) break;
    if (!ok) continue;
    const auto cut = [&](long v) {  // the token in front of which unit v cuts; behind the last: len + 1
      const long r = v - kStart;
      return r >= t.len ? t.len + 1L : r >= kLead ? r : r >= kLead / 2 ? (long)kLead : 0L;
    };
    const long from = cut(u0 - unit), to = cut(u1 - unit);
    if (from >= to) continue;
    t.t0 = (int)from;
    t1 = (int)min(to, (long)t.len);
    if (unit + kStart + t.len >= u1) w.b = w.end;  // the worker's last
    if (seq_state(a, t)) return true;
  }
  w.b = w.end;
  return false;
}

// Report a bad seq_start: called by the threads of one block of the grid.
__device__ __forceinline__ void seq_check(const SeqArgs& a, int tid, int nthr) {
  if (!a.start || !a.status) return;
  for (int b = tid; b < a.B; b += nthr) {
    const int s = a.start[b], e = a.start[b + 1];
    if (s < 0 || e < s || e > a.L) *a.status = ATLAS_ERR_INVALID;
  }
}

// Offset of token t of the tile's sequence.
__device__ __forceinline__ long seq_at(const SeqArgs& a, const SeqTile& t, int tok, long sb, long st) {
  return a.start ? (long)(t.first + tok) * st : (long)t.b * sb + (long)tok * st;
}

// ------------------------------------------------------------------ reductions

// Sums NV values over LANES lanes (lane bits STRIDE .. STRIDE * LANES / 2) by halving: each
// step sends half of the values and keeps the sums of the other half.  With NV >= LANES
// the lane numbered j among the LANES is left with v[0 .. NV / LANES) = the sums of values
// j * NV / LANES ..; with NV < LANES, value j * NV / LANES is left in LANES / NV lanes.
template <int NV, int LANES, int STRIDE>
__device__ __forceinline__ void lane_sums(float* v, int lane) {
  if constexpr (LANES > 1) {
    constexpr int M = LANES / 2 * STRIDE;
    if constexpr (NV > 1) {
      constexpr int H = NV / 2;
      const bool up = lane & M;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float send = up ? v[i] : v[i + H];
        const float keep = up ? v[i + H] : v[i];
        v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, M);
      }
      lane_sums<H, LANES / 2, STRIDE>(v, lane);
    } else {
      v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], M);
      lane_sums<1, LANES / 2, STRIDE>(v, lane);
    }
  }
}

}  // namespace atlas
