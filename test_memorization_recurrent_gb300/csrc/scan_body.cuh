// scan_body.cuh -- selective state space scan, for one element type (instantiated by
// scan_f32.cu, scan_bf16.cu, scan_f16.cu).
//
//   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = (C_t h_t + D x_t) SiLU(z_t)
//
// A channel's N states are split over LN lanes with four states a lane, the channel's y is
// their sum: batches of four tokens are added by halving (three shuffles for four tokens).
// x, dt, B, C of a tile of tokens lie in shared memory, where softplus has been taken once
// per token and channel.
//
// When sequences times channels do not fill the machine, the tokens are split into
// segments: a first pass finds each segment's end state from a zero start (with the sum of
// its dt: the decay over a segment is exp(A sum dt)), a second one joins them into start
// states, the third computes the outputs.
#pragma once
#include "ops_common.cuh"

namespace atlas {
namespace scan {

constexpr int kThreads = 128;
constexpr int kTile = 32;  // tokens in shared memory

template <int LN>
struct Shape {
  static constexpr int kNP = 4 * LN;               // padded states
  static constexpr int kCW = 32 / LN;              // channels of a warp
  static constexpr int kCB = kCW * kThreads / 32;  // channels of a block
};

// The block's channels: blocks do not cross groups.
struct Channels {
  int c0, n, g;  // first, count, group
};
template <int LN>
__device__ __forceinline__ Channels channels_of(const ScanArgs& a, int by) {
  const int per = a.D / a.G, bpg = (per + Shape<LN>::kCB - 1) / Shape<LN>::kCB;
  Channels k;
  k.g = by / bpg;
  const int at = (by % bpg) * Shape<LN>::kCB;
  k.c0 = k.g * per + at;
  k.n = min(Shape<LN>::kCB, per - at);
  return k;
}
template <int LN>
inline int channel_blocks(const ScanArgs& a) {
  const int per = a.D / a.G;
  return a.G * ((per + Shape<LN>::kCB - 1) / Shape<LN>::kCB);
}

// dt of a token and channel from its raw value.
__device__ __forceinline__ float step_of(const ScanArgs& a, float raw, int c) {
  const float r = a.bias ? raw + a.bias[c] : raw;
  return a.softplus ? softplusf(r) : r;
}

// Tokens t0 .. t0 + TT of dt (through softplus) and x into sd, those past `end` as zeros.
template <typename T, int V, int LN, int TT>
__device__ __forceinline__ void load_dx(const ScanArgs& a, const SeqTile& t, const Channels& k,
                                        int t0, int end, float2 (*sd)[Shape<LN>::kCB]) {
  constexpr int CV = Shape<LN>::kCB / V;
  for (int i = threadIdx.x; i < TT * CV; i += kThreads) {
    const int u = i / CV, cl = (i % CV) * V;
    if (t0 + u < end && cl < k.n) {
      const auto x = ld_pack<T, V>(reinterpret_cast<const T*>(a.x) + seq_at(a.s, t, t0 + u, a.xb, a.xt) + k.c0 + cl);
      const auto d = ld_pack<T, V>(reinterpret_cast<const T*>(a.dt) + seq_at(a.s, t, t0 + u, a.tb, a.tt) + k.c0 + cl);
#pragma unroll
      for (int j = 0; j < V; ++j) sd[u][cl + j] = make_float2(step_of(a, d.get(j), k.c0 + cl + j), x.get(j));
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) sd[u][cl + j] = make_float2(0.f, 0.f);
    }
  }
}

template <typename T, int LN, int TT>
__device__ __forceinline__ void load_states(const ScanArgs& a, const SeqTile& t, const Channels& k,
                                            int t0, int end, const void* p, long sb, long st,
                                            float (*s)[Shape<LN>::kNP]) {
  constexpr int NP = Shape<LN>::kNP;
  for (int i = threadIdx.x; i < TT * NP; i += kThreads) {
    const int u = i / NP, n = i % NP;
    s[u][n] = t0 + u < end && n < a.N
                  ? to_f(reinterpret_cast<const T*>(p)[seq_at(a.s, t, t0 + u, sb, st) + (long)k.g * a.N + n])
                  : 0.f;
  }
}

// This lane's four states at p (one channel's N states), 0 past N.
__device__ __forceinline__ void ld_states4(const float* p, int n0, int N, float* h) {
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = n0 + i < N ? p[n0 + i] : 0.f;
}
__device__ __forceinline__ void st_states4(float* p, int n0, int N, const float* h) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < N) p[n0 + i] = h[i];
}

// ENDS: only the end state of each segment but a sequence's last, from a zero start, into
// seg_h, and the sum of dt into seg_dt.  Otherwise the outputs, from seg_h (or, with one
// segment a sequence, from the sequence's state) on.
template <typename T, int V, int LN, bool ENDS>
__global__ void __launch_bounds__(kThreads)
    segment_kernel(ScanArgs a, int S, float* seg_h, float* seg_dt) {
  using P = Shape<LN>;
  __shared__ float2 sd[kTile][P::kCB];
  __shared__ __align__(16) float sB[kTile][P::kNP];
  __shared__ __align__(16) float sC[ENDS ? 1 : kTile][P::kNP];
  __shared__ float sy[ENDS ? 1 : kTile][P::kCB];
  if (blockIdx.x == 0 && blockIdx.y == 0) seq_check(a.s, threadIdx.x, kThreads);
  const long seg = blockIdx.x;
  SeqTile t;
  if (!seq_tile(a.s, seg, S, t)) return;
  const int end = min(t.t0 + S, t.len);
  if (ENDS && end == t.len) return;
  const Channels k = channels_of<LN>(a, blockIdx.y);
  const int lane = threadIdx.x & 31, nl = lane % LN, n0 = nl * 4;
  const int cl = (threadIdx.x >> 5) * P::kCW + lane / LN, c = k.c0 + cl;
  const bool live = cl < k.n;
  float A2[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  if (live) {
    ld_states4(a.A + (long)c * a.N, n0, a.N, A2);
    if (!ENDS) {
      if (seg_h)
        ld_states4(seg_h + (seg * a.D + c) * a.N, n0, a.N, h);
      else if (a.h_in && t.carry)
        ld_states4(a.h_in + ((long)t.slot * a.D + c) * a.N, n0, a.N, h);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] *= ATLAS_LOG2E;
  for (int t0 = t.t0; t0 < end; t0 += kTile) {
    __syncthreads();
    load_dx<T, V, LN, kTile>(a, t, k, t0, end, sd);
    load_states<T, LN, kTile>(a, t, k, t0, end, a.Bm, a.bb, a.bt, sB);
    if (!ENDS) load_states<T, LN, kTile>(a, t, k, t0, end, a.Cm, a.cb, a.ct, sC);
    __syncthreads();
    const int nt = min(kTile, end - t0);
    for (int u0 = 0; u0 < nt; u0 += 4) {
      float yp[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 d = sd[u0 + u][cl];
        const float4 b = *reinterpret_cast<const float4*>(&sB[u0 + u][n0]);
        const float g = d.x * d.y;
        h[0] = ex2(d.x * A2[0]) * h[0] + g * b.x;
        h[1] = ex2(d.x * A2[1]) * h[1] + g * b.y;
        h[2] = ex2(d.x * A2[2]) * h[2] + g * b.z;
        h[3] = ex2(d.x * A2[3]) * h[3] + g * b.w;
        if (ENDS) {
          sum += d.x;
        } else {
          const float4 q = *reinterpret_cast<const float4*>(&sC[u0 + u][n0]);
          yp[u] = h[0] * q.x + h[1] * q.y + h[2] * q.z + h[3] * q.w;
        }
      }
      if (!ENDS) {
        lane_sums<4, LN, 1>(yp, lane);
        if (LN <= 4) {
          constexpr int NV = LN <= 4 ? 4 / LN : 1;
#pragma unroll
          for (int i = 0; i < NV; ++i) sy[u0 + nl * NV + i][cl] = yp[i];
        } else if (nl % (LN > 4 ? LN / 4 : 1) == 0) {
          sy[u0 + nl / (LN > 4 ? LN / 4 : 1)][cl] = yp[0];
        }
      }
    }
    if (!ENDS) {
      __syncthreads();
      constexpr int CV = P::kCB / V;
      for (int i = threadIdx.x; i < nt * CV; i += kThreads) {
        const int u = i / CV, q = (i % CV) * V;
        if (q >= k.n) continue;
        Pack<T, V> z, o;
        if (a.z) z = ld_pack<T, V>(reinterpret_cast<const T*>(a.z) + seq_at(a.s, t, t0 + u, a.zb, a.zt) + k.c0 + q);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float y = sy[u][q + j];
          if (a.Dk) y += a.Dk[k.c0 + q + j] * sd[u][q + j].y;
          if (a.z) y *= siluf(z.get(j));
          o.set(j, y);
        }
        st_pack<T, V>(reinterpret_cast<T*>(a.y) + seq_at(a.s, t, t0 + u, a.yb, a.yt) + k.c0 + q, o);
      }
    }
  }
  if (!live) return;
  if (ENDS) {
    st_states4(seg_h + (seg * a.D + c) * a.N, n0, a.N, h);
    if (nl == 0) seg_dt[seg * a.D + c] = sum;
  } else if (a.h_out && end == t.len) {
    st_states4(a.h_out + ((long)t.slot * a.D + c) * a.N, n0, a.N, h);
  }
}

// Joins the segments of each sequence: seg_h becomes the state each segment starts from.
// One thread per (sequence, channel, state).
static __global__ void __launch_bounds__(256)
    join_kernel(ScanArgs a, int S, float* seg_h, const float* seg_dt) {
  const long dn = (long)a.D * a.N;
  const int b = blockIdx.y;
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  long seg;
  if (a.s.start) {
    const int s = a.s.start[b], e = a.s.start[b + 1];
    if (s < 0 || e < s || e > a.s.L) return;
    seg = (long)s / S + b;
  } else {
    seg = (long)b * seq_tiles_of(a.s.L, S);
  }
  SeqTile t;
  if (!seq_tile(a.s, seg, S, t) || i >= dn) return;
  const int c = (int)(i / a.N);
  const float A2 = a.A[i] * ATLAS_LOG2E;
  float h = a.h_in && t.carry ? a.h_in[(long)t.slot * dn + i] : 0.f;
  const int n = seq_tiles_of(t.len, S);
  for (int k = 0; k < n; ++k, ++seg) {
    const float own = k + 1 < n ? seg_h[seg * dn + i] : 0.f;
    const float d = k + 1 < n ? seg_dt[seg * a.D + c] : 0.f;
    seg_h[seg * dn + i] = h;
    h = ex2(A2 * d) * h + own;
  }
}

// One token a sequence: every lane takes four states of a channel, loads and stores them
// once.  Bound by the state's traffic.
template <typename T, int LN>
__global__ void __launch_bounds__(kThreads) token_kernel(ScanArgs a) {
  using P = Shape<LN>;
  SeqTile t;
  const int b = blockIdx.x;
  if (!seq_tile(a.s, b, 1, t)) return;
  const int lane = threadIdx.x & 31, nl = lane % LN, n0 = nl * 4;
  const int c = blockIdx.y * P::kCB + (threadIdx.x >> 5) * P::kCW + lane / LN;
  const bool live = c < a.D;
  float y = 0.f, x = 0.f;
  if (live) {
    float A[4], h[4] = {0.f, 0.f, 0.f, 0.f};
    ld_states4(a.A + (long)c * a.N, n0, a.N, A);
    if (a.h_in && t.carry) ld_states4(a.h_in + ((long)t.slot * a.D + c) * a.N, n0, a.N, h);
    x = to_f(reinterpret_cast<const T*>(a.x)[b * a.xb + c]);
    const float d = step_of(a, to_f(reinterpret_cast<const T*>(a.dt)[b * a.tb + c]), c);
    const long g = (long)(c / (a.D / a.G)) * a.N;
    const T* B = reinterpret_cast<const T*>(a.Bm) + b * a.bb + g;
    const T* C = reinterpret_cast<const T*>(a.Cm) + b * a.cb + g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n0 + i < a.N) {
        h[i] = ex2(d * (A[i] * ATLAS_LOG2E)) * h[i] + d * x * to_f(B[n0 + i]);
        y += h[i] * to_f(C[n0 + i]);
      }
    if (a.h_out) st_states4(a.h_out + ((long)t.slot * a.D + c) * a.N, n0, a.N, h);
  }
  lane_sums<1, LN, 1>(&y, lane);
  if (live && nl == 0) {
    if (a.Dk) y += a.Dk[c] * x;
    if (a.z) y *= siluf(to_f(reinterpret_cast<const T*>(a.z)[b * a.zb + c]));
    reinterpret_cast<T*>(a.y)[b * a.yb + c] = from_f<T>(y);
  }
}

// Segment length: one segment a sequence when the sequences alone give four blocks an SM;
// otherwise segments for that many, but not below 128 tokens, where the second pass over
// them costs more than it brings.  0: no segments.
inline int segment_tokens(const ScanArgs& a, long blocks_per_seq) {
  const long want = 152 * 4;
  const long rows = a.s.start ? a.s.L : (long)a.s.B * a.s.L;
  if (!a.s.start && a.s.B * blocks_per_seq >= want) return 0;
  if ((a.s.start ? a.s.L : a.s.L) <= 256) return 0;
  long S = rows * blocks_per_seq / want / kTile * kTile;
  if (S < 128) S = 128;
  if (S >= a.s.L) return 0;
  return (int)S;
}

template <int LN>
size_t workspace(const ScanArgs& a) {
  const int S = segment_tokens(a, channel_blocks<LN>(a));
  return S ? (size_t)seq_tiles(a.s, S) * a.D * (a.N + 1) * 4 : 0;
}

template <typename T, int V, int LN>
int forward(const ScanArgs& a, cudaStream_t st) {
  constexpr int VV = V < Shape<LN>::kCB ? V : Shape<LN>::kCB;
  const int by = channel_blocks<LN>(a);
  if (by > 65535 || a.s.B > 65535) return ATLAS_ERR_UNSUPPORTED;
  if (!a.s.start && a.s.L == 1) {
    const dim3 grid(a.s.B, (a.D + Shape<LN>::kCB - 1) / Shape<LN>::kCB);
    token_kernel<T, LN><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
  }
  int S = segment_tokens(a, by);
  float *seg_h = nullptr, *seg_dt = nullptr;
  if (S) {
    const long segs = seq_tiles(a.s, S);
    seg_h = reinterpret_cast<float*>(a.ws);
    seg_dt = seg_h + (size_t)segs * a.D * a.N;
    segment_kernel<T, VV, LN, true><<<dim3((unsigned)segs, by), kThreads, 0, st>>>(a, S, seg_h, seg_dt);
    const long dn = (long)a.D * a.N;
    join_kernel<<<dim3((unsigned)((dn + 255) / 256), a.s.B), 256, 0, st>>>(a, S, seg_h, seg_dt);
  } else {
    S = a.s.L > 0 ? a.s.L : 1;
  }
  const long segs = seq_tiles(a.s, S);
  segment_kernel<T, VV, LN, false><<<dim3((unsigned)segs, by), kThreads, 0, st>>>(a, S, seg_h, seg_dt);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <typename T, int V>
int forward_n(const ScanArgs& a, cudaStream_t st) {
  if (a.N <= 8) return forward<T, V, 2>(a, st);
  if (a.N <= 16) return forward<T, V, 4>(a, st);
  if (a.N <= 32) return forward<T, V, 8>(a, st);
  if (a.N <= 64) return forward<T, V, 16>(a, st);
  return forward<T, V, 32>(a, st);
}

}  // namespace scan
}  // namespace atlas
