// scan_bwd_body.cuh -- backward pass of the selective scan, for one element type.
//
// With a_t = exp(dt_t A), u_t = dt_t x_t and dy'_t = dy_t SiLU(z_t), per channel and state:
//   g_t = C_t dy'_t + a_{t+1} g_{t+1}                       (dL/dh_t)
//   dC_t = sum_c h_t dy'_t,   dB_t = sum_c g_t u_t,   s_t = sum_n g_t B_t
//   q_t = g_t a_t h_{t-1},    dA = sum_t q_t dt_t
//   dx_t = s_t dt_t + D dy'_t,   ddt_t = s_t x_t + sum_n q_t A,   through softplus' slope
//   dz_t = dy_t SiLU'(z_t) (sum_n C_t h_t + D x_t),   dD = sum dy'_t x_t
//
// Three passes over the tokens.  The first walks each segment forwards from a zero state
// and keeps the state every kSub tokens (with the sum of dt, which carries the segment's
// true start state to that place) and what the segment adds to the adjoint in front of it;
// a small kernel joins the segments in both directions; the main pass walks backwards,
// kSub tokens at a time, with their decays and states computed again into registers.  Sums
// over states and over channels are taken by halving over lanes; every block writes
// partial sums of dB, dC (per token) and dA, dD, ddt_bias (per segment), which the last
// kernel adds in a fixed order.
#pragma once
#include "scan_body.cuh"

namespace atlas {
namespace scan {

constexpr int kSub = 8;
constexpr int kBackThreads = 128;

template <int LN>
struct BackShape {
  static constexpr int kNP = 4 * LN;                   // padded states
  static constexpr int kCW = 32 / LN;                  // channels of a warp
  static constexpr int kCB = kCW * kBackThreads / 32;  // channels of a block
};

// Sizes and workspace of a backward call.
template <int LN>
struct Back {
  int S, nsub, cb;  // segment tokens, kept states a segment, channel blocks
  bool split;       // more than one segment a sequence is possible
  long segs, rows;
  float *keep_h, *keep_dt;  // [segs * nsub][D][N], [segs * nsub][D]
  float *seg_h, *seg_g, *seg_dt;  // [segs][D][N] (start state; adjoint behind the end), [segs][D]
  float *pA, *pD, *pb;      // [segs][D][N], [segs][D] twice
  float* pbc;               // [cb][rows][2][NP]
  size_t bytes;
  Back(const ScanArgs& a, void* ws) {
    cb = blocks_over<BackShape<LN>::kCB>(a);
    S = segment_tokens(a, cb);
    split = S != 0;
    if (!S) S = a.s.L > 0 ? a.s.L : 1;
    nsub = (S + kSub - 1) / kSub;
    segs = seq_tiles(a.s, S);
    rows = a.s.start ? a.s.L : (long)a.s.B * a.s.L;
    const size_t D = a.D, DN = D * a.N;
    float* p = reinterpret_cast<float*>(ws);
    bytes = 0;
    auto take = [&](float*& q, size_t n) {
      q = p ? p + bytes : nullptr;
      bytes += (n + 3) / 4 * 4;
    };
    take(keep_h, (size_t)segs * nsub * DN);
    take(keep_dt, (size_t)segs * nsub * D);
    take(seg_h, split ? segs * DN : 0);
    take(seg_g, split ? segs * DN : 0);
    take(seg_dt, split ? segs * D : 0);
    take(pA, segs * DN);
    take(pD, segs * D);
    take(pb, segs * D);
    take(pbc, (size_t)cb * rows * 2 * BackShape<LN>::kNP);
    bytes *= 4;
  }
};

// Tokens t0 .. t0 + TT of dt (through softplus) and x into sd, those past `end` as zeros.
template <typename T, int V, int LN, int TT>
__device__ __forceinline__ void load_dx(const ScanArgs& a, const SeqTile& t, const Channels& k,
                                        int t0, int end, float2 (*sd)[BackShape<LN>::kCB]) {
  constexpr int CV = BackShape<LN>::kCB / V;
  for (int i = threadIdx.x; i < TT * CV; i += kBackThreads) {
    const int u = i / CV, cl = (i % CV) * V;
    if (t0 + u < end && cl < k.n) {
      const auto x = ld_pack<T, V>(reinterpret_cast<const T*>(a.x) + seq_at(a.s, t, t0 + u, a.xb, a.xt) + k.c0 + cl);
      const auto d = ld_pack<T, V>(reinterpret_cast<const T*>(a.dt) + seq_at(a.s, t, t0 + u, a.tb, a.tt) + k.c0 + cl);
      float bias[V], step[V];
#pragma unroll
      for (int j = 0; j < V; ++j) bias[j] = a.bias ? a.bias[k.c0 + cl + j] : 0.f;
      steps_of<T, V>(a, d, bias, step);
#pragma unroll
      for (int j = 0; j < V; ++j) sd[u][cl + j] = make_float2(step[j], x.get(j));
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) sd[u][cl + j] = make_float2(0.f, 0.f);
    }
  }
}

template <typename T, int LN, int TT>
__device__ __forceinline__ void load_states(const ScanArgs& a, const SeqTile& t, const Channels& k,
                                            int t0, int end, const void* p, long sb, long st,
                                            float (*s)[BackShape<LN>::kNP]) {
  constexpr int NP = 4 * LN;
  const T* q = rows_of<T>(p, a, t, sb, st, k.g * a.N);
  for (int i = threadIdx.x; i < TT * NP; i += kBackThreads) {
    const int u = t0 + i / NP, n = i % NP;
    s[i / NP][n] = u < end && n < a.N ? to_f(q[(long)u * st + n]) : 0.f;
  }
}

// What the main pass needs of dy, z and softplus: dy SiLU(z), softplus' slope at the raw
// step (1 without softplus) and dy SiLU'(z).
template <typename T, int V, int LN>
__device__ __forceinline__ void load_up(const ScanArgs& a, const SeqTile& t, const Channels& k,
                                        int t0, int end, float (*dyg)[BackShape<LN>::kCB],
                                        float (*slope)[BackShape<LN>::kCB], float (*dyz)[BackShape<LN>::kCB]) {
  constexpr int CV = BackShape<LN>::kCB / V;
  for (int i = threadIdx.x; i < kSub * CV; i += kBackThreads) {
    const int u = i / CV, cl = (i % CV) * V;
    if (t0 + u < end && cl < k.n) {
      const auto dy = ld_pack<T, V>(reinterpret_cast<const T*>(a.dy) + seq_at(a.s, t, t0 + u, a.yb, a.yt) + k.c0 + cl);
      Pack<T, V> z, d;
      if (a.z) z = ld_pack<T, V>(reinterpret_cast<const T*>(a.z) + seq_at(a.s, t, t0 + u, a.zb, a.zt) + k.c0 + cl);
      if (slope) d = ld_pack<T, V>(reinterpret_cast<const T*>(a.dt) + seq_at(a.s, t, t0 + u, a.tb, a.tt) + k.c0 + cl);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g = dy.get(j);
        if (a.z) {
          const float zv = z.get(j), s = sigmoidf(zv);
          dyg[u][cl + j] = g * zv * s;
          if (dyz) dyz[u][cl + j] = g * silu_slope(zv, s);
        } else {
          dyg[u][cl + j] = g;
        }
        if (slope) {
          const int c = k.c0 + cl + j;
          slope[u][cl + j] = a.softplus ? sigmoidf(d.get(j) + (a.bias ? a.bias[c] : 0.f)) : 1.f;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        dyg[u][cl + j] = 0.f;
        if (slope) slope[u][cl + j] = 0.f;
        if (dyz) dyz[u][cl + j] = 0.f;
      }
    }
  }
}

template <typename T, int V, int LN>
__global__ void __launch_bounds__(kBackThreads) keep_kernel(ScanArgs a, Back<LN> w) {
  using P = BackShape<LN>;
  __shared__ float2 sd[kSub][P::kCB];
  __shared__ float sg[kSub][P::kCB];
  __shared__ __align__(16) float sB[kSub][P::kNP];
  __shared__ __align__(16) float sC[kSub][P::kNP];
  if (blockIdx.x == 0 && blockIdx.y == 0) seq_check(a.s, threadIdx.x, kBackThreads);
  const long seg = blockIdx.x;
  SeqTile t;
  if (!seq_tile(a.s, seg, w.S, t)) return;
  const int end = min(t.t0 + w.S, t.len);
  const Channels k = channels_at<BackShape<LN>::kCB>(a, blockIdx.y);
  const int lane = threadIdx.x & 31, nl = lane % LN, n0 = nl * 4;
  const int cl = (threadIdx.x >> 5) * P::kCW + lane / LN, c = k.c0 + cl;
  const bool live = cl < k.n;
  float A2[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  float p[4] = {1.f, 1.f, 1.f, 1.f}, g[4] = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    ld_states4(a.A + (long)c * a.N, n0, a.N, A2);
    if (!w.split && a.h_in && t.carry)
      ld_states4(a.h_in + ((long)t.b * a.D + c) * a.N, n0, a.N, h);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] *= ATLAS_LOG2E;
  for (int t0 = t.t0; t0 < end; t0 += kSub) {
    __syncthreads();
    load_dx<T, V, LN, kSub>(a, t, k, t0, end, sd);
    load_states<T, LN, kSub>(a, t, k, t0, end, a.Bm, a.bb, a.bt, sB);
    if (w.split) {
      load_states<T, LN, kSub>(a, t, k, t0, end, a.Cm, a.cb, a.ct, sC);
      load_up<T, V, LN>(a, t, k, t0, end, sg, nullptr, nullptr);
    }
    __syncthreads();
    if (live) {
      const long at = (seg * w.nsub + (t0 - t.t0) / kSub) * a.D + c;
      st_states4(w.keep_h + at * a.N, n0, a.N, h);
      if (nl == 0) w.keep_dt[at] = sum;
    }
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      const float2 d = sd[u][cl];
      const float gx = d.x * d.y;
      sum += d.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float e = ex2(d.x * A2[i]);
        h[i] = e * h[i] + gx * sB[u][n0 + i];
        if (w.split) {
          p[i] *= e;
          g[i] += p[i] * (sC[u][n0 + i] * sg[u][cl]);
        }
      }
    }
  }
  if (live && w.split) {
    const long at = seg * a.D + c;
    st_states4(w.seg_h + at * a.N, n0, a.N, h);
    st_states4(w.seg_g + at * a.N, n0, a.N, g);
    if (nl == 0) w.seg_dt[at] = sum;
  }
}

// seg_h becomes the state each segment starts from, seg_g the adjoint behind its last token;
// dh becomes dL/d h_in.
template <int LN>
__global__ void __launch_bounds__(256) join_back_kernel(ScanArgs a, Back<LN> w) {
  const long dn = (long)a.D * a.N;
  const int b = blockIdx.y;
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  long seg;
  if (a.s.start) {
    const int s = a.s.start[b], e = a.s.start[b + 1];
    if (s < 0 || e < s || e > a.s.L) return;
    seg = (long)s / w.S + b;
  } else {
    seg = (long)b * seq_tiles_of(a.s.L, w.S);
  }
  SeqTile t;
  if (!seq_tile(a.s, seg, w.S, t) || i >= dn) return;
  const int c = (int)(i / a.N);
  const float A2 = a.A[i] * ATLAS_LOG2E;
  const int n = seq_tiles_of(t.len, w.S);
  float h = a.h_in && t.carry ? a.h_in[(long)b * dn + i] : 0.f;
  for (int k = 0; k < n; ++k) {
    const float own = w.seg_h[(seg + k) * dn + i];
    w.seg_h[(seg + k) * dn + i] = h;
    h = ex2(A2 * w.seg_dt[(seg + k) * a.D + c]) * h + own;
  }
  float g = a.dh ? a.dh[(long)b * dn + i] : 0.f;
  for (int k = n - 1; k >= 0; --k) {
    const float own = w.seg_g[(seg + k) * dn + i];
    w.seg_g[(seg + k) * dn + i] = g;
    g = ex2(A2 * w.seg_dt[(seg + k) * a.D + c]) * g + own;
  }
  if (a.dh) a.dh[(long)b * dn + i] = t.carry ? g : 0.f;
}

template <typename T, int V, int LN>
__global__ void __launch_bounds__(kBackThreads) back_kernel(ScanArgs a, Back<LN> w) {
  using P = BackShape<LN>;
  __shared__ float2 sd[kSub][P::kCB];
  __shared__ float sg[kSub][P::kCB], ss[kSub][P::kCB], sz[kSub][P::kCB];
  __shared__ __align__(16) float sB[kSub][P::kNP];
  __shared__ __align__(16) float sC[kSub][P::kNP];
  __shared__ float sp[kBackThreads / 32][kSub][2 * P::kNP];
  __shared__ float so[3][kSub][P::kCB];
  const long seg = blockIdx.x;
  const Channels k = channels_at<BackShape<LN>::kCB>(a, blockIdx.y);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nl = lane % LN, n0 = nl * 4;
  const int chl = lane / LN, cl = warp * P::kCW + chl, c = k.c0 + cl;
  const bool live = cl < k.n;
  float A2[4] = {0.f, 0.f, 0.f, 0.f}, hs[4] = {0.f, 0.f, 0.f, 0.f}, gp[4] = {0.f, 0.f, 0.f, 0.f};
  float dA[4] = {0.f, 0.f, 0.f, 0.f}, dD = 0.f, db = 0.f;
  SeqTile t;
  const bool some = seq_tile(a.s, seg, w.S, t);
  if (some) {
    const int end = min(t.t0 + w.S, t.len);
    if (live) {
      ld_states4(a.A + (long)c * a.N, n0, a.N, A2);
      if (w.split) {
        ld_states4(w.seg_h + (seg * a.D + c) * a.N, n0, a.N, hs);
        ld_states4(w.seg_g + (seg * a.D + c) * a.N, n0, a.N, gp);
      } else if (a.dh) {
        ld_states4(a.dh + ((long)t.b * a.D + c) * a.N, n0, a.N, gp);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] *= ATLAS_LOG2E;
    const float Dk = a.Dk && live ? a.Dk[c] : 0.f;
    const long row0 = a.s.start ? t.first : (long)t.b * a.s.L;
    for (int sub = (end - t.t0 + kSub - 1) / kSub - 1; sub >= 0; --sub) {
      const int t0 = t.t0 + sub * kSub;
      __syncthreads();
      load_dx<T, V, LN, kSub>(a, t, k, t0, end, sd);
      load_states<T, LN, kSub>(a, t, k, t0, end, a.Bm, a.bb, a.bt, sB);
      load_states<T, LN, kSub>(a, t, k, t0, end, a.Cm, a.cb, a.ct, sC);
      load_up<T, V, LN>(a, t, k, t0, end, sg, ss, a.z ? sz : nullptr);
      float h[4] = {0.f, 0.f, 0.f, 0.f};
      if (live) {
        const long at = (seg * w.nsub + sub) * a.D + c;
        ld_states4(w.keep_h + at * a.N, n0, a.N, h);
        if (w.split) {
          const float cum = w.keep_dt[at];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] += ex2(A2[i] * cum) * hs[i];
        }
      }
      __syncthreads();
      float e[kSub][4], v[kSub][4];  // a_t and a_t h_{t-1}
#pragma unroll
      for (int u = 0; u < kSub; ++u) {
        const float2 d = sd[u][cl];
        const float4 b = *reinterpret_cast<const float4*>(&sB[u][n0]);
        const float bb[4] = {b.x, b.y, b.z, b.w}, gx = d.x * d.y;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[u][i] = ex2(d.x * A2[i]);
          v[u][i] = e[u][i] * h[i];
          h[i] = v[u][i] + gx * bb[i];
        }
      }
#pragma unroll
      for (int u0 = kSub - 4; u0 >= 0; u0 -= 4) {
        float ry[4], rs[4], rq[4];
#pragma unroll
        for (int uu = 3; uu >= 0; --uu) {
          const int u = u0 + uu;
          const float2 d = sd[u][cl];
          const float4 b4 = *reinterpret_cast<const float4*>(&sB[u][n0]);
          const float4 c4 = *reinterpret_cast<const float4*>(&sC[u][n0]);
          const float bb[4] = {b4.x, b4.y, b4.z, b4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
          const float gx = d.x * d.y, dyg = sg[u][cl];
          float m[8], y = 0.f, s = 0.f, q = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float g = gp[i] + cc[i] * dyg;
            const float ht = v[u][i] + gx * bb[i];
            const float qt = g * v[u][i];
            y += cc[i] * ht;
            s += g * bb[i];
            q += qt * A2[i];
            dA[i] += qt * d.x;
            m[i] = g * gx;
            m[4 + i] = ht * dyg;
            gp[i] = e[u][i] * g;
          }
          ry[uu] = y;
          rs[uu] = s;
          rq[uu] = q;
          lane_sums<8, P::kCW, LN>(m, lane);
          if (P::kCW <= 8) {
            constexpr int NV = P::kCW <= 8 ? 8 / P::kCW : 1;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              const int id = chl * NV + i;
              sp[warp][u][(id >> 2) * P::kNP + n0 + (id & 3)] = m[i];
            }
          } else if (chl % (P::kCW > 8 ? P::kCW / 8 : 1) == 0) {
            const int id = chl / (P::kCW > 8 ? P::kCW / 8 : 1);
            sp[warp][u][(id >> 2) * P::kNP + n0 + (id & 3)] = m[0];
          }
        }
        lane_sums<4, LN, 1>(ry, lane);
        lane_sums<4, LN, 1>(rs, lane);
        lane_sums<4, LN, 1>(rq, lane);
        constexpr int NV = LN <= 4 ? 4 / LN : 1, NR = LN > 4 ? LN / 4 : 1;
        if (nl % NR == 0) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int u = u0 + (LN <= 4 ? nl * NV + i : nl / NR);
            const float2 d = sd[u][cl];
            const float dyg = sg[u][cl];
            const float ddt = (rs[i] * d.y + rq[i] * (1.f / ATLAS_LOG2E)) * ss[u][cl];
            so[0][u][cl] = rs[i] * d.x + Dk * dyg;
            so[1][u][cl] = ddt;
            if (a.z) so[2][u][cl] = sz[u][cl] * (ry[i] + Dk * d.y);
            dD += dyg * d.y;
            db += ddt;
          }
        }
      }
      __syncthreads();
      constexpr int CV = P::kCB / V;
      for (int i = threadIdx.x; i < kSub * CV; i += kBackThreads) {
        const int u = i / CV, q = (i % CV) * V;
        if (t0 + u >= end || q >= k.n) continue;
        Pack<T, V> o;
#pragma unroll
        for (int j = 0; j < V; ++j) o.set(j, so[0][u][q + j]);
        st_pack<T, V>(reinterpret_cast<T*>(a.dx) + seq_at(a.s, t, t0 + u, a.xb, a.xt) + k.c0 + q, o);
#pragma unroll
        for (int j = 0; j < V; ++j) o.set(j, so[1][u][q + j]);
        st_pack<T, V>(reinterpret_cast<T*>(a.ddt) + seq_at(a.s, t, t0 + u, a.tb, a.tt) + k.c0 + q, o);
        if (a.z) {
#pragma unroll
          for (int j = 0; j < V; ++j) o.set(j, so[2][u][q + j]);
          st_pack<T, V>(reinterpret_cast<T*>(a.dz) + seq_at(a.s, t, t0 + u, a.zb, a.zt) + k.c0 + q, o);
        }
      }
      for (int i = threadIdx.x; i < kSub * 2 * P::kNP; i += kBackThreads) {
        const int u = i / (2 * P::kNP), q = i % (2 * P::kNP);
        if (t0 + u >= end) continue;
        float s = sp[0][u][q];
#pragma unroll
        for (int r = 1; r < kBackThreads / 32; ++r) s += sp[r][u][q];
        w.pbc[((long)blockIdx.y * w.rows + row0 + t0 + u) * 2 * P::kNP + q] = s;
      }
    }
  }
  // dD and ddt_bias lie in the lanes that owned the tokens
#pragma unroll
  for (int m = LN / 2; m; m >>= 1) {
    dD += __shfl_xor_sync(0xFFFFFFFFu, dD, m);
    db += __shfl_xor_sync(0xFFFFFFFFu, db, m);
  }
  if (!live) return;
  const long at = seg * a.D + c;
  st_states4(w.pA + at * a.N, n0, a.N, dA);
  if (nl == 0) {
    w.pD[at] = dD;
    w.pb[at] = db;
  }
  if (some && !w.split && a.dh) {
#pragma unroll
    for (int i = 0; i < 4; ++i) gp[i] = t.carry ? gp[i] : 0.f;
    st_states4(a.dh + ((long)t.b * a.D + c) * a.N, n0, a.N, gp);
  }
}

// Adds the partial sums: the first `nbc` blocks dB and dC, the others dA, dD and ddt_bias.
template <typename T, int LN>
__global__ void __launch_bounds__(256) finish_kernel(ScanArgs a, Back<LN> w, int nbc) {
  constexpr int NP = BackShape<LN>::kNP;
  if ((int)blockIdx.x < nbc) {
    const int bpg = w.cb / a.G;
    long lo = 0, hi = w.rows;
    if (a.s.start) {
      lo = min(max(a.s.start[0], 0), a.s.L);
      hi = min(max(a.s.start[a.s.B], 0), a.s.L);
    }
    const long n = w.rows * a.G * 2 * NP;
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)nbc * 256) {
      const int q = (int)(i % (2 * NP));
      const int g = (int)(i / (2 * NP) % a.G);
      const long r = i / (2 * NP) / a.G;
      if (q % NP >= a.N || r < lo || r >= hi) continue;
      float s = 0.f;
      for (int k = 0; k < bpg; ++k)
        s += w.pbc[((long)(g * bpg + k) * w.rows + r) * 2 * NP + q];
      const bool isC = q >= NP;
      const long sb = isC ? a.cb : a.bb, st = isC ? a.ct : a.bt;
      const long at = a.s.start ? r * st : r / a.s.L * sb + r % a.s.L * st;
      reinterpret_cast<T*>(isC ? a.dC : a.dB)[at + (long)g * a.N + q % NP] = from_f<T>(s);
    }
    return;
  }
  const long dn = (long)a.D * a.N;
  for (long i = (long)(blockIdx.x - nbc) * 256 + threadIdx.x; i < dn + 2 * a.D;
       i += (long)(gridDim.x - nbc) * 256) {
    const float* p = i < dn ? w.pA + i : i < dn + a.D ? w.pD + (i - dn) : w.pb + (i - dn - a.D);
    const long step = i < dn ? dn : a.D;
    float s = 0.f;
    for (long k = 0; k < w.segs; ++k) s += p[k * step];
    if (i < dn)
      a.dA[i] = s;
    else if (i < dn + a.D) {
      if (a.dD) a.dD[i - dn] = s;
    } else if (a.dbias) {
      a.dbias[i - dn - a.D] = s;
    }
  }
}

template <typename T, int V, int LN>
int backward(const ScanArgs& a, cudaStream_t st) {
  constexpr int VV = V < BackShape<LN>::kCB ? V : BackShape<LN>::kCB;
  const Back<LN> w(a, a.ws);
  if (w.cb > 65535 || a.s.B > 65535 || w.segs > 0x7FFFFFFFL) return ATLAS_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)w.segs, w.cb);
  if (w.segs > 0) keep_kernel<T, VV, LN><<<grid, kBackThreads, 0, st>>>(a, w);
  if (w.segs > 0 && w.split)
    join_back_kernel<LN><<<dim3((unsigned)(((long)a.D * a.N + 255) / 256), a.s.B), 256, 0, st>>>(a, w);
  if (w.segs > 0) back_kernel<T, VV, LN><<<grid, kBackThreads, 0, st>>>(a, w);
  const long nb = (w.rows * a.G * 2 * BackShape<LN>::kNP + 255) / 256;
  const int nbc = (int)(nb < 152 * 16 ? nb : 152 * 16);
  const long na = ((long)a.D * (a.N + 2) + 255) / 256;
  finish_kernel<T, LN><<<nbc + (int)(na < 4096 ? na : 4096), 256, 0, st>>>(a, w, nbc);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <typename T, int V>
int backward_n(const ScanArgs& a, cudaStream_t st) {
  if (a.N <= 8) return backward<T, V, 2>(a, st);
  if (a.N <= 16) return backward<T, V, 4>(a, st);
  if (a.N <= 32) return backward<T, V, 8>(a, st);
  if (a.N <= 64) return backward<T, V, 16>(a, st);
  return backward<T, V, 32>(a, st);
}

}  // namespace scan
}  // namespace atlas
