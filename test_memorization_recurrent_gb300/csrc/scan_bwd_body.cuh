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
//
// What bounds it: instruction issue in the main pass, 26 for 32 updates (17 of them in the
// walking warps: the decay and state twice, the adjoint, seven products, and the two kinds of
// sums).  Holding a tile's decays instead of taking them again costs 64 registers and with
// them half the warps.  4 x 2048 tokens x 2048 channels x 16 states, bf16, gated: 494 us, of
// which the main pass takes two thirds (55% of the issue slots) and the kept states a quarter; the first
// kernels, with one channel x four states a lane and loads in every warp's turn, took 1822.
#pragma once
#include "scan_body.cuh"

namespace atlas {
namespace scan {

constexpr int kWalkers = 4;                        // warps that walk; as many prepare and finish
constexpr int kBackThreads = 2 * kWalkers * kThreads;
constexpr int kBackRing = 4;  // tiles as they lie in memory: finished, walked, prepared, under way

template <int LN>
constexpr int kBackCB = kWalkers * Shape<LN>::kCB;  // channels of a block

// Segment length, 0 for one segment a sequence.  The main pass runs n blocks, two an SM at a
// time, for a little over S tokens each (30 more for a block's start): one round of blocks takes
// that long, several about half a round more than their share.  The shortest of the lengths
// from 128 on is taken (4 x 2048 tokens x 2048 channels, in the sweep that chose it: 478 us with 256, 501 with 128, 516 with
// 512, 624 with 2048; 8 x 512 x 2048: 252 with 512, 279 with 256).
inline int back_segment_tokens(const ScanArgs& a, long blocks_per_seq) {
  const long L = a.s.L, B = a.s.start ? 1 : a.s.B, more = a.s.start ? a.s.B : 0;
  int best = 0;
  double least = 0;
  for (long c = 128;; c = c % 3 ? c / 2 * 3 : c / 3 * 4) {  // 128, 192, 256, 384, ..
    const bool whole = c >= L;
    const long m = whole ? 1 : (L + c - 1) / c;  // segments a sequence
    const long S = whole ? L : ((L + m - 1) / m + kTile - 1) / kTile * kTile;
    const double n = (double)(B * m + more) * blocks_per_seq / (kSMs * 2);
    const double cost = n <= 1 ? 1.05 * S + 30 : (n + 0.5) * S + n * 30;
    if (best == 0 || cost < least) {
      best = whole ? -1 : (int)S;
      least = cost;
    }
    if (whole) break;
  }
  return best < 0 || best >= L ? 0 : best;
}

// Sizes and workspace of a backward call.
template <int LN>
struct Back {
  int S, cb;        // segment tokens, channel blocks
  bool split;       // more than one segment a sequence is possible
  long segs, rows;
  float *keep_h, *keep_dt;  // [places][D][N], [places][D]
  float *seg_h, *seg_g, *seg_dt;  // [segs][D][N] (start state; adjoint behind the end), [segs][D]
  float *pA, *pD, *pb;      // [segs][D][N], [segs][D] twice
  float* pbc;               // [cb][rows][2][NP]
  float* rising;            // a word, as an int: how many sequences count
  size_t bytes;
  Back(const ScanArgs& a, void* ws) {
    cb = blocks_over<kBackCB<LN>>(a);
    S = back_segment_tokens(a, cb);
    split = S != 0;
    if (!S) S = a.s.L > 0 ? a.s.L : 1;
    segs = seq_tiles(a.s, S);
    rows = a.s.start ? a.s.L : (long)a.s.B * a.s.L;
    const size_t D = a.D, DN = D * a.N;
    float* p = reinterpret_cast<float*>(ws);
    bytes = 0;
    auto take = [&](float*& q, size_t n) {
      q = p ? p + bytes : nullptr;
      bytes += (n + 3) / 4 * 4;
    };
    take(rising, kRisingBytes / 4);
    take(keep_h, kept_places(a.s) * DN);
    take(keep_dt, kept_places(a.s) * D);
    take(seg_h, split ? segs * DN : 0);
    take(seg_g, split ? segs * DN : 0);
    take(seg_dt, split ? segs * D : 0);
    take(pA, segs * DN);
    take(pD, segs * D);
    take(pb, segs * D);
    take(pbc, (size_t)cb * rows * 2 * Shape<LN>::kNP);
    bytes *= 4;
  }
  // in the kernels behind the first
  __device__ int rising_of(const SeqArgs& a) const { return a.start ? *reinterpret_cast<const int*>(rising) : a.B; }
  Segments segments() const {
    return Segments{S, split ? seg_h : nullptr, seg_dt, seg_g, keep_h, keep_dt, reinterpret_cast<int*>(rising), 0};
  }
};

// seg_h becomes the state each segment starts from, seg_g the adjoint behind its last token;
// dh becomes dL/d h_in.
template <int LN>
__global__ void __launch_bounds__(256) join_back_kernel(ScanArgs a, Back<LN> w) {
  const long dn = (long)a.D * a.N;
  const int b = blockIdx.y;
  const long i = (long)blockIdx.x * 256 + threadIdx.x;
  int s = 0, len = a.s.L;
  if (a.s.start) {
    const int e = a.s.start[b + 1], rising = w.rising_of(a.s);
    s = a.s.start[b];
    if (b >= rising || s < 0 || e < s || e > a.s.L) return;
    len = e - s;
  }
  if (i >= dn) return;
  const bool carry = a.s.carry ? a.s.carry[b] != 0 : true;
  const long seg = a.s.start ? (long)s / w.S + b : (long)b * seq_tiles_of(a.s.L, w.S);
  const int c = (int)(i / a.N);
  const float A2 = log2_decay(a.A[i]);
  const int n = seq_tiles_of(len, w.S);
  // eight segments' values are under way at a time
  constexpr int U = 8;
  float h = a.h_in && carry ? a.h_in[(long)b * dn + i] : 0.f;
  for (int k0 = 0; k0 < n; k0 += U) {
    float own[U], d[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      own[j] = k0 + j < n ? w.seg_h[(seg + k0 + j) * dn + i] : 0.f;
      d[j] = k0 + j < n ? w.seg_dt[(seg + k0 + j) * a.D + c] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (k0 + j < n) w.seg_h[(seg + k0 + j) * dn + i] = h;
      h = ex2(A2 * d[j]) * h + own[j];
    }
  }
  float g = a.dh ? a.dh[(long)b * dn + i] : 0.f;
  for (int k0 = n - 1; k0 >= 0; k0 -= U) {
    float own[U], d[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      own[j] = k0 - j >= 0 ? w.seg_g[(seg + k0 - j) * dn + i] : 0.f;
      d[j] = k0 - j >= 0 ? w.seg_dt[(seg + k0 - j) * a.D + c] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (k0 - j >= 0) w.seg_g[(seg + k0 - j) * dn + i] = g;
      g = ex2(A2 * d[j]) * g + own[j];
    }
  }
  if (a.dh) a.dh[(long)b * dn + i] = carry ? g : 0.f;
}

// Shared memory of back_kernel.
template <typename T, int LN>
struct BackShared {
  using P = Shape<LN>;
  struct Raw {  // tiles as they lie in memory, each preparing warp's channels apart
    alignas(16) T x[kWalkers][kSub][P::kCB];
    alignas(16) T dt[kWalkers][kSub][P::kCB];
    alignas(16) T z[kWalkers][kSub][P::kCB];
    alignas(16) T dy[kWalkers][kSub][P::kCB];
    alignas(16) T B[kSub][P::kNP];
    alignas(16) T C[kSub][P::kNP];
    alignas(16) float h[kWalkers][2][kThreads][4];  // the kept states of each walking lane's two
    alignas(16) float cum[kWalkers][P::kCB];        // channels, and the sum of dt there
  };
  alignas(16) float hs[kWalkers][2][kThreads][4];  // the states the segment starts from
  alignas(16) float2 d[2][kWalkers][kSub][P::kCB];     // dt, dt x
  alignas(16) float g[2][kWalkers][kSub][P::kCB];      // dy SiLU(z)
  alignas(16) float slope[2][kWalkers][kSub][P::kCB];  // of softplus
  alignas(16) float dz[2][kWalkers][kSub][P::kCB];     // dy SiLU'(z)
  alignas(16) float B[2][kSub][P::kNP];
  alignas(16) float C[2][kSub][P::kNP];
  alignas(16) float sums[2][3][kWalkers][kSub][P::kCB + 8];  // over states: C h, g B, q A
  alignas(16) float bc[2][kWalkers][kSub][2 * P::kNP];       // over a walker's channels: dB, dC
  Raw raw[kBackRing];
};

// ex2 that is not merged with an earlier one of the same argument: the decays of a whole tile
// would not fit the registers.
__device__ __forceinline__ pair32 pair_ex2_again(pair32 a) {
  float x, y;
  unpair(a, x, y);
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
  asm volatile("ex2.approx.ftz.f32 %0, %0;" : "+f"(y));
  return pair(x, y);
}

// The main pass.  A walker has two channels x four states a lane, as in the forward pass; it
// goes through kSub tokens forwards from the kept state, holding the states in registers, and
// then backwards.  Its partner prepares the tile before, and writes out the tile behind.
template <typename T, int V, int LN, bool NV>
__global__ void __launch_bounds__(kBackThreads, 2) back_kernel(ScanArgs a, Back<LN> w) {
  using P = Shape<LN>;
  using X = Tile<T, V, P::kCB, kSub>;
  constexpr int VN = !NV ? 1 : 16 / sizeof(T) < P::kNP ? 16 / sizeof(T) : P::kNP;
  using R = Tile<T, VN, P::kNP, kSub>;
  using Shared = BackShared<T, LN>;
  using Raw = typename Shared::Raw;
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  const long seg = blockIdx.x;
  const Channels kb = channels_at<kBackCB<LN>>(a, blockIdx.y);
  const int lane = threadIdx.x & 31, wi = (threadIdx.x >> 5) % kWalkers;
  const bool walks = threadIdx.x < kWalkers * kThreads;
  Channels k = kb;  // this warp's
  k.c0 += wi * P::kCB;
  k.n = max(0, min(P::kCB, kb.n - wi * P::kCB));
  const int rising = w.rising_of(a.s);
  SeqTile t;
  const bool some = seq_tile(a.s, rising, seg, w.S, t);
  const int end = some ? seq_tile_end(t, w.S) : 0;
  const int tiles = some ? (end - t.t0 + kSub - 1) / kSub : 0;
  const int first = tiles > 0 ? t.t0 + (tiles - 1) * kSub : 0;  // the last tile comes first

  if (!walks) {
    float dD[V], db[V], bias[V], skip[V];
    static_assert(kThreads % (P::kCB / V) == 0, "a thread's vectors share their channels");
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int ch = X::channel(0) + j;
      bias[j] = a.bias && ch < k.n ? a.bias[k.c0 + ch] : 0.f;
      skip[j] = a.Dk && ch < k.n ? a.Dk[k.c0 + ch] : 0.f;
      dD[j] = db[j] = 0.f;
    }
    if (tiles > 0) {
      X px(rows_of<T>(a.x, a, t, a.xb, a.xt, k.c0), a.xt, first);
      X pd(rows_of<T>(a.dt, a, t, a.tb, a.tt, k.c0), a.tt, first);
      X pz(rows_of<T>(a.z ? a.z : a.x, a, t, a.zb, a.zt, k.c0), a.zt, first);
      X py(rows_of<T>(a.dy, a, t, a.yb, a.yt, k.c0), a.yt, first);
      X ox(rows_of<T>(a.dx, a, t, a.xb, a.xt, k.c0), a.xt, first);
      X od(rows_of<T>(a.ddt, a, t, a.tb, a.tt, k.c0), a.tt, first);
      X oz(rows_of<T>(a.z ? a.dz : a.dx, a, t, a.zb, a.zt, k.c0), a.zt, first);
      // the first partner brings B, the second C
      R pn(rows_of<T>(wi ? a.Cm : a.Bm, a, t, wi ? a.cb : a.bb, wi ? a.ct : a.bt, k.g * a.N), wi ? a.ct : a.bt, first);
      const long row0 = (a.s.start ? t.first : (long)t.b * a.s.L) + first;
      float* pbc = w.pbc + ((long)blockIdx.y * w.rows + row0) * 2 * P::kNP;
      int rf = 0, rp = 0, rn = 0;
      int nf = 0, np = 0;  // tiles fetched, prepared
      constexpr int KN = P::kCB * LN / kThreads;
      static_assert(P::kCB * LN % kThreads == 0, "every lane has the same number of pieces");
      int kept_to[KN], kept_from[KN], kept_n[KN];  // places in the ring, offsets, states (of four)
      const long at = (kept_at(a.s, t) + tiles - 1) * a.D;
#pragma unroll
      for (int i = 0; i < KN; ++i) {
        const int q = i * kThreads + lane, ch = q / LN, n = q % LN * 4;
        kept_to[i] = ((ch & 1) * kThreads + q % LN * P::kPairs + ch / 2) * 4;
        kept_n[i] = ch < k.n ? max(0, min(4, a.N - n)) : 0;
        kept_from[i] = kept_n[i] > 0 ? (k.c0 + ch) * a.N + n : 0;
      }
      const float* kept = w.keep_h + at * a.N;
      const float* cum = w.keep_dt + at + (lane < k.n ? k.c0 + lane : 0);
      const auto step = [](int& r) { r = (r + 1) % kBackRing; };
      auto fetch = [&]() {
        if (nf < tiles) {
          const int left = nf == 0 ? end - first : kSub;
          Raw& r = s.raw[rf];
          px.copy(r.x[wi], left, k.n), px.back();
          pd.copy(r.dt[wi], left, k.n), pd.back();
          py.copy(r.dy[wi], left, k.n), py.back();
          if (a.z) pz.copy(r.z[wi], left, k.n), pz.back();
          if (wi == 0) pn.copy(r.B, left, a.N), pn.back();
          if (wi == 1) pn.copy(r.C, left, a.N), pn.back();
          // each lane's pieces of the kept states: where they go and come from stays but for the tile
#pragma unroll
          for (int i = 0; i < KN; ++i) {
            float* o = r.h[wi][0][0] + kept_to[i];
            if (a.N % 4 == 0) {
              cp_async<16>(o, kept + kept_from[i], kept_n[i] > 0);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) cp_async<4>(o + j, kept + kept_from[i] + (j < kept_n[i] ? j : 0), j < kept_n[i]);
            }
          }
          kept -= (long)a.D * a.N;
          if (lane < P::kCB) cp_async<4>(&r.cum[wi][lane], cum, lane < k.n);
          cum -= a.D;
        }
        cp_commit();
      };
      auto put = [&]() {
        if (nf < tiles) {
          Raw& r = s.raw[rf];
          px.put(r.x[wi]);
          pd.put(r.dt[wi]);
          py.put(r.dy[wi]);
          if (a.z) pz.put(r.z[wi]);
          if (wi == 0) pn.put(r.B);
          if (wi == 1) pn.put(r.C);
        }
        ++nf;
        step(rf);
      };
      auto prepare = [&](int p) {
        if (np >= tiles) return;
        const int left = np == 0 ? end - first : kSub;
        const Raw& r = s.raw[rp];
        ++np;
        step(rp);
#pragma unroll
        for (int i = 0; i < X::kN; ++i)
          if (X::inside(i)) {
            const int u = X::token(i), q = X::channel(i);
            float x[V], d[V], y[V], z[V], sl[V], sz[V];
            ld_pack<T, V>(&r.x[wi][u][q]).unpack(x);
            ld_pack<T, V>(&r.dt[wi][u][q]).unpack(d);
            ld_pack<T, V>(&r.dy[wi][u][q]).unpack(y);
            if (a.z) ld_pack<T, V>(&r.z[wi][u][q]).unpack(z);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              d[j] += bias[j];
              sl[j] = 1.f;
              if (a.softplus) {
                sl[j] = sigmoidf(d[j]);
                d[j] = softplusf(d[j]);
              }
              sz[j] = 0.f;
              if (a.z) {
                const float sg = sigmoidf(z[j]);
                sz[j] = y[j] * silu_slope(z[j], sg);
                y[j] *= z[j] * sg;
              }
            }
            if (left < kSub) {  // nothing behind the end
#pragma unroll
              for (int j = 0; j < V; ++j)
                if (u >= left) d[j] = sl[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) x[j] *= d[j];
            if (V == 1) {
              s.d[p][wi][u][q] = make_float2(d[0], x[0]);
            } else {
#pragma unroll
              for (int j = 0; j + 1 < V; j += 2)
                *reinterpret_cast<float4*>(&s.d[p][wi][u][2 * turned<V>(u, (q + j) / 2)]) =
                    make_float4(d[j], x[j], d[j + 1], x[j + 1]);
            }
            st_vec<V>(&s.g[p][wi][u][q], y);
            st_vec<V>(&s.slope[p][wi][u][q], sl);
            if (a.z) st_vec<V>(&s.dz[p][wi][u][q], sz);
          }
        if (wi < 2) {
#pragma unroll
          for (int i = lane; i < kSub * P::kNP / 4; i += kThreads) {
            const int u = i / (P::kNP / 4), n = i % (P::kNP / 4) * 4;
            float b[4];
            ld_pack<T, 4>(wi ? &r.C[u][n] : &r.B[u][n]).unpack(b);
            *reinterpret_cast<float4*>(wi ? &s.C[p][u][n] : &s.B[p][u][n]) = make_float4(b[0], b[1], b[2], b[3]);
          }
        }
      };
      auto finish = [&](int p, int left) {
        const Raw& r = s.raw[rn];
        step(rn);
#pragma unroll
        for (int i = 0; i < X::kN; ++i) {
          const int u = X::token(i), q = X::channel(i);
          if (!X::inside(i) || u >= left || q >= k.n) continue;
          float x[V], dx[V], dd[V], dz[V], dt[V], dyg[V], gB[V], qA[V], sl[V];
          ld_pack<T, V>(&r.x[wi][u][q]).unpack(x);
          if (V == 1) {
            dt[0] = s.d[p][wi][u][q].x;
          } else {
#pragma unroll
            for (int j = 0; j + 1 < V; j += 2) {
              const float4 d = *reinterpret_cast<const float4*>(&s.d[p][wi][u][2 * turned<V>(u, (q + j) / 2)]);
              dt[j] = d.x;
              dt[j + 1] = d.z;
            }
          }
          ld_vec<V>(&s.g[p][wi][u][q], dyg);
          ld_vec<V>(&s.sums[p][1][wi][u][q], gB);
          ld_vec<V>(&s.sums[p][2][wi][u][q], qA);
          ld_vec<V>(&s.slope[p][wi][u][q], sl);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            dx[j] = gB[j] * dt[j] + skip[j] * dyg[j];
            dd[j] = (gB[j] * x[j] + qA[j] * (1.f / ATLAS_LOG2E)) * sl[j];
            dD[j] += dyg[j] * x[j];
            db[j] += dd[j];
          }
          if (a.z) {
            float ch[V];
            ld_vec<V>(&s.dz[p][wi][u][q], dz);
            ld_vec<V>(&s.sums[p][0][wi][u][q], ch);
#pragma unroll
            for (int j = 0; j < V; ++j) dz[j] *= ch[j] + skip[j] * x[j];
          }
          Pack<T, V> o;
          o.pack(dx);
          st_pack<T, V>(ox.at(i), o);
          o.pack(dd);
          st_pack<T, V>(od.at(i), o);
          if (a.z) {
            o.pack(dz);
            st_pack<T, V>(oz.at(i), o);
          }
        }
        ox.back(), od.back(), oz.back();
        for (int i = wi * kThreads + lane; i < kSub * 2 * P::kNP; i += kWalkers * kThreads) {
          if (i / (2 * P::kNP) >= left) continue;
          float v = 0.f;
#pragma unroll
          for (int r2 = 0; r2 < kWalkers; ++r2) v += (&s.bc[p][r2][0][0])[i];
          pbc[i] = v;
        }
        pbc -= kSub * 2 * P::kNP;
      };
      for (int i = 0; i < 2; ++i) {
        fetch();
        put();
      }
      cp_wait<1>();
      __syncwarp();
      prepare(0);
      __syncthreads();
      for (int m = 0; m < tiles; ++m) {
        fetch();
        if (m > 0) finish((m - 1) & 1, m == 1 ? end - first : kSub);
        cp_wait<1>();
        __syncwarp();
        prepare((m + 1) & 1);
        put();
        __syncthreads();
      }
      cp_wait<0>();
      finish((tiles - 1) & 1, tiles == 1 ? end - first : kSub);
    }
    // a channel's tokens lie in the lanes that share its vector
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
      for (int m = P::kCB / V; m < 32; m *= 2) {
        dD[j] += __shfl_xor_sync(0xFFFFFFFFu, dD[j], m);
        db[j] += __shfl_xor_sync(0xFFFFFFFFu, db[j], m);
      }
      const int ch = lane * V + j;
      if (lane < P::kCB / V && ch < k.n) {
        w.pD[seg * a.D + k.c0 + ch] = dD[j];
        w.pb[seg * a.D + k.c0 + ch] = db[j];
      }
    }
    return;
  }

  const int nl = lane / P::kPairs, n0 = nl * 4, cp = lane % P::kPairs;
  pair32 A01[2], A23[2], g01[2], g23[2], dA01[2], dA23[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = k.c0 + 2 * cp + i;
    float A4[4] = {0.f, 0.f, 0.f, 0.f}, h4[4] = {0.f, 0.f, 0.f, 0.f}, g4[4] = {0.f, 0.f, 0.f, 0.f};
    if (some && 2 * cp + i < k.n) {
      ld_states4(a.A + (long)c * a.N, n0, a.N, A4);
      if (w.split) {
        ld_states4(w.seg_h + (seg * a.D + c) * a.N, n0, a.N, h4);
        ld_states4(w.seg_g + (seg * a.D + c) * a.N, n0, a.N, g4);
      } else if (a.dh) {
        ld_states4(a.dh + ((long)t.b * a.D + c) * a.N, n0, a.N, g4);
      }
    }
    A01[i] = pair(log2_decay(A4[0]), log2_decay(A4[1]));
    A23[i] = pair(log2_decay(A4[2]), log2_decay(A4[3]));
    // read by this lane alone
    *reinterpret_cast<float4*>(s.hs[wi][i][lane]) = make_float4(h4[0], h4[1], h4[2], h4[3]);
    g01[i] = pair(g4[0], g4[1]);
    g23[i] = pair(g4[2], g4[3]);
    dA01[i] = dA23[i] = pair(0.f, 0.f);
  }
  if (tiles > 0) __syncthreads();
  for (int m = 0; m < tiles; ++m) {
    const int p = m & 1;
    pair32 h01[2][kSub + 1], h23[2][kSub + 1];  // states in front of each token
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Raw& r = s.raw[m % kBackRing];
      const ulonglong2 h = *reinterpret_cast<const ulonglong2*>(r.h[wi][i][lane]);
      h01[i][0] = h.x;
      h23[i][0] = h.y;
      if (w.split) {
        const ulonglong2 hs = *reinterpret_cast<const ulonglong2*>(s.hs[wi][i][lane]);
        const float cum = r.cum[wi][2 * cp + i];
        const pair32 cc = pair(cum, cum);
        h01[i][0] = pair_fma(pair_ex2(pair_mul(cc, A01[i])), hs.x, h.x);
        h23[i][0] = pair_fma(pair_ex2(pair_mul(cc, A23[i])), hs.y, h.y);
      }
    }
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
      const float4 d = *reinterpret_cast<const float4*>(&s.d[p][wi][u][2 * turned<V>(u, cp)]);
      const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&s.B[p][u][n0]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float dt = i ? d.z : d.x, gx = i ? d.w : d.y;
        const pair32 dd = pair(dt, dt), gg = pair(gx, gx);
        h01[i][u + 1] = pair_fma(pair_ex2(pair_mul(dd, A01[i])), h01[i][u], pair_mul(gg, b.x));
        h23[i][u + 1] = pair_fma(pair_ex2(pair_mul(dd, A23[i])), h23[i][u], pair_mul(gg, b.y));
      }
    }
#pragma unroll
    for (int u0 = kSub - 4; u0 >= 0; u0 -= 4) {
      float ry[8], rs[8], rq[8];  // four tokens x two channels
#pragma unroll
      for (int uu = 3; uu >= 0; --uu) {
        const int u = u0 + uu;
        const float4 d = *reinterpret_cast<const float4*>(&s.d[p][wi][u][2 * turned<V>(u, cp)]);
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&s.B[p][u][n0]);
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&s.C[p][u][n0]);
        const float2 dy = *reinterpret_cast<const float2*>(&s.g[p][wi][u][2 * cp]);
        pair32 mB01, mB23, mC01, mC23;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float dt = i ? d.z : d.x, gx = i ? d.w : d.y, y = i ? dy.y : dy.x;
          const pair32 dd = pair(dt, dt), gg = pair(gx, gx), yy = pair(y, y);
          const pair32 e01 = pair_ex2_again(pair_mul(dd, A01[i])), e23 = pair_ex2_again(pair_mul(dd, A23[i]));
          const pair32 G01 = pair_fma(q.x, yy, g01[i]), G23 = pair_fma(q.y, yy, g23[i]);  // dL/dh_t
          const pair32 H01 = h01[i][u + 1], H23 = h23[i][u + 1];
          ry[2 * uu + i] = pair_sum(pair_fma(H23, q.y, pair_mul(H01, q.x)));
          rs[2 * uu + i] = pair_sum(pair_fma(G23, b.y, pair_mul(G01, b.x)));
          g01[i] = pair_mul(e01, G01);
          g23[i] = pair_mul(e23, G23);
          const pair32 q01 = pair_mul(g01[i], h01[i][u]), q23 = pair_mul(g23[i], h23[i][u]);
          rq[2 * uu + i] = pair_sum(pair_fma(q23, A23[i], pair_mul(q01, A01[i])));
          dA01[i] = pair_fma(q01, dd, dA01[i]);
          dA23[i] = pair_fma(q23, dd, dA23[i]);
          mB01 = i ? pair_fma(G01, gg, mB01) : pair_mul(G01, gg);
          mB23 = i ? pair_fma(G23, gg, mB23) : pair_mul(G23, gg);
          mC01 = i ? pair_fma(H01, yy, mC01) : pair_mul(H01, yy);
          mC23 = i ? pair_fma(H23, yy, mC23) : pair_mul(H23, yy);
        }
        float v[8];
        unpair(mB01, v[0], v[1]);
        unpair(mB23, v[2], v[3]);
        unpair(mC01, v[4], v[5]);
        unpair(mC23, v[6], v[7]);
        lane_sums<8, P::kPairs, 1>(v, lane);
        constexpr int M = P::kPairs <= 8 ? 8 / P::kPairs : 1, E = P::kPairs > 8 ? P::kPairs / 8 : 1;
        if (cp % E == 0) {
#pragma unroll
          for (int i = 0; i < M; ++i) {
            const int id = cp / E * M + i;
            s.bc[p][wi][u][(id >> 2) * P::kNP + n0 + (id & 3)] = v[i];
          }
        }
      }
      auto put = [&](int which, float* v) {
        lane_sums<8, LN, P::kPairs>(v, lane);
        constexpr int M = LN <= 8 ? 8 / LN : 1, E = LN > 8 ? LN / 8 : 1;  // (token, channel) order
        if (nl % E == 0) {
          if constexpr (M >= 2) {
#pragma unroll
            for (int i = 0; i < M; i += 2)
              *reinterpret_cast<float2*>(&s.sums[p][which][wi][u0 + (nl * M + i) / 2][2 * cp]) =
                  make_float2(v[i], v[i + 1]);
          } else {
            s.sums[p][which][wi][u0 + nl / E / 2][2 * cp + nl / E % 2] = v[0];
          }
        }
      };
      if (a.z) put(0, ry);
      put(1, rs);
      put(2, rq);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = k.c0 + 2 * cp + i;
    if (2 * cp + i >= k.n) continue;
    float v[4];
    unpair(dA01[i], v[0], v[1]);
    unpair(dA23[i], v[2], v[3]);
    st_states4(w.pA + (seg * a.D + c) * a.N, n0, a.N, v);
    if (some && !w.split && a.dh) {
      unpair(g01[i], v[0], v[1]);
      unpair(g23[i], v[2], v[3]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = t.carry ? v[j] : 0.f;
      st_states4(a.dh + ((long)t.b * a.D + c) * a.N, n0, a.N, v);
    }
  }
}

// Adds the partial sums: the first `nbc` blocks dB and dC, the others dA, dD and ddt_bias.
template <typename T, int LN>
__global__ void __launch_bounds__(256) finish_kernel(ScanArgs a, Back<LN> w, int nbc) {
  constexpr int NP = Shape<LN>::kNP;
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
#pragma unroll 8
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
#pragma unroll 8
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

template <typename T, int V, int LN, bool NV>
bool back_pass(const ScanArgs& a, const Back<LN>& w, cudaStream_t st) {
  constexpr size_t smem = sizeof(BackShared<T, LN>);
  auto* f = back_kernel<T, V, LN, NV>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return false;
  f<<<dim3((unsigned)w.segs, w.cb), kBackThreads, smem, st>>>(a, w);
  return true;
}

template <typename T, int V, int LN>
int backward(const ScanArgs& a, cudaStream_t st) {
  // four channels a vector: a tile of kSub tokens then has one for every lane
  constexpr int V4 = V > 4 ? 4 : V, VV = V4 < Shape<LN>::kCB ? V4 : Shape<LN>::kCB;
  const Back<LN> w(a, a.ws);
  const int by = blocks_over<Shape<LN>::kCB>(a);
  if (by > 65535 || a.s.B > 65535 || w.segs > 0x7FFFFFFFL) return ATLAS_ERR_UNSUPPORTED;
  if (w.segs > 0) {
    Segments sg = w.segments();
    find_rising<T>(a, sg, st);
    if (!segment_pass<T, V, LN, kKeep>(a, sg, st)) return ATLAS_ERR_CUDA;
    if (w.split)
      join_back_kernel<LN><<<dim3((unsigned)(((long)a.D * a.N + 255) / 256), a.s.B), 256, 0, st>>>(a, w);
    if (!(a.wide_n ? back_pass<T, VV, LN, true>(a, w, st) : back_pass<T, VV, LN, false>(a, w, st)))
      return ATLAS_ERR_CUDA;
  }
  const long nb = (w.rows * a.G * 2 * Shape<LN>::kNP + 255) / 256;
  const int nbc = (int)(nb < kSMs * 16 ? nb : kSMs * 16);
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
