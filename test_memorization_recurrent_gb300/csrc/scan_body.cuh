// scan_body.cuh -- selective state space scan, for one element type (instantiated by
// scan_f32.cu, scan_bf16.cu, scan_f16.cu).
//
//   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = (C_t h_t + D x_t) SiLU(z_t)
//
// A lane holds two channels x four states; the N states of a channel are split over LN lanes,
// whose sums over states are added by halving, four tokens at a time.  A block is two warps.
// The second takes softplus of a tile's dt, once per token and channel, and writes dt, dt x,
// B and C to shared memory while the first walks the tile before, and gates and stores the
// tile before that: one warp alone leaves most issue slots empty.
//
// What bounds it: for 32 updates of a state, one cycle of an SM for their exponentials (32 a
// cycle), 1.04 for what the lanes read from shared memory (four states' B and C and two
// channels' steps for eight updates) and 7.5 instructions; issue comes first.  So arithmetic
// is paired (one slot for two numbers; unpaired: 462 us against 438 at that step), and
// neighbouring lanes share B and C: a load whose lanes agree in pairs takes half the time of
// one whose addresses repeat every four lanes (2.2 against 4.0 cycles for 16 bytes a lane).
// With one channel x four states a lane the shared memory's 3 cycles were the bound.
// 8 x 4096 tokens x 2048 channels x 16 states, bf16, gated: 1793 us for the first kernel of
// one pass with everything in one warp's turn, 584 with a register tile prefetched, 525 with
// the second warp, 438 with the two kinds of warps spread over the schedulers, 343 with the
// second warp's addresses and conversions thinned out and seven blocks an SM: 4.3 times the
// traffic's floor, 3.2 times the exponentials', 65% of the issue slots.
//
// When sequences times channels do not fill the machine, the tokens are split into
// segments: a first pass finds each segment's end state from a zero start (with the sum of
// its dt: the decay over a segment is exp(A sum dt)); the second computes the outputs, each
// segment from the start state that it joins from those in front of it.  Three packed prompts of
// 16384 tokens x 1024 channels: 154 us.
#pragma once
#include "ops_common.cuh"

namespace atlas {
namespace scan {

constexpr int kThreads = 32;  // of each of a block's two warps
constexpr int kTile = 16;     // tokens in shared memory
constexpr int kRing = 5;      // tiles as they lie in memory: one to finish, one with the other
                              // warp, one to prepare, two under way

template <int LN>
struct Shape {
  static constexpr int kNP = 4 * LN;       // padded states
  static constexpr int kPairs = 32 / LN;   // pairs of channels of a block
  static constexpr int kCB = 2 * kPairs;   // its channels
};

// The block's channels: blocks do not cross groups.
struct Channels {
  int c0, n, g;  // first, count, group
};
template <int CB>
__device__ __forceinline__ Channels channels_at(const ScanArgs& a, int by) {
  const int per = a.D / a.G, bpg = (per + CB - 1) / CB;
  Channels k;
  k.g = by / bpg;
  const int at = (by % bpg) * CB;
  k.c0 = k.g * per + at;
  k.n = min(CB, per - at);
  return k;
}
template <int CB>
inline int blocks_over(const ScanArgs& a) {
  const int per = a.D / a.G;
  return a.G * ((per + CB - 1) / CB);
}

// Rows of one tensor from a tile's sequence: row tok at p + tok * st.
template <typename T>
__device__ __forceinline__ const T* rows_of(const void* p, const ScanArgs& a, const SeqTile& t, long sb,
                                            long st, int c) {
  return reinterpret_cast<const T*>(p) + seq_at(a.s, t, 0, sb, st) + c;
}

// A tile of TT tokens x W elements of a warp: vector i * kThreads + lane, the elements of a
// token innermost.  The object walks a tensor's rows from tile to tile.
template <typename T, int V, int W, int TT = kTile>
struct Tile {
  static constexpr int kN = (TT * W / V + kThreads - 1) / kThreads;
  static __device__ __forceinline__ int lane() { return threadIdx.x & 31; }
  static __device__ __forceinline__ int token(int i) { return (i * kThreads + lane()) / (W / V); }
  static __device__ __forceinline__ int channel(int i) { return (i * kThreads + lane()) % (W / V) * V; }
  static __device__ __forceinline__ bool inside(int i) {
    return TT * W / V % kThreads == 0 || i * kThreads + lane() < TT * W / V;
  }
  T* p;      // this lane's first vector of the tile
  long row;  // elements between tokens
  // rows from token t0 on at q
  __device__ __forceinline__ Tile(const T* q, long st, int t0) : row(st) {
    p = const_cast<T*>(q) + (long)(t0 + token(0)) * st + channel(0);
  }
  __device__ __forceinline__ T* at(int i) const {
    if (i == 0) return p;
    return p + (token(i) - token(0)) * row + (channel(i) - channel(0));
  }
  __device__ __forceinline__ void next() { p += TT * row; }
  __device__ __forceinline__ void back() { p -= TT * row; }
  // Asynchronous copies take at least four bytes; smaller elements come through registers,
  // loaded by copy() and stored by put(), with other work in between.
  static constexpr bool kAsync = V * sizeof(T) >= 4;
  T held[kAsync ? 1 : kN];
  // this tile into s; zeros from token `left` on and past element n
  __device__ __forceinline__ void copy(T (*s)[W], int left, int n) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      if (!inside(i)) continue;
      const int u = token(i), c = channel(i);
      const bool some = u < left && c < n;
      if constexpr (kAsync) {
        cp_async<V * sizeof(T)>(&s[u][c], some ? at(i) : p, some);
      } else {
        held[i] = some ? *at(i) : from_f<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ void put(T (*s)[W]) {
    if constexpr (!kAsync) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (inside(i)) s[token(i)][channel(i)] = held[i];
    }
  }
};

// V raw steps of channels c .. c + V to dt.
template <typename T, int V>
__device__ __forceinline__ void steps_of(const ScanArgs& a, const Pack<T, V>& raw, const float* bias, float* d) {
  raw.unpack(d);
#pragma unroll
  for (int j = 0; j < V; ++j) d[j] += bias[j];
  if (a.softplus) {
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = softplusf(d[j]);
  }
}

// A log2(e): exp(dt A) is 2 to its product with dt.  Held above -infinity, whose product with a step of 0 (as
// places behind a sequence's end have) would not be 0.
__device__ __forceinline__ float log2_decay(float A) {
  const float v = A * ATLAS_LOG2E;
  return v < -3.4e38f ? -3.4e38f : v;
}

// This lane's four states at p (one channel's N states), 0 past N.
__device__ __forceinline__ void ld_states4(const float* p, int n0, int N, float* h) {
  if (N % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    if (n0 < N) {
      const float4 v = *reinterpret_cast<const float4*>(p + n0);
      h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
    } else {
      h[0] = h[1] = h[2] = h[3] = 0.f;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = n0 + i < N ? p[n0 + i] : 0.f;
}
__device__ __forceinline__ void st_states4(float* p, int n0, int N, const float* h) {
  if (N % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    if (n0 < N) *reinterpret_cast<float4*>(p + n0) = make_float4(h[0], h[1], h[2], h[3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n0 + i < N) p[n0 + i] = h[i];
}

// Which of a token's pairs of channels lies at place p of its row: a thread stores V
// neighbouring channels, so the places are turned by the token and the threads of a store
// fall on different banks, as the pairs of a load do.
template <int V>
__device__ __forceinline__ int turned(int u, int p) {
  return V > 2 ? p ^ (u & (V / 2 - 1)) : p;
}

// What a walk over a segment is for: kOut, its outputs (kJoin: with several segments a sequence,
// a kernel of its own, whose start would cost kOut's loop registers); kEnds, its end state from a zero
// start; kKeep, for the backward pass: the state in front of every kSub tokens too, and what
// the segment's own tokens add to the adjoint in front of it.
enum Mode { kOut, kEnds, kKeep, kJoin };
constexpr int kSub = 8;

// Shared memory of segment_kernel.
template <typename T, int LN, Mode MODE>
struct SegmentShared {
  static constexpr bool ENDS = MODE == kEnds;
  using P = Shape<LN>;
  static constexpr int kOther = ENDS ? 1 : kTile;  // what the outputs alone need
  struct Raw {
    alignas(16) T x[kTile][P::kCB];
    alignas(16) T dt[kTile][P::kCB];
    alignas(16) T z[kOther][P::kCB];
    alignas(16) T B[kTile][P::kNP];
    alignas(16) T C[kOther][P::kNP];
    alignas(16) T dy[MODE == kKeep ? 1 : 0][kTile][P::kCB];
  };
  alignas(16) float2 d[2][kTile][P::kCB];  // dt, dt x
  alignas(16) float B[2][kTile][P::kNP];
  alignas(16) float C[2][kOther][P::kNP];
  alignas(16) float y[2][kOther][P::kCB + 8];  // the sums over states; kKeep: dy SiLU(z)
  Raw raw[kRing];
  int swap;
};

// Kept states lie by row, a place every kSub tokens of a sequence: a packed one's from start[b] / kSub + b
// on, L / kSub + B places in all however short the sequences are.
inline __host__ __device__ int kept_each(const SeqArgs& a) { return a.L / kSub + (a.L % kSub != 0); }
inline long kept_places(const SeqArgs& a) { return a.start ? (long)a.L / kSub + a.B : (long)a.B * kept_each(a); }
__device__ __forceinline__ long kept_at(const SeqArgs& a, const SeqTile& t) {  // of the token t.t0, a multiple of kSub
  return (a.start ? (long)t.first / kSub + t.b : (long)t.b * kept_each(a)) + t.t0 / kSub;
}

// Where the segments' states go: h and dt of kEnds and kKeep (kJoin reads them), the
// rest of kKeep.
struct Segments {
  int S;                          // tokens of a segment
  float *h, *dt;                  // [segments][D][N], [segments][D]
  float *g, *keep_h, *keep_dt;    // [segments][D][N], [places][D][N], [places][D]
  int* rising;                    // how many sequences count, for the kernels behind the one that finds it
  int known;                      // whether it is there already
};

// kOut starts from the sequence's state, kJoin from the segments in front, seg.h.  kEnds starts a sequence's first segment from its state, which the last
// segment's place receives too (kJoin may be overwriting it with the final one), and leaves the
// last segment out.  kKeep with seg.h starts from zeros, else from the
// sequence's state, and then leaves the adjoint out.  NV: B and C are copied in vectors too.
template <typename T, int V, int LN, Mode MODE, bool NV>
__global__ void __launch_bounds__(2 * kThreads, 7) segment_kernel(ScanArgs a, Segments sg) {
  constexpr bool ENDS = MODE == kEnds, KEEP = MODE == kKeep, JOIN = MODE == kJoin, OUT = MODE == kOut || JOIN;
  using P = Shape<LN>;
  using X = Tile<T, V, P::kCB>;
  constexpr int VN = !NV ? 1 : 16 / sizeof(T) < P::kNP ? 16 / sizeof(T) : P::kNP;
  using R = Tile<T, VN, P::kNP>;
  using Shared = SegmentShared<T, LN, MODE>;
  using Raw = typename Shared::Raw;
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *reinterpret_cast<Shared*>(smem);
  if (blockIdx.x == 0 && blockIdx.y == 0) seq_check(a.s, threadIdx.x, 2 * kThreads);
  const long seg = blockIdx.x;
  const int rising = !a.s.start ? a.s.B : sg.known ? *sg.rising : seq_rising(a.s);
  if ((ENDS || KEEP) && !sg.known && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *sg.rising = rising;
  SeqTile t;
  if (!seq_tile(a.s, rising, seg, sg.S, t)) return;
  const int end = seq_tile_end(t, sg.S);
  if (ENDS && end == t.len) return;  // (the last segment, or the only one)
  const Channels k = channels_at<P::kCB>(a, blockIdx.y);
  const int tiles = (end - t.t0 + kTile - 1) / kTile;
  const int lane = threadIdx.x & 31;
  // A warp stays on one of the four schedulers, by its number modulo 4; the two kinds of warps take
  // turns, so that each scheduler gets the exponentials of some blocks (without: 1.3 times the time).
  if (threadIdx.x == 0) {
    unsigned w;
    asm volatile("mov.u32 %0, %%warpid;" : "=r"(w));
    s.swap = (w >> 2) & 1;
  }
  __syncthreads();

  if ((threadIdx.x >= kThreads) != (s.swap != 0)) {  // the warp that prepares and finishes tiles
    X px(rows_of<T>(a.x, a, t, a.xb, a.xt, k.c0), a.xt, t.t0);
    X pd(rows_of<T>(a.dt, a, t, a.tb, a.tt, k.c0), a.tt, t.t0);
    X pz(rows_of<T>(a.z ? a.z : a.x, a, t, a.zb, a.zt, k.c0), a.zt, t.t0);
    X py(rows_of<T>(OUT ? a.y : a.x, a, t, a.yb, a.yt, k.c0), a.yt, t.t0);
    X pg(rows_of<T>(KEEP ? a.dy : a.x, a, t, a.yb, a.yt, k.c0), a.yt, t.t0);
    R pB(rows_of<T>(a.Bm, a, t, a.bb, a.bt, k.g * a.N), a.bt, t.t0);
    R pC(rows_of<T>(ENDS ? a.Bm : a.Cm, a, t, a.cb, a.ct, k.g * a.N), a.ct, t.t0);
    // a thread's vectors keep their channels from tile to tile
    static_assert(kThreads % (P::kCB / V) == 0, "a thread's vectors share their channels");
    float bias[V], skip[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int ch = X::channel(0) + j;
      bias[j] = a.bias && ch < k.n ? a.bias[k.c0 + ch] : 0.f;
      skip[j] = OUT && a.Dk && ch < k.n ? a.Dk[k.c0 + ch] : 0.f;
    }
    int rf = 0, rp = 0, rn = 0;  // places in the ring to fetch, prepare and finish next
    const auto step = [](int& r) { r = r + 1 == kRing ? 0 : r + 1; };
    int left_f = end - t.t0, left_p = left_f, left_n = left_f;  // tokens from there on
    auto fetch = [&]() {
      if (left_f > 0) {
        Raw& r = s.raw[rf];
        px.copy(r.x, left_f, k.n);
        pd.copy(r.dt, left_f, k.n);
        pB.copy(r.B, left_f, a.N);
        px.next(), pd.next(), pB.next();
        if (!ENDS) {
          if (a.z) pz.copy(r.z, left_f, k.n);
          pC.copy(r.C, left_f, a.N);
          pz.next(), pC.next();
        }
        if (KEEP) {
          pg.copy(r.dy[0], left_f, k.n);
          pg.next();
        }
      }
      cp_commit();
    };
    auto put = [&]() {
      if (left_f > 0) {
        Raw& r = s.raw[rf];
        px.put(r.x);
        pd.put(r.dt);
        pB.put(r.B);
        if (!ENDS) {
          if (a.z) pz.put(r.z);
          pC.put(r.C);
        }
        if (KEEP) pg.put(r.dy[0]);
      }
      left_f -= kTile;
      step(rf);
    };
    auto prepare = [&](int p) {
      const int left = left_p;
      if (left <= 0) return;
      const Raw& r = s.raw[rp];
      left_p -= kTile;
      step(rp);
#pragma unroll
      for (int i = 0; i < X::kN; ++i)
        if (X::inside(i)) {
          const int u = X::token(i), q = X::channel(i);
          float d[V], g[V];
          ld_pack<T, V>(&r.x[u][q]).unpack(g);
          steps_of<T, V>(a, ld_pack<T, V>(&r.dt[u][q]), bias, d);
          if (left < kTile) {  // past the end the state stays
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = u < left ? d[j] : 0.f;
          }
#pragma unroll
          for (int j = 0; j < V; ++j) g[j] *= d[j];
          if (V == 1) {
            s.d[p][u][q] = make_float2(d[0], g[0]);
          } else {
#pragma unroll
            for (int j = 0; j + 1 < V; j += 2)
              *reinterpret_cast<float4*>(&s.d[p][u][2 * turned<V>(u, (q + j) / 2)]) =
                  make_float4(d[j], g[j], d[j + 1], g[j + 1]);
          }
        }
      if (KEEP) {
#pragma unroll
        for (int i = 0; i < X::kN; ++i)
          if (X::inside(i)) {
            const int u = X::token(i), q = X::channel(i);
            float y[V], z[V];
            ld_pack<T, V>(&r.dy[0][u][q]).unpack(y);
            if (a.z) {
              ld_pack<T, V>(&r.z[u][q]).unpack(z);
#pragma unroll
              for (int j = 0; j < V; ++j) y[j] *= siluf(z[j]);
            }
            if (left < kTile) {
#pragma unroll
              for (int j = 0; j < V; ++j) y[j] = u < left ? y[j] : 0.f;
            }
            st_vec<V>(&s.y[p][u][q], y);
          }
      }
#pragma unroll
      for (int i = lane; i < kTile * P::kNP / 4; i += kThreads) {
        const int u = i / (P::kNP / 4), n = i % (P::kNP / 4) * 4;
        float b[4];
        ld_pack<T, 4>(&r.B[u][n]).unpack(b);
        *reinterpret_cast<float4*>(&s.B[p][u][n]) = make_float4(b[0], b[1], b[2], b[3]);
        if (!ENDS) {
          ld_pack<T, 4>(&r.C[u][n]).unpack(b);
          *reinterpret_cast<float4*>(&s.C[p][u][n]) = make_float4(b[0], b[1], b[2], b[3]);
        }
      }
    };
    auto finish = [&](int p) {
      if (!OUT) return;
      const Raw& r = s.raw[rn];
#pragma unroll
      for (int i = 0; i < X::kN; ++i) {
        const int u = X::token(i), q = X::channel(i);
        if (!X::inside(i) || u >= left_n || q >= k.n) continue;
        float y[V], z[V];
        ld_pack<T, V>(&r.x[u][q]).unpack(y);
        ld_vec<V>(&s.y[p][u][q], z);
#pragma unroll
        for (int j = 0; j < V; ++j) y[j] = fmaf(skip[j], y[j], z[j]);
        if (a.z) {
          ld_pack<T, V>(&r.z[u][q]).unpack(z);
#pragma unroll
          for (int j = 0; j < V; ++j) y[j] *= siluf(z[j]);
        }
        Pack<T, V> o;
        o.pack(y);
        st_pack<T, V>(py.at(i), o);
      }
      py.next();
      left_n -= kTile;
      step(rn);
    };
    for (int i = 0; i < 3; ++i) {
      fetch();
      put();
    }
    cp_wait<2>();
    __syncwarp();
    prepare(0);
    __syncthreads();
    for (int m = 0; m < tiles; ++m) {
      fetch();
      if (m > 0) finish((m - 1) & 1);
      cp_wait<2>();
      __syncwarp();
      prepare((m + 1) & 1);
      put();
      __syncthreads();
    }
    cp_wait<0>();
    if (tiles > 0) finish((tiles - 1) & 1);
    return;
  }

  const int nl = lane / P::kPairs, n0 = nl * 4, cp = lane % P::kPairs;
  pair32 A01[2], A23[2], h01[2], h23[2];
  pair32 p01[2], p23[2], g01[2], g23[2];  // kKeep: the decay so far, the adjoint
  float h4[4], sum[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    p01[i] = p23[i] = pair(1.f, 1.f);
    g01[i] = g23[i] = pair(0.f, 0.f);
    const int c = k.c0 + 2 * cp + i;
    float A4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) h4[j] = 0.f;
    if (2 * cp + i < k.n) {
      ld_states4(a.A + (long)c * a.N, n0, a.N, A4);
      const long first = seg - t.t0 / sg.S, last = first + seq_tiles_of(t.len, sg.S) - 1;
      if (JOIN && last > first) {
        // the sequence's state, then the segments in front, four under way at a time
        if (seg == first) {
          ld_states4(sg.h + (last * a.D + c) * a.N, n0, a.N, h4);
        } else {
#pragma unroll 1
          for (long q0 = first; q0 < seg; q0 += 4) {
            float own[4][4], d[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              d[q] = 0.f;
              own[q][0] = own[q][1] = own[q][2] = own[q][3] = 0.f;
              if (q0 + q < seg) {
                ld_states4(sg.h + ((q0 + q) * a.D + c) * a.N, n0, a.N, own[q]);
                d[q] = sg.dt[(q0 + q) * a.D + c];
              }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                h4[j] = ex2(log2_decay(A4[j]) * d[q]) * h4[j] + own[q][j];
          }
        }
      } else if (!KEEP && (!ENDS || seg == first) && a.h_in && t.carry) {
        ld_states4(a.h_in + ((long)t.slot * a.D + c) * a.N, n0, a.N, h4);
      } else if (KEEP && !sg.h && a.h_in && t.carry) {
        ld_states4(a.h_in + ((long)t.slot * a.D + c) * a.N, n0, a.N, h4);
      }
      if (ENDS && seg == first) st_states4(sg.h + (last * a.D + c) * a.N, n0, a.N, h4);
    }
    A01[i] = pair(log2_decay(A4[0]), log2_decay(A4[1]));
    A23[i] = pair(log2_decay(A4[2]), log2_decay(A4[3]));
    h01[i] = pair(h4[0], h4[1]);
    h23[i] = pair(h4[2], h4[3]);
  }
  // the operands of G tokens; those of the next G are loaded before the current ones are used,
  // and the sums over states of the last G taken among the products of the current ones
  constexpr int G = OUT ? 4 : 2;
  struct Few {
    float4 d[G];
    ulonglong2 b[G], q[G];
    float2 y[G];
  };
  // kKeep: the states in front of the next token, and the sum of dt so far
  long kept = KEEP ? kept_at(a.s, t) * a.D + k.c0 + 2 * cp : 0;
  auto keep = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (2 * cp + i >= k.n) continue;
      unpair(h01[i], h4[0], h4[1]);
      unpair(h23[i], h4[2], h4[3]);
      st_states4(sg.keep_h + (kept + i) * a.N, n0, a.N, h4);
      if (nl == 0) sg.keep_dt[kept + i] = sum[i];
    }
    kept += a.D;
  };
  __syncthreads();
  for (int m = 0; m < tiles; ++m) {
    const int p = m & 1;
    auto load = [&](int u0) {
      Few f;
#pragma unroll
      for (int u = 0; u < G; ++u) {
        f.d[u] = *reinterpret_cast<const float4*>(&s.d[p][u0 + u][2 * turned<V>(u0 + u, cp)]);
        f.b[u] = *reinterpret_cast<const ulonglong2*>(&s.B[p][u0 + u][n0]);
        if (!ENDS) f.q[u] = *reinterpret_cast<const ulonglong2*>(&s.C[p][u0 + u][n0]);
        if (KEEP) f.y[u] = *reinterpret_cast<const float2*>(&s.y[p][u0 + u][2 * cp]);
      }
      return f;
    };
    auto reduce = [&](int u0, float* yp) {
      lane_sums<8, LN, P::kPairs>(yp, lane);
      constexpr int M = LN <= 4 ? 8 / LN : LN == 8 ? 1 : 0;  // values left, in (token, channel) order
      if (M >= 2) {
#pragma unroll
        for (int i = 0; i < M; i += 2)
          *reinterpret_cast<float2*>(&s.y[p][u0 + (nl * M + i) / 2][2 * cp]) = make_float2(yp[i], yp[i + 1]);
      } else if (M == 1) {
        s.y[p][u0 + nl / 2][2 * cp + nl % 2] = yp[0];
      } else if (nl % (LN > 8 ? LN / 8 : 1) == 0) {
        const int v = nl / (LN > 8 ? LN / 8 : 1);
        s.y[p][u0 + v / 2][2 * cp + v % 2] = yp[0];
      }
    };
    Few f = load(0);
    float last[8];
#pragma unroll
    for (int u0 = 0; u0 < kTile; u0 += G) {
      Few next;
      if (u0 + G < kTile) next = load(u0 + G);
      if (KEEP && u0 % kSub == 0 && m * kTile + u0 < end - t.t0) keep();
      float yp[8];  // four tokens x two channels
#pragma unroll
      for (int u = 0; u < G; ++u) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float dt = i ? f.d[u].z : f.d[u].x, g = i ? f.d[u].w : f.d[u].y;
          const pair32 dd = pair(dt, dt), gg = pair(g, g);
          const pair32 e01 = pair_ex2(pair_mul(dd, A01[i])), e23 = pair_ex2(pair_mul(dd, A23[i]));
          h01[i] = pair_fma(e01, h01[i], pair_mul(gg, f.b[u].x));
          h23[i] = pair_fma(e23, h23[i], pair_mul(gg, f.b[u].y));
          if (!OUT) sum[i] += dt;
          if (KEEP) {
            const float y = i ? f.y[u].y : f.y[u].x;
            const pair32 yy = pair(y, y);
            p01[i] = pair_mul(p01[i], e01);
            p23[i] = pair_mul(p23[i], e23);
            g01[i] = pair_fma(p01[i], pair_mul(yy, f.q[u].x), g01[i]);
            g23[i] = pair_fma(p23[i], pair_mul(yy, f.q[u].y), g23[i]);
          }
          if (OUT) yp[2 * u + i] = pair_sum(pair_fma(h23[i], f.q[u].y, pair_mul(h01[i], f.q[u].x)));
        }
      }
      if (OUT) {
        if (u0 > 0) reduce(u0 - G, last);
#pragma unroll
        for (int i = 0; i < 8; ++i) last[i] = yp[i];
      }
      if (u0 + G < kTile) f = next;
    }
    if (OUT) reduce(kTile - G, last);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = k.c0 + 2 * cp + i;
    if (2 * cp + i >= k.n) continue;
    unpair(h01[i], h4[0], h4[1]);
    unpair(h23[i], h4[2], h4[3]);
    if (!OUT) {
      if (!sg.h) continue;
      st_states4(sg.h + (seg * a.D + c) * a.N, n0, a.N, h4);
      if (nl == 0) sg.dt[seg * a.D + c] = sum[i];
      if (KEEP) {
        unpair(g01[i], h4[0], h4[1]);
        unpair(g23[i], h4[2], h4[3]);
        st_states4(sg.g + (seg * a.D + c) * a.N, n0, a.N, h4);
      }
    } else if (a.h_out && end == t.len) {
      st_states4(a.h_out + ((long)t.slot * a.D + c) * a.N, n0, a.N, h4);
    }
  }
}

// One token a sequence: a lane takes four states of kTokenU channels, loads and stores them
// once.  Bound by the state's traffic, and for few sequences by latency: what does not depend
// on the sequence's slot is under way before the slot is looked up.
constexpr int kTokenThreads = 128, kTokenU = 2;
template <typename T, int LN>
__global__ void __launch_bounds__(kTokenThreads) token_kernel(ScanArgs a) {
  constexpr int CB = kTokenThreads / LN;  // channels of a block at a time
  const int b = blockIdx.x;
  const int lane = threadIdx.x & 31, nl = lane % LN, n0 = nl * 4;
  const int c0 = blockIdx.y * kTokenU * CB + (int)threadIdx.x / LN;
  float A[kTokenU][4], h[kTokenU][4], B[kTokenU][4], C[kTokenU][4];
  float x[kTokenU], d[kTokenU], z[kTokenU], skip[kTokenU];
#pragma unroll
  for (int i = 0; i < kTokenU; ++i) {
    const int c = c0 + i * CB;
#pragma unroll
    for (int j = 0; j < 4; ++j) A[i][j] = h[i][j] = B[i][j] = C[i][j] = 0.f;
    x[i] = d[i] = z[i] = skip[i] = 0.f;
    if (c >= a.D) continue;
    ld_states4(a.A + (long)c * a.N, n0, a.N, A[i]);
    x[i] = to_f(reinterpret_cast<const T*>(a.x)[b * a.xb + c]);
    d[i] = to_f(reinterpret_cast<const T*>(a.dt)[b * a.tb + c]) + (a.bias ? a.bias[c] : 0.f);
    if (a.z) z[i] = to_f(reinterpret_cast<const T*>(a.z)[b * a.zb + c]);
    if (a.Dk) skip[i] = a.Dk[c];
    const long g = a.G == 1 ? 0 : (long)(c / (a.D / a.G)) * a.N;
    const T* pB = reinterpret_cast<const T*>(a.Bm) + b * a.bb + g;
    const T* pC = reinterpret_cast<const T*>(a.Cm) + b * a.cb + g;
    if (a.wide_n) {
      if (n0 < a.N) {
        ld_pack<T, 4>(pB + n0).unpack(B[i]);
        ld_pack<T, 4>(pC + n0).unpack(C[i]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + j < a.N) B[i][j] = to_f(pB[n0 + j]), C[i][j] = to_f(pC[n0 + j]);
    }
  }
  SeqTile t;
  if (!seq_tile(a.s, a.s.B, b, 1, t)) return;
  if (a.h_in && t.carry) {
#pragma unroll
    for (int i = 0; i < kTokenU; ++i)
      if (c0 + i * CB < a.D) ld_states4(a.h_in + ((long)t.slot * a.D + c0 + i * CB) * a.N, n0, a.N, h[i]);
  }
#pragma unroll
  for (int i = 0; i < kTokenU; ++i) {
    const int c = c0 + i * CB;
    const float dt = a.softplus ? softplusf(d[i]) : d[i];
    float y = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[i][j] = ex2(dt * log2_decay(A[i][j])) * h[i][j] + dt * x[i] * B[i][j];
      y += h[i][j] * C[i][j];
    }
    lane_sums<1, LN, 1>(&y, lane);
    if (c >= a.D) continue;
    if (a.h_out) st_states4(a.h_out + ((long)t.slot * a.D + c) * a.N, n0, a.N, h[i]);
    if (nl == 0) {
      y += skip[i] * x[i];
      if (a.z) y *= siluf(z[i]);
      reinterpret_cast<T*>(a.y)[b * a.yb + c] = from_f<T>(y);
    }
  }
}

// Segment length, 0 for one segment a sequence.  The blocks of an SM share its throughput from
// about two of them on, and a second walk over the tokens costs two thirds of the first: one
// segment from 250 blocks on (4 x 4096 tokens x 1024 channels: 144 us, in segments 150 to 168;
// twice the sequences: 199 against 330).  Below, segments for seven blocks an SM, as many as run
// at once (three packed prompts of 16384 tokens x 1024, at the step that chose it: 170 us with six, 150
// with seven, 183 with eight), but none below 256 tokens.
inline int segment_tokens(const ScanArgs& a, long blocks_per_seq) {
  const long want = kSMs * 7;
  const long rows = a.s.start ? a.s.L : (long)a.s.B * a.s.L;
  if (!a.s.start && a.s.B * blocks_per_seq >= 250) return 0;
  if (a.s.L <= 256) return 0;
  long S = rows * blocks_per_seq / want / kTile * kTile;
  if (S < 256) S = 256;
  if (S >= a.s.L) return 0;
  return (int)S;
}

constexpr size_t kRisingBytes = 16;  // at the workspace's start; a word, the rest for alignment

template <int LN>
size_t workspace(const ScanArgs& a) {
  const int S = segment_tokens(a, blocks_over<Shape<LN>::kCB>(a));
  return S ? kRisingBytes + (size_t)seq_tiles(a.s, S) * a.D * (a.N + 1) * 4 : 0;
}

// How many sequences of a packed batch count, ahead of the first pass when they are many: its blocks
// would each look at all of them (4000 short sequences x 512 channels: 845 us, 678 so).
template <typename T>
__global__ void __launch_bounds__(1024) rising_kernel(SeqArgs a, int* out) {
  const int rising = seq_rising(a);
  if (threadIdx.x == 0) *out = rising;
}
template <typename T>
void find_rising(const ScanArgs& a, Segments& sg, cudaStream_t st) {
  sg.known = a.s.start && a.s.B > 2 * kThreads;
  if (sg.known) rising_kernel<T><<<1, 1024, 0, st>>>(a.s, sg.rising);
}

template <typename T, int V, int LN, Mode MODE, bool NV>
bool segment_pass(const ScanArgs& a, const Segments& sg, cudaStream_t st) {
  const dim3 grid((unsigned)seq_tiles(a.s, sg.S), blocks_over<Shape<LN>::kCB>(a));
  constexpr size_t smem = sizeof(SegmentShared<T, LN, MODE>);
  auto* f = segment_kernel<T, V, LN, MODE, NV>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return false;
  f<<<grid, 2 * kThreads, smem, st>>>(a, sg);
  return true;
}
template <typename T, int V, int LN, Mode MODE>
bool segment_pass(const ScanArgs& a, const Segments& sg, cudaStream_t st) {
  constexpr int VV = V < Shape<LN>::kCB ? V : Shape<LN>::kCB;
  return a.wide_n ? segment_pass<T, VV, LN, MODE, true>(a, sg, st)
                  : segment_pass<T, VV, LN, MODE, false>(a, sg, st);
}

template <typename T, int V, int LN>
int forward(const ScanArgs& a, cudaStream_t st) {
  const int by = blocks_over<Shape<LN>::kCB>(a);
  if (by > 65535) return ATLAS_ERR_UNSUPPORTED;
  if (!a.s.start && a.s.L == 1) {
    const long rows = ((long)a.D * LN + kTokenThreads * kTokenU - 1) / (kTokenThreads * kTokenU);
    if (rows > 65535) return ATLAS_ERR_UNSUPPORTED;
    token_kernel<T, LN><<<dim3(a.s.B, (unsigned)rows), kTokenThreads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
  }
  Segments sg = {};
  sg.S = segment_tokens(a, by);
  if (sg.S) {
    sg.rising = reinterpret_cast<int*>(a.ws);
    sg.h = reinterpret_cast<float*>(a.ws) + kRisingBytes / 4;
    sg.dt = sg.h + (size_t)seq_tiles(a.s, sg.S) * a.D * a.N;
    find_rising<T>(a, sg, st);
    if (!segment_pass<T, V, LN, kEnds>(a, sg, st)) return ATLAS_ERR_CUDA;
    sg.known = 1;
    if (!segment_pass<T, V, LN, kJoin>(a, sg, st)) return ATLAS_ERR_CUDA;
  } else {
    sg.S = a.s.L > 0 ? a.s.L : 1;
    if (!segment_pass<T, V, LN, kOut>(a, sg, st)) return ATLAS_ERR_CUDA;
  }
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
