// conv_body.cuh -- short causal convolution per channel and its backward pass, for one
// element type (instantiated by conv_f32.cu, conv_bf16.cu, conv_f16.cu).
//
//   p_t = b + sum_k w_k x_{t-W+1+k},  y_t = SiLU(p_t) or p_t
//   dp_t = dy_t SiLU'(p_t),  dx_s = sum_i w_{W-1-i} dp_{s+i},  dw_k = sum_t dp_t x_{t-W+1+k}
//
// Bound by memory: x (and dy) are read once and y (dx) written once.  A lane owns V adjacent
// channels and walks the tokens of its worker's pieces of the sequences with the last W - 1 inputs in
// registers, so that only the tokens in front of a piece (and, backward, those behind it) are read
// twice.  Workers have equal shares of the rows: 65536 rows x 2048 channels take 102 us in eight
// sequences, 104 in 256 equal ones, 105 with half of the rows in one of 256 (backward 176, 186, 187; with
// tiles of a length that went by the number of sequences 6385 and 6223 us for the last).  V is
// four: with eight, the taps, window and loads of a lane take 202 registers, and too few
// warps are left to cover the latency.  8 x 4096 tokens x 2048 channels of bf16, four taps:
// 126 us with eight, 59 with four, 53 (5.0 TB/s) without a second way to store, which spilled; 24
// warps an SM, against 91 us with 20, 65 with 28, 78 with 32 where 24 took 59.  Backward: 99 us (4.1
// TB/s; 672 with loads in the worker's turn, 150 with the ring but the edges' conditions at every token).
#pragma once
#include "ops_common.cuh"

namespace atlas {
namespace conv {

constexpr int kLanes = 32;  // channel vectors of a warp
constexpr int kWarps = 4;   // workers of a block

__device__ __forceinline__ long worker() { return (long)blockIdx.x * kWarps + threadIdx.y; }

// Offset of channel c of token tok in y's layout.
__device__ __forceinline__ long y_at(const ConvArgs& a, const SeqTile& t, int tok, int c) {
  const long o = seq_at(a.s, t, tok, a.yb, a.yt);
  return a.hd ? o + (long)(c / a.hd) * a.yh + c % a.hd : o + c;
}

// V channels as pairs (V = 1: one pair with an idle half).
template <int V>
constexpr int kPairs = V > 1 ? V / 2 : 1;

template <typename T, int V>
__device__ __forceinline__ void to_pairs(const Pack<T, V>& p, pair32* v) {
  float f[V > 1 ? V : 2] = {};
  p.unpack(f);
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) v[i] = pair(f[2 * i], f[2 * i + 1]);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> from_pairs(const pair32* v) {
  float f[V > 1 ? V : 2];
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) unpair(v[i], f[2 * i], f[2 * i + 1]);
  Pack<T, V> p;
  p.pack(f);
  return p;
}

// Taps and bias of V channels: the V x W taps are neighbours in memory.
template <typename WT, int V, int W>
__device__ __forceinline__ void load_taps_as(const ConvArgs& a, int c, pair32 (*w)[kPairs<V>], pair32* b) {
  float f[W * V + 1], g[V + 1];
#pragma unroll
  for (int i = 0; i < V; ++i) g[i] = 0.f;
  f[W * V] = g[V] = 0.f;
  const WT* p = reinterpret_cast<const WT*>(a.w) + (long)c * W;
  const WT* q = reinterpret_cast<const WT*>(a.bias) + c;
  if (c >= a.C) {
#pragma unroll
    for (int i = 0; i < W * V; ++i) f[i] = 0.f;
  } else if (V == 4 && (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(WT) - 1)) == 0) {
#pragma unroll
    for (int i = 0; i < W * V; i += 4) ld_pack<WT, 4>(p + i).unpack(f + i);
  } else {
#pragma unroll
    for (int i = 0; i < W * V; ++i) f[i] = to_f(p[i]);
  }
  if (a.bias && c < a.C) {
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = to_f(q[i]);
  }
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = pair(f[2 * i * W + k], V > 1 ? f[(2 * i + (V > 1)) * W + k] : 0.f);
    b[i] = pair(g[2 * i], V > 1 ? g[2 * i + (V > 1)] : 0.f);
  }
}
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvArgs& a, int c, pair32 (*w)[kPairs<V>], pair32* b) {
  if (a.wt == ATLAS_BF16)
    load_taps_as<__nv_bfloat16, V, W>(a, c, w, b);
  else if (a.wt == ATLAS_F16)
    load_taps_as<__half, V, W>(a, c, w, b);
  else
    load_taps_as<float, V, W>(a, c, w, b);
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kLanes * kWarps, W <= 4 ? 6 : 4) forward_kernel(ConvArgs a, long share) {
  constexpr int H = W - 1, N = kPairs<V>;
  const int lane = threadIdx.x, c = (blockIdx.y * kLanes + lane) * V;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    seq_check(a.s, threadIdx.y * kLanes + lane, kLanes * kWarps);
  pair32 w[W][N], b[N], win[W][N];
  load_taps<V, W>(a, c, w, b);
  SeqWalk walk = seq_walk(a.s, seq_rising(a.s), worker(), share);
  SeqTile t;
  int t1;
  while (seq_piece(a.s, walk, worker(), share, t, t1)) {
    if (c >= a.C) continue;
    const T* x = reinterpret_cast<const T*>(a.x) + seq_at(a.s, t, 0, a.xb, a.xt) + c;
    T* y = reinterpret_cast<T*>(a.y) + y_at(a, t, 0, c);
#pragma unroll
    for (int k = 0; k < H; ++k) {  // the last H inputs before the piece
      const int tok = t.t0 - H + k;
      Pack<T, V> v;
      if (tok >= 0)
        v = ld_pack<T, V>(x + (long)tok * a.xt);
      else if (a.st_in && t.carry)  // t0 == 0: a later piece begins kLead rows or more into its sequence
        v = ld_pack<T, V>(reinterpret_cast<const T*>(a.st_in) + ((long)t.slot * H + k) * a.C + c);
      else
        v.zero();
      to_pairs<T, V>(v, win[k]);
    }
    // the first piece alone reads the state, so it also writes the new one (the buffers may
    // be the same): the last H of (state, inputs)
    if (a.st_out && t.t0 == 0) {
      const T* s0 = a.st_in && t.carry ? reinterpret_cast<const T*>(a.st_in) + (long)t.slot * H * a.C + c : nullptr;
      T* o = reinterpret_cast<T*>(a.st_out) + (long)t.slot * H * a.C + c;
      Pack<T, V> v[W];
#pragma unroll
      for (int k = 0; k < H; ++k) {
        const int tok = t.len - H + k;
        if (tok >= 0)
          v[k] = ld_pack<T, V>(x + (long)tok * a.xt);
        else if (s0)
          v[k] = ld_pack<T, V>(s0 + (long)(tok + H) * a.C);
        else
          v[k].zero();
      }
#pragma unroll
      for (int k = 0; k < H; ++k) st_pack<T, V>(o + (long)k * a.C, v[k]);
    }
    constexpr int U = 8;  // tokens loaded ahead
    x += (long)t.t0 * a.xt;
    y += (long)t.t0 * a.yt;
    for (int left = t1 - t.t0; left > 0; left -= U) {
      Pack<T, V> in[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < left) in[u] = ld_pack<T, V>(x + u * a.xt);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u >= left) break;
        to_pairs<T, V>(in[u], win[H]);
        pair32 p[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          p[i] = b[i];
#pragma unroll
          for (int k = 0; k < W; ++k) p[i] = pair_fma(w[k][i], win[k][i], p[i]);
          if (a.act == ATLAS_ACT_SILU) {
            float lo, hi;
            unpair(p[i], lo, hi);
            p[i] = pair(siluf(lo), siluf(hi));
          }
#pragma unroll
          for (int k = 0; k < H; ++k) win[k][i] = win[k + 1][i];
        }
        const Pack<T, V> out = from_pairs<T, V>(p);
        st_pack<T, V>(y + u * a.yt, out);  // (heads hold whole vectors: else V is 1)
      }
      x += U * a.xt;
      y += U * a.yt;
    }
  }
}

// Rows of x and dy on their way to a worker of backward_kernel.  32-bit elements have two
// stages, so that three blocks fit an SM all the same.
constexpr int kChunk = 8;
template <typename T>
constexpr int kStages = sizeof(T) == 4 ? 2 : 4;
template <typename T, int V>
struct Ring {
  T x[kStages<T>][kChunk][kLanes * V];
  T dy[kStages<T>][kChunk][kLanes * V];
};

// A warp is a worker: it walks its pieces and keeps dw and db of its channels in registers; the
// block adds its workers in a fixed order and writes one row of partial sums
// part[block][(W + 1)][C].  A piece of n tokens is a stream of positions from -H to n + H, counted from
// its first token: the inputs in front of it (the state before a sequence's first token), its own
// tokens, and those whose dp reaches back into it; dx of a position is complete H positions later.
// Positions before a sequence give dL/d state, into ds.  The stream is copied to shared memory
// kStages - 1 chunks ahead.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kLanes * kWarps)
    backward_kernel(ConvArgs a, long share, float* part, float* ds) {
  constexpr int H = W - 1, N = kPairs<V>, S = kStages<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x, c = (blockIdx.y * kLanes + lane) * V;
  Ring<T, V>& ring = reinterpret_cast<Ring<T, V>*>(smem)[threadIdx.y];
  if (blockIdx.x == 0 && blockIdx.y == 0)
    seq_check(a.s, threadIdx.y * kLanes + lane, kLanes * kWarps);
  pair32 w[W][N], b[N], dw[W][N], db[N];
  load_taps<V, W>(a, c, w, b);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    db[i] = pair(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < W; ++k) dw[k][i] = db[i];
  }
  // copies: CL lanes a row, 16 bytes each (V = 1: one element each, at once)
  constexpr int CV = V == 1 ? 1 : 16 / sizeof(T), CL = kLanes * V / CV, RP = kLanes / CL;
  const int cc = (blockIdx.y * kLanes) * V + lane % CL * CV;  // the channels this lane copies
  const bool cin = cc < a.C;
  SeqWalk walk = seq_walk(a.s, seq_rising(a.s), worker(), share);
  SeqTile t;
  int t1;
  while (seq_piece(a.s, walk, worker(), share, t, t1)) {
    const int n = t1 - t.t0, rest = t.len - t.t0;  // its tokens, those to the sequence's end
    const bool first = t.t0 == 0;  // (else the positions in front of it are tokens)
    const T* x = reinterpret_cast<const T*>(a.x) + seq_at(a.s, t, t.t0, a.xb, a.xt) + cc;
    const T* dy = reinterpret_cast<const T*>(a.dy) + y_at(a, t, t.t0, cc);
    const T* st = a.st_in && t.carry ? reinterpret_cast<const T*>(a.st_in) + ((long)t.b * H + H) * a.C + cc : nullptr;
    const int from = first && !st ? 0 : -H, upto = min(rest, n + H);  // positions there are of x and dy
    auto fetch = [&](int stage, int base) {
      T vx[V > 1 ? 1 : kChunk], vy[V > 1 ? 1 : kChunk];  // V = 1: all loads before the first store
#pragma unroll
      for (int r = 0; r < kChunk; r += RP) {
        const int u = r + lane / CL, q = base + u;
        const bool fx = cin && q < rest && q >= from, fy = cin && q >= 0 && q < upto;
        const T* px = q < 0 && first ? st + (long)q * a.C : x + (long)q * a.xt;
        const T* py = dy + (long)q * a.yt;
        if constexpr (V > 1) {
          cp_async<16>(&ring.x[stage][u][lane % CL * CV], fx ? px : reinterpret_cast<const T*>(a.dx), fx);
          cp_async<16>(&ring.dy[stage][u][lane % CL * CV], fy ? py : reinterpret_cast<const T*>(a.dx), fy);
        } else {
          vx[r] = vy[r] = from_f<T>(0.f);
          if (fx) vx[r] = *px;
          if (fy) vy[r] = *py;
        }
      }
      if constexpr (V == 1) {
#pragma unroll
        for (int r = 0; r < kChunk; ++r) {
          ring.x[stage][r][lane] = vx[r];
          ring.dy[stage][r][lane] = vy[r];
        }
      }
    };
    pair32 win[W][N], dp[W][N];
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) win[k][i] = dp[k][i] = pair(0.f, 0.f);
    T* dx = reinterpret_cast<T*>(a.dx) + seq_at(a.s, t, t.t0, a.xb, a.xt) + c;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
      fetch(k, k * kChunk - H);
      cp_commit();
    }
    int stage = 0;
    // the positions of one chunk; EDGE: some of them are not plain tokens of the piece
    auto walk = [&](int base, auto edge) {
      constexpr bool EDGE = decltype(edge)::value;
      T* out = dx + (long)(base - H) * a.xt;
#pragma unroll
      for (int u = 0; u < kChunk; ++u) {
        const int q = base + u;
        if (EDGE && q >= n + H) break;
        pair32 g[N];
        to_pairs<T, V>(ld_pack<T, V>(&ring.x[stage][u][lane * V]), win[H]);
        to_pairs<T, V>(ld_pack<T, V>(&ring.dy[stage][u][lane * V]), g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          if (a.act == ATLAS_ACT_SILU) {  // SiLU'(p) = s (1 + p (1 - s)), s = 1 / (1 + exp(-p))
            const pair32 one = pair(1.f, 1.f);
            pair32 p = b[i];
#pragma unroll
            for (int k = 0; k < W; ++k) p = pair_fma(w[k][i], win[k][i], p);
            const pair32 e = pair_add(pair_ex2(pair_mul(p, pair(-ATLAS_LOG2E, -ATLAS_LOG2E))), one);
            float lo, hi;
            unpair(e, lo, hi);
            const pair32 s = pair(rcp(lo), rcp(hi));
            g[i] = pair_mul(g[i], pair_mul(s, pair_fma(p, pair_fma(s, pair(-1.f, -1.f), one), one)));
          }
          if (EDGE && (q < 0 || q >= rest)) g[i] = pair(0.f, 0.f);  // also where p is not finite
          dp[H][i] = g[i];
          if (!EDGE || (q >= 0 && q < n)) {  // (zero times a state that is not finite is not zero)
            db[i] = pair_add(db[i], g[i]);
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][i] = pair_fma(g[i], win[k][i], dw[k][i]);
          }
        }
        const int s = q - H;  // the position whose gradient is complete
        if (!EDGE || s >= (first ? -H : 0)) {
          pair32 o[N];
#pragma unroll
          for (int i = 0; i < N; ++i) {
            o[i] = pair_mul(w[H][i], dp[0][i]);
#pragma unroll
            for (int k = 1; k < W; ++k) o[i] = pair_fma(w[H - k][i], dp[k][i], o[i]);
          }
          if (!EDGE) {
            if (c < a.C) st_pack<T, V>(out, from_pairs<T, V>(o));
          } else if (c < a.C) {
            const int tail = s - (rest - H);  // row of dL/d state_out that is this position
            if (a.dstate && tail >= 0) {
              const float* d = a.dstate + ((long)t.b * H + tail) * a.C + c;
#pragma unroll
              for (int i = 0; i < N; ++i) o[i] = pair_add(o[i], pair(d[2 * i], V > 1 ? d[2 * i + 1] : 0.f));
            }
            if (s >= 0) {
              st_pack<T, V>(out, from_pairs<T, V>(o));
            } else if (a.dstate) {
              float* d = ds + ((long)t.b * H + s + H) * a.C + c;
#pragma unroll
              for (int i = 0; i < N; ++i) {
                float lo, hi;
                unpair(o[i], lo, hi);
                d[2 * i] = t.carry ? lo : 0.f;
                if (V > 1) d[2 * i + 1] = t.carry ? hi : 0.f;
              }
            }
          }
        }
        out += a.xt;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int k = 0; k < H; ++k) {
            win[k][i] = win[k + 1][i];
            dp[k][i] = dp[k + 1][i];
          }
      }
    };
    for (int base = -H; base < n + H; base += kChunk) {
      cp_wait<S - 2>();
      __syncwarp();  // this chunk is there for all lanes, and the one before has been read
      fetch(stage == 0 ? S - 1 : stage - 1, base + (S - 1) * kChunk);
      cp_commit();
      if (base >= H && base + kChunk <= min(n, rest - H))
        walk(base, std::false_type());
      else
        walk(base, std::true_type());
      stage = stage + 1 == S ? 0 : stage + 1;
    }
    cp_wait<0>();
  }
  // the block's workers, one after the other
  __syncthreads();  // the rings are no longer needed
  float* acc = reinterpret_cast<float*>(smem) + lane * V;  // [W + 1][32 V]
  for (int r = 0; r < kWarps; ++r) {
    __syncthreads();
    if (r == threadIdx.y) {
#pragma unroll
      for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          float lo, hi;
          unpair(k < W ? dw[k < W ? k : 0][j / 2] : db[j / 2], lo, hi);
          const float s = (r == 0 ? 0.f : acc[k * kLanes * V + j]) + (j % 2 ? hi : lo);
          if (r < kWarps - 1)
            acc[k * kLanes * V + j] = s;
          else if (c < a.C)
            part[((long)blockIdx.x * (W + 1) + k) * a.C + c + j] = s;
        }
    }
  }
}

// Sums the partial rows into dw and dbias and moves the states' gradients into place.
template <typename T>
__global__ void __launch_bounds__(256)
    finish_kernel(ConvArgs a, int nblk, const float* part, const float* ds) {
  __shared__ float s[8][33];
  const int W = a.W;
  const int cols = (W + 1) * a.C;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int nsum = (cols + 31) / 32;
  if ((int)blockIdx.x < nsum) {
    const int i = blockIdx.x * 32 + cx;
    float v = 0.f;
    if (i < cols)
      for (int r = ry; r < nblk; r += 8) v += part[(long)r * cols + i];
    s[ry][cx] = v;
    __syncthreads();
    if (ry == 0 && i < cols) {
#pragma unroll
      for (int r = 1; r < 8; ++r) v += s[r][cx];
      const int k = i / a.C, c = i % a.C;
      if (k < W)
        a.dw[(long)c * W + k] = v;
      else if (a.dbias)
        a.dbias[c] = v;
    }
  } else if (a.dstate) {
    const long n = (long)a.s.B * (W - 1) * a.C;
    const int rising = seq_rising(a.s);
    for (long i = (long)(blockIdx.x - nsum) * 256 + threadIdx.x; i < n;
         i += (long)(gridDim.x - nsum) * 256) {
      if (a.s.start) {  // sequences that are left out keep what they had
        const int b = (int)(i / ((long)(W - 1) * a.C));
        const int st = a.s.start[b], e = a.s.start[b + 1];
        if (b >= rising || st < 0 || e > a.s.L) continue;
      }
      a.dstate[i] = ds[i];
    }
  }
}

inline long lane_groups(const ConvArgs& a, int V) { return (a.C + kLanes * V - 1) / (kLanes * V); }

// Workers over the groups of channels: as many warps as run at once, so that few tokens are read twice
// (forward 24 an SM at up to four taps, backward twelve).
inline long workers(const ConvArgs& a, int V, int an_sm) {
  const long n = kSMs * an_sm / lane_groups(a, V) / kWarps * kWarps;
  return n < kWarps ? kWarps : n;
}
constexpr int kForwardWarps = 24, kBackWarps = 12;
// Blocks for a share of units.
inline long blocks_of(const ConvArgs& a, long share) {
  const long n = (seq_units(a.s) + share - 1) / share;
  return (n + kWarps - 1) / kWarps;
}

template <typename T, int V, int W>
int forward(const ConvArgs& a, cudaStream_t st) {
  const long share = seq_share(a.s, workers(a, V, kForwardWarps), 4);
  const long bx = blocks_of(a, share);
  const long by = lane_groups(a, V);
  if (by > 65535) return ATLAS_ERR_UNSUPPORTED;
  forward_kernel<T, V, W><<<dim3((unsigned)bx, (unsigned)by), dim3(kLanes, kWarps), 0, st>>>(a, share);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <typename T, int V, int W>
int backward(const ConvArgs& a, cudaStream_t st) {
  const long share = seq_share(a.s, workers(a, V, kBackWarps), 1);
  const int n = (int)blocks_of(a, share);
  const long by = lane_groups(a, V);
  if (by > 65535) return ATLAS_ERR_UNSUPPORTED;
  float* ds = reinterpret_cast<float*>(a.ws);
  float* part = ds + (a.dstate ? (size_t)a.s.B * (W - 1) * a.C : 0);
  constexpr size_t rings = kWarps * sizeof(Ring<T, V>), sums = (size_t)(W + 1) * kLanes * V * 4;
  constexpr size_t smem = rings > sums ? rings : sums;
  auto* f = backward_kernel<T, V, W>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return ATLAS_ERR_CUDA;
  if (n > 0)
    f<<<dim3((unsigned)n, (unsigned)by), dim3(kLanes, kWarps), smem, st>>>(a, share, part, ds);
  const int nsum = ((W + 1) * a.C + 31) / 32;
  const long moved = a.dstate ? ((long)a.s.B * (W - 1) * a.C + 255) / 256 : 0;
  finish_kernel<T><<<nsum + (unsigned)(moved < 1024 ? moved : 1024), 256, 0, st>>>(a, n, part, ds);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <typename T, int V>
int run(const ConvArgs& a, bool back, cudaStream_t st) {
#define ATLAS_W(W) \
  case W: return back ? backward<T, V, W>(a, st) : forward<T, V, W>(a, st);
  switch (a.W) {
    ATLAS_W(1) ATLAS_W(2) ATLAS_W(3) ATLAS_W(4) ATLAS_W(5) ATLAS_W(6) ATLAS_W(7) ATLAS_W(8)
    default: return ATLAS_ERR_UNSUPPORTED;
  }
#undef ATLAS_W
}

}  // namespace conv
}  // namespace atlas
