// conv_body.cuh -- short causal convolution per channel and its backward pass, for one
// element type (instantiated by conv_f32.cu, conv_bf16.cu, conv_f16.cu).
//
//   p_t = b + sum_k w_k x_{t-W+1+k},  y_t = SiLU(p_t) or p_t
//   dp_t = dy_t SiLU'(p_t),  dx_s = sum_i w_{W-1-i} dp_{s+i},  dw_k = sum_t dp_t x_{t-W+1+k}
//
// Bound by memory: x is read once and y written once.  A lane owns V adjacent channels
// (16 bytes forward, V = 4 backward) and walks the tokens of its tile with the last W - 1
// inputs in registers, so that only the W - 1 tokens in front of a tile are read twice.
#pragma once
#include "ops_common.cuh"

namespace atlas {
namespace conv {

constexpr int kLanes = 32;  // channel vectors of a warp
constexpr int kWarps = 4;   // tiles (forward) or workers (backward) of a block

// Offset of channel c of token tok in y's layout.
__device__ __forceinline__ long y_at(const ConvArgs& a, const SeqTile& t, int tok, int c) {
  const long o = seq_at(a.s, t, tok, a.yb, a.yt);
  return a.hd ? o + (long)(c / a.hd) * a.yh + c % a.hd : o + c;
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kLanes * kWarps) forward_kernel(ConvArgs a, int TT, long tiles) {
  const int lane = threadIdx.x, c = (blockIdx.y * kLanes + lane) * V;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    seq_check(a.s, threadIdx.y * kLanes + lane, kLanes * kWarps);
  const long tile = (long)blockIdx.x * kWarps + threadIdx.y;
  SeqTile t;
  if (tile >= tiles || !seq_tile(a.s, tile, TT, t) || c >= a.C) return;
  const T* x = reinterpret_cast<const T*>(a.x);
  T* y = reinterpret_cast<T*>(a.y);
  constexpr int H = W - 1;
  float w[W][V], b[V], win[W][V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][j] = ld_any(a.w, (long)(c + j) * W + k, a.wt);
    b[j] = a.bias ? ld_any(a.bias, c + j, a.wt) : 0.f;
  }
  Pack<T, V> st[W];  // the last H inputs before the tile
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const int tok = t.t0 - H + k;
    if (tok >= 0)
      st[k] = ld_pack<T, V>(x + seq_at(a.s, t, tok, a.xb, a.xt) + c);
    else if (a.st_in && t.carry)  // t0 == 0: a tile is never shorter than H
      st[k] = ld_pack<T, V>(reinterpret_cast<const T*>(a.st_in) + ((long)t.slot * H + k) * a.C + c);
    else
      st[k].zero();
  }
  // the first tile alone reads the state, so it also writes the new one (the buffers may
  // be the same): the last H of (state, inputs)
  if (a.st_out && t.t0 == 0) {
    T* o = reinterpret_cast<T*>(a.st_out) + (long)t.slot * H * a.C + c;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const int tok = t.len - H + k;
      Pack<T, V> v;
      if (tok >= 0) {
        v = ld_pack<T, V>(x + seq_at(a.s, t, tok, a.xb, a.xt) + c);
      } else {
        v = st[0];
#pragma unroll
        for (int i = 1; i < H; ++i)
          if (i == tok + H) v = st[i];
      }
      st_pack<T, V>(o + (long)k * a.C, v);
    }
  }
#pragma unroll
  for (int k = 0; k < H; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j) win[k][j] = st[k].get(j);
  const int t1 = min(t.t0 + TT, t.len);
  constexpr int U = 8;  // tokens loaded ahead
  for (int t0 = t.t0; t0 < t1; t0 += U) {
    Pack<T, V> in[U];
    const T* xp = x + seq_at(a.s, t, t0, a.xb, a.xt) + c;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (t0 + u < t1) in[u] = ld_pack<T, V>(xp + (long)u * a.xt);
    T* yp = y + y_at(a, t, t0, c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t0 + u >= t1) break;
      Pack<T, V> out;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        win[H][j] = in[u].get(j);
        float p = b[j];
#pragma unroll
        for (int k = 0; k < W; ++k) p += w[k][j] * win[k][j];
        out.set(j, a.act == ATLAS_ACT_SILU ? siluf(p) : p);
#pragma unroll
        for (int k = 0; k < H; ++k) win[k][j] = win[k + 1][j];
      }
      if (V == 1 || !a.hd || a.hd % V == 0) {
        st_pack<T, V>(yp + (long)u * a.yt, out);
      } else {  // a vector crosses heads
#pragma unroll
        for (int j = 0; j < V; ++j) y[y_at(a, t, t0 + u, c + j)] = out.e[j];
      }
    }
  }
}

// A warp is a worker: it walks tiles and keeps dw and db of its channels in registers; the
// block adds its workers in a fixed order and writes one row of partial sums
// part[block][(W + 1)][C].  Positions before a sequence give dL/d state, into ds.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kLanes * kWarps)
    backward_kernel(ConvArgs a, int TT, long tiles, float* part, float* ds) {
  extern __shared__ float sm[];
  const int lane = threadIdx.x, c = (blockIdx.y * kLanes + lane) * V;
  if (blockIdx.x == 0 && blockIdx.y == 0)
    seq_check(a.s, threadIdx.y * kLanes + lane, kLanes * kWarps);
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* dy = reinterpret_cast<const T*>(a.dy);
  T* dx = reinterpret_cast<T*>(a.dx);
  constexpr int H = W - 1;
  float w[W][V], b[V], dw[W][V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int k = 0; k < W; ++k) {
      w[k][j] = c < a.C ? ld_any(a.w, (long)(c + j) * W + k, a.wt) : 0.f;
      dw[k][j] = 0.f;
    }
    b[j] = a.bias && c < a.C ? ld_any(a.bias, c + j, a.wt) : 0.f;
    db[j] = 0.f;
  }
  for (long tile = (long)blockIdx.x * kWarps + threadIdx.y; tile < tiles;
       tile += (long)gridDim.x * kWarps) {
    SeqTile t;
    if (!seq_tile(a.s, tile, TT, t) || c >= a.C) continue;
    float win[W][V], dp[W][V];
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const int tok = t.t0 - H + k;
      Pack<T, V> v;
      if (tok >= 0)
        v = ld_pack<T, V>(x + seq_at(a.s, t, tok, a.xb, a.xt) + c);
      else if (a.st_in && t.carry)
        v = ld_pack<T, V>(reinterpret_cast<const T*>(a.st_in) + ((long)t.b * H + k) * a.C + c);
      else
        v.zero();
#pragma unroll
      for (int j = 0; j < V; ++j) win[k][j] = v.get(j), dp[k][j] = 0.f;
    }
    const int t1 = min(t.t0 + TT, t.len);
    // dp is needed H tokens past the tile; emission runs H tokens behind
    constexpr int U = 4;
    for (int q0 = t.t0; q0 < t1 + H; q0 += U) {
      Pack<T, V> in[U], up[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tok = q0 + u;
        if (tok < t.len && tok < t1 + H) {
          in[u] = ld_pack<T, V>(x + seq_at(a.s, t, tok, a.xb, a.xt) + c);
          if (V == 1 || !a.hd || a.hd % V == 0) {
            up[u] = ld_pack<T, V>(dy + y_at(a, t, tok, c));
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j) up[u].e[j] = dy[y_at(a, t, tok, c + j)];
          }
        } else {
          in[u].zero();
          up[u].zero();
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int tok = q0 + u;
        if (tok >= t1 + H) break;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          win[H][j] = in[u].get(j);
          float g = up[u].get(j);
          if (a.act == ATLAS_ACT_SILU) {
            float p = b[j];
#pragma unroll
            for (int k = 0; k < W; ++k) p += w[k][j] * win[k][j];
            g *= silu_slope(p, sigmoidf(p));
          }
          if (tok >= t.len) g = 0.f;
          dp[H][j] = g;
          if (tok < t1) {
            db[j] += g;
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][j] += g * win[k][j];
          }
        }
        const int s = tok - H;  // the position whose gradient is complete
        if (s >= t.t0 || t.t0 == 0) {
          float o[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            o[j] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) o[j] += w[H - i][j] * dp[i][j];
          }
          const int tail = s - (t.len - H);  // row of dL/d state_out that is this position
          if (a.dstate && tail >= 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] += a.dstate[((long)t.b * H + tail) * a.C + c + j];
          }
          if (s >= 0) {
            Pack<T, V> v;
#pragma unroll
            for (int j = 0; j < V; ++j) v.set(j, o[j]);
            st_pack<T, V>(dx + seq_at(a.s, t, s, a.xb, a.xt) + c, v);
          } else if (a.dstate) {
#pragma unroll
            for (int j = 0; j < V; ++j)
              ds[((long)t.b * H + s + H) * a.C + c + j] = t.carry ? o[j] : 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int k = 0; k < H; ++k) {
            win[k][j] = win[k + 1][j];
            dp[k][j] = dp[k + 1][j];
          }
      }
    }
  }
  // the block's workers, one after the other
  float* acc = sm + lane * V;  // [W + 1][32 V]
  for (int r = 0; r < kWarps; ++r) {
    __syncthreads();
    if (r == threadIdx.y) {
#pragma unroll
      for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float s = (r == 0 ? 0.f : acc[k * kLanes * V + j]) + (k < W ? dw[k < W ? k : 0][j] : db[j]);
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
    for (long i = (long)(blockIdx.x - nsum) * 256 + threadIdx.x; i < n;
         i += (long)(gridDim.x - nsum) * 256) {
      if (a.s.start) {  // sequences that are left out keep what they had
        const int b = (int)(i / ((long)(W - 1) * a.C));
        const int st = a.s.start[b], e = a.s.start[b + 1];
        if (st < 0 || e < st || e > a.s.L) continue;
      }
      a.dstate[i] = ds[i];
    }
  }
}

// Tokens per tile: long tiles read fewer tokens twice (W - 1 of each), short ones fill the
// machine; at least H so that one tile alone touches the state.
inline int tile_tokens(const ConvArgs& a, int V, long warps) {
  const long lanes = (a.C + kLanes * V - 1) / (kLanes * V);
  const long rows = a.s.start ? a.s.L : (long)a.s.B * a.s.L;
  int TT = 64;
  while (TT > 8 && rows / TT * lanes < warps) TT /= 2;
  return TT;
}

inline int back_blocks(const ConvArgs& a, int V, long tiles) {
  const long lanes = (a.C + kLanes * V - 1) / (kLanes * V);
  long n = (152 * 4 + lanes - 1) / lanes;  // four blocks an SM
  const long need = (tiles + kWarps - 1) / kWarps;
  return (int)(n < need ? n : need);
}

template <typename T, int V, int W>
int forward(const ConvArgs& a, cudaStream_t st) {
  const int TT = tile_tokens(a, V, 152 * 32);
  const long tiles = seq_tiles(a.s, TT);
  const long bx = (tiles + kWarps - 1) / kWarps;
  const long by = (a.C + kLanes * V - 1) / (kLanes * V);
  if (bx > 0x7FFFFFFFL || by > 65535) return ATLAS_ERR_UNSUPPORTED;
  forward_kernel<T, V, W><<<dim3((unsigned)bx, (unsigned)by), dim3(kLanes, kWarps), 0, st>>>(a, TT, tiles);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <typename T, int V, int W>
int backward(const ConvArgs& a, cudaStream_t st) {
  const int TT = tile_tokens(a, V, 152 * 16);
  const long tiles = seq_tiles(a.s, TT);
  const int n = back_blocks(a, V, tiles);
  const long by = (a.C + kLanes * V - 1) / (kLanes * V);
  if (by > 65535) return ATLAS_ERR_UNSUPPORTED;
  float* ds = reinterpret_cast<float*>(a.ws);
  float* part = ds + (a.dstate ? (size_t)a.s.B * (W - 1) * a.C : 0);
  const size_t smem = (size_t)(W + 1) * kLanes * V * 4;
  if (n > 0)
    backward_kernel<T, V, W><<<dim3((unsigned)n, (unsigned)by), dim3(kLanes, kWarps), smem, st>>>(
        a, TT, tiles, part, ds);
  const int nsum = ((W + 1) * a.C + 31) / 32;
  const long moved = a.dstate ? ((long)a.s.B * (W - 1) * a.C + 255) / 256 : 0;
  finish_kernel<T><<<nsum + (unsigned)(moved < 1024 ? moved : 1024), 256, 0, st>>>(a, n, part, ds);
  return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <typename T, int VF, int VB>
int run(const ConvArgs& a, bool back, cudaStream_t st) {
#define ATLAS_W(W) \
  case W: return back ? backward<T, VB, W>(a, st) : forward<T, VF, W>(a, st);
  switch (a.W) {
    ATLAS_W(1) ATLAS_W(2) ATLAS_W(3) ATLAS_W(4) ATLAS_W(5) ATLAS_W(6) ATLAS_W(7) ATLAS_W(8)
    default: return ATLAS_ERR_UNSUPPORTED;
  }
#undef ATLAS_W
}

}  // namespace conv
}  // namespace atlas
