// layernorm_bwd.cu -- layer norm, backward pass.
//
//   hat = (h - mu) rstd,  dx = rstd (w dy - mean(w dy) - hat mean(w dy hat)) + dh,
//   dw = sum over rows of dy hat,  db = sum over rows of dy
//
// Rows of up to 8192 channels: a block walks rows (short ones: lanes of a warp each), the next one or two
// on their way through shared memory; a row's four sums are taken about the mean of its first eight elements, as in the
// forward pass.  A thread's
// columns are the same in every row, so dw and db stay in its registers; blocks write partial sums,
// which a second launch adds in a fixed order.  Longer rows: a block a row, which reads it three times
// (from L2 but the first), then partial sums by column from the rows' kept statistics.
//
// Measured: 16384 x 2560 bf16 with a 32-bit stream 111 us, 78% of the copy rate (two rounds of sums: 126); 12001 x 1371 bf16 68 us,
// 22% (one by one, their type looked at each time: 92): 63% of the issue slots.
#include "layernorm_body.cuh"

namespace atlas {
namespace layernorm {
namespace {

constexpr int kMaxRow = 8192;
constexpr int kSums = 192;  // floats that a block's sums meet in: twice 16 fours (rows take turns), 16 fours

// One vector a thread while 512 threads are enough (2560 channels with a 32-bit stream: two vectors on half as many
// threads have a quarter fewer instructions, but too few warps: 139 us against 111; 80 registers 141, 112: 141).
template <int HB, int DB, int GB, int K, int AL>  // bytes of h, dy, dh (0: none)
__global__ void __maxnreg__(K == 1 ? 96 : 128) backward_rows(Args a, int tpr, int stages) {
  extern __shared__ __align__(16) float sm[];  // 3 x 64 for the sums, then [stage][row of the block]: h, dy, dh
  const int place = threadIdx.x % tpr, rpb = blockDim.x / tpr, mine = threadIdx.x / tpr;
  // (pairs: one row a block, an even grid)
  const int lane = AL == 2 ? 2 * place - (int)((reinterpret_cast<uintptr_t>(DB == 2 ? a.dy : a.x) / 2 + blockIdx.x * (DB == 2 ? a.sy : a.sr)) & 1) : place;
  float dw[K][8], db[K][8], w[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    load_params<AL>(a.w, a.wt, 1.f, k, a.d, tpr, lane, w[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = db[k][i] = 0.f;
  }
  const int hs = slot_bytes<HB, AL>(a.d), ds = slot_bytes<DB, AL>(a.d), bytes = hs + ds + slot_bytes<GB, AL>(a.d);
  char* ring = reinterpret_cast<char*>(sm + kSums) + mine * bytes;
  const Rows th = rows_of<HB>(a.x, a.sr, a.rows, a.d), td = rows_of<DB>(a.dy, a.sy, a.rows, a.d),
             tg = rows_of<GB>(a.r, a.sr, a.rows, a.d);
  const long step = (long)gridDim.x * rpb;
  auto fetch = [&](long row, int stage) {
    char* s = ring + stage * rpb * bytes;
    fetch_row<HB, K * HB / 2, AL>(s, th, row, a.rows, a.d, place, tpr);
    fetch_row<DB, K * DB / 2, AL>(s + hs, td, row, a.rows, a.d, place, tpr);
    fetch_row<GB, K * GB / 2, AL>(s + hs + ds, tg, row, a.rows, a.d, place, tpr);
    cp_commit();
  };
  auto next_done = [&] {
    if (stages == 3)
      cp_wait<1>();
    else
      cp_wait<0>();
  };
  const auto in = [&](int k, int i) { return inside(col<AL>(k, AL == 1 ? 0 : i, tpr, lane), a.d); };
  long row = (long)blockIdx.x * rpb + mine;
  for (int i = 0; i < stages - 1; ++i) fetch(row + i * step, i);
  next_done();
  __syncthreads();
  int stage = 0;
  for (int odd = 0; row - mine < a.rows; row += step, odd ^= 1) {
    const bool live = row < a.rows;
    fetch(row + (stages - 1) * step, stage == 0 ? stages - 1 : stage - 1);
    const char* s = ring + stage * rpb * bytes;
    stage = stage + 1 == stages ? 0 : stage + 1;
    float h[K][8], dy[K][8], gv[K][8];
    const int ah = AL == 1 || !live ? 0 : ahead(th, row), ad = AL == 1 || !live ? 0 : ahead(td, row), ag = AL == 1 || !live || GB == 0 ? 0 : ahead(tg, row);
    // (pairs: eight lanes' mean, 12001 x 1371 bf16 67.5 us for 69.6)
    float base = AL == 2 ? mean8(raw_float<HB>(ld_raw<HB>(s + ah, place & 7), a.rt)) : near_mean<HB, AL>(s + ah, a.rt, a.d);
    base = live ? within(base) : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      slot_floats<HB, AL>(s, ah, a.rt, k, a.d, tpr, lane, h[k]);
      slot_floats<DB, AL>(s + hs, ad, a.dt, k, a.d, tpr, lane, dy[k]);
      if constexpr (GB > 0) slot_floats<GB, AL>(s + hs + ds, ag, a.rt, k, a.d, tpr, lane, gv[k]);
      if (!live) {  // nothing was copied for a place of the block without a row
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = dy[k][i] = 0.f;
      }
    }
    next_done();  // the next row's copies, handed over by the barriers below
    if (tpr <= 32) __syncwarp();
    // Sums of t, t^2, w dy and t w dy, t = h - base, a number near the row's mean; and again about base + mean t where what the
    // differences cancel is more than what is left (as in the forward pass).
    float sum[4];
    const auto sums = [&](float minus, float times) {
      pair32 s1 = pair(0.f, 0.f), s2 = s1, s3 = s1, s4 = s1;
      const pair32 less = pair(-minus, -minus);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float t0, t1;
          unpair(pair_add(pair(h[k][i], h[k][i + 1]), less), t0, t1);
          if (!in(k, i)) t0 = 0.f;
          if (!in(k, i + 1)) t1 = 0.f;
          const pair32 t = pair(t0 * times, t1 * times), wdy = pair_mul(pair(w[k][i], w[k][i + 1]), pair(dy[k][i], dy[k][i + 1]));
          s1 = pair_add(s1, t);
          s2 = pair_fma(t, t, s2);
          s3 = pair_add(s3, wdy);
          s4 = pair_fma(t, wdy, s4);
        }
      sum[0] = pair_sum(s1), sum[1] = pair_sum(s2), sum[2] = pair_sum(s3), sum[3] = pair_sum(s4);
    };
    const auto meet = [&](float* red) {
      for (int m = min(tpr, 32) >> 1; m; m >>= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], m);
      if (tpr > 32) {
        if ((threadIdx.x & 31) == 0) *reinterpret_cast<float4*>(red + (threadIdx.x >> 5) * 4) = make_float4(sum[0], sum[1], sum[2], sum[3]);
        __syncthreads();
        float4 v = reinterpret_cast<const float4*>(red)[0];
        for (int i = 1; i < tpr / 32; ++i) {
          const float4 o = reinterpret_cast<const float4*>(red)[i];
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        sum[0] = v.x, sum[1] = v.y, sum[2] = v.z, sum[3] = v.w;
      }
    };
    sums(base, 1.f);
    meet(sm + odd * 64);
    float mean = sum[0] * a.inv_d, var = fmaf(sum[1], a.inv_d, -mean * mean), dot = fmaf(-mean, sum[2], sum[3]);
    const bool again = far<true>(mean, var);
    if (tpr > 32 ? again : __any_sync(0xFFFFFFFFu, again)) {
      const bool number = summed(mean);
      sums(number ? base + mean : 0.f, number ? 1.f : 0.f);
      meet(sm + 128);
      if (again) {
        base += mean;
        mean = sum[0] * a.inv_d;
        var = var_of(mean, sum[1], a.inv_d);
        dot = fmaf(-mean, sum[2], sum[3]);
        // (a row without a variance, as in the forward pass: nothing but dh reaches dx)
        if (!number || !(var < 3e38f)) base = dot = 0.f, mean = number ? 0.f : mean, var = __int_as_float(0x7F800000);
      }
      if (tpr > 32) __syncthreads();  // (the next row may come here too)
    }
    const float rstd = rsqrtf(fmaxf(var, 0.f) + a.eps), mdy = sum[2] * a.inv_d, mhat = rstd * dot * a.inv_d;
    // hat = (h - mu) rstd, mu = base + mean as two numbers;  dx = rstd (w dy - mdy - hat mhat) + dh
    const float mu = base + mean, off = ((mu - base) - mean) * rstd;
    const pair32 less = pair(-mu, -mu), rstd2 = pair(rstd, rstd), off2 = pair(off, off),
                 mdy2 = pair(-mdy, -mdy), mhat2 = pair(-mhat, -mhat);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const pair32 d2 = pair(dy[k][i], dy[k][i + 1]);
        const pair32 hat = pair_fma(pair_add(pair(h[k][i], h[k][i + 1]), less), rstd2, off2);
        unpair(pair_fma(d2, hat, pair(dw[k][i], dw[k][i + 1])), dw[k][i], dw[k][i + 1]);
        unpair(pair_add(d2, pair(db[k][i], db[k][i + 1])), db[k][i], db[k][i + 1]);
        const pair32 o = pair_fma(hat, mhat2, pair_fma(pair(w[k][i], w[k][i + 1]), d2, mdy2));
        unpair(GB ? pair_fma(rstd2, o, pair(gv[k][i], gv[k][i + 1])) : pair_mul(rstd2, o), h[k][i], h[k][i + 1]);
      }
    }
    if (live) store_row<K, AL>(a.y, row * a.sr, a.rt, a.d, tpr, lane, h);
  }
  cp_wait<0>();
  // The rows of a warp by its lanes, then the warps one by one (a block of 128 rows of 8 channels took 90 us row by row).
  const bool lanes = tpr <= 32;
  if (lanes) {
    for (int m = tpr; m < 32; m <<= 1)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[k][i] += __shfl_xor_sync(0xFFFFFFFFu, dw[k][i], m);
          db[k][i] += __shfl_xor_sync(0xFFFFFFFFu, db[k][i], m);
        }
  }
  const int groups = lanes ? blockDim.x / 32 : 1, group = lanes ? threadIdx.x / 32 : 0;
  const bool writes = !lanes || (threadIdx.x & 31) < tpr;
  float* acc = sm + kSums;  // over the rows' ring
  for (int which = 0; which < 2; ++which) {
    if (!(which ? a.db : a.dw)) continue;
    float* part = a.part + ((long)blockIdx.x * 2 + which) * a.d;
    for (int r = 0; r < groups; ++r) {
      __syncthreads();
      if (r == group && writes) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = col<AL>(k, i, tpr, lane);
            if (inside(c, a.d)) {
              const float v = (r == 0 ? 0.f : acc[c]) + (which ? db[k][i] : dw[k][i]);
              if (r == groups - 1)
                part[c] = v;
              else
                acc[c] = v;
            }
          }
      }
    }
  }
}

// dw[c] and db[c]: sums over the blocks' partial sums; 32 columns a block, 32 threads a column (8, with four loads under
// way: 10.6 us for 304 blocks' of 2560).
__global__ void __launch_bounds__(1024) sum_parts(const float* part, float* dw, float* db, int nblk, int d) {
  __shared__ float s[32][33];
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float v = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int r = ry; r < nblk; r += 32) v += part[((long)r * 2 + blockIdx.y) * d + c];
  }
  s[ry][cx] = v;
  __syncthreads();
  if (ry == 0 && c < d) {
#pragma unroll
    for (int r = 1; r < 32; ++r) v += s[r][cx];
    out[c] = v;
  }
}

// ------------------------------------------------------------------ rows of more than kMaxRow channels

constexpr int kLongBlock = 512;

// A block a row; stats receives (mu as two numbers whose sum it is, rstd) of each.
__global__ void __launch_bounds__(kLongBlock) long_rows(Args a, float4* stats) {
  __shared__ __align__(16) float red[96];
  clear_red(red, 96);
  const RowGroup g{kLongBlock, (int)threadIdx.x, (int)threadIdx.x};
  for (long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const auto h = [&](int c) { return ld_any(a.x, row * a.sr + c, a.rt); };
    const auto dy = [&](int c) { return ld_any(a.dy, row * a.sy + c, a.dt); };
    const auto w = [&](int c) { return a.w ? ld_any(a.w, c, a.wt) : 1.f; };
    float sum = 0.f, dsum = 0.f;
#pragma unroll 8
    for (int c = threadIdx.x; c < a.d; c += kLongBlock) sum += h(c), dsum = fmaf(w(c), dy(c), dsum);
    row_sums2(sum, dsum, g, red);
    float mean = sum * a.inv_d;
    const float mdy = dsum * a.inv_d;
    float rest = 0.f, ss = 0.f, dot = 0.f;
#pragma unroll 8
    for (int c = threadIdx.x; c < a.d; c += kLongBlock) {
      const float v = h(c) - mean;
      rest += v;
      ss = fmaf(v, v, ss);
      dot = fmaf(v, w(c) * dy(c), dot);
    }
    row_sums2(rest, ss, g, red + 32);
    dot = row_sum(dot, g, red + 64);
    rest *= a.inv_d;
    if (!(ss < 3e38f)) {  // no variance, as above: whether all elements are numbers
      float zero = 0.f, none = 0.f;
      for (int c = threadIdx.x; c < a.d; c += kLongBlock) zero = fmaf(h(c), 0.f, zero);
      __syncthreads();
      row_sums2(zero, none, g, red);
      __syncthreads();
      mean = zero, rest = dot = 0.f, ss = __int_as_float(0x7F800000);
    }
    const float rstd = rsqrtf(fmaxf(fmaf(ss, a.inv_d, -rest * rest), 0.f) + a.eps), off = -rest * rstd;
    const float mhat = rstd * (dot * a.inv_d - rest * mdy);
    if (threadIdx.x == 0 && stats) stats[row] = make_float4(mean, off, rstd, 0.f);
#pragma unroll 8
    for (int c = threadIdx.x; c < a.d; c += kLongBlock) {
      const float hat = fmaf(h(c) - mean, rstd, off);
      const float up = a.r ? ld_any(a.r, row * a.sr + c, a.rt) : 0.f;
      st_elem(a.y, row * a.sr + c, a.rt, rstd * (fmaf(w(c), dy(c), -mdy) - hat * mhat) + up);
    }
  }
}

// Partial sums of dy hat and dy over blockIdx.y's rows, 256 columns a block.
__global__ void __launch_bounds__(256) long_cols(Args a, const float4* stats) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.d) return;
  float dw = 0.f, db = 0.f;
#pragma unroll 4
  for (long row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float4 s = stats[row];
    const float dy = ld_any(a.dy, row * a.sy + c, a.dt);
    dw = fmaf(dy, fmaf(ld_any(a.x, row * a.sr + c, a.rt) - s.x, s.z, s.y), dw);
    db += dy;
  }
  a.part[((long)blockIdx.y * 2) * a.d + c] = dw;
  a.part[((long)blockIdx.y * 2 + 1) * a.d + c] = db;
}

// ------------------------------------------------------------------ launches

RowPlan back_plan(int d) { return forward_plan(d, false); }
// Partial sums: at most so many blocks.
int back_blocks(const Args& a) {
  const RowPlan p = back_plan(a.d);
  const long rpb = p.block / p.tpr, need = (a.rows + rpb - 1) / rpb;
  const long most = (long)kSMs * (p.block < 128 ? 8 : 1024 / p.block);
  return (int)(need < most ? need : most);
}
int long_splits(const Args& a) { return (int)(a.rows < 64 ? a.rows : 64); }

template <int HB, int DB, int GB, int K, int AL>
int run_rows(const Args& a, const RowPlan& p, int& blocks, cudaStream_t st) {
  const int rpb = p.block / p.tpr;
  const size_t row = slot_bytes<HB, AL>(a.d) + slot_bytes<DB, AL>(a.d) + slot_bytes<GB, AL>(a.d);
  auto* f = backward_rows<HB, DB, GB, K, AL>;
  const size_t sums = (size_t)a.d * 4;
  const auto bytes = [&](int stages) {
    const size_t ring = stages * rpb * row;
    return kSums * 4 + (ring > sums ? ring : sums);
  };
  // three stages where they cost no block of an SM (and fit)
  const int held = by_registers<backward_rows<HB, DB, GB, K, AL>>(p.block), stages = bytes(3) <= 200 * 1024 && resident(bytes(3), held) == resident(bytes(2), held) ? 3 : 2;
  const size_t smem = bytes(stages);
  if (const int rc = shared(f, smem)) return rc;
  const int most = kSMs * resident(smem, held);  // no more blocks than run at once
  blocks = blocks < most ? blocks : most;
  if (AL == 2) blocks &= ~1;
  f<<<blocks, p.block, smem, st>>>(a, p.tpr, stages);
  return status();
}
template <int HB, int DB, int GB, int AL>
int run(const Args& a, int& blocks, cudaStream_t st) {
  const RowPlan p = back_plan(a.d);
  return p.k == 1 ? run_rows<HB, DB, GB, 1, AL>(a, p, blocks, st) : run_rows<HB, DB, GB, 2, AL>(a, p, blocks, st);
}
template <int HB, int DB, int GB>
int run(const Args& a, int& blocks, cudaStream_t st) {
  if (a.wide) return run<HB, DB, GB, 1>(a, blocks, st);
  if constexpr (HB == 2 || DB == 2)
    if (a.d > 256 && a.rows >= 2 * kSMs &&
        pairs(a, {{a.x, a.sr, a.rt}, {a.dy, a.sy, a.dt}, {a.r, a.sr, a.rt}, {a.y, a.sr, a.rt}}, back_plan(a.d)))
      return run<HB, DB, GB, 2>(a, blocks, st);
  return run<HB, DB, GB, 0>(a, blocks, st);
}
template <int HB, int DB>
int run(const Args& a, int& blocks, cudaStream_t st) {
  return a.r ? run<HB, DB, HB>(a, blocks, st) : run<HB, DB, 0>(a, blocks, st);
}

}  // namespace
}  // namespace layernorm

int layernorm_run_f32(const LayerNormArgs& a, cudaStream_t st);
int layernorm_run_bf16(const LayerNormArgs& a, cudaStream_t st);
int layernorm_run_f16(const LayerNormArgs& a, cudaStream_t st);

int layernorm_forward_launch(const LayerNormArgs& args, cudaStream_t st) {
  LayerNormArgs a = args;
  a.inv_d = 1.f / a.d;
  a.ng = a.group ? (a.d + a.group - 1) / a.group : 1;
  for (a.gshift = 0; (1 << a.gshift) < a.group;) ++a.gshift;
  if (a.dt == ATLAS_BF16) return layernorm_run_bf16(a, st);
  if (a.dt == ATLAS_F16) return layernorm_run_f16(a, st);
  return layernorm_run_f32(a, st);
}

size_t layernorm_backward_workspace(const LayerNormArgs& a) {
  using namespace layernorm;
  if (a.d <= kMaxRow) return (size_t)back_blocks(a) * 2 * a.d * 4;
  return (size_t)a.rows * 16 + (size_t)long_splits(a) * 2 * a.d * 4;
}

int layernorm_backward_launch(const LayerNormArgs& args, cudaStream_t st) {
  using namespace layernorm;
  LayerNormArgs a = args;
  a.inv_d = 1.f / a.d;
  const bool sums = a.dw || a.db;
  int blocks = 0;
  if (a.rows > 0 && a.d <= kMaxRow) {
    blocks = back_blocks(a);
    const bool h4 = a.rt == ATLAS_F32, d4 = a.dt == ATLAS_F32;
    const int rc = h4 ? (d4 ? run<4, 4>(a, blocks, st) : run<4, 2>(a, blocks, st))
                      : (d4 ? run<2, 4>(a, blocks, st) : run<2, 2>(a, blocks, st));
    if (rc != ATLAS_OK) return rc;
  } else if (a.rows > 0) {
    float4* stats = sums ? reinterpret_cast<float4*>(a.part) : nullptr;
    a.part += sums ? a.rows * 4 : 0;
    const long most = 4L * kSMs;
    long_rows<<<(unsigned)(a.rows < most ? a.rows : most), kLongBlock, 0, st>>>(a, stats);
    blocks = long_splits(a);
    if (sums) long_cols<<<dim3((a.d + 255) / 256, blocks), 256, 0, st>>>(a, stats);
  }
  if (sums) sum_parts<<<dim3((a.d + 31) / 32, 2), 1024, 0, st>>>(a.part, a.dw, a.db, blocks, a.d);
  return status();
}

}  // namespace atlas
