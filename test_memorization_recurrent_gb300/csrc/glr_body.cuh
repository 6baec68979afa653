// glr_body.cuh -- gated linear recurrence, one state a channel: forward and backward.
//
//   s_t = c softplus(lambda) sigmoid(r_t),  a_t = exp(-s_t),  beta_t = sqrt(1 - a_t^2)
//   u_t = beta_t sigmoid(i_t) x_t,  h_t = a_t h_{t-1} + u_t,  y_t = h_t SiLU(z_t)
//   g_t = dL/dh_t = v_t + a_{t+1} g_{t+1},  v_t = dy_t SiLU(z_t)
//   dx = g beta sigma_i,  di = g u (1 - sigma_i),  dr = Q (1 - sigma_r),
//   Q = s dL/ds = g (u a^2 s / beta^2 - s a h_{t-1}),  dlambda = sum Q sigmoid(lambda) / softplus(lambda)
//
// A token's step is the map h -> a h + u, and such maps compose: (a, u) after (A, H) is (a A, a H + u).  The rows of a
// call are strings of maps, cut into tiles of kRows rows x kCh channels: equal work, whatever the sequences.
// Packed sequences (and short ones) are one string, in which a first token has the map h -> a h_0 + u, so that nothing
// passes from one sequence to the next; long sequences of one length are a string each.  A block takes tiles in order of a
// ticket.  Its threads hold a few tokens' maps each; lanes and warps compose them.  Where there are strings enough
// to keep all blocks busy, the tickets go from string to string, a tile takes the state that the one in front of it left
// long ago, and leaves its own.  Else the tile's map goes to memory at once, where the later tiles of its group of
// kGroup read it: each composes, always in the same order, what lies in front of it in its group with the state that
// the group before it left; a long sequence then costs one wait a group and not one a tile.  Everything is read once,
// and results do not depend on which block ran when.  A block waits only for tiles of earlier tickets, which running blocks
// hold.  A map travels as one 64-bit word that is all ones until it is there.
//
// A map's factor is held as d: 1 - a where a is near 1 (h + (u - d h) then rounds by h's last place, not by that of a,
// which would be the same in every step of a slow channel, and products of factors just below 1 would all be
// rounded down), else -a; 2 is a cut, which lets nothing through, not even what is not finite.  No factor is coded so: one
// that has left the range is -0 and multiplies, so NaN reaches the rest of its sequence however fast that decays and wherever
// its tiles end.
//
// Backward the same with the rows in reverse: c -> a (v + c) carries a g to the token in front.  The states inside a
// tile come from the state in front of it, which the forward pass keeps (one for kRows rows, in 32 bits).
//
// An element takes eight results of the exponential pipe and 65 instructions (147 backward), so issue and latency bound it,
// then memory.  Measured (copy rate 6.79 TB/s): 8 x 4096 x 2048 bf16, gated: 211 us, 47%, with the backward pass 691, 40%; with
// one string, 65536 x 512: 184 us, 22%; 9001 packed rows x 1500: 91 us.  A warp whose rows hold a factor below 0.70 or a first token, or
// are not all of a sequence and its channels, goes through the maps one by one: with one such channel in 32, 8 x 4096 x 2048 takes
// 333 us and 1174 with its backward pass, with no other channels 355 and 1218.  Tiles of 64 rows on blocks of four warps:
// 252 us; of 256 rows on sixteen: 234; three blocks of an SM (80 registers): 227.
#pragma once
#include "ops_common.cuh"

namespace atlas {
namespace glr {

constexpr int kCh = 32, kWarps = 8, kThreads = 32 * kWarps, kRows = 16 * kWarps, kGroup = 4 * kWarps;
constexpr int kPer = kRows / kWarps;  // rows of a warp
constexpr int kBlocks = 2;            // of an SM: a thread's elements and the work on them take 128 registers
constexpr unsigned long long kAbsent = ~0ull;
// Looks at a word until a wait gives up, most of a second; never reached unless two calls share a workspace.  Test builds only:
// with ATLAS_TEST_WITHHOLD_LOADS defined, the second tile of the first channels never hands on its map.
constexpr int kPolls = 1 << 20;
#ifdef ATLAS_TEST_WITHHOLD_LOADS
constexpr bool kWithhold = true;
#else
constexpr bool kWithhold = false;
#endif

// ------------------------------------------------------------------ workspace

struct Space {
  unsigned* ticket;                // and, behind it, whether a wait has given up
  float *rate, *rb, *ib;           // [groups * kCh]: c softplus(lambda), -log2(e) biases
  unsigned long long* words;       // [tiles][groups * kCh]
  int* tile_seq;                   // [tiles + 1]: packed, the sequence of a tile's first row
  int* state;                      // [B]: a sequence's state, -1: left out
  float* sums;                     // backward [tiles][3][D]
  float* kept;                     // backward without the forward's: [tiles][D]
  size_t bytes;
};

// (without sequences no row belongs to one, and seq_start has one element)
inline long rows_of(const GlrArgs& a) { return a.s.start && a.s.B > 0 ? a.s.L : (long)a.s.B * a.s.L; }
inline int groups_of(const GlrArgs& a) { return (a.D + kCh - 1) / kCh; }

// The strings of tiles.
struct Strings {
  long rows;                    // of the call
  unsigned n, tiles, groups;    // strings (1: all rows), tiles of each, groups of channels
  unsigned group;               // tiles of a group
  unsigned total;               // tiles x channels in all
};
// Sequences of one length are strings of their own where that leaves few places of tiles empty (a fifth at most: of 513
// rows, 127 of 640 places).  (As one string, 8 x 4096 x 2048 took 299 us against 211, its training pass 916 against 706.)
inline bool apart_of(const GlrArgs& a) { return !a.s.start && a.s.L > 0 && (a.s.L >= 4 * kRows || a.s.L % kRows == 0); }
inline long tiles_of(const GlrArgs& a) {  // in all
  if (apart_of(a)) return (long)a.s.B * ((a.s.L - 1L) / kRows + 1);
  return (rows_of(a) + kRows - 1) / kRows;
}
inline Strings strings(const GlrArgs& a) {
  Strings t;
  t.rows = rows_of(a);
  t.n = apart_of(a) ? a.s.B : 1;
  t.tiles = (unsigned)(tiles_of(a) / t.n);
  t.groups = groups_of(a);
  // a tile's predecessor in its string lies n x groups tickets behind it: done, if no more blocks run (in groups of tiles
  // all the same, 8 x 4096 x 2048 took 276 us against 211)
  t.group = (long)t.n * t.groups >= (long)kBlocks * kSMs ? 1 : kGroup;
  t.total = t.n * t.tiles * t.groups;
  return t;
}

inline Space space(const GlrArgs& a, bool back, bool keep) {
  Space s = {};
  char* p = reinterpret_cast<char*>(a.ws);
  size_t at = 0;
  const auto take = [&](size_t n) {
    char* q = p + at;
    at += (n + 15) / 16 * 16;
    return q;
  };
  const size_t tiles = tiles_of(a), width = (size_t)groups_of(a) * kCh;
  s.ticket = reinterpret_cast<unsigned*>(take(8));
  s.rate = reinterpret_cast<float*>(take(width * 4));
  s.rb = reinterpret_cast<float*>(take(width * 4));
  s.ib = reinterpret_cast<float*>(take(width * 4));
  s.words = reinterpret_cast<unsigned long long*>(take(tiles * width * 8));
  s.tile_seq = reinterpret_cast<int*>(take(a.s.start ? (tiles + 1) * 4 : 0));
  s.state = reinterpret_cast<int*>(take(a.s.start || a.s.slot ? (size_t)a.s.B * 4 : 0));
  if (back) s.sums = reinterpret_cast<float*>(take(tiles * 3 * a.D * 4));
  if (keep) s.kept = reinterpret_cast<float*>(take(tiles * a.D * 4));
  s.bytes = at;
  return s;
}

// ------------------------------------------------------------------ functions

// Of two elements at once: an instruction on a pair takes one issue slot, and those are what the kernels run out of.
__device__ __forceinline__ pair32 twice(float v) { return pair(v, v); }

// sigmoid of -b / log2(e): 1 / (1 + 2^b).
__device__ __forceinline__ pair32 gate(pair32 b) {
  float x, y;
  unpair(pair_add(twice(1.f), pair_ex2(b)), x, y);
  return pair(rcp(x), rcp(y));
}
// And 1 - sigmoid to its own relative precision, 2^b sigma.  The exponent is held below 126, so that it has no
// infinity; NONE: sigmoid is then 0, as beyond, and not 2^-126.
template <bool NONE>
__device__ __forceinline__ pair32 gate(pair32 b, pair32& rest) {
  float b0, b1, x, y;
  unpair(b, b0, b1);
  const pair32 e = pair(ex2(fminf(b0, 126.f)), ex2(fminf(b1, 126.f)));
  unpair(pair_add(twice(1.f), e), x, y);
  x = rcp(x), y = rcp(y);
  rest = pair_mul(e, pair(x, y));
  return NONE ? pair(b0 >= 126.f ? 0.f : x, b1 >= 126.f ? 0.f : y) : pair(x, y);
}

// 1 - exp(-s) for 0 <= s < kSlow: s P(s), P fitted to (1 - exp(-s)) / s at Chebyshev nodes (relative error 1.7e-8, 9e-8
// with the roundings of its evaluation).  Above, the exponential: decays below 0.70, which channels of long memory never have.
constexpr float kSlow = 0.36f;
__device__ __forceinline__ pair32 lost(pair32 s) {
  pair32 p = pair_fma(twice(0.0071831392f), s, twice(-0.041314516f));
  p = pair_fma(p, s, twice(0.16662203f));
  p = pair_fma(p, s, twice(-0.499998f));
  p = pair_fma(p, s, twice(1.f));
  return pair_mul(p, s);
}
__device__ __forceinline__ float lost(float s) {
  float m, dummy;
  unpair(lost(twice(s)), m, dummy);
  return m;
}
__device__ __forceinline__ float kept_of(float s) { return ex2(-ATLAS_LOG2E * s); }

// A factor a as d: 1 - a, or -a (2 a cut).
__device__ __forceinline__ bool is_kept(float d) { return __float_as_int(d) < 0; }
__device__ __forceinline__ bool is_cut(float d) { return d > 1.f; }
constexpr float kCut = 2.f;
__device__ __forceinline__ float factor(float d) { return is_kept(d) ? -d : 1.f - d; }
// Of 1 - a and a, both to their own precision.
__device__ __forceinline__ float coded(float m, float a) { return m < kSlow ? m : -a; }
// a c + u
__device__ __forceinline__ float apply(float d, float u, float c) {
  if (is_cut(d)) return u;
  const float t = fmaf(-d, c, u);
  return is_kept(d) ? t : c + t;
}
// The factor of d after e: a cut if one of them is.
__device__ __forceinline__ float after(float d, float e) {
  if (is_cut(d) || is_cut(e)) return kCut;
  const float m = fmaf(-d, e, d + e);  // of two that are 1 - a
  const float a = is_kept(d) || is_kept(e) ? factor(d) * factor(e) : 1.f - m;
  return is_kept(d) || is_kept(e) ? -a : coded(m, a);
}
__device__ __forceinline__ float root(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ pair32 root(pair32 v) {
  float x, y;
  unpair(v, x, y);
  return pair(root(x), root(y));
}

// softplus(lambda), and sigmoid(lambda) / softplus(lambda), which is 1 in the limit of -infinity.
__device__ __forceinline__ float soft(float x) { return x > 15.f ? x + __expf(-x) : log1pf(expf(x)); }
__device__ __forceinline__ float soft_ratio(float x) {
  if (x < -15.f) return 1.f - 0.5f * expf(x);  // log1p(e) = e (1 - e / 2 + ..), 1 / (1 + e) = 1 - e + ..
  return 1.f / (1.f + expf(-x)) / soft(x);
}

// The same of factors that are no cuts, held both ways until the end.
struct Map {
  float m, a, h;  // 1 - factor, factor, offset
  __device__ __forceinline__ void follow(float pm, float pa, float ph) {  // this after the other
    const float near = ph + fmaf(-m, ph, h), far = fmaf(a, ph, h);
    h = m < kSlow ? near : far;
    m = fmaf(-m, pm, m + pm);
    a *= pa;
  }
};

__device__ __forceinline__ unsigned long long word_of(float d, float H) {
  const unsigned long long w = (unsigned long long)__float_as_uint(d) << 32 | __float_as_uint(H);
  return w == kAbsent ? 0x7FFFFFFF7FFFFFFFull : w;  // (both NaN)
}
__device__ __forceinline__ unsigned long long peek(const unsigned long long* p) {
  unsigned long long v;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void post(unsigned long long* p, unsigned long long v) {
  asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}

// A word that another block leaves, once it is there.  By a whole warp, a channel each.  A wait that runs out is the last
// of the call: the others then give up at once, with NaN for what they miss.
__device__ __forceinline__ unsigned long long await(const unsigned long long* p, unsigned long long v, unsigned* lost, int* status) {
  for (int polls = 0; !__all_sync(0xFFFFFFFFu, v != kAbsent); ++polls) {
    const bool over = polls >= kPolls;
    if (over || (polls & 63) == 63) {
      if (over) {
        *reinterpret_cast<volatile unsigned*>(lost) = 1;
        if (status) *status = ATLAS_ERR_TIMEOUT;
      }
      if (__any_sync(0xFFFFFFFFu, over || *reinterpret_cast<volatile unsigned*>(lost))) break;
    }
    v = peek(p);
  }
  return v;
}
__device__ __forceinline__ float apply(unsigned long long word, float c) {
  return apply(__uint_as_float((unsigned)(word >> 32)), __uint_as_float((unsigned)word), c);
}

// Which tile a ticket is: string, place in it in walking order, tile (of all, and the first of the string), first channel.
struct alignas(16) Tile {
  unsigned string, at, k, first;
  int c0;
  bool some;  // false: behind the last ticket
  __device__ __forceinline__ void find(const Strings& t, unsigned n, bool reverse) {
    some = n < t.total;
    const unsigned q = n / t.groups;
    c0 = (int)(n - q * t.groups) * kCh;
    at = q / t.n;
    string = q - at * t.n;
    first = string * t.tiles;
    k = first + (reverse ? t.tiles - 1 - at : at);
  }
  // the call's row that the tile begins with
  __device__ __forceinline__ long row0(const GlrArgs& a) const { return (long)string * a.s.L + (long)(k - first) * kRows; }
};
// What a tile gets through the words of its group: those from place j0 on (and, first, what the group before left), where
// its string's carry begins.  Each warp asks for four neighbours at once and composes them.
struct Group {
  float2 part[kWarps][kCh];
  unsigned j0, lead;  // j0 == the tile's place: nothing reaches it
  __device__ __forceinline__ void begin(const Strings& t, const Tile& q, bool some, unsigned from) {
    const unsigned own = q.at / t.group * t.group;
    lead = own > 0 ? own - 1 : 0;
    j0 = !some ? q.at : from > lead ? from : lead;
  }
  __device__ __forceinline__ void gather(const Tile& q, const unsigned long long* words, size_t width, unsigned* lost, int* status) {
    const unsigned j = lead + (threadIdx.x >> 5) * 4;
    const auto there = [&](int i) { return j + i >= j0 && j + i < q.at; };
    unsigned long long v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (there(i)) v[i] = peek(words + (q.first + j + i) * width);
    float2 m = make_float2(0.f, 0.f);  // the identity
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (there(i)) {
        const unsigned long long word = await(words + (q.first + j + i) * width, v[i], lost, status);
        const float d = __uint_as_float((unsigned)(word >> 32));
        m.y = apply(word, m.y);
        m.x = after(d, m.x);
      }
    part[threadIdx.x >> 5][threadIdx.x & 31] = m;
  }
  __device__ __forceinline__ float carry() const {
    float2 m[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m[i] = part[i][threadIdx.x & 31];
    float c = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) c = apply(m[i].x, m[i].y, c);
    return c;
  }
};
static_assert(kGroup <= 4 * kWarps, "a group's words, and that of the group before, in its first tile's place");

// ------------------------------------------------------------------ rows

// A row's place: its sequence, and whether it takes part (rows of no sequence, or of one that is left out, do not) and is the
// first or last of it.
struct Row {
  int b;
  bool live, first, last;
};
__device__ __forceinline__ Row row_of(const GlrArgs& a, const Space& w, const Strings& t, const Tile& q, int r) {
  const Row none{0, false, false, false};
  Row o{0, true, false, false};
  if (a.s.start) {
    const long row = (long)q.k * kRows + r;
    int lo = w.tile_seq[q.k], hi = w.tile_seq[q.k + 1];  // the last sequence that starts at or before a row
    while (lo < hi) {
      const int mid = lo + (hi - lo + 1) / 2;
      if (a.s.start[mid] <= row)
        lo = mid;
      else
        hi = mid - 1;
    }
    o.b = lo;
    const int s = a.s.start[lo], e = a.s.start[lo + 1];
    if (row < s || row >= e) return none;
    o.first = row == s;
    o.last = row == e - 1;
  } else if (t.n > 1 || a.s.B == 1) {
    const long at = (long)(q.k - q.first) * kRows + r;
    if (at >= a.s.L) return none;
    o = Row{(int)q.string, true, at == 0, at == a.s.L - 1};
  } else {
    const long row = (long)q.k * kRows + r;
    if (row >= t.rows) return none;
    o.b = (int)(row / a.s.L);
    const int at = (int)(row - (long)o.b * a.s.L);
    o.first = at == 0;
    o.last = at == a.s.L - 1;
  }
  if ((a.s.start || a.s.slot) && w.state[o.b] < 0) return none;
  return o;
}
// A warp's rows of a tile: lane r of the first kPer has row r's sequence; a bit a row.
struct Info {
  int b;
  unsigned live, first, last;
  __device__ __forceinline__ void look(const GlrArgs& a, const Space& w, const Strings& t, const Tile& q) {
    const int r = threadIdx.x & (kPer - 1);
    const Row o = row_of(a, w, t, q, (threadIdx.x >> 5) * kPer + r);
    b = o.b;
    live = __ballot_sync(0xFFFFFFFFu, o.live);
    first = __ballot_sync(0xFFFFFFFFu, o.first);
    last = __ballot_sync(0xFFFFFFFFu, o.last);
  }
  // S rows from `from` on, of channels that there are.
  template <int S>
  __device__ __forceinline__ static unsigned bits(unsigned w, int from, bool in) {
    return in ? w >> from & ((1u << S) - 1u) : 0u;
  }
  __device__ __forceinline__ int seq(int r) const { return __shfl_sync(0xFFFFFFFFu, b, r); }  // by the whole warp
};
static_assert(kPer == 16, "a lane and its neighbour 16 further have one row");
__device__ __forceinline__ int state_of(const GlrArgs& a, const Space& w, int b) { return a.s.start || a.s.slot ? w.state[b] : b; }
// The state in front of sequence b.
__device__ __forceinline__ float start_of(const GlrArgs& a, const Space& w, int b, int c) {
  if (!a.h_in || (a.s.carry && !a.s.carry[b])) return 0.f;
  return a.h_in[(long)state_of(a, w, b) * a.D + c];
}

// A thread has V neighbours of S rows each: 4, 8 lanes a row, or 2 or 1 and 16 or 32 lanes where rows do not allow that.
template <int V>
struct Shape {
  static constexpr int lanes = kCh / V, groups = 32 / lanes, S = kPer / groups, N = S * V;
};

// Where a thread finds its channels of a tensor's rows.  FLAT: sequences lie one behind the other (or are packed), fewer than
// 2^31 rows of less than 2^32 bytes: one multiplication an address.
template <typename T, bool FLAT>
struct Cursor {
  char* p;
  long st, skip;  // bytes from row to row, and further for each sequence in front
  __device__ __forceinline__ Cursor(const void* base, long sb, long token, const GlrArgs& a, int c)
      : p(const_cast<char*>(reinterpret_cast<const char*>(base)) + (long)c * sizeof(T)), st(token * (long)sizeof(T)),
        skip(FLAT || a.s.start ? 0 : (sb - token * a.s.L) * (long)sizeof(T)) {}
  __device__ __forceinline__ T* at(long row, int b) const {  // b: the row's sequence
    if (FLAT) return reinterpret_cast<T*>(p + (unsigned long long)(unsigned)row * (unsigned)st);
    return reinterpret_cast<T*>(p + row * st + b * skip);
  }
};

// A thread's own elements on their way through shared memory: nobody else reads them.  (2-byte elements by themselves have no
// asynchronous copy.)
template <typename T, int V, int S>
struct Slots {
  Pack<T, V>* p;  // [S][kThreads], this thread's
  __device__ __forceinline__ Slots(char* base, int tensor) : p(reinterpret_cast<Pack<T, V>*>(base) + tensor * S * kThreads + threadIdx.x) {}
  __device__ __forceinline__ void fetch(int s, const T* from) const {
    if constexpr (sizeof(T) * V >= 4)
      cp_async<sizeof(T) * V>(p + s * kThreads, from, true);
    else
      p[s * kThreads] = ld_pack<T, V>(from);
  }
  // elements e .. e + 3 (e a multiple of four) as two pairs
  struct Four {
    pair32 lo, hi;
    __device__ __forceinline__ pair32 operator[](int j) const { return j ? hi : lo; }
  };
  __device__ __forceinline__ Four four(int e) const {
    float v[4];
    if constexpr (V == 4) {
      p[e / 4 * kThreads].unpack(v);
    } else if constexpr (V == 2) {
      p[e / 2 * kThreads].unpack(v);
      p[(e / 2 + 1) * kThreads].unpack(v + 2);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = p[(e + i) * kThreads].get(0);
    }
    return Four{pair(v[0], v[1]), pair(v[2], v[3])};
  }
  __device__ __forceinline__ pair32 two(int e) const { return four(e & ~3)[e >> 1 & 1]; }
};
template <typename T>
constexpr int slots_bytes(int tensors) {
  return tensors * kPer * kThreads * (int)sizeof(T);
}

// Elements e, e + 1 of values that rows share.
template <int V>
__device__ __forceinline__ pair32 two(const float* p, int e) {
  return V > 1 ? pair(p[e % V], p[e % V + (V > 1)]) : pair(p[0], p[0]);
}
__device__ __forceinline__ pair32 silu(pair32 z) {
  return pair_mul(z, gate(pair_mul(z, twice(-ATLAS_LOG2E))));
}

// ------------------------------------------------------------------ preparation

// Parameters, absent words, sequences' states, tiles' sequences; the states of empty sequences pass on.
static __global__ void __launch_bounds__(256) prepare(GlrArgs a, Space w, long tiles, int groups, int back) {
  const long id = (long)blockIdx.x * 256 + threadIdx.x, n = (long)gridDim.x * 256;
  if (id == 0) w.ticket[0] = w.ticket[1] = 0;
  for (long c = id; c < (long)groups * kCh; c += n) {
    const bool in = c < a.D;
    w.rate[c] = in ? a.c * soft(a.lam[c]) : 0.f;
    w.rb[c] = in && a.rb ? -ATLAS_LOG2E * a.rb[c] : 0.f;
    w.ib[c] = in && a.ib ? -ATLAS_LOG2E * a.ib[c] : 0.f;
  }
  for (long i = id; i < tiles * groups * (kCh / 2); i += n) reinterpret_cast<ulonglong2*>(w.words)[i] = make_ulonglong2(kAbsent, kAbsent);
  const bool packed = a.s.start;
  if (!packed && !a.s.slot && a.s.L > 0) return;
  int rising = a.s.B;
  if (packed) {
    rising = seq_rising(a.s);
    if (blockIdx.x == 0) seq_check(a.s, threadIdx.x, 256);
    for (long k = id; k <= tiles; k += n) {
      const long row = k * kRows < a.s.L ? k * kRows : (long)a.s.L - 1;
      int lo = 0, hi = rising > 0 ? rising - 1 : 0;
      while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (a.s.start[mid] <= row)
          lo = mid;
        else
          hi = mid - 1;
      }
      w.tile_seq[k] = lo;
    }
  }
  const int lane = threadIdx.x & 31;
  for (long b = id / 32; b < a.s.B; b += n / 32) {  // a warp each
    SeqTile t = {};
    t.b = (int)b;
    bool ok = true;
    if (packed) {
      const int s = a.s.start[b], e = a.s.start[b + 1];
      ok = b < rising && s >= 0 && e >= s && e <= a.s.L;
    }
    ok = ok && seq_state(a.s, t);
    if ((packed || a.s.slot) && lane == 0) w.state[b] = ok ? t.slot : -1;
  }
  // the states of empty sequences, 256 channels a warp
  if (!packed && a.s.L > 0) return;
  const long parts = (a.D + 255) / 256;
  for (long task = id / 32; task < a.s.B * parts; task += n / 32) {
    const long b = task / parts;
    SeqTile t = {};
    t.b = (int)b;
    if (packed) {
      const int s = a.s.start[b], e = a.s.start[b + 1];
      if (s != e || b >= rising || s < 0 || e > a.s.L) continue;
    }
    if (!seq_state(a.s, t)) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long c = (task - b * parts) * 256 + i * 32 + lane;
      v[i] = !back && a.h_in && t.carry && c < a.D ? a.h_in[(long)t.slot * a.D + c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const long c = (task - b * parts) * 256 + i * 32 + lane;
      if (c >= a.D) continue;
      if (!back && a.h_out) a.h_out[(long)t.slot * a.D + c] = v[i];
      if (back && a.dh && !t.carry) a.dh[b * a.D + c] = 0.f;
    }
  }
}

// ------------------------------------------------------------------ forward

// A block copies its next tile from when it has this one's maps.  It takes the ticket not before it begins a tile: tickets
// taken earlier would keep tiles waiting for others that no block has begun.
template <typename T, int V, bool FLAT>
__global__ void __launch_bounds__(kThreads, kBlocks) forward_tiles(GlrArgs a, Space w, Strings t) {
  typedef Shape<V> Sh;
  constexpr int S = Sh::S, N = Sh::N;
  extern __shared__ __align__(16) char buf[];  // x, r, i, z twice
  __shared__ float2 s_map[kWarps][kCh];
  __shared__ __align__(16) float s_carry[kWarps][kCh];
  __shared__ Group s_group;
  __shared__ Tile s_tile;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch = lane % Sh::lanes * V, tg = lane / Sh::lanes;
  const int r0 = warp * kPer + tg * S;  // the thread's first row
  const Slots<T, V, S> bx(buf, 0), br(buf, 1), bi(buf, 2);
  const bool gated = a.z && a.y;
  const size_t width = (size_t)t.groups * kCh;
  const auto fetch = [&](const Tile& q, const Info& info, int p) {
    const int c = q.c0 + ch;
    const unsigned live = Info::bits<S>(info.live, tg * S, c < a.D);
    const Cursor<const T, FLAT> px(a.x, a.xb, a.xt, a, c), pr(a.r, a.rbs, a.rt, a, c), pi(a.i, a.ibs, a.it, a, c), pz(a.z, a.zb, a.zt, a, c);
    const Slots<T, V, S> bz(buf, 3 + p);
    const long row = q.row0(a) + r0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int b = FLAT ? 0 : info.seq(tg * S + s);
      if (live >> s & 1) {
        bx.fetch(s, px.at(row + s, b));
        br.fetch(s, pr.at(row + s, b));
        if (a.i) bi.fetch(s, pi.at(row + s, b));
        if (gated) bz.fetch(s, pz.at(row + s, b));
      }
    }
    cp_commit();
  };
  if (threadIdx.x == 0) s_tile.find(t, atomicAdd(w.ticket, 1u), false);
  __syncthreads();
  Tile q = s_tile;
  __syncthreads();  // (the next ticket's tile takes its place; later ones have a pass's other barriers between)
  Info info;
  if (q.some) {
    info.look(a, w, t, q);
    fetch(q, info, 0);
  }
  for (int p = 0; q.some; p ^= 1) {
    unsigned next = 0;
    unsigned long long early = kAbsent;
    if (warp == 0) {  // on their way while the tile is computed
      if (lane == 0) next = atomicAdd(w.ticket, 1u);
      if (t.group == 1 && q.at > 0) early = peek(w.words + q.c0 + lane + (q.first + q.at - 1) * width);
    }
    const int c = q.c0 + ch;
    const unsigned live = Info::bits<S>(info.live, tg * S, c < a.D), first = Info::bits<S>(info.first, tg * S, c < a.D);
    float rate[V], rb[V], ib[V];
    ld_vec<V>(w.rate + c, rate);
    ld_vec<V>(w.rb + c, rb);
    ld_vec<V>(w.ib + c, ib);
    cp_wait<0>();
    // d and u of each element
    float M[N], U[N], top = 0.f;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      pair32 u = bx.two(e);
      const pair32 sv = pair_mul(two<V>(rate, e), gate(pair_fma(br.two(e), twice(-ATLAS_LOG2E), two<V>(rb, e))));
      if (a.i) u = pair_mul(u, gate(pair_fma(bi.two(e), twice(-ATLAS_LOG2E), two<V>(ib, e))));
      float s0, s1;
      unpair(sv, s0, s1);
      top = fmaxf(top, fmaxf(s0, s1));
      const pair32 m = lost(sv);
      unpair(m, M[e], M[e + 1]);
      u = pair_mul(u, root(pair_mul(m, pair_fma(m, twice(-1.f), twice(2.f)))));  // 1 - a^2 = m (2 - m)
      unpair(u, U[e], U[e + 1]);
    }
    // the thread's map of each channel, those of the lanes in front, and the warp's
    float fd[V], fh[V];
    // Rows that are no part of it, first rows and factors that are not near 1 go another way.
    const bool plain = !__any_sync(0xFFFFFFFFu, top >= kSlow || first || live != (1u << S) - 1u);
    if (plain) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Map g{M[v], 1.f - M[v], U[v]};
#pragma unroll
        for (int s = 1; s < S; ++s) {
          const float m = M[s * V + v];
          g.h += fmaf(-m, g.h, U[s * V + v]);
          g.m = fmaf(-m, g.m, g.m + m);
          if (S > 4) g.a = fmaf(-m, g.a, g.a);
        }
        if (S <= 4) g.a = 1.f - g.m;  // 0.17 at least: precise enough
#pragma unroll
        for (int d = Sh::lanes; d < 32; d *= 2) {
          const float pm = __shfl_up_sync(0xFFFFFFFFu, g.m, d), pa = __shfl_up_sync(0xFFFFFFFFu, g.a, d), ph = __shfl_up_sync(0xFFFFFFFFu, g.h, d);
          if (lane >= d) g.follow(pm, pa, ph);
        }
        fd[v] = coded(g.m, g.a), fh[v] = g.h;
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        float s[2], ig[2] = {1.f, 1.f}, xs[2];
        unpair(pair_mul(two<V>(rate, e), gate(pair_fma(br.two(e), twice(-ATLAS_LOG2E), two<V>(rb, e)))), s[0], s[1]);
        unpair(bx.two(e), xs[0], xs[1]);
        if (a.i) unpair(gate(pair_fma(bi.two(e), twice(-ATLAS_LOG2E), two<V>(ib, e))), ig[0], ig[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int f = e + j, row = f / V;
          if (!(s[j] < kSlow)) {
            const float A = kept_of(s[j]);
            M[f] = -A;
            U[f] = xs[j] * ig[j] * root((1.f - A) * (1.f + A));
          }
          if (!(live >> row & 1)) M[f] = kCut, U[f] = 0.f;
          const int b = info.seq(tg * S + row);
          if (first >> row & 1) {
            U[f] = apply(M[f], U[f], start_of(a, w, b, c + f % V));
            M[f] = kCut;
          }
        }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float d = M[v], h = U[v];
#pragma unroll
        for (int s = 1; s < S; ++s) {
          h = apply(M[s * V + v], U[s * V + v], h);
          d = after(M[s * V + v], d);
        }
#pragma unroll
        for (int k = Sh::lanes; k < 32; k *= 2) {
          const float pd = __shfl_up_sync(0xFFFFFFFFu, d, k), ph = __shfl_up_sync(0xFFFFFFFFu, h, k);
          if (lane >= k) {
            h = apply(d, h, ph);
            d = after(d, pd);
          }
        }
        fd[v] = d, fh[v] = h;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (tg == Sh::groups - 1) s_map[warp][ch + v] = make_float2(fd[v], fh[v]);
      if (Sh::groups > 1) {
        fd[v] = __shfl_up_sync(0xFFFFFFFFu, fd[v], Sh::lanes & 31), fh[v] = __shfl_up_sync(0xFFFFFFFFu, fh[v], Sh::lanes & 31);
      }
      if (tg == 0) fd[v] = fh[v] = 0.f;  // nothing in front: the identity
    }
    const unsigned long long* words = w.words + q.c0 + lane;
    const bool last = t.group == 1 || q.at % t.group == t.group - 1;
    bool some = false;
    if (warp == 0) {  // whether a state reaches the tile, and from where in its string
      const int b = info.seq(0);
      some = info.live & ~info.first & 1;
      if (t.group > 1 && lane == 0)
        s_group.begin(t, q, some, t.n > 1 || !some ? 0u : (unsigned)((a.s.start ? (long)a.s.start[b] : (long)b * a.s.L) / kRows));
      if (lane == 0) s_tile.find(t, next, false);
    }
    __syncthreads();
    const Tile q1 = s_tile;
    Info info1;
    if (t.group > 1) {
      if (warp == 1 && !last && !(kWithhold && q.at == 1 && q.c0 == 0)) {  // the tile's own map
        float2 o[kWarps];
#pragma unroll
        for (int i = 0; i < kWarps; ++i) o[i] = s_map[i][lane];
        float2 m = o[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) {
          m.y = apply(o[i].x, o[i].y, m.y);
          m.x = after(o[i].x, m.x);
        }
        post(w.words + q.c0 + lane + (q.first + q.at) * width, word_of(m.x, m.y));
      }
      s_group.gather(q, words, width, w.ticket + 1, a.s.status);
      __syncthreads();
    }
    if (warp == 0) {
      float cin = t.group > 1 ? s_group.carry() : some ? apply(await(words + (q.first + q.at - 1) * width, early, w.ticket + 1, a.s.status), 0.f) : 0.f;
      if (a.kept && q.c0 + lane < a.D) a.kept[(long)q.k * a.D + q.c0 + lane] = cin;
      float2 m[kWarps];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) m[i] = s_map[i][lane];
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        s_carry[i][lane] = cin;
        cin = apply(m[i].x, m[i].y, cin);
      }
      if (last) post(w.words + q.c0 + lane + (q.first + q.at) * width, word_of(kCut, cin));
    }
    if (q1.some) {  // the next tile's rows: x, r and i are in registers, z has another place
      info1.look(a, w, t, q1);
      fetch(q1, info1, p ^ 1);
    }
    __syncthreads();
    float h[V];
    ld_vec<V>(&s_carry[warp][ch], h);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = apply(fd[v], fh[v], h[v]);
    if (plain) {  // U: the states
#pragma unroll
      for (int e = 0; e < N; ++e) {
        h[e % V] += fmaf(-M[e], h[e % V], U[e]);
        U[e] = h[e % V];
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) U[e] = h[e % V] = apply(M[e], U[e], h[e % V]);
    }
    if (a.h_out && info.last) {
      const unsigned last = Info::bits<S>(info.last, tg * S, c < a.D);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int b = info.seq(tg * S + s);
        if (!(last >> s & 1)) continue;
        float* to = a.h_out + (long)state_of(a, w, b) * a.D + c;
#pragma unroll
        for (int v = 0; v < V; ++v) to[v] = U[s * V + v];
      }
    }
    if (a.y) {
      if (gated) {
        const Slots<T, V, S> bz(buf, 3 + p);
#pragma unroll
        for (int e = 0; e < N; e += 2) unpair(pair_mul(pair(U[e], U[e + 1]), silu(bz.two(e))), U[e], U[e + 1]);
      }
      const Cursor<T, FLAT> py(a.y, a.yb, a.yt, a, c);
      const long row = q.row0(a) + r0;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int b = FLAT ? 0 : info.seq(tg * S + s);
        Pack<T, V> y;
        y.pack(U + s * V);
        if (live >> s & 1) st_pack<T, V>(py.at(row + s, b), y);
      }
    }
    q = q1;
    info = info1;
  }
  cp_wait<0>();
}

// Single tokens, a sequence each: no string of maps.
template <typename T, int V>
__global__ void __launch_bounds__(128) forward_token(GlrArgs a) {
  SeqTile t = {};
  t.b = blockIdx.y;
  if (!seq_state(a.s, t)) return;
  const int c = (blockIdx.x * 128 + threadIdx.x) * V;
  if (c >= a.D) return;
  const long b = t.b, at = (long)t.slot * a.D + c;
  Pack<T, V> x = ld_pack<T, V>(reinterpret_cast<const T*>(a.x) + b * a.xb + c), r = ld_pack<T, V>(reinterpret_cast<const T*>(a.r) + b * a.rbs + c), i, z, y;
  i.zero(), z.zero();
  if (a.i) i = ld_pack<T, V>(reinterpret_cast<const T*>(a.i) + b * a.ibs + c);
  if (a.z) z = ld_pack<T, V>(reinterpret_cast<const T*>(a.z) + b * a.zb + c);
  float h[V], rate[V], rb[V], ib[V], o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    h[v] = a.h_in && t.carry ? a.h_in[at + v] : 0.f;
    rate[v] = a.lam[c + v];
    rb[v] = a.rb ? -ATLAS_LOG2E * a.rb[c + v] : 0.f;
    ib[v] = a.ib ? -ATLAS_LOG2E * a.ib[c + v] : 0.f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float sg, open = 1.f, dummy;
    unpair(gate(twice(fmaf(r.get(v), -ATLAS_LOG2E, rb[v]))), sg, dummy);
    if (a.i) unpair(gate(twice(fmaf(i.get(v), -ATLAS_LOG2E, ib[v]))), open, dummy);
    const float s = a.c * soft(rate[v]) * sg;
    const bool slow = s < kSlow;
    const float A = kept_of(s), m = slow ? lost(s) : 1.f - A;
    h[v] = apply(slow ? m : -A, root(m * (2.f - m)) * (open * x.get(v)), h[v]);
    o[v] = a.z ? h[v] * siluf(z.get(v)) : h[v];
    if (a.h_out) a.h_out[at + v] = h[v];
  }
  y.pack(o);
  st_pack<T, V>(reinterpret_cast<T*>(a.y) + b * a.yb + c, y);
}

// ------------------------------------------------------------------ backward

template <typename T>
constexpr int back_stages() {
  return sizeof(T) == 2 ? 2 : 1;
}
template <typename T, int V, bool FLAT>
__global__ void __launch_bounds__(kThreads, kBlocks) backward_tiles(GlrArgs a, Space w, Strings t, const float* kept) {
  typedef Shape<V> Sh;
  constexpr int S = Sh::S, N = Sh::N;
  constexpr bool kAhead = back_stages<T>() == 2;  // the next tile's copies under way (32-bit elements: no room)
  extern __shared__ __align__(16) char buf[];     // [stage]: x, r, i, z, dy
  __shared__ float s_map[3][kWarps][kCh];
  __shared__ __align__(16) float s_carry[2][kWarps][kCh];
  __shared__ float s_sum[kWarps][3][kCh];
  __shared__ Group s_group;
  __shared__ Tile s_tile;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, ch = lane % Sh::lanes * V, tg = lane / Sh::lanes;
  const int r0 = warp * kPer + tg * S;
  const size_t width = (size_t)t.groups * kCh;
  const auto fetch = [&](const Tile& q, const Info& info, int p) {
    const int c = q.c0 + ch;
    char* stage = buf + (kAhead ? p : 0) * slots_bytes<T>(5);
    const Slots<T, V, S> bx(stage, 0), br(stage, 1), bi(stage, 2), bz(stage, 3), by(stage, 4);
    const unsigned live = Info::bits<S>(info.live, tg * S, c < a.D);
    const Cursor<const T, FLAT> px(a.x, a.xb, a.xt, a, c), pr(a.r, a.rbs, a.rt, a, c), pi(a.i, a.ibs, a.it, a, c), pz(a.z, a.zb, a.zt, a, c),
        py(a.dy, a.yb, a.yt, a, c);
    const long row = q.row0(a) + r0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int b = FLAT ? 0 : info.seq(tg * S + s);
      if (live >> s & 1) {
        bx.fetch(s, px.at(row + s, b));
        br.fetch(s, pr.at(row + s, b));
        by.fetch(s, py.at(row + s, b));
        if (a.i) bi.fetch(s, pi.at(row + s, b));
        if (a.z) bz.fetch(s, pz.at(row + s, b));
      }
    }
    cp_commit();
  };
  if (threadIdx.x == 0) s_tile.find(t, atomicAdd(w.ticket, 1u), true);
  __syncthreads();
  Tile q = s_tile;
  __syncthreads();  // (the next ticket's tile takes its place; later ones have a pass's other barriers between)
  Info info;
  if (q.some) {
    info.look(a, w, t, q);
    fetch(q, info, 0);
  }
  for (int p = 0; q.some; p ^= 1) {
    unsigned next = 0;
    unsigned long long early = kAbsent;
    if (warp == kWarps - 1) {
      if (lane == 0) next = atomicAdd(w.ticket, 1u);
      if (t.group == 1 && q.at > 0) early = peek(w.words + q.c0 + lane + (q.first + q.at - 1) * width);
    }
    const int c = q.c0 + ch;
    char* stage = buf + (kAhead ? p : 0) * slots_bytes<T>(5);
    const Slots<T, V, S> bx(stage, 0), br(stage, 1), bi(stage, 2), bz(stage, 3), by(stage, 4);
    const unsigned live = Info::bits<S>(info.live, tg * S, c < a.D), first = Info::bits<S>(info.first, tg * S, c < a.D),
                   last = Info::bits<S>(info.last, tg * S, c < a.D);
    float rate[V], rb[V], ib[V];
    ld_vec<V>(w.rate + c, rate);
    ld_vec<V>(w.rb + c, rb);
    ld_vec<V>(w.ib + c, ib);
    cp_wait<0>();
    float M[N], U[N], G[N], top = 0.f;
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      pair32 u = bx.two(e), g = by.two(e);
      const pair32 sv = pair_mul(two<V>(rate, e), gate(pair_fma(br.two(e), twice(-ATLAS_LOG2E), two<V>(rb, e))));
      if (a.i) u = pair_mul(u, gate(pair_fma(bi.two(e), twice(-ATLAS_LOG2E), two<V>(ib, e))));
      if (a.z) g = pair_mul(g, silu(bz.two(e)));
      float s0, s1;
      unpair(sv, s0, s1);
      const pair32 m = lost(sv);
      unpair(m, M[e], M[e + 1]);
      u = pair_mul(u, root(pair_mul(m, pair_fma(m, twice(-1.f), twice(2.f)))));
      unpair(u, U[e], U[e + 1]);
      unpair(g, G[e], G[e + 1]);
      top = fmaxf(top, fmaxf(s0, s1));
    }
    // plain: all rows take part, none is a first one (of which the factor is cut for what passes, but not for its own
    // gradient), all factors are near 1
    const bool plain = !__any_sync(0xFFFFFFFFu, top >= kSlow || first || live != (1u << S) - 1u);
    if (!plain) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        float s[2], ig[2] = {1.f, 1.f}, xs[2];
        unpair(pair_mul(two<V>(rate, e), gate(pair_fma(br.two(e), twice(-ATLAS_LOG2E), two<V>(rb, e)))), s[0], s[1]);
        unpair(bx.two(e), xs[0], xs[1]);
        if (a.i) unpair(gate(pair_fma(bi.two(e), twice(-ATLAS_LOG2E), two<V>(ib, e))), ig[0], ig[1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int f = e + j;
          if (!(s[j] < kSlow)) {
            const float A = kept_of(s[j]);
            M[f] = -A;
            U[f] = xs[j] * ig[j] * root((1.f - A) * (1.f + A));
          }
          if (!(live >> f / V & 1)) M[f] = kCut, U[f] = G[f] = 0.f;
        }
      }
    }
    if (a.dh && info.last) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int b = info.seq(tg * S + s);
        if (!(last >> s & 1)) continue;
#pragma unroll
        for (int v = 0; v < V; ++v) G[s * V + v] += a.dh[(long)b * a.D + c + v];
      }
    }
    // forward: the maps of the lanes in front; in reverse: of those behind
    float fd[V], fh[V], bd[V], bc[V];
    if (plain) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Map f{M[v], 1.f - M[v], U[v]};
#pragma unroll
        for (int s = 1; s < S; ++s) {
          const float m = M[s * V + v];
          f.h += fmaf(-m, f.h, U[s * V + v]);
          f.m = fmaf(-m, f.m, f.m + m);
          if (S > 4) f.a = fmaf(-m, f.a, f.a);
        }
        if (S <= 4) f.a = 1.f - f.m;
        Map r{f.m, f.a, 0.f};
#pragma unroll
        for (int s = S - 1; s >= 0; --s) {
          const float x = G[s * V + v] + r.h;
          r.h = fmaf(-M[s * V + v], x, x);
        }
#pragma unroll
        for (int d = Sh::lanes; d < 32; d *= 2) {
          const float pm = __shfl_up_sync(0xFFFFFFFFu, f.m, d), pa = __shfl_up_sync(0xFFFFFFFFu, f.a, d), ph = __shfl_up_sync(0xFFFFFFFFu, f.h, d);
          const float nm = __shfl_down_sync(0xFFFFFFFFu, r.m, d), na = __shfl_down_sync(0xFFFFFFFFu, r.a, d), nh = __shfl_down_sync(0xFFFFFFFFu, r.h, d);
          if (lane >= d) f.follow(pm, pa, ph);
          if (lane + d < 32) r.follow(nm, na, nh);
        }
        fd[v] = coded(f.m, f.a), fh[v] = f.h;
        bd[v] = coded(r.m, r.a), bc[v] = r.h;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float d = 0.f, h = 0.f, g = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
          const int e = s * V + v, b = info.seq(tg * S + s);
          if (first >> s & 1) {
            h = apply(M[e], U[e], start_of(a, w, b, c + v));
            d = kCut;
          } else {
            h = apply(M[e], U[e], h);
            d = after(M[e], d);
          }
        }
#pragma unroll
        for (int s = S - 1; s >= 0; --s) g = first >> s & 1 ? 0.f : apply(M[s * V + v], 0.f, G[s * V + v] + g);
        float r = d;
#pragma unroll
        for (int k = Sh::lanes; k < 32; k *= 2) {
          const float pd = __shfl_up_sync(0xFFFFFFFFu, d, k), ph = __shfl_up_sync(0xFFFFFFFFu, h, k);
          const float nd = __shfl_down_sync(0xFFFFFFFFu, r, k), ng = __shfl_down_sync(0xFFFFFFFFu, g, k);
          if (lane >= k) {
            h = apply(d, h, ph);
            d = after(d, pd);
          }
          if (lane + k < 32) {
            g = apply(r, g, ng);
            r = after(r, nd);
          }
        }
        fd[v] = d, fh[v] = h, bd[v] = r, bc[v] = g;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (tg == Sh::groups - 1) s_map[0][warp][ch + v] = fd[v], s_map[1][warp][ch + v] = fh[v];
      if (tg == 0) s_map[2][warp][ch + v] = bc[v];
      if (Sh::groups > 1) {
        fd[v] = __shfl_up_sync(0xFFFFFFFFu, fd[v], Sh::lanes & 31), fh[v] = __shfl_up_sync(0xFFFFFFFFu, fh[v], Sh::lanes & 31);
        bd[v] = __shfl_down_sync(0xFFFFFFFFu, bd[v], Sh::lanes & 31), bc[v] = __shfl_down_sync(0xFFFFFFFFu, bc[v], Sh::lanes & 31);
      }
      if (tg == 0) fd[v] = fh[v] = 0.f;
      if (tg == Sh::groups - 1) bd[v] = bc[v] = 0.f;
    }
    const unsigned long long* words = w.words + q.c0 + lane;
    const bool end = t.group == 1 || q.at % t.group == t.group - 1;
    bool some = false;
    if (warp == kWarps - 1) {  // whether a gradient reaches the tile, and from where in its string (its rows are the last)
      const int b = info.seq(kPer - 1);
      some = (info.live & ~info.last) >> (kPer - 1) & 1;
      if (t.group > 1 && lane == 0)
        s_group.begin(t, q, some, t.n > 1 || !some ? 0u : t.tiles - 1 - (unsigned)(((a.s.start ? (long)a.s.start[b + 1] : (long)(b + 1) * a.s.L) - 1) / kRows));
      if (lane == 0) s_tile.find(t, next, true);
    }
    __syncthreads();
    const Tile q1 = s_tile;
    Info info1;
    if (t.group > 1) {
      if (warp == 1 && !end) {
        float d = s_map[0][kWarps - 1][lane], g = s_map[2][kWarps - 1][lane];
#pragma unroll
        for (int i = kWarps - 2; i >= 0; --i) {
          g = apply(s_map[0][i][lane], s_map[2][i][lane], g);
          d = after(s_map[0][i][lane], d);
        }
        post(w.words + q.c0 + lane + (q.first + q.at) * width, word_of(d, g));
      }
      s_group.gather(q, words, width, w.ticket + 1, a.s.status);
      __syncthreads();
    }
    if (warp == 0) {  // the states in front of the warps
      float h = q.c0 + lane < a.D ? kept[(long)q.k * a.D + q.c0 + lane] : 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        s_carry[0][i][lane] = h;
        h = apply(s_map[0][i][lane], s_map[1][i][lane], h);
      }
    } else if (warp == kWarps - 1) {  // the gradients behind them
      float cin = t.group > 1 ? s_group.carry() : some ? apply(await(words + (q.first + q.at - 1) * width, early, w.ticket + 1, a.s.status), 0.f) : 0.f;
#pragma unroll
      for (int i = kWarps - 1; i >= 0; --i) {
        s_carry[1][i][lane] = cin;
        cin = apply(s_map[0][i][lane], s_map[2][i][lane], cin);
      }
      if (end) post(w.words + q.c0 + lane + (q.first + q.at) * width, word_of(kCut, cin));
    }
    if (q1.some) {
      info1.look(a, w, t, q1);
      if (kAhead) fetch(q1, info1, p ^ 1);
    }
    __syncthreads();
    float h[V], g[V], sum[3][V];
    ld_vec<V>(&s_carry[0][warp][ch], h);
    ld_vec<V>(&s_carry[1][warp][ch], g);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      h[v] = apply(fd[v], fh[v], h[v]);
      g[v] = apply(bd[v], bc[v], g[v]);
      sum[0][v] = sum[1][v] = sum[2][v] = 0.f;
    }
    // G: dL/dh of each token
    if (plain) {
#pragma unroll
      for (int e = N - 1; e >= 0; --e) {
        G[e] += g[e % V];
        g[e % V] = fmaf(-M[e], G[e], G[e]);
      }
    } else {
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        const int b = info.seq(tg * S + s);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int e = s * V + v;
          if (live >> s & 1) G[e] += g[v];
          g[v] = apply(M[e], 0.f, G[e]);
          if (first >> s & 1) {
            if (a.dh) a.dh[(long)b * a.D + c + v] = a.s.carry && !a.s.carry[b] ? 0.f : g[v];
            g[v] = 0.f;
          }
        }
      }
    }
    const Cursor<T, FLAT> ox(a.dx, a.xb, a.xt, a, c), orr(a.dr, a.rbs, a.rt, a, c), oi(a.di, a.ibs, a.it, a, c), oz(a.dz, a.zb, a.zt, a, c);
    const long row0 = q.row0(a) + r0;
    constexpr int P = V > 1 ? 1 : 2;  // rows that a step takes, whose elements are pairs
    // Two copies: what the other way asks for is a tenth of this one's instructions.  The other is a loop, its values in local
    // memory: run by few warps, and longer than what it would share the instruction cache with (unrolled too: 706 us for 695,
    // of packed documents 239 for 235).
    const auto put = [&](auto is_plain) {
      constexpr bool kPlain = decltype(is_plain)::value;
      constexpr int kUnroll = kPlain ? S / P : 1;
      float lM[N], lU[N], lG[N];
#pragma unroll
      for (int e = 0; e < N; ++e) lM[e] = M[e], lU[e] = U[e], lG[e] = G[e];
#pragma unroll kUnroll
      for (int s = 0; s < S; s += P) {
        float before[P * V], here[P * V], dx[P * V], dr[P * V], di[P * V], dz[P * V];
#pragma unroll
        for (int f = 0; f < P * V; ++f) {
          const int e = s * V + f, v = f % V;
          if (!kPlain) {
            const int b = info.seq(tg * S + e / V);
            if (first >> e / V & 1) h[v] = start_of(a, w, b, c + v);
          }
          before[f] = h[v];
          if (kPlain)
            h[v] += fmaf(-lM[e], h[v], lU[e]);
          else
            h[v] = apply(lM[e], lU[e], h[v]);
          here[f] = h[v];
        }
#pragma unroll
        for (int f = 0; f < P * V; f += 2) {
          const int e = s * V + f, v = f % V;
          const pair32 G2 = pair(lG[e], lG[e + 1]), U2 = pair(lU[e], lU[e + 1]);
          pair32 rrest, irest = twice(0.f), m = pair(lM[e], lM[e + 1]), ig = twice(1.f), A2;
          const pair32 rg = gate<true>(pair_fma(br.two(e), twice(-ATLAS_LOG2E), two<V>(rb, e)), rrest);
          if (a.i) ig = gate<false>(pair_fma(bi.two(e), twice(-ATLAS_LOG2E), two<V>(ib, e)), irest);
          const pair32 sv = pair_mul(two<V>(rate, e), rg);
          if (kPlain) {
            A2 = pair_fma(m, twice(-1.f), twice(1.f));
          } else {
            const float a0 = factor(lM[e]), a1 = factor(lM[e + 1]);
            A2 = pair(a0, a1);
            m = pair(is_kept(lM[e]) ? 1.f - a0 : lM[e], is_kept(lM[e + 1]) ? 1.f - a1 : lM[e + 1]);
          }
          const pair32 b2 = pair_mul(m, pair_fma(m, twice(-1.f), twice(2.f)));
          float q0, q1;
          unpair(b2, q0, q1);
          // s / beta^2 is 1/2 in the limit of s = 0, where u is 0 too
          const pair32 ratio = pair_mul(sv, pair(rcp(fmaxf(q0, 1e-37f)), rcp(fmaxf(q1, 1e-37f))));
          // Q = G (u a^2 ratio - s a h) = G a (u a ratio - s h)
          const pair32 in2 = pair_fma(pair_mul(U2, A2), ratio, pair_mul(pair_mul(sv, twice(-1.f)), pair(before[f], before[f + 1])));
          pair32 Q = pair_mul(pair_mul(G2, A2), in2), r2 = pair_mul(Q, rrest), i2 = pair_mul(pair_mul(G2, U2), irest);
          unpair(r2, dr[f], dr[f + 1]);
          unpair(i2, di[f], di[f + 1]);
          unpair(pair_mul(pair_mul(G2, root(b2)), ig), dx[f], dx[f + 1]);
          if (a.z) {
            const pair32 zv = bz.two(e);
            pair32 zr;
            const pair32 zg = gate<true>(pair_mul(zv, twice(-ATLAS_LOG2E)), zr);
            const pair32 slope = pair_mul(zg, pair_fma(zv, zr, twice(1.f)));
            unpair(pair_mul(pair_mul(by.two(e), pair(here[f], here[f + 1])), slope), dz[f], dz[f + 1]);
          }
          if (!kPlain) {  // a slot without a row may hold anything
            const float l0 = live >> e / V & 1 ? 1.f : 0.f, l1 = live >> (e + 1) / V & 1 ? 1.f : 0.f;
            const auto masked = [&](pair32 x) {
              float x0, x1;
              unpair(x, x0, x1);
              return pair(l0 != 0.f ? x0 : 0.f, l1 != 0.f ? x1 : 0.f);
            };
            Q = masked(Q), r2 = masked(r2), i2 = masked(i2);
          }
          const auto add = [&](float* to, pair32 x) {
            if (V > 1)
              unpair(pair_add(pair(to[v], to[v + (V > 1)]), x), to[v], to[v + (V > 1)]);
            else
              to[0] += pair_sum(x);
          };
          add(sum[0], Q);
          add(sum[1], r2);
          add(sum[2], i2);
        }
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const int b = FLAT ? 0 : info.seq(tg * S + s + j);
          if (!kPlain && !(live >> (s + j) & 1)) continue;
          const long row = row0 + s + j;
          Pack<T, V> o;
          o.pack(dx + j * V);
          st_pack<T, V>(ox.at(row, b), o);
          o.pack(dr + j * V);
          st_pack<T, V>(orr.at(row, b), o);
          if (a.i) {
            o.pack(di + j * V);
            st_pack<T, V>(oi.at(row, b), o);
          }
          if (a.z) {
            o.pack(dz + j * V);
            st_pack<T, V>(oz.at(row, b), o);
          }
        }
      }
    };
    if (plain)
      put(std::true_type());
    else
      put(std::false_type());
#pragma unroll
    for (int j = 0; j < 3; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int d = Sh::lanes; d < 32; d *= 2) sum[j][v] += __shfl_xor_sync(0xFFFFFFFFu, sum[j][v], d);
        if (tg == 0) s_sum[warp][j][ch + v] = sum[j][v];
      }
    __syncthreads();
    if (threadIdx.x < 3 * kCh) {
      const int j = threadIdx.x / kCh, cl = threadIdx.x % kCh;
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) x += s_sum[i][j][cl];
      if (q.c0 + cl < a.D) w.sums[((long)q.k * 3 + j) * a.D + q.c0 + cl] = x;
    }
    q = q1;
    info = info1;
    if (!kAhead && q.some) fetch(q, info, p ^ 1);
  }
  cp_wait<0>();
}

// dlambda and the biases' gradients from the tiles' sums; 32 channels a block, 32 threads each.
static __global__ void __launch_bounds__(1024) add_sums(GlrArgs a, const float* sums, long tiles) {
  __shared__ float s[32][33];
  const int j = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  float* out = j == 0 ? a.dlam : j == 1 ? a.drb : a.dib;
  if (!out) return;
  float v = 0.f;
  if (c < a.D) {
#pragma unroll 4
    for (long k = threadIdx.y; k < tiles; k += 32) v += sums[(k * 3 + j) * a.D + c];
  }
  s[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < a.D) {
#pragma unroll
    for (int i = 1; i < 32; ++i) v += s[i][threadIdx.x];
    out[c] = j == 0 ? v * soft_ratio(a.lam[c]) : v;
  }
}

// ------------------------------------------------------------------ launches

inline int status() { return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA; }

inline int run_prepare(const GlrArgs& a, const Space& w, bool back, cudaStream_t st) {
  const long tiles = tiles_of(a), fill = tiles * groups_of(a) * (kCh / 2), tasks = (long)a.s.B * (a.s.start ? 1 + (a.D + 255) / 256 : 1) * 32;
  long n = (fill / 4 > tasks ? fill / 4 : tasks) / 256 + 1;
  n = n < 4L * kSMs ? n : 4L * kSMs;
  prepare<<<(unsigned)n, 256, 0, st>>>(a, w, tiles, groups_of(a), back);
  return status();
}

// Whether sequences lie one behind the other in every tensor, and offsets of rows are products of 32-bit numbers.
inline bool flat(const GlrArgs& a, int e) {
  const long st[] = {a.xt, a.rt, a.it, a.zt, a.yt}, sb[] = {a.xb, a.rbs, a.ibs, a.zb, a.yb};
  for (int i = 0; i < 5; ++i) {
    if (!a.s.start && a.s.B > 1 && sb[i] != st[i] * a.s.L) return false;
    if (st[i] * e > 0xFFFFFFFFL) return false;
  }
  return rows_of(a) < 0x7FFFFFFFL;
}

template <typename F, typename... X>
int launch(F* f, int smem, const Strings& t, cudaStream_t st, X... args) {
  if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return ATLAS_ERR_CUDA;
  const unsigned most = kBlocks * kSMs;
  f<<<t.total < most ? t.total : most, kThreads, smem, st>>>(args...);
  return status();
}

// The forward pass over tiles; y null: the kept states alone.
template <typename T, int V>
int forward(const GlrArgs& a, const Space& w, cudaStream_t st) {
  if (const int rc = run_prepare(a, w, false, st)) return rc;
  if (tiles_of(a) == 0) return ATLAS_OK;
  const Strings t = strings(a);
  return launch(flat(a, sizeof(T)) ? forward_tiles<T, V, true> : forward_tiles<T, V, false>, slots_bytes<T>(5), t, st, a, w, t);
}

template <typename T, int V>
int run_forward(const GlrArgs& a, cudaStream_t st) {
  if (!a.s.start && a.s.L == 1 && a.y) {
    forward_token<T, V><<<dim3((a.D - 1) / (128 * V) + 1, a.s.B), 128, 0, st>>>(a);
    return status();
  }
  return forward<T, V>(a, space(a, false, false), st);
}

template <typename T, int V>
int run_backward(const GlrArgs& a, cudaStream_t st) {
  const Space w = space(a, true, !a.kept);
  const float* kept = a.kept;
  const bool some = tiles_of(a) > 0;
  if (!kept && some) {  // the forward pass once more, for the kept states alone
    GlrArgs f = a;
    f.y = nullptr;
    f.h_out = nullptr;
    f.kept = w.kept;
    if (const int rc = forward<T, V>(f, w, st)) return rc;
    kept = w.kept;
  }
  if (const int rc = run_prepare(a, w, true, st)) return rc;
  if (some) {
    const Strings t = strings(a);
    const int smem = slots_bytes<T>(5) * back_stages<T>();
    if (const int rc = launch(flat(a, sizeof(T)) ? backward_tiles<T, V, true> : backward_tiles<T, V, false>, smem, t, st, a, w, t, kept)) return rc;
  }
  add_sums<<<dim3((a.D + 31) / 32, 3), dim3(32, 32), 0, st>>>(a, w.sums, tiles_of(a));
  return status();
}

template <typename T, int V>
int run(const GlrArgs& a, bool back, cudaStream_t st) {
  return back ? run_backward<T, V>(a, st) : run_forward<T, V>(a, st);
}
template <typename T>
int run(const GlrArgs& a, bool back, cudaStream_t st) {
  return a.wide == 4 ? run<T, 4>(a, back, st) : a.wide == 2 ? run<T, 2>(a, back, st) : run<T, 1>(a, back, st);
}

}  // namespace glr
}  // namespace atlas
