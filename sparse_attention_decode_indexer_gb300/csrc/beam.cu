// beam.cu -- the next tokens of beams: the best (beam, token) pairs of every
// group, and the beams' states in their new order.
//
// With x[r][t] the logits of beam r, a candidate's score is
//   score[r] + x[r][t] - ln sum_t' exp(x[r][t']);
// a beam that has ended has one candidate, (r, eos) at score[r].  The K = beams
// best of a group win, the first beam and then the first token among equals.
//
// What bounds it: the logits, read once.  A CTA takes a part of a row, 64 bytes a
// thread at a time with the next 64 in flight, and leaves the sum of their
// exponentials and the K best; the last CTA of a group (a ticket) puts these
// together.  41 M logits are 270,000 to an SM, so every instruction per logit
// counts: 16-bit logits stay in words, two to a maximum, and the exponential is
// one product, 2^(x log2e - c).
//
// The K best of what the threads of a CTA hold: the greatest of each four
// threads; the K-th of these 64 is a bound that at least K values reach, and so
// is the K-th best of the chunks before.  The values that reach it, few more
// than K, go to a list, in which each finds its rank by counting; values are
// compared together with their index, so no two are equal and the order of the
// list does not matter.  Where many values equal the bound (a mask of one finite
// value) the list would overflow: then the bound is taken over (value, index) of
// each thread, which at most K threads' values reach.
//
// Sums are 64-bit integers in units of 2^-40, which do not depend on any order.  The
// reference moves when a thread's sum of a chunk passes its number of logits, so the
// terms average at most one and 2^23 of them come to 2^63.  Double arithmetic (two
// operations a clock and SM here) makes the logarithms and adds the scores, so that
// candidates of different beams are ordered by what they are and not by a rounding
// to fp32: an exponential is off by about 2^-22, an average over many by less.
// 2^(x L), L = log2e rounded to fp32, in place of e^x is off by 2e-8 of the row's
// entropy.
//
// Measured: 32 x 8 beams of 160,000 bf16 logits, histories of 4,096: 38 us (82 MB, 12
// at the copy rate; 300 instructions a warp and chunk at 0.42 of the issue rate);
// 64 x 1 of 131,072: 13 us; 1 x 4 of 32,000: 10.7 us, of which the last CTA's choice
// is 5 (64 us for the first of these before loads went out together and double
// comparisons became integers, 231 at first).  Chunks of 64 bytes a thread: two more
// in flight through shared memory measured the same (39).  64 registers allow four
// CTAs; the 16-bit kernels spill 32 bytes for it.
// Beyond 2^20 (masks of some large number) c, an fp32 product, would no longer be
// the logit it stands for: there sums are taken against the logit itself.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "rope.cuh"

namespace ssa {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 4;                  // per SM
constexpr int kBytes = 64;                // of a chunk of logits, a thread
constexpr int kMaxBeams = 32;
constexpr int kMaxGroups = 65535;
constexpr int kMaxLists = 1024;           // (row, part) lists of a group
constexpr int kList = kMaxBeams * 33;     // values in a CTA's list: K threads' 32, and K kept
constexpr int kFinal = 512;               // candidates in a group's list
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGreatest = 0x1p126f;     // logits above it count as it: its product with kLog2e is finite
constexpr float kUnit = 0x1p40f;          // of the sums
constexpr float kFar = 0x1p20f;           // references further out are logits, not octaves

struct Part {                             // of a row: sum * 2^(c - 40) is its sum of 2^(x kLog2e)
  uint64_t sum;
  float c;                                // -infinity: no logit
  float ref;                              // the reference as a logit, where it is beyond kFar; else infinity
};
struct Cand {                             // logit and token; token < 0: none
  float x;
  int t;
};

struct Params {
  const void* logits;
  int64_t stride;
  int K, V, parts, chunks, max_len, eos;  // parts of a row, chunks of a part
  const float* scores;
  const uint8_t* ended;
  const int32_t *history, *hist_len, *seq_lens;
  float* scores_out;
  uint8_t* ended_out;
  int32_t *history_out, *hist_len_out, *new_lens, *parent, *token;
  int32_t* status;
  Part* part;                             // [row][part]
  Cand* cand;                             // [row][part][K]
  int32_t* ticket;                        // [group], zero between calls
  int32_t* old_len;                       // [group], for the kernel that moves the histories
  int move_here;                          // histories are moved by the group's last CTA
};

// Numbers in their order as integers: the larger, the greater.
__device__ __forceinline__ uint32_t rank32(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unrank32(uint32_t b) {
  return __uint_as_float(b ^ ((int32_t)b < 0 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ uint64_t rank64(double x) {
  const uint64_t b = (uint64_t)__double_as_longlong(x);
  return b ^ ((int64_t)b < 0 ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unrank64(uint64_t b) {
  return __longlong_as_double((int64_t)(b ^ ((int64_t)b < 0 ? 1ull << 63 : ~0ull)));
}
// A logit and its token (or another index): the greater logit, then the lower index.
// (The sum makes both zeros one.)
__device__ __forceinline__ uint64_t key_of(float x, uint32_t t) {
  return (uint64_t)rank32(x + 0.0f) << 32 | (uint32_t)~t;
}
__device__ __forceinline__ float key_x(uint64_t k) { return unrank32((uint32_t)(k >> 32)); }

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// A thread's logits of a chunk, in 16-byte pieces 16 * kThreads bytes apart.
template <typename T> struct Logits {
  static constexpr int N = 16 / sizeof(T);              // of a piece
  static constexpr int W = kBytes / 4;                  // words
  static constexpr int M = kBytes / sizeof(T);          // logits
  static constexpr int kChunk = M * kThreads;
  uint32_t w[W];

  static __device__ __forceinline__ float lowest() {    // that is finite
    if constexpr (sizeof(T) == 4) return -FLT_MAX;
    else return std::is_same_v<T, __half> ? -65504.0f : -0x1.FEp127f;
  }
  static __device__ __forceinline__ uint32_t none() {   // a word of -infinity
    if constexpr (sizeof(T) == 4) return 0xFF800000u;
    else return std::is_same_v<T, __half> ? 0xFC00FC00u : 0xFF80FF80u;
  }
  __device__ __forceinline__ void load(const T* row, long long first, int V, bool vec) {
#pragma unroll
    for (int j = 0; j < M / N; ++j) {
      const long long at = first + (j * kThreads + (int)threadIdx.x) * N;
      if (vec && at + N <= V) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + at));
        w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[4 * j + i] = none();
          if constexpr (sizeof(T) == 4) {
            if (at + i < V) w[4 * j + i] = __float_as_uint(row[at + i]);
          } else {
            const uint16_t* h = reinterpret_cast<const uint16_t*>(row);
            uint32_t lo = none() & 0xFFFFu, hi = lo;
            if (at + 2 * i < V) lo = h[at + 2 * i];
            if (at + 2 * i + 1 < V) hi = h[at + 2 * i + 1];
            w[4 * j + i] = lo | hi << 16;
          }
        }
      }
    }
  }
  // the greatest, NaN aside
  __device__ __forceinline__ float most() const {
    if constexpr (sizeof(T) == 4) {
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < W; ++i) m[i & 3] = fmaxf(m[i & 3], __uint_as_float(w[i]));
      return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    } else {
      uint32_t m = none();
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if constexpr (std::is_same_v<T, __half>) asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
        else asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
      }
      const float2 f = unpack<T>(m);
      return fmaxf(f.x, f.y);
    }
  }
  // f(logit, its place in the thread's order)
  template <typename F> __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(T) == 4) {
        f(__uint_as_float(w[i]), i);
      } else {
        const float2 x = unpack<T>(w[i]);
        f(x.x, 2 * i);
        f(x.y, 2 * i + 1);
      }
    }
  }
  // the sum of 2^(x kLog2e - c)
  __device__ __forceinline__ float sum(float c) const {
    const uint64_t l2 = pack2(kLog2e, kLog2e), c2 = pack2(-c, -c);
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < M / 2; ++i) {
      uint64_t x;
      if constexpr (sizeof(T) == 4) {
        x = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      } else {
        const float2 f = unpack<T>(w[i]);
        x = pack2(f.x, f.y);
      }
      const float2 t = unpack2(fma2(x, l2, c2));
      s[i & 1] = add2(s[i & 1], pack2(fast_exp2(t.x), fast_exp2(t.y)));
    }
    const float2 r = unpack2(add2(s[0], s[1]));
    return r.x + r.y;
  }
  // the same, NaN aside
  __device__ __forceinline__ float sum_clean(float c) const {
    float s = 0.0f;
    each([&](float v, int) {
      if (v == v) s += fast_exp2(fmaf(v, kLog2e, -c));
    });
    return s;
  }
  // the sum of e^(x - ref), NaN aside: any magnitude
  __device__ __forceinline__ float sum_from(float ref) const {
    float s = 0.0f;
    each([&](float v, int) {
      if (v == v) s += fast_exp2((fminf(v, kGreatest) - ref) * kLog2e);
    });
    return s;
  }
  // which of them are at least `least` (never a NaN): bit i the thread's i-th
  __device__ __forceinline__ uint32_t reach(float least) const {
    uint32_t bits = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) bits |= __uint_as_float(w[i]) >= least ? 1u << i : 0u;
    } else {
      const uint32_t l = pack<T>(least, least);          // exact, or (fp16) infinity
#pragma unroll
      for (int i = 0; i < W; ++i) {
        uint32_t m;
        if constexpr (std::is_same_v<T, __half>)
          m = __hge2_mask(*reinterpret_cast<const __half2*>(&w[i]), *reinterpret_cast<const __half2*>(&l));
        else
          m = __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), *reinterpret_cast<const __nv_bfloat162*>(&l));
        bits |= m & (1u << i | 0x10000u << i);           // the even ones low, the odd ones high
      }
    }
    return bits;
  }
  // the logit at a place (registers have no index: a chain of selects)
  __device__ __forceinline__ float at(int place) const {
    const int j = sizeof(T) == 4 ? place : place >> 1;
    uint32_t v = w[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v = j == i ? w[i] : v;
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(v);
    } else {
      const float2 f = unpack<T>(v);
      return place & 1 ? f.y : f.x;
    }
  }
  // the place of a bit of reach()
  static __device__ __forceinline__ int place(int bit) {
    return sizeof(T) == 4 ? bit : (bit & 15) * 2 + (bit >> 4);
  }
  static __device__ __forceinline__ int token(int first, int i) {
    return first + ((i / N) * kThreads + (int)threadIdx.x) * N + i % N;
  }
};

// A reference of a sum in octaves: whole ones, or a far logit's.
__device__ __forceinline__ double octaves(float c, float far) {
  return far < INFINITY ? (double)far * (double)kLog2e : (double)c;
}
// A sum beside the reference (c, far) as one beside (c1, far1), which is not below it
// but for the rounding of a far c.  Whole octaves are a shift; between far references a
// part of an octave is left.
__device__ __forceinline__ uint64_t beside(uint64_t z, float c, float far, float c1, float far1) {
  if (!(far < INFINITY) && !(far1 < INFINITY)) return z >> (int)fminf(c1 - c, 63.0f);
  const double d = octaves(c1, far1) - octaves(c, far);
  if (!(d < 63.0)) return 0;
  const int n = max((int)d, 0);
  const uint64_t f = (uint64_t)(exp2f((float)((double)n - d)) * 0x1p31f);     // at most a little above 2^31
  return __umul64hi(z >> n, f << 32) << 1;
}

struct Score {                            // of a candidate, and its place in the group
  uint64_t s;                             // rank64 of the score; 0: none
  uint64_t at;                            // row << 32 | token
};
__device__ __forceinline__ bool better(const Score& a, const Score& b) {
  return a.s > b.s || (a.s == b.s && a.at < b.at);
}

// Scratch of a CTA: its list, or the group's.
union Scratch {
  uint64_t list[kList];
  Score score[kFinal];
  int32_t move[2048];
};

// ln z, z > 0, to about 2^-35: z = 2^e m with m about one, ln m = 2 atanh(s), s =
// (m - 1) / (m + 1), |s| < 0.172; the series' first two terms in double.  A
// double operation takes an SM 16 clocks a warp, so few of them.
__device__ __forceinline__ double ln_of(uint64_t z) {
  const int lead = __clzll((long long)z);
  const uint64_t f = z << lead;           // the leading bit on top
  const bool high = f >= 0xB504F333F9DE6485ull;           // above sqrt(2)
  const int e = 63 - lead + (high ? 1 : 0);
  const double m = __longlong_as_double((long long)(((high ? 1022ull : 1023ull) << 52) | (f << 1 >> 12)));
  const double d = m + 1.0;
  double r = (double)(1.0f / (float)d);
  r = fma(r, fma(-d, r, 1.0), r);
  const double s = (m - 1.0) * r;
  const float t = (float)s, t2 = t * t;
  const float tail = t2 * t2 * t * fmaf(t2, fmaf(t2, fmaf(t2, fmaf(t2, 1.0f / 13, 1.0f / 11), 1.0f / 9), 1.0f / 7), 0.2f);
  const double sum = s + (s * s * s * (1.0 / 3) + (double)tail);
  return fma((double)e, 0.69314718055994530942, 2.0 * sum);
}

// The K-th greatest of the threads' numbers (0: none), or something below it that
// no more than K reach; N numbers a thread.
template <int N> __device__ __forceinline__ uint32_t kth(const uint32_t (&x)[N], int K) {
  __shared__ uint32_t s_and, s_or;
  if (threadIdx.x == 0) { s_and = ~0u; s_or = 0; }
  uint32_t all = ~0u, any = 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (x[i]) { all &= x[i]; any |= x[i]; }
  all = __reduce_and_sync(0xffffffffu, all);
  any = __reduce_or_sync(0xffffffffu, any);
  __syncthreads();
  if ((threadIdx.x & 31) == 0 && any) { atomicAnd(&s_and, all); atomicOr(&s_or, any); }
  __syncthreads();
  // the leading bits that all have in common need no search
  const uint32_t differ = s_and ^ s_or;
  uint32_t lo = 0;                        // at least K reach it, or it is 0
  if (s_or) {
    uint32_t bit = differ ? 0x80000000u >> __clz(differ) : 0u;
    const uint32_t common = bit ? s_and & ~(2 * bit - 1) : s_and;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __syncthreads_count(x[i] != 0);
    if (n > K) {
      for (lo = common; bit; bit >>= 1) {
        const uint32_t mid = lo | bit;
        n = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) n += __syncthreads_count(x[i] >= mid);
        if (n >= K) lo = mid;
        if (n == K) break;
      }
    }
  }
  __syncthreads();
  return lo;
}

// The group's choice and the new states, by the group's last CTA.  What it takes
// is round trips to L2, one after another, so loads go out together: the parts,
// the candidates and the old states.  (Of very many candidates the lists' first;
// then the K lists whose first are the best, among which the K best are.)
__device__ __noinline__ void choose(const Params& p, int g, Scratch& sc) {
  constexpr int kPerThread = kMaxLists / kThreads;
  const int K = p.K, lists = K * p.parts, tid = threadIdx.x, lane = tid & 31;
  __shared__ double s_add[kMaxBeams], s_ref[kMaxBeams], s_ln[kMaxBeams];
  __shared__ uint64_t s_z[kMaxBeams];
  __shared__ float s_c[kMaxBeams], s_far[kMaxBeams];
  __shared__ int s_n, s_lists, s_parent[kMaxBeams], s_token[kMaxBeams], s_lens[kMaxBeams];
  __shared__ uint16_t s_list[kMaxLists];
  __shared__ uint8_t s_old[kMaxBeams], s_taken[kMaxLists];
  __shared__ float s_score[kMaxBeams];
  const int row0 = g * K;
  const int2* cand = reinterpret_cast<const int2*>(p.cand + (size_t)row0 * p.parts * K);
  // all candidates where a thread can hold its share of them, else the lists' first,
  // which are their best
  const bool every = lists * K <= kMaxLists;
  const int held = every ? lists * K : lists, of_row = every ? p.parts * K : p.parts;
  int2 head[kPerThread];
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = tid + j * kThreads;
    head[j] = i < held ? __ldcg(cand + (size_t)i * (every ? 1 : K)) : make_int2(0, -1);
  }
  // everything old: in and out may be the same
  float add = 0.0f;
  uint8_t old = 0;
  int lens = 0, len = 0;
  if (tid < K) {
    add = p.scores[row0 + tid];
    if (p.ended) old = p.ended[row0 + tid];
    if (p.seq_lens) lens = p.seq_lens[row0 + tid];
  }
  if (p.history) len = p.hist_len[g];
  for (int r = tid >> 5; r < K; r += kThreads / 32) {
    const uint4* part = reinterpret_cast<const uint4*>(p.part + (size_t)(row0 + r) * p.parts);
    float c = -INFINITY, far = -INFINITY;
    uint64_t z = 0;
    for (int i = lane; i < p.parts; i += 32) {
      const uint4 u = __ldcg(part + i);
      const uint64_t s = (uint64_t)u.y << 32 | u.x;
      const float pc = __uint_as_float(u.z);
      const float pf = __uint_as_float(u.w);
      if (pc > c || (pc == c && pf > far)) {
        z = (c > -INFINITY ? beside(z, c, far, pc, pf) : 0) + s;
        c = pc;
        far = pf;
      } else if (pc > -INFINITY) {
        z += beside(s, pc, pf, c, far);
      }
    }
    const float top = warp_max(c), top_far = warp_max(c == top ? far : -INFINITY);
    z = warp_sum(c > -INFINITY ? beside(z, c, far, top, top_far) : 0);
    if (lane == 0) { s_z[r] = z; s_c[r] = top; s_far[r] = top_far; }
  }
  if (tid < K) {
    s_add[tid] = add;
    s_old[tid] = old;
    s_lens[tid] = lens;
    s_parent[tid] = s_token[tid] = -1;
    s_score[tid] = -INFINITY;
  }
  if (tid == 0) s_n = s_lists = 0;
  __syncthreads();
  if (tid < K) {
    // ln of the sum = ref + ln, apart: beside a far reference ln would be lost
    const bool none = s_old[tid] || s_z[tid] == 0;
    s_ref[tid] = none ? 0.0 : s_far[tid] < INFINITY ? (double)s_far[tid] : (double)s_c[tid] * (1.0 / (double)kLog2e);
    s_ln[tid] = none ? 0.0 : ln_of(s_z[tid]) - 40.0 * 0.69314718055994530942;
  }
  __syncthreads();

  const auto score_of = [&](int r, int2 c) {
    Score s{0, ~0ull};
    if (c.y >= 0) {
      const double v = ((double)__int_as_float(c.x) - s_ref[r]) - s_ln[r] + s_add[r];
      if (v > -INFINITY) { s.s = rank64(v); s.at = (uint64_t)r << 32 | (uint32_t)c.y; }
    }
    return s;
  };
  // (the upper half of a score's rank is in its order)
  Score mine[kPerThread];
  uint32_t most[kPerThread];
  const auto listed = [&](int n) {        // of the first n candidates, those among the K best, or equal to them
    const uint32_t bound = n <= kThreads ? kth<1>({most[0]}, K) : kth<kPerThread>(most, K);
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      if (most[j] && most[j] >= bound) {
        const int at = atomicAdd(&s_n, 1);
        if (at < kFinal) sc.score[at] = mine[j];
      }
  };
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) {
    const int i = tid + j * kThreads;
    mine[j] = Score{0, ~0ull};
    if (i < held) mine[j] = score_of(i / of_row, head[j]);
    most[j] = (uint32_t)(mine[j].s >> 32);
  }
  if (every) {
    listed(held);
  } else {
    // the K lists that begin best, and of theirs the K best
    const uint32_t bound = lists <= kThreads ? kth<1>({most[0]}, K) : kth<kPerThread>(most, K);
#pragma unroll
    for (int j = 0; j < kPerThread; ++j)
      if (most[j] && most[j] >= bound) s_list[atomicAdd(&s_lists, 1)] = (uint16_t)(tid + j * kThreads);
    __syncthreads();
    const int some = s_lists * K;
    if (some <= kMaxLists) {
#pragma unroll
      for (int j = 0; j < kPerThread; ++j) {
        const int i = tid + j * kThreads;
        mine[j] = Score{0, ~0ull};
        if (i < some) {
          const int list = s_list[i / K];
          mine[j] = score_of(list / p.parts, __ldcg(cand + (size_t)list * K + i % K));
        }
        most[j] = (uint32_t)(mine[j].s >> 32);
      }
      listed(some);
    } else if (tid == 0) {
      s_n = kFinal + 1;
    }
  }
  __syncthreads();
  const int n = s_n;
  const auto place = [&](const Score& s, int r) {
    s_parent[r] = (int)(s.at >> 32);
    s_token[r] = (int)(uint32_t)s.at;
    s_score[r] = (float)unrank64(s.s);
  };
  if (n <= kFinal) {
    for (int i = tid; i < n; i += kThreads) {
      const Score s = sc.score[i];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) r += better(sc.score[j], s);
      if (r < K) place(s, r);
    }
  } else {
    // more than the list holds (many that are equal): the best of the lists'
    // next ones, K times
    for (int i = tid; i < lists; i += kThreads) s_taken[i] = 0;
    __syncthreads();
    for (int r = 0; r < K; ++r) {
      Score top{0, ~0ull};
      for (int i = tid; i < lists; i += kThreads)
        if (s_taken[i] < K) {
          const Score s = score_of(i / p.parts, __ldcg(cand + (size_t)i * K + s_taken[i]));
          if (better(s, top)) {
            top = s;
            s_list[tid] = (uint16_t)i;    // the list it came from
          }
        }
      sc.score[tid] = top;
      __syncthreads();
      if (tid == 0) {
        int from = 0;
        for (int i = 1; i < kThreads; ++i)
          if (better(sc.score[i], sc.score[from])) from = i;
        if (sc.score[from].s) {
          place(sc.score[from], r);
          s_taken[s_list[from]] += 1;
        }
      }
      __syncthreads();
    }
  }
  __syncthreads();

  if (tid < K) {
    const int par = s_parent[tid];
    p.parent[row0 + tid] = par < 0 ? -1 : row0 + par;
    p.token[row0 + tid] = s_token[tid];
    p.scores_out[row0 + tid] = s_score[tid];
    if (p.ended_out) p.ended_out[row0 + tid] = par >= 0 && (s_old[par] || s_token[tid] == p.eos);
    if (p.new_lens) p.new_lens[row0 + tid] = par >= 0 ? s_lens[par] + 1 : 0;
  }
  if (!p.history) return;
  const bool full = len < 0 || len >= p.max_len;
  if (full && tid == 0) set_status(p.status, SSA_ST_BAD_POS);
  len = min(max(len, 0), p.max_len);
  if (p.move_here) {                      // K * max_len fit the scratch
    for (int i = 0; i < K; ++i)
      if (s_parent[i] >= 0)
        for (int c = tid; c < len; c += kThreads)
          sc.move[i * len + c] = p.history[(long long)(row0 + s_parent[i]) * p.max_len + c];
    __syncthreads();
    for (int i = 0; i < K; ++i)
      if (s_parent[i] >= 0)
        for (int c = tid; c < len; c += kThreads)
          p.history_out[(long long)(row0 + i) * p.max_len + c] = sc.move[i * len + c];
  } else if (tid == 0) {
    p.old_len[g] = len;
  }
  if (!full && tid < K && s_parent[tid] >= 0) p.history_out[(long long)(row0 + tid) * p.max_len + len] = s_token[tid];
  if (tid == 0) p.hist_len_out[g] = full ? len : len + 1;
}

// A CTA takes a part of a row, chunk after chunk, the next one's loads in flight.
template <typename T>
__global__ void __launch_bounds__(kThreads, kCtas) beam_kernel(const __grid_constant__ Params p, bool vec) {
  using X = Logits<T>;
  __shared__ Scratch sc;
  __shared__ uint64_t s_best[kThreads], s_keep[kMaxBeams];
  __shared__ __align__(16) uint32_t s_key[64];
  __shared__ uint64_t s_bound, s_sum[kThreads / 32];
  __shared__ uint32_t s_least;
  __shared__ __align__(16) float s_max[kThreads / 32];
  __shared__ int s_n, s_last;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = p.K;
  const int row = (int)(blockIdx.x / (unsigned)p.parts), part = (int)(blockIdx.x % (unsigned)p.parts);
  const int g = row / K;
  Cand* out = p.cand + ((size_t)row * p.parts + part) * K;
  Part* left = p.part + (size_t)row * p.parts + part;

  if (p.ended && p.ended[row]) {
    // one candidate, at the beam's score
    if (tid < K) out[tid] = Cand{0.0f, part == 0 && tid == 0 ? p.eos : -1};
    if (tid == 0) *left = Part{0, -INFINITY, INFINITY};
  } else {
    const T* logits = static_cast<const T*>(p.logits) + row * p.stride;
    const long long begin = (long long)part * p.chunks * X::kChunk;
    const long long end = min((long long)p.V, begin + (long long)p.chunks * X::kChunk);
    X x;
    x.load(logits, begin, p.V, vec);
    if (tid == 0) s_n = 0;
    int kept = 0;                         // of the list, the best so far
    float reached = X::lowest();          // the K-th best so far
    float c = -INFINITY;                  // the reference of the sum: whole octaves, so that parts add by shifts,
    float far = INFINITY;                 // or this logit, where it is far out
    uint64_t z = 0;                       // the thread's sum
    // the chunk's greatest becomes the reference where it is above it
    const auto refer = [&](float top) {
      if (top > -INFINITY) {
        const bool is_far = fabsf(top) >= kFar;
        const float tc = is_far ? fmaxf(top, -kGreatest) * kLog2e : ceilf(top * kLog2e);
        if (tc > c || (tc == c && is_far && top > far)) {
          const float tf = is_far ? top : INFINITY;
          if (c > -INFINITY) z = beside(z, c, far, tc, tf);
          c = tc;
          far = tf;
        }
      }
    };
    const auto block_top = [&]() {
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kThreads / 128; ++w) {
        const float4 f = reinterpret_cast<const float4*>(s_max)[w];
        top = fmaxf(fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)), top);
      }
      return top;
    };
    for (long long first = begin; first < end; first += X::kChunk) {
      X next;
      if (first + X::kChunk < end) next.load(logits, first + X::kChunk, p.V, vec);
      const float m = fminf(x.most(), kGreatest);
      float least = reached;
      if (kept < K) {                     // no bound yet: one of this chunk's own
        float q = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 2));
        // the lowest six bits tell groups apart: a bound rounded down is still one
        if ((tid & 3) == 0) s_key[tid >> 2] = (rank32(q) & ~63u) | (uint32_t)(tid >> 2);
        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 4));
        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 8));
        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 16));
        if (lane == 0) s_max[warp] = q;
        __syncthreads();
        refer(block_top());
        if (tid < 64) {
          const uint32_t k = s_key[tid];
          int rank = 0;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint4 u = reinterpret_cast<const uint4*>(s_key)[j];
            rank += (u.x > k) + (u.y > k) + (u.z > k) + (u.w > k);
          }
          if (rank == K - 1) s_least = k & ~63u;
        }
        __syncthreads();
        least = fmaxf(unrank32(s_least), reached);        // (a NaN where fewer than K are finite)
      }
      // the list of what reaches the bound
      int flags = 0;
      if (m >= least) {
        flags = 1;
        for (uint32_t bits = x.reach(least); bits; bits &= bits - 1) {
          const int at = kept + atomicAdd(&s_n, 1);
          if (at >= kList) break;
          const int i = x.place(__ffs(bits) - 1);
          sc.list[at] = key_of(fminf(x.at(i), kGreatest), (uint32_t)x.token((int)first, i));
        }
      }
      float sum = 0.0f;
      if (c > -INFINITY) sum = far < INFINITY ? x.sum_from(far) : x.sum(c);
      // above: a NaN, or logits above the reference of the chunks before
      if (!(sum <= (float)X::M) || (c == -INFINITY && m > -INFINITY)) flags |= 2;
      // The size of the list is read between two barriers: a warp that is done with a
      // chunk which lists nothing (a NaN alone brought it here) may add to the next
      // one's while another still decides, and they would part ways.
      int found = 0;
      if (__syncthreads_or(flags != 0)) {
        found = s_n;
        if (__syncthreads_or((flags & 2) != 0)) {
          const float q = warp_max(m);
          if (lane == 0) s_max[warp] = q;
          __syncthreads();
          refer(block_top());
          sum = 0.0f;
          if (c > -INFINITY) sum = far < INFINITY ? x.sum_from(far) : x.sum_clean(c);
          __syncthreads();                // s_max is the next chunk's from here on
        }
      }
      z += (uint64_t)(sum * kUnit);
      if (found > 0) {
        int n = kept + found;
        if (n > kList) {
          // many equal ones: bounded over (value, token) instead
          uint64_t best = 0;
          x.each([&](float v, int i) {
            if (v == v) {
              const uint64_t k = key_of(fminf(v, kGreatest), (uint32_t)x.token((int)first, i));
              if (k > best) best = k;
            }
          });
          s_best[tid] = best;
          __syncthreads();
          if (tid == 0) s_n = 0;
          int rank = 0;
          for (int j = 0; j < kThreads; ++j) rank += s_best[j] > best || (s_best[j] == best && j < tid);
          if (rank == K - 1) s_bound = best;
          __syncthreads();
          const uint64_t bound = s_bound;
          if (best >= bound)
            x.each([&](float v, int i) {
              if (v == v && v > -INFINITY) {
                const uint64_t k = key_of(fminf(v, kGreatest), (uint32_t)x.token((int)first, i));
                if (k >= bound) sc.list[kept + atomicAdd(&s_n, 1)] = k;
              }
            });
          __syncthreads();
          n = kept + s_n;
        }
        for (int i = tid; i < n; i += kThreads) {
          const uint64_t k = sc.list[i];
          int r = 0;
#pragma unroll 4
          for (int j = 0; j < n; ++j) r += sc.list[j] > k;
          if (r < K) s_keep[r] = k;
        }
        __syncthreads();
        kept = min(n, K);
        if (tid < kept) sc.list[tid] = s_keep[tid];
        if (kept == K) reached = fmaxf(key_x(s_keep[K - 1]), reached);
        if (tid == 0) s_n = 0;
        __syncthreads();
      }
      x = next;
    }
    z = warp_sum(z);
    if (lane == 0) s_sum[warp] = z;
    __syncthreads();
    if (tid < K) out[tid] = tid < kept ? Cand{key_x(s_keep[tid]), (int)~(uint32_t)s_keep[tid]} : Cand{0.0f, -1};
    if (tid == 0) {
      uint64_t s = 0;
      for (int w = 0; w < kThreads / 32; ++w) s += s_sum[w];
      *left = Part{s, c, far};
    }
  }
  // the last CTA of the group goes on: one thread's release covers what the CTA wrote before the
  // barrier, its acquire what the others released
  __syncthreads();
  if (tid == 0) {
    uint32_t before;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.ticket + g) : "memory");
    const bool last = before == (uint32_t)(K * p.parts - 1);
    if (last) p.ticket[g] = 0;
    s_last = last;
  }
  __syncthreads();
  if (!s_last) return;
  choose(p, g, sc);
}

// Histories of a group in their new order: a thread per column, which reads it in
// every row before it writes one, so in and out may be the same.
constexpr int kMoveThreads = 128;
__global__ void __launch_bounds__(kMoveThreads) beam_move_kernel(const __grid_constant__ Params p) {
  extern __shared__ int32_t s_col[];      // [K][kMoveThreads]
  pdl_trigger();
  pdl_wait();
  const int g = blockIdx.y, K = p.K, tid = threadIdx.x;
  const int c = blockIdx.x * kMoveThreads + tid;
  const long long row0 = (long long)g * K;
  if (c >= p.old_len[g]) return;
#pragma unroll 8
  for (int i = 0; i < K; ++i) {
    const int par = p.parent[row0 + i];
    if (par >= 0) s_col[i * kMoveThreads + tid] = p.history[(long long)par * p.max_len + c];
  }
#pragma unroll 8
  for (int i = 0; i < K; ++i)
    if (p.parent[row0 + i] >= 0) p.history_out[(row0 + i) * p.max_len + c] = s_col[i * kMoveThreads + tid];
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// A workspace begins with a ticket for every group that a call may have: what a call
// of any size leaves behind them is never another's ticket.
constexpr size_t kTickets = ((size_t)kMaxGroups * sizeof(int32_t) + 255) & ~(size_t)255;

template <typename T>
cudaError_t launch(Params p, int groups, cudaStream_t s) {
  constexpr int N = 16 / sizeof(T);
  const bool vec = !((uintptr_t)p.logits & 15) && (p.stride % N == 0 || groups * p.K == 1);
  // parts of a row: as many as one wave of CTAs has room for, whole chunks each
  const int rows = groups * p.K, all = (int)(((long long)p.V + Logits<T>::kChunk - 1) / Logits<T>::kChunk);
  const int room = std::max(1, std::min(kMaxLists, current_device_info().sms * kCtas) / rows);
  p.chunks = (all + room - 1) / room;
  p.parts = (all + p.chunks - 1) / p.chunks;
  cudaError_t e = launch_pdl(beam_kernel<T>, dim3((unsigned)(rows * p.parts)), dim3(kThreads), 0, s, p, vec);
  count_launch();
  if (e != cudaSuccess || !p.history || p.move_here) return e;
  e = launch_pdl(beam_move_kernel, dim3((p.max_len + kMoveThreads - 1) / kMoveThreads, groups), dim3(kMoveThreads),
                 (size_t)p.K * kMoveThreads * sizeof(int32_t), s, p);
  count_launch();
  return e;
}

}  // namespace
}  // namespace ssa

extern "C" {

size_t ssa_beam_workspace_size(int groups, int beams) {
  using namespace ssa;
  if (groups < 1 || beams < 1 || beams > kMaxBeams) return 0;
  const size_t lists = std::max((size_t)groups * beams, (size_t)kMaxLists);
  return kTickets + align256((size_t)groups * 4) + align256(lists * sizeof(Part)) + align256(lists * beams * sizeof(Cand));
}

int ssa_beam_select(int dtype, int groups, int beams, int vocab, const void* logits, int64_t row_stride,
                    const ssa_beams* in, const ssa_beams* out, int max_len, int eos, int32_t* parent,
                    int32_t* token, const int32_t* seq_lens_opt, int32_t* new_lens_opt, int32_t* status,
                    void* ws, ssa_stream_t stream) {
  using namespace ssa;
  if (dtype < SSA_BF16 || dtype > SSA_F32) return SSA_ERR_UNSUPPORTED;
  if (groups < 1 || beams < 1 || vocab < 1 || max_len < 0 || eos < -1 || eos >= vocab) return SSA_ERR_INVALID_ARG;
  if (beams > kMaxBeams || groups > kMaxGroups || vocab > 1 << 23) return SSA_ERR_UNSUPPORTED;
  if (!logits || !in || !out || !in->scores || !out->scores || !parent || !token || !ws) return SSA_ERR_INVALID_ARG;
  if ((uintptr_t)logits & (dtype == SSA_F32 ? 3 : 1)) return SSA_ERR_INVALID_ARG;
  if (row_stride < vocab && (long long)groups * beams > 1) return SSA_ERR_INVALID_ARG;
  // beams end where there is an eos, and only there
  if ((eos >= 0) != (in->finished != nullptr) || (eos >= 0) != (out->finished != nullptr)) return SSA_ERR_INVALID_ARG;
  for (const ssa_beams* b : {in, out})
    if ((max_len > 0) != (b->history != nullptr) || (max_len > 0) != (b->hist_len != nullptr)) return SSA_ERR_INVALID_ARG;
  if ((seq_lens_opt != nullptr) != (new_lens_opt != nullptr)) return SSA_ERR_INVALID_ARG;
  if ((uintptr_t)ws & 255) return SSA_ERR_INVALID_ARG;

  Params p{};
  p.logits = logits; p.stride = row_stride;
  p.K = beams; p.V = vocab; p.max_len = max_len; p.eos = eos;
  p.scores = in->scores; p.ended = in->finished; p.history = in->history; p.hist_len = in->hist_len;
  p.scores_out = out->scores; p.ended_out = out->finished; p.history_out = out->history;
  p.hist_len_out = out->hist_len;
  p.seq_lens = seq_lens_opt; p.new_lens = new_lens_opt; p.parent = parent; p.token = token;
  p.status = status;
  p.move_here = (long long)beams * max_len <= (long long)(sizeof(Scratch::move) / 4);
  char* w = static_cast<char*>(ws);
  p.ticket = reinterpret_cast<int32_t*>(w);
  w += kTickets;
  p.old_len = reinterpret_cast<int32_t*>(w);
  w += align256((size_t)groups * 4);
  p.part = reinterpret_cast<Part*>(w);
  w += align256(std::max((size_t)groups * beams, (size_t)kMaxLists) * sizeof(Part));
  p.cand = reinterpret_cast<Cand*>(w);
  cudaError_t e;
  switch (dtype) {
    case SSA_BF16: e = launch<__nv_bfloat16>(p, groups, (cudaStream_t)stream); break;
    case SSA_F16: e = launch<__half>(p, groups, (cudaStream_t)stream); break;
    default: e = launch<float>(p, groups, (cudaStream_t)stream); break;
  }
  return e == cudaSuccess ? SSA_OK : record_cuda_error(e);
}

}  // extern "C"
