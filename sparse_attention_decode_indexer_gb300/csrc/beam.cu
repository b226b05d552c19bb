// beam.cu -- the next tokens of beams: the best (beam, token) pairs of every
// group, and the beams' states in their new order.
//
// With x[r][t] the logits of beam r, a candidate's score is
//   score[r] + x[r][t] - ln sum_t' exp(x[r][t']);
// a beam that has ended has one candidate, (r, eos) at score[r].  The K = beams
// best of a group win, the first beam and then the first token among equals.
//
// What bounds it: the logits, read once.  A CTA takes 8,192 of a row's logits
// into registers and leaves their maximum, the sum of their exponentials and
// the K best; the last CTA of a group (a ticket) puts these together.
//
// The K best of what the threads of a CTA hold: each thread's own best; the
// K-th of those bests is a bound that at least K values reach, and values that
// reach it lie in at most K threads, so they go to a short list, in which each
// finds its rank by counting.  Values are compared together with their index,
// so that no two are equal and the order of the list does not matter.
//
// Sums: fp32 within a thread (32 values), double above; scores are compared in
// double, so that candidates of different beams are ordered by what they are
// and not by a rounding to fp32 (an exponential is off by about 2^-22, an
// average over many by less).
#include <algorithm>
#include <cfloat>
#include <climits>

#include "rope.cuh"

namespace ssa {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 32;                  // logits of a thread
constexpr int kSlice = kThreads * kPer;
constexpr int kMaxBeams = 32;
constexpr int kMaxLists = 1024;           // (row, slice) lists of a group

struct Part {                             // of a slice
  double sum;                             // of exp(x - max)
  float max;
  int pad;
};
struct Cand {                             // logit and token; token < 0: none
  float x;
  int t;
};

struct Params {
  const void* logits;
  int64_t stride;
  int K, V, slices, max_len, eos;
  const float* scores;
  const uint8_t* ended;
  const int32_t *history, *hist_len, *seq_lens;
  float* scores_out;
  uint8_t* ended_out;
  int32_t *history_out, *hist_len_out, *new_lens, *parent, *token;
  int32_t* status;
  Part* part;                             // [row][slice]
  Cand* cand;                             // [row][slice][K]
  int32_t* ticket;                        // [group], zero between calls
};

// Larger keys are better: the logit's order above, the lower token first below.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t t) {
  const uint32_t b = __float_as_uint(x);
  return (uint64_t)(b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u)) << 32 | (uint32_t)~t;
}
__device__ __forceinline__ float key_x(uint64_t k) {
  const uint32_t b = (uint32_t)(k >> 32);
  return __uint_as_float(b ^ ((int32_t)b < 0 ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A logit as the sums take it: NaN is no candidate, +infinity the greatest number.
__device__ __forceinline__ float clean(float x) { return x == x ? fminf(x, FLT_MAX) : -INFINITY; }

template <typename T>
__device__ __forceinline__ void load_slice(const T* row, int first, int V, bool vec, float* x) {
  constexpr int N = 16 / sizeof(T);
#pragma unroll
  for (int j = 0; j < kPer / N; ++j) {
    const int at = first + (j * kThreads + threadIdx.x) * N;
    if (vec && at + N <= V) {
      const uint4 u = *reinterpret_cast<const uint4*>(row + at);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          x[j * N + i] = __uint_as_float(w[i]);
        } else {
          const float2 f = unpack<T>(w[i]);
          x[j * N + 2 * i] = f.x;
          x[j * N + 2 * i + 1] = f.y;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[j * N + i] = at + i < V ? one_in(row[at + i]) : -INFINITY;
    }
  }
}
// the token of a thread's i-th logit
template <typename T> __device__ __forceinline__ int token_of(int first, int i) {
  constexpr int N = 16 / sizeof(T);
  return first + ((i / N) * kThreads + (int)threadIdx.x) * N + i % N;
}

struct Score {                            // of a candidate, and its place in the group
  double s;
  long long at;                           // row * V + token
};
__device__ __forceinline__ bool better(const Score& a, const Score& b) {
  return a.s > b.s || (a.s == b.s && a.at < b.at);
}

// The group's choice and the new states, by the group's last CTA.
template <typename T>
__device__ void choose(const Params& p, int g, uint8_t* smem) {
  const int K = p.K, lists = K * p.slices, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ double s_score0[kMaxBeams], s_lse[kMaxBeams];
  __shared__ Score s_best[kThreads];
  __shared__ Score s_bound;
  __shared__ int s_n, s_parent[kMaxBeams], s_token[kMaxBeams];
  __shared__ uint8_t s_ended[kMaxBeams];
  __shared__ int s_len[kMaxBeams];
  __shared__ float s_score[kMaxBeams];
  const long long row0 = (long long)g * K;
  for (int r = warp; r < K; r += kThreads / 32) {
    const bool ended = p.ended && p.ended[row0 + r];
    float m = -INFINITY;
    for (int i = lane; i < p.slices; i += 32) m = fmaxf(m, __ldcg(&p.part[(row0 + r) * p.slices + i].max));
    m = warp_max(m);
    double z = 0.0;
    for (int i = lane; i < p.slices; i += 32) {
      const Part* q = &p.part[(row0 + r) * p.slices + i];
      const float qm = __ldcg(&q->max);
      if (qm > -INFINITY) z += __ldcg(&q->sum) * exp((double)qm - (double)m);
    }
    z = warp_sum(z);
    if (lane == 0) {
      s_score0[r] = p.scores[row0 + r];
      s_lse[r] = ended || z == 0.0 ? 0.0 : (double)m + log(z);
    }
  }
  if (tid == 0) s_n = 0;
  if (tid < K) {
    s_parent[tid] = -1;
    s_token[tid] = -1;
    s_score[tid] = -INFINITY;
  }
  __syncthreads();

  const auto score_of = [&](int list, int k) {
    const int r = list / p.slices;
    const int2 c = __ldcg(reinterpret_cast<const int2*>(p.cand + (row0 * p.slices + list) * K + k));
    Score s{-INFINITY, LLONG_MAX};
    if (c.y >= 0) {
      const double v = ((double)__int_as_float(c.x) - s_lse[r]) + s_score0[r];
      if (v > -INFINITY) { s.s = v; s.at = (long long)r * p.V + c.y; }
    }
    return s;
  };
  // a list is sorted: its first is its best
  Score best{-INFINITY, LLONG_MAX};
  for (int i = tid; i < lists; i += kThreads) {
    const Score s = score_of(i, 0);
    if (better(s, best)) best = s;
  }
  s_best[tid] = best;
  if (tid == 0) s_bound = Score{-INFINITY, LLONG_MAX};
  __syncthreads();
  int rank = 0;
  for (int j = 0; j < kThreads; ++j) rank += better(s_best[j], best);
  if (rank == K - 1 && best.s > -INFINITY) s_bound = best;
  __syncthreads();
  const Score bound = s_bound;
  Score* list = reinterpret_cast<Score*>(smem);
  if (best.s > -INFINITY && !better(bound, best))
    for (int i = tid; i < lists; i += kThreads)
      for (int k = 0; k < K; ++k) {
        const Score s = score_of(i, k);
        if (s.s == -INFINITY || better(bound, s)) break;
        list[atomicAdd(&s_n, 1)] = s;
      }
  __syncthreads();
  const int n = s_n;
  for (int i = tid; i < n; i += kThreads) {
    const Score s = list[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += better(list[j], s);
    if (r < K) {
      s_parent[r] = (int)(s.at / p.V);
      s_token[r] = (int)(s.at % p.V);
      s_score[r] = (float)s.s;
    }
  }
  __syncthreads();

  // states: everything old is read before anything new is written, in and out may be the same
  if (tid < K) {
    const int par = s_parent[tid];
    s_ended[tid] = par >= 0 && p.ended ? (uint8_t)(p.ended[row0 + par] != 0 || s_token[tid] == p.eos) : (uint8_t)0;
    s_len[tid] = par >= 0 && p.seq_lens ? p.seq_lens[row0 + par] + 1 : 0;
  }
  int len = 0;
  if (p.history) len = p.hist_len[g];
  __syncthreads();
  if (tid < K) {
    const int par = s_parent[tid];
    p.parent[row0 + tid] = par < 0 ? -1 : (int)(row0 + par);
    p.token[row0 + tid] = s_token[tid];
    p.scores_out[row0 + tid] = s_score[tid];
    if (p.ended_out) p.ended_out[row0 + tid] = s_ended[tid];
    if (p.new_lens) p.new_lens[row0 + tid] = s_len[tid];
  }
  if (!p.history) return;
  const bool full = len < 0 || len >= p.max_len;
  if (full && tid == 0) set_status(p.status, SSA_ST_BAD_POS);
  len = min(max(len, 0), p.max_len);
  int32_t* column = reinterpret_cast<int32_t*>(smem);       // [K][kThreads], a thread its own
  for (int c = tid; c < len; c += kThreads) {
    for (int i = 0; i < K; ++i)
      if (s_parent[i] >= 0) column[i * kThreads + tid] = p.history[(row0 + s_parent[i]) * p.max_len + c];
    for (int i = 0; i < K; ++i)
      if (s_parent[i] >= 0) p.history_out[(row0 + i) * p.max_len + c] = column[i * kThreads + tid];
  }
  if (!full && tid < K && s_parent[tid] >= 0) p.history_out[(row0 + tid) * p.max_len + len] = s_token[tid];
  if (tid == 0) p.hist_len_out[g] = full ? len : len + 1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_kernel(const __grid_constant__ Params p, bool vec) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t s_best[kThreads];
  __shared__ uint64_t s_bound;
  __shared__ double s_sum[kThreads / 32];
  __shared__ float s_max[kThreads / 32];
  __shared__ int s_n, s_last;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, K = p.K;
  const long long row = blockIdx.x / p.slices;
  const int slice = blockIdx.x % p.slices, g = (int)(row / K);
  Cand* out = p.cand + ((long long)row * p.slices + slice) * K;
  Part* part = p.part + (long long)row * p.slices + slice;

  if (p.ended && p.ended[row]) {
    // one candidate, at the beam's score
    if (tid < K) out[tid] = Cand{0.0f, slice == 0 && tid == 0 ? p.eos : -1};
    if (tid == 0) *part = Part{0.0, -INFINITY, 0};
  } else {
    float x[kPer];
    const int first = slice * kSlice;
    load_slice<T>(static_cast<const T*>(p.logits) + row * p.stride, first, p.V, vec, x);
    if (tid == 0) { s_n = 0; s_bound = 0; }
    float m = -INFINITY;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      x[i] = clean(x[i]);
      if (x[i] > m) { m = x[i]; at = i; }
    }
    const uint64_t best = key_of(m, (uint32_t)token_of<T>(first, at));
    s_best[tid] = best;
    float top = warp_max(m);
    if (lane == 0) s_max[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, s_max[w]);
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < kThreads; ++j) rank += s_best[j] > best;
    if (rank == K - 1) s_bound = best;
    float sum[4] = {0, 0, 0, 0};
    if (top > -INFINITY) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum[i & 3] += fast_exp2((x[i] - top) * 1.4426950408889634f);
    }
    const double z = warp_sum((double)((sum[0] + sum[1]) + (sum[2] + sum[3])));
    if (lane == 0) s_sum[warp] = z;
    __syncthreads();
    const uint64_t bound = s_bound;
    uint64_t* list = reinterpret_cast<uint64_t*>(smem);
    if (best >= bound) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint64_t k = key_of(x[i], (uint32_t)token_of<T>(first, i));
        if (k >= bound && x[i] > -INFINITY) list[atomicAdd(&s_n, 1)] = k;
      }
    }
    __syncthreads();
    const int n = s_n;
    if (tid < K && tid >= n) out[tid] = Cand{0.0f, -1};
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t k = list[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += list[j] > k;
      if (r < K) out[r] = Cand{key_x(k), (int)~(uint32_t)k};
    }
    if (tid == 0) {
      double s = 0.0;
      for (int w = 0; w < kThreads / 32; ++w) s += s_sum[w];
      *part = Part{s, top, 0};
    }
  }
  // the last CTA of the group goes on
  __threadfence();
  __syncthreads();
  if (tid == 0) {
    const int last = atomicAdd(p.ticket + g, 1) == K * p.slices - 1;
    if (last) p.ticket[g] = 0;
    s_last = last;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  choose<T>(p, g, smem);
}

int slices_of(int V) { return (V + kSlice - 1) / kSlice; }

size_t align16(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T>
cudaError_t launch(const Params& p, int groups, cudaStream_t s) {
  constexpr int N = 16 / sizeof(T);
  const bool vec = !((uintptr_t)p.logits & 15) && (p.stride % N == 0 || groups * p.K == 1);
  const int per = (p.K * p.slices + kThreads - 1) / kThreads;        // lists of a thread
  size_t smem = (size_t)p.K * kPer * sizeof(uint64_t);
  smem = std::max(smem, (size_t)p.K * per * p.K * sizeof(Score));
  if (p.history) smem = std::max(smem, (size_t)p.K * kThreads * sizeof(int32_t));
  cudaError_t e = cudaFuncSetAttribute(beam_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long ctas = (long long)groups * p.K * p.slices;
  if (ctas > INT_MAX) return cudaErrorInvalidValue;
  e = launch_pdl(beam_kernel<T>, dim3((unsigned)ctas), dim3(kThreads), smem, s, p, vec);
  count_launch();
  return e;
}

}  // namespace
}  // namespace ssa

extern "C" {

size_t ssa_beam_workspace_size(int groups, int beams) {
  using namespace ssa;
  if (groups < 1 || beams < 1 || beams > kMaxBeams) return 0;
  const size_t lists = (size_t)groups * kMaxLists;
  return align16((size_t)groups * 4) + align16(lists * sizeof(Part)) + align16(lists * beams * sizeof(Cand));
}

int ssa_beam_select(int dtype, int groups, int beams, int vocab, const void* logits, int64_t row_stride,
                    const ssa_beams* in, const ssa_beams* out, int max_len, int eos, int32_t* parent,
                    int32_t* token, const int32_t* seq_lens_opt, int32_t* new_lens_opt, int32_t* status,
                    void* ws, ssa_stream_t stream) {
  using namespace ssa;
  if (dtype < SSA_BF16 || dtype > SSA_F32) return SSA_ERR_UNSUPPORTED;
  if (groups < 1 || beams < 1 || vocab < 1 || max_len < 0 || eos < -1 || eos >= vocab) return SSA_ERR_INVALID_ARG;
  if (beams > kMaxBeams || (long long)beams * slices_of(vocab) > kMaxLists) return SSA_ERR_UNSUPPORTED;
  if ((long long)groups * beams > INT_MAX) return SSA_ERR_UNSUPPORTED;
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
  p.K = beams; p.V = vocab; p.slices = slices_of(vocab); p.max_len = max_len; p.eos = eos;
  p.scores = in->scores; p.ended = in->finished; p.history = in->history; p.hist_len = in->hist_len;
  p.scores_out = out->scores; p.ended_out = out->finished; p.history_out = out->history;
  p.hist_len_out = out->hist_len;
  p.seq_lens = seq_lens_opt; p.new_lens = new_lens_opt; p.parent = parent; p.token = token;
  p.status = status;
  char* w = static_cast<char*>(ws);
  p.ticket = reinterpret_cast<int32_t*>(w);
  w += align16((size_t)groups * 4);
  p.part = reinterpret_cast<Part*>(w);
  w += align16((size_t)groups * kMaxLists * sizeof(Part));
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
