// rope.cu -- rotary positions of queries and keys.
//
// Pair i of a head, (a, b) = (x[i], x[i + rd/2]) or interleaved (x[2i],
// x[2i+1]), turns by the angle pos * theta_i:
//   a' = a c - b s,  b' = b c + a s,  (c, s) = m (cos, sin)(pos * theta_i)
// (the inverse, and the gradient, with -s); dimensions past rd stay.
//
// Angles: theta_i / 2 pi is kept as a 64-bit fixed-point fraction of a turn,
// so pos * theta_i modulo a turn is one wrapping 64-bit product, exact for
// any position (an fp32 product is off by 0.06 rad at a million tokens).  The
// nearest quarter turn comes off as its top bits; the rest, at most an eighth
// of a turn, goes to sincospif.
//
// What bounds it: each element read and written once, HBM (3 flop per 4
// bytes).  The angles are shared by all layers and heads of a token, so a CTA
// serves one token: its threads start their first loads, rd/2 of them put the
// token's cos and sin into shared memory, and all rotate with 16-byte
// accesses.  Few tokens (a decode step) split a token's layers and heads over
// more CTAs, each of which computes the rd/2 pairs again.
#include <cmath>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace ssa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;           // units in flight per thread

template <typename T> struct Conv;
template <> struct Conv<float> {
  static __device__ __forceinline__ float in(float x) { return x; }
  static __device__ __forceinline__ float out(float x) { return x; }
};
template <> struct Conv<__half> {
  static __device__ __forceinline__ float in(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half out(float x) { return __float2half_rn(x); }
};
template <> struct Conv<__nv_bfloat16> {
  static __device__ __forceinline__ float in(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 out(float x) { return __float2bfloat16_rn(x); }
};

// V elements moved as one access (16 bytes, or one element)
template <typename T, int V> struct alignas(sizeof(T) * V) Vec { T x[V]; };

// (cos, sin) of pos * f turns, f a 64-bit fraction
__device__ __forceinline__ float2 turn(uint64_t pos, uint64_t f) {
  const uint64_t ph = pos * f;
  const uint64_t q = (ph + (1ull << 61)) >> 62;             // nearest quarter turn
  const long long r = (long long)(ph - (q << 62));          // the rest, |r| <= 2^61
  float s, c;
  sincospif(__ll2float_rn(r) * 0x1p-63f, &s, &c);
  if (q & 1) { const float t = c; c = -s; s = t; }
  if (q & 2) { c = -c; s = -s; }
  return make_float2(c, s);
}

struct RopeParams {
  RopeTensor x[2];
  int n_x;
  const uint64_t* freq;
  const void* pos;
  int64_t offset;
  float factor;
  int pos64, inverse, D, rd, L, T;
  int u_rot, units, rows_x0, rows;       // units of a row: rotated, with the tail; rows of q, of both
  int per_cta;                           // units of one CTA
};

// INTER: V elements hold V / 2 pairs.  Else a unit is V elements of each half.
// V counts elements per access; with INTER a scalar unit is one pair in two
// accesses (V = 1, NA = 2).
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  extern __shared__ float2 s_cs[];
  using A = Vec<T, V>;
  // accesses of a unit and the pairs in it
  constexpr int NA = (INTER && V > 1) ? 1 : 2;
  constexpr int NP = (INTER && V > 1) ? V / 2 : V;
  pdl_trigger();
  pdl_wait();
  const int t = blockIdx.x, tid = threadIdx.x;
  const int half = p.rd / 2;
  const int u0 = blockIdx.y * p.per_cta;
  const int u1 = min(u0 + p.per_cta, p.rows * p.units);

  // unit u of the token: which row, where its accesses are
  struct Place { const T* in; T* out; int64_t step; int pair; int n; };
  auto place = [&](int u) -> Place {
    int row = u / p.units;
    const int w = u - row * p.units;
    const RopeTensor& x = p.x[row >= p.rows_x0];
    if (row >= p.rows_x0) row -= p.rows_x0;
    const int l = row / x.heads, h = row - l * x.heads;
    Place r;
    r.in = static_cast<const T*>(x.in) + l * x.is[0] + t * x.is[1] + h * x.is[2];
    r.out = static_cast<T*>(x.out) + l * x.os[0] + t * x.os[1] + h * x.os[2];
    int e;
    if (w < p.u_rot) {
      r.pair = w * NP;
      e = INTER ? w * NP * 2 : w * V;
      r.step = INTER ? V : half;
      r.n = NA;
    } else {                              // the dimensions that stay
      r.pair = -1;
      e = p.rd + (w - p.u_rot) * V;
      r.step = 0;
      r.n = 1;
    }
    r.in += e;
    r.out += e;
    return r;
  };

  bool have_table = false;
  for (int base = u0; base < u1; base += kRopeThreads * kRopeUnroll) {
    A a[kRopeUnroll][NA];
#pragma unroll
    for (int i = 0; i < kRopeUnroll; ++i) {
      const int u = base + i * kRopeThreads + tid;
      if (u < u1) {
        const Place r = place(u);
        a[i][0] = *reinterpret_cast<const A*>(r.in);
        if (NA > 1 && r.n > 1) a[i][NA - 1] = *reinterpret_cast<const A*>(r.in + r.step);
      }
    }
    if (!have_table) {                    // while the first loads are in flight
      const int64_t raw = p.pos64 ? static_cast<const int64_t*>(p.pos)[t]
                                  : (int64_t) static_cast<const int32_t*>(p.pos)[t];
      const uint64_t pos = (uint64_t)raw + (uint64_t)p.offset;
      for (int i = tid; i < half; i += kRopeThreads) {
        const float2 cs = turn(pos, p.freq[i]);
        s_cs[i] = make_float2(cs.x * p.factor, (p.inverse ? -cs.y : cs.y) * p.factor);
      }
      __syncthreads();
      have_table = true;
    }
#pragma unroll
    for (int i = 0; i < kRopeUnroll; ++i) {
      const int u = base + i * kRopeThreads + tid;
      if (u < u1) {
        const Place r = place(u);
        if (r.pair >= 0) {
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            const float2 cs = s_cs[r.pair + k];
            T& ea = NA == 1 ? a[i][0].x[2 * k % V] : a[i][0].x[k % V];
            T& eb = NA == 1 ? a[i][0].x[(2 * k + 1) % V] : a[i][NA - 1].x[k % V];
            const float x = Conv<T>::in(ea), y = Conv<T>::in(eb);
            ea = Conv<T>::out(x * cs.x - y * cs.y);
            eb = Conv<T>::out(y * cs.x + x * cs.y);
          }
        }
        *reinterpret_cast<A*>(r.out) = a[i][0];
        if (NA > 1 && r.n > 1) *reinterpret_cast<A*>(r.out + r.step) = a[i][NA - 1];
      }
    }
  }
}

// every access of V elements of this tensor is aligned
bool aligned(const RopeTensor& x, int V, int esz, int L, int T) {
  const int64_t step[2][3] = {{x.is[0], x.is[1], x.is[2]}, {x.os[0], x.os[1], x.os[2]}};
  const int n[3] = {L, T, x.heads};
  if ((((uintptr_t)x.in | (uintptr_t)x.out) & (size_t)(V * esz - 1)) != 0) return false;
  for (auto& st : step)
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && st[i] % V != 0) return false;
  return true;
}

template <typename T, int V, bool INTER>
cudaError_t launch_rope_t(RopeParams p, bool copy_tail, int num_sms, cudaStream_t s) {
  const int np = (INTER && V > 1) ? V / 2 : V;                 // pairs per unit
  p.u_rot = p.rd / 2 / np;
  p.units = p.u_rot + (copy_tail ? (p.D - p.rd) / V : 0);
  const long long total = (long long)p.rows * p.units;         // of one token
  if (total > 0x3FFFFFFF) return cudaErrorInvalidValue;
  // one CTA per token where there are enough tokens to fill the machine
  // (8 CTAs of 256 threads per SM), else a token's units over several CTAs,
  // down to one unit per thread
  const long long full = 8LL * num_sms;
  long long split = (full + p.T - 1) / p.T;
  const long long most = (total + kRopeThreads - 1) / kRopeThreads;
  if (split > most) split = most;
  if (split > 65535) split = 65535;
  p.per_cta = (int)((total + split - 1) / split);
  const unsigned gy = (unsigned)((total + p.per_cta - 1) / p.per_cta);
  cudaError_t e = launch_pdl(rope_kernel<T, V, INTER>, dim3((unsigned)p.T, gy), dim3(kRopeThreads),
                             (size_t)p.rd / 2 * sizeof(float2), s, p);
  count_launch();
  return e;
}

template <typename T>
cudaError_t launch_rope_d(const RopeParams& p, bool inter, bool copy_tail, int num_sms,
                          cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  bool vec = p.D % V == 0 && (inter ? p.rd : p.rd / 2) % V == 0;
  for (int i = 0; i < p.n_x; ++i) vec = vec && aligned(p.x[i], V, sizeof(T), p.L, p.T);
  if (vec)
    return inter ? launch_rope_t<T, V, true>(p, copy_tail, num_sms, s)
                 : launch_rope_t<T, V, false>(p, copy_tail, num_sms, s);
  return inter ? launch_rope_t<T, 1, true>(p, copy_tail, num_sms, s)
               : launch_rope_t<T, 1, false>(p, copy_tail, num_sms, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  RopeParams p{};
  p.n_x = a.n_x;
  bool copy_tail = false;
  for (int i = 0; i < a.n_x; ++i) {
    p.x[i] = a.x[i];
    copy_tail = copy_tail || (a.x[i].in != a.x[i].out);
  }
  copy_tail = copy_tail && a.rd < a.D;
  p.freq = a.freq;
  p.pos = a.pos;
  p.pos64 = a.pos64;
  p.offset = a.offset;
  p.factor = a.factor;
  p.inverse = a.inverse;
  p.D = a.D; p.rd = a.rd; p.L = a.n_layers; p.T = a.n_tokens;
  p.rows_x0 = a.n_layers * a.x[0].heads;
  p.rows = p.rows_x0 + (a.n_x > 1 ? a.n_layers * a.x[1].heads : 0);
  switch (a.dtype) {
    case SSA_BF16: return launch_rope_d<__nv_bfloat16>(p, a.interleaved, copy_tail, a.num_sms, s);
    case SSA_F16: return launch_rope_d<__half>(p, a.interleaved, copy_tail, a.num_sms, s);
    default: return launch_rope_d<float>(p, a.interleaved, copy_tail, a.num_sms, s);
  }
}

int rope_frequencies(int rd, double base, int scaling, double factor, double original_len,
                     double low, double high, uint64_t* freq, double* attn_factor) {
  const double two_pi = 6.283185307179586476925286766559;
  if (rd < 2 || rd > SSA_ROPE_MAX_DIM || rd % 2 || !freq || !(base > 1.0) || !std::isfinite(base))
    return SSA_ERR_INVALID_ARG;
  if (scaling < SSA_ROPE_PLAIN || scaling > SSA_ROPE_YARN) return SSA_ERR_UNSUPPORTED;
  if (scaling != SSA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return SSA_ERR_INVALID_ARG;
  const bool banded = scaling == SSA_ROPE_BANDS || scaling == SSA_ROPE_YARN;
  if (banded && (!(original_len > 0.0) || !(low > 0.0) || !(high > low) ||
                 !std::isfinite(original_len) || !std::isfinite(high)))
    return SSA_ERR_INVALID_ARG;
  if (scaling == SSA_ROPE_NTK && rd > 2) base *= std::pow(factor, (double)rd / (rd - 2));
  // YaRN: the pair whose wavelength fits r times into the original length
  auto pair_of = [&](double r) {
    return rd * std::log(original_len / (two_pi * r)) / (2.0 * std::log(base));
  };
  double lo = 0, hi = 0;
  if (scaling == SSA_ROPE_YARN) {
    lo = std::fmax(std::floor(pair_of(high)), 0.0);
    hi = std::fmin(std::ceil(pair_of(low)), rd - 1.0);
  }
  for (int i = 0; i < rd / 2; ++i) {
    double th = std::pow(base, -2.0 * i / rd);
    if (scaling == SSA_ROPE_LINEAR) {
      th /= factor;
    } else if (scaling == SSA_ROPE_BANDS) {
      double mix = (original_len * th / two_pi - low) / (high - low);
      mix = std::fmin(std::fmax(mix, 0.0), 1.0);
      th = th * mix + th / factor * (1.0 - mix);
    } else if (scaling == SSA_ROPE_YARN) {
      double ramp = (i - lo) / std::fmax(hi - lo, 1e-3);
      ramp = std::fmin(std::fmax(ramp, 0.0), 1.0);
      th = th / factor * ramp + th * (1.0 - ramp);
    }
    freq[i] = (uint64_t)std::nearbyint(std::ldexp(th / two_pi, 64));
  }
  if (attn_factor) *attn_factor = scaling == SSA_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return SSA_OK;
}

}  // namespace ssa
