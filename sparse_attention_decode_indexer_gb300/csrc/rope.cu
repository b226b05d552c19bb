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
// bytes).  The angles are shared by all layers and heads of a token, so a warp
// serves one token: its lanes start their first loads, compute the token's cos
// and sin once (a pair or more per lane, exchanged through shared memory), and
// then only move and rotate 16-byte pieces.  Few tokens (a decode step) split
// a token's layers and heads over more warps, each of which computes the rd/2
// pairs again.
#include <cmath>
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace ssa {
namespace {

constexpr int kRopeThreads = 256;

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
  const uint64_t* freq;
  const void* pos;
  int64_t offset;
  float factor;
  int pos64, inverse, D, rd, L, T;
  int heads0, heads;                     // of q, of both
  int u_rot, units;                      // units of a row that turn, and with the tail
  int lanes_row, rows_pass;              // lanes on a row, rows side by side in a warp
  int split, per_warp;                   // warps on one token, rows of one of them
  int dl, dh;                            // rows_pass rows on, as layers and heads
};

// Rows in flight per lane: four 16-byte loads.
template <int NA> constexpr int rope_unroll() { return NA == 1 ? 4 : 2; }

// A unit is what a lane moves at once: V elements of each half of a head (or
// one pair), INTER: V elements that hold V / 2 pairs (or one pair, V = 1).  A
// lane keeps its unit, and its cos and sin, and walks over the token's
// (layer, head) rows.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeParams p) {
  extern __shared__ float2 s_cs[];       // [warps][rd / 2]
  using A = Vec<T, V>;
  constexpr int NA = (INTER && V > 1) ? 1 : 2;      // accesses of a unit
  constexpr int NP = (INTER && V > 1) ? V / 2 : V;  // pairs of a unit
  constexpr int NR = rope_unroll<NA>();
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = p.rd / 2;
  const long long gw = (long long)blockIdx.x * (kRopeThreads / 32) + warp;
  const long long tok = gw / p.split;
  if (tok >= p.T) return;
  const int part = (int)(gw - tok * p.split);
  float2* cs_w = s_cs + warp * half;
  const int col = lane % p.lanes_row, first = lane / p.lanes_row;
  const int r1 = min((part + 1) * p.per_warp, p.L * p.heads);

  bool have_table = false;
  for (int w0 = 0; w0 < p.units; w0 += p.lanes_row) {
    const int w = w0 + col;
    const bool turns = w < p.u_rot;
    // this unit's first element, and the distance to its second access
    const int e = turns ? (INTER ? w * NP * 2 : w * V) : p.rd + (w - p.u_rot) * V;
    const int step = INTER ? V : half;
    // the lanes left over idle
    int r = w < p.units && first < p.rows_pass ? part * p.per_warp + first : r1;
    int l = r / p.heads, h = r - l * p.heads;
    float2 cs[NP];
    for (int base = part * p.per_warp; base < r1; base += p.rows_pass * NR) {
      A a[NR][NA];
      T* out[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        out[i] = nullptr;
        if (r < r1) {
          const bool second = h >= p.heads0;
          const RopeTensor& x = p.x[second];
          const int hh = second ? h - p.heads0 : h;
          const T* in = static_cast<const T*>(x.in) + l * x.is[0] + tok * x.is[1] + hh * x.is[2] + e;
          out[i] = static_cast<T*>(x.out) + l * x.os[0] + tok * x.os[1] + hh * x.os[2] + e;
          a[i][0] = *reinterpret_cast<const A*>(in);
          if (NA > 1 && turns) a[i][NA - 1] = *reinterpret_cast<const A*>(in + step);
        }
        r += p.rows_pass;
        h += p.dh;
        l += p.dl;
        if (h >= p.heads) { h -= p.heads; ++l; }
      }
      if (!have_table) {                  // while the first loads are in flight
        const int64_t raw = p.pos64 ? static_cast<const int64_t*>(p.pos)[tok]
                                    : (int64_t) static_cast<const int32_t*>(p.pos)[tok];
        for (int i = lane; i < half; i += 32) {
          const float2 t = turn((uint64_t)raw + (uint64_t)p.offset, p.freq[i]);
          cs_w[i] = make_float2(t.x * p.factor, (p.inverse ? -t.y : t.y) * p.factor);
        }
        __syncwarp();
        have_table = true;
      }
      if (base == part * p.per_warp && turns) {
#pragma unroll
        for (int k = 0; k < NP; ++k) cs[k] = cs_w[w * NP + k];
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        if (!out[i]) continue;
        if (turns) {
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            T& ea = NA == 1 ? a[i][0].x[2 * k % V] : a[i][0].x[k % V];
            T& eb = NA == 1 ? a[i][0].x[(2 * k + 1) % V] : a[i][NA - 1].x[k % V];
            const float x = Conv<T>::in(ea), y = Conv<T>::in(eb);
            ea = Conv<T>::out(x * cs[k].x - y * cs[k].y);
            eb = Conv<T>::out(y * cs[k].x + x * cs[k].y);
          }
          if (NA > 1) *reinterpret_cast<A*>(out[i] + step) = a[i][NA - 1];
        }
        *reinterpret_cast<A*>(out[i]) = a[i][0];
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
  p.lanes_row = p.units < 32 ? p.units : 32;
  p.rows_pass = 32 / p.lanes_row;
  const int rows = p.L * p.heads;                              // of one token
  // a warp per token where the tokens fill the machine (32 warps per SM), else
  // a token's rows over several warps, down to one pass each
  const long long want = 32LL * num_sms;
  long long split = (want + p.T - 1) / p.T;
  const long long most = (rows + p.rows_pass - 1) / p.rows_pass;
  if (split > most) split = most;
  p.per_warp = (int)(((rows + split - 1) / split + p.rows_pass - 1) / p.rows_pass * p.rows_pass);
  p.split = (rows + p.per_warp - 1) / p.per_warp;
  p.dl = p.rows_pass / p.heads;
  p.dh = p.rows_pass % p.heads;
  const long long warps = (long long)p.T * p.split;
  const long long ctas = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  cudaError_t e = launch_pdl(rope_kernel<T, V, INTER>, dim3((unsigned)ctas), dim3(kRopeThreads),
                             (size_t)(kRopeThreads / 32) * p.rd / 2 * sizeof(float2), s, p);
  count_launch();
  return e;
}

template <typename T>
cudaError_t launch_rope_d(const RopeParams& p, bool inter, bool copy_tail, int num_sms,
                          cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  bool vec = p.D % V == 0 && (inter ? p.rd : p.rd / 2) % V == 0;
  for (int i = 0; i < (p.heads > p.heads0 ? 2 : 1); ++i)
    vec = vec && aligned(p.x[i], V, sizeof(T), p.L, p.T);
  if (vec)
    return inter ? launch_rope_t<T, V, true>(p, copy_tail, num_sms, s)
                 : launch_rope_t<T, V, false>(p, copy_tail, num_sms, s);
  return inter ? launch_rope_t<T, 1, true>(p, copy_tail, num_sms, s)
               : launch_rope_t<T, 1, false>(p, copy_tail, num_sms, s);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  RopeParams p{};
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
  p.heads0 = a.x[0].heads;
  p.heads = p.heads0 + (a.n_x > 1 ? a.x[1].heads : 0);
  if ((long long)p.L * p.heads > 0x0FFFFFFF) return cudaErrorInvalidValue;
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
