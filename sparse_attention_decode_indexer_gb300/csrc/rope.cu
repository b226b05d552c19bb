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

#include "rope.cuh"

namespace ssa {
namespace {

constexpr int kRopeCtas = 4;             // per SM
constexpr int kRopeRows = 4;             // accesses in flight per lane

// What a lane moves at once (a unit): with V > 1 16 bytes of each half of a
// head, or 16 bytes of interleaved pairs; with V = 1 one pair.
template <typename T, int V, bool INTER> struct Unit {
  static constexpr int NP = V;                      // pairs
  static constexpr int NA = 2;                      // accesses
  uint4 a, b;
  __device__ __forceinline__ void load(const T* p, int step, bool two) {
    a = *reinterpret_cast<const uint4*>(p);
    if (two) b = *reinterpret_cast<const uint4*>(p + step);
  }
  __device__ __forceinline__ void store(T* p, int step, bool two) const {
    *reinterpret_cast<uint4*>(p) = a;
    if (two) *reinterpret_cast<uint4*>(p + step) = b;
  }
  __device__ __forceinline__ void turn(const float2* cs) {
    uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        float u = __uint_as_float(x[i]), v = __uint_as_float(y[i]);
        rotate(u, v, cs[i]);
        x[i] = __float_as_uint(u);
        y[i] = __float_as_uint(v);
      } else {
        float2 u = unpack<T>(x[i]), v = unpack<T>(y[i]);
        rotate(u.x, v.x, cs[2 * i]);
        rotate(u.y, v.y, cs[2 * i + 1]);
        x[i] = pack<T>(u.x, u.y);
        y[i] = pack<T>(v.x, v.y);
      }
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
    b = make_uint4(y[0], y[1], y[2], y[3]);
  }
};

template <typename T, int V> struct Unit<T, V, true> {
  static constexpr int NP = V / 2;
  static constexpr int NA = 1;
  uint4 a;
  __device__ __forceinline__ void load(const T* p, int, bool) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store(T* p, int, bool) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void turn(const float2* cs) {
    uint32_t x[4] = {a.x, a.y, a.z, a.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float u = __uint_as_float(x[2 * i]), v = __uint_as_float(x[2 * i + 1]);
        rotate(u, v, cs[i]);
        x[2 * i] = __float_as_uint(u);
        x[2 * i + 1] = __float_as_uint(v);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 u = unpack<T>(x[i]);
        rotate(u.x, u.y, cs[i]);
        x[i] = pack<T>(u.x, u.y);
      }
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
  }
};

template <typename T> struct Pair {
  static constexpr int NP = 1;
  static constexpr int NA = 2;
  T a, b;
  __device__ __forceinline__ void load(const T* p, int step, bool two) {
    a = p[0];
    if (two) b = p[step];
  }
  __device__ __forceinline__ void store(T* p, int step, bool two) const {
    p[0] = a;
    if (two) p[step] = b;
  }
  __device__ __forceinline__ void turn(const float2* cs) {
    float u = one_in(a), v = one_in(b);
    rotate(u, v, *cs);
    a = one_out<T>(u);
    b = one_out<T>(v);
  }
};
template <typename T> struct Unit<T, 1, false> : Pair<T> {};
template <typename T> struct Unit<T, 1, true> : Pair<T> {};

struct RopeParams {
  RopeRows x[2];
  int n_x;
  const uint64_t* freq;
  const void* pos;
  int64_t offset;
  float factor;
  int pos64, inverse, D, rd, L, T;
  int u_rot, units;                      // units of a row that turn, and with the tail
  int lanes_row, rows_pass;              // lanes on a row, rows side by side in a warp
  int split;                             // warps on one token
};

// A lane keeps its unit of the head, and its cos and sin, and walks over the
// token's (layer, head) rows, a few of them in flight: up to 64 bytes.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeParams p) {
  extern __shared__ float2 s_cs[];       // [warps][rd / 2]
  using U = Unit<T, V, INTER>;
  constexpr int NP = U::NP, NR = kRopeRows / U::NA;
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = p.rd / 2;
  const long long gw = (long long)blockIdx.x * (kRopeThreads / 32) + warp;
  const long long tok = gw / p.split;
  if (tok >= p.T) return;
  const int part = (int)(gw - tok * p.split);
  float2* cs_w = s_cs + warp * half;
  const int col = lane % p.lanes_row, first = lane / p.lanes_row;

  bool have_table = false;
  for (int w0 = 0; w0 < p.units; w0 += p.lanes_row) {
    const int w = w0 + col;
    const bool turns = w < p.u_rot;
    // this unit's first element, and the distance to its second access
    const int e = turns ? (INTER ? w * NP * 2 : w * NP) : p.rd + (w - p.u_rot) * V;
    const int step = INTER ? 1 : half;
    const bool on = w < p.units && first < p.rows_pass;           // the lanes left over idle
    float2 cs[NP];
    bool have_cs = false;
    for (int xi = 0; xi < p.n_x; ++xi) {
      const RopeRows& x = p.x[xi];
      const int heads = x.x.heads, rows = p.L * heads;
      const int base = part * x.per_warp, r1 = min(base + x.per_warp, rows);
      int left = on ? r1 - base - first : 0;                      // rows from this lane's on
      const int l = (base + first) / heads;
      int h = base + first - l * heads;
      const T* in = static_cast<const T*>(x.x.in) + l * x.x.is[0] + tok * x.x.is[1] + h * x.x.is[2] + e;
      T* out = static_cast<T*>(x.x.out) + l * x.x.os[0] + tok * x.x.os[1] + h * x.x.os[2] + e;
      for (int r = base; r < r1; r += p.rows_pass * NR) {
        U u[NR];
        uint32_t wraps = 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          if (left > i * p.rows_pass) u[i].load(in, step, turns);
          in += x.in_step;
          h += x.dh;
          if (h >= heads) {
            h -= heads;
            in += x.in_wrap;
            wraps |= 1u << i;
          }
        }
        if (!have_table) {                // while the first loads are in flight
          const int64_t raw = p.pos64 ? static_cast<const int64_t*>(p.pos)[tok]
                                      : (int64_t) static_cast<const int32_t*>(p.pos)[tok];
          for (int i = lane; i < half; i += 32) {
            const float2 t = turn((uint64_t)raw + (uint64_t)p.offset, p.freq[i]);
            cs_w[i] = make_float2(t.x * p.factor, (p.inverse ? -t.y : t.y) * p.factor);
          }
          __syncwarp();
          have_table = true;
        }
        if (!have_cs) {
          have_cs = true;
#pragma unroll
          for (int k = 0; k < NP; ++k) cs[k] = turns ? cs_w[w * NP + k] : make_float2(1.0f, 0.0f);
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          if (left > i * p.rows_pass) {
            if (turns) u[i].turn(cs);
            u[i].store(out, step, turns);
          }
          out += x.out_step;
          if (wraps >> i & 1) out += x.out_wrap;
        }
        left -= NR * p.rows_pass;
      }
    }
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch_rope_t(RopeParams p, bool copy_tail, int num_sms, cudaStream_t s) {
  const int np = (INTER && V > 1) ? V / 2 : V;                 // pairs per unit
  p.u_rot = p.rd / 2 / np;
  p.units = p.u_rot + (copy_tail ? (p.D - p.rd) / V : 0);
  p.lanes_row = p.units < 32 ? p.units : 32;
  p.rows_pass = 32 / p.lanes_row;
  // a warp per token where the tokens fill the machine (32 warps per SM), else
  // a token's rows over several warps, down to one pass each
  long long rows = 0;                                          // of one token
  for (int i = 0; i < p.n_x; ++i) rows += (long long)p.L * p.x[i].x.heads;
  const long long want = 32LL * num_sms;
  long long split = (want + p.T - 1) / p.T;
  const long long most = (rows + p.rows_pass - 1) / p.rows_pass;
  if (split > most) split = most;
  p.split = (int)split;
  for (int i = 0; i < p.n_x; ++i) {
    RopeRows& x = p.x[i];
    const long long n = (long long)p.L * x.x.heads;
    const long long per = (n + split - 1) / split;
    x.per_warp = (int)((per + p.rows_pass - 1) / p.rows_pass * p.rows_pass);
    const int dl = p.rows_pass / x.x.heads;
    x.dh = p.rows_pass % x.x.heads;
    x.in_step = dl * x.x.is[0] + x.dh * x.x.is[2];
    x.out_step = dl * x.x.os[0] + x.dh * x.x.os[2];
    x.in_wrap = x.x.is[0] - x.x.heads * x.x.is[2];
    x.out_wrap = x.x.os[0] - x.x.heads * x.x.os[2];
  }
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
  for (int i = 0; i < p.n_x; ++i) vec = vec && aligned(p.x[i].x, V, sizeof(T), p.L, p.T);
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
    p.x[i].x = a.x[i];
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
  p.n_x = a.n_x;
  for (int i = 0; i < a.n_x; ++i)
    if ((long long)a.n_layers * a.x[i].heads > 0x0FFFFFFF) return cudaErrorInvalidValue;
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
