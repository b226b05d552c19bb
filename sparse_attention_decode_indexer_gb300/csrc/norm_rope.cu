// norm_rope.cu -- norms of queries and keys, head by head, and their rotary
// positions in the same pass.
//
// For every head x[D] of q (weights wq) and of k (wk):
//   y = x / sqrt(mean(x^2) + eps) * w[layer],
// then the rotation of rope.cu on y, in fp32, rounded once at the end.
//
// What bounds it: each element read and written once, HBM.  As in rope.cu a
// warp serves one token (few tokens: a share of its rows), computes the token's
// cos and sin once, and walks over its (layer, head) rows.  A row lies in the
// registers of 2^n lanes, 16 bytes of each half of the rotated part (or of the
// interleaved pairs, or of the rest) to a lane, so that the sum of squares is n
// shuffles and the row is read once.  A lane's weights stay in registers while
// the layer does.
#include "rope.cuh"

namespace ssa {
namespace {

constexpr int kCtas = 3;                 // per SM
constexpr int kInFlight = 4;             // 16-byte loads of a lane

struct NormParams {
  RopeRows x[2];
  const float* w[2];                     // null: ones
  int64_t w_step[2];                     // floats from a layer's weights to the next's
  int n_x;
  const uint64_t* freq;
  const void* pos;
  int64_t offset;
  float factor, eps;
  int pos64, D, rd, L, T;
  int u_rot, units;                      // 16-byte units of a row that turn, and all
  int lanes_row, rows_pass;              // lanes on a row (a power of two), rows side by side
  int split;                             // warps on one token
};

// The token's cos and sin, a pair a lane and round.
__device__ __forceinline__ void fill_table(const NormParams& p, long long tok, int lane, float2* cs) {
  const int64_t raw = p.pos64 ? static_cast<const int64_t*>(p.pos)[tok]
                              : (int64_t) static_cast<const int32_t*>(p.pos)[tok];
  for (int i = lane; i < p.rd / 2; i += 32) {
    const float2 t = turn((uint64_t)raw + (uint64_t)p.offset, p.freq[i]);
    cs[i] = make_float2(t.x * p.factor, t.y * p.factor);
  }
  __syncwarp();
}

// 16 bytes as floats, and back.
template <typename T, int V> __device__ __forceinline__ void widen(uint4 u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = __uint_as_float(w[i]);
    } else {
      const float2 f = unpack<T>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}
template <typename T, int V> __device__ __forceinline__ uint4 narrow(const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
    else w[i] = pack<T>(x[2 * i], x[2 * i + 1]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows in registers: D and rd / 2 (INTER: rd) multiples of V = 16 bytes, at
// most 32 units to a row.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kCtas) norm_rope_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ float2 s_cs[];       // [warps][rd / 2]
  constexpr int V = 16 / sizeof(T);
  constexpr int NA = INTER ? 1 : 2;      // accesses of a unit that turns
  constexpr int NP = INTER ? V / 2 : V;  // its pairs
  constexpr int NR = kInFlight / NA;     // rows in flight
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * (kRopeThreads / 32) + warp;
  const long long tok = gw / p.split;
  if (tok >= p.T) return;
  const int part = (int)(gw - tok * p.split);
  float2* cs_w = s_cs + warp * (p.rd / 2);
  const int col = lane & (p.lanes_row - 1), first = lane / p.lanes_row;
  const bool on = col < p.units, turns = col < p.u_rot, two = NA == 2 && turns;
  const int e = turns ? col * NP * (INTER ? 2 : 1) : p.rd + (col - p.u_rot) * V;
  const int step = p.rd / 2;
  const float inv_d = 1.0f / (float)p.D;

  bool have = false;
  float2 cs[NP];
  for (int xi = 0; xi < p.n_x; ++xi) {
    const RopeRows& x = p.x[xi];
    const int heads = x.x.heads, rows = p.L * heads;
    const int base = part * x.per_warp, r1 = min(base + x.per_warp, rows);
    int left = r1 - base - first;                               // rows from this lane's on
    int l = (base + first) / heads, h = base + first - l * heads;
    const int dl = p.rows_pass / heads;
    const T* in = static_cast<const T*>(x.x.in) + l * x.x.is[0] + tok * x.x.is[1] + h * x.x.is[2] + e;
    T* out = static_cast<T*>(x.x.out) + l * x.x.os[0] + tok * x.x.os[1] + h * x.x.os[2] + e;
    int w_of = -1;                                              // the layer of wa, wb
    __align__(16) float wa[V], wb[V];
#pragma unroll
    for (int i = 0; i < V; ++i) wa[i] = wb[i] = 1.0f;
    for (int r = base; r < r1; r += p.rows_pass * NR) {
      uint4 a[NR], b[NR];
      int layer[NR];
      uint32_t wraps = 0;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        a[i] = b[i] = make_uint4(0, 0, 0, 0);
        layer[i] = l;
        if (on && left > i * p.rows_pass) {
          a[i] = *reinterpret_cast<const uint4*>(in);
          if (two) b[i] = *reinterpret_cast<const uint4*>(in + step);
        }
        in += x.in_step;
        h += x.dh;
        l += dl;
        if (h >= heads) {
          h -= heads;
          ++l;
          in += x.in_wrap;
          wraps |= 1u << i;
        }
      }
      if (!have) {                        // while the first loads are in flight
        fill_table(p, tok, lane, cs_w);
#pragma unroll
        for (int k = 0; k < NP; ++k) cs[k] = turns ? cs_w[col * NP + k] : make_float2(1.0f, 0.0f);
        have = true;
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const bool mine = on && left > i * p.rows_pass;
        if (mine && p.w[xi] && layer[i] != w_of) {
          w_of = layer[i];
          const float* w = p.w[xi] + w_of * p.w_step[xi] + e;
#pragma unroll
          for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(wa + k) = *reinterpret_cast<const float4*>(w + k);
          if (two) {
#pragma unroll
            for (int k = 0; k < V; k += 4)
              *reinterpret_cast<float4*>(wb + k) = *reinterpret_cast<const float4*>(w + step + k);
          }
        }
        float u[V], v[V];
        widen<T, V>(a[i], u);
        if constexpr (NA == 2) widen<T, V>(b[i], v);
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < V; ++k) ss = fmaf(u[k], u[k], ss);
        if constexpr (NA == 2) {
#pragma unroll
          for (int k = 0; k < V; ++k) ss = fmaf(v[k], v[k], ss);
        }
        for (int o = 1; o < p.lanes_row; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float f = rsqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
        for (int k = 0; k < V; ++k) u[k] *= f * wa[k];
        if constexpr (NA == 2) {
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] *= f * wb[k];
          if (turns) {
#pragma unroll
            for (int k = 0; k < V; ++k) rotate(u[k], v[k], cs[k]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < NP; ++k) rotate(u[2 * k], u[2 * k + 1], cs[k]);
        }
        if (mine) {
          *reinterpret_cast<uint4*>(out) = narrow<T, V>(u);
          if constexpr (NA == 2) {
            if (two) *reinterpret_cast<uint4*>(out + step) = narrow<T, V>(v);
          }
        }
        out += x.out_step;
        if (wraps >> i & 1) out += x.out_wrap;
      }
      left -= NR * p.rows_pass;
    }
  }
}

// Any dimensions, strides and alignment: a warp per row, element by element,
// the row read twice.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_any_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ float2 s_cs[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = p.rd / 2;
  const long long gw = (long long)blockIdx.x * (kRopeThreads / 32) + warp;
  const long long tok = gw / p.split;
  if (tok >= p.T) return;
  const int part = (int)(gw - tok * p.split);
  float2* cs = s_cs + warp * half;
  fill_table(p, tok, lane, cs);
  for (int xi = 0; xi < p.n_x; ++xi) {
    const RopeRows& x = p.x[xi];
    const int heads = x.x.heads, rows = p.L * heads;
    const int base = part * x.per_warp, r1 = min(base + x.per_warp, rows);
    for (int r = base; r < r1; ++r) {
      const int l = r / heads, h = r - l * heads;
      const T* in = static_cast<const T*>(x.x.in) + l * x.x.is[0] + tok * x.x.is[1] + h * x.x.is[2];
      T* out = static_cast<T*>(x.x.out) + l * x.x.os[0] + tok * x.x.os[1] + h * x.x.os[2];
      const float* w = p.w[xi] ? p.w[xi] + l * p.w_step[xi] : nullptr;
      float ss = 0.0f;
      for (int i = lane; i < p.D; i += 32) {
        const float v = one_in(in[i]);
        ss = fmaf(v, v, ss);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float f = rsqrtf(ss / (float)p.D + p.eps);
      // (in place: a lane writes what it alone reads from here on)
      for (int i = lane; i < half; i += 32) {
        const int i0 = INTER ? 2 * i : i, i1 = INTER ? 2 * i + 1 : i + half;
        float a = one_in(in[i0]) * (f * (w ? w[i0] : 1.0f)), b = one_in(in[i1]) * (f * (w ? w[i1] : 1.0f));
        rotate(a, b, cs[i]);
        out[i0] = one_out<T>(a);
        out[i1] = one_out<T>(b);
      }
      for (int i = p.rd + lane; i < p.D; i += 32) out[i] = one_out<T>(one_in(in[i]) * (f * (w ? w[i] : 1.0f)));
    }
  }
}

template <typename T, bool INTER>
cudaError_t launch_t(NormParams p, int num_sms, cudaStream_t s) {
  constexpr int V = 16 / sizeof(T);
  bool vec = p.D % V == 0 && (INTER ? p.rd : p.rd / 2) % V == 0;
  for (int i = 0; i < p.n_x; ++i)
    vec = vec && aligned(p.x[i].x, V, sizeof(T), p.L, p.T) && !((uintptr_t)p.w[i] & 15) && p.w_step[i] % 4 == 0;
  p.u_rot = p.rd / (INTER ? V : 2 * V);
  p.units = p.u_rot + (p.D - p.rd) / V;
  vec = vec && p.units <= 32;
  p.lanes_row = 1;
  while (p.lanes_row < p.units && p.lanes_row < 32) p.lanes_row *= 2;
  if (!vec) p.lanes_row = 32;
  p.rows_pass = 32 / p.lanes_row;
  // a warp per token where the tokens fill the machine (32 warps per SM), else
  // a token's rows over several warps, down to one pass each
  long long rows = 0;
  for (int i = 0; i < p.n_x; ++i) rows += (long long)p.L * p.x[i].x.heads;
  const long long most = (rows + p.rows_pass - 1) / p.rows_pass;
  long long split = (32LL * num_sms + p.T - 1) / p.T;
  if (split > most) split = most;
  p.split = (int)split;
  for (int i = 0; i < p.n_x; ++i) {
    RopeRows& x = p.x[i];
    const long long n = (long long)p.L * x.x.heads, per = (n + split - 1) / split;
    x.per_warp = (int)((per + p.rows_pass - 1) / p.rows_pass * p.rows_pass);
    const int dl = p.rows_pass / x.x.heads;
    x.dh = p.rows_pass % x.x.heads;
    x.in_step = dl * x.x.is[0] + x.dh * x.x.is[2];
    x.out_step = dl * x.x.os[0] + x.dh * x.x.os[2];
    x.in_wrap = x.x.is[0] - x.x.heads * x.x.is[2];
    x.out_wrap = x.x.os[0] - x.x.heads * x.x.os[2];
  }
  const long long ctas = ((long long)p.T * p.split + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const cudaError_t e = launch_pdl(vec ? norm_rope_kernel<T, INTER> : norm_rope_any_kernel<T, INTER>,
                                   dim3((unsigned)ctas), dim3(kRopeThreads),
                                   (size_t)(kRopeThreads / 32) * p.rd / 2 * sizeof(float2), s, p);
  count_launch();
  return e;
}

template <typename T>
cudaError_t launch_d(const NormParams& p, bool inter, int num_sms, cudaStream_t s) {
  return inter ? launch_t<T, true>(p, num_sms, s) : launch_t<T, false>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeArgs& a, const float* const* w, int64_t w_step, float eps,
                             cudaStream_t s) {
  NormParams p{};
  for (int i = 0; i < a.n_x; ++i) {
    if ((long long)a.n_layers * a.x[i].heads > 0x0FFFFFFF) return cudaErrorInvalidValue;
    p.x[i].x = a.x[i];
    p.w[i] = w[i];
    p.w_step[i] = w_step;
  }
  p.n_x = a.n_x;
  p.freq = a.freq;
  p.pos = a.pos;
  p.pos64 = a.pos64;
  p.offset = a.offset;
  p.factor = a.factor;
  p.eps = eps;
  p.D = a.D; p.rd = a.rd; p.L = a.n_layers; p.T = a.n_tokens;
  switch (a.dtype) {
    case SSA_BF16: return launch_d<__nv_bfloat16>(p, a.interleaved, a.num_sms, s);
    case SSA_F16: return launch_d<__half>(p, a.interleaved, a.num_sms, s);
    default: return launch_d<float>(p, a.interleaved, a.num_sms, s);
  }
}

}  // namespace ssa
