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
// shuffles and the row is read once.
#include "rope.cuh"

namespace ssa {
namespace {

constexpr int kCtas = 4;                 // per SM
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

// The token of a warp (more than one warp a token only where they fit 32 bits).
__device__ __forceinline__ long long token_of(const NormParams& p, long long gw) {
  return p.split == 1 ? gw : (long long)((uint32_t)gw / (uint32_t)p.split);
}

// 16 bytes as pairs of floats, and back.
template <typename T, int V> __device__ __forceinline__ void widen(uint4 u, uint64_t* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    if constexpr (sizeof(T) == 4) {
      x[i] = pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else {
      const float2 f = unpack<T>(w[i]);
      x[i] = pack2(f.x, f.y);
    }
  }
}
template <typename T, int V> __device__ __forceinline__ uint4 narrow(const uint64_t* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float2 f = unpack2(x[i]);
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(f.x);
      w[2 * i + 1] = __float_as_uint(f.y);
    } else {
      w[i] = pack<T>(f.x, f.y);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows in registers: D and rd / 2 (INTER: rd) multiples of V = 16 bytes, at
// most 32 units to a row.  Weights, cosines and sines are multiplied once a token
// (and layer) into a table of the warp's own in shared memory: a turned pair is
//   a' = (f a) (wa c) - (f b) (wb s),  b' = (f b) (wb c) + (f a) (wa s),
// f the row's norm, four factors a pair (elements that do not turn: one factor).
// (32,768 tokens of 36 heads of 128 in bf16: 106 us, the bytes at the copy rate take
// 89.  The factors in registers took 120: 80 registers, 24 warps per SM.  64 registers
// allow 32 warps; the 16-bit kernel for two halves spills 32 bytes for it.)
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kCtas) norm_rope_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) float4 s_f[];          // [warps][units * NF], then cos and sin [warps][rd / 2]
  constexpr int V = 16 / sizeof(T);
  constexpr int NA = INTER ? 1 : 2;      // accesses of a unit that turns
  constexpr int H = V / 2;               // pairs of floats of an access
  constexpr int NF = INTER ? H : V;      // entries of a unit
  constexpr int NR = kInFlight / NA;     // rows in flight
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long gw = (long long)blockIdx.x * (kRopeThreads / 32) + warp;
  const long long tok = token_of(p, gw);
  if (tok >= p.T) return;
  const int part = (int)(gw - tok * p.split);
  float4* fac = s_f + warp * p.units * NF;
  float2* cs_w = reinterpret_cast<float2*>(s_f + (kRopeThreads / 32) * p.units * NF) + warp * (p.rd / 2);
  const int col = lane & (p.lanes_row - 1), first = lane / p.lanes_row;
  const bool on = col < p.units, turns = col < p.u_rot, two = NA == 2 && turns;
  const int e = turns ? col * V : p.rd + (col - p.u_rot) * V;
  const int step = p.rd / 2;
  const float inv_d = 1.0f / (float)p.D;
  const float4* my = fac + (on ? col : 0);               // entry c of unit u at [c * units + u]: no bank twice

  bool have = false;
  for (int xi = 0; xi < p.n_x; ++xi) {
    const RopeRows& x = p.x[xi];
    const int heads = x.x.heads, base = part * x.per_warp, r1 = min(base + x.per_warp, p.L * heads);
    const float* weights = p.w[xi];
    int w_of = -1;                                              // the layer of the factors
    for (int r = base; r < r1;) {                               // a layer's rows together
      const int l = r / heads, h0 = r - l * heads, n = min(heads - h0, r1 - r);
      const T* in = static_cast<const T*>(x.x.in) + l * x.x.is[0] + tok * x.x.is[1] + (h0 + first) * x.x.is[2] + e;
      T* out = static_cast<T*>(x.x.out) + l * x.x.os[0] + tok * x.x.os[1] + (h0 + first) * x.x.os[2] + e;
      for (int k = 0; k < n; k += p.rows_pass * NR) {
        uint4 a[NR], b[NR];
        const int left = on ? n - k - first : 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          a[i] = b[i] = make_uint4(0, 0, 0, 0);
          if (left > i * p.rows_pass) {
            a[i] = *reinterpret_cast<const uint4*>(in);
            if (two) b[i] = *reinterpret_cast<const uint4*>(in + step);
          }
          in += x.in_step;
        }
        const float* w = weights ? weights + l * p.w_step[xi] : nullptr;
        float2 early[2];                  // the first factors' weights, on their way with the rows
        if (!have) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            early[j] = make_float2(1.0f, 1.0f);
            const int at = lane + 32 * j;
            if (w && at < p.u_rot * NF)
              early[j] = INTER ? make_float2(w[2 * at], w[2 * at + 1]) : make_float2(w[at], w[at + step]);
          }
          fill_table(p, tok, lane, cs_w);
        }
        if (w_of < 0 || (p.w_step[xi] && w_of != l)) {
          w_of = l;
          __syncwarp();
#pragma unroll 2
          for (int j = lane; j < p.units * NF; j += 32) {
            float4 f = make_float4(1, 0, 0, 0);
            if (j < p.u_rot * NF) {
              const int i0 = INTER ? 2 * j : j, i1 = INTER ? 2 * j + 1 : j + step;
              float wa, wb;
              if (!have && j < 64) {
                wa = j < 32 ? early[0].x : early[1].x;
                wb = j < 32 ? early[0].y : early[1].y;
              } else {
                wa = w ? w[i0] : 1.0f;
                wb = w ? w[i1] : 1.0f;
              }
              const float2 c = cs_w[j];
              // NA == 2: wa c, wa s, wb c, -wb s; INTER: wa c, wb c, -wb s, wa s
              f = INTER ? make_float4(wa * c.x, wb * c.x, -wb * c.y, wa * c.y)
                        : make_float4(wa * c.x, wa * c.y, wb * c.x, -wb * c.y);
            } else if (INTER) {
              const int i0 = p.rd + 2 * (j - p.u_rot * NF);
              f = make_float4(w ? w[i0] : 1.0f, w ? w[i0 + 1] : 1.0f, 0, 0);
            } else if (w) {
              f.x = w[p.rd + j - p.u_rot * NF];
            }
            float* at = reinterpret_cast<float*>(fac + (INTER ? j % NF : j % NF & ~1) * p.units + j / NF);
            if (INTER) {
              *reinterpret_cast<float4*>(at) = f;
            } else {                      // two pairs' factors side by side, as they are multiplied
              at += j & 1;
              at[0] = f.x;
              at[2] = f.y;
              at[4 * p.units] = f.z;
              at[4 * p.units + 2] = f.w;
            }
          }
          __syncwarp();
        }
        have = true;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          uint64_t u[H], v[H], s2 = 0;
          widen<T, V>(a[i], u);
#pragma unroll
          for (int c = 0; c < H; ++c) s2 = fma2(u[c], u[c], s2);
          if constexpr (NA == 2) {
            widen<T, V>(b[i], v);
#pragma unroll
            for (int c = 0; c < H; ++c) s2 = fma2(v[c], v[c], s2);
          }
          const float2 s1 = unpack2(s2);
          float ss = s1.x + s1.y;
          for (int o = 1; o < p.lanes_row; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float f = rsqrtf(fmaf(ss, inv_d, p.eps));
          if (left > i * p.rows_pass) {
            const uint64_t f2 = pack2(f, f);
#pragma unroll
            for (int c = 0; c < H; ++c) {
              u[c] = mul2(u[c], f2);
              if constexpr (NA == 2) {
                v[c] = mul2(v[c], f2);
                const ulonglong2 ga = *reinterpret_cast<const ulonglong2*>(my + 2 * c * p.units);
                const ulonglong2 gb = *reinterpret_cast<const ulonglong2*>(my + (2 * c + 1) * p.units);
                const uint64_t z = fma2(v[c], gb.y, mul2(u[c], ga.x));
                v[c] = fma2(u[c], ga.y, mul2(v[c], gb.x));
                u[c] = z;
              } else {
                const ulonglong2 g = *reinterpret_cast<const ulonglong2*>(my + c * p.units);
                const float2 t = unpack2(u[c]);
                u[c] = fma2(pack2(t.y, t.x), g.y, mul2(u[c], g.x));
              }
            }
            *reinterpret_cast<uint4*>(out) = narrow<T, V>(u);
            if constexpr (NA == 2) {
              if (two) *reinterpret_cast<uint4*>(out + step) = narrow<T, V>(v);
            }
          }
          out += x.out_step;
        }
      }
      r += n;
    }
  }
}

// Any dimensions, strides and alignment: a warp per row, element by element,
// the row read twice.  (One row in flight, 2 bytes a lane: 32,768 tokens of 36 heads in
// bf16 one element off take 328 us, 1.8 TB/s; heads of 80, 40 of them turned, 362,
// 1.0 TB/s.)
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_any_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ float2 s_cs[];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = p.rd / 2;
  const long long gw = (long long)blockIdx.x * (kRopeThreads / 32) + warp;
  const long long tok = token_of(p, gw);
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
  // a warp per token where the tokens fill the machine, else a token's rows over
  // several warps, down to one pass each (rounded down: 4,099 tokens x 48 rows in one
  // wave of a warp each 36 us, in 1.7 waves of half a token 48)
  long long rows = 0;
  for (int i = 0; i < p.n_x; ++i) rows += (long long)p.L * p.x[i].x.heads;
  const long long most = (rows + p.rows_pass - 1) / p.rows_pass;
  long long split = (long long)kCtas * (kRopeThreads / 32) * num_sms / p.T;
  if (split > most) split = most;
  if (split < 1) split = 1;
  p.split = (int)split;
  for (int i = 0; i < p.n_x; ++i) {
    RopeRows& x = p.x[i];
    const long long n = (long long)p.L * x.x.heads, per = (n + split - 1) / split;
    x.per_warp = (int)((per + p.rows_pass - 1) / p.rows_pass * p.rows_pass);
    x.in_step = p.rows_pass * x.x.is[2];
    x.out_step = p.rows_pass * x.x.os[2];
  }
  const long long ctas = ((long long)p.T * p.split + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  size_t smem = (size_t)(kRopeThreads / 32) * p.rd / 2 * sizeof(float2);
  if (vec) smem += (size_t)(kRopeThreads / 32) * p.units * (INTER ? V / 2 : V) * sizeof(float4);
  const auto kernel = vec ? norm_rope_kernel<T, INTER> : norm_rope_any_kernel<T, INTER>;
  if (smem > 48 * 1024)
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) return e;
  const cudaError_t e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(kRopeThreads), smem, s, p);
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
