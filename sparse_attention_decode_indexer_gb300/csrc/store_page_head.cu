// store_page_head.cu -- the store of the page_head formats: 8-bit K and V codes
// with one fp32 scale per (page, KV head) for K and one for V, the host
// mirror's and the pool's copies, and the indexer slab.
//
// The mathematics, per page, KV head and tensor, for the tokens x a call
// stores into the page (amax over the finite values; qmax = 127 or 448):
//   need = amax / qmax
//   s'   = need on a page without tokens (slab count 0), else max(s, need)
//   codes already there, when s' > s: Q(code * (s / s'))
//   new codes: Q(x / s'), all zero when s' = 0
// Q rounds to nearest even (int8: clamped to +-127; e4m3: saturating).  IEEE
// fp32 division and rounding throughout, one operation at a time, so that the
// codes follow from the definition bit for bit.
//
// What bounds it: bf16 K and V in (4 Hkv D bytes a token) and codes out
// (2 Hkv D, and as many again to the mirror over the host link), so HBM or the
// host link; an append of one token per request is latency, a chain of
// dependent reads (position, slot, scale).
//
// A run is the consecutive tokens of one page in a call.  Three ways to store
// one, the division x / s' being most of their arithmetic.  s' is the block's,
// so its reciprocal is computed once and each quotient is corrected from its
// fused residual (after Markstein 1990), two elements per f32x2 instruction: 3
// instead of about 20 per pair.
//   * a whole page (prefill): a CTA per head.  Its rows wait in shared memory
//     while the scale becomes known, so that each input is read once.  A thread
//     has 8 dimensions of 4 consecutive tokens at a time, so V leaves as whole
//     words of its d-major block through a swizzled tile.  The heads meet only
//     in the slab's scale (max over all heads): they form a cluster and push
//     their maxima into each other's shared memory;
//   * other runs, a decode step's single tokens above all: a warp per head,
//     four dimensions a lane, the heads of a run in one CTA, so that a run costs
//     three dependent reads (position, state, scale).  16 rows of one 16-byte
//     unit of V leave as units; a single token writes one byte in every row of
//     its block, 32-byte sectors that come to about half of a large append's
//     time (1,000 tokens of 12 layers and 4 heads, 118 us);
//   * whole pages with values that are not finite, or scales near the ends of
//     fp32: 128 threads, one per dimension, plain division.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace ssa {
namespace {

constexpr int kHD = 128;                 // head_dim
constexpr int kMaxP = 128;
constexpr int kRowUnits = kHD * 2 / 16;  // 16-byte units of a bf16 token row
constexpr int kMaxPiece = 128;           // most tokens whose runs one CTA of the append kernel stores
constexpr int kTokBatch = 4;             // tokens of a run in flight, for their maxima

struct StorePHParams {
  uint8_t *k_pool, *v_pool;
  float *k_scale, *v_scale;
  uint8_t *k_mir, *v_mir;
  float *k_scale_m, *v_scale_m;
  int8_t* slab;
  float* slab_scale;
  float* slab_sum;
  int32_t* slab_cnt;
  const int32_t* slot_of;
  const __nv_bfloat16 *k, *v;            // [n_layers][T][Hkv][D]
  const int64_t* pos;
  int32_t* status;
  int T, layer0, Lp, S, Hkv;
  int chunk;                             // append: tokens whose runs one CTA stores
  int whole;                             // append: whole pages are the other kernel's
};

// A 4-byte word into the same shared variable of CTA `rank` of the cluster,
// counted by that CTA's barrier.
__device__ __forceinline__ void push_f32(const float* p, uint64_t* bar, int rank, float v) {
  uint32_t a, m;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(m) : "r"(smem_u32(bar)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
               ::"r"(a), "r"(__float_as_uint(v)), "r"(m) : "memory");
}

template <bool I8>
__device__ __forceinline__ uint8_t quant(float x) {
  if (I8) {
    // NaN has no int8 code: 0
    const float r = fminf(fmaxf(rintf(x), -127.0f), 127.0f);
    return x != x ? 0 : (uint8_t)(int8_t)(int)r;
  }
  return (uint8_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

template <bool I8>
__device__ __forceinline__ float value(uint8_t c) {
  if (I8) return (float)(int8_t)c;
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// The codes already in a block of one tensor, again at the scale that grew by
// 1 / ratio: from the pool's copy where there is one (the mirror's bytes are
// the same), to both.  (One unit in flight per thread: an append of 64 tokens,
// 12 layers and 4 heads takes 25 us where 6 % of the blocks' scales grow and 48
// where all do, against 7.7 without.)
template <bool I8>
__device__ __forceinline__ void rescale_block(uint8_t* mir, uint8_t* pool, int bytes, float ratio,
                                              int tid, int nthreads) {
  const uint8_t* from = pool ? pool : mir;
  for (int u = tid; u < bytes / 16; u += nthreads) {
    uint4 w = reinterpret_cast<const uint4*>(from)[u];
    uint8_t* b = reinterpret_cast<uint8_t*>(&w);
#pragma unroll
    for (int i = 0; i < 16; ++i) b[i] = quant<I8>(value<I8>(b[i]) * ratio);
    if (mir) reinterpret_cast<uint4*>(mir)[u] = w;
    if (pool) reinterpret_cast<uint4*>(pool)[u] = w;
  }
}

// Where one page's block of one head is held: block number in the mirror and
// in the pool, -1 where it is not (K's and V's blocks and scales are alike).
struct Block {
  long long m, s;
  __device__ __forceinline__ Block(const StorePHParams& p, int layer, int pg, int slot, int h) {
    m = p.k_mir ? ((long long)layer * p.Lp + pg) * p.Hkv + h : -1;
    s = slot >= 0 ? ((long long)layer * p.S + slot) * p.Hkv + h : -1;
  }
  // the scale, from the pool where it is there (the mirror's is the same)
  __device__ __forceinline__ float scale(const float* mir, const float* pool) const {
    return s >= 0 ? pool[s] : (m >= 0 ? mir[m] : 0.0f);
  }
  __device__ __forceinline__ void set_scale(float* mir, float* pool, float v) const {
    if (m >= 0) mir[m] = v;
    if (s >= 0) pool[s] = v;
  }
  __device__ __forceinline__ uint8_t* mirror(uint8_t* base, int pe) const {
    return m >= 0 ? base + m * pe : nullptr;
  }
  __device__ __forceinline__ uint8_t* slot(uint8_t* base, int pe) const {
    return s >= 0 ? base + s * pe : nullptr;
  }
};

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Divides by one block's scale, to quotients whose codes are those of the IEEE
// quotients.  With ny = -RN(1 / s) and nx = -x, one step corrects the quotient
// by its residual q s - x; the signs are such that a zero keeps its own.  The
// result is RN(x / s + e) with |e| < 2^-45 x / s, so it can differ from
// RN(x / s), and then by one unit, only where x / s lies that close to the
// middle between two floats; and a code can differ only where one of the two
// is a border between codes (at most 9 significant bits).  x has 8 significant
// bits and s 24, and the only such s has all of them set (with x a power of
// two): the search over every border is a test.  So: any s in [2^-90, 2^100]
// but those, x finite; nothing on the way over- or underflows then unless the
// quotient is below 2^-12 (every code 0).
struct Divider {
  uint64_t s2, ny2;
  __device__ __forceinline__ Divider(float2 s) : s2(pack2(s.x, s.x)), ny2(pack2(s.y, s.y)) {}
  // two negated elements -> the two quotients
  __device__ __forceinline__ uint64_t operator()(float nx0, float nx1) const {
    const uint64_t nx = pack2(nx0, nx1);
    const uint64_t q = mul2(nx, ny2);
    return fma2(fma2(q, s2, nx), ny2, q);
  }
};

__device__ __forceinline__ bool divides(float s) {
  return s >= 0x1p-90f && s <= 0x1p100f && (__float_as_uint(s) & 0x7FFFFFu) != 0x7FFFFFu;
}

// Four quotients -> four codes, the first in byte 0.
template <bool I8>
__device__ __forceinline__ uint32_t codes4(uint64_t a, uint64_t b) {
  float x0, x1, x2, x3;
  unpack2(a, x0, x1);
  unpack2(b, x2, x3);
  if (I8) {
    // |x| <= 127 (1 + 2^-24): adding 1.5 * 2^23 rounds to nearest even and
    // leaves the code in the low byte
    const float m = 12582912.0f;
    const uint32_t lo = __byte_perm(__float_as_uint(x0 + m), __float_as_uint(x1 + m), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(x2 + m), __float_as_uint(x3 + m), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  return f32x4_to_e4m3x4(x0, x1, x2, x3);
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ void copy_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
               : "memory");
}

// Largest |bf16| so far per half, NaN if there is one (so: bits from 0x7F80 on
// where a value is not finite)
__device__ __forceinline__ void absmax(__nv_bfloat162& m, uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
}

__device__ __forceinline__ uint32_t max_bits(__nv_bfloat162 m) {
  const uint32_t w = *reinterpret_cast<uint32_t*>(&m);
  return __reduce_max_sync(0xffffffffu, max(w >> 16, w & 0xFFFFu));
}

// E consecutive bf16 of a row, as they lie in memory.
template <int E> struct Row;
template <> struct Row<1> {
  __nv_bfloat16 v;
  __device__ __forceinline__ float at(int) const { return __bfloat162float(v); }
};
template <> struct Row<4> {
  uint2 v;
  __device__ __forceinline__ float at(int i) const {
    const uint32_t w = i < 2 ? v.x : v.y;
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};

// Stores a run of one head, whatever its tokens and values, with 128 / E
// threads that have E dimensions each: a warp (E = 4), or four (E = 1; then
// every thread of the CTA calls it, `active` those with a dimension, and s_max
// [2][4] is their scratch).  row_of(r): the page's row of token r.  kin, vin:
// the thread's elements of the first token, rows HD apart; k0, v0: their
// values.  sum: the slab's sums, updated.
template <bool I8, int P, int E, typename RowOf>
__device__ __forceinline__ void store_run(const StorePHParams& p, const Block& blk, bool active,
                                          int d, const Row<E>* kin, const Row<E>* vin, Row<E> k0,
                                          Row<E> v0, int HD, int R, RowOf row_of, int cnt0,
                                          float (&sum)[E], float (*s_max)[4]) {
  constexpr float kQmax = I8 ? 127.0f : 448.0f;
  constexpr int pe = P * kHD;              // codes of one head of one page
  constexpr int NT = kHD / E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rs = HD / E;
  const float old_k = cnt0 > 0 ? blk.scale(p.k_scale_m, p.k_scale) : 0.0f;
  const float old_v = cnt0 > 0 ? blk.scale(p.v_scale_m, p.v_scale) : 0.0f;
  // finite maxima of the run
  float ak = 0.0f, av = 0.0f;
  bool finite = true;
  auto take = [&](float& m, const Row<E>& x) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float a = fabsf(x.at(e));
      if (a < INFINITY) m = fmaxf(m, a);
      else finite = false;
    }
  };
  if (active) {
    take(ak, k0);
    take(av, v0);
    for (int r0 = 1; r0 < R; r0 += kTokBatch) {
      Row<E> xk[kTokBatch], xv[kTokBatch];
#pragma unroll
      for (int i = 0; i < kTokBatch; ++i)
        if (r0 + i < R) {
          xk[i] = kin[(size_t)(r0 + i) * rs];
          xv[i] = vin[(size_t)(r0 + i) * rs];
        }
#pragma unroll
      for (int i = 0; i < kTokBatch; ++i)
        if (r0 + i < R) {
          take(ak, xk[i]);
          take(av, xv[i]);
        }
    }
  }
  ak = warp_max(ak);
  av = warp_max(av);
  if constexpr (E == 1) {
    if (active && lane == 0) {
      s_max[0][warp] = ak;
      s_max[1][warp] = av;
    }
    __syncthreads();                       // (every thread has read the old scales)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      ak = fmaxf(ak, s_max[0][w]);
      av = fmaxf(av, s_max[1][w]);
    }
  } else {
    __syncwarp();                          // (every lane has read the old scales)
  }
  const float need_k = ak / kQmax, need_v = av / kQmax;
  const float sk = cnt0 > 0 ? fmaxf(old_k, need_k) : need_k;
  const float sv = cnt0 > 0 ? fmaxf(old_v, need_v) : need_v;
  uint8_t *km = blk.mirror(p.k_mir, pe), *kp = blk.slot(p.k_pool, pe);
  uint8_t *vm = blk.mirror(p.v_mir, pe), *vp = blk.slot(p.v_pool, pe);
  if (active) {
    if (d == 0) {
      blk.set_scale(p.k_scale_m, p.k_scale, sk);
      blk.set_scale(p.v_scale_m, p.v_scale, sv);
    }
    const bool gk = cnt0 > 0 && sk > old_k, gv = cnt0 > 0 && sv > old_v;
    if ((km || kp) && gk) rescale_block<I8>(km, kp, pe, old_k / sk, d / E, NT);
    if ((km || kp) && gv) rescale_block<I8>(vm, vp, pe, old_v / sv, d / E, NT);
  }
  // the new codes go on top
  if (E == 1) __syncthreads();
  else __syncwarp();
  if (!active) return;
  float2 dsk = make_float2(sk, 0.0f), dsv = make_float2(sv, 0.0f);
  bool exact = false;
  if (E == 4) {
    exact = __all_sync(0xffffffffu, finite) && divides(sk) && divides(sv);
    dsk.y = exact ? -(1.0f / sk) : 0.0f;
    dsv.y = exact ? -(1.0f / sv) : 0.0f;
  }
  const Divider dk(dsk), dv(dsv);
  Row<E> xk = k0, xv = v0;                 // token r
  for (int r = 0; r < R;) {
    const int j = row_of(r);
    if constexpr (E == 4) {
      // 16 rows of one unit of V: 16-byte stores instead of 16 byte stores
      if (exact && j % 16 == 0 && r + 16 <= R && row_of(r + 15) == j + 15) {
        uint32_t cv[4][4];                 // [dimension][4 tokens]
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          Row<E> yk[4], yv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            yk[i] = kin[(size_t)(r + 4 * q + i) * rs];
            yv[i] = vin[(size_t)(r + 4 * q + i) * rs];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t ck = codes4<I8>(dk(-yk[i].at(0), -yk[i].at(1)),
                                           dk(-yk[i].at(2), -yk[i].at(3)));
            const int off = (j + 4 * q + i) * kHD + d;
            if (km) *reinterpret_cast<uint32_t*>(km + off) = ck;
            if (kp) *reinterpret_cast<uint32_t*>(kp + off) = ck;
#pragma unroll
            for (int e = 0; e < E; ++e) sum[e] = sum[e] + yk[i].at(e);
          }
#pragma unroll
          for (int e = 0; e < E; ++e)
            cv[e][q] = codes4<I8>(dv(-yv[0].at(e), -yv[1].at(e)), dv(-yv[2].at(e), -yv[3].at(e)));
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint4 w = make_uint4(cv[e][0], cv[e][1], cv[e][2], cv[e][3]);
          if (vm) *reinterpret_cast<uint4*>(vm + (d + e) * P + j) = w;
          if (vp) *reinterpret_cast<uint4*>(vp + (d + e) * P + j) = w;
        }
        r += 16;
        if (r < R) {
          xk = kin[(size_t)r * rs];
          xv = vin[(size_t)r * rs];
        }
        continue;
      }
    }
    Row<E> nk = xk, nv = xv;               // token r + 1, on its way
    if (r + 1 < R) {
      nk = kin[(size_t)(r + 1) * rs];
      nv = vin[(size_t)(r + 1) * rs];
    }
    uint32_t ck = 0, cv = 0;
    if (E == 4 && exact) {
      ck = codes4<I8>(dk(-xk.at(0), -xk.at(1 % E)), dk(-xk.at(2 % E), -xk.at(3 % E)));
      cv = codes4<I8>(dv(-xv.at(0), -xv.at(1 % E)), dv(-xv.at(2 % E), -xv.at(3 % E)));
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        ck |= (uint32_t)(sk > 0.0f ? quant<I8>(xk.at(e) / sk) : 0) << (8 * e);
        cv |= (uint32_t)(sv > 0.0f ? quant<I8>(xv.at(e) / sv) : 0) << (8 * e);
      }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint8_t c = (uint8_t)(cv >> (8 * e));
      if (vm) vm[(d + e) * P + j] = c;
      if (vp) vp[(d + e) * P + j] = c;
      sum[e] = sum[e] + xk.at(e);          // the slab: fp32, token order
    }
    if (E == 1) {
      if (km) km[j * kHD + d] = (uint8_t)ck;
      if (kp) kp[j * kHD + d] = (uint8_t)ck;
    } else {
      if (km) *reinterpret_cast<uint32_t*>(km + j * kHD + d) = ck;
      if (kp) *reinterpret_cast<uint32_t*>(kp + j * kHD + d) = ck;
    }
    xk = nk;
    xv = nv;
    ++r;
  }
}

__device__ __forceinline__ int slab_code(float mean, float amax, float s) {
  return amax > 0.0f ? (int)fminf(fmaxf(rintf(mean / s), -127.0f), 127.0f) : 0;
}

// A whole page of tokens starts at t (given its position x): by its ends, which
// is all of it where positions increase.
template <int P>
__device__ __forceinline__ bool whole_page(const StorePHParams& p, int t, int64_t x) {
  return x % P == 0 && p.T - t >= P && p.pos[t + P - 1] == x + P - 1;
}

// Runs of any kind, but for whole pages where the other kernel stores those
// (p.whole).  A warp per KV head, four dimensions a lane; grid (CTAs, layers):
// a CTA stores the runs that start at its tokens, one or, MANY, up to p.chunk,
// as far apart as there are CTAs, so that a few single tokens behind a prefill
// are not left to a few CTAs.
template <bool I8, int P, bool MANY>
__global__ void __launch_bounds__(256, MANY ? 3 : 0) append_page_head_kernel(
    const __grid_constant__ StorePHParams p) {
  __shared__ int s_row[P];
  __shared__ int s_run;
  __shared__ float s_head[8];
  __shared__ uint32_t s_starts[kMaxPiece / 32];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, h = tid >> 5;
  const int Hkv = p.Hkv, HD = Hkv * kHD, d = 4 * lane;
  const int li = blockIdx.y, layer = p.layer0 + li;
  // the runs that start at its tokens: a lane per token, MANY: 32 of them per
  // warp; alone, in one round trip with the token's K and V
  const int first = blockIdx.x, step = gridDim.x;
  auto run_starts = [&](int i) -> bool {
    const long long at = first + (long long)i * step;
    if (at >= p.T) return false;
    const int t = (int)at;
    const int64_t x = p.pos[t], prev = t > 0 ? p.pos[t - 1] : -1;
    if (x < 0 || x / P >= p.Lp) {
      set_status(p.status, SSA_ST_BAD_ID);
      return false;
    }
    if (t > 0) {
      if (prev >= x) set_status(p.status, SSA_ST_BAD_POS);
      if (prev >= 0 && prev / P == x / P) return false;              // inside a run
    }
    return !(MANY && p.whole && whole_page<P>(p, t, x));
  };
  int words = 1;
  uint32_t runs = 0;
  Row<4> k0, v0;
  if (MANY) {
    words = (p.chunk + 31) / 32;
    for (int w = h; w < words; w += Hkv) {
      const uint32_t m = __ballot_sync(0xffffffffu, run_starts(32 * w + lane));
      if (lane == 0) s_starts[w] = m;
    }
    __syncthreads();
  } else {
    const size_t in_c = (((size_t)li * p.T + first) * HD + h * kHD + d) / 4;
    k0 = reinterpret_cast<const Row<4>*>(p.k)[in_c];
    v0 = reinterpret_cast<const Row<4>*>(p.v)[in_c];
    runs = run_starts(0) ? 1u : 0u;    // (the same in every thread)
  }
#pragma unroll 1
  for (int w = 0; w < words; ++w) {
    if (MANY) runs = s_starts[w];
#pragma unroll 1
    for (; runs; runs &= runs - 1) {
      const int t0 = first + (32 * w + __ffs(runs) - 1) * step;
      const size_t in_c = (((size_t)li * p.T + t0) * HD + h * kHD + d) / 4;
      const Row<4>* kin = reinterpret_cast<const Row<4>*>(p.k) + in_c;
      const Row<4>* vin = reinterpret_cast<const Row<4>*>(p.v) + in_c;
      if (MANY) {
        k0 = *kin;
        v0 = *vin;
      }
      const int pg = (int)(p.pos[t0] / P);
      const size_t lp = (size_t)layer * p.Lp + pg;
      const size_t so = lp * HD + h * kHD + d;
      const float4 old_sum = *reinterpret_cast<const float4*>(p.slab_sum + so);
      const int cnt0 = p.slab_cnt[lp];
      int slot = p.slot_of[lp];
      // the run's length
      if (tid == 0) s_run = P;
      __syncthreads();
      for (int r = tid; r < P; r += blockDim.x) {
        const int t = t0 + r;
        const int64_t x = t < p.T ? p.pos[t] : -1;
        if (x < 0 || x / P != pg) {
          atomicMin(&s_run, r);
        } else {
          s_row[r] = (int)(x % P);
          if (r > 0 && x <= p.pos[t - 1]) set_status(p.status, SSA_ST_BAD_POS);
        }
      }
      if (slot >= p.S) {                     // corrupt state: never write through it
        if (tid == 0) set_status(p.status, SSA_ST_BAD_ID);
        slot = -1;
      }
      const Block blk(p, layer, pg, slot, h);
      __syncthreads();
      const int R = s_run;
      float sum[4] = {old_sum.x, old_sum.y, old_sum.z, old_sum.w};
      store_run<I8, P, 4>(p, blk, true, d, kin, vin, k0, v0, HD, R, [&](int r) { return s_row[r]; },
                          cnt0, sum, nullptr);
      *reinterpret_cast<float4*>(p.slab_sum + so) = make_float4(sum[0], sum[1], sum[2], sum[3]);
      const int cnt = cnt0 + R;
      float mean[4], a = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mean[e] = sum[e] / (float)cnt;
        a = fmaxf(a, fabsf(mean[e]));
      }
      a = warp_max(a);
      if (lane == 0) s_head[h] = a;
      __syncthreads();
      float amax = 0.0f;
      for (int w = 0; w < Hkv; ++w) amax = fmaxf(amax, s_head[w]);
      const float s = amax / 127.0f;
      char4 code;
      code.x = (signed char)slab_code(mean[0], amax, s);
      code.y = (signed char)slab_code(mean[1], amax, s);
      code.z = (signed char)slab_code(mean[2], amax, s);
      code.w = (signed char)slab_code(mean[3], amax, s);
      *reinterpret_cast<char4*>(p.slab + so) = code;
      if (tid == 0) {
        p.slab_cnt[lp] = cnt;
        p.slab_scale[lp] = s;
      }
      if (!MANY) return;
      __syncthreads();                       // s_run, s_row, s_head: the next run's
    }
    if (!MANY) return;
  }
}

// Threads of a CTA and 16-byte units of K (and of V) a thread holds: 4 tokens
// at a time, at most 8 units.
constexpr int store_threads(int P) { return P == 128 ? 256 : 128; }
constexpr int store_units(int P) { return P == 32 ? 4 : 8; }
// dynamic shared memory: K and V rows as they came; V's codes on their way out
// take the place of K's
inline size_t store_smem_bytes(int P) { return (size_t)P * kHD * 4; }

// The whole pages of a call: a cluster per P tokens, in which at most one
// starts, a CTA per head.  MIR: the cache has a host mirror.
template <bool I8, int P, bool MIR>
__global__ void __launch_bounds__(store_threads(P), P == 128 ? 3 : 6)
store_page_head_kernel(const __grid_constant__ StorePHParams p) {
  constexpr int NT = store_threads(P), NU = store_units(P), NW = NT / 32;
  constexpr int G = NT / kRowUnits;      // groups of 4 tokens side by side
  static_assert(NT * NU == P * kRowUnits, "every unit of a page has its thread");
  extern __shared__ __align__(16) uint8_t dsm[];
  uint4* kx = reinterpret_cast<uint4*>(dsm);                       // [r][16 units]
  uint4* vx = kx + P * kRowUnits;
  uint32_t* vt = reinterpret_cast<uint32_t*>(dsm);                 // [d][P / 4 words], swizzled
  __shared__ int s_first;                // the page's first token
  __shared__ uint32_t s_bits[2][NW];
  __shared__ float s_max[2][4], s_slab[2];
  __shared__ float s_heads[8];           // the heads' maxima, pushed by each of them
  __shared__ uint64_t s_bar;             // counts their bytes
  constexpr float kQmax = I8 ? 127.0f : 448.0f;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    mbar_init(&s_bar, 1);
    fence_barrier_init();
    s_first = -1;
  }
  pdl_trigger();
  // every head's barrier is there before the first push (waited for below)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_wait();
  const int c = tid % kRowUnits, g = tid / kRowUnits;              // dims 8c.., tokens 4g..
  const int h = blockIdx.x % p.Hkv, Hkv = p.Hkv, HD = Hkv * kHD;   // h: the cluster's rank
  const int li = blockIdx.y, layer = p.layer0 + li;
  __syncthreads();
  // the page that starts in the cluster's tokens (each head finds the same)
  const int t = (int)(blockIdx.x / p.Hkv) * P + tid;
  if (tid < P && t < p.T) {
    const int64_t x = p.pos[t], prev = t > 0 ? p.pos[t - 1] : -1;
    if (t > 0 && prev >= x && h == 0) set_status(p.status, SSA_ST_BAD_POS);
    const bool inside = prev >= 0 && prev / P == x / P;
    if (x >= 0 && x / P < p.Lp && !inside && whole_page<P>(p, t, x)) {
      // one where positions increase; the last one otherwise
      atomicMax(&s_first, t);
    }
  }
  __syncthreads();
  const int t0 = s_first;
  if (t0 < 0) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return;
  }

  const int pg = (int)(p.pos[t0] / P);
  const size_t lp = (size_t)layer * p.Lp + pg;
  const size_t so = (lp * Hkv + h) * kHD;
  const size_t row0 = ((size_t)li * p.T + t0) * HD + h * kHD;
  // its rows of this head into shared memory (asynchronous copies, so that no
  // register waits for them).  A thread copies the units that it works on.
  auto token = [&](int i) { return (i >> 2) * (4 * G) + 4 * g + (i & 3); };
  {
    const uint4* kg = reinterpret_cast<const uint4*>(p.k + row0) + c;
    const uint4* vg = reinterpret_cast<const uint4*>(p.v + row0) + c;
    const int rs = HD / 8;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      copy_async16(&kx[token(i) * kRowUnits + c], kg + token(i) * rs);
      copy_async16(&vx[token(i) * kRowUnits + c], vg + token(i) * rs);
    }
  }
  const int cnt0 = p.slab_cnt[lp], cnt = cnt0 + P;
  const float fcnt = (float)cnt;
  int slot = p.slot_of[lp];
  if (slot >= p.S) {                       // corrupt state: never write through it
    if (tid == 0 && h == 0) set_status(p.status, SSA_ST_BAD_ID);
    slot = -1;
  }
  const Block blk(p, layer, pg, slot, h);
  float2 sum = make_float2(0.0f, 0.0f), mean = sum;      // of dims 2 tid, 2 tid + 1
  if (tid < kHD / 2) sum = reinterpret_cast<const float2*>(p.slab_sum + so)[tid];
  const float old_k = cnt0 > 0 ? blk.scale(p.k_scale_m, p.k_scale) : 0.0f;
  const float old_v = cnt0 > 0 ? blk.scale(p.v_scale_m, p.v_scale) : 0.0f;
  asm volatile("cp.async.wait_all;" ::: "memory");
  // the largest magnitudes
  {
    __nv_bfloat162 mk2 = __floats2bfloat162_rn(0.0f, 0.0f), mv2 = mk2;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      absmax(mk2, kx[token(i) * kRowUnits + c]);
      absmax(mv2, vx[token(i) * kRowUnits + c]);
    }
    const uint32_t mk = max_bits(mk2), mv = max_bits(mv2);
    if (lane == 0) {
      s_bits[0][warp] = mk;
      s_bits[1][warp] = mv;
    }
  }
  __syncthreads();                         // (every thread has read the old scales)
  // (scale, -1 / scale, or 0 where values are not finite or the Divider's range ends)
  auto scale_of = [&](const uint32_t* bits, float old) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = max(m, bits[w]);
    const float need = __uint_as_float(m << 16) / kQmax;
    const float s = cnt0 > 0 ? fmaxf(old, need) : need;
    return make_float2(s, m < 0x7F80u && divides(s) ? -(1.0f / s) : 0.0f);
  };
  const float2 sck = scale_of(s_bits[0], old_k), scv = scale_of(s_bits[1], old_v);
  if (tid < kHD / 2) {
    // fp32 running sums in token order, two dimensions per thread
    const uint32_t* col = reinterpret_cast<const uint32_t*>(kx) + tid;
    uint64_t acc = pack2(sum.x, sum.y);
#pragma unroll 16
    for (int r = 0; r < P; ++r) {
      const uint32_t w = col[r * (kHD / 2)];
      acc = add2(acc, pack2(lo_f(w), hi_f(w)));
    }
    unpack2(acc, sum.x, sum.y);
    reinterpret_cast<float2*>(p.slab_sum + so)[tid] = sum;
    mean = make_float2(sum.x / fcnt, sum.y / fcnt);
    const float a = warp_max(fmaxf(fabsf(mean.x), fabsf(mean.y)));
    if (lane == 0) s_slab[warp] = a;
  }
  // the page's heads exchange their maxima while V's codes are made
  auto exchange = [&]() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid == 0) mbar_arrive_expect_tx(&s_bar, 4 * Hkv);
    if (tid < Hkv) push_f32(&s_heads[h], &s_bar, tid, fmaxf(s_slab[0], s_slab[1]));
  };
  if (sck.y != 0.0f && scv.y != 0.0f) {
    if (tid == 0) {
      blk.set_scale(p.k_scale_m, p.k_scale, sck.x);
      blk.set_scale(p.v_scale_m, p.v_scale, scv.x);
    }
    constexpr int pe = P * kHD;            // codes of one head of one page
    constexpr uint32_t kNeg = 0x80008000u;
    // K: 8 codes of a row per unit
    const Divider dk(sck), dv(scv);
    uint8_t* kp = blk.slot(p.k_pool, pe);
    uint8_t* km = MIR ? blk.mirror(p.k_mir, pe) : nullptr;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint4 x = kx[token(i) * kRowUnits + c];
      const uint32_t w[4] = {x.x ^ kNeg, x.y ^ kNeg, x.z ^ kNeg, x.w ^ kNeg};
      uint64_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = dk(lo_f(w[k]), hi_f(w[k]));
      const uint2 out = make_uint2(codes4<I8>(q[0], q[1]), codes4<I8>(q[2], q[3]));
      const int off = token(i) * kHD + 8 * c;
      if (MIR) *reinterpret_cast<uint2*>(km + off) = out;
      if (kp) *reinterpret_cast<uint2*>(kp + off) = out;
    }
    __syncthreads();                       // K's rows make room for V's codes
    exchange();
    // V: words of 4 tokens per dimension; word r / 4 of row d goes to a place
    // that spreads the 16 dimension groups over the banks
    constexpr int kWords = P / 4, kVec = P / 16;         // words, 16-byte units of a row
#pragma unroll
    for (int i = 0; i < NU; i += 4) {
      const int at_w = (token(i) >> 2) ^ (c & (kWords - 1));
      uint4 vr[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) vr[m] = vx[token(i + m) * kRowUnits + c];
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        auto word = [&](const uint4& v) {
          return (k < 2 ? v.x : (k < 4 ? v.y : (k < 6 ? v.z : v.w))) ^ kNeg;
        };
        const uint32_t w[4] = {word(vr[0]), word(vr[1]), word(vr[2]), word(vr[3])};
        const uint32_t o0 = codes4<I8>(dv(lo_f(w[0]), lo_f(w[1])), dv(lo_f(w[2]), lo_f(w[3])));
        const uint32_t o1 = codes4<I8>(dv(hi_f(w[0]), hi_f(w[1])), dv(hi_f(w[2]), hi_f(w[3])));
        vt[(8 * c + k) * kWords + at_w] = o0;
        vt[(8 * c + k + 1) * kWords + at_w] = o1;
      }
    }
    __syncthreads();
    uint8_t* vp = blk.slot(p.v_pool, pe);
    uint8_t* vm = MIR ? blk.mirror(p.v_mir, pe) : nullptr;
#pragma unroll
    for (int u0 = 0; u0 < kHD * kVec; u0 += NT) {
      const int u = u0 + tid;
      const int d = u / kVec, x = u % kVec, sw = (d >> 3) & (kWords - 1);
      // the unit's words lie together, in another order
      const uint4 q = *reinterpret_cast<const uint4*>(vt + d * kWords + ((4 * x) ^ (sw & ~3)));
      const bool b0 = sw & 1, b1 = sw & 2;
      const uint2 e = b1 ? make_uint2(q.z, q.w) : make_uint2(q.x, q.y);
      const uint2 f = b1 ? make_uint2(q.x, q.y) : make_uint2(q.z, q.w);
      const uint4 out = b0 ? make_uint4(e.y, e.x, f.y, f.x) : make_uint4(e.x, e.y, f.x, f.y);
      if (MIR) reinterpret_cast<uint4*>(vm)[u] = out;
      if (vp) reinterpret_cast<uint4*>(vp)[u] = out;
    }
  } else {
    // values or scales out of the ordinary: a thread per dimension
    const int d = tid & (kHD - 1);
    const Row<1>* kin = reinterpret_cast<const Row<1>*>(p.k + row0 + d);
    const Row<1>* vin = reinterpret_cast<const Row<1>*>(p.v + row0 + d);
    float unused[1] = {0.0f};
    store_run<I8, P, 1>(p, blk, tid < kHD, d, kin, vin, *kin, *vin, HD, P, [](int r) { return r; },
                        cnt0, unused, s_max);
    __syncthreads();
    exchange();
  }

  // the page's slab row, now that every head's maximum is there
  if (!mbar_wait<true>(&s_bar, 0, nullptr)) {
    set_status(p.status, SSA_ST_TIMEOUT);
    return;
  }
  float amax = 0.0f;
  for (int r = 0; r < Hkv; ++r) amax = fmaxf(amax, s_heads[r]);
  const float s = amax / 127.0f;
  if (tid < kHD / 2)
    reinterpret_cast<char2*>(p.slab + so)[tid] = make_char2(
        (signed char)slab_code(mean.x, amax, s), (signed char)slab_code(mean.y, amax, s));
  if (tid == 0 && h == 0) {                // every head has read the count by now
    p.slab_cnt[lp] = cnt;
    p.slab_scale[lp] = s;
  }
}

// Calls below kWholeTokens go to the append kernel alone: mostly a batch's
// decode step, for which a second launch is 3 us; longer ones leave whole
// pages to the other kernel.  (Pages of 16 tokens are one step of a warp, and
// stay there.)
constexpr int kWholeTokens = 256;
// CTAs of the append kernel in such a call: single tokens want many, but a
// prefill's find nothing to do at 1 us a thousand.  (12 layers: 4,096 tokens of
// whole pages, then 256 single ones behind them and 1,000 single ones alone:
// 1,024 CTAs 36.6, 72.7 and 144 us, 2,048 37.3, 66.6 and 118 us, 8,192 43.2,
// 64.0 and 112 us.)
constexpr int kAppendCtas = 2048;

template <bool I8, int P, bool MIR>
cudaError_t launch_m(const StorePHParams& p, int n_layers, cudaStream_t s) {
  const size_t smem = store_smem_bytes(P);
  cudaError_t e = cudaFuncSetAttribute(store_page_head_kernel<I8, P, MIR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long nchunk = (p.T + (long long)P - 1) / P;
  if (nchunk * p.Hkv > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nchunk * p.Hkv), (unsigned)n_layers);
  cfg.blockDim = dim3(store_threads(P));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.Hkv;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, store_page_head_kernel<I8, P, MIR>, p);
  count_launch();
  return e;
}

template <bool I8, int P>
cudaError_t launch_t(StorePHParams p, int n_layers, cudaStream_t s) {
  const dim3 block((unsigned)(p.Hkv * 32));
  cudaError_t e;
  if (p.T < kWholeTokens) {
    e = launch_pdl(append_page_head_kernel<I8, P, false>, dim3((unsigned)p.T, (unsigned)n_layers),
                   block, 0, s, p);
    count_launch();
    return e;
  }
  // (pages of 16: a prefill's CTAs store every page; 32,768 tokens of 3 layers
  // and 2 heads 74.0 us with one times as many, 60.8 with four, 72.9 with 16)
  constexpr int kCtas = P == 16 ? 4 * kAppendCtas : kAppendCtas;
  const long long per = ((long long)p.T * n_layers + kCtas - 1) / kCtas;
  p.chunk = per < 4 ? 4 : (per > kMaxPiece ? kMaxPiece : (int)per);
  // odd, so that runs that start 16 or 32 tokens apart reach all CTAs
  const unsigned ctas = (unsigned)(((long long)p.T + p.chunk - 1) / p.chunk) | 1u;
  p.whole = P > 16;
  e = launch_pdl(append_page_head_kernel<I8, P, true>,
                 dim3(ctas, (unsigned)n_layers), block, 0, s, p);
  count_launch();
  if (e != cudaSuccess) return e;
  if constexpr (P > 16)
    e = p.k_mir ? launch_m<I8, P, true>(p, n_layers, s) : launch_m<I8, P, false>(p, n_layers, s);
  return e;
}

template <bool I8>
cudaError_t launch_p(const StorePHParams& p, int P, int n_layers, cudaStream_t s) {
  switch (P) {
    case 16: return launch_t<I8, 16>(p, n_layers, s);
    case 32: return launch_t<I8, 32>(p, n_layers, s);
    case 64: return launch_t<I8, 64>(p, n_layers, s);
    case 128: return launch_t<I8, 128>(p, n_layers, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_store_page_head(const Dims& d, const ssa_cache& c, int layer0, int n_layers,
                                   const void* k, const void* v, const int64_t* pos, int T,
                                   int32_t* status, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  if (d.D != kHD || d.P > kMaxP || d.Hkv > 8) return cudaErrorInvalidValue;
  StorePHParams p{};
  p.k_pool = static_cast<uint8_t*>(c.k_pool);
  p.v_pool = static_cast<uint8_t*>(c.v_pool);
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.k_mir = static_cast<uint8_t*>(c.k_mirror);
  p.v_mir = static_cast<uint8_t*>(c.v_mirror);
  p.k_scale_m = c.k_scale_mirror;
  p.v_scale_m = c.v_scale_mirror;
  p.slab = c.slab;
  p.slab_scale = c.slab_scale;
  p.slab_sum = c.slab_sum;
  p.slab_cnt = c.slab_cnt;
  p.slot_of = c.slot_of;
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.pos = pos;
  p.status = status;
  p.T = T;
  p.layer0 = layer0; p.Lp = d.Lp; p.S = d.S; p.Hkv = d.Hkv;
  return d.kind == SSA_KV_INT8_PAGE_HEAD ? launch_p<true>(p, d.P, n_layers, s)
                                         : launch_p<false>(p, d.P, n_layers, s);
}

}  // namespace ssa
