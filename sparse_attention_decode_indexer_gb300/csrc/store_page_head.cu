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
// Two kernels, by the length of the call as in store.cu: a call of 4,096
// tokens or more is a prefill, whose runs (consecutive tokens of one page) are
// mostly whole pages; a shorter one is mostly an append, whose runs are one or
// a few tokens.
//
// Prefill: one CTA per (run, layer, KV head), which keeps the run's rows of
// its head in shared memory while the scale becomes known, so that each input
// is read once.  A thread holds 8 dimensions of 4 consecutive tokens, so V leaves
// as whole words of its d-major block through a swizzled tile.  The heads of a
// page meet only in the slab's scale (max over all heads): they form a cluster
// and read each other's maximum through distributed shared memory.
// Its arithmetic is the division x / s'.  s' is the block's, so the reciprocal
// is computed once and each quotient is corrected from its exact residual
// twice (Markstein 1990: a faithful quotient plus its fused residual times the
// correctly rounded reciprocal is the correctly rounded quotient), two
// elements per f32x2 instruction: 5 instead of about 20 per pair.
//
// Append: one CTA per (run, layer) with a warp per head, so that a head's
// maxima are a warp's and only the slab's scale meets in shared memory; a run
// costs three dependent reads (position, state, scale), and 64 requests of 12
// layers are all resident at once.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace ssa {
namespace {

constexpr int kHD = 128;                 // head_dim
constexpr int kMaxP = 128;
constexpr int kRowUnits = kHD * 2 / 16;  // 16-byte units of a bf16 token row
constexpr int kTokBatch = 8;             // append: tokens in flight per thread

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
// the same), to both.
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
// [2][4] is their scratch).  kin, vin: the thread's elements of the first
// token, rows HD apart; k0, v0: their values.  sum: the slab's sums, updated.
template <bool I8, int P, int E>
__device__ __forceinline__ void store_run(const StorePHParams& p, const Block& blk, bool active,
                                          int d, const Row<E>* kin, const Row<E>* vin, Row<E> k0,
                                          Row<E> v0, int HD, int R, const int* s_row, int cnt0,
                                          float (&sum)[E], float (*s_max)[4]) {
  constexpr float kQmax = I8 ? 127.0f : 448.0f;
  constexpr int pe = P * kHD;              // codes of one head of one page
  constexpr int NT = kHD / E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rs = HD / E;
  const float old_k = cnt0 > 0 ? blk.scale(p.k_scale_m, p.k_scale) : 0.0f;
  const float old_v = cnt0 > 0 ? blk.scale(p.v_scale_m, p.v_scale) : 0.0f;
  // finite maxima of the run
  float ak = 0.0f, av = 0.0f;
  auto take = [](float& m, const Row<E>& x) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float a = fabsf(x.at(e));
      if (a < INFINITY) m = fmaxf(m, a);
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
  if (E == 1) {
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
  for (int r = 0; r < R; ++r) {
    const Row<E> xk = r == 0 ? k0 : kin[(size_t)r * rs], xv = r == 0 ? v0 : vin[(size_t)r * rs];
    const int j = s_row[r];
    uint32_t ck = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float fk = xk.at(e), fv = xv.at(e);
      ck |= (uint32_t)(sk > 0.0f ? quant<I8>(fk / sk) : 0) << (8 * e);
      const uint8_t c = sv > 0.0f ? quant<I8>(fv / sv) : 0;
      if (vm) vm[(d + e) * P + j] = c;
      if (vp) vp[(d + e) * P + j] = c;
      sum[e] = sum[e] + fk;                // the slab: fp32, token order
    }
    if (E == 1) {
      if (km) km[j * kHD + d] = (uint8_t)ck;
      if (kp) kp[j * kHD + d] = (uint8_t)ck;
    } else {
      if (km) *reinterpret_cast<uint32_t*>(km + j * kHD + d) = ck;
      if (kp) *reinterpret_cast<uint32_t*>(kp + j * kHD + d) = ck;
    }
  }
}

__device__ __forceinline__ int slab_code(float mean, float amax, float s) {
  return amax > 0.0f ? (int)fminf(fmaxf(rintf(mean / s), -127.0f), 127.0f) : 0;
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
// A warp per KV head, four dimensions a lane; grid (tokens, layers): the CTA
// of a run's first token stores the run, the others return.
template <bool I8, int P>
__global__ void __launch_bounds__(256) append_page_head_kernel(StorePHParams p) {
  __shared__ int s_row[P];
  __shared__ int s_run;
  __shared__ float s_head[8];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, h = tid >> 5;
  const int Hkv = p.Hkv, HD = Hkv * kHD, d = 4 * lane;
  const int t0 = blockIdx.x, li = blockIdx.y, layer = p.layer0 + li;
  // this token's position and the ones around it, in one round trip with the
  // run's first token
  const int64_t pos0 = p.pos[t0];
  const int64_t prev = t0 > 0 ? p.pos[t0 - 1] : -1;
  const size_t in0 = (((size_t)li * p.T + t0) * HD + h * kHD + d) / 4;
  const Row<4>* kin = reinterpret_cast<const Row<4>*>(p.k) + in0;
  const Row<4>* vin = reinterpret_cast<const Row<4>*>(p.v) + in0;
  const Row<4> k0 = *kin, v0 = *vin;
  if (pos0 < 0 || pos0 / P >= p.Lp) {
    if (tid == 0) set_status(p.status, SSA_ST_BAD_ID);
    return;
  }
  const int pg = (int)(pos0 / P);
  if (t0 > 0) {
    if (tid == 0 && prev >= pos0) set_status(p.status, SSA_ST_BAD_POS);
    if (prev >= 0 && prev / P == pg) return;                 // inside a run
  }
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
  if (slot >= p.S) {                       // corrupt state: never write through it
    if (tid == 0) set_status(p.status, SSA_ST_BAD_ID);
    slot = -1;
  }
  const Block blk(p, layer, pg, slot, h);
  __syncthreads();
  const int R = s_run;
  float sum[4] = {old_sum.x, old_sum.y, old_sum.z, old_sum.w};
  store_run<I8, P, 4>(p, blk, true, d, kin, vin, k0, v0, HD, R, s_row, cnt0, sum, nullptr);
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
}

// ---------------------------------------------------------------------------
// prefill
// ---------------------------------------------------------------------------
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

// Divides by one block's scale.  With ny = -RN(1 / s) and nx = -x, each step
// corrects the quotient by its residual q s - x (exact in one fma); the signs
// are such that a zero keeps its own.  For s in [2^-90, 2^100] and x finite:
// nothing on the way over- or underflows then unless the quotient is below
// 2^-12 (every code 0).
struct Divider {
  uint64_t s2, ny2;
  __device__ __forceinline__ Divider(float2 s) : s2(pack2(s.x, s.x)), ny2(pack2(s.y, s.y)) {}
  // two negated elements -> the two quotients
  __device__ __forceinline__ uint64_t operator()(float nx0, float nx1) const {
    const uint64_t nx = pack2(nx0, nx1);
    uint64_t q = mul2(nx, ny2);
    q = fma2(fma2(q, s2, nx), ny2, q);
    q = fma2(fma2(q, s2, nx), ny2, q);
    return q;
  }
};

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

// Threads of a CTA and 16-byte units of K (and of V) a thread holds: 4 tokens
// at a time, at most 8 units.
constexpr int prefill_threads(int P) { return P == 128 ? 256 : 128; }
constexpr int prefill_units(int P) { return P <= 32 ? 4 : 8; }
// dynamic shared memory: K and V rows as they came; V's codes on their way out
// take the place of K's
inline size_t prefill_smem(int P) { return (size_t)P * kHD * 4; }

// MIR: the cache has a host mirror.
template <bool I8, int P, bool MIR>
__global__ void __launch_bounds__(prefill_threads(P), P == 128 ? 3 : 6)
prefill_page_head_kernel(StorePHParams p) {
  constexpr int NT = prefill_threads(P), NU = prefill_units(P), NW = NT / 32;
  constexpr int G = NT / kRowUnits;      // groups of 4 tokens side by side
  extern __shared__ __align__(16) uint8_t dsm[];
  uint4* kx = reinterpret_cast<uint4*>(dsm);                       // [r][16 units]
  uint4* vx = kx + P * kRowUnits;
  uint32_t* vt = reinterpret_cast<uint32_t*>(dsm);                 // [d][P / 4 words], swizzled
  __shared__ int64_t s_pos[2 * P];       // positions of the chunk and of the run it may end in
  __shared__ uint32_t s_start[(P + 31) / 32];
  __shared__ int s_row[P];               // the run's tokens' rows j, ascending
  __shared__ int s_run;
  __shared__ uint32_t s_bits[2][NW];
  __shared__ float s_max[2][4], s_slab[4];
  __shared__ float2 s_scale[2];          // K's, V's: (scale, -1 / scale, 0 outside the exact range)
  // the heads' maxima of two runs, and their barriers: head r of the cluster
  // writes entry r of every head.  (Two of each: a head can be one run ahead.)
  __shared__ float s_heads[2][8];
  __shared__ uint64_t s_bar[2];
  constexpr float kQmax = I8 ? 127.0f : 448.0f;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    mbar_init(&s_bar[0], 1);
    mbar_init(&s_bar[1], 1);
    fence_barrier_init();
  }
  pdl_trigger();
  // every head's barriers are there before the first push (waited for below)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  const int c = tid % kRowUnits, g = tid / kRowUnits;              // dims 8c.., tokens 4g..
  const int h = blockIdx.x % p.Hkv, Hkv = p.Hkv, HD = Hkv * kHD;   // h: the cluster's rank
  const int li = blockIdx.y, layer = p.layer0 + li;

  // the chunk's positions, and the runs that start in it (each head finds the same)
  const int c0 = (int)(blockIdx.x / p.Hkv) * P, nc = min(P, p.T - c0);
  const int64_t before = c0 > 0 ? p.pos[c0 - 1] : -1;
#pragma unroll
  for (int i = tid; i < 2 * P; i += NT)
    if (c0 + i < p.T) s_pos[i] = p.pos[c0 + i];
  __syncthreads();
  if (tid < (P + 31) / 32 * 32) {
    bool start = false;
    if (tid < nc) {
      const int64_t x = s_pos[tid], prev = tid > 0 ? s_pos[tid - 1] : before;
      start = x >= 0 && x / P < p.Lp;
      if (!start && h == 0) set_status(p.status, SSA_ST_BAD_ID);
      if (start && c0 + tid > 0) {
        if (prev >= x && h == 0) set_status(p.status, SSA_ST_BAD_POS);
        if (prev >= 0 && prev / P == x / P) start = false;         // inside a run
      }
    }
    const uint32_t m = __ballot_sync(0xffffffffu, start);
    if (lane == 0) s_start[warp] = m;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

  int run = 0;
#pragma unroll 1
  for (int at = 0; at < P; ++at) {
    const uint32_t ahead = s_start[at >> 5] >> (at & 31);
    if (!ahead) { at |= 31; continue; }
    at += __ffs(ahead) - 1;
    const int t0 = c0 + at;
    const int64_t page = s_pos[at] / P;
    const int pg = (int)page;
    const size_t lp = (size_t)layer * p.Lp + pg;
    // the page's state, loaded now: its latency overlaps the run's scan
    const size_t so = (lp * Hkv + h) * kHD;
    const int cnt0 = p.slab_cnt[lp];
    int slot = p.slot_of[lp];
    // run length: consecutive tokens of the same page (at most P)
    if (tid == 0) s_run = P;
    __syncthreads();
    bool in_place = true;                  // token r in row r
    if (tid < P) {
      bool ends = t0 + tid >= p.T;
      if (!ends) {
        const int64_t x = s_pos[at + tid];
        ends = x < 0 || x / P != page;
        if (!ends) {
          s_row[tid] = (int)(x % P);
          in_place = x % P == tid;
          if (tid > 0 && x <= s_pos[at + tid - 1] && h == 0) set_status(p.status, SSA_ST_BAD_POS);
        }
      }
      if (ends) {
        atomicMin(&s_run, tid);
        in_place = false;
      }
    }
    const bool full = __syncthreads_and(in_place);     // the run is the whole page
    const int R = s_run;
    const size_t row0 = ((size_t)li * p.T + t0) * HD + h * kHD;
    if (slot >= p.S) {                     // corrupt state: never write through it
      if (tid == 0 && h == 0) set_status(p.status, SSA_ST_BAD_ID);
      slot = -1;
    }
    const Block blk(p, layer, pg, slot, h);
    const int cnt = cnt0 + R;
    const float fcnt = (float)cnt;

    // a whole page: its rows of this head into shared memory (asynchronous
    // copies, so that no register waits for them); the largest magnitudes.  A
    // thread copies the units that it works on itself.
    auto token = [&](int i) { return (i >> 2) * (4 * G) + 4 * g + (i & 3); };
    constexpr bool kIdle = NT * NU > P * kRowUnits;    // threads without tokens (P = 16)
    const bool mine = !kIdle || token(0) < P;
    float2 mean = make_float2(0.0f, 0.0f);             // of dims 2 tid, 2 tid + 1
    if (full) {
      const uint4* kg = reinterpret_cast<const uint4*>(p.k + row0) + c;
      const uint4* vg = reinterpret_cast<const uint4*>(p.v + row0) + c;
      const int rs = HD / 8;
      if (mine) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          copy_async16(&kx[token(i) * kRowUnits + c], kg + token(i) * rs);
          copy_async16(&vx[token(i) * kRowUnits + c], vg + token(i) * rs);
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      // warps 0 and 1 have the slab's sums to make, warp 2 (3) K's (V's) scale
      float2 sum = make_float2(0.0f, 0.0f);
      float old = 0.0f;
      if (tid < kHD / 2) sum = reinterpret_cast<const float2*>(p.slab_sum + so)[tid];
      if (tid == 64 && cnt0 > 0) old = blk.scale(p.k_scale_m, p.k_scale);
      if (tid == 96 && cnt0 > 0) old = blk.scale(p.v_scale_m, p.v_scale);
      __nv_bfloat162 mk2 = __floats2bfloat162_rn(0.0f, 0.0f), mv2 = mk2;
      if (mine) {
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          absmax(mk2, kx[token(i) * kRowUnits + c]);
          absmax(mv2, vx[token(i) * kRowUnits + c]);
        }
      }
      const uint32_t mk = max_bits(mk2), mv = max_bits(mv2);
      if (lane == 0) {
        s_bits[0][warp] = mk;
        s_bits[1][warp] = mv;
      }
      __syncthreads();
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
      } else if (tid == 64 || tid == 96) {
        uint32_t m = 0;
        for (int w = 0; w < NW; ++w) m = max(m, s_bits[warp - 2][w]);
        const float need = __uint_as_float(m << 16) / kQmax;
        const float s = cnt0 > 0 ? fmaxf(old, need) : need;
        // finite values, and a scale that keeps the quotients exact (see Divider)
        const bool exact = m < 0x7F80u && s >= 0x1p-90f && s <= 0x1p100f;
        s_scale[warp - 2] = make_float2(s, exact ? -(1.0f / s) : 0.0f);
      }
      __syncthreads();
    }
    const float2 sck = s_scale[0], scv = s_scale[1];
    const bool fast = full && sck.y != 0.0f && scv.y != 0.0f;
    if (fast) {
      if (tid == 0) {
        blk.set_scale(p.k_scale_m, p.k_scale, sck.x);
        blk.set_scale(p.v_scale_m, p.v_scale, scv.x);
      }
    } else {
      // part of a page, or values or scales out of the ordinary
      const int d = tid & (kHD - 1);
      const bool active = tid < kHD;
      const Row<1>* kin = reinterpret_cast<const Row<1>*>(p.k + row0 + d);
      const Row<1>* vin = reinterpret_cast<const Row<1>*>(p.v + row0 + d);
      // (a whole page has its sums already)
      float sum[1] = {active && !full ? p.slab_sum[so + d] : 0.0f};
      store_run<I8, P, 1>(p, blk, active, d, kin, vin, *kin, *vin, HD, R, s_row, cnt0, sum, s_max);
      if (!full && active) {
        p.slab_sum[so + d] = sum[0];
        mean.x = sum[0] / fcnt;
        const float a = warp_max(fabsf(mean.x));
        if (lane == 0) s_slab[warp] = a;
      }
      __syncthreads();
    }
    // the page's heads exchange their maxima while the codes are made
    const int par = run & 1;
    if (tid == 0) mbar_arrive_expect_tx(&s_bar[par], 4 * Hkv);
    if (tid < Hkv) {
      float a = fmaxf(s_slab[0], s_slab[1]);
      if (!full) a = fmaxf(a, fmaxf(s_slab[2], s_slab[3]));
      push_f32(&s_heads[par][h], &s_bar[par], tid, a);
    }

    if (fast) {
      constexpr int pe = P * kHD;          // codes of one head of one page
      constexpr uint32_t kNeg = 0x80008000u;
      // K: 8 codes of a row per unit
      const Divider dk(sck), dv(scv);
      uint8_t* kp = blk.slot(p.k_pool, pe);
      uint8_t* km = MIR ? blk.mirror(p.k_mir, pe) : nullptr;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (!mine) break;
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
      __syncthreads();                     // K's rows make room for V's codes
      // V: words of 4 tokens per dimension; word r / 4 of row d goes to a place
      // that spreads the 16 dimension groups over the banks
      constexpr int kWords = P / 4, kVec = P / 16;       // words, 16-byte units of a row
#pragma unroll
      for (int i = 0; i < NU; i += 4) {
        if (!mine) break;
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
    }

    // the page's slab row, now that every head's maximum is there
    if (!mbar_wait(&s_bar[par], (run >> 1) & 1, nullptr)) {
      set_status(p.status, SSA_ST_TIMEOUT);
      return;
    }
    float amax = 0.0f;
    for (int r = 0; r < Hkv; ++r) amax = fmaxf(amax, s_heads[par][r]);
    const float s = amax / 127.0f;
    if (full) {
      if (tid < kHD / 2)
        reinterpret_cast<char2*>(p.slab + so)[tid] = make_char2(
            (signed char)slab_code(mean.x, amax, s), (signed char)slab_code(mean.y, amax, s));
    } else if (tid < kHD) {
      p.slab[so + tid] = (int8_t)slab_code(mean.x, amax, s);
    }
    if (tid == 0 && h == 0) {              // every head has read the count by now
      p.slab_cnt[lp] = cnt;
      p.slab_scale[lp] = s;
    }
    ++run;
    __syncthreads();                       // the tiles and s_row: the next run's
  }
}

// Calls of at least this many tokens take the prefill kernel.
constexpr int kPrefillTokens = 4096;

template <bool I8, int P, bool MIR>
cudaError_t launch_prefill(const StorePHParams& p, int n_layers, cudaStream_t s) {
  const size_t smem = prefill_smem(P);
  cudaError_t e = cudaFuncSetAttribute(prefill_page_head_kernel<I8, P, MIR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long nchunk = (p.T + (long long)P - 1) / P;
  if (nchunk * p.Hkv > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nchunk * p.Hkv), (unsigned)n_layers);
  cfg.blockDim = dim3(prefill_threads(P));
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
  e = cudaLaunchKernelEx(&cfg, prefill_page_head_kernel<I8, P, MIR>, p);
  count_launch();
  return e;
}

template <bool I8, int P>
cudaError_t launch_t(const StorePHParams& p, int n_layers, cudaStream_t s) {
  if (p.T >= kPrefillTokens)
    return p.k_mir ? launch_prefill<I8, P, true>(p, n_layers, s)
                   : launch_prefill<I8, P, false>(p, n_layers, s);
  cudaError_t e = launch_pdl(append_page_head_kernel<I8, P>,
                             dim3((unsigned)p.T, (unsigned)n_layers),
                             dim3((unsigned)(p.Hkv * 32)), 0, s, p);
  count_launch();
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
