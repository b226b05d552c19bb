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
// host link; each input is read once, into shared memory, because the scale
// has to be known before the first code.
//
// Split: one CTA per (run of consecutive tokens of one page, layer, KV head),
// so that a decode append (one token per request) spreads over requests x
// layers x heads, and a page's tokens of one head fit in shared memory as they
// came.  The heads of a page meet only in the slab's scale (max over all
// heads): they form a cluster of Hkv CTAs and read each other's maximum
// through distributed shared memory.  Runs are found per chunk of tokens as in
// store.cu: chunks of one token for short calls, of one page for long ones.
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace ssa {
namespace {

constexpr int kHD = 128;                 // head_dim
constexpr int kThreads = 128;            // one per head dimension
constexpr int kMaxP = 128;
constexpr int kUnitsPerRow = kHD * 2 / 16;     // 16-byte units of a bf16 token row
constexpr int kLoads = 8;                // input loads in flight per thread and tensor

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
  int T, chunk, layer0, Lp, S, Hkv;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// a float of the same shared variable in CTA `rank` of the cluster
__device__ __forceinline__ float cluster_read(const float* p, int rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
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

// |x| of the finite ones of 8 bf16 values, maximum
__device__ __forceinline__ float finite_absmax(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (w[i] << 16) & 0x7FFF0000u, hi = w[i] & 0x7FFF0000u;
    if (lo < 0x7F800000u) m = fmaxf(m, __uint_as_float(lo));
    if (hi < 0x7F800000u) m = fmaxf(m, __uint_as_float(hi));
  }
  return m;
}

// dynamic shared memory: the run's K and V rows of one head as they came
// (2 * P * 256 B), then the codes of one tensor on their way out (P * 128 B)
inline size_t smem_bytes(int P) { return (size_t)P * (2 * kHD * 2 + kHD); }

template <bool I8, int P>
__global__ void __launch_bounds__(kThreads) store_page_head_kernel(StorePHParams p) {
  extern __shared__ __align__(16) uint8_t dsm[];
  __nv_bfloat16* kx = reinterpret_cast<__nv_bfloat16*>(dsm);       // [R][D]
  __nv_bfloat16* vx = kx + P * kHD;
  uint8_t* codes = reinterpret_cast<uint8_t*>(vx + P * kHD);       // K: [j][D]; V: [D][j]
  __shared__ int s_start[P];
  __shared__ int s_row[P];               // the run's tokens' rows j, ascending
  __shared__ int s_at[P];                // the token of row j in this run, or -1
  __shared__ int s_nstart, s_run;
  __shared__ float s_red[2][kThreads / 32];
  __shared__ float s_head_amax;          // read by the other heads of the cluster
  constexpr float kQmax = I8 ? 127.0f : 448.0f;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.Hkv, Hkv = p.Hkv;                   // the cluster's rank
  const int li = blockIdx.y, layer = p.layer0 + li;

  // the runs that start in this cluster's chunk (each head finds the same)
  const int c0 = (int)(blockIdx.x / p.Hkv) * p.chunk, nc = min(p.chunk, p.T - c0);
  for (int i = tid; i < nc; i += kThreads) {
    const int t = c0 + i;
    const int64_t x = p.pos[t];
    bool start = true;
    if (x < 0 || x / P >= p.Lp) {
      if (h == 0) set_status(p.status, SSA_ST_BAD_ID);
      start = false;
    } else if (t > 0) {
      const int64_t prev = p.pos[t - 1];
      if (prev >= x && h == 0) set_status(p.status, SSA_ST_BAD_POS);
      if (prev >= 0 && prev / P == x / P) start = false;           // inside a run
    }
    s_start[i] = start ? t : -1;
  }
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int i = 0; i < nc; ++i)
      if (s_start[i] >= 0) s_start[n++] = s_start[i];
    s_nstart = n;
  }
  __syncthreads();
  const int nstart = s_nstart;

  for (int ri = 0; ri < nstart; ++ri) {
    const int t0 = s_start[ri];
    const int pg = (int)(p.pos[t0] / P);
    const size_t lp = (size_t)layer * p.Lp + pg;
    // the page's state, loaded now: its latency overlaps the run's scan
    const size_t so = (lp * Hkv + h) * kHD + tid;
    float sum = p.slab_sum[so];
    const int cnt0 = p.slab_cnt[lp];
    int slot = p.slot_of[lp];
    if (slot >= p.S) {                     // corrupt state: never write through it
      if (tid == 0 && h == 0) set_status(p.status, SSA_ST_BAD_ID);
      slot = -1;
    }
    // run length: consecutive tokens of the same page (at most P)
    if (tid == 0) s_run = P;
    if (tid < P) s_at[tid] = -1;
    __syncthreads();
    if (tid < P) {
      const int t = t0 + tid;
      bool ends = t >= p.T;
      if (!ends) {
        const int64_t x = p.pos[t];
        ends = x < 0 || x / P != pg;
        if (!ends) s_row[tid] = (int)(x % P);
        if (!ends && tid > 0 && x <= p.pos[t - 1] && h == 0) set_status(p.status, SSA_ST_BAD_POS);
      }
      if (ends) atomicMin(&s_run, tid);
    }
    __syncthreads();
    const int R = s_run;
    if (tid < R) s_at[s_row[tid]] = tid;

    // the run's rows of this head, into shared memory; their finite maxima
    float ak = 0.0f, av = 0.0f;
    {
      const size_t row0 = ((size_t)li * p.T + t0) * Hkv + h;       // token r: row0 + r * Hkv
      const uint4* kg = reinterpret_cast<const uint4*>(p.k);
      const uint4* vg = reinterpret_cast<const uint4*>(p.v);
      const int n = R * kUnitsPerRow;
      for (int u0 = tid; u0 < n; u0 += kThreads * kLoads) {
        uint4 bk[kLoads], bv[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int u = u0 + i * kThreads;
          if (u < n) {
            const size_t g = (row0 + (size_t)(u / kUnitsPerRow) * Hkv) * kUnitsPerRow + u % kUnitsPerRow;
            bk[i] = kg[g];
            bv[i] = vg[g];
          }
        }
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int u = u0 + i * kThreads;
          if (u < n) {
            reinterpret_cast<uint4*>(kx)[u] = bk[i];
            reinterpret_cast<uint4*>(vx)[u] = bv[i];
            ak = fmaxf(ak, finite_absmax(bk[i]));
            av = fmaxf(av, finite_absmax(bv[i]));
          }
        }
      }
    }
    ak = warp_max(ak);
    av = warp_max(av);
    if (lane == 0) {
      s_red[0][warp] = ak;
      s_red[1][warp] = av;
    }
    __syncthreads();                       // rows, s_at and the maxima are in place
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      ak = fmaxf(ak, s_red[0][w]);
      av = fmaxf(av, s_red[1][w]);
    }

    // K, then V: scale, the codes already there, the new codes
    const size_t pe = (size_t)P * kHD;     // codes of one head of one page
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      float* sc_m = which ? p.v_scale_m : p.k_scale_m;
      float* sc_p = which ? p.v_scale : p.k_scale;
      uint8_t* mir = which ? p.v_mir : p.k_mir;
      uint8_t* pool = which ? p.v_pool : p.k_pool;
      const __nv_bfloat16* xs = which ? vx : kx;
      if (mir) mir += (lp * Hkv + h) * pe;
      pool = slot >= 0 ? pool + (((size_t)layer * p.S + slot) * Hkv + h) * pe : nullptr;
      sc_m = sc_m ? sc_m + lp * Hkv + h : nullptr;
      sc_p = slot >= 0 ? sc_p + ((size_t)layer * p.S + slot) * Hkv + h : nullptr;
      if (!mir && !pool) continue;         // the page is held nowhere
      // the pool's copy where there is one (the mirror's bytes are the same)
      const float need = (which ? av : ak) / kQmax;
      const float old = cnt0 > 0 ? (sc_p ? *sc_p : *sc_m) : 0.0f;
      const float s = cnt0 > 0 ? fmaxf(old, need) : need;
      const bool grow = cnt0 > 0 && s > old;
      const float ratio = grow ? old / s : 1.0f;
      __syncthreads();                     // every thread has read the old scale
      if (tid == 0) {
        if (sc_m) *sc_m = s;
        if (sc_p) *sc_p = s;
      }
      const uint8_t* from = pool ? pool : mir;
      if (grow) {                          // the whole block at its new scale
        for (int u = tid; u < (int)pe / 16; u += kThreads) {
          uint4 w = reinterpret_cast<const uint4*>(from)[u];
          uint8_t* b = reinterpret_cast<uint8_t*>(&w);
#pragma unroll
          for (int i = 0; i < 16; ++i) b[i] = quant<I8>(value<I8>(b[i]) * ratio);
          reinterpret_cast<uint4*>(codes)[u] = w;
        }
        __syncthreads();
      }
      // new codes: K rows [j][D]; V transposed to [D][j]
      for (int r = 0; r < R; ++r) {
        const float x = __bfloat162float(xs[r * kHD + tid]);
        const uint8_t c = s > 0.0f ? quant<I8>(x / s) : 0;
        codes[which ? tid * P + s_row[r] : s_row[r] * kHD + tid] = c;
      }
      __syncthreads();
      // out: 16-byte units whose codes are all known, single codes otherwise
      for (int u = tid; u < (int)pe / 16; u += kThreads) {
        const uint4 w = reinterpret_cast<const uint4*>(codes)[u];
        if (!which) {
          if (grow || s_at[u / (kHD / 16)] >= 0) {
            if (mir) reinterpret_cast<uint4*>(mir)[u] = w;
            if (pool) reinterpret_cast<uint4*>(pool)[u] = w;
          }
          continue;
        }
        const int j0 = u * 16 % P;
        uint32_t known = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) known |= (grow || s_at[j0 + i] >= 0 ? 1u : 0u) << i;
        if (known == 0xFFFFu) {
          if (mir) reinterpret_cast<uint4*>(mir)[u] = w;
          if (pool) reinterpret_cast<uint4*>(pool)[u] = w;
        } else {
          for (; known; known &= known - 1) {
            const int i = __ffs(known) - 1;
            const uint8_t c = codes[u * 16 + i];
            if (mir) mir[u * 16 + i] = c;
            if (pool) pool[u * 16 + i] = c;
          }
        }
      }
      __syncthreads();                     // codes are rewritten for V, and by the next run
    }

    // the slab: fp32 running sum in token order, the page's row again
    for (int r = 0; r < R; ++r) sum = sum + __bfloat162float(kx[r * kHD + tid]);
    p.slab_sum[so] = sum;
    const int cnt = cnt0 + R;
    const float mean = sum / (float)cnt;
    float a = warp_max(fabsf(mean));
    if (lane == 0) s_red[0][warp] = a;
    __syncthreads();
    if (tid == 0) {
      a = 0.0f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) a = fmaxf(a, s_red[0][w]);
      s_head_amax = a;
    }
    cluster_sync();
    float amax = 0.0f;
    for (int r = 0; r < Hkv; ++r) amax = fmaxf(amax, cluster_read(&s_head_amax, r));
    cluster_sync();                        // read before it is rewritten, or the CTA ends
    const float s = amax / 127.0f;
    int c = 0;
    if (amax > 0.0f) c = (int)fminf(fmaxf(rintf(mean / s), -127.0f), 127.0f);
    p.slab[so] = (int8_t)c;
    if (tid == 0 && h == 0) {              // every head has read the count by now
      p.slab_cnt[lp] = cnt;
      p.slab_scale[lp] = s;
    }
    __syncthreads();                       // s_row, s_at, s_run, the rows: the next run's
  }
}

template <bool I8, int P>
cudaError_t launch_t(const StorePHParams& p, int n_layers, cudaStream_t s) {
  const size_t smem = smem_bytes(P);
  cudaError_t e = cudaFuncSetAttribute(store_page_head_kernel<I8, P>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const long long nchunk = (p.T + (long long)p.chunk - 1) / p.chunk;
  if (nchunk * p.Hkv > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(nchunk * p.Hkv), (unsigned)n_layers);
  cfg.blockDim = dim3(kThreads);
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
  e = cudaLaunchKernelEx(&cfg, store_page_head_kernel<I8, P>, p);
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
  p.chunk = T >= 4096 ? d.P : 1;
  p.layer0 = layer0; p.Lp = d.Lp; p.S = d.S; p.Hkv = d.Hkv;
  return d.kind == SSA_KV_INT8_PAGE_HEAD ? launch_p<true>(p, d.P, n_layers, s)
                                         : launch_p<false>(p, d.P, n_layers, s);
}

}  // namespace ssa
