// prompt.cu -- attention over whole prompts: packed sequences, grouped heads.
//
// For query token i of a sequence of Lq query tokens and Lk keys, and query
// head hq = h * G + g,
//   out = sum_j w_j v_j,  w = softmax_j(scale q . k_j),  j <= i + Lk - Lq
// (causal) or all j < Lk; zeros where no key is seen.
//
// What bounds it: the two products, 4 * 128 flop per pair of query row and
// key, on the tensor cores; Q K^T reads both operands from shared memory, which
// at 64 keys a product gives 48 of the 32 clocks it would take, and the
// exponentials come next (a quarter of the products' time).  The work:
//   * A row is a (token, head of the group) pair, so that the G heads that
//     share K and V share every byte of them that is loaded.  A CTA owns two
//     tiles of up to 128 rows (128 / G tokens each) and walks over the keys in
//     blocks of 128, which TMA brings through a ring of five stages.
//   * The packed token axis is cut into tiles wherever sequences begin or end;
//     each row knows the range [lo, hi) of packed keys that it sees (one
//     binary search in the sequence table).  The keys that a tile's rows see
//     lie next to one another, so a tile walks from the least lo to the
//     greatest hi; scores outside a row's range are set to -inf.
//   * S = Q K^T and O += P V are tcgen05 MMAs with accumulators in tensor
//     memory: O, 128 columns a tile, and S in two half blocks of 64 keys, so
//     that one is made while the softmax has the other; P, rounded to the type
//     of V, lies over its S.  A warp a tile issues them: with one half block the
//     products of a tile and its softmax took turns (24,576 tokens, 16/2 heads:
//     1.82 ms with blocks of 128, 1.63 with half blocks; one warp for both tiles
//     reached the next wait too late).
//   * A thread per row: the 64 scores of a half block in registers, maximum,
//     exponentials, P.  (Two threads per row, P handed over in two halves,
//     or the scores read twice from tensor memory measured slower.)
//   * Softmax in one pass against a lazy reference: the maximum that p is taken
//     against moves only when a score exceeds it by 8 octaves; then the row's O
//     is rescaled in tensor memory.  Sums and references are fp32; P in 16 bits
//     is off by half a step of its type, as the inputs are, and divided by the sum
//     of the rounded weights: a row's error is sum_j w_j d_j (v_j - out), d_j the
//     roundings, so that of a weight near one cancels.  (The logarithm is that of the
//     sum before rounding.  The second sum costs packed prompts 3 %, prompts of some
//     hundred tokens 3 to 6 %, 24,576 tokens 1 %.)  For fp16 the reference
//     lies 7 octaves below the maximum (p up to 2^15 of 65,504): weights keep their
//     bits down to 2^-21 of the greatest, where 2^-14 would cut the many small ones
//     of a long context.
//   * Masked scores give p = 0, and 0 times an infinite or NaN v would still
//     be NaN.  Four spare warps look through the V of those blocks that some
//     row does not see all of, and set what is not finite to zero; the epilogue
//     then adds it for the rows that do see it, which read these blocks again.
//   * Few rows and many keys: the key blocks of a tile are split over several
//     CTAs; their unnormalised outputs are joined by a second kernel.
// Measured: 24,576 tokens x 16/2 heads causal 1.70 to 1.83 ms (1,350 to 1,455
// TFLOP/s, by how far the power limit lets the clock); 24 prompts of 69 to 3,712
// tokens, 32/4 heads, 384 us (885: a third of a CTA's time is its start and its end);
// 8 tokens behind 65,528 24 us (2.8 TB/s), 17 tokens 6.3 us.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "tc5.cuh"
#include "tmap.cuh"

namespace ssa {
namespace {

constexpr int kD = 128;                   // head size
constexpr int kRows = 128;                // rows of a tile
constexpr int kBlk = 128;                 // keys of a block, as they are loaded
constexpr int kSub = 64;                  // and as they are multiplied
constexpr int kThreads = 480;             // 8 softmax warps; TMA, an MMA warp a tile, 4 that look over V
constexpr int kTma = 8, kMma = 9, kLook = 11, kLooks = 4;           // these warps
constexpr int kTable = 256;               // entries of the sequence tables held on chip
constexpr int kStages = 5;                // K and V blocks in flight
constexpr int kHalf = kRows * 128;        // bytes of 64 of the 128 dimensions
constexpr int kTile = 2 * kHalf;
constexpr float kLazy = 8.0f;             // octaves
template <typename T> constexpr float kBelow = std::is_same_v<T, __half> ? 7.0f : 0.0f;     // reference below the maximum

struct Shared {                           // behind the tiles
  uint64_t full[kStages], empty[kStages], clean[kStages];
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_full[2][2];   // [tile][buffer]
  uint64_t drain;
  uint32_t tmem;
  int abort;
  int dirty[2];                           // first and last block in which V was not finite
  int4 seen[8];                           // of each 32 rows: least lo, greatest hi, greatest lo, least hi
  int cu_q[kTable], cu_k[kTable];
};
constexpr size_t kSmem = (size_t)(2 + kStages) * kTile + sizeof(Shared);
static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");

struct Params {
  const int32_t *cu_q, *cu_k;
  int n_seqs, Tq, Tk, Hq, Hkv, G, tpt;    // tpt: tokens of a tile
  int tiles, n_ctas, n_split, causal;     // tiles of a CTA, CTAs of a head and part
  float scale_log2;
  int64_t v_tok, v_head, o_tok, o_head;   // strides in elements
  const void* v;
  void* out;
  float* lse;
  float *part_o, *part_ml;                // [CTA][head][split][2 * kRows][kD], [..][4]: reference, two sums
  int32_t* status;
};

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tm, uint64_t* bar, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
               " [%0], [%1, {%2, %3, %4}], [%5];"
               ::"r"(smem_u32(dst)), "l"(tm), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tm, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
               " [%0], [%1, {%2, %3, %4, %5}], [%6];"
               ::"r"(smem_u32(dst)), "l"(tm), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)) : "memory");
}

template <typename T> __device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (std::is_same_v<T, __half>) return pack_f16(lo, hi);
  else return pack_bf16(lo, hi);
}
// a and b and the two elements of a word.
template <typename T> __device__ __forceinline__ void add16(uint32_t w, float& a, float& b) {
  if constexpr (std::is_same_v<T, __half>)
    asm("{\n.reg .b16 x, y;\nmov.b32 {x, y}, %2;\nadd.f32.f16 %0, x, %0;\nadd.f32.f16 %1, y, %1;\n}"
        : "+f"(a), "+f"(b) : "r"(w));
  else
    asm("{\n.reg .b16 x, y;\nmov.b32 {x, y}, %2;\nadd.f32.bf16 %0, x, %0;\nadd.f32.bf16 %1, y, %1;\n}"
        : "+f"(a), "+f"(b) : "r"(w));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <typename T> __device__ __forceinline__ float to_f32(T x) {
  if constexpr (std::is_same_v<T, __half>) return __half2float(x);
  else return __bfloat162float(x);
}

template <typename T> __device__ __forceinline__ T from_f32(float x) {
  if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// The range of packed keys that query token `tok` sees.  False where no
// sequence holds it.
__device__ __forceinline__ bool row_keys(const Params& p, const int32_t* cu_q, const int32_t* cu_k, int tok, int& lo,
                                         int& hi) {
  lo = hi = 0;
  int a = 0, b = p.n_seqs + 1;            // cu_q[a - 1] <= tok < cu_q[b]
  while (a < b) {
    const int m = (a + b) >> 1;
    if (cu_q[m] <= tok) a = m + 1;
    else b = m;
  }
  if (a == 0 || a > p.n_seqs) return false;
  const int q1 = cu_q[a];
  lo = min(max(cu_k[a - 1], 0), p.Tk);
  hi = min(max(cu_k[a], lo), p.Tk);
  if (p.causal) hi = (int)max((long long)lo, (long long)hi - (q1 - 1 - tok));
  return true;
}

// Whether one of eight elements is infinite or NaN: its exponent, all ones, and
// one more carry into the sign's place.
template <typename T> __device__ __forceinline__ bool any_odd(uint4 u) {
  constexpr uint32_t e = std::is_same_v<T, __half> ? 0x7C007C00u : 0x7F807F80u;
  constexpr uint32_t one = std::is_same_v<T, __half> ? 0x04000400u : 0x00800080u;
  return (((u.x & e) + one) | ((u.y & e) + one) | ((u.z & e) + one) | ((u.w & e) + one)) & 0x80008000u;
}
// A word without those.
template <typename T> __device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  constexpr uint32_t e = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;
  if ((w & e) == e) w &= 0xFFFF0000u;
  if ((w & e << 16) == e << 16) w &= 0x0000FFFFu;
  return w;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const Params p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) uint8_t base[];
  if (smem_u32(base) & 1023) {            // the swizzle goes by addresses; there is no room to align here
    set_status(p.status, SSA_ST_INTERNAL);
    return;
  }
  uint8_t* s_q = base;
  uint8_t* s_kv = base + 2 * kTile;
  Shared& sh = *reinterpret_cast<Shared*>(base + (2 + kStages) * kTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr bool BF = !std::is_same_v<T, __half>;

  const int id = blockIdx.x, split = id % p.n_split, rest = id / p.n_split;
  const int head = rest % p.Hkv, place = p.n_ctas - 1 - rest / p.Hkv;   // the longest rows first
  const int tok0 = place * p.tiles * p.tpt;

  if (threadIdx.x < kStages) {
    mbar_init(&sh.full[threadIdx.x], 1);
    mbar_init(&sh.empty[threadIdx.x], 2 + kLooks);   // two MMA warps, and those that look through V
    mbar_init(&sh.clean[threadIdx.x], kLooks);
    fence_barrier_init();
  } else if (threadIdx.x >= 8 && threadIdx.x < 12) {
    const int t = threadIdx.x & 1, b = threadIdx.x >> 1 & 1;
    mbar_init(&sh.s_full[t][b], 1);
    mbar_init(&sh.p_full[t][b], 4);
    mbar_init(&sh.o_full[t][b], 1);
    fence_barrier_init();
  } else if (threadIdx.x == 12) {
    mbar_init(&sh.q_full[0], 1);
    mbar_init(&sh.q_full[1], 1);
    mbar_init(&sh.drain, 2);
    sh.abort = 0;
    sh.dirty[0] = INT_MAX;
    sh.dirty[1] = -1;
    fence_barrier_init();
  }
  if (warp == kMma) tmem_alloc_all(&sh.tmem);
  if (threadIdx.x == 256) { prefetch_tmap(&tm_q); prefetch_tmap(&tm_k); prefetch_tmap(&tm_v); }
  pdl_trigger();
  pdl_wait();
  const bool on_chip = p.n_seqs < kTable;
  if (on_chip && threadIdx.x <= p.n_seqs) {
    sh.cu_q[threadIdx.x] = p.cu_q[threadIdx.x];
    sh.cu_k[threadIdx.x] = p.cu_k[threadIdx.x];
  }
  tc5_fence_before();
  __syncthreads();
  tc5_fence_after();

  // rows: threads 0..127 tile 0, 128..255 tile 1
  const int tile = (threadIdx.x >> 7) & 1, r = threadIdx.x & 127;
  const int tok = tok0 + tile * p.tpt + r / p.G;
  int lo = 0, hi = 0;
  bool in_seq = false;
  if (threadIdx.x < 256) {
    if (tile < p.tiles && r < p.tpt * p.G && tok < p.Tq)
      in_seq = on_chip ? row_keys(p, sh.cu_q, sh.cu_k, tok, lo, hi) : row_keys(p, p.cu_q, p.cu_k, tok, lo, hi);
    const bool any = lo < hi;
    const int least = __reduce_min_sync(~0u, any ? lo : INT_MAX), most = __reduce_max_sync(~0u, any ? hi : 0);
    const int lo_max = __reduce_max_sync(~0u, any ? lo : 0), hi_min = __reduce_min_sync(~0u, any ? hi : INT_MAX);
    if (lane == 0) sh.seen[warp] = make_int4(least, most, lo_max, hi_min);
  } else if (warp == kTma) {
    // q needs no range
    for (int t = 0; lane == 0 && t < 2; ++t)
      if (t < p.tiles && tok0 + t * p.tpt < p.Tq) {
        mbar_arrive_expect_tx(&sh.q_full[t], 2u * 128u * p.G * p.tpt);
        for (int h = 0; h < 2; ++h)
          tma_load_4d(s_q + t * kTile + h * kHalf, &tm_q, &sh.q_full[t], h * 64, 0, head, tok0 + t * p.tpt);
      }
  } else if (id == 0) {                   // the tables themselves: ascending, inside the tensors
    bool bad = false;
    for (int i = threadIdx.x - 288; i <= p.n_seqs; i += kThreads - 288) {
      const int a = p.cu_q[i], b = p.cu_k[i];
      bad = bad || a < (i ? p.cu_q[i - 1] : 0) || b < (i ? p.cu_k[i - 1] : 0) || a > p.Tq || b > p.Tk;
    }
    if (bad) set_status(p.status, SSA_ST_BAD_POS);
  }
  __syncthreads();

  // blocks of this CTA, and of each tile in it
  int x0 = INT_MAX, end = 0, lo_max = 0, hi_min = INT_MAX, t_lo[2], t_hi[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    t_lo[t] = INT_MAX;
    t_hi[t] = 0;
#pragma unroll
    for (int w = 4 * t; w < 4 * t + 4; ++w) {
      const int4 u = sh.seen[w];
      t_lo[t] = min(t_lo[t], u.x);
      t_hi[t] = max(t_hi[t], u.y);
      lo_max = max(lo_max, u.z);          // what every row sees begins here
      hi_min = min(hi_min, u.w);          // and ends here
    }
    x0 = min(x0, t_lo[t]);
    end = max(end, t_hi[t]);
  }
  const int nb = end > 0 ? (end - x0 + kBlk - 1) / kBlk : 0;
  const int b0 = (int)((long long)nb * split / p.n_split), b1 = (int)((long long)nb * (split + 1) / p.n_split);
  int tb0[2], tb1[2], j1[2];              // j1: the first half block that a tile does not need
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    tb0[t] = tb1[t] = b1;
    if (t_hi[t] > 0) {
      tb0[t] = max(b0, (t_lo[t] - x0) / kBlk);
      tb1[t] = min(b1, (t_hi[t] - x0 + kBlk - 1) / kBlk);
      if (tb1[t] <= tb0[t]) tb0[t] = tb1[t] = b1;         // none in this part
    }
    j1[t] = tb0[t] < tb1[t] ? min(2 * tb1[t], (t_hi[t] - x0 + kSub - 1) / kSub) : 2 * tb0[t];
  }
  const uint32_t tmem = sh.tmem;
  volatile int* abort = &sh.abort;
  const auto give_up = [&](int bits) { sh.abort = 1; set_status(p.status, bits); };

  if (warp == kTma && lane == 0) {
    // ---- loads ----
    int it = 0;
    bool ok = true;
    for (int i = b0; ok && i < b1; ++i)
      for (int v = 0; ok && v < 2; ++v, ++it) {
        const int st = it % kStages, use = it / kStages;
        if (use > 0 && !mbar_wait(&sh.empty[st], (use - 1) & 1, abort)) { give_up(SSA_ST_TIMEOUT); ok = false; break; }
        mbar_arrive_expect_tx(&sh.full[st], kTile);
        for (int h = 0; h < 2; ++h)
          tma_load_3d(s_kv + st * kTile + h * kHalf, v ? (const void*)&tm_v : (const void*)&tm_k, &sh.full[st],
                      h * 64, head, x0 + i * kBlk);
      }
    // copies in flight land before the CTA goes: q's of rows without keys, and all if it gives up
    for (int t = 0; t < 2; ++t)
      if (t < p.tiles && tok0 + t * p.tpt < p.Tq) mbar_wait(&sh.q_full[t], 0, nullptr);
    if (*abort) {
      for (int j = max(0, it - kStages); j < it; ++j)
        mbar_wait(&sh.full[j % kStages], (j / kStages) & 1, nullptr);
    }
  } else if (warp == kMma || warp == kMma + 1) {
    // ---- MMAs: a warp a tile, its lanes together ----
    // Scores of two half blocks lie in tensor memory: while the softmax has one of
    // them the other is made, so that it never waits for the products of its own
    // tile.  S of half block j + 2 follows P V of j, whose P it overwrites.
    constexpr uint32_t id_qk = tc5_idesc(BF, kSub, false), id_pv = tc5_idesc(BF, kD, true);
    const int t = warp - kMma;
    const uint32_t q = tc5_desc(smem_u32(s_q + t * kTile), 16), a_k = tc5_desc(smem_u32(s_kv), 16),
                   a_v = tc5_desc(smem_u32(s_kv), kHalf);
    const uint32_t S = tmem + t * 128, O = tmem + 256 + t * 128;
    const int i0 = t ? tb0[1] : tb0[0], i1 = t ? tb1[1] : tb1[0], first = 2 * i0, last = t ? j1[1] : j1[0];
    bool ok = true;
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(~0u, mbar_wait(bar, parity, abort));
      if (!ok) give_up(SSA_ST_TIMEOUT);
    };
    // a stage is free when the MMAs that read it are done; a tile that reads
    // nothing of it lets it go at once
    const auto release = [&](uint64_t* bar, bool used) {
      if (used) tc5_commit(bar);
      else if (lane == 0) mbar_arrive(bar);
      __syncwarp();
    };
    // stages of the K and of the V at hand, and the phases of their barriers (V comes
    // to a stage every fifth block, K and V by turns)
    int ks = 0, vs = 1, v5 = 0;
    uint32_t kp = 0, vp = 0;
    const auto next_k = [&](bool used) {
      release(&sh.empty[ks], used);
      ks += 2;
      if (ks >= kStages) { ks -= kStages; kp ^= 1; }
    };
    const auto next_v = [&](bool used) {
      release(&sh.empty[vs], used);
      vs += 2;
      if (vs >= kStages) vs -= kStages;
      if (++v5 == kStages) { v5 = 0; vp ^= 1; }
    };
    const auto skip = [&](int n) {        // blocks that this tile does not need
      for (int i = 0; ok && i < n; ++i) {
        wait(&sh.full[ks], kp);
        if (ok) next_k(false);
        wait(&sh.clean[vs], vp);
        if (ok) next_v(false);
      }
    };
    const auto scores = [&](int j) {
      if (!(j & 1)) wait(&sh.full[ks], kp);
      if (!ok) return;
      const uint32_t kb = a_k + ks * (kTile >> 4) + (j & 1) * (kSub * 128 >> 4);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
        tc5_mma(S + (j & 1) * kSub, q + off, kb + off, id_qk, k > 0);
      }
      tc5_commit(&sh.s_full[t][j & 1]);
      if ((j & 1) || j == last - 1) next_k(true);
    };
    skip(i0 - b0);
    if (i0 < i1) {
      wait(&sh.q_full[t], 0);
      for (int j = first; ok && j < min(first + 2, last); ++j) scores(j);
      for (int j = first; ok && j < last; ++j) {
        if (!(j & 1)) wait(&sh.clean[vs], vp);
        wait(&sh.p_full[t][j & 1], ((j - first) >> 1) & 1);
        if (!ok) break;
        tc5_fence_after();
        const uint32_t v = a_v + vs * (kTile >> 4) + (j & 1) * (kSub * 128 >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) tc5_mma_ta(O, S + (j & 1) * kSub + k * 8, v + k * 128, id_pv, j > first || k > 0);
        tc5_commit(&sh.o_full[t][j & 1]);
        if (j + 2 < last) scores(j + 2);
        if ((j & 1) || j == last - 1) next_v(true);
      }
    }
    skip(b1 - max(i1, i0));
    release(&sh.drain, i0 < i1);          // no MMA is in flight when the CTA goes
    mbar_wait(&sh.drain, 0, nullptr);
  } else if (warp >= kLook) {
    // ---- V of the blocks that some row does not see all of: what is not finite becomes zero ----
    // They wait for K too, and a stage is free only when they have seen what it held:
    // copies land in any order, and the phase before the one waited for reads as a
    // phase that is done, so that a use that a waiter leaves out lets it pass too early.
    int st = 0;
    uint32_t ph = 0;
    const auto seen = [&](uint64_t* clean) {
      if (lane == 0) {
        if (clean) mbar_arrive(clean);
        mbar_arrive(&sh.empty[st]);
      }
      if (++st == kStages) { st = 0; ph ^= 1; }
    };
    for (int i = b0; i < b1; ++i) {
      if (!__all_sync(~0u, mbar_wait(&sh.full[st], ph, abort))) { give_up(SSA_ST_TIMEOUT); break; }
      seen(nullptr);
      if (!__all_sync(~0u, mbar_wait(&sh.full[st], ph, abort))) { give_up(SSA_ST_TIMEOUT); break; }
      if (x0 + i * kBlk < lo_max || x0 + (i + 1) * kBlk > hi_min) {
        uint4* v = reinterpret_cast<uint4*>(s_kv + st * kTile);
        bool found = false;
#pragma unroll 8
        for (int j = threadIdx.x - kLook * 32; j < kTile / 16; j += kLooks * 32) {
          const uint4 w = v[j];
          if (any_odd<T>(w)) {
            v[j] = make_uint4(finite_part<T>(w.x), finite_part<T>(w.y), finite_part<T>(w.z), finite_part<T>(w.w));
            found = true;
          }
        }
        if (found) {
          atomicMin(&sh.dirty[0], i);
          atomicMax(&sh.dirty[1], i);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
      }
      seen(&sh.clean[st]);
    }
  } else if (warp < 8) {
    // ---- softmax: a thread per row ----
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t S = tmem + tile * 128 + lanes, O = tmem + 256 + tile * 128 + lanes;
    const bool live = lo < hi;
    // a warp goes on together or not at all
    const auto all = [&](bool got) {
      const bool ok = __all_sync(~0u, got);
      if (!ok) give_up(SSA_ST_TIMEOUT);
      return ok;
    };
    // The first n products P V are done.  Each of the two barriers is at most one
    // phase short: the scores of half block n - 1 came behind the product n - 3,
    // which used the barrier of n - 1 before it.
    const auto o_done = [&](int n) { return mbar_wait(&sh.o_full[tile][(n - 1) & 1], ((n - 1) >> 1) & 1, abort); };
    float m = -INFINITY, l = 0.0f, z = 0.0f;              // reference, sum, sum of the rounded
    int n = 0;
    bool ok = true;
    const int first = 2 * (tile ? tb0[1] : tb0[0]), last = tile ? j1[1] : j1[0];
    for (int j = first; j < last; ++j, ++n) {
      const uint32_t Sj = S + (j & 1) * kSub;
      if (!all(mbar_wait(&sh.s_full[tile][j & 1], (n >> 1) & 1, abort))) { ok = false; break; }
      tc5_fence_after();
      const int x = x0 + j * kSub;
      const bool cut = __any_sync(~0u, live && (x < lo || x + kSub > hi));
      const uint32_t from = lo - x, len = hi - lo;
      uint32_t s[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c) tmem_ld32(s[c], Sj + 32 * c);
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        tmem_wait_ld(s[c]);
        if (cut) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((uint32_t)(32 * c + e) - from >= len) s[c][e] = 0xFF800000u;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
          mx[e & 3] = max3(mx[e & 3], __uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1]));
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
      const bool move = live && top > m + (kLazy + kBelow<T>);
      if (__any_sync(~0u, move)) {
        const float to = top - kBelow<T>, a = move ? fast_exp2(m - to) : 1.0f;
        if (move) m = to;
        l *= a;
        z *= a;
        if (n > 0) {
          if (!all(o_done(n))) { ok = false; break; }
          tc5_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld16(o, O + 16 * c);
            tmem_wait_ld16(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
            tmem_st16(O + 16 * c, o);
          }
        }
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2), ref2 = pack2(-ref, -ref);
      uint64_t sum[4] = {0, 0, 0, 0};
      float rounded[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 t = unpack2(fma2(pack2(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1])), scale2, ref2));
          const float e0 = fast_exp2(t.x), e1 = fast_exp2(t.y);
          sum[e & 3] = add2(sum[e & 3], pack2(e0, e1));
          w[e] = pack16<T>(e0, e1);
          add16<T>(w[e], rounded[2 * (e & 1)], rounded[2 * (e & 1) + 1]);
        }
        tmem_st16(Sj + 16 * c, w);        // over the scores
      }
      const float2 total = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
      l += total.x + total.y;
      z += (rounded[0] + rounded[1]) + (rounded[2] + rounded[3]);
      tmem_wait_st();
      tc5_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[tile][j & 1]);
    }
    // ---- epilogue ----
    if (ok && n > 0) ok = all(o_done(n));
    // (without a product nobody has waited for the queries, whose place is used below)
    if (ok && n == 0 && tile < p.tiles && tok0 + tile * p.tpt < p.Tq) ok = all(mbar_wait(&sh.q_full[tile], 0, abort));
    if (ok) {
      tc5_fence_after();
      const bool seen = live && n > 0;
      if (!live) { m = -INFINITY; l = z = 0.0f; }      // (a row without keys ran along)
      const size_t row = (((size_t)place * p.Hkv + head) * p.n_split + split) * (2 * kRows) + threadIdx.x;
      const int hq = head * p.G + r % p.G;
      if (p.n_split > 1) {
        if (tile < p.tiles && r < p.tpt * p.G && tok < p.Tq)
          reinterpret_cast<float4*>(p.part_ml)[row] = make_float4(m, in_seq ? l : -1.0f, z, 0.0f);
      } else if (in_seq && p.lse) {
        p.lse[(size_t)tok * p.Hq + hq] = l != 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
      // The warp's 32 rows go through the shared memory of its tile's queries, whose
      // products are done, so that a row is written by neighbouring lanes: 32 lanes
      // on 32 rows took 6,000 clocks.  256 bytes of a row at a time (all of it, or
      // half of the fp32 row of a split), 16-byte pieces turned by the row.
      uint8_t* const mine = s_q + tile * kTile + (warp & 3) * 32 * 256;
      const int64_t at_row = p.n_split > 1 ? (int64_t)row * kD : tok * p.o_tok + hq * p.o_head;
      const uint32_t rows = __ballot_sync(~0u, in_seq);
      const float f = p.n_split > 1 ? 1.0f : seen && z != 0.0f ? 1.0f / z : 0.0f;
      const auto write = [&](char* dst, int size) {
        __syncwarp();
        const int piece = lane & 15;
#pragma unroll 8
        for (int e = 0; e < 16; ++e) {
          const int rr = 2 * e + (lane >> 4);
          const int64_t at = __shfl_sync(~0u, at_row, rr);
          if (rows >> rr & 1)
            *reinterpret_cast<uint4*>(dst + at * size + 16 * piece) =
                *reinterpret_cast<const uint4*>(mine + rr * 256 + ((piece ^ (rr & 15)) << 4));
        }
        __syncwarp();
      };
      // What was set to zero, for the rows that see it: added to the staged row, elements
      // of type E, dimensions from `col` on.
      const int dirty0 = max(b0, sh.dirty[0]), dirty1 = min(b1, sh.dirty[1] + 1);
      const auto restore = [&](auto* type, int col, int dims) {
        using E = std::remove_const_t<std::remove_pointer_t<decltype(type)>>;
        if (!seen || dirty0 >= dirty1) return;
        const T* v = static_cast<const T*>(p.v) + head * p.v_head + col;
        for (int x = max(lo, x0 + dirty0 * kBlk); x < min(hi, x0 + dirty1 * kBlk); ++x)
#pragma unroll 4
          for (int e = 0; e < dims; ++e) {
            const float y = to_f32<T>(v[(int64_t)x * p.v_tok + e]);
            if (isfinite(y)) continue;
            const int at = e * (int)sizeof(E);
            E* z = reinterpret_cast<E*>(mine + lane * 256 + ((at >> 4 ^ (lane & 15)) << 4) + (at & 15));
            if constexpr (sizeof(E) == 4) *z += y;
            else *z = from_f32<T>(to_f32<T>(*z) + y);
          }
      };
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {       // 64 of the 128 dimensions
        uint32_t o[2][32];
        if (n > 0) {
          tmem_ld32(o[0], O + 64 * h);
          tmem_ld32(o[1], O + 64 * h + 32);
          tmem_wait_ld(o[0]);
          tmem_wait_ld(o[1]);
        }
        if (!seen) {
#pragma unroll
          for (int e = 0; e < 64; ++e) o[e >> 5][e & 31] = 0;
        }
        if (p.n_split > 1) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            *reinterpret_cast<uint4*>(mine + lane * 256 + ((e ^ (lane & 15)) << 4)) =
                *reinterpret_cast<uint4*>(&o[e >> 3][4 * (e & 7)]);
          restore(static_cast<const float*>(nullptr), 64 * h, 64);
          write(reinterpret_cast<char*>(p.part_o + 64 * h), 4);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t* x = &o[e >> 2][8 * (e & 3)];
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack16<T>(__uint_as_float(x[2 * i]) * f, __uint_as_float(x[2 * i + 1]) * f);
            *reinterpret_cast<uint4*>(mine + lane * 256 + (((8 * h + e) ^ (lane & 15)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (p.n_split == 1) {
        restore(static_cast<const T*>(nullptr), 0, kD);
        write(static_cast<char*>(p.out), 2);
      }
    }
    tc5_fence_before();
  }
  __syncwarp();
  __syncthreads();
  if (warp == kMma) {
    tc5_fence_after();
    tmem_free_all(tmem);
  }
}

// out = sum_s w_s O_s / sum_s w_s z_s, w_s = 2^(m_s - max m): `warps` warps a row, four
// dimensions a lane, eight splits of a warp in flight (each read is a round trip to
// L2: with one warp a row 76 splits took 25 us).  Always in the same order.
template <typename T>
__global__ void __launch_bounds__(256) prompt_join_kernel(const Params p, int warps) {
  __shared__ float4 s_o[8][32];
  __shared__ float s_m[8], s_l[8], s_z[8];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp & (warps - 1);
  const long long i = (long long)blockIdx.x * (8 / warps) + warp / warps;
  const int tok = (int)(i / p.Hq), hq = (int)(i % p.Hq);
  bool mine = tok < p.Tq;
  float m = -INFINITY, l = 0.0f, z = 0.0f;
  float4 o = make_float4(0, 0, 0, 0);
  if (mine) {
    const int head = hq / p.G, of_cta = p.tiles * p.tpt, in = tok % of_cta;
    const int r = in / p.tpt * kRows + in % p.tpt * p.G + hq % p.G;
    const size_t row0 = ((size_t)(tok / of_cta) * p.Hkv + head) * p.n_split * (2 * kRows) + r;
    for (int s0 = w; s0 < p.n_split; s0 += 8 * warps) {
      float4 ml[8];
      float4 y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const size_t row = row0 + (size_t)min(s0 + e * warps, p.n_split - 1) * 2 * kRows;
        ml[e] = reinterpret_cast<const float4*>(p.part_ml)[row];
        y[e] = reinterpret_cast<const float4*>(p.part_o + row * kD)[lane];
        if (s0 + e * warps >= p.n_split) ml[e] = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
      }
      if (ml[0].y < 0.0f) mine = false;   // not a token of any sequence: every split says so
      float top = m;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, ml[e].x);
      const float old = m == -INFINITY ? 0.0f : fast_exp2(m - top);
      m = top;
      l *= old;
      z *= old;
      o.x *= old; o.y *= old; o.z *= old; o.w *= old;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (ml[e].y == 0.0f) continue;    // saw no key
        const float f = fast_exp2(ml[e].x - m);
        l += f * ml[e].y;
        z += f * ml[e].z;
        o.x += f * y[e].x; o.y += f * y[e].y; o.z += f * y[e].z; o.w += f * y[e].w;
      }
    }
  }
  if (warps > 1) {
    s_o[warp][lane] = o;
    if (lane == 0) { s_m[warp] = m; s_l[warp] = l; s_z[warp] = z; }
    __syncthreads();
    if (w != 0) return;
    float top = m;
    for (int e = 1; e < warps; ++e) top = fmaxf(top, s_m[warp + e]);
    const float f0 = m == -INFINITY ? 0.0f : fast_exp2(m - top);
    l *= f0;
    z *= f0;
    o.x *= f0; o.y *= f0; o.z *= f0; o.w *= f0;
    for (int e = 1; e < warps; ++e) {
      if (s_l[warp + e] == 0.0f) continue;
      const float f = fast_exp2(s_m[warp + e] - top);
      const float4 y = s_o[warp + e][lane];
      l += f * s_l[warp + e];
      z += f * s_z[warp + e];
      o.x += f * y.x; o.y += f * y.y; o.z += f * y.z; o.w += f * y.w;
    }
    m = top;
  }
  if (!mine) return;
  const float f = z != 0.0f ? 1.0f / z : 0.0f;
  T* dst = static_cast<T*>(p.out) + tok * p.o_tok + hq * p.o_head + 4 * lane;
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<T>(o.x * f, o.y * f), pack16<T>(o.z * f, o.w * f));
  if (p.lse && lane == 0)
    p.lse[(size_t)tok * p.Hq + hq] = l != 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// One of k and v, [tokens][heads][128] with any strides: 128 tokens of one head.
bool map_kv(CUtensorMap* tm, const ssa_prompt_tensor& x, int n, bool bf) {
  cuuint64_t dims[3] = {kD, (cuuint64_t)x.heads, (cuuint64_t)n};
  cuuint64_t str[2] = {(cuuint64_t)(x.heads > 1 ? x.stride[1] : kD) * 2, (cuuint64_t)(n > 1 ? x.stride[0] : kD) * 2};
  cuuint32_t box[3] = {64, 1, kBlk}, one[3] = {1, 1, 1};
  auto fn = encode_fn();
  return fn && fn(tm, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, x.data, dims, str,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [tokens][KV heads][G][128]: a tile's tokens of one KV head.
bool map_q(CUtensorMap* tm, const ssa_prompt_tensor& x, int n, int Hkv, int tpt, bool bf) {
  const int G = x.heads / Hkv;
  const cuuint64_t hs = (cuuint64_t)(x.heads > 1 ? x.stride[1] : kD) * 2;
  cuuint64_t dims[4] = {kD, (cuuint64_t)G, (cuuint64_t)Hkv, (cuuint64_t)n};
  cuuint64_t str[3] = {hs, hs * G, (cuuint64_t)(n > 1 ? x.stride[0] : kD) * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)tpt}, one[4] = {1, 1, 1, 1};
  auto fn = encode_fn();
  return fn && fn(tm, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, x.data, dims, str,
                  box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
cudaError_t launch_prompt(const Params& p, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          cudaStream_t s) {
  // once a device: the attribute stays, and asking for it is a tenth of a small call
  static std::atomic<bool> asked[kMaxDevices];
  std::atomic<bool>& done = asked[current_device_ordinal()];
  cudaError_t e;
  if (!done.load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(prompt_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    if (e != cudaSuccess) return e;
    done.store(true, std::memory_order_relaxed);
  }
  const long long n = (long long)p.n_ctas * p.Hkv * p.n_split;
  if (n > INT_MAX) return cudaErrorInvalidValue;
  e = launch_pdl(prompt_kernel<T>, dim3((unsigned)n), dim3(kThreads), kSmem, s, p, q, k, v);
  count_launch();
  if (e != cudaSuccess || p.n_split == 1) return e;
  const long long rows = (long long)p.Tq * p.Hq;
  int warps = 1;                          // of a row: no more than eight splits to each
  while (warps < 8 && 8 * warps < p.n_split) warps *= 2;
  e = launch_pdl(prompt_join_kernel<T>, dim3((unsigned)((rows * warps + 7) / 8)), dim3(256), 0, s, p, warps);
  count_launch();
  return e;
}

// Partial rows of one launch: a split launch has no more CTAs than SMs.
size_t part_rows(int sms) { return (size_t)sms * 2 * kRows; }

// Parts that the keys of a CTA's rows are split into, where CTAs would not fill the
// machine.  How many keys a CTA walks over stands in the tables on the device; the
// host goes by the average sequence, and by the keys of all the sequences that
// share a CTA's tokens.  A CTA takes about 1 us for 80 keys (one tile: 140); a part more costs 528
// bytes of every row written and read, 0.26 ns a row, and the second kernel 5 us.
// (Before the second sum: 1,000 tokens, 16/2 heads: 18.8 us whole, 24.1 in two; 2,000 tokens, 8/1: 31.3 and
// 30.8; 64 tokens behind 8,000, 16/2: 109 whole, 18.0 in 15, 18.9 in 19; one token each
// of 8 sequences of 4,000: 370 whole, 19.6 in 62; one behind 30,000: 13.9 in 58,
// 16.9 in 152, so four blocks at least to a part.)
int splits(const Params& p, int n_seqs, int sms) {
  const long long units = (long long)p.n_ctas * p.Hkv;
  const double rows = (double)p.Tq * p.Hq;
  const double walk = std::min((double)p.Tk, std::max((double)p.Tk / n_seqs, (double)p.Tk / p.Tq * p.tiles * p.tpt));
  const double whole = walk / (p.tiles == 1 ? 140 : 80), row_cost = rows * 2.6e-4;                      // us
  const double best = std::min({(double)(sms / units), walk / (4 * kBlk), std::sqrt(whole / row_cost)});
  const int n = best > 2 ? (int)best : best >= 1.5 ? 2 : 1;
  if (n < 2 || n * units > sms) return 1;
  return whole * (1.0 - 1.0 / n) > 5 + row_cost * n ? n : 1;
}

int check_tensor(const ssa_prompt_tensor* x, int n) {
  if (!x || x->heads < 1) return SSA_ERR_INVALID_ARG;
  if (n > 0 && (!x->data || ((uintptr_t)x->data & 15))) return SSA_ERR_INVALID_ARG;
  const int size[2] = {n, x->heads};
  for (int i = 0; i < 2; ++i)
    if (size[i] > 1 && (x->stride[i] <= 0 || x->stride[i] % 8 || x->stride[i] >= 1ll << 38)) return SSA_ERR_INVALID_ARG;
  // (no address space has more; what follows stays within 64 bits)
  if (n > 0 && (double)(n - 1) * (n > 1 ? x->stride[0] : 0) + (double)(x->heads - 1) * (x->heads > 1 ? x->stride[1] : 0) > 0x1p56)
    return SSA_ERR_INVALID_ARG;
  return SSA_OK;
}

// Rows of kD elements, n tokens by heads.
struct Rows {
  int64_t at;                             // the first's address in elements
  int64_t n, heads, tok, head;            // counts and strides
  int64_t end() const { return at + (n - 1) * tok + (heads - 1) * head + kD; }
};
Rows rows_of(const ssa_prompt_tensor& x, int n) {
  return Rows{(int64_t)((uintptr_t)x.data / 2), n, x.heads, n > 1 ? x.stride[0] : 0, x.heads > 1 ? x.stride[1] : 0};
}
// Whether |c + k * step| < kD for some k in [k0, k1]: the one nearest to -c / step.
bool meets(int64_t c, int64_t step, int64_t k0, int64_t k1) {
  int64_t k = step ? -c / step : 0;
  for (int64_t i = k - 1; i <= k + 1; ++i) {
    const int64_t d = c + std::min(std::max(i, k0), k1) * step;
    if (d > -kD && d < kD) return true;
  }
  return false;
}
// Whether a row of a and a row of b share an element.  Slices of one buffer lie between
// each other's rows; token strides that differ there are taken for an overlap.
bool overlap(const Rows& a, const Rows& b) {
  if (a.at >= b.end() || b.at >= a.end()) return false;
  if (a.n > 1 && b.n > 1 && a.tok != b.tok) return true;
  const int64_t step = std::max(a.tok, b.tok);
  const bool alike = a.head == b.head || a.heads == 1 || b.heads == 1;
  const int64_t head = std::max(a.head, b.head);
  for (int64_t h = 0; h < a.heads; ++h)
    for (int64_t i = 0; i < b.heads; ++i) {
      // heads alike: only their difference counts, -(b.heads - 1) .. a.heads - 1
      if (alike && h > 0 && i > 0) break;
      if (meets(a.at - b.at + (alike ? (h - i) * head : h * a.head - i * b.head), step, 1 - b.n, a.n - 1)) return true;
    }
  return false;
}
// Whether two rows of x share an element.
bool overlaps_itself(const Rows& x) {
  if (x.heads > 1 && x.head < kD) return true;
  if (x.n == 1) return false;
  if (x.tok >= (x.heads - 1) * x.head + kD) return false;
  for (int64_t h = 0; h < x.heads; ++h)   // another token's, h heads on
    if (meets(h * x.head, x.tok, 1 - x.n, -1)) return true;
  return false;
}

}  // namespace
}  // namespace ssa

extern "C" {

size_t ssa_prompt_workspace_size(void) {
  return ssa::part_rows(ssa::current_device_info().sms) * (ssa::kD + 4) * sizeof(float);
}

int ssa_prompt_attention(int dtype, int head_dim, int n_seqs, int n_q, int n_kv, const ssa_prompt_tensor* q,
                         const ssa_prompt_tensor* k, const ssa_prompt_tensor* v, const ssa_prompt_tensor* out,
                         const int32_t* cu_q, const int32_t* cu_kv, int causal, float sm_scale, float* lse_opt,
                         int32_t* status, void* ws, ssa_stream_t stream) {
  using namespace ssa;
  if (dtype != SSA_BF16 && dtype != SSA_F16) return SSA_ERR_UNSUPPORTED;
  if (head_dim != kD) return SSA_ERR_UNSUPPORTED;
  if (n_seqs < 0 || n_q < 0 || n_kv < 0 || !cu_q || !cu_kv || !ws) return SSA_ERR_INVALID_ARG;
  if (!(sm_scale >= 0.0f) || !(sm_scale < INFINITY)) return SSA_ERR_INVALID_ARG;
  for (const ssa_prompt_tensor* x : {q, k, v, out})
    if (int e = check_tensor(x, x == q || x == out ? n_q : n_kv)) return e;
  if (k->heads != v->heads || q->heads != out->heads) return SSA_ERR_INVALID_ARG;
  if (q->heads % k->heads || q->heads / k->heads > kRows) return SSA_ERR_UNSUPPORTED;
  if ((uintptr_t)ws & 15) return SSA_ERR_INVALID_ARG;
  // (a tile's result may come before another's reads)
  if (n_q > 0) {
    const Rows o = rows_of(*out, n_q);
    if (overlaps_itself(o) || overlap(o, rows_of(*q, n_q))) return SSA_ERR_INVALID_ARG;
    if (n_kv > 0 && (overlap(o, rows_of(*k, n_kv)) || overlap(o, rows_of(*v, n_kv)))) return SSA_ERR_INVALID_ARG;
  }
  if (n_q > INT_MAX / 2 || n_kv > INT_MAX / 2) return SSA_ERR_UNSUPPORTED;
  if (n_q == 0 || n_seqs == 0) return SSA_OK;

  Params p{};
  p.cu_q = cu_q; p.cu_k = cu_kv;
  p.n_seqs = n_seqs; p.Tq = n_q; p.Tk = n_kv;
  p.Hq = q->heads; p.Hkv = k->heads; p.G = p.Hq / p.Hkv;
  p.tpt = kRows / p.G;
  // two tiles a CTA share its K and V; where one tile each fits the machine at once
  // the CTAs are twice as many and each is done sooner (2,000 tokens x 8/1 heads:
  // two tiles 31.5 us, one 25.5 before the second sum and 27.4 with it)
  const int sms = current_device_info().sms, n_tiles = (n_q + p.tpt - 1) / p.tpt;
  p.tiles = (long long)n_tiles * p.Hkv <= sms ? 1 : 2;
  p.n_ctas = (n_tiles + p.tiles - 1) / p.tiles;
  p.causal = causal ? 1 : 0;
  // not zero: masked scores are -inf, and stay so when scaled
  p.scale_log2 = std::max(sm_scale * 1.4426950408889634f, FLT_MIN);
  p.v = v->data; p.v_tok = v->stride[0]; p.v_head = v->stride[1];
  p.out = out->data; p.o_tok = out->stride[0]; p.o_head = out->stride[1];
  p.lse = lse_opt;
  p.status = status;
  p.n_split = splits(p, n_seqs, sms);
  p.part_o = static_cast<float*>(ws);
  p.part_ml = p.part_o + part_rows(sms) * kD;

  const bool bf = dtype == SSA_BF16;
  CUtensorMap mq, mk, mv;
  // without keys nothing is loaded through these two
  ssa_prompt_tensor none = *q;
  none.heads = k->heads;
  if (!map_q(&mq, *q, n_q, p.Hkv, p.tpt, bf) || !map_kv(&mk, n_kv ? *k : none, n_kv ? n_kv : 1, bf) ||
      !map_kv(&mv, n_kv ? *v : none, n_kv ? n_kv : 1, bf))
    return record_cuda_error(cudaErrorInvalidValue);
  const cudaError_t e = bf ? launch_prompt<__nv_bfloat16>(p, mq, mk, mv, (cudaStream_t)stream)
                           : launch_prompt<__half>(p, mq, mk, mv, (cudaStream_t)stream);
  return e == cudaSuccess ? SSA_OK : record_cuda_error(e);
}

}  // extern "C"
