// pages.cu -- who owns the pages of the cache: copying pages, forking, growing
// and freeing requests, compacting the logical page space.
//
// State: the block table [B][n_max], the lengths [B] and a reference count per
// logical page (rows that name it, plus what the caller pins).  A page is free
// when nothing refers to it.
//
// Fork.  Row i becomes a continuation of old row parent[i] (-1: of nothing),
// grown to new_lens[i] tokens.  Full pages are shared, by reference.  The
// partly filled last page g of the parent will be written by whoever continues
// it: with n_g rows continuing g and ref[g] - n_g other references left, the
// lowest of those rows keeps g if no other reference is left, and every other
// one gets a copy of it in a new page.  New pages are the lowest free ids, in
// row order (a row's copy first, then its growth).  Two launches:
//   plan   each row's old references off, its new ones on (g counts once per
//          row that continues it), the old table kept aside and the pages that
//          rows go on holding marked; then the last CTA to finish finds the free
//          pages (count 0 and not held: a held page that nothing counts is
//          flagged and counted), resolves the claims, scans the rows' needs and
//          lists that many free pages;
//   apply  the rows, and per layer the copies, the cleared slab rows of new
//          pages and the slots of freed ones.
//
// Compact.  With n live pages, the k-th live page at or above n moves to the
// k-th free id below it (both ascending): slab row and mirror block are
// copied, the two pages trade slots, so pool bytes stay where they are.
//
// What bounds them: the copies move each byte once in and once out (HBM; the
// mirror's over the host link); the tables are latency, a few dependent
// passes over B n_max and Lp words.  Copies: one CTA per 32 KB of a page's K or
// V and layer, eight 16-byte loads in flight per thread (with 16 KB and four,
// 400 pages of 12 layers took 118 us, now 101).
#include "common.cuh"
#include "internal.h"

namespace ssa {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll;     // 16-byte units per CTA
constexpr int kMoveUnroll = 4;                             // compaction: units per lane
constexpr int kPlanThreads = 1024;
constexpr int kPlanWords = 4096;         // words of page bits kept in shared memory
constexpr int kPlanList = 1024;          // new pages kept there
// most dynamic shared memory of a fork's plan: batch * max_sel <= 16384 and
// max_sel >= 10 leave 1638 rows, of seven words each
constexpr size_t kForkSmem = (7 * 1638 + kPlanWords) * sizeof(int32_t);

// The cache as the page calls see it.
struct PageCache {
  uint8_t *k_pool, *v_pool, *k_mir, *v_mir;
  float *k_scale, *v_scale, *ks_mir, *vs_mir;
  int8_t* slab;
  float *slab_scale, *slab_sum;
  int32_t *slab_cnt, *slot_of, *page_of, *last_use;
  int32_t* status;
  long long pb16;            // 16-byte units of a page's K (and V)
  int n_scale, HD, Lp, S;
  bool mirror() const { return k_mir != nullptr; }
};

__device__ __forceinline__ bool valid_page(const PageCache& c, int id) {
  return id >= 0 && id < c.Lp;
}

__device__ __forceinline__ int slot_at(const PageCache& c, int layer, int id) {
  const int s = c.slot_of[(size_t)layer * c.Lp + id];
  return s >= 0 && s < c.S ? s : -1;
}

// dst := src in one layer: where the pages are, and their 16-byte units, the
// concatenation [K | V | slab sums | slab codes] (the scales and counts apart).
// DST_SLOT: a pool slot that dst holds is written too.  POOL: K and V move in
// the pool as well (else only in the mirror).
template <bool DST_SLOT, bool POOL>
struct PageCopy {
  size_t ls, ld, ps, pd;
  int ss, sd;
  bool mir, can;
  long long kv16;
  __device__ __forceinline__ PageCopy(const PageCache& c, int layer, int src, int dst) {
    ls = (size_t)layer * c.Lp + src;
    ld = (size_t)layer * c.Lp + dst;
    mir = c.k_mir != nullptr;
    const bool kv = POOL || mir;
    ss = kv ? slot_at(c, layer, src) : -1;
    sd = DST_SLOT ? slot_at(c, layer, dst) : -1;
    ps = (size_t)layer * c.S + max(ss, 0);
    pd = (size_t)layer * c.S + max(sd, 0);
    can = kv && (ss >= 0 || mir) && (mir || sd >= 0);
    kv16 = can ? 2 * c.pb16 : 0;
  }
  __device__ __forceinline__ long long units(const PageCache& c) const {
    return kv16 + c.HD / 4 + c.HD / 16;
  }
  // unit u: read from `from`, written to `to`; K's and V's only where they
  // move in the mirror alone (compaction: !DST_SLOT, !POOL)
  __device__ __forceinline__ void unit(const PageCache& c, long long u, const uint4*& from,
                                       uint4*& to) const {
    if (!POOL && u < kv16) {
      const bool v = u >= c.pb16;
      if (v) u -= c.pb16;
      const uint4* pool = reinterpret_cast<const uint4*>(v ? c.v_pool : c.k_pool);
      uint4* m = reinterpret_cast<uint4*>(v ? c.v_mir : c.k_mir);
      from = ss >= 0 ? pool + ps * c.pb16 + u : m + ls * c.pb16 + u;
      to = m + ld * c.pb16 + u;
    } else if ((u -= kv16) < c.HD / 4) {
      uint4* sum = reinterpret_cast<uint4*>(c.slab_sum);
      from = sum + ls * (c.HD / 4) + u;
      to = sum + ld * (c.HD / 4) + u;
    } else {
      u -= c.HD / 4;
      uint4* code = reinterpret_cast<uint4*>(c.slab);
      from = code + ls * (c.HD / 16) + u;
      to = code + ld * (c.HD / 16) + u;
    }
  }
  // the scales, and the slab row's scale and count: threads i of n
  __device__ __forceinline__ void small(const PageCache& c, int i0, int n) const {
    if (i0 == 0) {
      c.slab_scale[ld] = c.slab_scale[ls];
      c.slab_cnt[ld] = c.slab_cnt[ls];
    }
    if (!can) return;
    for (int i = i0; i < 2 * c.n_scale; i += n) {
      const bool v = i >= c.n_scale;
      const int j = v ? i - c.n_scale : i;
      float* pool = v ? c.v_scale : c.k_scale;
      float* m = v ? c.vs_mir : c.ks_mir;
      const float s = ss >= 0 ? pool[ps * c.n_scale + j] : m[ls * c.n_scale + j];
      if (mir) m[ld * c.n_scale + j] = s;
      if (sd >= 0) pool[pd * c.n_scale + j] = s;
    }
  }
};

// One CTA's share, chunk `x`: 32 KB of K or V, or (the last chunk) the slab
// row, scales and counts.  `go` is asked, by every thread, once the loads are
// on their way: false leaves dst as it is.
template <bool DST_SLOT, bool POOL, typename Go>
__device__ __forceinline__ void copy_page(const PageCache& c, int layer, int src, int dst, int x,
                                          Go go) {
  const PageCopy<DST_SLOT, POOL> pc(c, layer, src, dst);
  const int pb16 = (int)c.pb16;
  const int nk = (pb16 + kCopyChunk - 1) / kCopyChunk;      // chunks of K, and of V
  const int tid = threadIdx.x;
  if (x < 2 * nk) {
    const bool v = x >= nk;
    const int u0 = (v ? x - nk : x) * kCopyChunk + tid;
    uint4* pool = reinterpret_cast<uint4*>(v ? c.v_pool : c.k_pool);
    uint4* m = reinterpret_cast<uint4*>(v ? c.v_mir : c.k_mir);
    const uint4* from = (pc.ss >= 0 ? pool + pc.ps * c.pb16 : m + pc.ls * c.pb16) + u0;
    uint4 buf[kCopyUnroll];
    if (pc.can) {
#pragma unroll
      for (int i = 0; i < kCopyUnroll; ++i)
        if (u0 + i * kCopyThreads < pb16) buf[i] = from[i * kCopyThreads];
    }
    if (!go() || !pc.can) return;
    auto put = [&](uint4* to) {
#pragma unroll
      for (int i = 0; i < kCopyUnroll; ++i)
        if (u0 + i * kCopyThreads < pb16) to[i * kCopyThreads] = buf[i];
    };
    if (pc.mir) put(m + pc.ld * c.pb16 + u0);
    if (pc.sd >= 0) put(pool + pc.pd * c.pb16 + u0);
    return;
  }
  uint4 buf[2];                            // HD <= 1024: at most 320 units of slab row
  const int units = c.HD / 4 + c.HD / 16;
  const uint4* from;
  uint4* to[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    to[i] = nullptr;
    if (tid + i * kCopyThreads < units) {
      pc.unit(c, pc.kv16 + tid + i * kCopyThreads, from, to[i]);
      buf[i] = *from;
    }
  }
  if (!go()) return;
  if (!pc.can && tid == 0) set_status(c.status, SSA_ST_UNRESOLVED);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (to[i]) *to[i] = buf[i];
  pc.small(c, tid, kCopyThreads);
}

// The slot a page holds becomes free (host tier: the mirror holds the page).
__device__ __forceinline__ void release_slot(const PageCache& c, int layer, int id) {
  int32_t* so = c.slot_of + (size_t)layer * c.Lp + id;
  const int s = *so;
  if (s < 0) return;
  if (s < c.S && c.page_of[(size_t)layer * c.S + s] == id) {
    c.page_of[(size_t)layer * c.S + s] = -1;
    c.last_use[(size_t)layer * c.S + s] = -1;
  }
  *so = -1;
}

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------

// Pair i is copied: both ids in range and different, dst[i] not the dst of an
// earlier pair nor the src of any (so no copy reads what another writes and
// the result does not depend on their order).

// This lane's share of the search for a pair that clashes with pair i.
__device__ __forceinline__ bool pair_clash(const int32_t* src, const int32_t* dst, int n, int i,
                                           int d, int first, int step) {
  bool clash = false;
  for (int j = first; j < n; j += step) {
    const int a = src[j], b = dst[j];
    if (a < 0 || b < 0 || j == i) continue;                 // padding, itself
    clash = clash || a == d || (j < i && b == d);
  }
  return clash;
}

// ok[i], a warp per pair
__global__ void copy_check_kernel(const int32_t* src, const int32_t* dst, int n, int32_t* ok,
                                  PageCache c) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= n) return;
  const int s = src[i], d = dst[i];
  bool good = false;
  if (s >= 0 && d >= 0) {
    const bool in = valid_page(c, s) && valid_page(c, d);
    good = in && !__any_sync(0xffffffffu, pair_clash(src, dst, n, i, d, lane, 32));
    if (!good && lane == 0) set_status(c.status, SSA_ST_BAD_ID);
  }
  if (lane == 0) ok[i] = good && s != d;
}

// FUSED: a few pairs, each CTA looks for clashes itself while its loads are on
// their way (1 pair of 2 layers: a microsecond less than with a launch that
// checks; 400 of 12 layers: a tenth more); else ok has the answer.
template <bool FUSED>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const int32_t* src,
                                                                  const int32_t* dst, int n,
                                                                  const int32_t* ok, PageCache c) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.y, layer = blockIdx.z;
  if (!FUSED && !ok[i]) return;
  const int s = src[i], d = dst[i];
  if (FUSED) {
    if (s < 0 || d < 0) return;
    if (!valid_page(c, s) || !valid_page(c, d)) {
      if (threadIdx.x == 0) set_status(c.status, SSA_ST_BAD_ID);
      return;
    }
  }
  copy_page<true, true>(c, layer, s, d, blockIdx.x, [&]() -> bool {
    if (!FUSED) return true;
    const bool clash = __syncthreads_or(pair_clash(src, dst, n, i, d, threadIdx.x, kCopyThreads));
    if (clash && threadIdx.x == 0) set_status(c.status, SSA_ST_BAD_ID);
    return !clash && s != d;
  });
}

// ---------------------------------------------------------------------------
// tables
// ---------------------------------------------------------------------------

struct Table {
  int32_t *bt, *lens, *ref;
  int B, nmax, P;
};

__device__ __forceinline__ int row_len(const Table& t, int i, int32_t* status) {
  const int n = t.lens[i];
  const long long most = (long long)t.nmax * t.P;
  if (n < 0 || n > most) {
    set_status(status, SSA_ST_BAD_POS);
    return n < 0 ? 0 : (int)most;
  }
  return n;
}

__global__ void count_refs_kernel(Table t, int Lp, int32_t* status) {
  pdl_trigger();
  pdl_wait();
  const long long n = (long long)t.B * t.nmax;
  for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < n;
       x += (long long)gridDim.x * blockDim.x) {
    const int i = (int)(x / t.nmax), p = (int)(x - (long long)i * t.nmax);
    const int len = row_len(t, i, status);
    if (p >= (len + t.P - 1) / t.P) continue;
    const int id = t.bt[x];
    if (id >= 0 && id < Lp) atomicAdd(&t.ref[id], 1);
    else set_status(status, SSA_ST_BAD_ID);
  }
}

// What a fork leaves in the workspace between its launches.
struct ForkWs {
  int32_t *old_bt, *old_len;     // [B][nmax], [B]
  uint32_t* bits;                // [ceil(Lp / 32)] free pages
  uint8_t* held;                 // [Lp] 1: a row holds the page after the call; zero between calls
  int32_t* list;                 // the new pages, in rank order
  int2* from;                    // [B] {the partly filled page the row continues or -1, the
                                 // parent's length}
  int4* plan;                    // [B] {parent, its length, new length, rank of its growth}
  int2* copy;                    // [B] {src, dst} of the row's copy; src -1: the last page is
                                 // kept, -2: it should have been copied
  int32_t* ticket;
};

__device__ __forceinline__ int parent_of(const int32_t* parent, int i, int B, int32_t* status) {
  const int j = parent[i];
  if (j >= -1 && j < B) return j;
  set_status(status, SSA_ST_BAD_ID);
  return i;
}

// One bit per page by one CTA: ref > 0 (live), or, FREE, neither counted nor
// held; into the workspace and, where it fits, shared memory, which is what
// the CTA goes on with.  FREE clears the marks for the next call, and a held
// page that nothing counts gets a count of one.
template <bool FREE>
__device__ __forceinline__ const uint32_t* page_bits(int32_t* ref, uint8_t* held, int Lp,
                                                     uint32_t* bits, uint32_t* s_bits,
                                                     int32_t* status) {
  constexpr int kBatch = 8;               // words a warp loads before it writes any
  const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  const int words = (Lp + 31) / 32;
  const bool fits = words <= kPlanWords;
  for (int w0 = threadIdx.x >> 5; w0 < words; w0 += kBatch * nw) {
    int n[kBatch];
    uint8_t h[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int id = (w0 + k * nw) * 32 + lane;
      n[k] = id < Lp ? __ldcg(&ref[id]) : (FREE ? 1 : 0);
      h[k] = FREE && id < Lp ? __ldcg(&held[id]) : 0;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int w = w0 + k * nw, id = w * 32 + lane;
      if (w >= words) break;
      if (FREE && h[k]) {
        held[id] = 0;
        if (n[k] <= 0) {
          ref[id] = 1;
          set_status(status, SSA_ST_BAD_ID);
        }
      }
      const uint32_t m = __ballot_sync(0xffffffffu, FREE ? n[k] <= 0 && !h[k] : n[k] > 0);
      if (lane == 0) {
        bits[w] = m;
        if (fits) s_bits[w] = m;
      }
    }
  }
  return fits ? s_bits : bits;
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(Table t, const int32_t* parent,
                                                                 const int32_t* new_lens, ForkWs w,
                                                                 PageCache c) {
  extern __shared__ int32_t dyn[];
  __shared__ int s_tmp[33];
  __shared__ int s_last;
  __shared__ int32_t s_list[kPlanList];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, B = t.B, P = t.P;
  // the references, and what each row continues
  {
    const int n = B * t.nmax;             // at most 1638 x 49152
    for (int x = blockIdx.x * kPlanThreads + tid; x < n; x += gridDim.x * kPlanThreads) {
      const int i = x / t.nmax, p = x - i * t.nmax;
      const int id = t.bt[x], len = row_len(t, i, c.status);
      const int j = parent_of(parent, i, B, c.status);
      const int jid = j >= 0 ? t.bt[j * t.nmax + p] : -1;
      const int jlen = j >= 0 ? row_len(t, j, c.status) : 0;
      w.old_bt[x] = id;
      if (p == 0) w.old_len[i] = len;
      if (p == (jlen % P ? jlen / P : 0))
        w.from[i] = make_int2(jlen % P && valid_page(c, jid) ? jid : -1, jlen);
      const bool out = j != i && p < (len + P - 1) / P, in = p < (jlen + P - 1) / P;
      if ((out && !valid_page(c, id)) || (in && !valid_page(c, jid)))
        set_status(c.status, SSA_ST_BAD_ID);
      if (out && valid_page(c, id)) atomicAdd(&t.ref[id], -1);
      if (in && valid_page(c, jid)) {
        w.held[jid] = 1;
        if (j != i) atomicAdd(&t.ref[jid], 1);
      }
    }
  }
  __syncthreads();
  if (gridDim.x > 1) {
    if (tid == 0) {
      __threadfence();
      s_last = atomicAdd(w.ticket, 1) == (int)gridDim.x - 1;
      if (s_last) {
        *w.ticket = 0;                    // ready for the next call
        __threadfence();
      }
    }
    __syncthreads();
    if (!s_last) return;
  }

  // the last CTA: which pages are free, what each row needs
  int32_t* gs = dyn;                      // [B] the partly filled page a row continues, or -1
  int32_t* refg = gs + B;                 // [B] references of it
  int32_t* plens = refg + B;              // [B] the parent's length
  int32_t* nlens = plens + B;             // [B] the new length
  int32_t* copies = nlens + B;            // [B] 1: the row needs a copy of that page
  int32_t* need = copies + B;             // [B] new pages
  int32_t* ranks = need + B;              // [B] the first of them in the list
  uint32_t* s_bits = reinterpret_cast<uint32_t*>(ranks + B);       // [kPlanWords] or none
  for (int i = tid; i < B; i += kPlanThreads) {
    const int2 f = __ldcg(&w.from[i]);
    const int want = new_lens ? new_lens[i] : 0;
    gs[i] = f.x;
    plens[i] = f.y;
    refg[i] = f.x >= 0 ? __ldcg(&t.ref[f.x]) : 0;
    const int most = t.nmax * P;
    if (want > most) set_status(c.status, SSA_ST_BAD_POS);
    nlens[i] = max(f.y, min(want, most));
  }
  const uint32_t* bits = page_bits<true>(t.ref, w.held, c.Lp, w.bits, s_bits, c.status);
  __syncthreads();
  for (int i = tid; i < B; i += kPlanThreads) {
    const int g = gs[i];
    int n = 0, first = i, left = 0;
    if (g >= 0) {
      for (int k = 0; k < B; ++k)
        if (gs[k] == g) {
          ++n;
          first = min(first, k);
        }
      left = max(refg[i] - n, 0);
      if (first == i) t.ref[g] = max(left, 1);               // the first row settles the count
    }
    copies[i] = first != i || left > 0;
    need[i] = copies[i] + (nlens[i] + P - 1) / P - (plens[i] + P - 1) / P;
  }
  __syncthreads();
  int total = 0;
  for (int base = 0; base < B; base += kPlanThreads) {
    const int i = base + tid;
    int sum;
    const int e = block_exclusive_scan(i < B ? need[i] : 0, s_tmp, sum);
    if (i < B) ranks[i] = total + e;
    total += sum;
  }
  // the lowest `total` free pages
  const int words = (c.Lp + 31) / 32;
  int got = 0;
  for (int base = 0; base < words && got < total; base += kPlanThreads) {
    const int x = base + tid;
    uint32_t m = x < words ? bits[x] : 0u;
    int sum;
    int r = got + block_exclusive_scan(__popc(m), s_tmp, sum);
    for (; m && r < total; m &= m - 1, ++r) {
      const int id = x * 32 + __ffs(m) - 1;
      w.list[r] = id;
      if (r < kPlanList) s_list[r] = id;
      t.ref[id] = 1;
    }
    got += sum;
  }
  if (got > total) got = total;
  __syncthreads();                        // the list is written
  for (int i = tid; i < B; i += kPlanThreads) {
    const int plen = plens[i], base = ranks[i], copy = copies[i];
    int nlen = nlens[i];
    const int avail = min(max(got - base, 0), need[i]);
    if (avail < need[i]) {                // too few free pages: the row is cut to what it has
      set_status(c.status, SSA_ST_NO_PAGES);
      if (copy && avail == 0) nlen = plen / P * P;
      else nlen = min(nlen, ((plen + P - 1) / P + avail - copy) * P);
    }
    w.copy[i] = copy ? (avail > 0 ? make_int2(gs[i], base < kPlanList ? s_list[base] : w.list[base]) : make_int2(-2, -1))
                     : make_int2(-1, -1);
    w.plan[i] = make_int4(parent_of(parent, i, B, nullptr), plen, nlen, base + copy);
  }
}

// grid (chunks, B, layers + 1): the last z writes the rows
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(Table t, ForkWs w, PageCache c) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.y, P = t.P, layer = blockIdx.z;
  const int4 pl = w.plan[i];
  const int2 cp = w.copy[i];
  const int j = pl.x, plen = pl.y, growth = pl.w;
  const int full = plen / P, pn = (plen + P - 1) / P, nn = (pl.z + P - 1) / P;
  const int first = blockIdx.x * kCopyThreads + threadIdx.x, step = gridDim.x * kCopyThreads;
  if (layer == (int)gridDim.z - 1) {
    for (int p = first; p < t.nmax; p += step) {
      int id = -1;
      if (p < nn) {
        if (p < full || (p < pn && cp.x == -1)) id = w.old_bt[(long long)j * t.nmax + p];
        else if (p < pn) id = cp.y;
        else id = w.list[growth + p - pn];
      }
      t.bt[(long long)i * t.nmax + p] = id;
    }
    if (first == 0) t.lens[i] = pl.z;
    return;
  }
  const bool mir = c.k_mir != nullptr;
  if (cp.x >= 0) {
    // a new page of a host-tier cache holds no slot: its copy goes to the mirror
    auto yes = []() { return true; };
    if (mir) {
      if (first == 0) release_slot(c, layer, cp.y);
      copy_page<false, true>(c, layer, cp.x, cp.y, blockIdx.x, yes);
    } else {
      copy_page<true, true>(c, layer, cp.x, cp.y, blockIdx.x, yes);
    }
  }
  // pages the row grew by: empty slab rows, no slot
  const int HD4 = c.HD / 4, HD16 = c.HD / 16;
  const int per = HD4 + HD16;
  for (long long u = first; u < (long long)(nn - pn) * per; u += step) {
    const int k = (int)(u / per), r = (int)(u - (long long)k * per);
    const int id = w.list[growth + k];
    const size_t lp = (size_t)layer * c.Lp + id;
    const uint4 z = make_uint4(0, 0, 0, 0);
    if (r < HD4) reinterpret_cast<uint4*>(c.slab_sum + lp * c.HD)[r] = z;
    else reinterpret_cast<uint4*>(c.slab + lp * c.HD)[r - HD4] = z;
    if (r == 0) {
      c.slab_scale[lp] = 0.0f;
      c.slab_cnt[lp] = 0;
      if (mir) release_slot(c, layer, id);
    }
  }
  // pages the row let go that nothing refers to now: their slots are free
  if (mir && j != i) {
    const int on = (w.old_len[i] + P - 1) / P;
    for (int p = first; p < on; p += step) {
      const int id = w.old_bt[(long long)i * t.nmax + p];
      if (valid_page(c, id) && (w.bits[id >> 5] >> (id & 31) & 1)) release_slot(c, layer, id);
    }
  }
}

// ---------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------

struct CompactWs {
  uint32_t* bits;                // live pages
  int32_t *from, *to, *map;      // the moves, ascending; map[from] = to
  int32_t* count;                // {live pages, moves}
};

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(Table t, CompactWs w, int Lp,
                                                                    int32_t* from_opt,
                                                                    int32_t* to_opt,
                                                                    int32_t* n_opt) {
  __shared__ int s_tmp[33];
  __shared__ uint32_t s_bits[kPlanWords];
  pdl_trigger();
  pdl_wait();
  const uint32_t* bits = page_bits<false>(t.ref, nullptr, Lp, w.bits, s_bits, nullptr);
  __syncthreads();
  const int tid = threadIdx.x, words = (Lp + 31) / 32;
  // live pages in all, then those below that number
  int mine = 0, n_live, below;
  for (int x = tid; x < words; x += kPlanThreads) mine += __popc(bits[x]);
  block_exclusive_scan(mine, s_tmp, n_live);
  mine = 0;
  for (int x = tid; x * 32 < n_live; x += kPlanThreads) {
    const int k = n_live - x * 32;
    mine += __popc(bits[x] & (k >= 32 ? 0xffffffffu : (1u << k) - 1u));
  }
  block_exclusive_scan(mine, s_tmp, below);
  const int moves = n_live - below;
  int seen = 0;                           // live pages before this round's words
  for (int base = 0; base < words && moves > 0; base += kPlanThreads) {
    const int x = base + tid;
    const uint32_t m = x < words ? bits[x] : 0u;
    int sum;
    const int pre = seen + block_exclusive_scan(__popc(m), s_tmp, sum);
    const int k = n_live - x * 32;        // ids of this word below n_live
    const uint32_t low = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
    if (x < words) {
      int r = x * 32 - pre;               // free ids before this word
      for (uint32_t h = ~m & low; h; h &= h - 1, ++r) w.to[r] = x * 32 + __ffs(h) - 1;
      r = pre + __popc(m & low) - below;  // moved pages before this word's
      for (uint32_t h = m & ~low; h; h &= h - 1, ++r) w.from[r] = x * 32 + __ffs(h) - 1;
    }
    seen += sum;
  }
  __syncthreads();
  for (int r = tid; r < moves; r += kPlanThreads) {
    const int a = w.from[r], b = w.to[r];
    w.map[a] = b;
    if (from_opt) from_opt[r] = a;
    if (to_opt) to_opt[r] = b;
  }
  if (tid == 0) {
    w.count[0] = n_live;
    w.count[1] = moves;
    if (n_opt) *n_opt = moves;
  }
}

// The moves: a warp per (page, layer, 128 of its 16-byte units), four of them
// in flight per lane.
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(CompactWs w, PageCache c,
                                                                    int layers, int chunks) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long items = (long long)w.count[1] * layers * chunks;
  const long long step = (long long)gridDim.x * (kCopyThreads / 32);
  for (long long it = (long long)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5); it < items;
       it += step) {
    const long long rest = it / chunks;
    const int x = (int)(it - rest * chunks), r = (int)(rest / layers);
    const PageCopy<false, false> pc(c, (int)(rest - (long long)r * layers), w.from[r], w.to[r]);
    const int units = (int)pc.units(c);
    uint4 buf[kMoveUnroll];
    uint4* to[kMoveUnroll];
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i) {
      const int u = (x * kMoveUnroll + i) * 32 + lane;
      to[i] = nullptr;
      if (u < units) {
        const uint4* from;
        pc.unit(c, u, from, to[i]);
        buf[i] = *from;
      }
    }
#pragma unroll
    for (int i = 0; i < kMoveUnroll; ++i)
      if (to[i]) *to[i] = buf[i];
    if (x == 0) pc.small(c, lane, 32);
  }
}

// The tables: rows, counts, and per layer the two pages' slots change hands.
__global__ void compact_tables_kernel(Table t, CompactWs w, PageCache c, int layers) {
  pdl_trigger();
  pdl_wait();
  const long long step = (long long)gridDim.x * blockDim.x;
  const long long first = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const int n_live = w.count[0], moves = w.count[1];
  for (long long x = first; x < (long long)t.B * t.nmax; x += step) {
    const int i = (int)(x / t.nmax), p = (int)(x - (long long)i * t.nmax);
    const int len = row_len(t, i, c.status);
    if (p >= (len + t.P - 1) / t.P) continue;
    const int id = t.bt[x];
    if (!valid_page(c, id) || !(w.bits[id >> 5] >> (id & 31) & 1))
      set_status(c.status, SSA_ST_BAD_ID);          // no page, or one nothing counts
    else if (id >= n_live)
      t.bt[x] = w.map[id];
  }
  for (long long x = first; x < (long long)moves * layers; x += step) {
    const int layer = (int)(x / moves), r = (int)(x - (long long)layer * moves);
    const int a = w.from[r], b = w.to[r];
    if (layer == 0) {
      t.ref[b] = t.ref[a];
      t.ref[a] = 0;
    }
    int32_t* so = c.slot_of + (size_t)layer * c.Lp;
    int32_t* po = c.page_of + (size_t)layer * c.S;
    const int sa = so[a], sb = so[b];
    so[b] = sa;
    so[a] = sb;
    if (sa >= 0 && sa < c.S) po[sa] = b;
    if (sb >= 0 && sb < c.S) po[sb] = a;
  }
}

PageCache page_cache(const Dims& d, const ssa_cache& c, int32_t* status) {
  PageCache p{};
  p.k_pool = static_cast<uint8_t*>(c.k_pool);
  p.v_pool = static_cast<uint8_t*>(c.v_pool);
  p.k_mir = static_cast<uint8_t*>(c.k_mirror);
  p.v_mir = static_cast<uint8_t*>(c.v_mirror);
  p.k_scale = c.k_scale; p.v_scale = c.v_scale;
  p.ks_mir = c.k_scale_mirror; p.vs_mir = c.v_scale_mirror;
  p.slab = c.slab;
  p.slab_scale = c.slab_scale; p.slab_sum = c.slab_sum;
  p.slab_cnt = c.slab_cnt;
  p.slot_of = c.slot_of; p.page_of = c.page_of; p.last_use = c.last_use;
  p.status = status;
  p.pb16 = (long long)d.page_bytes() / 16;
  p.n_scale = d.scale_floats();
  p.HD = d.Hkv * d.D;
  p.Lp = d.Lp; p.S = d.S;
  return p;
}

// CTAs of copy_page for one page and layer.
unsigned page_chunks(const PageCache& c) {
  return (unsigned)(2 * ((c.pb16 + kCopyChunk - 1) / kCopyChunk) + 1);
}

Table table_of(const Dims& d, const ssa_requests& r) {
  return Table{r.block_table, r.seq_lens, r.ref, d.B, d.nmax, d.P};
}

unsigned table_blocks(const Dims& d) {
  const long long n = ((long long)d.B * d.nmax + 255) / 256;
  return (unsigned)(n < 1024 ? n : 1024);
}

// Pairs up to which a copy looks for clashes itself.
constexpr int kFusedPairs = 64;

}  // namespace

cudaError_t launch_page_refs(const Dims& d, const ssa_requests& r, int32_t* status,
                             cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(r.ref, 0, (size_t)d.Lp * sizeof(int32_t), s);
  if (e != cudaSuccess) return e;
  e = launch_pdl(count_refs_kernel, dim3(table_blocks(d)), dim3(256), 0, s, table_of(d, r), d.Lp,
                 status);
  count_launch();
  return e;
}

cudaError_t launch_copy_pages(const Dims& d, const ssa_cache& c, const int32_t* src,
                              const int32_t* dst, int n, int32_t* status, const PageWs& w,
                              cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const PageCache pc = page_cache(d, c, status);
  const dim3 grid(page_chunks(pc), n, d.Lyr);
  cudaError_t e;
  if (n <= kFusedPairs) {
    e = launch_pdl(copy_pages_kernel<true>, grid, dim3(kCopyThreads), 0, s, src, dst, n,
                   (const int32_t*)nullptr, pc);
    count_launch();
    return e;
  }
  constexpr int kWarps = kCopyThreads / 32;
  e = launch_pdl(copy_check_kernel, dim3((n + kWarps - 1) / kWarps), dim3(kCopyThreads), 0, s, src,
                 dst, n, w.ok, pc);
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(copy_pages_kernel<false>, grid, dim3(kCopyThreads), 0, s, src, dst, n,
                 (const int32_t*)w.ok, pc);
  count_launch();
  return e;
}

cudaError_t launch_fork(const Dims& d, const ssa_cache& c, const ssa_requests& r,
                        const int32_t* parent, const int32_t* new_lens, int32_t* status,
                        const PageWs& w, int num_sms, cudaStream_t s) {
  const PageCache pc = page_cache(d, c, status);
  const Table t = table_of(d, r);
  const ForkWs fw{w.old_bt,       w.old_len,      w.bits,        w.held,  w.list,
                  (int2*)w.from,  (int4*)w.plan,  (int2*)w.copy, w.ticket};
  // one CTA up to four entries a thread (it then needs no ticket), else up to
  // two per SM
  const long long entries = (long long)d.B * d.nmax;
  long long ctas = entries <= 4 * kPlanThreads ? 1 : (entries + kPlanThreads - 1) / kPlanThreads;
  if (ctas > 2 * num_sms) ctas = 2 * num_sms;
  const int words = (d.Lp + 31) / 32;
  const size_t smem = ((size_t)7 * d.B + (words <= kPlanWords ? words : 0)) * sizeof(int32_t);
  if (smem > kForkSmem) return cudaErrorInvalidValue;
  // every call sets the same limit, so none lowers another's before its launch
  cudaError_t e = cudaFuncSetAttribute(
      fork_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kForkSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(fork_plan_kernel, dim3((unsigned)ctas), dim3(kPlanThreads), smem, s, t, parent,
                 new_lens, fw, pc);
  count_launch();
  if (e != cudaSuccess) return e;
  // growth can be many pages of few rows: eight CTAs a row and layer at least
  unsigned chunks = page_chunks(pc);
  if (new_lens && chunks < 8) chunks = 8;
  e = launch_pdl(fork_apply_kernel, dim3(chunks, d.B, d.Lyr + 1), dim3(kCopyThreads), 0, s, t, fw,
                 pc);
  count_launch();
  return e;
}

cudaError_t launch_compact(const Dims& d, const ssa_cache& c, const ssa_requests& r,
                           int32_t* moved_from, int32_t* moved_to, int32_t* n_moved,
                           int32_t* status, const PageWs& w, int num_sms, cudaStream_t s) {
  const PageCache pc = page_cache(d, c, status);
  const Table t = table_of(d, r);
  const CompactWs cw{w.bits, w.list, w.to, w.map, w.count};
  cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, t,
                             cw, d.Lp, moved_from, moved_to, n_moved);
  count_launch();
  if (e != cudaSuccess) return e;
  const long long per = (pc.mirror() ? 2 * pc.pb16 : 0) + pc.HD / 4 + pc.HD / 16;
  constexpr int kWarpUnits = 32 * kMoveUnroll;
  e = launch_pdl(compact_move_kernel, dim3(8 * num_sms), dim3(kCopyThreads), 0, s, cw, pc, d.Lyr,
                 (int)((per + kWarpUnits - 1) / kWarpUnits));
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(compact_tables_kernel, dim3(2 * num_sms), dim3(256), 0, s, t, cw, pc, d.Lyr);
  count_launch();
  return e;
}

}  // namespace ssa
