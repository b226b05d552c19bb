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
// row order (a row's copy first, then its growth).  Three launches:
//   count  each row's old references off, its new ones on (g counts once per
//          row that continues it, so a page is free exactly when its count is
//          0); the old table kept aside;
//   plan   one bit per free page; the last CTA to finish resolves the claims,
//          scans the rows' needs and lists that many free pages;
//   apply  the rows, and per layer the copies, the cleared slab rows of new
//          pages and the slots of freed ones.
//
// Compact.  With n live pages, the k-th live page at or above n moves to the
// k-th free id below it (both ascending): slab row and mirror block are
// copied, the two pages trade slots, so pool bytes stay where they are.
//
// What bounds them: the copies move each byte once in and once out (HBM; the
// mirror's over the host link); the tables are latency, a few dependent
// passes over B n_max and Lp words.  Copies: one CTA per 16 KB of a page and
// layer, four 16-byte loads in flight per thread.
#include "common.cuh"
#include "internal.h"

namespace ssa {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll;     // 16-byte units per CTA
constexpr int kPlanThreads = 512;

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

// One CTA's share of dst := src in one layer: chunk `x` of the concatenation
// [K | V | slab sums | slab codes], with chunk 0 the scales and counts.
// DST_SLOT: a pool slot that dst holds is written too.  POOL: pool and scale
// blocks move (else only the mirror's and the slab).
template <bool DST_SLOT, bool POOL>
__device__ __forceinline__ void copy_page(const PageCache& c, int layer, int src, int dst, int x) {
  const size_t ls = (size_t)layer * c.Lp + src, ld = (size_t)layer * c.Lp + dst;
  const bool mir = c.k_mir != nullptr;
  const bool kv = POOL || mir;
  const int ss = kv ? slot_at(c, layer, src) : -1;
  const int sd = DST_SLOT ? slot_at(c, layer, dst) : -1;
  const size_t ps = (size_t)layer * c.S + max(ss, 0), pd = (size_t)layer * c.S + max(sd, 0);
  const bool can = kv && (ss >= 0 || mir) && (mir || sd >= 0);
  if (kv && !can && x == 0 && threadIdx.x == 0) set_status(c.status, SSA_ST_UNRESOLVED);
  const long long kv16 = can ? 2 * c.pb16 : 0;
  const long long total = kv16 + c.HD / 4 + c.HD / 16;
  uint4 buf[kCopyUnroll];
  uint4 *d0[kCopyUnroll], *d1[kCopyUnroll];
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i) {
    long long u = (long long)x * kCopyChunk + i * kCopyThreads + threadIdx.x;
    d0[i] = d1[i] = nullptr;
    if (u >= total) continue;
    const uint4* from;
    if (u < kv16) {
      const bool v = u >= c.pb16;
      if (v) u -= c.pb16;
      const uint8_t* pool = v ? c.v_pool : c.k_pool;
      const uint8_t* m = v ? c.v_mir : c.k_mir;
      from = ss >= 0 ? reinterpret_cast<const uint4*>(pool) + ps * c.pb16 + u
                     : reinterpret_cast<const uint4*>(m) + ls * c.pb16 + u;
      if (mir) d0[i] = reinterpret_cast<uint4*>(v ? c.v_mir : c.k_mir) + ld * c.pb16 + u;
      if (sd >= 0) d1[i] = reinterpret_cast<uint4*>(v ? c.v_pool : c.k_pool) + pd * c.pb16 + u;
    } else if ((u -= kv16) < c.HD / 4) {
      from = reinterpret_cast<const uint4*>(c.slab_sum + ls * c.HD) + u;
      d0[i] = reinterpret_cast<uint4*>(c.slab_sum + ld * c.HD) + u;
    } else {
      u -= c.HD / 4;
      from = reinterpret_cast<const uint4*>(c.slab + ls * c.HD) + u;
      d0[i] = reinterpret_cast<uint4*>(c.slab + ld * c.HD) + u;
    }
    buf[i] = *from;
  }
#pragma unroll
  for (int i = 0; i < kCopyUnroll; ++i) {
    if (d0[i]) *d0[i] = buf[i];
    if (d1[i]) *d1[i] = buf[i];
  }
  if (x != 0) return;
  if (threadIdx.x == 0) {
    c.slab_scale[ld] = c.slab_scale[ls];
    c.slab_cnt[ld] = c.slab_cnt[ls];
  }
  if (!can) return;
  for (int i = threadIdx.x; i < 2 * c.n_scale; i += kCopyThreads) {
    const bool v = i >= c.n_scale;
    const int j = v ? i - c.n_scale : i;
    const float* pool = v ? c.v_scale : c.k_scale;
    const float* m = v ? c.vs_mir : c.ks_mir;
    const float s = ss >= 0 ? pool[ps * c.n_scale + j] : m[ls * c.n_scale + j];
    if (mir) (v ? c.vs_mir : c.ks_mir)[ld * c.n_scale + j] = s;
    if (sd >= 0) (v ? c.v_scale : c.k_scale)[pd * c.n_scale + j] = s;
  }
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

// ok[i] = pair i is copied: both ids in range and different, dst[i] not the
// dst of an earlier pair nor the src of any (so no copy reads what another
// writes and the result does not depend on their order).
__global__ void copy_check_kernel(const int32_t* src, const int32_t* dst, int n, int32_t* ok,
                                  PageCache c) {
  __shared__ int2 tile[kCopyThreads];
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x * kCopyThreads + threadIdx.x;
  const int s = i < n ? src[i] : -1, d = i < n ? dst[i] : -1;
  bool clash = false;
  for (int base = 0; base < n; base += kCopyThreads) {
    const int j = base + threadIdx.x;
    __syncthreads();
    tile[threadIdx.x] = j < n ? make_int2(src[j], dst[j]) : make_int2(-1, -1);
    __syncthreads();
    const int m = min(kCopyThreads, n - base);
    for (int k = 0; k < m; ++k) {
      const int2 o = tile[k];
      if (o.x < 0 || o.y < 0) continue;                     // padding
      if (base + k != i && o.x == d) clash = true;
      if (base + k < i && o.y == d) clash = true;
    }
  }
  if (i >= n) return;
  int good = 0;
  if (s >= 0 && d >= 0) {
    if (!valid_page(c, s) || !valid_page(c, d) || clash) set_status(c.status, SSA_ST_BAD_ID);
    else good = s != d;
  }
  ok[i] = good;
}

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const int32_t* src,
                                                                  const int32_t* dst,
                                                                  const int32_t* ok, PageCache c) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.y;
  if (!ok[i]) return;
  copy_page<true, true>(c, blockIdx.z, src[i], dst[i], blockIdx.x);
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
  int32_t* list;                 // the new pages, in rank order
  int4* plan;                    // [B] {parent, base, new length, 1 copy | 2 keep}
  int2* copy;                    // [B] {src, dst} of the row's copy, or -1
  int32_t* ticket;
};

__device__ __forceinline__ int parent_of(const int32_t* parent, int i, int B, int32_t* status) {
  const int j = parent[i];
  if (j >= -1 && j < B) return j;
  set_status(status, SSA_ST_BAD_ID);
  return i;
}

__global__ void fork_count_kernel(Table t, const int32_t* parent, ForkWs w, PageCache c) {
  pdl_trigger();
  pdl_wait();
  const long long n = (long long)t.B * t.nmax;
  auto add = [&](int id, int v) {
    if (valid_page(c, id)) atomicAdd(&t.ref[id], v);
    else set_status(c.status, SSA_ST_BAD_ID);
  };
  for (long long x = (long long)blockIdx.x * blockDim.x + threadIdx.x; x < n;
       x += (long long)gridDim.x * blockDim.x) {
    const int i = (int)(x / t.nmax), p = (int)(x - (long long)i * t.nmax);
    const int id = t.bt[x], len = row_len(t, i, c.status);
    w.old_bt[x] = id;
    if (p == 0) w.old_len[i] = len;
    const int j = parent_of(parent, i, t.B, c.status);
    if (j == i) continue;
    if (p < (len + t.P - 1) / t.P) add(id, -1);
    if (j >= 0 && p < (row_len(t, j, c.status) + t.P - 1) / t.P) add(t.bt[(long long)j * t.nmax + p], 1);
  }
}

// One bit per page: ref > 0 (live) or not, by the whole grid; the last CTA to
// finish gets true.
__device__ __forceinline__ bool page_bits(const int32_t* ref, int Lp, uint32_t* bits, bool live,
                                          int32_t* ticket) {
  __shared__ int s_last;
  const int lane = threadIdx.x & 31;
  const int words = (Lp + 31) / 32;
  const int warps = gridDim.x * (blockDim.x >> 5);
  for (int w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < words; w += warps) {
    const int id = w * 32 + lane;
    const bool bit = id < Lp && (__ldcg(&ref[id]) > 0) == live;
    const uint32_t m = __ballot_sync(0xffffffffu, bit);
    if (lane == 0) bits[w] = m;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    s_last = atomicAdd(ticket, 1) == (int)gridDim.x - 1;
    if (s_last) {
      *ticket = 0;                        // ready for the next call
      __threadfence();
    }
  }
  __syncthreads();
  return s_last;
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(Table t, const int32_t* parent,
                                                                 const int32_t* new_lens, ForkWs w,
                                                                 PageCache c) {
  extern __shared__ int32_t dyn[];
  __shared__ int s_tmp[33];
  pdl_trigger();
  pdl_wait();
  if (!page_bits(t.ref, c.Lp, w.bits, false, w.ticket)) return;
  const int tid = threadIdx.x, B = t.B, P = t.P;
  int32_t* gs = dyn;                      // [B] the partly filled page a row continues, or -1
  int32_t* others = gs + B;               // [B] its other references, -1 where another row settles them
  int32_t* need = others + B;             // [B] new pages
  for (int i = tid; i < B; i += kPlanThreads) {
    const int j = parent_of(parent, i, B, nullptr);
    const int plen = j >= 0 ? w.old_len[j] : 0;
    int g = -1;
    if (plen % P) {
      g = w.old_bt[(long long)j * t.nmax + plen / P];
      if (!valid_page(c, g)) g = -1;      // flagged by the count; carried as it is
    }
    gs[i] = g;
  }
  __syncthreads();
  for (int i = tid; i < B; i += kPlanThreads) {
    const int j = parent_of(parent, i, B, nullptr);
    const int plen = j >= 0 ? w.old_len[j] : 0;
    const int g = gs[i];
    int n = 0, first = i, left = 0, flags = 2;
    if (g >= 0) {
      for (int k = 0; k < B; ++k)
        if (gs[k] == g) {
          ++n;
          first = min(first, k);
        }
      left = __ldcg(&t.ref[g]) - n;
      flags = first == i && left <= 0 ? 2 : 1;
      if (first != i) left = -1;          // only the first row settles the count
      else left = max(left, 0);
    }
    others[i] = left;
    int nlen = plen;
    if (new_lens) {
      int want = new_lens[i];
      const long long most = (long long)t.nmax * P;
      if (want > most) {
        set_status(c.status, SSA_ST_BAD_POS);
        want = (int)most;
      }
      nlen = max(plen, want);
    }
    need[i] = (flags == 1) + (nlen + P - 1) / P - (plen + P - 1) / P;
    w.plan[i] = make_int4(j, 0, nlen, flags);
  }
  __syncthreads();
  int total = 0;
  for (int base = 0; base < B; base += kPlanThreads) {
    const int i = base + tid;
    int sum;
    const int v = i < B ? need[i] : 0;
    const int e = block_exclusive_scan(v, s_tmp, sum);
    if (i < B) {
      w.plan[i].y = total + e;
      if (gs[i] >= 0 && others[i] >= 0) t.ref[gs[i]] = max(others[i], 1);
    }
    total += sum;
  }
  // the lowest `total` free pages
  const int words = (c.Lp + 31) / 32;
  int got = 0;
  for (int base = 0; base < words && got < total; base += kPlanThreads) {
    const int x = base + tid;
    uint32_t m = x < words ? __ldcg(&w.bits[x]) : 0u;
    int sum;
    int r = got + block_exclusive_scan(__popc(m), s_tmp, sum);
    for (; m && r < total; m &= m - 1, ++r) {
      const int id = x * 32 + __ffs(m) - 1;
      w.list[r] = id;
      t.ref[id] = 1;
    }
    got += sum;
  }
  if (got > total) got = total;
  __syncthreads();                        // the list is written
  for (int i = tid; i < B; i += kPlanThreads) {
    int4 pl = w.plan[i];
    const int plen = pl.x >= 0 ? w.old_len[pl.x] : 0;
    const int avail = min(max(got - pl.y, 0), need[i]);
    if (avail < need[i]) {                // too few free pages: the row is cut to what it has
      set_status(c.status, SSA_ST_NO_PAGES);
      if (pl.w == 1 && avail == 0) pl.z = plen / P * P;
      else pl.z = min(pl.z, ((plen + P - 1) / P + avail - (pl.w == 1)) * P);
    }
    w.copy[i] = pl.w == 1 && avail > 0 ? make_int2(gs[i], w.list[pl.y]) : make_int2(-1, -1);
    w.plan[i] = pl;
  }
}

// grid (chunks, B, layers + 1): the last z writes the rows
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(Table t, ForkWs w, PageCache c) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.y, P = t.P, layer = blockIdx.z;
  const int4 pl = w.plan[i];
  const int2 cp = w.copy[i];
  const int j = pl.x;
  const int plen = j >= 0 ? w.old_len[j] : 0;
  const int full = plen / P, pn = (plen + P - 1) / P, nn = (pl.z + P - 1) / P;
  const int first = blockIdx.x * kCopyThreads + threadIdx.x, step = gridDim.x * kCopyThreads;
  const int growth = pl.y + (pl.w == 1);             // rank of the row's first growth page
  if (layer == (int)gridDim.z - 1) {
    for (int p = first; p < t.nmax; p += step) {
      int id = -1;
      if (p < nn) {
        if (p < full || (p < pn && pl.w == 2)) id = w.old_bt[(long long)j * t.nmax + p];
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
    if (mir) {
      if (first == 0) release_slot(c, layer, cp.y);
      copy_page<false, true>(c, layer, cp.x, cp.y, blockIdx.x);
    } else {
      copy_page<true, true>(c, layer, cp.x, cp.y, blockIdx.x);
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
  int32_t* ticket;
};

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(Table t, CompactWs w, int Lp,
                                                                    int32_t* from_opt,
                                                                    int32_t* to_opt,
                                                                    int32_t* n_opt) {
  __shared__ int s_tmp[33];
  pdl_trigger();
  pdl_wait();
  if (!page_bits(t.ref, Lp, w.bits, true, w.ticket)) return;
  const int tid = threadIdx.x, words = (Lp + 31) / 32;
  // live pages in all, then those below that number
  int mine = 0, n_live, below;
  for (int x = tid; x < words; x += kPlanThreads) mine += __popc(__ldcg(&w.bits[x]));
  block_exclusive_scan(mine, s_tmp, n_live);
  mine = 0;
  for (int x = tid; x * 32 < n_live; x += kPlanThreads) {
    const int k = n_live - x * 32;
    mine += __popc(__ldcg(&w.bits[x]) & (k >= 32 ? 0xffffffffu : (1u << k) - 1u));
  }
  block_exclusive_scan(mine, s_tmp, below);
  const int moves = n_live - below;
  int seen = 0;                           // live pages before this round's words
  for (int base = 0; base < words && moves > 0; base += kPlanThreads) {
    const int x = base + tid;
    const uint32_t m = x < words ? __ldcg(&w.bits[x]) : 0u;
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

__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(CompactWs w, PageCache c,
                                                                    int layers, int chunks) {
  pdl_trigger();
  pdl_wait();
  const long long items = (long long)w.count[1] * layers * chunks;
  for (long long it = blockIdx.x; it < items; it += gridDim.x) {
    const int x = (int)(it % chunks);
    const long long rest = it / chunks;
    const int layer = (int)(rest % layers), r = (int)(rest / layers);
    copy_page<false, false>(c, layer, w.from[r], w.to[r], x);
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

unsigned page_chunks(const PageCache& c, bool kv) {
  const long long total = (kv ? 2 * c.pb16 : 0) + c.HD / 4 + c.HD / 16;
  return (unsigned)((total + kCopyChunk - 1) / kCopyChunk);
}

Table table_of(const Dims& d, const ssa_requests& r) {
  return Table{r.block_table, r.seq_lens, r.ref, d.B, d.nmax, d.P};
}

unsigned table_blocks(const Dims& d) {
  const long long n = ((long long)d.B * d.nmax + 255) / 256;
  return (unsigned)(n < 1024 ? n : 1024);
}

// CTAs of the bit pass: a few words per warp
unsigned bit_blocks(const Dims& d) {
  const long long words = (d.Lp + 31) / 32, per = 8 * (kPlanThreads / 32);
  const long long n = (words + per - 1) / per;
  return (unsigned)(n < 1 ? 1 : n > 256 ? 256 : n);
}

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
  cudaError_t e = launch_pdl(copy_check_kernel, dim3((n + kCopyThreads - 1) / kCopyThreads),
                             dim3(kCopyThreads), 0, s, src, dst, n, w.ok, pc);
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(copy_pages_kernel, dim3(page_chunks(pc, true), n, d.Lyr), dim3(kCopyThreads), 0, s,
                 src, dst, (const int32_t*)w.ok, pc);
  count_launch();
  return e;
}

cudaError_t launch_fork(const Dims& d, const ssa_cache& c, const ssa_requests& r,
                        const int32_t* parent, const int32_t* new_lens, int32_t* status,
                        const PageWs& w, cudaStream_t s) {
  const PageCache pc = page_cache(d, c, status);
  const Table t = table_of(d, r);
  const ForkWs fw{w.old_bt, w.old_len, w.bits, w.list, (int4*)w.plan, (int2*)w.copy, w.ticket};
  cudaError_t e = launch_pdl(fork_count_kernel, dim3(table_blocks(d)), dim3(256), 0, s, t, parent,
                             fw, pc);
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(fork_plan_kernel, dim3(bit_blocks(d)), dim3(kPlanThreads),
                 (size_t)3 * d.B * sizeof(int32_t), s, t, parent, new_lens, fw, pc);
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(fork_apply_kernel, dim3(page_chunks(pc, true), d.B, d.Lyr + 1), dim3(kCopyThreads),
                 0, s, t, fw, pc);
  count_launch();
  return e;
}

cudaError_t launch_compact(const Dims& d, const ssa_cache& c, const ssa_requests& r,
                           int32_t* moved_from, int32_t* moved_to, int32_t* n_moved,
                           int32_t* status, const PageWs& w, int num_sms, cudaStream_t s) {
  const PageCache pc = page_cache(d, c, status);
  const Table t = table_of(d, r);
  const CompactWs cw{w.bits, w.list, w.to, w.map, w.count, w.ticket};
  cudaError_t e = launch_pdl(compact_plan_kernel, dim3(bit_blocks(d)), dim3(kPlanThreads), 0, s, t,
                             cw, d.Lp, moved_from, moved_to, n_moved);
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(compact_move_kernel, dim3(8 * num_sms), dim3(kCopyThreads), 0, s, cw, pc, d.Lyr,
                 (int)page_chunks(pc, pc.mirror()));
  count_launch();
  if (e != cudaSuccess) return e;
  e = launch_pdl(compact_tables_kernel, dim3(2 * num_sms), dim3(256), 0, s, t, cw, pc, d.Lyr);
  count_launch();
  return e;
}

}  // namespace ssa
