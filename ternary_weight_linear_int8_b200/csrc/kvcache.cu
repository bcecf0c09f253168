// Paged key-value cache: growing sequences, writing new rows, and the page
// operations of a serving pool (fork, free, compact, copy).
//
// The tables live on the device and every decision is made there, so that a
// captured step replays with whatever the tables hold then.  A page is free
// when its reference count is 0.  Pages are always taken lowest index first,
// in the order of the request, so each result is a function of the tables
// alone.  The calls that take pages either do all of their work or change
// nothing.
//
// The tables are small (4 bytes a page), so one block of 1024 threads plans a
// call: each scan over the counts reads 16 KB per step and is bound by the
// block's barriers, not by bandwidth.  The bytes are in the pages themselves,
// which the copy kernel moves with the whole card.
#include "attention.cuh"

namespace bitnet {

constexpr int kKvThreads = 1024;
constexpr int kKvMaxSlots = 65536;           // slots fit two shared-memory bit sets

// Lists the free pages in order until `want` are found; returns how many were
// (at most `want`).  Called by the whole block.
__device__ __forceinline__ int list_free_pages(const int32_t* refs, int n_pages, int want,
                                               int32_t* out, int* red) {
  int found = 0;
  for (int base = 0; base < n_pages && found < want; base += 4 * kKvThreads) {
    const int p0 = base + 4 * threadIdx.x;
    bool free[4];
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      free[i] = p0 + i < n_pages && refs[p0 + i] == 0;
      n += free[i];
    }
    int total, at = found + block_exclusive_sum(n, red, total);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (free[i]) {
        if (at < want) out[at] = p0 + i;
        ++at;
      }
    found += total;
  }
  __syncthreads();                           // the list is written
  return min(found, want);
}

__device__ __forceinline__ bool slot_ok(const KvTables& kv, int s) {
  return s >= 0 && s < kv.n_slots;
}
// Length of a slot, or -1 if it does not fit the table.
__device__ __forceinline__ int slot_len(const KvTables& kv, int s) {
  const int n = kv.lens[s];
  return n < 0 || (int64_t)n > (int64_t)kv.max_pages * kv.page_size ? -1 : n;
}
__device__ __forceinline__ bool set_bit(uint32_t* bits, int i) {   // true if it was set
  return (atomicOr(&bits[i >> 5], 1u << (i & 31)) >> (i & 31)) & 1u;
}

// The entries of one row's new tokens, [e0, e1) of slot s.
struct NewEntries {
  int s, e0, e1;
};
// Calls f(row of lane `src`, src) with the whole warp for every lane whose row
// has more than a few new entries (a prompt); the other rows (one token, as a
// rule) are left to their lanes.
constexpr int kFewEntries = 4;
template <typename F>
__device__ __forceinline__ void for_wide_rows(const NewEntries& r, F f) {
  unsigned m = __ballot_sync(0xffffffffu, r.e1 - r.e0 > kFewEntries);
  while (m) {
    const int src = __ffs(m) - 1;
    m &= m - 1;
    NewEntries w;
    w.s = __shfl_sync(0xffffffffu, r.s, src);
    w.e0 = __shfl_sync(0xffffffffu, r.e0, src);
    w.e1 = __shfl_sync(0xffffffffu, r.e1, src);
    f(w, src);
  }
}
// How many of a row's new entries name no page, for each lane's row.
__device__ __forceinline__ int count_missing(const KvTables& kv, const NewEntries& r) {
  int k = 0;
  if (r.e1 - r.e0 <= kFewEntries)
    for (int e = r.e0; e < r.e1; ++e) k += kv.table[(int64_t)r.s * kv.max_pages + e] < 0;
  for_wide_rows(r, [&](const NewEntries& w, int src) {
    int c = 0;
    for (int e = w.e0 + (threadIdx.x & 31); e < w.e1; e += 32)
      c += kv.table[(int64_t)w.s * kv.max_pages + e] < 0;
    c = __reduce_add_sync(0xffffffffu, c);
    if ((threadIdx.x & 31) == src) k = c;
  });
  return k;
}

// Sequences grow by add[i] tokens: entries of the new tokens that have no page
// get one.  A thread has a row.  ws: the free list [n_pages].  short_pages:
// see the header.
__global__ void __launch_bounds__(kKvThreads) kv_extend_kernel(KvTables kv, const int32_t* slots,
                                                               const int32_t* add, int n,
                                                               int32_t* short_pages,
                                                               int32_t* ws) {
  __shared__ uint32_t used[kKvMaxSlots / 32];
  __shared__ int red[33];
  __shared__ long long red64[32];
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const int words = (kv.n_slots + 31) / 32;
  for (int i = threadIdx.x; i < words; i += kKvThreads) used[i] = 0;
  __syncthreads();
  // check everything and count the pages wanted
  bool bad = false;
  long long want = 0;
  for (int base = 0; base < n; base += kKvThreads) {
    const int i = base + threadIdx.x;
    NewEntries r{0, 0, 0};
    if (i < n) {
      const int s = slots ? slots[i] : i, more = add[i];
      const int len = slot_ok(kv, s) && !set_bit(used, s) ? slot_len(kv, s) : -1;
      if (len < 0 || more < 0 || (int64_t)len + more > (int64_t)kv.max_pages * kv.page_size)
        bad = true;
      else
        r = NewEntries{s, (len + kv.page_size - 1) / kv.page_size,
                       (len + more + kv.page_size - 1) / kv.page_size};
    }
    want += count_missing(kv, r);
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      record_error(BITNET_ERR_PAGES);
      if (short_pages) *short_pages = -1;
    }
    return;
  }
  // The sum is 64 bits wide: a row may want more than the pool has, and all
  // rows together more than 2^31.  No more pages than there are get listed, and
  // the call goes on only if the list holds every page that it will take.
  const long long wanted = block_sum(want, red64);
  const int got = list_free_pages(kv.refs, kv.n_pages, (int)min(wanted, (long long)kv.n_pages), ws,
                                  red);
  if (got < wanted) {
    if (threadIdx.x == 0) {
      record_error(BITNET_ERR_PAGES);
      if (short_pages) *short_pages = (int)min(wanted - got, 0x7fffffffll);
    }
    return;
  }
  int taken = 0;
  for (int base = 0; base < n; base += kKvThreads) {
    const int i = base + threadIdx.x;
    NewEntries r{0, 0, 0};
    int len = 0;
    if (i < n) {
      r.s = slots ? slots[i] : i;
      const int old = kv.lens[r.s];
      len = old + add[i];
      r.e0 = (old + kv.page_size - 1) / kv.page_size;
      r.e1 = (len + kv.page_size - 1) / kv.page_size;
    }
    if (got > 0) {
      const int k = count_missing(kv, r);
      int sum;
      int at = taken + block_exclusive_sum(k, red, sum);
      taken += sum;
      for_wide_rows(r, [&](const NewEntries& w, int src) {
        int to = __shfl_sync(0xffffffffu, at, src);
        for (int e = w.e0; e < w.e1; e += 32) {
          int32_t* t = kv.table + (int64_t)w.s * kv.max_pages + e + lane;
          const bool take = e + lane < w.e1 && *t < 0;
          const unsigned m = __ballot_sync(0xffffffffu, take);
          if (take) {
            const int page = ws[to + __popc(m & ((1u << lane) - 1))];
            *t = page;
            kv.refs[page] = 1;
          }
          to += __popc(m);
        }
      });
      if (r.e1 - r.e0 <= kFewEntries)
        for (int e = r.e0; e < r.e1; ++e) {
          int32_t* t = kv.table + (int64_t)r.s * kv.max_pages + e;
          if (*t >= 0) continue;
          const int page = ws[at++];
          *t = page;
          kv.refs[page] = 1;
        }
    }
    if (i < n) kv.lens[r.s] = len;
  }
  if (short_pages && threadIdx.x == 0) *short_pages = 0;
}

// Tables of up to this many entries are finished by the planning block itself
// instead of a second launch: 48 forks of rows of 23 entries take 5.9 us of
// device time in one launch and 6.4 in two (and 2 us less of the host's), 128
// of rows of 64 entries 10.0 and 7.5 (the check of the parents' entries came to
// both later); compactions of 2208 entries 4.6 and 5.2.
constexpr int64_t kKvOneBlock = 4096;

// Entries first, first + step, .. of the children's table rows, and the counts
// of the pages they share.
__device__ __forceinline__ void fork_rows(const KvTables& kv, const int32_t* parents,
                                          const int32_t* children, int n, const int32_t* fresh,
                                          int64_t first, int64_t step) {
  for (int64_t x = first; x < (int64_t)n * kv.max_pages; x += step) {
    const int i = (int)(x / kv.max_pages), e = (int)(x % kv.max_pages);
    const int p = parents[i], c = children[i], len = kv.lens[p], full = len / kv.page_size;
    int page = -1;
    if (e < full) {                          // inside the pool: the plan has checked
      page = kv.table[(int64_t)p * kv.max_pages + e];
      atomicAdd(&kv.refs[page], 1);          // integer: the order does not matter
    } else if (e == full) {
      page = fresh[i];
    }
    kv.table[(int64_t)c * kv.max_pages + e] = page;
  }
}

// Plans a fork: checks the pairs, takes a page for each child whose parent
// ends inside a page and lists the copy.  ws: [0] go flag, then the children's
// new pages [n] (-1: none), then the free list.
__global__ void __launch_bounds__(kKvThreads) kv_fork_plan_kernel(
    KvTables kv, const int32_t* parents, const int32_t* children, int n, int32_t* pairs,
    int32_t* n_pairs, int32_t* short_pages, int32_t* ws, bool one_block) {
  __shared__ uint32_t is_child[kKvMaxSlots / 32], is_parent[kKvMaxSlots / 32];
  __shared__ int red[33];
  pdl_wait();
  const int words = (kv.n_slots + 31) / 32;
  for (int i = threadIdx.x; i < words; i += kKvThreads) is_child[i] = is_parent[i] = 0;
  __syncthreads();
  int32_t* fresh = ws + 4;
  int32_t* list = fresh + n;
  bool bad = false;
  int want = 0;
  for (int i = threadIdx.x; i < n; i += kKvThreads) {
    const int p = parents[i], c = children[i];
    if (!slot_ok(kv, p) || !slot_ok(kv, c) || set_bit(is_child, c) || kv.lens[c] != 0) {
      bad = true;
      continue;
    }
    const int len = slot_len(kv, p);
    if (len < 0) { bad = true; continue; }
    want += len % kv.page_size != 0;
  }
  __syncthreads();                           // every child is marked
  for (int i = threadIdx.x; i < n && !bad; i += kKvThreads)
    if ((is_child[parents[i] >> 5] >> (parents[i] & 31)) & 1u) bad = true;   // parent and child
  bad = __syncthreads_or(bad);
  if (!bad) {
    // every entry that a parent's tokens lie in names a page: a warp per
    // parent, however often it is named, 16 entries a lane on their way.  Costs
    // 0.6 us for 48 children of 6 parents of 22 entries (5.6 -> 6.2 us), 1.2 for 16
    // children of 4 parents of 1875 (5.4 -> 6.6); loads one after the other cost 6.5
    // there.
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < n; i += kKvThreads / 32) {
      const int p = parents[i];
      int again = 0;
      if (lane == 0) again = set_bit(is_parent, p);
      if (__shfl_sync(0xffffffffu, again, 0)) continue;
      const int held = (kv.lens[p] + kv.page_size - 1) / kv.page_size;
      const int32_t* t = kv.table + (int64_t)p * kv.max_pages;
      for (int e0 = lane; e0 < held; e0 += 32 * 16) {
        unsigned page[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) page[x] = e0 + 32 * x < held ? t[e0 + 32 * x] : 0;
#pragma unroll
        for (int x = 0; x < 16; ++x) bad |= page[x] >= (unsigned)kv.n_pages;
      }
    }
    bad = __syncthreads_or(bad);
  }
  int total = 0, got = 0;
  if (!bad) {
    block_exclusive_sum(want, red, total);
    got = list_free_pages(kv.refs, kv.n_pages, total, list, red);
  }
  const bool go = !bad && got == total;
  if (threadIdx.x == 0) {
    if (!go) record_error(BITNET_ERR_PAGES);
    if (short_pages) *short_pages = bad ? -1 : total - got;
    *n_pairs = go ? total : 0;
    ws[0] = go;
  }
  if (!go) return;
  int taken = 0;
  for (int base = 0; base < n; base += kKvThreads) {
    const int i = base + threadIdx.x;
    int p = 0, len = 0;
    if (i < n) {
      p = parents[i];
      len = kv.lens[p];
    }
    const int k = len % kv.page_size != 0;
    int sum, at = taken + block_exclusive_sum(k, red, sum);
    if (i < n) {
      const int page = k ? list[at] : -1;
      fresh[i] = page;
      if (k) {
        kv.refs[page] = 1;
        pairs[2 * at] = kv.table[(int64_t)p * kv.max_pages + len / kv.page_size];
        pairs[2 * at + 1] = page;
      }
      kv.lens[children[i]] = len;
    }
    taken += sum;
  }
  if (one_block) {
    __syncthreads();
    fork_rows(kv, parents, children, n, fresh, threadIdx.x, kKvThreads);
  }
}

__global__ void __launch_bounds__(256) kv_fork_rows_kernel(KvTables kv, const int32_t* parents,
                                                           const int32_t* children, int n,
                                                           const int32_t* ws) {
  pdl_wait();
  if (!ws[0]) return;
  fork_rows(kv, parents, children, n, ws + 4, blockIdx.x * 256ll + threadIdx.x, gridDim.x * 256ll);
}

// Drops the pages of sequences.  An entry is taken out by an exchange, so a
// slot that is named twice gives its pages back once.
__global__ void __launch_bounds__(256) kv_free_kernel(KvTables kv, const int32_t* slots, int n) {
  pdl_wait();
  for (int64_t x = blockIdx.x * 256ll + threadIdx.x; x < (int64_t)n * kv.max_pages;
       x += gridDim.x * 256ll) {
    const int i = (int)(x / kv.max_pages), e = (int)(x % kv.max_pages);
    const int s = slots[i];
    if (!slot_ok(kv, s)) {
      if (e == 0) record_error(BITNET_ERR_PAGES);
      continue;
    }
    int32_t* t = kv.table + (int64_t)s * kv.max_pages + e;
    if (*t >= 0) {
      const int page = atomicExch(t, -1);
      if (page >= 0) {
        if (page >= kv.n_pages) {
          record_error(BITNET_ERR_PAGES);
        } else if (atomicSub(&kv.refs[page], 1) <= 0) {   // no count held the entry: it stays free
          atomicAdd(&kv.refs[page], 1);
          record_error(BITNET_ERR_PAGES);
        }
      }
    }
    if (e == 0) kv.lens[s] = 0;
  }
}

// Table entries first, first + step, .. that name a page at or above `used`.
__device__ __forceinline__ void compact_entries(const KvTables& kv, int used, const int32_t* to,
                                                int64_t first, int64_t step) {
  for (int64_t x = first; x < (int64_t)kv.n_slots * kv.max_pages; x += step) {
    const int p = kv.table[x];
    if (p < used) continue;
    const int dst = p < kv.n_pages ? to[p] : -1;
    if (dst < 0) record_error(BITNET_ERR_PAGES);   // an entry that no count holds
    kv.table[x] = dst;
  }
}

// Plans a compaction: with L pages in use, those at L and above move into the
// free ones below, both in order.  ws: [0] L, then the new page of each page
// at L and above [n_pages], then the free list.
__global__ void __launch_bounds__(kKvThreads) kv_compact_plan_kernel(KvTables kv, int32_t* pairs,
                                                                     int32_t* n_pairs,
                                                                     int32_t* live, int32_t* ws,
                                                                     bool one_block) {
  __shared__ int red[33];
  pdl_wait();
  int mine = 0;
#pragma unroll 8
  for (int p = threadIdx.x; p < kv.n_pages; p += kKvThreads) mine += kv.refs[p] != 0;
  int used;
  block_exclusive_sum(mine, red, used);
  int32_t* to = ws + 4;
  int32_t* holes = to + kv.n_pages;
  // as many pages in use lie at or above `used` as free ones lie below it
  const int moves = list_free_pages(kv.refs, used, used, holes, red);
  int at0 = 0;
  for (int base = used; base < kv.n_pages; base += 4 * kKvThreads) {
    const int p0 = base + 4 * threadIdx.x;
    int r[4], n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = p0 + i < kv.n_pages ? kv.refs[p0 + i] : 0;
      n += r[i] != 0;
    }
    int sum;
    int at = at0 + block_exclusive_sum(n, red, sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + i;
      if (p >= kv.n_pages) break;
      int dst = -1;
      if (r[i] != 0) {
        dst = holes[at];
        pairs[2 * at] = p;
        pairs[2 * at + 1] = dst;
        kv.refs[dst] = r[i];
        kv.refs[p] = 0;
        ++at;
      }
      to[p] = dst;
    }
    at0 += sum;
  }
  if (threadIdx.x == 0) {
    *n_pairs = moves;
    if (live) *live = used;
    ws[0] = used;
  }
  if (one_block) {
    __syncthreads();
    compact_entries(kv, used, to, threadIdx.x, kKvThreads);
  }
}

__global__ void __launch_bounds__(256) kv_compact_table_kernel(KvTables kv, const int32_t* ws) {
  pdl_wait();
  compact_entries(kv, ws[0], ws + 4, blockIdx.x * 256ll + threadIdx.x, gridDim.x * 256ll);
}

// Copies pages within the caches of up to kCopyLayers layers.  The list is on
// the device; a pair outside the pool is skipped and recorded.
constexpr int kCopyLayers = 64;
struct KvCopyArgs {
  uint4* base[2 * kCopyLayers];              // keys and values of each layer
  const int32_t* pairs;
  const int32_t* n_pairs;
  int max_pairs, n_pages, planes;            // planes = 2 * layers
  int64_t page_chunks;                       // 16-byte chunks per page
};

constexpr int kCopyThreads = 256, kCopyPer = 8;   // chunks in flight per thread
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const __grid_constant__ KvCopyArgs a) {
  pdl_wait();
  const int n = min(*a.n_pairs, a.max_pairs);
  const int64_t piece = kCopyThreads * kCopyPer;
  const int64_t pieces = (a.page_chunks + piece - 1) / piece;   // per page
  const int64_t work = n > 0 ? (int64_t)n * a.planes * pieces : 0;
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int64_t pc = w % pieces, rest = w / pieces;
    const int pl = (int)(rest % a.planes), i = (int)(rest / a.planes);
    const int src = a.pairs[2 * i], dst = a.pairs[2 * i + 1];
    if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages) {
      if (threadIdx.x == 0) record_error(BITNET_ERR_PAGES);
      continue;
    }
    const uint4* s = a.base[pl] + (int64_t)src * a.page_chunks;
    uint4* d = a.base[pl] + (int64_t)dst * a.page_chunks;
    uint4 v[kCopyPer];
#pragma unroll
    for (int x = 0; x < kCopyPer; ++x) {
      const int64_t c = pc * piece + x * kCopyThreads + threadIdx.x;
      if (c < a.page_chunks) v[x] = s[c];
    }
#pragma unroll
    for (int x = 0; x < kCopyPer; ++x) {
      const int64_t c = pc * piece + x * kCopyThreads + threadIdx.x;
      if (c < a.page_chunks) d[c] = v[x];
    }
  }
}

// New key and value rows into their pages: row r of batch row b goes to
// position lens[slot] - (rows of b) + r.  One warp per token.
struct KvAppendArgs {
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* cu;                         // [B + 1]
  const int32_t* slots;
  KvTables kv;
  uint16_t* k_pages;
  uint16_t* v_pages;
  int64_t k_stride, v_stride;
  int B, T, Hkv;
};

template <int D>
__global__ void __launch_bounds__(256) kv_append_kernel(const KvAppendArgs a) {
  constexpr int CH = D / 8;                  // 16-byte chunks per head
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= a.T) return;
  // the last b with cu[b] <= r, 32 candidates at a time
  int lo = 0, n = a.B + 1;                   // cu[lo .. lo + n - 1]
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lane * step;
    const bool le = i < n && a.cu[lo + i] <= r;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (!(m & 1u)) return;                   // before the first sequence
    const int k = 31 - __clz(m);
    lo += k * step;
    n = min(step, n - k * step);
  }
  const int b = lo;
  if (b >= a.B) return;                      // behind the last sequence
  const int c0 = a.cu[b], c1 = a.cu[b + 1];
  if (r < c0 || r >= c1) return;
  const int s = a.slots ? a.slots[b] : b;
  int64_t page = -1;
  int row = 0;
  if (slot_ok(a.kv, s)) {
    const int len = slot_len(a.kv, s);
    // below len, since r < c1; in 64 bits, whatever the bounds are
    const int64_t pos = (int64_t)len - c1 + r;
    if (len >= 0 && pos >= 0) {
      const int e = (int)(pos / a.kv.page_size);
      row = (int)(pos - (int64_t)e * a.kv.page_size);
      page = a.kv.table[(int64_t)s * a.kv.max_pages + e];
    }
  }
  if (page < 0 || page >= a.kv.n_pages) {
    if (lane == 0) record_error(BITNET_ERR_PAGES);
    return;
  }
  const uint4* ks = reinterpret_cast<const uint4*>(a.k + (int64_t)r * a.k_stride);
  const uint4* vs = reinterpret_cast<const uint4*>(a.v + (int64_t)r * a.v_stride);
  uint4* kd = reinterpret_cast<uint4*>(a.k_pages);
  uint4* vd = reinterpret_cast<uint4*>(a.v_pages);
  // four chunks of the keys and four of the values on their way per lane
  for (int x0 = lane; x0 < a.Hkv * CH; x0 += 128) {
    uint4 kv4[4], vv4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = x0 + 32 * i;
      if (x < a.Hkv * CH) {
        kv4[i] = ks[x];
        vv4[i] = vs[x];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = x0 + 32 * i;
      if (x < a.Hkv * CH) {
        const int64_t o = ((page * a.Hkv + x / CH) * a.kv.page_size + row) * CH + x % CH;
        kd[o] = kv4[i];
        vd[o] = vv4[i];
      }
    }
  }
}

}  // namespace bitnet
