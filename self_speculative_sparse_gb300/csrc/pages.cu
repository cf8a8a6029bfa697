// The page pool of a paged cache: rows of the block table grown, cut, forked and freed, and
// live pages moved down to the front of the pool.
//
// The state is three integer arrays on the device: the block table, the pages each row
// holds, and a reference count per page (0: free).  A request never waits for the host:
// one cluster of CTAs gives pages back, counts what is free, and hands out the lowest free
// pages to the requests in order, so a result depends on the state and the request alone
// (counts are added to atomically, but sums of integers do not depend on the order).
// What has to be read is the reference counts (4 bytes a page) and the rows that a request
// names; the rest is latency: the phases are separated by cluster barriers, and the cluster
// grows with the pool (one CTA up to kPagesPerCta pages), since a barrier of one CTA is
// several times cheaper than one of sixteen.
//
// Page contents move in a second kernel, launched as a programmatic dependent over all SMs,
// from a list of (source page, destination page, tokens) that the first one leaves: reads
// and writes of whole 16-byte vectors, bound by memory (8 layers of 1024 pages with holes, 1.05 GB:
// 166 us, 6.3 TB/s; 64 forks over 16 layers, 208 MB: 34 us, 6.1 TB/s).  Sources and destinations are
// disjoint (destinations were free), so the copies need no order.
#include <cooperative_groups.h>

#include <climits>

#include "vg_common.cuh"
#include "vg_internal.h"

namespace vg {
namespace {

namespace cg = cooperative_groups;

constexpr int kPageThreads = 1024;
constexpr int kPageMaxCluster = 16;
constexpr int kPagesPerCta = 8192;
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = 16384;  // bytes of one copy item
constexpr int kShareChunk = 1024;  // table entries of one share item

// Exclusive scan over the CTA's threads; *total gets the sum.  All threads.
__device__ __forceinline__ int block_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += t;
  }
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = lane < kPageThreads / 32 ? sh[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += t;
    }
    sh[lane] = y;
  }
  __syncthreads();
  const int base = warp > 0 ? sh[warp - 1] : 0;
  *total = sh[kPageThreads / 32 - 1];
  __syncthreads();
  return base + x - v;
}

// This thread's contiguous run of pages [lo, hi): the pool is cut into equal runs, a
// multiple of four pages each.
__device__ __forceinline__ void page_run(int n_pages, int rank, int nctas, int& lo, int& hi) {
  const int threads = nctas * kPageThreads;
  const int per = ((n_pages + threads - 1) / threads + 3) & ~3;
  const int64_t at = static_cast<int64_t>(rank * kPageThreads + threadIdx.x) * per;
  lo = static_cast<int>(at < n_pages ? at : n_pages);
  hi = static_cast<int>(at + per < n_pages ? at + per : n_pages);
}

// Pages of the run that are free (other CTAs' counts come through L2).
__device__ __forceinline__ int count_free(const int32_t* refs, int lo, int hi) {
  int n = 0;
  int i = lo;
  for (; i + 4 <= hi; i += 4) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(refs + i));
    n += (v.x <= 0) + (v.y <= 0) + (v.z <= 0) + (v.w <= 0);
  }
  for (; i < hi; ++i) n += __ldcg(refs + i) <= 0;
  return n;
}

struct ClusterShared {
  int sh[32];
  int counts[kPageMaxCluster];  // every CTA's count, pushed by its owner
};

// Cluster barriers, where a cluster of one CTA needs no more than its own (a request for
// 16 rows: 5.2 us, with the cluster's 6.2).
__device__ __forceinline__ void cluster_arrive(int C) {
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait(int C) {
  if (C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync(int C) {
  if (C > 1) cg::this_cluster().sync();
  else __syncthreads();
}

// Grow, cut or fork rows (one cluster).
__global__ void __launch_bounds__(kPageThreads) pages_request_kernel(const PagesParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), C = static_cast<int>(cluster.num_blocks());
  __shared__ ClusterShared s;
  const int tid = threadIdx.x, lane = tid & 31;
  const int gt = rank * kPageThreads + tid, GT = C * kPageThreads;  // thread of the cluster
  const int gw = gt >> 5, GW = GT >> 5;                             // warp of the cluster
  pdl_wait();
  // ---- which request names each row first (a row named twice: the later ones are refused)
  for (int j = gt; j < p.n; j += GT) {
    const int c = p.seq ? p.seq[j] : j;
    if (c >= 0 && c < p.n_seqs) p.owner[c] = INT_MAX;
    if (p.parent) {
      const int f = p.parent[j];
      if (f >= 0 && f < p.n_seqs) p.owner[f] = INT_MAX;
    }
  }
  cluster_sync(C);
  for (int j = gt; j < p.n; j += GT) {
    const int c = p.seq ? p.seq[j] : j;
    if (c >= 0 && c < p.n_seqs) atomicMin(p.owner + c, j);
  }
  cluster_sync(C);
  // ---- check each request, give back what its row no longer holds
  for (int j = gw; j < p.n; j += GW) {
    const int c = p.seq ? p.seq[j] : j;
    const int len = p.length[j];
    bool ok = c >= 0 && c < p.n_seqs && __ldcg(p.owner + c) == j && len >= 0;
    int total = 0, have = 0, held = 0;
    if (ok) {
      held = p.held[c];
      const int64_t want = (static_cast<int64_t>(len) + p.room + p.page_size - 1) / p.page_size;
      ok = held >= 0 && held <= p.pages_per_seq && want <= p.pages_per_seq;
      total = static_cast<int>(want);
    }
    if (ok && p.parent) {
      const int f = p.parent[j];
      ok = f >= 0 && f < p.n_seqs && __ldcg(p.owner + f) == INT_MAX;
      if (ok) {
        const int fh = p.held[f];
        ok = fh >= 0 && fh <= p.pages_per_seq && len <= static_cast<int64_t>(fh) * p.page_size;
      }
    }
    int keep = 0;
    if (ok) {
      if (p.parent) {
        have = len / p.page_size;  // whole pages shared with the parent
      } else {
        have = keep = min(held, total);
      }
      int32_t* row = p.table + static_cast<int64_t>(c) * p.pages_per_seq;
      for (int i = keep + lane; i < held; i += 32) {
        const int pg = row[i];
        if (pg >= 0 && pg < p.n_pages) atomicSub(p.refs + pg, 1);
        else report(p.status, VG_ERR_DEVICE_BOUNDS);
        row[i] = -1;
      }
    } else if (lane == 0) {
      report(p.status, VG_ERR_DEVICE_BOUNDS);
    }
    if (lane == 0) {
      p.need[j] = ok ? total - have : 0;
      p.have[j] = ok ? have : -1;
    }
  }
  cluster_sync(C);
  // ---- free pages of every CTA's share; each request's rank among the pages handed out
  int lo, hi, mine, run_free;
  page_run(p.n_pages, rank, C, lo, hi);
  run_free = count_free(p.refs, lo, hi);
  const int before = block_scan(run_free, s.sh, &mine);
  if (tid < C) *cluster.map_shared_rank(s.counts + rank, tid) = mine;
  if (rank == C - 1) {
    const int per = (p.n + kPageThreads - 1) / kPageThreads;
    const int a = min(tid * per, p.n), b = min(a + per, p.n);
    int sum = 0, all;
    for (int j = a; j < b; ++j) sum += __ldcg(p.need + j);
    int at = block_scan(sum, s.sh, &all);
    for (int j = a; j < b; ++j) {
      p.start[j] = at;
      at += __ldcg(p.need + j);
    }
    if (tid == 0) *p.needed = all;
  }
  cluster_sync(C);
  // ---- the lowest free pages, as many as are asked for
  int base = before, free_all = 0;
  for (int c = 0; c < C; ++c) {
    if (c < rank) base += s.counts[c];
    free_all += s.counts[c];
  }
  const int needed = __ldcg(p.needed);
  if (base < needed) {
    for (int i = lo; i < hi && base < needed; ++i)
      if (__ldcg(p.refs + i) <= 0) p.freelist[base++] = i;
  }
  cluster_sync(C);
  pdl_launch_dependents();
  // ---- fill the rows
  for (int j = gw; j < p.n; j += GW) {
    const int have = __ldcg(p.have + j);
    if (p.copies && lane == 0) p.copies[j] = make_int4(0, 0, 0, 0);
    if (have < 0) continue;
    const int c = p.seq ? p.seq[j] : j;
    const int need = __ldcg(p.need + j), start = __ldcg(p.start + j);
    int32_t* row = p.table + static_cast<int64_t>(c) * p.pages_per_seq;
    if (need > 0 && start + need > free_all) {  // the pool ran out at an earlier request or here
      if (lane == 0) {
        report(p.status, VG_ERR_DEVICE_PAGES);
        p.held[c] = p.parent ? 0 : have;
        if (p.parent) p.have[j] = -1;
      }
      continue;
    }
    if (p.parent) {
      const int part = p.length[j] % p.page_size;
      if (lane == 0 && part > 0) {
        const int src = p.table[static_cast<int64_t>(p.parent[j]) * p.pages_per_seq + have];
        const int dst = __ldcg(p.freelist + start);
        if (src >= 0 && src < p.n_pages)
          p.copies[j] = make_int4(src, dst, part, 0);
        else
          report(p.status, VG_ERR_DEVICE_BOUNDS);
      }
    }
    for (int i = lane; i < need; i += 32) {
      const int pg = __ldcg(p.freelist + start + i);
      row[have + i] = pg;
      p.refs[pg] = 1;
    }
    if (lane == 0) p.held[c] = have + need;
  }
}

// The same for up to kSmallRequests requests and a pool of kSmallPages: every CTA has what all the
// requests ask in its own shared memory, so that two cluster barriers are left, and nothing but the
// reference counts passes through global memory: (1) a thread a request checks it; a hash table
// finds the first request that names a row; (2) a warp a request gives back the pages that its
// row no longer holds; (3) every CTA counts the free pages of its share of the pool, kept as a
// mask in registers; (4) the thread of a free page finds the request whose page it becomes by
// its rank, and writes it there.  A request for 16 rows of a pool of 1024 pages takes 5.2 us so
// and 11 us with the kernel above; for 512 rows of 131072 pages 9 to 12 us and 16 to 17.  (256 threads for
// a small pool are no faster.)
constexpr int kSmallRequests = 1024;
constexpr int kSmallPages = kPageMaxCluster * kPageThreads * 32;
constexpr int kHash = 2048;
static_assert(kSmallRequests <= kPageThreads && 2 * kSmallRequests <= kHash && kHash == 1 << (32 - 21), "see slot_of");

__global__ void __launch_bounds__(kPageThreads) pages_request_small_kernel(const PagesParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), C = static_cast<int>(cluster.num_blocks());
  __shared__ ClusterShared s;
  __shared__ int hash_row[kHash], hash_first[kHash];
  __shared__ int child[kSmallRequests], have_of[kSmallRequests], start_of[kSmallRequests];
  __shared__ int2 give[kSmallRequests];  // entries of its row that a request gives back: first, end
  int* need_of = hash_row;               // (once the hash table has been read)
  const int tid = threadIdx.x, lane = tid & 31;
  const int gw = (rank * kPageThreads + tid) >> 5, GW = (C * kPageThreads) >> 5;
  for (int i = tid; i < kHash; i += kPageThreads) {
    hash_row[i] = -1;
    hash_first[i] = INT_MAX;
  }
  cluster_arrive(C);
  __syncthreads();
  pdl_wait();
  // ---- check the requests
  auto slot_of = [&](int row) { return static_cast<int>((static_cast<uint32_t>(row) * 2654435761u) >> 21); };
  int c = -1, f = -1, len = 0, held = 0, fh = 0;
  if (tid < p.n) {
    c = p.seq ? p.seq[tid] : tid;
    len = p.length[tid];
    f = p.parent ? p.parent[tid] : 0;
    if (c >= 0 && c < p.n_seqs) {
      held = p.held[c];
      int h = slot_of(c);
      for (;; h = (h + 1) & (kHash - 1)) {  // (at most half of the entries are taken)
        const int was = atomicCAS(&hash_row[h], -1, c);
        if (was == -1 || was == c) break;
      }
      atomicMin(&hash_first[h], tid);
    }
    if (p.parent && f >= 0 && f < p.n_seqs) fh = p.held[f];
  }
  __syncthreads();
  auto first_of = [&](int row) {  // the first request that names a row, INT_MAX: none
    for (int h = slot_of(row);; h = (h + 1) & (kHash - 1)) {
      if (hash_row[h] == row) return hash_first[h];
      if (hash_row[h] == -1) return INT_MAX;
    }
  };
  int need = 0, have = -1;
  if (tid < p.n) {
    const int64_t want = (static_cast<int64_t>(len) + p.room + p.page_size - 1) / p.page_size;
    bool ok = c >= 0 && c < p.n_seqs && len >= 0 && first_of(c) == tid && held >= 0 && held <= p.pages_per_seq &&
              want <= p.pages_per_seq;
    if (ok && p.parent)
      ok = f >= 0 && f < p.n_seqs && first_of(f) == INT_MAX && fh >= 0 && fh <= p.pages_per_seq &&
           len <= static_cast<int64_t>(fh) * p.page_size;
    if (ok) {
      have = p.parent ? len / p.page_size : min(held, static_cast<int>(want));  // whole pages shared, or kept
      need = static_cast<int>(want) - have;
    } else if (rank == 0) {
      report(p.status, VG_ERR_DEVICE_BOUNDS);
    }
    child[tid] = c;
    have_of[tid] = have;
    give[tid] = ok ? make_int2(p.parent ? 0 : have, held) : make_int2(0, 0);
  }
  __syncthreads();  // (the hash table has been read)
  if (tid < p.n) need_of[tid] = need;
  // ---- give back what the rows no longer hold
  for (int j = gw; j < p.n; j += GW) {
    const int2 range = give[j];
    if (range.x >= range.y) continue;
    int32_t* row = p.table + static_cast<int64_t>(child[j]) * p.pages_per_seq;
    for (int i0 = range.x + lane; i0 < range.y; i0 += 128) {
      int pg[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) pg[u] = i0 + 32 * u < range.y ? row[i0 + 32 * u] : -1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (i0 + 32 * u >= range.y) break;
        if (pg[u] >= 0 && pg[u] < p.n_pages) atomicSub(p.refs + pg[u], 1);
        else report(p.status, VG_ERR_DEVICE_BOUNDS);
        row[i0 + 32 * u] = -1;
      }
    }
  }
  cluster_wait(C);  // every CTA runs: its shared memory may be written
  cluster_sync(C);
  // ---- the free pages of every CTA's share (and, while the counts come, the requests' places among
  // the pages handed out)
  int lo, hi, mine, needed, start = 0;
  page_run(p.n_pages, rank, C, lo, hi);
  uint32_t mask = 0;  // free pages of this thread's run (32 at most)
  for (int i0 = lo;; i0 += 8) {  // (the run starts at a multiple of four)
    int4 v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int i = i0 + 4 * u;
      v[u] = make_int4(1, 1, 1, 1);
      if (i + 4 <= hi) {
        v[u] = __ldcg(reinterpret_cast<const int4*>(p.refs + i));
      } else {
        if (i < hi) v[u].x = __ldcg(p.refs + i);
        if (i + 1 < hi) v[u].y = __ldcg(p.refs + i + 1);
        if (i + 2 < hi) v[u].z = __ldcg(p.refs + i + 2);
      }
    }
    if (i0 == lo) {
      start = block_scan(need, s.sh, &needed);
      if (tid < p.n) start_of[tid] = start;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (i0 + 4 * u < hi)
        mask |= ((v[u].x <= 0 ? 1u : 0u) | (v[u].y <= 0 ? 2u : 0u) | (v[u].z <= 0 ? 4u : 0u) | (v[u].w <= 0 ? 8u : 0u))
                << (i0 + 4 * u - lo);
    if (i0 + 8 >= hi) break;
  }
  const int before = block_scan(__popc(mask), s.sh, &mine);
  if (tid < C) *cluster.map_shared_rank(s.counts + rank, tid) = mine;
  cluster_sync(C);
  pdl_launch_dependents();
  int base = before, free_all = 0;
  for (int r = 0; r < C; ++r) {
    if (r < rank) base += s.counts[r];
    free_all += s.counts[r];
  }
  // ---- the lowest free pages, in order, to the rows that get them.  The request of rank r is the
  // last one that starts at r or before (it asks for pages, as the one behind it would start there
  // too); the next page's is the same or one soon behind it
  int a = 0, first = 0, end = 0;
  int32_t* row = nullptr;
  for (; mask != 0 && base < needed; mask &= mask - 1, ++base) {
    const int pg = lo + __ffs(mask) - 1;
    if (row == nullptr) {
      for (int b = p.n - 1; a < b;) {
        const int mid = (a + b + 1) >> 1;
        if (start_of[mid] <= base) a = mid; else b = mid - 1;
      }
    }
    if (base >= end) {
      while ((end = (first = start_of[a]) + need_of[a]) <= base) ++a;
      row = p.table + static_cast<int64_t>(child[a]) * p.pages_per_seq + have_of[a];
    }
    if (end > free_all) continue;  // not served
    const int i = base - first;
    row[i] = pg;
    p.refs[pg] = 1;
    if (i == 0 && p.copies) {
      const int part = p.length[a] % p.page_size;
      if (part > 0) {
        const int src = p.table[static_cast<int64_t>(p.parent[a]) * p.pages_per_seq + have_of[a]];
        const bool good = src >= 0 && src < p.n_pages;
        p.copies[a] = good ? make_int4(src, pg, part, 0) : make_int4(0, 0, 0, 0);
        if (!good) report(p.status, VG_ERR_DEVICE_BOUNDS);
      }
    }
  }
  // ---- what the rows hold
  if (rank == C - 1 && tid < p.n) {
    const bool served = need == 0 || start + need <= free_all;
    if (p.copies) {
      if (have < 0 || !served || need == 0 || len % p.page_size == 0) p.copies[tid] = make_int4(0, 0, 0, 0);
      p.have[tid] = served ? have : -1;
    }
    if (have >= 0) {
      if (!served) report(p.status, VG_ERR_DEVICE_PAGES);
      p.held[c] = served ? have + need : (p.parent ? 0 : have);
    }
  }
}

// Live pages past the count of live pages take the free ones below it, in order.
__global__ void __launch_bounds__(kPageThreads) pages_compact_kernel(const PagesParams p) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank()), C = static_cast<int>(cluster.num_blocks());
  __shared__ ClusterShared s;
  const int tid = threadIdx.x;
  const int gt = rank * kPageThreads + tid, GT = C * kPageThreads;
  cluster_arrive(C);
  pdl_wait();
  int lo, hi, mine;
  page_run(p.n_pages, rank, C, lo, hi);
  const int run_free = count_free(p.refs, lo, hi);
  const int before = block_scan(run_free, s.sh, &mine);
  cluster_wait(C);  // every CTA runs: its shared memory may be written
  if (tid < C) *cluster.map_shared_rank(s.counts + rank, tid) = mine;
  cluster_sync(C);
  int free_before = before, free_all = 0;  // free pages before this run, in all
  for (int c = 0; c < C; ++c) {
    if (c < rank) free_before += s.counts[c];
    free_all += s.counts[c];
  }
  const int n_live = p.n_pages - free_all;
  // holes (free pages below n_live) in ascending order; movers (live pages from n_live on)
  // counted from the last one, which needs no count of the holes
  int f = free_before;
  for (int i = lo; i < hi; ++i) {
    const int r = p.refs[i];
    if (i == n_live) *p.needed = f;  // holes, and so movers
    if (r <= 0) {
      if (i < n_live) {
        p.freelist[f] = i;
      } else {
        p.refs_out[i] = 0;
        p.moved_to[i] = -1;
      }
      ++f;
    } else if (i >= n_live) {
      p.movers[n_live - 1 - (i - f)] = i;
    } else {
      p.refs_out[i] = r;
    }
  }
  if (n_live == p.n_pages && gt == 0) *p.needed = 0;  // (no page at index n_live)
  if (gt == 0) *p.n_live = n_live;
  cluster_sync(C);
  const int moves = __ldcg(p.needed);
  pdl_launch_dependents();
  for (int r = gt; r < moves; r += GT) {
    const int hole = __ldcg(p.freelist + r), from = __ldcg(p.movers + moves - 1 - r);
    p.moved_to[from] = hole;
    const int refs = p.refs[from];
    p.refs_out[hole] = refs;
    p.refs_out[from] = 0;
  }
}

__host__ __device__ __forceinline__ int share_chunks(const PagesParams& p) {
  return (p.pages_per_seq + kShareChunk - 1) / kShareChunk;
}

// One 16 KB piece of a page's tokens.
__device__ __forceinline__ void copy_piece(const char* src, char* dst, int bytes) {
  constexpr int U = kCopyBytes / (16 * kCopyThreads);  // vectors a thread
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = (u * kCopyThreads + threadIdx.x) * 16;
    if (at < bytes) v[u] = *reinterpret_cast<const uint4*>(src + at);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = (u * kCopyThreads + threadIdx.x) * 16;
    if (at < bytes) *reinterpret_cast<uint4*>(dst + at) = v[u];
  }
}

// Page contents of a fork (list of p.n) or a compaction (list of *p.needed, whole pages),
// over every layer's K and V.  After a fork also the whole pages that a row shares with its parent
// (here, over all SMs, rather than by the one cluster before: 64 forks at 100 to 2000
// tokens, pages of 64, took that 3 us longer); after a compaction also the rows of the table.
template <bool COMPACT>
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const PagesParams p, const PageLayers layers) {
  pdl_wait();
  const int64_t page_bytes = static_cast<int64_t>(p.page_size) * p.token_bytes;
  const int pieces = static_cast<int>((page_bytes + kCopyBytes - 1) / kCopyBytes);
  const int n = COMPACT ? *p.needed : p.n;
  const int64_t work = static_cast<int64_t>(n) * 2 * p.n_layers * pieces;
  if constexpr (!COMPACT) {
    const int chunks = share_chunks(p);
    const int64_t shares = static_cast<int64_t>(n) * chunks;
    for (int64_t w = blockIdx.x; w < shares; w += gridDim.x) {
      const int j = static_cast<int>(w / chunks), i0 = static_cast<int>(w - static_cast<int64_t>(j) * chunks) * kShareChunk;
      const int have = p.have[j];
      if (i0 >= have) continue;  // (refused: -1)
      const int32_t* from = p.table + static_cast<int64_t>(p.parent[j]) * p.pages_per_seq;
      int32_t* row = p.table + static_cast<int64_t>(p.seq[j]) * p.pages_per_seq;
      constexpr int U = kShareChunk / kCopyThreads;
      int pg[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kCopyThreads + threadIdx.x;
        if (i < have) pg[u] = from[i];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * kCopyThreads + threadIdx.x;
        if (i >= have) continue;
        row[i] = pg[u];
        if (pg[u] >= 0 && pg[u] < p.n_pages) atomicAdd(p.refs + pg[u], 1);
        else report(p.status, VG_ERR_DEVICE_BOUNDS);
      }
    }
  }
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int64_t j = w / pieces;
    const int piece = static_cast<int>(w - j * pieces);
    const int lk = static_cast<int>(j % (2 * p.n_layers)), m = static_cast<int>(j / (2 * p.n_layers));
    int src, dst;
    int64_t bytes;
    if constexpr (COMPACT) {
      src = p.movers[n - 1 - m];
      dst = p.freelist[m];
      bytes = page_bytes;
    } else {
      const int4 c = p.copies[m];
      src = c.x;
      dst = c.y;
      bytes = static_cast<int64_t>(c.z) * p.token_bytes;
    }
    const int64_t at = static_cast<int64_t>(piece) * kCopyBytes;
    if (at >= bytes) continue;
    char* base = static_cast<char*>(layers.base[lk]);
    copy_piece(base + src * page_bytes + at, base + dst * page_bytes + at,
               static_cast<int>(bytes - at < kCopyBytes ? bytes - at : kCopyBytes));
  }
  if constexpr (COMPACT) {
    const int n_live = *p.n_live;
    const int64_t entries = static_cast<int64_t>(p.n_seqs) * p.pages_per_seq;
    for (int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries;
         e += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
      const int s = static_cast<int>(e / p.pages_per_seq), i = static_cast<int>(e - static_cast<int64_t>(s) * p.pages_per_seq);
      int pg = p.table[e];
      if (i < p.held[s]) {
        if (pg < 0 || pg >= p.n_pages)
          report(p.status, VG_ERR_DEVICE_BOUNDS);
        else if (pg >= n_live) {
          const int to = p.moved_to[pg];
          if (to >= 0) pg = to;
          else report(p.status, VG_ERR_DEVICE_BOUNDS);  // a row holds a page that nothing counts
        }
      }
      p.table_out[e] = pg;
    }
  }
}

template <typename K>
cudaError_t launch_cluster(K* kernel, const PagesParams& p, cudaStream_t stream) {
  int C = (p.n_pages + kPagesPerCta - 1) / kPagesPerCta;
  C = C < 1 ? 1 : (C > kPageMaxCluster ? kPageMaxCluster : C);
  cudaError_t e;
  if (C > 8 && (e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kPageThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool COMPACT>
cudaError_t launch_copy(const PagesParams& p, const PageLayers& layers, int64_t most, int sms, cudaStream_t stream) {
  const int64_t cap = 8 * static_cast<int64_t>(sms);
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(most < 1 ? 1 : (most < cap ? most : cap)));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_copy_kernel<COMPACT>, p, layers);
}

int64_t page_pieces(const PagesParams& p) {
  return (static_cast<int64_t>(p.page_size) * p.token_bytes + kCopyBytes - 1) / kCopyBytes * 2 * p.n_layers;
}

}  // namespace

cudaError_t launch_pages_request(const PagesParams& p, const PageLayers& layers, int sms, cudaStream_t stream) {
  const bool small = p.n <= kSmallRequests && p.n_pages <= kSmallPages;
  const cudaError_t e = launch_cluster(small ? pages_request_small_kernel : pages_request_kernel, p, stream);
  if (e != cudaSuccess || !p.copies) return e;
  const int64_t pieces = p.n * page_pieces(p), shares = static_cast<int64_t>(p.n) * share_chunks(p);
  return launch_copy<false>(p, layers, pieces > shares ? pieces : shares, sms, stream);
}

cudaError_t launch_pages_compact(const PagesParams& p, const PageLayers& layers, int sms, cudaStream_t stream) {
  const cudaError_t e = launch_cluster(pages_compact_kernel, p, stream);
  if (e != cudaSuccess) return e;
  const int64_t pieces = static_cast<int64_t>(p.n_pages / 2) * page_pieces(p);
  const int64_t rows = (static_cast<int64_t>(p.n_seqs) * p.pages_per_seq + kCopyThreads - 1) / kCopyThreads;
  return launch_copy<true>(p, layers, pieces > rows ? pieces : rows, sms, stream);
}

}  // namespace vg
