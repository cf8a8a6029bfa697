// A tree of drafted tokens: who attends whom, and the walk and commit of what is accepted.
//
// vg_tree_build.  A node's ancestors are its parent's and itself: thread i of a sequence's CTA walks
// up from node i through the parents in shared memory, setting bits and counting steps.  parent[i] < i
// makes every walk end; parents that break this are taken as -1 when they are staged.  What bounds
// it is latency: a launch, one round of loads, and the deepest node's walk of some 30 cycles a step.
//
// vg_tree_accept.  Node i goes on from its parent iff its token is the one that the target continues the
// parent with; the lowest such child of a node is its next one (an atomic minimum in shared
// memory: of integers, so the order does not matter), and the accepted path is a list walk
// from node 0.  The move of the accepted rows: a path ascends, path[j] >= j, so that row j's new place
// is never the old place of a later one, and a thread that takes the same 16 bytes of every row, j
// ascending, loads before it overwrites.  Threads never meet: each has its own bytes of a layer's K
// or V.
//
// One launch for both: the CTAs of a sequence are a cluster, each walks for itself (a round of loads and
// some 30 cycles a node), and they meet once after reading the prefix length, before the first of
// them may advance it.  What bounds it is the rows' bytes for many layers, else latency.
#include "tree_step.h"
#include "vg_common.cuh"
#include "vg_internal.h"

namespace vg {
namespace {

constexpr int kMaxNodes = VG_TREE_MAX_NODES;
static_assert(kMaxNodes % 64 == 0, "");

// Nodes of sequence b (reported and none, if out of range).
__device__ __forceinline__ int tree_nodes(const int32_t* len, int b, int n_nodes, int32_t* status) {
  if (!len) return n_nodes;
  const int n = len[b];
  if (n >= 0 && n <= n_nodes) return n;
  if (threadIdx.x == 0) report(status, VG_ERR_DEVICE_BOUNDS);
  return 0;
}

// The parent of node i, -1 (and reported) where it is none that a walk could follow.
__device__ __forceinline__ int tree_parent(int p, int i, int32_t* status) {
  if (p >= -1 && p < i) return p;
  report(status, VG_ERR_DEVICE_BOUNDS);
  return -1;
}

__global__ void __launch_bounds__(kMaxNodes) tree_build_kernel(const TreeBuildParams p) {
  __shared__ int up[kMaxNodes];
  const int b = blockIdx.x, i = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int n = tree_nodes(p.len, b, p.n_nodes, p.status);
  const int pre = p.prefix_len ? p.prefix_len[b] : 0;
  if (i < n) up[i] = tree_parent(p.parent[b * p.parent_stride + i], i, p.status);
  __syncthreads();
  if (i >= n) return;
  uint64_t sees[kMaxNodes / 64] = {};
  int depth = -1;
  for (int j = i; j >= 0; j = up[j]) {
    ++depth;
#pragma unroll
    for (int w = 0; w < kMaxNodes / 64; ++w)
      if (j >> 6 == w) sees[w] |= uint64_t{1} << (j & 63);
  }
  const size_t row = static_cast<size_t>(b) * p.n_nodes + i;
  if (p.position) p.position[row] = static_cast<int32_t>(static_cast<uint32_t>(pre) + static_cast<uint32_t>(depth));
  if (p.visible) {
    const int words = (p.n_nodes + 63) >> 6;
#pragma unroll
    for (int w = 0; w < kMaxNodes / 64; ++w)
      if (w < words) p.visible[row * words + w] = sees[w];
  }
}

// Threads of a CTA of the acceptance, and the rows it has on the way (a thread's 16 bytes of each).
constexpr int kAcceptThreads = 512;
constexpr int kMoveBatch = 8;
constexpr int kAcceptCluster = 8;  // most CTAs of a sequence

__global__ void __launch_bounds__(kAcceptThreads) tree_accept_kernel(const TreeAcceptParams p, const PageLayers layers) {
  __shared__ int up[kMaxNodes], tgt[kMaxNodes], next[kMaxNodes], path[kMaxNodes];
  __shared__ int64_t from[kMaxNodes], to[kMaxNodes];
  __shared__ int count;
  const int b = blockIdx.y, part = blockIdx.x, parts = gridDim.x, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int n = tree_nodes(p.len, b, p.n_nodes, p.status);
  const int pre = p.prefix_len[b];
  const bool room = pre >= 0 && pre <= p.max_len && pre <= 0x7fffffff - kMaxNodes;  // (kv_slot's positions have 31 bits)
  const size_t row0 = static_cast<size_t>(b) * p.n_nodes;
  int token = 0;
  if (tid < n) {
    int x = tree_parent(p.parent[b * p.parent_stride + tid], tid, p.status);
    up[tid] = x;
    tgt[tid] = p.target[row0 + tid];
    token = p.draft[row0 + tid];
  }
  if (tid < kMaxNodes) next[tid] = kMaxNodes;
  __syncthreads();
  // (a row without any token draws -1, drafts' rows and the target's: no token that both have)
  if (tid < n && up[tid] >= 0 && token >= 0 && token == tgt[up[tid]]) atomicMin(&next[up[tid]], tid);
  __syncthreads();
  if (tid == 0) {
    int a = 0;
    for (int cur = 0; cur < n; cur = next[cur]) path[a++] = cur;
    count = a;  // nodes of the path, node 0 among them
  }
  __syncthreads();
  const int a = count;
  // Every CTA of the cluster has read the prefix length: it may be advanced.
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (part == 0) {
    if (tid < p.n_nodes) p.path[row0 + tid] = tid < a ? path[tid] : -1;
    if (tid == 0) {
      if (!room) report(p.status, VG_ERR_DEVICE_BOUNDS);
      p.n_accept[b] = max(a - 1, 0);
      p.next_token[b] = a ? tgt[path[a - 1]] : -1;
      if (p.advance_len && room) p.advance_len[b] += a;
    }
  }
  if (!room || a < 2 || p.n_tensors == 0) return;
  if (tid < a) {
    from[tid] = kv_slot(p.seq_offset, p.ptab, p.psize, p.pstride, p.capacity, b, static_cast<int64_t>(pre) + path[tid]);
    to[tid] = kv_slot(p.seq_offset, p.ptab, p.psize, p.pstride, p.capacity, b, static_cast<int64_t>(pre) + tid);
    if (from[tid] < 0 || to[tid] < 0) {
      if (path[tid] != tid) report(p.status, VG_ERR_DEVICE_BOUNDS);
      from[tid] = to[tid] = 0;
    }
  }
  __syncthreads();
  const int units = p.token_bytes / 16;  // of a row
  for (int e = part * kAcceptThreads + tid; e < p.n_tensors * units; e += parts * kAcceptThreads) {
    const int t = e / units, u = e - t * units;
    uint4* base = reinterpret_cast<uint4*>(layers.base[t]) + u;
    for (int j0 = 1; j0 < a; j0 += kMoveBatch) {
      uint4 v[kMoveBatch];
#pragma unroll
      for (int k = 0; k < kMoveBatch; ++k)
        if (j0 + k < a && from[j0 + k] != to[j0 + k]) v[k] = base[from[j0 + k] * units];
#pragma unroll
      for (int k = 0; k < kMoveBatch; ++k)
        if (j0 + k < a && from[j0 + k] != to[j0 + k]) base[to[j0 + k] * units] = v[k];
    }
  }
}

}  // namespace

cudaError_t launch_tree_build(const TreeBuildParams& p, cudaStream_t stream) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B);
  cfg.blockDim = dim3((p.n_nodes + 31) / 32 * 32);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_build_kernel, p);
}

cudaError_t launch_tree_accept(const TreeAcceptParams& p, const PageLayers& layers, cudaStream_t stream) {
  const int64_t work = static_cast<int64_t>(p.n_tensors) * (p.token_bytes / 16);
  int parts = 1;
  while (parts < kAcceptCluster && parts * kAcceptThreads < work) parts *= 2;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = parts;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts, p.B);
  cfg.blockDim = dim3(kAcceptThreads);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_accept_kernel, p, layers);
}

}  // namespace vg
