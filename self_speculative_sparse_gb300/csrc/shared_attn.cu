// Verification attention for a batch whose groups share a prefix.
//
// The rows of all members of a group read the group's shared tokens once: per KV head they
// form one tall matrix of members * (gamma + 1) * G query rows, cut into tiles of 128, and a
// tile of 128 keys serves a whole tile of rows in one tensor-core product.  The tokens that
// only one sequence has (past the shared prefix) are a second, smaller problem of the same
// shape with that sequence's rows.  A softmax over a union of key sets is the merge of the
// sets' (max, sum, output), so both leave unnormalised partials, and a combine kernel merges
// them with the verify rows' own causal keys.
//
// The shared range is used in whole key tiles: what a shared prefix has past a multiple of
// 128 tokens is read as private tokens (every sequence's own row of the block table names
// them), so the tall problem needs no mask at all.
//
// Attention kernel.  One persistent CTA per SM; the flattened list of steps is split evenly
// over the CTAs.  A CTA has two "lanes" of eight softmax warps, each with its own 128 rows, S / P
// and O in tensor memory; a step is one key tile for both lanes:
//   pair   the lanes are two row tiles of one KV head and share the step's K and V tile;
//   heads  the lanes are the same row tile of two KV heads, each with its own K and V tile
//          (a group's odd last row tile, and every private range).
// While one lane's warps run the softmax of their tile, the tensor cores work for the other
// (P V of its tile, then Q K^T of its next): the lanes' issuers take turns.  P goes back to tensor
// memory as bf16, over the columns of S, and is the A operand of P V from there: it never passes
// shared memory.  The rows' sums are of the rounded P, so that weights sum to one and the rounding
// moves an output by at most 2^-8 of sum p |v - out|.  A second product with what the rounding drops
// lengthens a step by 1024 of its 2750 cycles: only ranges of few keys have it (kLowKeys).
// Warps: 0-7 and 8-15 the lanes (two threads a row), 16 and 18 the TMA producers, 17 and 19
// the lanes' MMA issuers; 16 also plans the CTA's runs.
//
// What bounds it: 2048 cycles of tensor-core work a step of two lanes with d = 128, or 128 KB of
// keys and values a step in heads mode.  In the middle of a run a pair step takes 2750 cycles,
// about the rate at which a plain bf16 product runs on this card; a run's start and end (the first
// tile's latency, the first maximum, partials of 64 KB a lane) cost it another 8000.  64 sequences of
// 8 rows and 32 heads over 16384 shared and 100 to 1000 private tokens take it 115 us (140 GFLOP:
// 1.22 PFLOP/s, 64% of a plain product's rate); 16 of one row over 32768 tokens 38 us
// (134 MB of shared keys and values: 3.5 TB/s; the first tile is there after 18000 of 69000 cycles).
#include "vg_common.cuh"
#include "vg_internal.h"

namespace vg {
namespace {

constexpr int KT = kSharedTileKeys;  // keys of a tile, and rows of a lane
static_assert(KT == 128, "a lane's rows and a tile's keys are the 128 tensor-memory lanes");
// A row's running max is raised only when the P of one half of a tile, 64 keys, sum to more than this:
// P stays below 2^8 and O is rescaled rarely.  (The sum is needed anyway: 64 sequences over 16384 shared
// tokens take 166 us a call so, and 172 with a maximum of every half tile of S beside it.)
constexpr float kMostSum = 256.f;
constexpr int kMaxSlots = 12;  // ring slots (K or V tiles) at most
// A private range of a sequence with at most this many prefix tokens, and a shared range of at most
// as many, carry P as a bf16 high part plus a bf16 low part (exact to 2^-17), as vg_verify_attn does:
// with so few keys, rows whose weight sits on two or three of them are likely, and there the rounding of P
// to one bf16 can pass the output's own.  (The smallest call, two sequences of 512 tokens: 17.3 us, 15.5
// with P in one part.)
constexpr int kLowKeys = 1024;

// ---------------------------------------------------------------- the batch's layout
// Everything the kernels need about lengths and groups, in the workspace: built from the
// device arrays by one CTA of a first small kernel, copied to shared memory by the others (built by
// every attention CTA for itself, in place of that kernel, it takes the CTAs 6 us).  An item is one unit
// of rows (a pair of row tiles of a KV head, or one row tile of two KV heads) and its whole key range.
// Its steps are its key tiles and, before them, kItemSteps more for what filling a run's pipeline and
// writing its partials costs a CTA; the attention CTAs split the steps of all items evenly, the shared
// ones first.  (Attention kernel with 1, 2, 3 and 4 such steps, measured when it summed unrounded weights
// and was 2% faster: 131, 117, 110 and 115 us for 64 sequences
// of 16384 shared and 100 to 1000 private tokens, 55, 57, 57 and 58 for eight of 20011 in three groups,
// 38 for 16 of 32768 with each.)
constexpr int kItemSteps = kSharedItemSteps;

struct Meta {
  int* gs;     // [ng + 1] first sequence of a group
  int* eff;    // [ng + 1] tokens of a group read once (a multiple of 128)
  int* stepS;  // [ng + 1] attention steps before a group
  int* itemS;  // [ng + 1] items before a group
  int* scS;    // [ng + 1] score items before a group
  int* nlen;   // [B] checked prefix length, -1: out of range
  int* grp;    // [B] group of a sequence
  int* stepP;  // [B + 1] attention steps of private ranges before a sequence
  int* scP;    // [B + 1] score items of private ranges before a sequence
};

// What the combine kernel needs of a sequence, in one load; the record after the last sequence's
// has the totals.
struct __align__(16) SeqRec {
  int n, eff;         // checked length; tokens read once for its group
  int row0, pairs;    // its first query row among the group's; row-tile pairs of the group
  int stepS, itemS;   // shared steps and items before its group
  int stepP, pad;     // private steps before it
};

__host__ __device__ inline int meta_ints(int B, int ng) { return 5 * (ng + 1) + 2 * B + 2 * (B + 1); }

__device__ __forceinline__ Meta meta_at(int* base, int B, int ng) {
  Meta m;
  m.gs = base;
  m.eff = m.gs + ng + 1;
  m.stepS = m.eff + ng + 1;
  m.itemS = m.stepS + ng + 1;
  m.scS = m.itemS + ng + 1;
  m.nlen = m.scS + ng + 1;
  m.grp = m.nlen + B;
  m.stepP = m.grp + B;
  m.scP = m.stepP + B + 1;
  return m;
}

// Row tiles of a group's KV head: `pairs` pairs of them, and whether one is left over.
__device__ __forceinline__ void row_tiles(int members, const SharedParams& p, int& pairs, int& odd) {
  const int rt = (members * p.M + p.RT - 1) / p.RT;
  pairs = rt >> 1;
  odd = rt & 1;
}

// Exclusive scans of N values over a CTA of WARPS warps, and their totals.  All threads; sh is
// not used again before the next barrier.
template <int N, int WARPS>
__device__ __forceinline__ void cta_scan(const int (&v)[N], int (&before)[N], int (&total)[N], int (*sh)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    x[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] += t;
    }
    if (lane == 31) sh[k][warp] = x[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {  // (every warp scans the warps' totals for itself)
    const int mine = lane < WARPS ? sh[k][lane] : 0;
    int y = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += t;
    }
    total[k] = __shfl_sync(0xffffffffu, y, 31);
    before[k] = __shfl_sync(0xffffffffu, y - mine, warp) + x[k] - v[k];
  }
}

// Last index i in [0, n) with cum[i] <= x, skipping empty entries (cum[i] == cum[i + 1]).
__device__ __forceinline__ int find(const int* cum, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The layout, by a CTA of WARPS warps (all threads).  A length out of range makes its sequence's
// nlen -1, groups that do not partition the batch or a shared length beyond a member's prefix
// make the sequences' ranges private; the caller reports what is returned as false.
template <int WARPS>
__device__ bool build_layout(const SharedParams& p, const Meta& m, int (*sh)[32]) {
  constexpr int NT = WARPS * 32, PER = (kMaxBatch + NT - 1) / NT;
  const int tid = threadIdx.x, B = p.B, ng = p.n_groups, Hp = (p.Hkv + 1) / 2;
  bool good = true;
  // (asked for together with the lengths)
  const int start0 = p.group_start && tid <= ng ? p.group_start[tid] : 0, shared0 = tid < ng ? p.shared_len[tid] : 0;
  for (int b = tid; b < B; b += NT) {
    int n = p.prefix_len[b];
    bool ok = n >= 0 && n <= p.max_len;
    if (ok) {
      if (p.ptab) {
        ok = static_cast<int64_t>(n) + p.R <= static_cast<int64_t>(p.pstride) * p.psize;
      } else {
        const int64_t off = p.seq_offset[b];
        ok = off >= 0 && off + static_cast<int64_t>(n) + p.R <= p.capacity;
      }
    }
    good &= ok;
    m.nlen[b] = ok ? n : -1;
    m.grp[b] = 0;
  }
  int* least = m.stepS;   // (until the scan) the shortest member
  int* shared = m.itemS;  // (until the scan) the shared length asked for
  for (int g = tid; g <= ng; g += NT) {
    m.gs[g] = !p.group_start ? (g ? B : 0) : g == tid ? start0 : p.group_start[g];
    if (g < ng) {
      shared[g] = g == tid ? shared0 : p.shared_len[g];
      least[g] = 0x7fffffff;
    }
  }
  __syncthreads();
  bool shape = true;
  for (int g = tid; g < ng; g += NT) shape &= m.gs[g] >= 0 && m.gs[g] <= m.gs[g + 1] && m.gs[g + 1] <= B;
  if (tid == 0) shape &= m.gs[0] == 0 && m.gs[ng] == B;
  shape = __syncthreads_and(shape);
  good &= shape;
  if (shape) {
    for (int b = tid; b < B; b += NT) {
      const int g = find(m.gs, ng, b);
      m.grp[b] = g;
      if (m.nlen[b] >= 0) atomicMin(&least[g], m.nlen[b]);
    }
  }
  __syncthreads();
  int steps[PER], items[PER], sc[PER], eff[PER], sum[3] = {0, 0, 0};
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int g = tid * PER + k;
    steps[k] = items[k] = sc[k] = eff[k] = 0;
    if (g < ng && shape && m.gs[g] < m.gs[g + 1]) {
      const int members = m.gs[g + 1] - m.gs[g];
      int len = shared[g];
      if (m.nlen[m.gs[g]] < 0) {
        len = 0;  // no row to read the prefix through
      } else if (len < 0 || len > least[g]) {
        good = false;
        len = 0;
      }
      eff[k] = len / KT * KT;
      int pairs, odd;
      row_tiles(members, p, pairs, odd);
      const int tiles = eff[k] / KT;
      items[k] = tiles ? p.Hkv * pairs + odd * Hp : 0;
      steps[k] = items[k] * (tiles + kItemSteps);
      sc[k] = tiles * ((members + p.nsc - 1) / p.nsc);
    }
    sum[0] += steps[k];
    sum[1] += items[k];
    sum[2] += sc[k];
  }
  int at[3], tot[3];
  cta_scan<3, WARPS>(sum, at, tot, sh);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int g = tid * PER + k;
    if (g < ng) {
      m.eff[g] = eff[k];
      m.stepS[g] = at[0];
      m.itemS[g] = at[1];
      m.scS[g] = at[2];
    }
    at[0] += steps[k];
    at[1] += items[k];
    at[2] += sc[k];
  }
  if (tid == 0) {
    m.eff[ng] = 0;
    m.stepS[ng] = tot[0];
    m.itemS[ng] = tot[1];
    m.scS[ng] = tot[2];
  }
  __syncthreads();
  int tiles[PER], sum2[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int b = tid * PER + k;
    tiles[k] = b < B && m.nlen[b] >= 0 ? (m.nlen[b] - m.eff[m.grp[b]] + KT - 1) / KT : 0;
    sum2[0] += tiles[k] > 0 ? (tiles[k] + kItemSteps) * Hp : 0;
    sum2[1] += tiles[k];
  }
  int at2[2], tot2[2];
  cta_scan<2, WARPS>(sum2, at2, tot2, sh);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int b = tid * PER + k;
    if (b < B) {
      m.stepP[b] = at2[0];
      m.scP[b] = at2[1];
    }
    at2[0] += tiles[k] > 0 ? (tiles[k] + kItemSteps) * Hp : 0;
    at2[1] += tiles[k];
  }
  if (tid == 0) {
    m.stepP[B] = tot2[0];
    m.scP[B] = tot2[1];
  }
  __syncthreads();
  return good;
}

// The first kernel of a call.  CTA 0: the layout.  The others (with scores), one a sequence: the sum
// of its masked query rows of each KV head, in fp32, as three bf16 parts whose sum is it to 2^-24.
// 512 threads: 6.0 to 6.7 us with 16 sequences by itself, most of it the launch and a dozen dependent
// steps (1024 threads take 0.7 us more, 128 with scores 3 us more).
constexpr int kPrepThreads = 512;
__global__ void __launch_bounds__(kPrepThreads) shared_prep_kernel(const SharedParams p) {
  __shared__ int space[5 * (kMaxBatch + 1) + 2 * kMaxBatch + 2 * (kMaxBatch + 1)], sh[3][32];
  pdl_launch_dependents();
  pdl_wait();
  if (blockIdx.x > 0) {
    const int b = blockIdx.x - 1, width = p.Hkv * p.D;
    const size_t part = static_cast<size_t>(p.Bpad) * width;
    for (int e = threadIdx.x; e < width; e += kPrepThreads) {
      const int g = e / p.D, d = e - g * p.D;
      float acc = 0.f;
      for (uint32_t bits = p.mask; bits != 0u; bits &= bits - 1u) {
        const int t = __ffs(bits) - 1;
        const __nv_bfloat16* src = p.q + ((static_cast<size_t>(b) * p.R + t) * p.Hq + g * p.G) * p.D + d;
#pragma unroll 4
        for (int h = 0; h < p.G; ++h) acc += __bfloat162float(src[h * p.D]);
      }
      __nv_bfloat16* dst = p.qsum + static_cast<size_t>(b) * width + e;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const __nv_bfloat16 h = __float2bfloat16_rn(acc);
        dst[k * part] = h;
        acc -= __bfloat162float(h);
      }
    }
    return;
  }
  const Meta m = meta_at(space, p.B, p.n_groups);
  if (!build_layout<kPrepThreads / 32>(p, m, sh)) report(p.status, VG_ERR_DEVICE_BOUNDS);
  for (int i = threadIdx.x; i < meta_ints(p.B, p.n_groups); i += kPrepThreads) p.meta[i] = space[i];
  SeqRec* rec = reinterpret_cast<SeqRec*>(p.rec);
  for (int b = threadIdx.x; b <= p.B; b += kPrepThreads) {
    if (b == p.B) {
      rec[b] = SeqRec{0, 0, 0, 0, m.stepS[p.n_groups], m.itemS[p.n_groups], m.stepP[p.B], 0};
    } else {
      const int g = m.grp[b];
      int pairs, odd;
      row_tiles(m.gs[g + 1] - m.gs[g], p, pairs, odd);
      rec[b] = SeqRec{m.nlen[b], m.eff[g], (b - m.gs[g]) * p.M, pairs, m.stepS[g], m.itemS[g], m.stepP[b], 0};
    }
  }
}

// A contiguous run of key tiles of one item, as one CTA works on it.
enum RunMode { kPair, kHeads, kSingle };
struct Run {
  int mode;
  int tile0, ntiles;  // key tiles of the item's range
  int row;            // the unit's first sequence, whose tokens locate the keys
  int tok0, ntok;     // first token of the range, tokens in it
  int rows;           // query rows of the unit
  int head[2];        // KV head of each lane
  int r0[2];          // first query row of each lane
  bool priv;
  bool low;           // P's low part is multiplied too
  int item;           // index of its partials among the shared / private items
};

// A run as the planner leaves it in shared memory, in a ring of kRuns.
constexpr int kRuns = 4;
struct __align__(16) RunRec {
  int mode, ntiles, tile0, ntok;  // ntiles -1: no further run
  int tok0, row, rows, priv;
  int head[2], r0[2];
  int unit;  // of its partials (for lane 0)
  int low, pad[2];
};
static_assert(sizeof(RunRec) == 64, "");

// The run at step x of a CTA that ends at xend; x moves past it (ntiles may be 0 or less).
__device__ __forceinline__ Run make_run(const SharedParams& p, const Meta& m, int& x, int xend) {
  Run r;
  const int Hp = (p.Hkv + 1) / 2, totS = m.stepS[p.n_groups];
  int off, len;  // step within the item, the item's steps
  if (x < totS) {
    const int g = find(m.stepS, p.n_groups, x);
    const int members = m.gs[g + 1] - m.gs[g];
    int pairs, odd;
    row_tiles(members, p, pairs, odd);
    len = m.eff[g] / KT + kItemSteps;
    off = x - m.stepS[g];
    const int it = off / len;
    off -= it * len;
    r.row = m.gs[g];
    r.rows = members * p.M;
    r.tok0 = 0;
    r.ntok = m.eff[g];
    r.priv = false;
    r.low = r.ntok <= kLowKeys;
    r.item = m.itemS[g] + it;
    const int np = p.Hkv * pairs;
    if (it < np) {
      r.mode = kPair;
      r.head[0] = r.head[1] = it / pairs;
      r.r0[0] = (it - r.head[0] * pairs) * 2 * p.RT;
      r.r0[1] = r.r0[0] + p.RT;
    } else {
      const int hp = it - np;
      r.mode = 2 * hp + 1 < p.Hkv ? kHeads : kSingle;
      r.head[0] = 2 * hp;
      r.head[1] = 2 * hp + 1;
      r.r0[0] = r.r0[1] = pairs * 2 * p.RT;
    }
  } else {
    const int b = find(m.stepP, p.B, x - totS);
    const int eff = m.eff[m.grp[b]];
    len = (m.nlen[b] - eff + KT - 1) / KT + kItemSteps;
    off = x - totS - m.stepP[b];
    const int hp = off / len;
    off -= hp * len;
    r.row = b;
    r.rows = p.M;
    r.tok0 = eff;
    r.ntok = m.nlen[b] - eff;
    r.priv = true;
    r.low = m.nlen[b] <= kLowKeys;
    r.item = b * Hp + hp;
    r.mode = 2 * hp + 1 < p.Hkv ? kHeads : kSingle;
    r.head[0] = 2 * hp;
    r.head[1] = 2 * hp + 1;
    r.r0[0] = r.r0[1] = 0;
  }
  const int take = min(len - off, xend - x);  // (the item's first steps have no tile)
  r.tile0 = max(off - kItemSteps, 0);
  r.ntiles = off + take - kItemSteps - r.tile0;
  x += take;
  return r;
}

// Ring order of a run's tiles (uses counted from the run's first): the order in which the MMA
// issuer takes them.  Pair and single: K(0), then V(n), K(n + 1).  Heads: K0(0), K1(0), then
// V0(n), K0(n + 1), V1(n), K1(n + 1).
__device__ __forceinline__ int v_use(int mode, int w, int n, int last) {
  if (mode != kHeads) return 2 * n + 1;
  return w == 0 ? 4 * n + 2 : (n < last ? 4 * n + 4 : 4 * n + 3);
}
__device__ __forceinline__ int run_uses(int mode, int ntiles) { return mode == kHeads ? 4 * ntiles : 2 * ntiles; }

template <int D>
struct SCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_BYTES = KT * 128;     // 64 columns of a tile
  static constexpr int TILE_BYTES = KT * D * 2;   // a K or V tile, or a lane's Q
  static constexpr int OFF_RING = 2 * TILE_BYTES;
  // full, empty, then s_full, p_full, q_full, o_full, q_empty, fin, turn [2], run_full, run_empty [kRuns]
  static constexpr int NBAR = 2 * kMaxSlots + 14 + 2 * kRuns;
  static constexpr int TAIL = NBAR * 8 + 16 + kRuns * static_cast<int>(sizeof(RunRec));
  static_assert(NBAR % 2 == 0, "the records are 16-byte aligned");
  static constexpr int THREADS = 20 * 32;
  static constexpr uint32_t TMEM_COLS = 512;      // S of the lanes at 0 and 128, O at 256 and 256 + D
  static constexpr uint32_t COL_O = 256;
  static int slots(int meta, size_t optin) {
    const long room = static_cast<long>(optin) - 1024 - OFF_RING - TAIL - 4l * meta;
    const long n = room / TILE_BYTES;
    return static_cast<int>(n > kMaxSlots ? kMaxSlots : n);
  }
  static size_t smem(int slots, int meta) {
    return 1024 + OFF_RING + static_cast<size_t>(slots) * TILE_BYTES + TAIL + 4 * static_cast<size_t>(meta);
  }
};

// Three times 16 columns of this thread's tensor-memory lane, loaded and waited for in one
// statement.
__device__ __forceinline__ void tc_ld16x3_sync(uint32_t t0, uint32_t t1, uint32_t t2, float (&v)[3][16]) {
  uint32_t r[48];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%48];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%49];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47}, [%50];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(r[0]), "=&r"(r[1]), "=&r"(r[2]), "=&r"(r[3]), "=&r"(r[4]), "=&r"(r[5]), "=&r"(r[6]), "=&r"(r[7]), "=&r"(r[8]), "=&r"(r[9]), "=&r"(r[10]), "=&r"(r[11]), "=&r"(r[12]), "=&r"(r[13]), "=&r"(r[14]), "=&r"(r[15]), "=&r"(r[16]), "=&r"(r[17]), "=&r"(r[18]), "=&r"(r[19]), "=&r"(r[20]), "=&r"(r[21]), "=&r"(r[22]), "=&r"(r[23]), "=&r"(r[24]), "=&r"(r[25]), "=&r"(r[26]), "=&r"(r[27]), "=&r"(r[28]), "=&r"(r[29]), "=&r"(r[30]), "=&r"(r[31]), "=&r"(r[32]), "=&r"(r[33]), "=&r"(r[34]), "=&r"(r[35]), "=&r"(r[36]), "=&r"(r[37]), "=&r"(r[38]), "=&r"(r[39]), "=&r"(r[40]), "=&r"(r[41]), "=&r"(r[42]), "=&r"(r[43]), "=&r"(r[44]), "=&r"(r[45]), "=&r"(r[46]), "=&r"(r[47])
      : "r"(t0), "r"(t1), "r"(t2)
      : "memory");
#pragma unroll
  for (int i = 0; i < 48; ++i) v[i / 16][i % 16] = __uint_as_float(r[i]);
}
// 16 columns, likewise.
__device__ __forceinline__ void tc_ld16_sync(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// 64 columns, likewise.
__device__ __forceinline__ void tc_ld64_sync(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}
// Bit patterns to 32 and 16 columns of this thread's lane.
__device__ __forceinline__ void tc_st32b(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31]) : "memory");
}
__device__ __forceinline__ void tc_st16b(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}
// One fp32 value to a column of this thread's lane, and from one (waited for).
__device__ __forceinline__ void tc_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)) : "memory");
}
__device__ __forceinline__ float tc_ld1_sync(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r)
               : "r"(taddr)
               : "memory");
  return __uint_as_float(r);
}
// Named barrier of n threads that returns whether any of them brought `v`.
__device__ __forceinline__ bool named_bar_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}
// tma_load_2d to a shared-memory address; 3-D.
__device__ __forceinline__ void tma_load_2d_at(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y,
                                               uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// a * b + c on two fp32 values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The issuing forms below are run by a whole warp, convergent, so that their operands can stay in
// uniform registers (in a branch of one thread each operand is moved there for each
// instruction: 50 to 75 cycles an MMA instead of its 64); the instruction itself is predicated
// on the elected thread.
// D[tmem] (+)= A[smem] * B[smem]^T.
__device__ __forceinline__ void tc_mma_one(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: the A operand's rows are the lanes, two bf16 a column.
__device__ __forceinline__ void tc_mma_ta_one(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tc_commit_one(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// One try of a phase for a whole warp, suspended for up to 20 us.
__device__ __forceinline__ bool warp_try(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return __all_sync(0xffffffffu, done != 0);
}
// The rest of a wait that the first try did not end (not inlined: a kernel of several roles is
// slow to start while its code is not in the instruction cache).
__device__ __noinline__ bool warp_wait_on(uint32_t bar, uint32_t parity, int32_t* status, volatile int* abort) {
  const unsigned long long t0 = globaltimer();
  while (true) {
    if (warp_try(bar, parity)) return true;
    if (__any_sync(0xffffffffu, *abort != 0)) return false;
    if (__any_sync(0xffffffffu, globaltimer() - t0 > kWaitLimitNs)) {
      *abort = 1;
      report(status, VG_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
}
// mbar_wait_ab for a whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status, volatile int* abort) {
  const uint32_t addr = smem_u32(bar);
  return warp_try(addr, parity) || warp_wait_on(addr, parity, status, abort);
}

// Wait until use number (lap, slot) of a ring is filled.  A wait by parity is right only while
// its barrier is at most one phase behind, and `full` alone does not ensure that here: with the
// lanes taking turns, the slot's previous use may be the other lane's, and its copies may land
// (or be read) later than those of a use this lane has already had.  So the previous use's
// release is awaited first.  That wait is not ambiguous: the caller has had a use u' within
// the last NS - 1 (rings have four slots or more); the producers fill in order, and to fill u' they had
// seen everything up to u' - NS released, the slot's use of two laps ago among it.
__device__ __forceinline__ bool filled(uint64_t* full, uint64_t* empty, int st, int lap, int32_t* status,
                                       volatile int* abort) {
  return (lap == 0 || warp_wait(&empty[st], (lap - 1) & 1, status, abort)) &&
         warp_wait(&full[st], lap & 1, status, abort);
}

// Row (in the cache seen as rows of slots) of the TMA box that starts at token `tok` of
// sequence `row`, or -1 if its page is outside the pool (reported).
__device__ __forceinline__ int box_slot(const SharedParams& p, int row, int tok) {
  if (!p.ptab) return static_cast<int>(p.seq_offset[row]) + tok;
  const int pi = tok / p.psize;
  const int w = pi < p.pstride ? p.ptab[static_cast<size_t>(row) * p.pstride + pi] : -1;
  if (w < 0 || (static_cast<int64_t>(w) + 1) * p.psize > p.capacity) {
    report(p.status, VG_ERR_DEVICE_BOUNDS);
    return -1;
  }
  return w * p.psize + (tok - pi * p.psize);
}

template <int D>
__global__ void __launch_bounds__(SCfg<D>::THREADS, 1)
    shared_attn_kernel(const SharedParams p, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ) {
  using C = SCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int NS = p.nslots;
  uint8_t* ring = smem + C::OFF_RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + static_cast<size_t>(NS) * C::TILE_BYTES);
  uint64_t* empty = full + kMaxSlots;
  uint64_t* s_full = empty + kMaxSlots;
  uint64_t* p_full = s_full + 2;
  uint64_t* q_full = s_full + 4;
  uint64_t* o_full = s_full + 6;
  uint64_t* q_empty = s_full + 8;
  uint64_t* fin = s_full + 10;
  uint64_t* turn = s_full + 12;
  uint64_t* run_full = s_full + 14;
  uint64_t* run_empty = run_full + kRuns;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + C::NBAR);
  // Raised by the first wait that runs out; every later wait then gives up at once.
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  RunRec* recs = reinterpret_cast<RunRec*>(tmem_slot + 4);
  int* mbase = reinterpret_cast<int*>(recs + kRuns);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 2);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w], 8);
      mbar_init(&q_full[w], 1);
      mbar_init(&q_empty[w], 1);
      mbar_init(&o_full[w], 1);
      mbar_init(&fin[w], 1);
      mbar_init(&turn[w], 1);
    }
    for (int k = 0; k < kRuns; ++k) {
      mbar_init(&run_full[k], 1);
      mbar_init(&run_empty[k], 20);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 17) tc_alloc(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tmem_slot;
  // Nothing in global memory is read before this; every thread calls it once.
  auto begin = [&] {
    pdl_wait();
    for (int i = threadIdx.x; i < meta_ints(p.B, p.n_groups); i += C::THREADS) mbase[i] = p.meta[i];
    __syncthreads();
    pdl_launch_dependents();
  };
  // The CTA's run number k (nullptr: no more, or a wait gave up), held until the warp lets it go.
  auto run_at = [&](int k) -> const RunRec* {
    const RunRec* r = recs + k % kRuns;
    return warp_wait(&run_full[k % kRuns], (k / kRuns) & 1, p.status, abort) && r->ntiles >= 0 ? r : nullptr;
  };
  auto run_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&run_empty[k % kRuns]);
  };

  if (warp == 16 || warp == 18) {
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    begin();
    // ---------------------------------------------------------------- TMA producers
    // A tile is 128 / box_rows boxes (page pieces) of 64 columns: one box a lane, the boxes of
    // every tile dealt out to two warps in turn (a warp issues its lanes' boxes one by one).
    // Warp 16 also finds the CTA's runs, each while the copies of the one before are on their way, and
    // leaves them in shared memory (each of the 20 warps for itself took 3000 cycles a run, most
    // of it for instructions out of cache).
    const Meta m = meta_at(mbase, p.B, p.n_groups);
    const int T = m.stepS[p.n_groups] + m.stepP[p.B], nc = min(T, p.nctas), cta = blockIdx.x;
    int x = cta < nc ? static_cast<int>(split_begin(cta, T, nc)) : 0, planned = 0;
    const int x1 = cta < nc ? static_cast<int>(split_begin(cta + 1, T, nc)) : 0;
    bool ended = false;
    auto plan = [&] {
      if (ended) return true;
      RunRec out{kPair, -1, 0, 0, 0, 0, 0, 0, {0, 0}, {0, 0}, 0, 0, {0, 0}};
      while (x < x1 && out.ntiles <= 0) {
        const Run r = make_run(p, m, x, x1);
        out = RunRec{r.mode, r.ntiles, r.tile0, r.ntok, r.tok0, r.row, r.rows, r.priv, {r.head[0], r.head[1]},
                     {r.r0[0], r.r0[1]}, (cta + r.item) * 2, r.low, {0, 0}};
      }
      ended = out.ntiles <= 0;
      if (ended) out.ntiles = -1;
      if (planned >= kRuns &&
          !warp_wait(&run_empty[planned % kRuns], (planned / kRuns - 1) & 1, p.status, abort))
        return false;
      if (lane == 0) {
        recs[planned % kRuns] = out;
        mbar_arrive(&run_full[planned % kRuns]);
      }
      __syncwarp();
      ++planned;
      return true;
    };
    const int BR = p.box_rows;
    const int e = 2 * lane + (warp == 18 ? 1 : 0);
    const int box = e / C::HALVES, half = e % C::HALVES;
    const bool has_box = box < KT / BR;
    const uint32_t dst0 = smem_u32(ring) + half * C::HALF_BYTES + box * BR * 128;
    int off0 = 0;
    int u = 0, st = 0, lap = 0;  // ring uses so far, slot and lap of the next one
    bool ok = true;
    const bool leader = elect_one();
    const int sh = (p.psize & (p.psize - 1)) == 0 ? __ffs(p.psize) - 1 : -1;  // (most page sizes)
    bool zeros = false;  // a slot may hold zeros that the softmax warps wrote
    auto load = [&](const CUtensorMap* map, int head, int y) {
      if (lap > 0) ok = warp_wait(&empty[st], (lap - 1) & 1, p.status, abort);
      if (!ok) return;
      const uint32_t have = __ballot_sync(0xffffffffu, y >= 0);
      if (leader) {
        if (zeros) fence_proxy_async_smem();
        mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(__popc(have) * BR * 128));
      }
      __syncwarp();
      if (y >= 0)
        tma_load_2d_at(dst0 + st * C::TILE_BYTES, map, head * D + half * 64, y, &full[st]);
      __syncwarp();
      ++u;
      if (++st == NS) {
        st = 0;
        ++lap;
      }
    };
    const int lw = warp == 18 ? 1 : 0;  // this warp brings the query tiles of that lane
    uint32_t qpar = 1;                  // (the first wait passes)
    if (lw == 0) ok = plan();
    for (int k = 0; ok; ++k) {
      const RunRec* rec = run_at(k);
      if (!rec) break;
      const RunRec r = *rec;
      const int r0 = lw ? r.r0[1] : r.r0[0], my_head = lw ? r.head[1] : r.head[0];
      run_done(k);
      // page-table word of this lane's box in tile n, loaded a tile ahead; its slot row (-1: no
      // box, or reported) when the tile is issued
      auto word = [&](int n) {
        const int tok = (r.tile0 + n) * KT + box * BR;
        if (!has_box || n >= r.ntiles || tok >= r.ntok) return -1;
        if (!p.ptab) return 0;
        const int pi = sh >= 0 ? (r.tok0 + tok) >> sh : (r.tok0 + tok) / p.psize;
        return pi < p.pstride ? p.ptab[static_cast<size_t>(r.row) * p.pstride + pi] : -1;
      };
      auto slot_row = [&](int n, int w) {
        const int tok = (r.tile0 + n) * KT + box * BR;
        if (!has_box || n >= r.ntiles || tok >= r.ntok) return -1;
        if (!p.ptab) return off0 + r.tok0 + tok;
        if (w < 0 || (static_cast<int64_t>(w) + 1) * p.psize > p.capacity) {
          report(p.status, VG_ERR_DEVICE_BOUNDS);
          return -1;
        }
        return w * p.psize + (sh >= 0 ? (r.tok0 + tok) & (p.psize - 1) : (r.tok0 + tok) % p.psize);
      };
      off0 = p.ptab ? 0 : static_cast<int>(p.seq_offset[r.row]);
      int w0 = word(0), w1 = word(1);
      if (r.mode != kSingle || lw == 0) {
        ok = warp_wait(&q_empty[lw], qpar, p.status, abort);
        qpar ^= 1;
        if (ok && leader) {
          mbar_arrive_expect_tx(&q_full[lw], static_cast<uint32_t>(p.RT * 128 * C::HALVES));
#pragma unroll
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(smem_u32(smem) + lw * C::TILE_BYTES + h * C::HALF_BYTES, &tmQ, h * 64, my_head * p.G,
                        r.row * p.R + r0 / p.G, &q_full[lw]);
        }
        __syncwarp();
      }
      int y = slot_row(0, w0);
      if (ok) load(&tmK, r.head[0], y);
      if (ok && r.mode == kHeads) load(&tmK, r.head[1], y);
      for (int n = 0; ok && n < r.ntiles; ++n) {
        const bool more = n + 1 < r.ntiles;
        const int w2 = word(n + 2);
        load(&tmV, r.head[0], y);
        const int yn = slot_row(n + 1, w1);
        if (ok && more) load(&tmK, r.head[0], yn);
        if (r.mode == kHeads) {
          if (ok) load(&tmV, r.head[1], y);
          if (ok && more) load(&tmK, r.head[1], yn);
        }
        y = yn;
        w1 = w2;
        if (ok && n == 0 && lw == 0) ok = plan();
      }
      zeros |= r.priv != 0;
    }
    // No copy may still be in flight when the CTA exits: normally the issuers have waited
    // for every one; after a lost wait the last ones issued here get 2 ms each to land.
    if (!ok && lane == 0) {
      volatile int never = 0;
      for (int i = u > NS ? u - NS : 0; i < u; ++i)
        mbar_wait_ab(&full[i % NS], (i / NS) & 1, nullptr, &never, 2000000ull);
    }
    __syncwarp();
  } else if (warp == 17 || warp == 19) {
    begin();
    // ---------------------------------------------------------------- MMA issuers, one a lane
    // The whole warp waits, one elected thread issues.  Descriptors are a base plus offsets in
    // units of 16 bytes (addresses stay below 2^18, so the sums stay in the address field).
    // A ring slot is free after two arrivals: one from each lane that reads it, or two from its
    // only reader (see filled).  Where its lane has no tile (kSingle), lane 1 waits and arrives.
    constexpr uint32_t idS = tc_idesc_bf16(128, KT, 0, 0), idO = tc_idesc_bf16(128, D, 0, 1);
    const int w = __shfl_sync(0xffffffffu, warp == 19 ? 1 : 0, 0);
    const uint64_t dq = tc_desc_sw128(smem_u32(smem) + w * C::TILE_BYTES, 16, 1024);
    const uint64_t dk = tc_desc_sw128(smem_u32(ring), 16, 1024), dv = tc_desc_sw128(smem_u32(ring), C::HALF_BYTES, 1024);
    const uint32_t ts = tm + w * 128, to = tm + C::COL_O + w * D;
    const uint32_t lead = elect_one() ? 1u : 0u;
    int st = 0, lap = 0;  // ring slot of the next use, its lap
    uint32_t qpar = 0, ppar = 0, tpar = 0;
    bool ok = true, sole = false;  // sole: this lane is its slots' only reader
    auto skip = [&](int n) {
      st += n;
      if (st >= NS) {
        st -= NS;
        ++lap;
      }
    };
    auto release = [&] {
      tc_commit_one(lead, &empty[st]);
      if (sole) tc_commit_one(lead, &empty[st]);
    };
    // S = Q K^T from the next use (filled); end: Q has no further reader in this run
    auto qk = [&](bool end) {
      tc_fence_after();
      const uint64_t db = dk + static_cast<uint64_t>(st * (C::TILE_BYTES / 16));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        constexpr int H = C::HALF_BYTES / 16;
        tc_mma_one(lead, ts, dq + (kk >> 2) * H + (kk & 3) * 2, db + (kk >> 2) * H + (kk & 3) * 2, idS,
                   kk > 0 ? 1u : 0u);
      }
      tc_commit_one(lead, &s_full[w]);
      release();
      if (end) tc_commit_one(lead, &q_empty[w]);
    };
    // O (+)= P V from the next use (filled), P written (low: its low part too)
    auto pv = [&](bool first, bool end, bool low) {
      tc_fence_after();
      const uint64_t db = dv + static_cast<uint64_t>(st * (C::TILE_BYTES / 16));
#pragma unroll
      for (int kk = 0; kk < KT / 16; ++kk)
        tc_mma_ta_one(lead, to, ts + kk * (low ? 16 : 8), db + kk * 128, idO, (kk > 0 || !first) ? 1u : 0u);
      if (low) {
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk) tc_mma_ta_one(lead, to, ts + kk * 16 + 8, db + kk * 128, idO, 1u);
      }
      release();
      if (end) tc_commit_one(lead, &o_full[w]);
    };
    auto have = [&](int ahead) {  // the use `ahead` of the next one is filled
      const int s2 = st + ahead < NS ? st + ahead : st + ahead - NS;
      return filled(full, empty, s2, st + ahead < NS ? lap : lap + 1, p.status, abort);
    };
    for (int k = 0; ok; ++k) {
      const RunRec* rec = run_at(k);
      if (!rec) break;
      const int ntiles = __shfl_sync(0xffffffffu, rec->ntiles, 0), mode = __shfl_sync(0xffffffffu, rec->mode, 0);
      const bool low = __shfl_sync(0xffffffffu, rec->low, 0) != 0;
      run_done(k);
      const int last = ntiles - 1;
      if (mode == kSingle && w == 1) {
        for (int i = 0; ok && i < 2 * ntiles; ++i) {
          ok = filled(full, empty, st, lap, p.status, abort);
          if (lane == 0) mbar_arrive(&empty[st]);
          skip(1);
        }
        continue;
      }
      // uses of a heads run: K0(0) K1(0), then V0(n) K0(n + 1) V1(n) K1(n + 1); else K(0), then
      // V(n) K(n + 1)
      sole = mode == kHeads;
      ok = warp_wait(&q_full[w], qpar, p.status, abort);
      qpar ^= 1;
      if (sole) skip(w);
      if (!(ok = ok && have(0))) break;
      qk(last == 0);
      skip(sole ? 2 - w : 1);
      // The lanes take turns: a lane issues P V and the next Q K^T together, lane 0 first.  Left to
      // themselves the two issuers' products mix, both lanes' S come late and at the same time, and
      // the tensor cores wait while both are in their softmax
      const bool turns = mode != kSingle;
      if (turns && w == 1 && lane == 0) mbar_arrive(&turn[0]);
      for (int n = 0; n <= last; ++n) {
        const bool end = n == last;
        const int theirs = sole ? (end ? 1 : 2) : 0;
        if (w) skip(theirs);
        // V(n), K(n + 1) and the turn are awaited before P, whose arrival is what the products wait
        // for
        ok = have(0) && (end || have(1)) && (!turns || warp_wait(&turn[w], tpar, p.status, abort)) &&
             warp_wait(&p_full[w], ppar, p.status, abort);
        if (!ok) break;
        tpar ^= turns;
        ppar ^= 1;
        pv(n == 0, end, low);
        skip(1);
        if (!end) {
          qk(n + 1 == last);
          skip(1);
        }
        if (turns && lane == 0 && (w == 0 || !end)) mbar_arrive(&turn[w ^ 1]);
        if (!w) skip(theirs);
      }
    }
    tc_commit_one(lead, &fin[w]);  // every MMA of this thread complete before the CTA tears down
    warp_wait(&fin[w], 0, p.status, abort);
  } else {
    // ---------------------------------------------------------------- softmax lanes
    // Two threads a row: half 0 takes keys 0 .. 63 of each tile, half 1 the others, and each half
    // of the output's columns where those are touched.  They use one running maximum, the row's
    // maximum at the last time it was raised: while no half tile's P sum to more than kMostSum, a
    // thread needs nothing of the other but the word that this holds for both (which the
    // barrier that lets P overwrite S brings along), and the maximum is off the path from S to P.
    constexpr int HK = KT / 2;
    const int w = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3, row = 32 * quad + lane;
    const int pair_bar = 1 + 4 * w + quad;  // named barrier of the two warps that share rows
    const uint32_t tq = tm + (static_cast<uint32_t>(32 * quad) << 16);
    const uint32_t ts = tq + w * 128, to = tq + C::COL_O + w * D + half * (D / 2);
    const float c2 = p.scale_log2;
    const uint32_t to_mine = to, to_other = tq + C::COL_O + w * D + (half ^ 1) * (D / 2);
    int base = 0, ns = 0, nr = 0;  // ring uses, tiles and runs of this lane so far
    // Run -1 takes a tile of whatever tensor memory holds through the code, without a wait, an
    // arrival or a store, while the previous kernel ends and the first tiles are on their way:
    // the first real tile then finds its instructions in the caches (it took 11,000 cycles to
    // go from S to P without that, of a decode step's 75,000).
    for (int k = -1;; ++k) {
      const bool real = k >= 0;
      if (k == 0) begin();
      const RunRec* rec = recs;
      int mode = kPair, last = 0, keys = KT, nrows = KT;
      if (real) {
        rec = run_at(k);
        // (the two warps of a pair meet at named barriers, which have no limit: after a lost wait they
        // leave together)
        if (named_bar_or(pair_bar, 64, rec == nullptr)) break;
        mode = rec->mode;
        last = rec->ntiles - 1;
        keys = rec->ntok - rec->tile0 * KT;
        nrows = min(p.RT, rec->rows - rec->r0[w]);
        if (mode == kSingle && w == 1) {
          base += run_uses(mode, last + 1);
          run_done(k);
          continue;
        }
      }
      const bool live = 32 * quad < nrows;  // (a warp without rows only keeps the barriers' count)
      float mx = neg_inf(), l = 0.f;        // the maximum in use (log2 units), this half's sum
      for (int n = 0; n <= last; ++n) {
        const int left = keys - n * KT;  // keys of the tile (128 or more: all)
        if (real) warp_wait(&s_full[w], ns++ & 1, p.status, abort);
        tc_fence_after();
        if (left < KT) {
          // value rows past the range hold whatever was there: zeroed, so that 0 * V is 0 (after
          // the wait for S, which orders this tile's V within NS uses of its K: see filled)
          const int use = base + v_use(mode, w, n, last);
          filled(full, empty, use % NS, use / NS, p.status, abort);
          uint8_t* vt = ring + static_cast<size_t>(use % NS) * C::TILE_BYTES;
          for (int e = threadIdx.x & 255; e < C::HALVES * KT * 8; e += 256) {
            const int h = e / (KT * 8), i = (e >> 3) & (KT - 1);
            if (i >= left)
              *reinterpret_cast<uint4*>(vt + h * C::HALF_BYTES + i * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (!live) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[w]);
          continue;
        }
        const int valid = left - HK * half;  // keys of this half (64 or more: all)
        uint32_t pk[HK / 2];
        auto load_s = [&](float (&s)[HK]) {
          tc_ld64_sync(ts + HK * half, s);
          if (valid < HK) {
#pragma unroll
            for (int i = 0; i < HK; ++i)
              if (i >= valid) s[i] = neg_inf();
          }
        };
        if (n == 0) {
          // The run's first tile gives the maximum to begin with.  The row's two threads tell each
          // other their half's through the first column of their half of O, which is read out and
          // not yet written again
          float s[HK];
          load_s(s);
          float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 0; i < HK; i += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j) t4[j] = max3(t4[j], s[i + 2 * j], s[i + 2 * j + 1]);
          const float t = fmaxf(max3(t4[0], t4[1], t4[2]), t4[3]) * c2;
          tc_st1(to_mine, t);
          tc_wait_st();
          tc_fence_before();
          named_bar_or(pair_bar, 64, false);
          tc_fence_after();
          mx = fmaxf(t, tc_ld1_sync(to_other));
        }
        float ls = 0.f;
        for (bool raised = false;; raised = true) {
          // P = 2^(s c2 - mx) of this half, and its sum, of the bf16 values that P V multiplies: a row's
          // weights sum to one
          float s[HK];
          load_s(s);
          float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < HK; i += 2) {
            const float2 e = fma2(make_float2(s[i], s[i + 1]), make_float2(c2, c2), make_float2(-mx, -mx));
            pk[i / 2] = pack_bf16(ex2(e.x), ex2(e.y));
            a4[(i >> 1) & 3] = add_bf16x2_f32(pk[i / 2], a4[(i >> 1) & 3]);
          }
          ls = (a4[0] + a4[1]) + (a4[2] + a4[3]);
          // (both threads of each row have read S after the barrier: P may overwrite it)
          if (!named_bar_or(pair_bar, 64, row < nrows && ls > kMostSum) || raised) break;
          // rare: the row's maximum over the whole tile, which both threads of the row read for
          // themselves, becomes the one in use; then P again.  (A sum of 64 beyond kMostSum has a P of
          // 4 or more in it: two above the maximum in use)
          float t = neg_inf();
#pragma unroll 1
          for (int c0 = 0; c0 < KT; c0 += 32) {
            float v[32];
            tc_ld32_sync(ts + c0, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) t = fmaxf(t, c0 + i < left ? v[i] : neg_inf());
          }
          t *= c2;
          const float mn = t > mx + 1.f ? t : mx;
          // (P V of the lane's previous tile has completed: the commit that brought this S
          // came after it)
          const float alpha = mn != mx ? ex2(mx - mn) : 1.f;
          l *= alpha;
#pragma unroll 1
          for (int c0 = 0; c0 < D / 2; c0 += 32) {
            float o[32];
            tc_ld32_sync(to + c0, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            tc_st32(to + c0, o);
          }
          mx = mn;
        }
        if (real && rec->low != 0) {
          // P in two parts, over S in place: a step of 16 keys of the product has its high parts in the
          // first eight of their columns of S and its low parts in the others
          ls = 0.f;
#pragma unroll 1
          for (int c0 = 0; c0 < HK; c0 += 16) {
            float v[16];
            uint32_t part[16];
            tc_ld16_sync(ts + HK * half + c0, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float p0 = c0 + 2 * i < valid ? ex2(fmaf(v[2 * i], c2, -mx)) : 0.f;
              const float p1 = c0 + 2 * i + 1 < valid ? ex2(fmaf(v[2 * i + 1], c2, -mx)) : 0.f;
              split_bf16(p0, p1, part[i], part[8 + i]);
              ls = add_bf16x2_f32(part[8 + i], add_bf16x2_f32(part[i], ls));
            }
            tc_st16b(ts + HK * half + c0, part);
          }
          tc_wait_st();
        } else if (real) {
          tc_st32b(ts + (HK / 2) * half, pk);
          tc_wait_st();
        }
        l += ls;
        tc_fence_before();
        __syncwarp();
        if (real && lane == 0) mbar_arrive(&p_full[w]);
      }
      if (!real) continue;
      // the run's partial: (O, max, sum) of each row once P V of its last tile has landed
      warp_wait(&o_full[w], nr & 1, p.status, abort);
      ++nr;
      tc_fence_after();
      if (live) {
        // four columns of 32 rows lie together: a warp's stores are 512 contiguous bytes
        const bool priv = rec->priv != 0;
        const int height = priv ? p.Mpad : KT;
        const size_t unit = static_cast<size_t>(rec->unit + w);
        float* po = (priv ? p.partp_o : p.parts_o) + (unit * D + half * (D / 2)) * height + row * 4;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2; c0 += 32) {
          float o[32];
          tc_ld32_sync(to + c0, o);
          if (row < nrows) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(po + static_cast<size_t>(c0 + i) * height) =
                  make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        // (max, sum of each half of the keys, unused)
        float* pml = (priv ? p.partp_ml : p.parts_ml) + (unit * height + row) * 4;
        if (row < nrows) {
          if (half == 0) *reinterpret_cast<float2*>(pml) = make_float2(mx, l);
          else pml[2] = l;
        }
      }
      tc_fence_before();
      base += run_uses(mode, last + 1);
      run_done(k);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tc_dealloc(tm, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- combine
// A CTA merges ROWS consecutive rows of a (sequence, KV head).  A thread has four columns of every
// eighth row (ROWS >= 8), or of one row and every fourth of its partials (ROWS = 2).  Everything
// is asked for in two rounds: the sequence's record, then the partials, their maxima and sums, the
// query rows and the verify rows' own keys and values; where each of these lies is worked out
// once, by one thread each.  A warp a row takes the causal logits of the row's own keys
// u = 0 .. t, and the maximum and the sum over those and the row's partials (lanes across
// partials).  Then the threads of a column add up: the row's shared partials by CTA, its
// private ones by CTA, the causal values: a fixed order.
//
// What bounds it is instructions, most of them addresses and the short sums: there are some ten
// products for each of a row's 128 columns (64 sequences x 32 rows x 8 heads: 27 us at 0.7
// instructions a cycle and partition, whether 4, 5 or 6 CTAs fit an SM; 32 us with 16 rows a CTA, 36
// with 32.  Of its time the logits take about 4 us, the staging of the verify rows' keys and values 4).
template <int D, int ROWS>
__global__ void __launch_bounds__(2 * D) shared_combine_kernel(const SharedParams p) {
  constexpr int PER = D / 32, WARPS = D / 16, CH = D / 8, NT = 2 * D;
  constexpr int SG = ROWS < 8 ? 8 / ROWS : 1;      // threads that share a row's four columns
  constexpr int RPT = ROWS < 8 ? 1 : ROWS / 8;     // rows a thread
  constexpr int NB = ROWS == 2 ? 8 : 4;            // partials in flight a thread
  constexpr int NW = 64;                           // partials of a row whose weights are kept
  __shared__ float lgs[ROWS][16], rowM[ROWS], rowL[ROWS], wts[ROWS][NW];
  // the row's shared and private partials: how many, and the first one's place in units of 16
  // bytes (of O, then of its row of maximum and sums)
  __shared__ int cnt[ROWS][2];
  __shared__ uint32_t at[ROWS][4];
  __shared__ int64_t slots[16];  // of the verify rows in the cache
  __shared__ __align__(16) __nv_bfloat16 kvs[2][16][D];
  __shared__ float4 part_sum[SG][ROWS][D / 4];
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rblocks = (p.M + ROWS - 1) / ROWS;
  const int bg = blockIdx.x / rblocks, r0 = (blockIdx.x - bg * rblocks) * ROWS;
  const int b = bg / p.Hkv, g = bg - b * p.Hkv;
  const int rows = min(ROWS, p.M - r0);
  const int tmax = (r0 + rows - 1) / p.G;
  pdl_wait();
  const SeqRec rec = reinterpret_cast<const SeqRec*>(p.rec)[b];
  const int n = rec.n;
  if (n < 0) return;  // the whole CTA
  if (tid < rows) {
    // the first kItemSteps steps of an item have no tile (see make_run); every CTA that owns a later one
    // left a partial
    const SeqRec tot = reinterpret_cast<const SeqRec*>(p.rec)[p.B];
    const int r = r0 + tid, tiles = rec.eff / KT, ptiles = (n - rec.eff + KT - 1) / KT;
    cnt[tid][0] = cnt[tid][1] = 0;
    const int T = tot.stepS + tot.stepP, nc = min(T, p.nctas);
    if (tiles > 0) {
      const int rr = rec.row0 + r, rt = rr / p.RT;
      const bool pair = (rt >> 1) < rec.pairs;
      const int it = pair ? g * rec.pairs + (rt >> 1) : p.Hkv * rec.pairs + (g >> 1);
      const int s0 = rec.stepS + it * (tiles + kItemSteps) + kItemSteps;  // its first tile
      const int cs = static_cast<int>(owner_cta(s0, T, nc));
      cnt[tid][0] = static_cast<int>(owner_cta(s0 + tiles - 1, T, nc)) - cs + 1;
      const uint32_t u = (cs + rec.itemS + it) * 2 + (pair ? rt & 1 : g & 1);
      at[tid][0] = u * (KT * D / 4) + (rr - rt * p.RT);
      at[tid][1] = u * KT + (rr - rt * p.RT);
    }
    if (ptiles > 0) {
      const int s0 = tot.stepS + rec.stepP + (g >> 1) * (ptiles + kItemSteps) + kItemSteps;
      const int cp = static_cast<int>(owner_cta(s0, T, nc));
      cnt[tid][1] = static_cast<int>(owner_cta(s0 + ptiles - 1, T, nc)) - cp + 1;
      const uint32_t u = (cp + b * ((p.Hkv + 1) / 2) + (g >> 1)) * 2 + (g & 1);
      at[tid][2] = u * (p.Mpad * (D / 4)) + r;
      at[tid][3] = u * p.Mpad + r;
    }
  } else if (tid >= 32 && tid < 48 && tid - 32 <= tmax) {
    const int64_t slot = kv_slot(p.seq_offset, p.ptab, p.psize, p.pstride, p.capacity, b, n + tid - 32);
    slots[tid - 32] = slot;
    if (slot < 0) report(p.status, VG_ERR_DEVICE_BOUNDS);  // a page outside the pool: neither read nor written
  }
  __syncthreads();
  // (max, sum) row and O of partial i of a row (from one CTA's partial to the next's two lanes' rows
  // lie between)
  auto ml_at = [&](int rl, int i, int nS) {
    return i < nS ? reinterpret_cast<const float4*>(p.parts_ml) + (at[rl][1] + static_cast<uint32_t>(i) * (2 * KT))
                  : reinterpret_cast<const float4*>(p.partp_ml) + (at[rl][3] + static_cast<uint32_t>(i - nS) * (2 * p.Mpad));
  };
  // a thread's four columns of a row: its partials' places (by number), how many shared and in all
  struct Row {
    const float4 *s, *p;
    int nS, n;
  };
  auto row_at = [&](int rl, int c) {
    Row x{nullptr, nullptr, 0, 0};
    if (rl < rows) {
      x.nS = cnt[rl][0];
      x.n = x.nS + cnt[rl][1];
      x.s = reinterpret_cast<const float4*>(p.parts_o) + (at[rl][0] + c * KT);
      x.p = reinterpret_cast<const float4*>(p.partp_o) + (at[rl][2] + c * p.Mpad);
    }
    return x;
  };
  auto o_at = [&](const Row& x, int i) {
    return i < x.nS ? x.s + static_cast<size_t>(i) * (2 * KT * D / 4)
                    : x.p + static_cast<size_t>(static_cast<uint32_t>(i - x.nS) * (2 * p.Mpad * (D / 4)));
  };
  const int rl0 = tid % (ROWS < 8 ? ROWS : 8), sg = ROWS < 8 ? tid / ROWS % SG : 0, c = tid / 8;
  struct Batch {
    float4 v[NB];
  };
  auto fetch = [&](Batch& x, const Row& row, int i0) {  // partials i0 + sg, i0 + sg + SG ... of a row
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int i = i0 + sg + q * SG;
      x.v[q] = i < row.n ? *o_at(row, i) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  Batch now, next;
  Row here = row_at(rl0, c);
  fetch(now, here, 0);
  auto load_ml = [&](int rl, int i, float& ms, float& ls) {  // (max, sum) of partial i of a row
    ms = neg_inf();
    ls = 0.f;
    if (rl >= rows) return;
    const int nS = cnt[rl][0];
    if (i >= nS + cnt[rl][1]) return;
    const float4 x = *ml_at(rl, i, nS);
    ms = x.x;
    ls = x.y + x.z;
  };
  // the first maxima and sums and the query row of each of the warp's rows, asked for together
  constexpr int RPW = (ROWS + WARPS - 1) / WARPS;
  float first_m[RPW][2], first_l[RPW][2];
  uint32_t qrow[RPW][PER / 2];
#pragma unroll
  for (int k = 0; k < RPW; ++k) {
    const int wr = warp + k * WARPS;
    load_ml(wr, lane, first_m[k][0], first_l[k][0]);
    load_ml(wr, lane + 32, first_m[k][1], first_l[k][1]);
    const int r = r0 + min(wr, rows - 1), t = r / p.G, jh = r - t * p.G;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        p.q + ((static_cast<size_t>(b) * p.R + t) * p.Hq + g * p.G + jh) * D + lane * PER);
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) qrow[k][e] = src[e];
  }
  for (int e = tid; e < 2 * 16 * CH; e += NT) {
    const int which = e / (16 * CH), u = e / CH % 16, cc = e % CH;
    if (u > tmax) continue;
    const __nv_bfloat16* fresh = which ? p.v_new : p.k_new;
    const int64_t slot = slots[u];
    const __nv_bfloat16* src = fresh ? fresh + ((static_cast<size_t>(b) * p.R + u) * p.Hkv + g) * D
                                     : (which ? p.V : p.K) + ((slot < 0 ? 0 : slot) * p.Hkv + g) * D;
    uint4 x = reinterpret_cast<const uint4*>(src)[cc];
    if (!fresh && slot < 0) x = make_uint4(0u, 0u, 0u, 0u);
    reinterpret_cast<uint4*>(&kvs[which][u][0])[cc] = x;
  }
  __syncthreads();
#pragma unroll
  for (int kr = 0; kr < RPW; ++kr) {
    const int wr = warp + kr * WARPS;
    if (wr >= rows) break;
    const int t = (r0 + wr) / p.G;
    const int np = cnt[wr][0] + cnt[wr][1];
    const float pm = first_m[kr][0], pl = first_l[kr][0], pm2 = first_m[kr][1], pl2 = first_l[kr][1];
    float qv[PER];
#pragma unroll
    for (int e = 0; e < PER / 2; ++e) {
      qv[2 * e] = __uint_as_float(qrow[kr][e] << 16);
      qv[2 * e + 1] = __uint_as_float(qrow[kr][e] & 0xffff0000u);
    }
    float pmax = fmaxf(pm, pm2);
    for (int u0 = 0; u0 <= t; u0 += 8) {
      // eight keys at a time; their sums over the lanes in nine exchanges, after which lanes 4 j .. 4 j + 3
      // have key j's
      float dot[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dot[j] = 0.f;
        if (u0 + j <= t) {
#pragma unroll
          for (int e = 0; e < PER; e += 2) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(&kvs[0][u0 + j][lane * PER + e]);
            dot[j] += qv[e] * __uint_as_float(x << 16);
            dot[j] += qv[e + 1] * __uint_as_float(x & 0xffff0000u);
          }
        }
      }
#pragma unroll
      for (int h = 4; h > 0; h >>= 1)
#pragma unroll
        for (int j = 0; j < h; ++j) {
          const bool up = (lane & (4 * h)) != 0;
          const float keep = up ? dot[j + h] : dot[j], give = up ? dot[j] : dot[j + h];
          dot[j] = keep + __shfl_xor_sync(0xffffffffu, give, 4 * h);
        }
      float x = dot[0];
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x *= p.scale_log2;
      const int u = u0 + (lane >> 2);
      if (u <= t) {
        if (!p.k_new && slots[u] < 0) x = neg_inf();  // (a key that the cache does not have)
        pmax = fmaxf(pmax, x);
        if ((lane & 3) == 0) lgs[wr][u] = x;
      }
    }
    for (int i = 64; i < np; i += 32) {
      float ms, ls;
      load_ml(wr, i + lane, ms, ls);
      pmax = fmaxf(pmax, ms);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) pmax = fmaxf(pmax, __shfl_xor_sync(0xffffffffu, pmax, o));
    const float M = pmax;
    const float w1 = pm != neg_inf() ? ex2(pm - M) : 0.f, w2 = pm2 != neg_inf() ? ex2(pm2 - M) : 0.f;
    wts[wr][lane] = w1;
    wts[wr][lane + 32] = w2;
    float l = w1 * pl + w2 * pl2;
    for (int i = 64; i < np; i += 32) {
      float ms, ls;
      load_ml(wr, i + lane, ms, ls);
      if (ms != neg_inf()) l += ex2(ms - M) * ls;
    }
    __syncwarp();
    const float w = lane <= t ? ex2(lgs[wr][lane] - M) : 0.f;  // (t < 16)
    l += w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if (lane <= t) lgs[wr][lane] = w;
    if (lane == 0) {
      rowM[wr] = M;
      rowL[wr] = l;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < RPT; ++k) {
    const int rl = rl0 + 8 * k;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const Row row = here;
    if (k + 1 < RPT) {
      here = row_at(rl + 8, c);
      fetch(next, here, 0);  // the next row's, while this one's are added
    }
    auto add = [&](float w, const float4& v) {
      acc.x += w * v.x;
      acc.y += w * v.y;
      acc.z += w * v.z;
      acc.w += w * v.w;
    };
    for (int i0 = 0; i0 < min(row.n, NW); i0 += NB * SG) {
      if (i0 > 0) fetch(now, row, i0);
#pragma unroll
      for (int q = 0; q < NB; ++q) add(wts[rl][i0 + sg + q * SG], now.v[q]);
    }
    for (int i = NW + sg; i < row.n; i += SG) {  // (a row of very many partials)
      const float m = ml_at(rl, i, row.nS)->x;
      add(m != neg_inf() ? ex2(m - rowM[rl]) : 0.f, *o_at(row, i));
    }
    if constexpr (SG > 1) {
      part_sum[sg][rl][c] = acc;
      __syncthreads();
      if (sg > 0) return;
#pragma unroll
      for (int j = 1; j < SG; ++j) {
        const float4 x = part_sum[j][rl][c];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
    }
    if (k + 1 < RPT) now = next;
    if (rl >= rows) return;
    const int r = r0 + rl, t = r / p.G, jh = r - t * p.G;
    for (int u = 0; u <= t; ++u) {
      const float w = lgs[rl][u];
      const uint2 x = *reinterpret_cast<const uint2*>(&kvs[1][u][4 * c]);
      acc.x += w * __uint_as_float(x.x << 16);
      acc.y += w * __uint_as_float(x.x & 0xffff0000u);
      acc.z += w * __uint_as_float(x.y << 16);
      acc.w += w * __uint_as_float(x.y & 0xffff0000u);
    }
    const float inv = 1.f / rowL[rl];
    *reinterpret_cast<uint2*>(p.out + ((static_cast<size_t>(b) * p.R + t) * p.Hq + g * p.G + jh) * D + 4 * c) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (p.k_new && jh == 0 && slots[t] >= 0) {  // append verify row t
      const size_t dst = (slots[t] * p.Hkv + g) * D + 4 * c;
      *reinterpret_cast<uint2*>(p.K + dst) = *reinterpret_cast<const uint2*>(&kvs[0][t][4 * c]);
      *reinterpret_cast<uint2*>(p.V + dst) = *reinterpret_cast<const uint2*>(&kvs[1][t][4 * c]);
    }
  }
}

// ---------------------------------------------------------------- scores
// scores[b][i] = scale * sum over the mask's rows and all heads of q . K_i = scale * sum over
// KV heads g of Q_b,g . K_i,g with Q_b,g the sum of the sequence's masked query rows of head g.
// Q is fp32 and enters the tensor cores as three bf16 parts.
//
// One item is a tile of 128 keys and up to N members: S^T[keys][members] on the tensor cores
// (the keys are the M rows, so few members cost little), one KV head at a time into a double
// buffer, the three parts of the members' queries side by side as columns; four warps add the
// parts and the heads' tiles in fp32 registers (the tensor core's own sum runs over one part of
// one head) and write rows of consecutive positions.  A private range has one member: its
// items bring and multiply the 16 columns an MMA has at least.
//
// What bounds it: the keys' bytes, once its ring is full: 8 sequences over three prompts of 20011 tokens
// and 8 KV heads take 29.5 us for 123 MB of shared keys, a stage of 32 KB every 1200 cycles (7.8 TB/s,
// partly out of L2) after a start of 7000.  64 members over one prompt bring 24 KB of query parts with
// each 32 KB of keys, and three stages do not cover the latency: 29 us for 105 MB.
template <int D, int N>
struct ZCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_BYTES = KT * 128;
  static constexpr int K_BYTES = KT * D * 2;
  static constexpr int Z_HALF = 3 * N * 128;      // 64 columns of the query parts
  static constexpr int STAGE = K_BYTES + HALVES * Z_HALF;
  static constexpr int NST = 196608 / STAGE > 6 ? 6 : 196608 / STAGE;
  static constexpr int NBAR = 2 * NST + 6;
  static constexpr int THREADS = 224;
  static constexpr uint32_t TMEM_COLS = N == 16 ? 128 : 256;  // two buffers of 3 N columns
  static constexpr uint32_t COL_B = TMEM_COLS / 2;
  static size_t smem(int meta) { return 1024 + NST * STAGE + NBAR * 8 + 16 + 4 * static_cast<size_t>(meta); }
};

template <int D, int N>
__global__ void __launch_bounds__(ZCfg<D, N>::THREADS, 1)
    shared_score_kernel(const SharedParams p, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmZ, const __grid_constant__ CUtensorMap tmZ1) {
  using C = ZCfg<D, N>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::NST * C::STAGE);
  uint64_t* empty = full + C::NST;
  uint64_t* s_full = empty + C::NST;
  uint64_t* s_free = s_full + 2;
  uint64_t* fin = s_full + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + C::NBAR);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* mbase = reinterpret_cast<int*>(tmem_slot + 4);
  const Meta m = meta_at(mbase, p.B, p.n_groups);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 32) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 4);
    }
    mbar_init(fin, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 5) tc_alloc(tmem_slot, C::TMEM_COLS);
  pdl_wait();
  for (int i = threadIdx.x; i < meta_ints(p.B, p.n_groups); i += C::THREADS) mbase[i] = p.meta[i];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tmem_slot;
  pdl_launch_dependents();
  const int totS = m.scS[p.n_groups], T = totS + m.scP[p.B];
  struct Item {
    int row, tok0, ntok, tile, seq0, members, cols;
  };
  auto item = [&](int x) {
    Item i;
    if (x < totS) {
      const int g = find(m.scS, p.n_groups, x);
      const int nm = m.gs[g + 1] - m.gs[g], mb = (nm + N - 1) / N, off = x - m.scS[g];
      i.tile = off / mb;
      const int blk = off - i.tile * mb;
      i.row = m.gs[g];
      i.tok0 = 0;
      i.ntok = m.eff[g];
      i.seq0 = m.gs[g] + blk * N;
      i.members = min(N, nm - blk * N);
    } else {
      const int b = find(m.scP, p.B, x - totS);
      i.tile = x - totS - m.scP[b];
      i.row = i.seq0 = b;
      i.tok0 = m.eff[m.grp[b]];
      i.ntok = m.nlen[b] - i.tok0;
      i.members = 1;
    }
    i.cols = x < totS ? N : 16;  // columns of one part
    return i;
  };
  if (warp == 4 || warp == 6) {
    // the boxes of a tile dealt out to two warps, one a lane, as in the attention kernel; the halves
    // of the query parts likewise
    const int BR = p.box_rows, second = warp == 6 ? 1 : 0;
    const int e = 2 * lane + second, box = e / C::HALVES, half = e % C::HALVES;
    int u = 0, st = 0, lap = 0;
    bool ok = true;
    for (int x = blockIdx.x; ok && x < T; x += gridDim.x) {
      const Item it = item(x);
      const int at = it.tile * KT + box * BR;
      const int y = box < KT / BR && at < it.ntok ? box_slot(p, it.row, it.tok0 + at) : -1;
      const int boxes = __popc(__ballot_sync(0xffffffffu, y >= 0));
      for (int g = 0; g < p.Hkv; ++g) {
        if (lap > 0) ok = warp_wait(&empty[st], (lap - 1) & 1, p.status, abort);
        if (!ok) break;
        const uint32_t dst = smem_u32(smem) + st * C::STAGE;
        const bool z = second < C::HALVES;
        if (lane == 0) {
          mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(boxes * BR * 128 + (z ? 3 * it.cols * 128 : 0)));
          if (z)  // the three parts of `cols` members, one after another
            tma_load_3d(dst + C::K_BYTES + second * C::Z_HALF, it.cols == N ? &tmZ : &tmZ1, g * D + second * 64, it.seq0,
                        0, &full[st]);
        }
        __syncwarp();
        if (y >= 0)
          tma_load_2d_at(dst + half * C::HALF_BYTES + box * BR * 128, &tmK, g * D + half * 64, y, &full[st]);
        __syncwarp();
        ++u;
        if (++st == C::NST) {
          st = 0;
          ++lap;
        }
      }
    }
    // (as in the attention kernel: no copy is in flight at the end of a normal run)
    if (!ok && lane == 0) {
      volatile int never = 0;
      for (int i = u > C::NST ? u - C::NST : 0; i < u; ++i)
        mbar_wait_ab(&full[i % C::NST], (i / C::NST) & 1, nullptr, &never, 2000000ull);
    }
    __syncwarp();
  } else if (warp == 5) {
    int u = 0, st = 0;
    uint32_t par = 0;
    bool ok = true;
    const uint32_t lead = elect_one() ? 1u : 0u;
    const uint64_t dk = tc_desc_sw128(smem_u32(smem), 16, 1024);
    const uint64_t dz = tc_desc_sw128(smem_u32(smem) + C::K_BYTES, 16, 1024);
    for (int x = blockIdx.x; ok && x < T; x += gridDim.x) {
      const Item it = item(x);
      const uint32_t id = tc_idesc_bf16(128, 3 * it.cols, 0, 0);
      for (int g = 0; ok && g < p.Hkv; ++g, ++u) {
        ok = warp_wait(&full[st], par, p.status, abort) &&
             (u < 2 || warp_wait(&s_free[u & 1], ((u - 2) >> 1) & 1, p.status, abort));
        if (!ok) break;
        tc_fence_after();
        const uint64_t da = dk + static_cast<uint64_t>(st * (C::STAGE / 16));
        const uint64_t db = dz + static_cast<uint64_t>(st * (C::STAGE / 16));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma_one(lead, tm + (u & 1) * C::COL_B, da + (kk >> 2) * (C::HALF_BYTES / 16) + (kk & 3) * 2,
                     db + (kk >> 2) * (C::Z_HALF / 16) + (kk & 3) * 2, id, kk > 0 ? 1u : 0u);
        tc_commit_one(lead, &s_full[u & 1]);
        tc_commit_one(lead, &empty[st]);
        if (++st == C::NST) {
          st = 0;
          par ^= 1;
        }
      }
    }
    tc_commit_one(lead, fin);  // every MMA of this thread complete before the CTA tears down
    warp_wait(fin, 0, p.status, abort);
  } else if (warp < 4) {
    int u = 0;
    const uint32_t tl = tm + (static_cast<uint32_t>(32 * warp) << 16);
    for (int x = blockIdx.x; x < T; x += gridDim.x) {
      const Item it = item(x);
      float acc[N];
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] = 0.f;
      for (int g = 0; g < p.Hkv; ++g, ++u) {
        warp_wait(&s_full[u & 1], (u >> 1) & 1, p.status, abort);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < N; c += 16) {
          if (c < it.cols) {
            float v[3][16];
            const uint32_t at = tl + (u & 1) * C::COL_B + c;
            tc_ld16x3_sync(at, at + it.cols, at + 2 * it.cols, v);
            // (the small parts first: the large sum is rounded into last)
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[c + k] += v[0][k] + (v[1][k] + v[2][k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[u & 1]);
      }
      const int at = it.tile * KT + 32 * warp + lane;
      if (at < it.ntok) {
        float* dst = p.scores + it.seq0 * p.score_stride + it.tok0 + at;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          if (k < it.members) *dst = acc[k] * p.scale;
          dst += p.score_stride;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tc_dealloc(tm, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- launches
struct Launch {
  cudaLaunchAttribute at[1];
  cudaLaunchConfig_t cfg = {};
  Launch(int grid, int block, size_t smem, cudaStream_t stream) {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
};

template <int D, int N>
cudaError_t launch_scores(const SharedParams& p, const CUtensorMap& tmK, const CUtensorMap& tmZ,
                          const CUtensorMap& tmZ1, cudaStream_t stream) {
  using C = ZCfg<D, N>;
  const size_t smem = C::smem(meta_ints(p.B, p.n_groups));
  cudaError_t e = ensure_smem<shared_score_kernel<D, N>>(smem);
  if (e != cudaSuccess) return e;
  Launch z(p.nctas, C::THREADS, smem, stream);
  return cudaLaunchKernelEx(&z.cfg, shared_score_kernel<D, N>, p, tmK, tmZ, tmZ1);
}

template <int D>
cudaError_t launch_shared_t(const SharedParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                            const CUtensorMap& tmQ, const CUtensorMap& tmZ, const CUtensorMap& tmZ1,
                            cudaStream_t stream) {
  cudaError_t e;
  Launch f(p.mask ? 1 + p.B : 1, kPrepThreads, 0, stream);
  if ((e = cudaLaunchKernelEx(&f.cfg, shared_prep_kernel, p)) != cudaSuccess) return e;
  if (p.mask) {
    e = p.nsc == 16 ? launch_scores<D, 16>(p, tmK, tmZ, tmZ1, stream) : launch_scores<D, 32>(p, tmK, tmZ, tmZ1, stream);
    if (e != cudaSuccess) return e;
  }
  using C = SCfg<D>;
  const size_t smem = C::smem(p.nslots, meta_ints(p.B, p.n_groups));
  if ((e = ensure_smem<shared_attn_kernel<D>>(smem)) != cudaSuccess) return e;
  Launch a(p.nctas, C::THREADS, smem, stream);
  if ((e = cudaLaunchKernelEx(&a.cfg, shared_attn_kernel<D>, p, tmK, tmV, tmQ)) != cudaSuccess) return e;
  // rows of a CTA share their staging, but fewer CTAs than SMs leave SMs idle (16 sequences of one
  // row and 4 heads a KV head: 9.5 us with two rows a CTA, 12.5 with eight; 8 sequences of 7
  // rows: 14.9 and 10.8; 64 of 8 rows: 91 and 27)
  const int bg = p.B * p.Hkv;
  if (bg * ((p.M + 7) / 8) >= p.nctas) {
    Launch c(bg * ((p.M + 7) / 8), 2 * D, 0, stream);
    return cudaLaunchKernelEx(&c.cfg, shared_combine_kernel<D, 8>, p);
  }
  Launch c(bg * ((p.M + 1) / 2), 2 * D, 0, stream);
  return cudaLaunchKernelEx(&c.cfg, shared_combine_kernel<D, 2>, p);
}

}  // namespace

int shared_meta_ints(int B, int n_groups) { return meta_ints(B, n_groups); }

size_t shared_rec_bytes(int B) { return sizeof(SeqRec) * (static_cast<size_t>(B) + 1); }

int shared_slots(int D, int B, int n_groups, size_t smem_optin) {
  const int n = meta_ints(B, n_groups);
  return D == 64 ? SCfg<64>::slots(n, smem_optin) : SCfg<128>::slots(n, smem_optin);
}

cudaError_t launch_shared(const SharedParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          const CUtensorMap& tmQ, const CUtensorMap& tmZ, const CUtensorMap& tmZ1,
                          cudaStream_t stream) {
  return p.D == 64 ? launch_shared_t<64>(p, tmK, tmV, tmQ, tmZ, tmZ1, stream)
                   : launch_shared_t<128>(p, tmK, tmV, tmQ, tmZ, tmZ1, stream);
}

}  // namespace vg
