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
// over the CTAs.  A CTA has two softmax warpgroups, "lanes", each with its own 128 rows, S / P
// and O in tensor memory; a step is one key tile for both lanes:
//   pair   the lanes are two row tiles of one KV head and share the step's K and V tile;
//   heads  the lanes are the same row tile of two KV heads, each with its own K and V tile
//          (a group's odd last row tile, and every private range).
// While one lane's warps run the softmax of their tile, the tensor cores work for the other
// (P V of its tile, then Q K^T of its next).  P goes back to tensor memory as bf16, over the
// columns of S, and is the A operand of P V from there: it never passes shared memory.
// Warps: 0-3 and 4-7 the lanes (a thread is a row: no exchange between threads), 8 the TMA
// producer, 9 the MMA issuer.
#include "vg_common.cuh"
#include "vg_internal.h"

namespace vg {
namespace {

constexpr int KT = kSharedTileKeys;  // keys of a tile, and rows of a lane
static_assert(KT == 128, "a lane's rows and a tile's keys are the 128 tensor-memory lanes");
// A row's running max is raised only when a tile exceeds it by more than this (log2 units):
// P stays below 2^8 and O is rescaled rarely.
constexpr float kRescaleSlack = 8.f;
constexpr int kMaxSlots = 12;  // ring slots (K or V tiles)

// ---------------------------------------------------------------- the batch's layout
// Everything the kernels need about lengths and groups, from the device arrays; built by one
// warp of each CTA (B <= 1024), and left in the workspace for the combine kernel.
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

__device__ __forceinline__ int warp_incl(int v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  return v;
}

// Row tiles of a group's KV head: `pairs` pairs of them, and whether one is left over.
__device__ __forceinline__ void row_tiles(int members, int M, int& pairs, int& odd) {
  const int rt = (members * M + KT - 1) / KT;
  pairs = rt >> 1;
  odd = rt & 1;
}

// One warp.
__device__ void build_meta(const SharedParams& p, const Meta& m) {
  const int lane = threadIdx.x & 31;
  const int B = p.B, ng = p.n_groups, Hp = (p.Hkv + 1) / 2;
  bool bad = false;
  for (int b = lane; b < B; b += 32) {
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
    bad |= !ok;
    m.nlen[b] = ok ? n : -1;
    m.grp[b] = 0;
  }
  bool shape_ok = true;
  for (int g = lane; g <= ng; g += 32) {
    const int v = p.group_start ? p.group_start[g] : (g ? B : 0);
    const int next = g < ng ? (p.group_start ? p.group_start[g + 1] : B) : B;
    shape_ok &= v >= 0 && v <= next && next <= B && (g > 0 || v == 0) && (g < ng || v == B);
    m.gs[g] = v;
  }
  shape_ok = __all_sync(0xffffffffu, shape_ok);
  __syncwarp();
  int c0 = 0, c1 = 0, c2 = 0;
  for (int g0 = 0; g0 < ng; g0 += 32) {
    const int g = g0 + lane;
    int steps = 0, items = 0, sc = 0;
    if (g < ng) {
      int eff = 0;
      if (shape_ok) {
        const int s0 = m.gs[g], s1 = m.gs[g + 1];
        if (s0 < s1) {
          const int shared = p.shared_len[g];
          int least = 0x7fffffff;
          for (int b = s0; b < s1; ++b) {
            m.grp[b] = g;
            if (m.nlen[b] >= 0) least = min(least, m.nlen[b]);
          }
          if (m.nlen[s0] < 0) least = 0;  // no row to read the prefix through (reported above)
          else if (shared < 0 || shared > least) {
            bad = true;
            least = 0;
          }
          eff = min(shared, least) / KT * KT;
          int pairs, odd;
          row_tiles(s1 - s0, p.M, pairs, odd);
          const int tiles = eff / KT;
          items = tiles ? p.Hkv * pairs + odd * Hp : 0;
          steps = tiles * items;
          sc = tiles * ((s1 - s0 + p.nsc - 1) / p.nsc);
        }
      }
      m.eff[g] = eff;
    }
    const int a = warp_incl(steps), b = warp_incl(items), c = warp_incl(sc);
    if (g < ng) {
      m.stepS[g] = c0 + a - steps;
      m.itemS[g] = c1 + b - items;
      m.scS[g] = c2 + c - sc;
    }
    c0 += __shfl_sync(0xffffffffu, a, 31);
    c1 += __shfl_sync(0xffffffffu, b, 31);
    c2 += __shfl_sync(0xffffffffu, c, 31);
  }
  if (lane == 0) {
    m.eff[ng] = 0;
    m.stepS[ng] = c0;
    m.itemS[ng] = c1;
    m.scS[ng] = c2;
  }
  __syncwarp();
  c0 = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    int tiles = 0;
    if (b < B && m.nlen[b] >= 0) tiles = (m.nlen[b] - m.eff[m.grp[b]] + KT - 1) / KT;
    const int a = warp_incl(tiles);
    if (b < B) {
      m.scP[b] = c0 + a - tiles;
      m.stepP[b] = (c0 + a - tiles) * Hp;
    }
    c0 += __shfl_sync(0xffffffffu, a, 31);
  }
  if (lane == 0) {
    m.scP[B] = c0;
    m.stepP[B] = c0 * Hp;
  }
  if (bad || !shape_ok) report(p.status, VG_ERR_DEVICE_BOUNDS);
  __syncwarp();
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

// A contiguous run of key tiles of one item, as one CTA works on it.
enum RunMode { kPair, kHeads, kSingle };
struct Run {
  int mode;
  int tile0, ntiles;  // key tiles of the item's range
  int row;            // sequence whose tokens locate the keys
  int tok0, ntok;     // first token of the range, tokens in it
  int seq0, rows;     // first sequence and number of query rows of the unit
  int head[2];        // KV head of each lane
  int r0[2];          // first query row of each lane
  bool priv;
  int item;           // index of its partials among the shared / private items
};

__device__ __forceinline__ Run make_run(const SharedParams& p, const Meta& m, int x, int xend) {
  Run r;
  const int Hp = (p.Hkv + 1) / 2;
  const int totS = m.stepS[p.n_groups];
  if (x < totS) {
    const int g = find(m.stepS, p.n_groups, x);
    const int tiles = m.eff[g] / KT;
    int pairs, odd;
    row_tiles(m.gs[g + 1] - m.gs[g], p.M, pairs, odd);
    const int off = x - m.stepS[g];
    const int it = off / tiles;
    r.tile0 = off - it * tiles;
    r.ntiles = min(tiles - r.tile0, xend - x);
    r.row = r.seq0 = m.gs[g];
    r.rows = (m.gs[g + 1] - m.gs[g]) * p.M;
    r.tok0 = 0;
    r.ntok = m.eff[g];
    r.priv = false;
    r.item = m.itemS[g] + it;
    const int np = p.Hkv * pairs;
    if (it < np) {
      r.mode = kPair;
      r.head[0] = r.head[1] = it / pairs;
      r.r0[0] = (it - r.head[0] * pairs) * 2 * KT;
      r.r0[1] = r.r0[0] + KT;
    } else {
      const int hp = it - np;
      r.mode = 2 * hp + 1 < p.Hkv ? kHeads : kSingle;
      r.head[0] = 2 * hp;
      r.head[1] = 2 * hp + 1;
      r.r0[0] = r.r0[1] = pairs * 2 * KT;
    }
  } else {
    const int y = x - totS;
    const int b = find(m.stepP, p.B, y);
    const int eff = m.eff[m.grp[b]];
    const int tiles = (m.nlen[b] - eff + KT - 1) / KT;
    const int off = y - m.stepP[b];
    const int hp = off / tiles;
    r.tile0 = off - hp * tiles;
    r.ntiles = min(tiles - r.tile0, xend - x);
    r.row = r.seq0 = b;
    r.rows = p.M;
    r.tok0 = eff;
    r.ntok = m.nlen[b] - eff;
    r.priv = true;
    r.item = b * Hp + hp;
    r.mode = 2 * hp + 1 < p.Hkv ? kHeads : kSingle;
    r.head[0] = 2 * hp;
    r.head[1] = 2 * hp + 1;
    r.r0[0] = r.r0[1] = 0;
  }
  return r;
}

// Ring order of a run's tiles (uses counted from the run's first): the order in which the MMA
// issuer takes them.  Pair and single: K(0), then V(n), K(n + 1).  Heads: K0(0), K1(0), then
// V0(n), K0(n + 1), V1(n), K1(n + 1).
__device__ __forceinline__ int k_use(int mode, int w, int n) {
  if (mode != kHeads) return 2 * n;
  return n == 0 ? w : 4 * n - 1 + 2 * w;
}
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
  static constexpr int NBAR = 2 * kMaxSlots + 10;  // full, empty, then s_full, p_full, q_full, o_full [2], fin
  static constexpr int TAIL = NBAR * 8 + 16;
  static constexpr int THREADS = 320;
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

// 32 columns of this thread's tensor-memory lane; the caller waits (tc_wait_ld) before use.
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Bit patterns to 32 columns of this thread's lane.
__device__ __forceinline__ void tc_st32b(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: the A operand's rows are the lanes, two bf16 a column.
__device__ __forceinline__ void tc_mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait_ab(bar, parity, status, abort));
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
                       const __grid_constant__ CUtensorMap tmV) {
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
  uint64_t* fin = s_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + C::NBAR);
  // Raised by the first wait that runs out; every later wait then gives up at once.
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* mbase = reinterpret_cast<int*>(tmem_slot + 4);
  const Meta m = meta_at(mbase, p.B, p.n_groups);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&s_full[w], 1);
      mbar_init(&p_full[w], 4);
      mbar_init(&q_full[w], 4);
      mbar_init(&o_full[w], 1);
    }
    mbar_init(fin, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) tc_alloc(tmem_slot, C::TMEM_COLS);
  pdl_wait();
  if (warp == 0) build_meta(p, m);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tmem_slot;
  if (blockIdx.x == 0) {
    const int n = meta_ints(p.B, p.n_groups);
    for (int i = threadIdx.x; i < n; i += C::THREADS) p.meta[i] = mbase[i];
  }
  pdl_launch_dependents();

  const int T = m.stepS[p.n_groups] + m.stepP[p.B];
  const int x0 = static_cast<int>(split_begin(blockIdx.x, T, p.nctas));
  const int x1 = static_cast<int>(split_begin(blockIdx.x + 1, T, p.nctas));

  if (x0 < x1 && warp == 8) {
    // ---------------------------------------------------------------- TMA producer
    // A tile is 128 / box_rows boxes (page pieces) of 64 columns: one box a lane.
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int BR = p.box_rows;
    const int box = lane / C::HALVES, half = lane % C::HALVES;
    const bool has_box = box < KT / BR;
    int u = 0;  // ring uses so far
    bool ok = true;
    for (int x = x0; ok && x < x1;) {
      const Run r = make_run(p, m, x, x1);
      x += r.ntiles;
      // slot rows of this lane's box in tile n (-1: not loaded), looked up a tile ahead
      auto lookup = [&](int n) {
        const int at = (r.tile0 + n) * KT + box * BR;
        return has_box && at < r.ntok ? box_slot(p, r.row, r.tok0 + at) : -1;
      };
      auto load = [&](const CUtensorMap* map, int head, int y) {
        const int st = u % NS;
        if (lane == 0 && u >= NS) ok = mbar_wait_ab(&empty[st], ((u / NS) - 1) & 1, p.status, abort);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) return;
        const int boxes = __popc(__ballot_sync(0xffffffffu, y >= 0));
        if (lane == 0) {
          fence_proxy_async_smem();  // the slot may hold zeros written by the generic proxy
          mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(boxes * BR * 128));
        }
        __syncwarp();
        if (y >= 0)
          tma_load_2d(ring + static_cast<size_t>(st) * C::TILE_BYTES + half * C::HALF_BYTES + box * BR * 128, map,
                      head * D + half * 64, y, &full[st]);
        ++u;
      };
      int y = lookup(0);
      load(&tmK, r.head[0], y);
      if (ok && r.mode == kHeads) load(&tmK, r.head[1], y);
      for (int n = 0; ok && n < r.ntiles; ++n) {
        const bool more = n + 1 < r.ntiles;
        const int yn = more ? lookup(n + 1) : -1;
        load(&tmV, r.head[0], y);
        if (ok && more) load(&tmK, r.head[0], yn);
        if (r.mode == kHeads) {
          if (ok) load(&tmV, r.head[1], y);
          if (ok && more) load(&tmK, r.head[1], yn);
        }
        y = yn;
      }
    }
    // no copy may still be in flight when the CTA exits (normally all were consumed)
    if (lane == 0)
      for (int i = u > NS ? u - NS : 0; i < u; ++i) mbar_wait(&full[i % NS], (i / NS) & 1, p.status);
    __syncwarp();
  } else if (x0 < x1 && warp == 9 && lane == 0) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t idS = tc_idesc_bf16(128, KT, 0, 0), idO = tc_idesc_bf16(128, D, 0, 1);
    const uint32_t qbase = smem_u32(smem), rbase = smem_u32(ring);
    int base = 0, nrun[2] = {0, 0}, np[2] = {0, 0};
    bool ok = true;
    auto wait_use = [&](int use) { return mbar_wait_ab(&full[use % NS], (use / NS) & 1, p.status, abort); };
    for (int x = x0; ok && x < x1;) {
      const Run r = make_run(p, m, x, x1);
      x += r.ntiles;
      const int lanes = r.mode == kSingle ? 1 : 2, last = r.ntiles - 1;
      auto qk = [&](int w, int n) {
        const int use = base + k_use(r.mode, w, n);
        if (!(ok = ok && wait_use(use))) return;
        tc_fence_after();
        const uint32_t ka = rbase + (use % NS) * C::TILE_BYTES, qa = qbase + w * C::TILE_BYTES;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc_mma(tm + w * 128, tc_desc_sw128(qa + (kk >> 2) * C::HALF_BYTES + (kk & 3) * 32, 16, 1024),
                 tc_desc_sw128(ka + (kk >> 2) * C::HALF_BYTES + (kk & 3) * 32, 16, 1024), idS, kk > 0 ? 1u : 0u);
        tc_commit(&s_full[w]);
        if (r.mode != kPair || w == 1) tc_commit(&empty[use % NS]);
      };
      for (int w = 0; w < lanes; ++w) {
        ok = ok && mbar_wait_ab(&q_full[w], nrun[w]++ & 1, p.status, abort);
        qk(w, 0);
      }
      for (int n = 0; ok && n < r.ntiles; ++n) {
        for (int w = 0; ok && w < lanes; ++w) {
          const int use = base + v_use(r.mode, w, n, last);
          ok = mbar_wait_ab(&p_full[w], np[w]++ & 1, p.status, abort) && wait_use(use);
          if (!ok) break;
          tc_fence_after();
          const uint32_t va = rbase + (use % NS) * C::TILE_BYTES;
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            tc_mma_ta(tm + C::COL_O + w * D, tm + w * 128 + kk * 8,
                      tc_desc_sw128(va + kk * 2048, C::HALF_BYTES, 1024), idO, (n > 0 || kk > 0) ? 1u : 0u);
          if (r.mode != kPair || w == 1) tc_commit(&empty[use % NS]);
          if (n == last) tc_commit(&o_full[w]);
          else qk(w, n + 1);
        }
      }
      base += run_uses(r.mode, r.ntiles);
    }
    tc_commit(fin);  // every MMA of this thread complete before the CTA tears down
    mbar_wait(fin, 0, p.status);
  } else if (x0 < x1 && warp < 8) {
    // ---------------------------------------------------------------- softmax lanes
    const int w = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
    const uint32_t ts = tm + (static_cast<uint32_t>(32 * quad) << 16) + w * 128;
    const uint32_t to = tm + (static_cast<uint32_t>(32 * quad) << 16) + C::COL_O + w * D;
    const float c2 = p.scale_log2;
    uint8_t* sQ = smem + w * C::TILE_BYTES;
    int base = 0, ns = 0, nr = 0;  // ring uses, tiles and runs of this lane so far
    for (int x = x0; x < x1;) {
      const Run r = make_run(p, m, x, x1);
      x += r.ntiles;
      if (r.mode == kSingle && w == 1) {
        base += run_uses(r.mode, r.ntiles);
        continue;
      }
      const int g = r.head[w], last = r.ntiles - 1;
      const int nrows = min(KT, r.rows - r.r0[w]);
      // query rows: row i of the unit is (member and verify row i / G, head i % G)
      for (int e = lane; e < 32 * (D / 8); e += 32) {
        const int i = quad * 32 + e / (D / 8), c = e % (D / 8);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (i < nrows) {
          const int rr = r.r0[w] + i;
          const int bt = rr / p.G, hh = rr - bt * p.G;
          v = *reinterpret_cast<const uint4*>(
              p.q + ((static_cast<size_t>(r.seq0) * p.R + bt) * p.Hq + g * p.G + hh) * D + c * 8);
        }
        *reinterpret_cast<uint4*>(sQ + (c >> 3) * C::HALF_BYTES + i * 128 + (((c & 7) ^ (i & 7)) << 4)) = v;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[w]);

      float mx = neg_inf(), l = 0.f;
      for (int n = 0; n < r.ntiles; ++n) {
        const int valid = r.ntok - (r.tile0 + n) * KT;  // keys of the tile (128 or more: all)
        warp_wait(&s_full[w], ns & 1, p.status, abort);
        ++ns;
        tc_fence_after();
        if (valid < KT) {
          // value rows past the range hold whatever was there: zeroed, so that 0 * V is 0.  (After
          // the wait for S: by then the issuer has seen the slot's previous use filled, so this
          // wait's parity is not that of an older phase.)
          const int use = base + v_use(r.mode, w, n, last);
          warp_wait(&full[use % NS], (use / NS) & 1, p.status, abort);
          uint8_t* vt = ring + static_cast<size_t>(use % NS) * C::TILE_BYTES;
          for (int e = quad * 32 + lane; e < C::HALVES * KT * 8; e += 128) {
            const int h = e / (KT * 8), i = (e >> 3) & (KT - 1);
            if (i >= valid)
              *reinterpret_cast<uint4*>(vt + h * C::HALF_BYTES + i * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tc_ld32(ts + 32 * c, s[c]);
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
        float t = neg_inf();
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            asm volatile("" : "+r"(s[c][k]));  // (no use before the wait)
            if (valid < KT && 32 * c + k >= valid) s[c][k] = 0xff800000u;
            t = fmaxf(t, __uint_as_float(s[c][k]));
          }
        t *= c2;
        const bool first = n == 0;
        const float mn = first || t > mx + kRescaleSlack ? fmaxf(mx, t) : mx;
        const bool resc = !first && mn != mx;
        if (__any_sync(0xffffffffu, resc)) {
          // rare: the running max rises (P V of the lane's previous tile has completed: the
          // commit that brought this S came after it)
          const float alpha = resc ? ex2(mx - mn) : 1.f;
          l *= alpha;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            float o[32];
            tc_ld32_sync(to + c0, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] *= alpha;
            tc_st32(to + c0, o);
          }
        }
        mx = mn;
        float ls = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            const uint32_t a = s[2 * h + (k >> 5)][k & 31], b = s[2 * h + (k >> 5)][(k & 31) + 1];
            // the sum takes the bf16 values that P V multiplies: a row's weights sum to one up
            // to fp32 rounding, and what bf16 leaves off a dominant weight cancels
            pk[k / 2] = pack_bf16(ex2(fmaf(__uint_as_float(a), c2, -mx)), ex2(fmaf(__uint_as_float(b), c2, -mx)));
            ls = add_bf16x2_f32(pk[k / 2], ls);
          }
          tc_st32b(ts + 32 * h, pk);
        }
        l += ls;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[w]);
      }
      // the run's partial: (O, max, sum) of each row once P V of its last tile has landed
      warp_wait(&o_full[w], nr & 1, p.status, abort);
      ++nr;
      tc_fence_after();
      const size_t prow =
          r.priv ? (static_cast<size_t>(blockIdx.x + r.item) * 2 + w) * p.Mpad + row
                 : (static_cast<size_t>(blockIdx.x + r.item) * 2 + w) * KT + row;
      float* po = (r.priv ? p.partp_o : p.parts_o) + prow * D;
      if (32 * quad < nrows) {
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
          tc_ld32_sync(to + c0, o);
          if (row < nrows) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(po + c0 + k) = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          }
        }
        if (row < nrows) *reinterpret_cast<float2*>((r.priv ? p.partp_ml : p.parts_ml) + prow * 2) = make_float2(mx, l);
      }
      tc_fence_before();
      base += run_uses(r.mode, r.ntiles);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tc_dealloc(tm, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- combine
// One warp per output row, lanes across d: the partials of the row's shared item by CTA, of
// its private item by CTA, then its causal keys u = 0 .. t: a fixed order.
constexpr int kCombWarps = 8;

template <int D>
__global__ void __launch_bounds__(kCombWarps * 32) shared_combine_kernel(const SharedParams p) {
  constexpr int PER = D / 32;
  __shared__ float lgs[kCombWarps][16];
  __shared__ __align__(16) __nv_bfloat16 kvs[2][16][D];
  pdl_launch_dependents();
  pdl_wait();
  const Meta m = meta_at(p.meta, p.B, p.n_groups);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rblocks = (p.M + kCombWarps - 1) / kCombWarps;
  const int bg = blockIdx.x / rblocks, r0 = (blockIdx.x - bg * rblocks) * kCombWarps;
  const int r = r0 + warp, g = bg % p.Hkv, b = bg / p.Hkv;
  const int n = m.nlen[b];
  if (n < 0) return;  // the whole CTA
  const bool active = r < p.M;
  const int t = active ? r / p.G : 0, jh = r - t * p.G;
  const int tmax = min(p.M - 1, r0 + kCombWarps - 1) / p.G;
  constexpr int CH = D / 8;
  for (int e = tid; e < 2 * (tmax + 1) * CH; e += kCombWarps * 32) {
    const int which = e / ((tmax + 1) * CH), rem = e - which * (tmax + 1) * CH;
    const int u = rem / CH, c = rem - u * CH;
    const __nv_bfloat16* fresh = which ? p.v_new : p.k_new;
    const __nv_bfloat16* src = nullptr;
    if (fresh) {
      src = fresh + ((static_cast<size_t>(b) * p.R + u) * p.Hkv + g) * D;
    } else {
      const int64_t slot = kv_slot(p.seq_offset, p.ptab, p.psize, p.pstride, p.capacity, b, n + u);
      if (slot >= 0) src = (which ? p.V : p.K) + (slot * p.Hkv + g) * D;
    }
    reinterpret_cast<uint4*>(&kvs[which][u][0])[c] =
        src ? reinterpret_cast<const uint4*>(src)[c] : make_uint4(0u, 0u, 0u, 0u);
  }
  // where the row's partials are: shared ones from CTA cs on, private ones from CTA cp on
  const int grp = m.grp[b], Hp = (p.Hkv + 1) / 2;
  const int totS = m.stepS[p.n_groups];
  const int T = totS + m.stepP[p.B];
  int cs = 0, nS = 0, cp = 0, nP = 0;
  size_t baseS = 0, strideS = 2 * KT, baseP = 0;
  if (active) {
    const int tiles = m.eff[grp] / KT;
    if (tiles > 0) {
      int pairs, odd;
      row_tiles(m.gs[grp + 1] - m.gs[grp], p.M, pairs, odd);
      const int rr = (b - m.gs[grp]) * p.M + r, rt = rr / KT;
      int it, w;
      if ((rt >> 1) < pairs) {
        it = g * pairs + (rt >> 1);
        w = rt & 1;
      } else {
        it = p.Hkv * pairs + (g >> 1);
        w = g & 1;
      }
      const int s0 = m.stepS[grp] + it * tiles;
      cs = static_cast<int>(owner_cta(s0, T, p.nctas));
      nS = static_cast<int>(owner_cta(s0 + tiles - 1, T, p.nctas)) - cs + 1;
      baseS = (static_cast<size_t>(cs + m.itemS[grp] + it) * 2 + w) * KT + (rr - rt * KT);
    }
    const int ptiles = (n - m.eff[grp] + KT - 1) / KT;
    if (ptiles > 0) {
      const int s0 = totS + m.stepP[b] + (g >> 1) * ptiles;
      cp = static_cast<int>(owner_cta(s0, T, p.nctas));
      nP = static_cast<int>(owner_cta(s0 + ptiles - 1, T, p.nctas)) - cp + 1;
      baseP = (static_cast<size_t>(cp + b * Hp + (g >> 1)) * 2 + (g & 1)) * p.Mpad + r;
    }
  }
  const int nseg = nS + nP;
  // (a CTA between the first and the last has steps of the item: T >= nctas there, or it is
  // skipped as empty)
  auto nonempty = [&](int i) { return split_nonempty(i < nS ? cs + i : cp + i - nS, T, p.nctas); };
  auto prow = [&](int i) {
    return i < nS ? baseS + static_cast<size_t>(i) * strideS : baseP + static_cast<size_t>(i - nS) * 2 * p.Mpad;
  };
  float qv[PER];
  if (active) {
    const __nv_bfloat16* qrow = p.q + ((static_cast<size_t>(b) * p.R + t) * p.Hq + g * p.G + jh) * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) qv[e] = __bfloat162float(qrow[e]);
  }
  __syncthreads();
  if (!active) return;
  float* lg = lgs[warp];
  float M = neg_inf();
  for (int u = 0; u <= t; ++u) {
    float acc = 0.f;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc += qv[e] * __bfloat162float(kvs[0][u][lane * PER + e]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    acc *= p.scale_log2;
    M = fmaxf(M, acc);
    if (lane == 0) lg[u] = acc;
  }
  __syncwarp();
  auto load_ml = [&](int i, float& ms, float& ls) {
    ms = neg_inf();
    ls = 0.f;
    if (i < nseg && nonempty(i)) {
      const float2 v = *reinterpret_cast<const float2*>((i < nS ? p.parts_ml : p.partp_ml) + prow(i) * 2);
      ms = v.x;
      ls = v.y;
    }
  };
  float pm, pl;
  load_ml(lane, pm, pl);
  float pmax = pm;
  for (int s0 = 32; s0 < nseg; s0 += 32) {
    float ms, ls;
    load_ml(s0 + lane, ms, ls);
    pmax = fmaxf(pmax, ms);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) pmax = fmaxf(pmax, __shfl_xor_sync(0xffffffffu, pmax, off));
  M = fmaxf(M, pmax);
  float acc[PER] = {}, l = 0.f;
  for (int s0 = 0; s0 < nseg; s0 += 32) {
    float ms = pm, ls = pl;
    if (s0 > 0) load_ml(s0 + lane, ms, ls);
    const float wgt = ms != neg_inf() ? ex2(ms - M) : 0.f;
    float wl = wgt * ls;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) wl += __shfl_xor_sync(0xffffffffu, wl, off);
    l += wl;
    const int cnt = min(32, nseg - s0);
    for (int q0 = 0; q0 < cnt; q0 += 4) {
      float v[4][PER];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = s0 + q0 + q;
        const bool have = i < nseg && nonempty(i);
        const float* src = (i < nS ? p.parts_o : p.partp_o) + (have ? prow(i) : 0) * D + lane * PER;
#pragma unroll
        for (int e = 0; e < PER; e += 2) {
          const float2 x = have ? *reinterpret_cast<const float2*>(src + e) : make_float2(0.f, 0.f);
          v[q][e] = x.x;
          v[q][e + 1] = x.y;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float wq = __shfl_sync(0xffffffffu, wgt, (q0 + q) & 31);
        if (q0 + q < cnt) {
#pragma unroll
          for (int e = 0; e < PER; ++e) acc[e] += wq * v[q][e];
        }
      }
    }
  }
  for (int u = 0; u <= t; ++u) {
    const float wu = ex2(lg[u] - M);
    l += wu;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] += wu * __bfloat162float(kvs[1][u][lane * PER + e]);
  }
  const float inv = 1.f / l;
  __nv_bfloat16* o = p.out + ((static_cast<size_t>(b) * p.R + t) * p.Hq + g * p.G + jh) * D + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; ++e) o[e] = __float2bfloat16_rn(acc[e] * inv);
  if (p.k_new && jh == 0) {  // append verify row t
    const int64_t slot = kv_slot(p.seq_offset, p.ptab, p.psize, p.pstride, p.capacity, b, n + t);
    if (slot >= 0) {
      const size_t dst = (slot * p.Hkv + g) * D + lane * PER;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        p.K[dst + e] = kvs[0][t][lane * PER + e];
        p.V[dst + e] = kvs[1][t][lane * PER + e];
      }
    }
  }
}

// ---------------------------------------------------------------- scores
// scores[b][i] = scale * sum over the mask's rows and all heads of q . K_i = scale * sum over
// KV heads g of Q_b,g . K_i,g with Q_b,g the sum of the sequence's masked query rows of head g.
// Q is fp32; it enters the tensor cores as three bf16 parts whose sum is Q to 2^-24.
__global__ void __launch_bounds__(128) shared_qsum_kernel(const SharedParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int b = blockIdx.x / p.Hkv, g = blockIdx.x - b * p.Hkv, d = threadIdx.x;
  if (d >= p.D) return;
  float acc = 0.f;
  for (uint32_t bits = p.mask; bits != 0u; bits &= bits - 1u) {
    const int t = __ffs(bits) - 1;
    const __nv_bfloat16* src = p.q + ((static_cast<size_t>(b) * p.R + t) * p.Hq + g * p.G) * p.D + d;
    for (int h = 0; h < p.G; ++h) acc += __bfloat162float(src[h * p.D]);
  }
  const size_t width = static_cast<size_t>(p.Hkv) * p.D, part = static_cast<size_t>(p.Bpad) * width;
  __nv_bfloat16* dst = p.qsum + b * width + g * p.D + d;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const __nv_bfloat16 h = __float2bfloat16_rn(acc);
    dst[k * part] = h;
    acc -= __bfloat162float(h);
  }
}

// One item is a tile of 128 keys and up to N members: S^T[keys][members] on the tensor cores
// (the keys are the M rows, so few members cost little), one KV head at a time into a double
// buffer; four warps add the heads' tiles in fp32 registers (the tensor core's own sum runs
// over one head only) and write rows of consecutive positions.
template <int D, int N>
struct ZCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int HALF_BYTES = KT * 128;
  static constexpr int K_BYTES = KT * D * 2;
  static constexpr int PART = N * D * 2;
  static constexpr int STAGE = K_BYTES + 3 * PART;
  static constexpr int NST = 163840 / STAGE > 6 ? 6 : 163840 / STAGE;
  static constexpr int NBAR = 2 * NST + 6;
  static constexpr int THREADS = 192;
  static constexpr uint32_t TMEM_COLS = 2 * N < 32 ? 32 : 2 * N;
  static size_t smem(int meta) { return 1024 + NST * STAGE + NBAR * 8 + 16 + 4 * static_cast<size_t>(meta); }
};

template <int D, int N>
__global__ void __launch_bounds__(ZCfg<D, N>::THREADS, 1)
    shared_score_kernel(const SharedParams p, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmZ) {
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
      mbar_init(&full[s], 1);
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
  if (warp == 0) build_meta(p, m);
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
    i.cols = (i.members + 15) & ~15;
    return i;
  };
  if (warp == 4) {
    const int BR = p.box_rows, box = lane / C::HALVES, half = lane % C::HALVES;
    int u = 0;
    bool ok = true;
    for (int x = blockIdx.x; ok && x < T; x += gridDim.x) {
      const Item it = item(x);
      const int at = it.tile * KT + box * BR;
      const int y = box < KT / BR && at < it.ntok ? box_slot(p, it.row, it.tok0 + at) : -1;
      const int boxes = __popc(__ballot_sync(0xffffffffu, y >= 0));
      const int zb = it.cols / 16 * 3 * C::HALVES;  // boxes of 16 members of a part, 64 columns
      for (int g = 0; ok && g < p.Hkv; ++g, ++u) {
        const int st = u % C::NST;
        if (lane == 0 && u >= C::NST) ok = mbar_wait_ab(&empty[st], ((u / C::NST) - 1) & 1, p.status, abort);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(boxes * BR * 128 + zb * 16 * 128));
        __syncwarp();
        uint8_t* dst = smem + st * C::STAGE;
        if (y >= 0) tma_load_2d(dst + half * C::HALF_BYTES + box * BR * 128, &tmK, g * D + half * 64, y, &full[st]);
        for (int e = lane; e < zb; e += 32) {
          const int h = e % C::HALVES, q = e / C::HALVES, part = q % 3, blk = q / 3;
          tma_load_2d(dst + C::K_BYTES + part * C::PART + h * (N * 128) + blk * 16 * 128, &tmZ, g * D + h * 64,
                      part * p.Bpad + it.seq0 + blk * 16, &full[st]);
        }
      }
    }
    if (lane == 0)
      for (int i = u > C::NST ? u - C::NST : 0; i < u; ++i) mbar_wait(&full[i % C::NST], (i / C::NST) & 1, p.status);
    __syncwarp();
  } else if (warp == 5 && lane == 0) {
    int u = 0;
    bool ok = true;
    const uint32_t base = smem_u32(smem);
    for (int x = blockIdx.x; ok && x < T; x += gridDim.x) {
      const Item it = item(x);
      const uint32_t id = tc_idesc_bf16(128, it.cols, 0, 0);
      for (int g = 0; ok && g < p.Hkv; ++g, ++u) {
        const int st = u % C::NST;
        ok = mbar_wait_ab(&full[st], (u / C::NST) & 1, p.status, abort) &&
             (u < 2 || mbar_wait_ab(&s_free[u & 1], ((u - 2) >> 1) & 1, p.status, abort));
        if (!ok) break;
        tc_fence_after();
        const uint32_t ka = base + st * C::STAGE, za = ka + C::K_BYTES;
        // smallest part first: the large sum is rounded into last
#pragma unroll
        for (int part = 2; part >= 0; --part)
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc_mma(tm + (u & 1) * N, tc_desc_sw128(ka + (kk >> 2) * C::HALF_BYTES + (kk & 3) * 32, 16, 1024),
                   tc_desc_sw128(za + part * C::PART + (kk >> 2) * (N * 128) + (kk & 3) * 32, 16, 1024), id,
                   (part < 2 || kk > 0) ? 1u : 0u);
        tc_commit(&s_full[u & 1]);
        tc_commit(&empty[st]);
      }
    }
    tc_commit(fin);  // every MMA of this thread complete before the CTA tears down
    mbar_wait(fin, 0, p.status);
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
            uint32_t v[16];
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
                "tcgen05.wait::ld.sync.aligned;"
                : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                  "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                : "r"(tl + (u & 1) * N + c)
                : "memory");
#pragma unroll
            for (int k = 0; k < 16; ++k) acc[c + k] += __uint_as_float(v[k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[u & 1]);
      }
      const int at = it.tile * KT + 32 * warp + lane;
      if (at < it.ntok) {
        float* dst = p.scores + it.tok0 + at;
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (k < it.members && m.nlen[it.seq0 + k] >= 0)
            dst[static_cast<size_t>(it.seq0 + k) * p.score_stride] = acc[k] * p.scale;
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
cudaError_t launch_scores(const SharedParams& p, const CUtensorMap& tmK, const CUtensorMap& tmZ, cudaStream_t stream) {
  using C = ZCfg<D, N>;
  const size_t smem = C::smem(meta_ints(p.B, p.n_groups));
  cudaError_t e = ensure_smem<shared_score_kernel<D, N>>(smem);
  if (e != cudaSuccess) return e;
  Launch q(p.B * p.Hkv, 128, 0, stream);
  if ((e = cudaLaunchKernelEx(&q.cfg, shared_qsum_kernel, p)) != cudaSuccess) return e;
  Launch z(p.nctas, C::THREADS, smem, stream);
  return cudaLaunchKernelEx(&z.cfg, shared_score_kernel<D, N>, p, tmK, tmZ);
}

template <int D>
cudaError_t launch_shared_t(const SharedParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                            const CUtensorMap& tmZ, cudaStream_t stream) {
  cudaError_t e;
  if (p.mask) {
    e = p.nsc == 16 ? launch_scores<D, 16>(p, tmK, tmZ, stream) : launch_scores<D, 64>(p, tmK, tmZ, stream);
    if (e != cudaSuccess) return e;
  }
  using C = SCfg<D>;
  const size_t smem = C::smem(p.nslots, meta_ints(p.B, p.n_groups));
  if ((e = ensure_smem<shared_attn_kernel<D>>(smem)) != cudaSuccess) return e;
  Launch a(p.nctas, C::THREADS, smem, stream);
  if ((e = cudaLaunchKernelEx(&a.cfg, shared_attn_kernel<D>, p, tmK, tmV)) != cudaSuccess) return e;
  Launch c(p.B * p.Hkv * ((p.M + kCombWarps - 1) / kCombWarps), kCombWarps * 32, 0, stream);
  return cudaLaunchKernelEx(&c.cfg, shared_combine_kernel<D>, p);
}

}  // namespace

int shared_meta_ints(int B, int n_groups) { return meta_ints(B, n_groups); }

int shared_slots(int D, int B, int n_groups, size_t smem_optin) {
  const int n = meta_ints(B, n_groups);
  return D == 64 ? SCfg<64>::slots(n, smem_optin) : SCfg<128>::slots(n, smem_optin);
}

cudaError_t launch_shared(const SharedParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                          const CUtensorMap& tmZ, cudaStream_t stream) {
  return p.D == 64 ? launch_shared_t<64>(p, tmK, tmV, tmZ, stream) : launch_shared_t<128>(p, tmK, tmV, tmZ, stream);
}

}  // namespace vg
