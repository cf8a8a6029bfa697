// The attention kernel of the calls with tall row matrices: shared prefixes (shared_attn.cu) and trees
// (tree_attn.cu).  A Plan names the call's parameters and finds the runs of a CTA.
//
// Attention kernel.  One persistent CTA per SM; the Plan deals the steps out: the flattened list of them is split
// evenly over the CTAs, or, for trees with several units a head, pieces of ranges (tasks) go round.  A CTA has two
// "lanes" of eight softmax warps, each with its own 128 rows, S / P and O in tensor memory; a step is one key tile for
// both lanes:
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
// (Plan::kScores: while they wait for S, the softmax warps multiply the keys of some runs with the heads' summed queries.  A ring slot
// then takes sixteen more arrivals: theirs, or at once the producer's.)
// A tree's runs (Plan::kTree) end inside a key tile, and their last tokens, the nodes, are attended
// by the bit sets of the rows' nodes.  A run that holds an item's whole key range writes the
// output itself; partials are two a CTA at most: of its first run and its last, or, where tasks go round and
// ranges are cut, of its two tasks.
#pragma once

#include "vg_common.cuh"
#include "vg_internal.h"

namespace vg {
namespace {

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)), "r"(n)
               : "memory");
}

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
  int n;              // tree: tokens of the prefix, before the nodes
  bool whole;         // tree: the item's whole key range
  int z;              // tree: bit w: the keys of lane w's head are scored in this run
};

// A run as the planner leaves it in shared memory, in a ring of kRuns.
constexpr int kRuns = 4;
struct __align__(16) RunRec {
  int mode, ntiles, tile0, ntok;  // ntiles -1: no further run
  int tok0, row, rows, priv;
  int head[2], r0[2];
  int unit;  // of its partials (for lane 0)
  int low, n, whole;  // (n, whole, z: trees)
  int z, pad[3];
};
static_assert(sizeof(RunRec) % 16 == 0, "");

// Ring order of a run's tiles (uses counted from the run's first): the order in which the MMA
// issuer takes them.  Pair and single: K(0), then V(n), K(n + 1).  Heads: K0(0), K1(0), then
// V0(n), K0(n + 1), V1(n), K1(n + 1).
__device__ __forceinline__ int v_use(int mode, int w, int n, int last) {
  if (mode != kHeads) return 2 * n + 1;
  return w == 0 ? 4 * n + 2 : (n < last ? 4 * n + 4 : 4 * n + 3);
}
__device__ __forceinline__ int k_use(int mode, int w, int n) {
  return mode != kHeads ? 2 * n : n == 0 ? w : 4 * n - 1 + 2 * w;
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

// Two bf16, 0 in place of one that is not finite.
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  const uint32_t is = ~x & 0x7f807f80u;  // (a half of 0: not finite)
  return x & (((is & 0xffffu) ? 0xffffu : 0u) | ((is >> 16) ? 0xffff0000u : 0u));
}

// A tree's value tile, by a lane's 256 threads: rows from `left` on become 0, and so do elements that are not finite of the rows from
// `nodes` on, for the rows that do not attend them (the others have them added at the end: *odd).
template <int HALVES>
__device__ __noinline__ void clear_values(uint8_t* tile, int nodes, int left, volatile int* odd) {
  for (int e = (threadIdx.x & 255) + nodes * 8; e < KT * 8; e += 256) {
    const int i = e >> 3;
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      uint4* x = reinterpret_cast<uint4*>(tile + h * (KT * 128) + e * 16);
      if (i >= left) {
        *x = make_uint4(0u, 0u, 0u, 0u);
        continue;
      }
      const uint4 v = *x;
      const uint4 f = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
      if (f.x != v.x || f.y != v.y || f.z != v.z || f.w != v.w) {
        *odd = 1;
        __threadfence_block();  // (who finds the zeros finds that)
        *x = f;
      }
    }
  }
  fence_proxy_async_smem();
}

// The products of keys m0 .. m0 + 7 of a tile (as TMA left it at `tile`) with a summed query, for the first `count` keys of the
// tile.  One warp: lane l takes a quarter of key l % 8, so that eight lanes' 16 bytes lie in different banks.  (On the warp-level
// tensor path, 16 keys a warp, the small products wait for the large ones: 16 trees of 64 nodes 293 us.)
template <int D>
__device__ __forceinline__ void score_keys(uint32_t tile, const float* z, float* dst, int m0, int count) {
  const int lane = threadIdx.x & 31, row = m0 + (lane & 7), q = lane >> 3;
  float acc[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int chunk = q * (D / 32) + i;  // 16 bytes of a row; 8 to a half of the tile
    uint32_t x[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(tile + (chunk >> 3) * (KT * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)));
    const float4 z0 = reinterpret_cast<const float4*>(z)[2 * chunk], z1 = reinterpret_cast<const float4*>(z)[2 * chunk + 1];
    const float zs[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[0] = fmaf(__uint_as_float(x[e] << 16), zs[2 * e], acc[0]);
      acc[1] = fmaf(__uint_as_float(x[e] & 0xffff0000u), zs[2 * e + 1], acc[1]);
    }
  }
  float sum = acc[0] + acc[1];
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  sum += __shfl_xor_sync(0xffffffffu, sum, 16);
  if (lane < 8 && row < count) dst[row] = sum;
}

template <int D, class Plan>
__global__ void __launch_bounds__(SCfg<D>::THREADS, 1)
    lane_attn_kernel(const typename Plan::Params p, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ) {
  using C = SCfg<D>;
  constexpr bool TREE = Plan::kTree, SCORES = Plan::kScores;
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
  volatile int* odd = reinterpret_cast<volatile int*>(tmem_slot + 2);  // tree: a node's value has not been finite
  RunRec* recs = reinterpret_cast<RunRec*>(tmem_slot + 4);
  int* mbase = reinterpret_cast<int*>(recs + kRuns);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 2);
      mbar_init(&empty[s], 2 + (SCORES ? 16 : 0));
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
    *odd = 0;
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
    Plan::load(p, mbase, C::THREADS);
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
    int x, x1, planned = 0;
    Plan::steps(p, mbase, x, x1);
    bool ended = false;
    auto plan = [&] {
      if (ended) return true;
      RunRec out{kPair, -1, 0, 0, 0, 0, 0, 0, {0, 0}, {0, 0}, 0, 0, 0, 0, 0, {0, 0, 0}};
      while (x < x1 && out.ntiles <= 0) {
        const Run r = Plan::next(p, mbase, x, x1);
        out = RunRec{r.mode, r.ntiles, r.tile0, r.ntok, r.tok0, r.row, r.rows, r.priv, {r.head[0], r.head[1]},
                     {r.r0[0], r.r0[1]}, Plan::unit(r), r.low, r.n, r.whole, r.z, {0, 0, 0}};
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
    const int lw = warp == 18 ? 1 : 0;  // this warp brings the query tiles of that lane
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
    auto load = [&](const CUtensorMap* map, int head, int y, bool scored) {
      if (lap > 0) ok = warp_wait(&empty[st], (lap - 1) & 1, p.status, abort);
      if (!ok) return;
      const uint32_t have = __ballot_sync(0xffffffffu, y >= 0);
      if (leader) {
        if (zeros) fence_proxy_async_smem();
        mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(__popc(have) * BR * 128));
        if (SCORES && !scored && lw == 0) mbar_arrive_n(&empty[st], 16);
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
      if (ok) load(&tmK, r.head[0], y, r.z != 0);
      if (ok && r.mode == kHeads) load(&tmK, r.head[1], y, r.z != 0);
      for (int n = 0; ok && n < r.ntiles; ++n) {
        const bool more = n + 1 < r.ntiles;
        const int w2 = word(n + 2);
        if (TREE) zeros |= (r.tile0 + n) * KT > r.n;  // (the tile before this one had nodes)
        load(&tmV, r.head[0], y, false);
        const int yn = slot_row(n + 1, w1);
        if (ok && more) load(&tmK, r.head[0], yn, r.z != 0);
        if (r.mode == kHeads) {
          if (ok) load(&tmV, r.head[1], y, false);
          if (ok && more) load(&tmK, r.head[1], yn, r.z != 0);
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
    const RunRec* rec = recs;
    // Maximum (log2 units) of this thread's whole row of S in a tile with `left` keys of the range from token
    // `tok` on.
    auto row_max = [&](int left, int tok, bool nodes) {
      uint64_t b[2] = {~uint64_t{0}, ~uint64_t{0}};
      if (TREE && nodes) {
        b[0] = Plan::bits(p, *rec, rec->r0[w] + row, tok);
        b[1] = Plan::bits(p, *rec, rec->r0[w] + row, tok + HK);
      }
      float t = neg_inf();
#pragma unroll 1
      for (int c0 = 0; c0 < KT; c0 += 32) {
        float v[32];
        tc_ld32_sync(ts + c0, v);
        const uint32_t x = static_cast<uint32_t>(b[c0 >> 6] >> (c0 & 32));
#pragma unroll
        for (int i = 0; i < 32; ++i)
          t = fmaxf(t, (TREE ? (x >> i & 1u) != 0 : c0 + i < left) ? v[i] : neg_inf());
      }
      return t * c2;
    };
    int base = 0, ns = 0, nr = 0;  // ring uses, tiles and runs of this lane so far
    // Run -1 takes a tile of whatever tensor memory holds through the code, without a wait, an
    // arrival or a store, while the previous kernel ends and the first tiles are on their way:
    // the first real tile then finds its instructions in the caches (it took 11,000 cycles to
    // go from S to P without that, of a decode step's 75,000).
    for (int k = -1;; ++k) {
      const bool real = k >= 0;
      if (k == 0) begin();
      int mode = kPair, last = 0, keys = KT, nrows = KT, end = KT, prefix = KT;
      if (real) {
        rec = run_at(k);
        // (the two warps of a pair meet at named barriers, which have no limit: after a lost wait they
        // leave together)
        if (named_bar_or(pair_bar, 64, rec == nullptr)) break;
        mode = rec->mode;
        last = rec->ntiles - 1;
        keys = rec->ntok - rec->tile0 * KT;
        nrows = min(p.RT, rec->rows - rec->r0[w]);
        end = rec->ntok;
        prefix = rec->n;
        if (mode == kSingle && w == 1) {
          base += run_uses(mode, last + 1);
          run_done(k);
          continue;
        }
      }
      const bool live = 32 * quad < nrows;  // (a warp without query rows only keeps the barriers' count)
      float mx = neg_inf(), l = 0.f;        // the maximum in use (log2 units), this half's sum
      bool bare = false;                    // tree: a row of these warps has perhaps nothing that weighs anything yet
      for (int n = 0; n <= last; ++n) {
        const int left = keys - n * KT;  // keys of the tile (128 or more: all)
        // S is awaited, and in the meantime the keys are scored (a pair's two lanes share the tile).  A run's first
        // tile only after its S: a lane may have left out runs before, and a wait for its keys would not know their lap (see
        // filled)
        auto await_s = [&] { warp_wait(&s_full[w], ns++ & 1, p.status, abort); };
        if (real && (!SCORES || n == 0)) await_s();
        if (SCORES && real && rec->z != 0) {
          const int use = base + k_use(mode, w, n), slot = use % NS, tok = end - left, count = prefix - tok;
          if (filled(full, empty, slot, use / NS, p.status, abort) && count > 0) {
            const uint32_t tile = smem_u32(ring) + slot * C::TILE_BYTES;
            const float* z = Plan::sums(p, *rec, rec->head[w]);
            float* dst = Plan::scores(p, *rec, rec->head[w]) + tok;
            const int i = warp & 7;
            score_keys<D>(tile, z, dst, 8 * (mode == kPair ? 8 * w + i : i), count);
            if (mode != kPair) score_keys<D>(tile, z, dst, 64 + 8 * i, count);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive_n(&empty[slot], mode == kPair ? 1 : 2);
        }
        if (SCORES && real && n > 0) await_s();
        tc_fence_after();
        const int tok = end - left;  // the tile's first token
        // tree: a tile that reaches into the nodes is masked by the row's bits, else by the range's end
        const bool nodes = TREE && real && tok + KT > prefix;
        // value rows past the range hold whatever was there: zeroed, so that 0 * V is 0 (after
        // the wait for S, which orders this tile's V within NS uses of its K: see filled)
        if (TREE ? nodes : left < KT) {
          const int use = base + v_use(mode, w, n, last);
          filled(full, empty, use % NS, use / NS, p.status, abort);
          uint8_t* vt = ring + static_cast<size_t>(use % NS) * C::TILE_BYTES;
          if constexpr (TREE) {
            clear_values<C::HALVES>(vt, max(prefix - tok, 0), left, odd);
          } else {
            for (int e = threadIdx.x & 255; e < C::HALVES * KT * 8; e += 256) {
              const int h = e / (KT * 8), i = (e >> 3) & (KT - 1);
              if (i >= left)
                *reinterpret_cast<uint4*>(vt + h * C::HALF_BYTES + i * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
        }
        if (!live) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[w]);
          continue;
        }
        const int valid = left - HK * half;  // keys of this half (64 or more: all)
        uint64_t bits = ~uint64_t{0};
        if (TREE && nodes) bits = Plan::bits(p, *rec, rec->r0[w] + row, tok + HK * half);
        uint32_t pk[HK / 2];
        auto load_s = [&](float (&s)[HK]) {
          tc_ld64_sync(ts + HK * half, s);
          if (TREE) {
            if (nodes) {
#pragma unroll
              for (int i = 0; i < HK; ++i)
                if (!((i < 32 ? static_cast<uint32_t>(bits) : static_cast<uint32_t>(bits >> 32)) >> (i & 31) & 1u))
                  s[i] = neg_inf();
            }
          } else if (valid < HK) {
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
          // (bare: of a half, which a row's other half may make up for; the next tile settles it)
          bare = named_bar_or(pair_bar, 64, TREE && row < nrows && t == neg_inf()) && TREE;
          tc_fence_after();
          mx = fmaxf(t, tc_ld1_sync(to_other));
        } else if (TREE && bare) {
          // (O is in use: each thread reads its row's whole tile.  What such a row has of O is 0)
          const float t = row_max(left, tok, nodes);
          if (mx == neg_inf()) mx = t;
          bare = named_bar_or(pair_bar, 64, row < nrows && mx == neg_inf());
        }
        float ls = 0.f;
        for (bool raised = false;; raised = true) {
          // P = 2^(s c2 - mx) of this half, and its sum, of the bf16 values that P V multiplies: a row's
          // weights sum to one
          float s[HK];
          load_s(s);
          const float ref = TREE && mx == neg_inf() ? 0.f : mx;  // (nothing attended yet: every P is 0)
          float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < HK; i += 2) {
            const float2 e = fma2(make_float2(s[i], s[i + 1]), make_float2(c2, c2), make_float2(-ref, -ref));
            pk[i / 2] = pack_bf16(ex2(e.x), ex2(e.y));
            a4[(i >> 1) & 3] = add_bf16x2_f32(pk[i / 2], a4[(i >> 1) & 3]);
          }
          ls = (a4[0] + a4[1]) + (a4[2] + a4[3]);
          // (both threads of each row have read S after the barrier: P may overwrite it)
          if (!named_bar_or(pair_bar, 64, row < nrows && ls > kMostSum) || raised) break;
          // rare: the row's maximum over the whole tile, which both threads of the row read for
          // themselves, becomes the one in use; then P again.  (A sum of 64 beyond kMostSum has a P of
          // 4 or more in it: two above the maximum in use)
          const float t = row_max(left, tok, nodes);
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
          const float ref = TREE && mx == neg_inf() ? 0.f : mx;
          auto in = [&](int i) { return TREE ? (bits >> i & 1u) != 0 : i < valid; };
#pragma unroll 1
          for (int c0 = 0; c0 < HK; c0 += 16) {
            float v[16];
            uint32_t part[16];
            tc_ld16_sync(ts + HK * half + c0, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float p0 = in(c0 + 2 * i) ? ex2(fmaf(v[2 * i], c2, -ref)) : 0.f;
              const float p1 = in(c0 + 2 * i + 1) ? ex2(fmaf(v[2 * i + 1], c2, -ref)) : 0.f;
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
      if (TREE && live && rec->whole) {
        // half a row of the output a thread.  The row's sum is both halves', exchanged like the first maximum: by the first
        // column of each half of O, which has been read by then
        __nv_bfloat16* dst = Plan::out(p, *rec, rec->r0[w] + row, w) + half * (D / 2);
        float inv = 0.f;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2; c0 += 32) {
          float o[32];
          tc_ld32_sync(to + c0, o);
          if (c0 == 0) {
            tc_st1(to_mine, l);
            tc_wait_st();
            tc_fence_before();
            named_bar(pair_bar, 64);
            tc_fence_after();
            const float sum = l + tc_ld1_sync(to_other);
            inv = sum > 0.f ? 1.f / sum : 0.f;
          }
          if (row < nrows) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(dst + c0 + i) =
                  make_uint4(pack_bf16(o[i] * inv, o[i + 1] * inv), pack_bf16(o[i + 2] * inv, o[i + 3] * inv),
                             pack_bf16(o[i + 4] * inv, o[i + 5] * inv), pack_bf16(o[i + 6] * inv, o[i + 7] * inv));
          }
        }
        if constexpr (TREE) {
          if (*odd != 0 && row < nrows)
            Plan::add_odd(p, rec->row, (rec->r0[w] + row) / p.G, rec->head[w], half * (D / 2), D / 2, dst);
          __syncwarp();
        }
      } else if (live) {
        // four columns of 32 rows lie together: a warp's stores are 512 contiguous bytes
        const bool priv = !TREE && rec->priv != 0;
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
  if constexpr (TREE) {
    if (threadIdx.x == 0) Plan::leave_odd(p, *odd);
  }
  if (warp == 17) {
    tc_fence_after();
    tc_dealloc(tm, C::TMEM_COLS);
  }
}

}  // namespace
}  // namespace vg
