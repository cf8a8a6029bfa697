// Verification attention for trees of drafted tokens.
//
// A node attends the whole prefix and, of the nodes, those that its bit set names.  Both lie one
// after the other in the sequence's slots or pages, so a row's softmax runs over one range of prefix_len + len
// tokens whose last len are masked by bits.  Per KV head a sequence's nodes form a matrix of len * G
// query rows, cut into tiles of 128 and multiplied with tiles of 128 keys on the tensor cores
// (lane_attn.cuh): two row tiles of a head side by side, or a last odd one of two heads.
//
// How the steps (one key tile of one unit: a pair of row tiles of a head, or the last odd one of two heads) are dealt out:
//   even   where every key tile is read by one unit, the flattened list of steps is split evenly over the SMs, wherever
//          that cuts a unit's range;
//   waves  where several units of a head read the same keys, their ranges are cut at the same places, and the pieces (tasks) go
//          to the SMs in the order of sequence, piece, unit: units that read the same tiles do so at the same time, and
//          all but one find them in L2.  Number and length of the pieces are the ones that make the longest SM's list
//          shortest.  (45 nodes of 8 heads over 131072 tokens, three row tiles: split evenly the keys come from memory twice and
//          the kernel takes 205 us.)
// A unit whose whole range falls to one CTA is finished there; of one that is split, every CTA leaves a
// partial (O, max, sum), and a combine kernel merges them, a CTA 32 rows and 64 columns at a time.  There are two partials a CTA
// at most, so they take a fixed 40 MB however large the batch.
//
// Scores (the summed logits of every prefix entry) need no softmax: they are products of the keys with the sum of the named
// nodes' queries, which a first kernel forms in fp32.  The softmax warps of one of the units that read a key tile multiply it with
// its head's sum while it is in shared memory; the combine adds up the heads.  (As three bf16 rows more of a row tile, where that had
// room for them, the warps of those rows held up the others: 8 ragged trees of 13 nodes 228 us; in a kernel of its own, which reads
// the keys again, 16 trees of 64 nodes took 123 us more.)
//
// A weight of 0 times an infinity or NaN is no 0: what is not finite of the nodes' values is zeroed in the tiles that hold them, and added
// at the end to the rows that attend it (2 to 3% of the calls of one sequence, less of others).
//
// What bounds it: the keys' bytes where a sequence has few row tiles (8 ragged trees of 13 nodes over 4096 to 65536 tokens, with
// scores: 225 us a call, 5.6 TB/s); the lanes' steps, softmax beside products, where it has many (45 nodes of 8 heads a KV head over
// 131072 tokens: 175 to 179 us, 1.1 PFLOP/s, the tensor pipe active 55% of the kernel); both where each would take about as long (16
// trees of 64 nodes over 16384 tokens: 219 us, with scores 271 to 282: the warps that multiply the keys with the summed queries
// are the softmax's).  What the plan does not do is balance batches of very different lengths that have several units a head: pieces are
// cut by the longest range, and with more than two units an SM not at all (131072 and 31 times 2048 tokens under 128 nodes each:
// 1657 us, the floor 216; 24 trees of 80 nodes over 512 to 65536 tokens: 872, 236).  With d = 64 the softmax warps keep some of the row
// masks' values in local memory (204 to 208 bytes a thread stored, 304 to 332 loaded; none with d = 128), which holds them up: 16
// trees of 64 nodes over 16384 tokens take 682 us, with d = 128 215.
#include "lane_attn.cuh"
#include "tree_bits.h"
#include "tree_step.h"

namespace vg {
namespace {

// A unit whose range is split, for the combine: its parts lie at `first`, then `second`, second + step and so on.
struct __align__(16) Split {
  int parts;  // 0: none
  int first, second, step;
  int seq, mode, rows;
  int odd;  // (of record c: CTA c has met values that are not finite)
  int head[2], r0[2];
};

// Prefix tokens and nodes of sequence b, and whether the call serves it: lengths in range, tokens of 31 bits (to the end of
// their last tile), and room for all of them in the cache.  The same answer for all three kernels: what is not served is neither
// appended nor attended nor scored.
struct Served {
  int n, m;
  bool ok;
};
__device__ __forceinline__ Served served(const TreeParams& p, int b) {
  Served s{p.prefix_len[b], p.tree_len ? p.tree_len[b] : p.R, false};
  const int64_t off = p.ptab ? 0 : p.seq_offset[b];
  const int64_t tokens = static_cast<int64_t>(s.n) + s.m;
  s.ok = s.n >= 0 && s.n <= p.max_len && s.m >= 0 && s.m <= p.R && tokens <= 0x7fffffff - KT &&
         (p.ptab ? tokens <= static_cast<int64_t>(p.pstride) * p.psize
                 : off >= 0 && off <= p.capacity && off + tokens <= p.capacity);
  return s;
}

struct TreePlan {
  using Params = TreeParams;
  static constexpr bool kTree = true, kScores = false;

  // n[B] prefix tokens, m[B] nodes, at[B + 1] steps (waves: tasks) before a sequence; key tiles of a task (0: even)
  struct Layout {
    int *n, *m, *at, *piece;
  };
  static __device__ __forceinline__ Layout layout(const TreeParams& p, int* mem) {
    return Layout{mem, mem + p.B, mem + 2 * p.B, mem + 3 * p.B + 1};
  }
  static __device__ __forceinline__ void units(const TreeParams& p, int m, int& pairs, int& units) {
    const int tiles = (m * p.G + p.RT - 1) / p.RT;
    pairs = tiles >> 1;
    units = p.Hkv * pairs + (tiles & 1) * ((p.Hkv + 1) / 2);
  }
  static __device__ __forceinline__ int key_tiles(int n, int m) { return m ? (n + m + KT - 1) / KT : 0; }
  // All threads of the CTA; a barrier follows.
  static __device__ __forceinline__ void load(const TreeParams& p, int* mem, int threads) {
    const Layout l = layout(p, mem);
    for (int b = threadIdx.x; b < p.B; b += threads) {
      const Served x = served(p, b);
      if (!x.ok && blockIdx.x == 0) report(p.status, VG_ERR_DEVICE_BOUNDS);
      l.n[b] = x.n;
      l.m[b] = x.ok ? x.m : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      // several units a head anywhere?  The longest range
      int longest = 0, several = 0, all = 0;
      for (int b = lane; b < p.B; b += 32) {
        int pairs, us;
        units(p, l.m[b], pairs, us);
        several |= (l.m[b] * p.G + p.RT - 1) / p.RT > 2;
        longest = max(longest, key_tiles(l.n[b], l.m[b]));
        all += us;
      }
      several = __any_sync(0xffffffffu, several);
      longest = __reduce_max_sync(0xffffffffu, longest);
      all = __reduce_add_sync(0xffffffffu, all);
      int piece = several ? longest : 0;
      if (several && all <= 2 * p.nctas) {
        // Lane j: the longest range cut into j + 1 pieces, the others into pieces of that length; the time of the
        // SM with the most tasks, if the split ones' partials have room.
        const int k = (longest + lane) / (lane + 1);
        int tasks = 0;
        for (int b = 0; b < p.B; ++b) {
          int pairs, us;
          units(p, l.m[b], pairs, us);
          tasks += us * ((key_tiles(l.n[b], l.m[b]) + k - 1) / k);
        }
        const int waves = (tasks + p.nctas - 1) / p.nctas;
        const uint32_t cost = tasks > all && tasks > 2 * p.nctas ? 0xffffffffu
                                                                 : static_cast<uint32_t>(waves) * (k + kSharedItemSteps);
        const uint32_t best = __reduce_min_sync(0xffffffffu, cost);
        const uint32_t who = __ballot_sync(0xffffffffu, cost == best);
        piece = __shfl_sync(0xffffffffu, k, __ffs(who) - 1);
      }
      int sum = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane;
        int v = 0;
        if (b < p.B) {
          int pairs, us;
          units(p, l.m[b], pairs, us);
          const int tiles = key_tiles(l.n[b], l.m[b]);
          v = us * (piece ? (tiles + piece - 1) / piece : tiles + kSharedItemSteps);
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += t;
        }
        if (b < p.B) l.at[b + 1] = sum + v;
        sum += __shfl_sync(0xffffffffu, v, 31);
      }
      if (lane == 0) {
        l.at[0] = 0;
        *l.piece = piece;
      }
    }
  }
  static __device__ __forceinline__ int sequence(const TreeParams& p, const Layout& l, int x) {
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {  // the last sequence that begins at x or before
      const int mid = (lo + hi + 1) >> 1;
      if (l.at[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
  }
  // Unit u of sequence b, with all its key tiles.
  static __device__ __forceinline__ Run unit_run(const TreeParams& p, const Layout& l, int b, int u) {
    Run r = {};
    r.row = b;
    r.n = l.n[b];
    r.rows = l.m[b] * p.G;
    r.ntok = r.n + l.m[b];
    r.priv = true;
    r.low = r.ntok <= kLowKeys;
    r.ntiles = key_tiles(l.n[b], l.m[b]);
    int pairs, us;
    units(p, l.m[b], pairs, us);
    const int np = p.Hkv * pairs;
    if (u < np) {
      r.mode = kPair;
      r.head[0] = r.head[1] = u / pairs;
      const int pair = u - r.head[0] * pairs;
      r.r0[0] = pair * 2 * p.RT;
      r.r0[1] = r.r0[0] + p.RT;
      r.z = pair == pairs - 1 && us == np ? 2 : 0;
    } else {
      const int hp = u - np;
      r.mode = 2 * hp + 1 < p.Hkv ? kHeads : kSingle;
      r.head[0] = 2 * hp;
      r.head[1] = 2 * hp + 1;
      r.r0[0] = r.r0[1] = pairs * 2 * p.RT;
      r.z = 3;
    }
    return r;
  }
  static __device__ __forceinline__ Split split_of(const Run& r, int parts, int first, int second, int step) {
    return Split{parts, first, second, step, r.row, r.mode, r.rows, 0, {r.head[0], r.head[1]}, {r.r0[0], r.r0[1]}};
  }
  // Task t (waves): its run; `parts` its unit is cut into, of which it is number j; units of its sequence.
  static __device__ __forceinline__ Run task(const TreeParams& p, const Layout& l, int t, int& j, int& parts, int& us) {
    const int b = sequence(p, l, t);
    int pairs;
    units(p, l.m[b], pairs, us);
    j = (t - l.at[b]) / us;
    Run r = unit_run(p, l, b, t - l.at[b] - j * us);
    const int tiles = r.ntiles;
    parts = (tiles + *l.piece - 1) / *l.piece;
    r.tile0 = j * tiles / parts;
    r.ntiles = (j + 1) * tiles / parts - r.tile0;
    r.whole = parts == 1;
    r.item = t;
    return r;
  }

  // This CTA's steps [x, x1) (waves: its first task, and all tasks); the producer warp 16 also leaves the split units that
  // begin with it, two at most.
  static __device__ __forceinline__ void steps(const TreeParams& p, int* mem, int& x, int& x1) {
    const Layout l = layout(p, mem);
    const int T = l.at[p.B], cta = blockIdx.x;
    Split s[2] = {};
    if (*l.piece) {
      x = cta;
      x1 = T;
      if (threadIdx.x == 16 * 32) {
        for (int k = 0; k < 2; ++k) {
          const int t = cta + k * p.nctas;
          if (t >= T) continue;
          int j, parts, us;
          const Run r = task(p, l, t, j, parts, us);
          if (j == 0 && parts > 1) s[k] = split_of(r, parts, t, t + us, us);
        }
      }
    } else {
      const int nc = min(T, p.nctas);
      x = cta < nc ? static_cast<int>(split_begin(cta, T, nc)) : 0;
      x1 = cta < nc ? static_cast<int>(split_begin(cta + 1, T, nc)) : 0;
      if (threadIdx.x == 16 * 32 && x < x1) {
        const int b = sequence(p, l, x1 - 1), len = key_tiles(l.n[b], l.m[b]) + kSharedItemSteps;
        const int u = (x1 - 1 - l.at[b]) / len, begin = l.at[b] + u * len, first = begin + kSharedItemSteps;
        if (first >= x && first < x1 && begin + len > x1)
          s[0] = split_of(unit_run(p, l, b, u), static_cast<int>(owner_cta(begin + len - 1, T, nc)) - cta + 1, 2 * cta + 1,
                          2 * (cta + 1), 2);
      }
    }
    if (threadIdx.x == 16 * 32) {
      Split* to = reinterpret_cast<Split*>(p.rec);
      to[cta] = s[0];
      to[cta + p.nctas] = s[1];
    }
  }
  static __device__ __forceinline__ Run next(const TreeParams& p, int* mem, int& x, int x1) {
    const Layout l = layout(p, mem);
    if (*l.piece) {
      int j, parts, us;
      const Run r = task(p, l, x, j, parts, us);
      x += p.nctas;
      return r;
    }
    const int b = sequence(p, l, x), len = key_tiles(l.n[b], l.m[b]) + kSharedItemSteps, u = (x - l.at[b]) / len;
    Run r = unit_run(p, l, b, u);
    const int off = x - l.at[b] - u * len, take = min(len - off, x1 - x), tiles = r.ntiles;
    r.tile0 = max(off - kSharedItemSteps, 0);  // (the unit's first steps have no tile)
    r.ntiles = off + take - kSharedItemSteps - r.tile0;
    r.whole = r.ntiles == tiles;
    // its partial: 0 of the unit that this CTA goes on with, 1 of the one that it leaves unfinished
    r.item = 2 * static_cast<int>(blockIdx.x) + (r.tile0 > 0 ? 0 : 1);
    x += take;
    return r;
  }
  static __device__ __forceinline__ int unit(const Run& r) { return r.item * 2; }

  // The summed query of a head; where the head's scores go.
  static __device__ __forceinline__ const float* sums(const TreeParams& p, const RunRec& r, int head) {
    return p.zsum + (static_cast<size_t>(r.row) * p.Hkv + head) * p.D;
  }
  static __device__ __forceinline__ float* scores(const TreeParams& p, const RunRec& r, int head) {
    return p.part_s + (static_cast<size_t>(r.row) * p.Hkv + head) * p.s_stride;
  }

  // Which of the tokens first .. first + 63 of the range query row `row` of the item attends.
  static __device__ __forceinline__ uint64_t bits(const TreeParams& p, const RunRec& r, int row, int first) {
    return tree_bits(p.visible, p.R, p.words, p.G, r.row, r.rows, row, r.n, r.ntok, first);
  }
  // Adds to columns col .. col + count - 1 of a node's output, at dst, what its nodes' values hold there that is not finite (slow,
  // for trees that have such values: a weight above 0 makes no other number of them).
  static __device__ __noinline__ void add_odd(const TreeParams& p, int b, int node, int head, int col, int count,
                                              __nv_bfloat16* dst) {
    const int n = p.prefix_len[b], m = p.tree_len ? p.tree_len[b] : p.R;
    for (int u = 0; u < m; ++u) {
      if (!(p.visible[(static_cast<size_t>(b) * p.R + node) * p.words + u / 64] >> (u & 63) & 1)) continue;
      const int64_t slot = kv_slot(p.seq_offset, p.ptab, p.psize, p.pstride, p.capacity, b, static_cast<int64_t>(n) + u);
      if (slot < 0) continue;
      const __nv_bfloat16* v = p.V + (slot * p.Hkv + head) * p.D + col;
      for (int i = 0; i < count; ++i) {
        const float x = __bfloat162float(v[i]);
        if (!isfinite(x)) dst[i] = __float2bfloat16(__bfloat162float(dst[i]) + x);
      }
    }
  }
  // Whether the CTA has met such values, for the combine.
  static __device__ __forceinline__ void leave_odd(const TreeParams& p, int odd) {
    reinterpret_cast<Split*>(p.rec)[blockIdx.x].odd = odd;
  }
  // Output of query row `row` of lane w.
  static __device__ __forceinline__ __nv_bfloat16* out(const TreeParams& p, const RunRec& r, int row, int w) {
    const int node = row / p.G, j = row - node * p.G;
    return p.out + ((static_cast<size_t>(r.row) * p.R + node) * p.Hq + r.head[w] * p.G + j) * p.D;
  }
};

struct ScoredTreePlan : TreePlan {
  static constexpr bool kScores = true;
};

// ---------------------------------------------------------------- combine
// A block of work is 32 rows and 64 columns of one lane of a split unit: a warp takes twice four columns, a lane a row, 512 contiguous
// bytes of each partial; partials, maxima and sums are asked for four at a time and merged in order.  Every CTA finds the split
// units among the attention CTAs' records for itself and takes every so many blocks (a CTA for every block that there could
// be, most of them empty, took 20 us more).  Then it takes its share of the tokens whose heads' scores are to be added up, a
// thread four of them.
constexpr int kTreeCombineThreads = 256;
constexpr int kScoreChunk = kTreeCombineThreads * 4;

template <int D, int GROUPS>
__device__ __forceinline__ void tree_merge(const TreeParams& p, const Split& s, int y, __nv_bfloat16 (*rows)[64 + 8]) {
  constexpr int AT_ONCE = 4, COLS = D / (32 * GROUPS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = y / (4 * COLS), q0 = (y / COLS & 3) * 32, g0 = y % COLS * 8 * GROUPS;
  if (w == 1 && s.mode == kSingle) return;
  const int nrows = min(p.RT, s.rows - s.r0[w]) - q0;
  if (nrows <= 0) return;
  const int row = q0 + lane;
  float4 acc[GROUPS] = {};
  float top = neg_inf(), l = 0.f;
  for (int i0 = 0; i0 < s.parts; i0 += AT_ONCE) {
    float4 ml[AT_ONCE], o[AT_ONCE][GROUPS];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int i = i0 + k;
      if (i >= s.parts) {
        ml[k] = make_float4(neg_inf(), 0.f, 0.f, 0.f);
        continue;
      }
      const size_t unit = static_cast<size_t>(i == 0 ? s.first : s.second + (i - 1) * s.step) * 2 + w;
      ml[k] = reinterpret_cast<const float4*>(p.parts_ml)[unit * KT + row];
#pragma unroll
      for (int h = 0; h < GROUPS; ++h)
        o[k][h] = reinterpret_cast<const float4*>(p.parts_o)[(unit * (D / 4) + g0 + warp + 8 * h) * KT + row];
    }
    float m = top;
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) m = fmaxf(m, ml[k].x);
    if (m != neg_inf()) {
      const float f = ex2(top - m);  // (0 of -inf)
#pragma unroll
      for (int h = 0; h < GROUPS; ++h) {
        acc[h].x *= f;
        acc[h].y *= f;
        acc[h].z *= f;
        acc[h].w *= f;
      }
      l *= f;
      top = m;
    }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      if (ml[k].x == neg_inf() && !(ml[k].y + ml[k].z != 0.f)) continue;  // (a key of NaN raises no maximum, but is in the sum)
      const float f = ex2(ml[k].x - top);
#pragma unroll
      for (int h = 0; h < GROUPS; ++h) {
        acc[h].x += f * o[k][h].x;
        acc[h].y += f * o[k][h].y;
        acc[h].z += f * o[k][h].z;
        acc[h].w += f * o[k][h].w;
      }
      l += f * (ml[k].y + ml[k].z);
    }
  }
  const float z = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int h = 0; h < GROUPS; ++h)
    *reinterpret_cast<uint2*>(&rows[lane][4 * (warp + 8 * h)]) =
        make_uint2(pack_bf16(acc[h].x * z, acc[h].y * z), pack_bf16(acc[h].z * z, acc[h].w * z));
  __syncthreads();
  constexpr int U = 4 * GROUPS;  // 16-byte units of a row
  const int r = threadIdx.x / U, k = threadIdx.x % U;
  if (r < 32 && r < nrows) {
    const int rr = s.r0[w] + q0 + r, node = rr / p.G, j = rr - node * p.G;
    __nv_bfloat16* dst = p.out + ((static_cast<size_t>(s.seq) * p.R + node) * p.Hq + s.head[w] * p.G + j) * D + 4 * g0;
    *reinterpret_cast<uint4*>(dst + 8 * k) = *reinterpret_cast<const uint4*>(&rows[r][8 * k]);
  }
  __syncthreads();
}

// What the rows of a block (of one of `cols` parts of the columns) attend that is not finite.
__device__ __noinline__ void tree_finish(const TreeParams& p, const Split& s, int y, int cols) {
  const int w = y / (4 * cols), q0 = (y / cols & 3) * 32, width = p.D / cols;
  if (w == 1 && s.mode == kSingle) return;
  const int nrows = min(p.RT, s.rows - s.r0[w]) - q0, r = threadIdx.x >> 3, part = width / 8;
  if (r >= nrows) return;
  const int rr = s.r0[w] + q0 + r, node = rr / p.G, j = rr - node * p.G, col = y % cols * width + (threadIdx.x & 7) * part;
  TreePlan::add_odd(p, s.seq, node, s.head[w], col, part,
                    p.out + ((static_cast<size_t>(s.seq) * p.R + node) * p.Hq + s.head[w] * p.G + j) * p.D + col);
}

template <int D>
__global__ void __launch_bounds__(kTreeCombineThreads, 4) tree_combine_kernel(const TreeParams p, int chunks) {
  constexpr int BLOCKS = 2 * 4 * (D / 64), WARPS = kTreeCombineThreads / 32;  // blocks of a unit
  extern __shared__ int list[];  // the split units' records, in order
  __shared__ int counts[WARPS];
  __shared__ __align__(16) __nv_bfloat16 rows[32][64 + 8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  const Split* records = reinterpret_cast<const Split*>(p.rec);
  int found = 0, odd = 0;
  for (int i0 = 0; i0 < 2 * p.nctas; i0 += kTreeCombineThreads) {
    const int i = i0 + tid;
    const bool in = i < 2 * p.nctas;
    const uint32_t mask = __ballot_sync(0xffffffffu, in && records[i].parts > 0);
    const bool met = __any_sync(0xffffffffu, in && records[i].odd != 0);
    if (lane == 0) counts[warp] = __popc(mask) + (met ? 64 : 0);
    __syncthreads();
    int before = found;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const int c = counts[k];
      if (k < warp) before += c & 63;
      found += c & 63;
      odd |= c & 64;
    }
    if (mask >> lane & 1) list[before + __popc(mask & ((1u << lane) - 1u))] = i;
    __syncthreads();
  }
  // (few units: twice as many blocks of half the columns, 165 us for one sequence of 131072 tokens, with wide ones 170; many: 16
  // sequences of 16384 tokens 213 us with wide ones, 225)
  if (found * BLOCKS >= static_cast<int>(gridDim.x)) {
    for (int x = blockIdx.x; x < found * BLOCKS; x += gridDim.x)
      tree_merge<D, 2>(p, records[list[x / BLOCKS]], x % BLOCKS, rows);
  } else {
    for (int x = blockIdx.x; x < found * 2 * BLOCKS; x += gridDim.x)
      tree_merge<D, 1>(p, records[list[x / (2 * BLOCKS)]], x % (2 * BLOCKS), rows);
  }
  if (odd) {  // (the rows that this CTA has written)
    const bool wide = found * BLOCKS >= static_cast<int>(gridDim.x);
    const int blocks = wide ? BLOCKS : 2 * BLOCKS;
    for (int x = blockIdx.x; x < found * blocks; x += gridDim.x)
      tree_finish(p, records[list[x / blocks]], x % blocks, blocks / 8);
  }
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int per = (p.max_len + kScoreChunk - 1) / kScoreChunk;
    const int b = c / per, i = (c - b * per) * kScoreChunk + 4 * tid;
    const Served seq = served(p, b);
    const int n = seq.n;
    if (!seq.ok || i >= n) continue;  // (nobody has left its heads' scores)
    const float* src = p.part_s + static_cast<size_t>(b) * p.Hkv * p.s_stride + i;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < (seq.m > 0 ? p.Hkv : 0); ++k) {
      const float4 x = *reinterpret_cast<const float4*>(src + k * p.s_stride);
      sum.x += x.x;
      sum.y += x.y;
      sum.z += x.z;
      sum.w += x.w;
    }
    float* dst = p.scores + b * p.score_stride + i;
    const float y[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < n) dst[e] = y[e] * p.scale;
  }
}

// ---------------------------------------------------------------- before: append, summed queries
// CTAs 0 .. B * R - 1 (k_new given): the key and value of a node to its slot.  The others (with scores), one a sequence
// and KV head: the sum of the named nodes' queries, in fp32.
constexpr int kTreePrepThreads = 256;
__global__ void __launch_bounds__(kTreePrepThreads) tree_prep_kernel(const TreeParams p, int appends) {
  __shared__ float part[kTreePrepThreads];
  pdl_wait();
  pdl_launch_dependents();
  const int width = p.Hkv * p.D, tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) < appends) {
    const int b = blockIdx.x / p.R, t = blockIdx.x - b * p.R;
    const Served seq = served(p, b);
    if (!seq.ok || t >= seq.m) return;  // (reported by the attention kernel)
    const int64_t slot = kv_slot(p.seq_offset, p.ptab, p.psize, p.pstride, p.capacity, b, static_cast<int64_t>(seq.n) + t);
    if (slot < 0) {
      if (tid == 0) report(p.status, VG_ERR_DEVICE_BOUNDS);
      return;
    }
    const uint4* k = reinterpret_cast<const uint4*>(p.k_new + static_cast<size_t>(blockIdx.x) * width);
    const uint4* v = reinterpret_cast<const uint4*>(p.v_new + static_cast<size_t>(blockIdx.x) * width);
    for (int e = tid; e < width / 8; e += kTreePrepThreads) {
      const uint4 x = k[e], y = v[e];
      reinterpret_cast<uint4*>(p.K + slot * width)[e] = x;
      reinterpret_cast<uint4*>(p.V + slot * width)[e] = y;
    }
    return;
  }
  const int x = blockIdx.x - appends, b = x / p.Hkv, g = x - b * p.Hkv, D = p.D;
  const Served seq = served(p, b);
  const int m = seq.ok ? seq.m : 0;
  const __nv_bfloat16* q = p.q + (static_cast<size_t>(b) * p.R * p.Hq + g * p.G) * D;  // node 0's rows of the head
  // the sum: thread (s, d) takes column d of every S-th head of the named nodes
  const int S = kTreePrepThreads / D, d = tid % D, s0 = tid / D;
  float acc = 0.f;
  for (int w = 0; 64 * w < m; ++w) {
    uint64_t named = p.score_rows[static_cast<size_t>(b) * p.words + w];
    if (m - 64 * w < 64) named &= (uint64_t{1} << (m - 64 * w)) - 1;
    for (; named != 0; named &= named - 1) {
      const __nv_bfloat16* row = q + static_cast<size_t>(64 * w + __ffsll(static_cast<long long>(named)) - 1) * p.Hq * D + d;
#pragma unroll 4
      for (int j = s0; j < p.G; j += S) acc += __bfloat162float(row[j * D]);
    }
  }
  part[tid] = acc;
  __syncthreads();
  if (tid < D) {
    for (int s = 1; s < S; ++s) acc += part[s * D + d];
    p.zsum[(static_cast<size_t>(b) * p.Hkv + g) * D + d] = acc;
  }
}

struct Launch {
  cudaLaunchAttribute at[1];
  cudaLaunchConfig_t cfg = {};
  Launch(dim3 grid, int block, size_t smem, cudaStream_t stream) {
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
};

int tree_words(int B) { return 3 * B + 2; }

template <int D>
cudaError_t launch_tree_t(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmQ,
                          cudaStream_t stream) {
  cudaError_t e;
  const int appends = p.k_new ? p.B * p.R : 0, sums = p.scores ? p.B * p.Hkv : 0;
  if (appends + sums > 0) {
    Launch f(dim3(appends + sums), kTreePrepThreads, 0, stream);
    if ((e = cudaLaunchKernelEx(&f.cfg, tree_prep_kernel, p, appends)) != cudaSuccess) return e;
  }
  using C = SCfg<D>;
  const size_t smem = C::smem(p.nslots, tree_words(p.B));
  Launch a(dim3(p.nctas), C::THREADS, smem, stream);
  if (p.scores) {
    if ((e = ensure_smem<lane_attn_kernel<D, ScoredTreePlan>>(smem)) != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&a.cfg, lane_attn_kernel<D, ScoredTreePlan>, p, tmK, tmV, tmQ);
  } else {
    if ((e = ensure_smem<lane_attn_kernel<D, TreePlan>>(smem)) != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&a.cfg, lane_attn_kernel<D, TreePlan>, p, tmK, tmV, tmQ);
  }
  if (e != cudaSuccess) return e;
  const int64_t chunks = p.scores ? static_cast<int64_t>(p.B) * ((p.max_len + kScoreChunk - 1) / kScoreChunk) : 0;
  // at most a CTA for every block of a unit, or chunk of scores, that there can be
  const int tiles = (p.R * p.G + p.RT - 1) / p.RT;
  const int64_t units = static_cast<int64_t>(p.B) * (p.Hkv * (tiles / 2) + (p.Hkv + 1) / 2), most = units * 8 * (D / 32) + chunks;
  Launch c(dim3(static_cast<unsigned>(most < 8 * p.nctas ? most : 8 * p.nctas)), kTreeCombineThreads,
           static_cast<size_t>(2 * p.nctas) * 4, stream);
  return cudaLaunchKernelEx(&c.cfg, tree_combine_kernel<D>, p, static_cast<int>(chunks));
}

}  // namespace

int tree_slots(int D, int B, size_t smem_optin) {
  return D == 64 ? SCfg<64>::slots(tree_words(B), smem_optin) : SCfg<128>::slots(tree_words(B), smem_optin);
}

size_t tree_split_bytes(int nctas) { return sizeof(Split) * 2 * static_cast<size_t>(nctas); }

cudaError_t launch_tree_verify(const TreeParams& p, const CUtensorMap& tmK, const CUtensorMap& tmV,
                               const CUtensorMap& tmQ, cudaStream_t stream) {
  return p.D == 64 ? launch_tree_t<64>(p, tmK, tmV, tmQ, stream) : launch_tree_t<128>(p, tmK, tmV, tmQ, stream);
}

}  // namespace vg
