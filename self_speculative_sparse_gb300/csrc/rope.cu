// Rotary positions of new q and k rows, and the append of k and v to the cache.
//
// A pair (x, y) of a row at position pos, with the pair's frequency f, becomes
//   (x cos(a) - y sin(a), x sin(a) + y cos(a)) * mscale,   a = pos * f.
// The angle is never formed in radians: a frequency is held as F = f / 2pi * 2^64, a
// fraction of a turn per position in 64-bit fixed point, so the 64-bit product pos * F
// drops whole turns by overflow and is the fraction of the turn, exact up to pos * 2^-65
// of a turn (the rounding of F) at any position.  Its top 32 bits, as a signed fraction in
// [-1/2, 1/2), go through sincospif: an absolute error of about 2^-25 of a turn, far below
// the bf16 rounding of the result, where a 32-bit pos * f would be off by 2^-8 of a turn at
// position 65536.  Everything between the bf16 loads and stores is fp32.
//
// The step is bound by memory: a row's heads are read once and written once (23977 rows of 48 heads
// of 128: 589 MB in 95 us, 6.2 TB/s, 91% of a plain copy's rate).  A CTA takes
// a few rows; its threads compute the rows' sines and cosines once into shared
// memory (they are the same for every head), then walk over units of 16 elements of the
// rows' q, k and v heads.  A unit holds both members of its pairs, so q may be rotated in
// place.
#include "vg_common.cuh"
#include "vg_internal.h"

namespace vg {
namespace {

constexpr int kRopeThreads = 256;

// How a head's elements are cut into units.  kHalf16: pairs (i, i + rot / 2), rot a multiple
// of 16: 8 consecutive i and their partners, as two 16-byte vectors.  kInter16: pairs
// (2i, 2i + 1): 16 consecutive elements.  kHalf2: pairs (i, i + rot / 2) for any other even
// rot: one pair, element by element (its partner vectors are not 16-byte aligned): 23977 rows of 48 heads
// with 100 of 128 elements turned take 510 us, with all 128 95.
enum RopeUnits { kHalf16, kInter16, kHalf2 };

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Sequence of packed row r: the last b with row_start[b] <= r (B <= 1024: two rounds of one
// load a lane).  Whole warp.
__device__ __forceinline__ int row_sequence(const int32_t* row_start, int B, int r) {
  const int lane = threadIdx.x & 31;
  const int step = (B + 31) / 32;  // <= 32
  const int i = lane * step;
  const bool le = i < B && row_start[i] <= r;
  const int seg = max(0, __popc(__ballot_sync(0xffffffffu, le)) - 1) * step;
  const int j = seg + lane;
  const bool le2 = lane < step && j < B && row_start[j] <= r;
  return seg + max(0, __popc(__ballot_sync(0xffffffffu, le2)) - 1);
}

// A unit: where it comes from and goes, which head and pair it starts at.  Units of a row: the q
// heads', then the k heads', then the v heads'.
struct RopeUnit {
  const __nv_bfloat16* src;
  int rr, h, u;
};

template <int UNITS, bool FEW>
__global__ void __launch_bounds__(kRopeThreads, FEW ? 1 : 8) rope_kernel(const RopeParams p, int rows_per_cta) {
  __shared__ float2 cs[kRopeMaxRows][64];  // (cos, sin) * mscale of the rows' pairs
  __shared__ int spos[kRopeMaxRows];       // position (-1: the row is left alone)
  __shared__ int64_t sslot[kRopeMaxRows];  // cache slot, -1: outside the cache
  constexpr int NB = FEW ? (UNITS == kHalf2 ? 4 : 3) : 1;  // units a thread has on the way
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = p.D, half = p.rot >> 1;
  const int upr = UNITS == kHalf2 ? D / 2 : D / 16;  // units of a head
  const int heads = p.Hq + 2 * p.Hkv, per_row = heads * upr;
  pdl_wait();
  pdl_launch_dependents();
  const int r0 = blockIdx.x * rows_per_cta;
  const int nr = min(rows_per_cta, p.n_rows - r0), total = nr * per_row;
  auto unit = [&](int e) {
    RopeUnit x;
    x.rr = e / per_row;
    e -= x.rr * per_row;
    x.h = e / upr;
    x.u = e - x.h * upr;
    const int64_t row = r0 + x.rr;
    x.src = x.h < p.Hq            ? p.q + row * p.q_stride + x.h * D
            : x.h < p.Hq + p.Hkv ? p.k + row * p.k_stride + (x.h - p.Hq) * D
                                  : p.v + row * p.v_stride + (x.h - p.Hq - p.Hkv) * D;
    return x;
  };
  // first and second element (or vector) of a unit
  auto places = [&](const RopeUnit& x, int& i, int& j) {
    const bool turn = x.h < p.Hq + p.Hkv;
    if constexpr (UNITS == kHalf2) {
      i = x.u < half ? x.u : p.rot + 2 * (x.u - half);
      j = x.u < half ? x.u + half : i + 1;
    } else {
      i = 16 * x.u;
      j = i + 8;
      if (UNITS == kHalf16 && turn && 16 * x.u < p.rot) {
        i = 8 * x.u;
        j = half + 8 * x.u;
      }
    }
  };
  struct Two {
    uint4 a, b;
  };
  auto fetch = [&](Two (&t)[NB], int e0) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int e = e0 + k * kRopeThreads;
      if (e >= total) continue;
      const RopeUnit x = unit(e);
      if (spos[x.rr] < 0) continue;
      int i, j;
      places(x, i, j);
      if constexpr (UNITS == kHalf2) {
        t[k].a.x = *reinterpret_cast<const uint16_t*>(x.src + i);
        t[k].b.x = *reinterpret_cast<const uint16_t*>(x.src + j);
      } else {
        t[k].a = *reinterpret_cast<const uint4*>(x.src + i);
        t[k].b = *reinterpret_cast<const uint4*>(x.src + j);
      }
    }
  };
  if (warp < nr) {
    const int r = r0 + warp;
    int b, t;
    if (p.row_start) {
      b = row_sequence(p.row_start, p.B, r);
      t = r < p.row_start[p.B] ? r - p.row_start[b] : -1;  // rows behind the last sequence
    } else {
      b = r / p.R;
      t = r - b * p.R;
    }
    const int n = p.prefix_len[b];
    int pos = -1;
    int64_t slot = -1;
    if (t >= 0) {
      if (n < 0 || n > p.max_len || static_cast<int64_t>(n) + t > 0x7fffffffLL) {
        if (lane == 0) report(p.status, VG_ERR_DEVICE_BOUNDS);
      } else {
        pos = n + t;
        slot = kv_slot(p.seq_offset, p.ptab, p.psize, p.pstride, p.capacity, b, pos);
        if (slot < 0 && lane == 0) report(p.status, VG_ERR_DEVICE_BOUNDS);
      }
    }
    if (lane == 0) {
      spos[warp] = pos;
      sslot[warp] = slot;
    }
  }
  __syncthreads();
  Two now[NB];
  fetch(now, tid);
  for (int e = tid; e < nr * half; e += kRopeThreads) {
    const int rr = e / half, i = e - rr * half;
    const uint64_t phase = static_cast<uint64_t>(static_cast<uint32_t>(max(spos[rr], 0))) * p.freq[i];
    const float turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-32f;
    float s, c;
    sincospif(2.f * turns, &s, &c);
    cs[rr][i] = make_float2(c * p.mscale, s * p.mscale);
  }
  __syncthreads();
  for (int e0 = tid; e0 < total; e0 += NB * kRopeThreads) {
    if (e0 != tid) fetch(now, e0);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int e = e0 + k * kRopeThreads;
      if (e >= total) continue;
      const RopeUnit x = unit(e);
      if (spos[x.rr] < 0) continue;
      const int64_t slot = sslot[x.rr];
      const bool turn = x.h < p.Hq + p.Hkv;
      if (x.h >= p.Hq && slot < 0) continue;
      __nv_bfloat16* dst = x.h < p.Hq ? p.q_out + (r0 + x.rr) * p.q_out_stride + x.h * D
                           : turn     ? p.K + (slot * p.Hkv + x.h - p.Hq) * D
                                      : p.V + (slot * p.Hkv + x.h - p.Hq - p.Hkv) * D;
      int i, j;
      places(x, i, j);
      const float2* w = cs[x.rr];
      if constexpr (UNITS == kHalf2) {
        if (turn && x.u < half) {
          const float fx = __uint_as_float(now[k].a.x << 16), fy = __uint_as_float(now[k].b.x << 16);
          dst[i] = __float2bfloat16_rn(fx * w[x.u].x - fy * w[x.u].y);
          dst[j] = __float2bfloat16_rn(fx * w[x.u].y + fy * w[x.u].x);
        } else {
          *reinterpret_cast<uint16_t*>(dst + i) = static_cast<uint16_t>(now[k].a.x);
          *reinterpret_cast<uint16_t*>(dst + j) = static_cast<uint16_t>(now[k].b.x);
        }
      } else {
        uint32_t a[4] = {now[k].a.x, now[k].a.y, now[k].a.z, now[k].a.w};
        uint32_t b[4] = {now[k].b.x, now[k].b.y, now[k].b.z, now[k].b.w};
        if (turn && 16 * x.u < p.rot) {
          const int f0 = 8 * x.u;
          if constexpr (UNITS == kHalf16) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 w0 = w[f0 + 2 * q], w1 = w[f0 + 2 * q + 1];
              const float x0 = bf_lo(a[q]), x1 = bf_hi(a[q]), y0 = bf_lo(b[q]), y1 = bf_hi(b[q]);
              a[q] = pack_bf16(x0 * w0.x - y0 * w0.y, x1 * w1.x - y1 * w1.y);
              b[q] = pack_bf16(x0 * w0.y + y0 * w0.x, x1 * w1.y + y1 * w1.x);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              uint32_t& v = q < 4 ? a[q] : b[q - 4];
              if (f0 + q < half) {  // (rot may end inside the unit)
                const float x0 = bf_lo(v), y0 = bf_hi(v);
                v = pack_bf16(x0 * w[f0 + q].x - y0 * w[f0 + q].y, x0 * w[f0 + q].y + y0 * w[f0 + q].x);
              }
            }
          }
        }
        *reinterpret_cast<uint4*>(dst + i) = make_uint4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<uint4*>(dst + j) = make_uint4(b[0], b[1], b[2], b[3]);
      }
    }
  }
}

template <int UNITS>
cudaError_t launch_rope_t(const RopeParams& p, int sms, cudaStream_t stream) {
  // Few rows (all CTAs resident at once): one row a CTA and up to four units a thread on the way, so
  // that the call is one round of loads: 56 rows of 48 heads of 128 take 5.3 us so and 7.3 us with
  // four rows a CTA.  Many: occupancy hides the loads better than a thread's own loads in flight
  // (23977 rows of 48 heads of 128: 97 us with one unit and 8 CTAs an SM, 100 with two, 118 with one
  // and the 4 CTAs that fit when registers are not limited), and a CTA for every four rows
  // better than CTAs that stay (107 us).
  const bool few = p.n_rows <= 4 * sms;
  const int per = few ? 1 : kRopeMaxRows;
  const int need = (p.n_rows + per - 1) / per;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(need);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? rope_kernel<UNITS, true> : rope_kernel<UNITS, false>, p, per);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t stream) {
  if (p.interleaved) return launch_rope_t<kInter16>(p, sms, stream);
  return p.rot % 16 == 0 ? launch_rope_t<kHalf16>(p, sms, stream) : launch_rope_t<kHalf2>(p, sms, stream);
}

}  // namespace vg
