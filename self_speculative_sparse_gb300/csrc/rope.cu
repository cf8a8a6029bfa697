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
// The step is bound by memory: a row's heads are read once and written once.  A CTA takes
// a few rows at a time; its threads compute the rows' sines and cosines once into shared
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
// rot: one pair, element by element (its partner vectors are not 16-byte aligned).
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

template <int UNITS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, int rows_per_cta) {
  __shared__ float2 cs[kRopeMaxRows][64];  // (cos, sin) * mscale of the rows' pairs
  __shared__ int spos[kRopeMaxRows];       // position (-1: the row is left alone)
  __shared__ int64_t sslot[kRopeMaxRows];  // cache slot, -1: outside the cache
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = p.D, half = p.rot >> 1;
  const int upr = UNITS == kHalf2 ? D / 2 : D / 16;  // units of a head
  const int heads = p.Hq + 2 * p.Hkv;
  pdl_wait();
  pdl_launch_dependents();
  for (int r0 = blockIdx.x * rows_per_cta; r0 < p.n_rows; r0 += gridDim.x * rows_per_cta) {
    const int nr = min(rows_per_cta, p.n_rows - r0);
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
    for (int e = tid; e < nr * half; e += kRopeThreads) {
      const int rr = e / half, i = e - rr * half;
      const uint64_t phase = static_cast<uint64_t>(static_cast<uint32_t>(max(spos[rr], 0))) * p.freq[i];
      const float turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-32f;
      float s, c;
      sincospif(2.f * turns, &s, &c);
      cs[rr][i] = make_float2(c * p.mscale, s * p.mscale);
    }
    __syncthreads();
    const int total = nr * heads * upr;
    for (int e = tid; e < total; e += kRopeThreads) {
      const int rh = e / upr, u = e - rh * upr;
      const int rr = rh / heads, h = rh - rr * heads;
      if (spos[rr] < 0) continue;
      const int64_t row = r0 + rr;
      const int64_t slot = sslot[rr];
      const __nv_bfloat16* src;
      __nv_bfloat16* dst;
      bool turn = true;
      if (h < p.Hq) {
        src = p.q + row * p.q_stride + h * D;
        dst = p.q_out + row * p.q_out_stride + h * D;
      } else {
        if (slot < 0) continue;
        const int g = h - p.Hq;
        if (g < p.Hkv) {
          src = p.k + row * p.k_stride + g * D;
          dst = p.K + (slot * p.Hkv + g) * D;
        } else {
          src = p.v + row * p.v_stride + (g - p.Hkv) * D;
          dst = p.V + (slot * p.Hkv + g - p.Hkv) * D;
          turn = false;
        }
      }
      if constexpr (UNITS == kHalf2) {
        int i = u, j = u + half;
        if (u >= half) {
          i = p.rot + 2 * (u - half);
          j = i + 1;
        }
        const __nv_bfloat16 x = src[i], y = src[j];
        if (turn && u < half) {
          const float2 w = cs[rr][u];
          const float fx = __bfloat162float(x), fy = __bfloat162float(y);
          dst[i] = __float2bfloat16_rn(fx * w.x - fy * w.y);
          dst[j] = __float2bfloat16_rn(fx * w.y + fy * w.x);
        } else {
          dst[i] = x;
          dst[j] = y;
        }
      } else {
        int i = 16 * u, j = i + 8, f0 = 8 * u;
        if (UNITS == kHalf16 && turn && 16 * u < p.rot) {
          i = 8 * u;
          j = half + 8 * u;
        }
        const uint4 a = *reinterpret_cast<const uint4*>(src + i), b = *reinterpret_cast<const uint4*>(src + j);
        uint4 oa = a, ob = b;
        if (turn && 16 * u < p.rot) {
          if constexpr (UNITS == kHalf16) {
            const uint32_t xa[4] = {a.x, a.y, a.z, a.w}, xb[4] = {b.x, b.y, b.z, b.w};
            uint32_t ya[4], yb[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 w0 = cs[rr][f0 + 2 * q], w1 = cs[rr][f0 + 2 * q + 1];
              const float x0 = bf_lo(xa[q]), x1 = bf_hi(xa[q]), y0 = bf_lo(xb[q]), y1 = bf_hi(xb[q]);
              ya[q] = pack_bf16(x0 * w0.x - y0 * w0.y, x1 * w1.x - y1 * w1.y);
              yb[q] = pack_bf16(x0 * w0.y + y0 * w0.x, x1 * w1.y + y1 * w1.x);
            }
            oa = make_uint4(ya[0], ya[1], ya[2], ya[3]);
            ob = make_uint4(yb[0], yb[1], yb[2], yb[3]);
          } else {
            uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              if (f0 + q < half) {  // (rot may end inside the unit)
                const float2 w = cs[rr][f0 + q];
                const float x0 = bf_lo(x[q]), y0 = bf_hi(x[q]);
                x[q] = pack_bf16(x0 * w.x - y0 * w.y, x0 * w.y + y0 * w.x);
              }
            }
            oa = make_uint4(x[0], x[1], x[2], x[3]);
            ob = make_uint4(x[4], x[5], x[6], x[7]);
          }
        }
        *reinterpret_cast<uint4*>(dst + i) = oa;
        *reinterpret_cast<uint4*>(dst + j) = ob;
      }
    }
    __syncthreads();
  }
}

template <int UNITS>
cudaError_t launch_rope_t(const RopeParams& p, int sms, cudaStream_t stream) {
  const int per = kRopeMaxRows;
  const int need = (p.n_rows + per - 1) / per;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(need < 8 * sms ? need : 8 * sms);
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<UNITS>, p, per);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int sms, cudaStream_t stream) {
  if (p.interleaved) return launch_rope_t<kInter16>(p, sms, stream);
  return p.rot % 16 == 0 ? launch_rope_t<kHalf16>(p, sms, stream) : launch_rope_t<kHalf2>(p, sms, stream);
}

}  // namespace vg
