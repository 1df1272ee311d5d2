// The experts' products on microscaled (MX) operands: e2m1 weights, e2m1 or
// e4m3 token rows, one e8m0 scale per 32 elements along K on both sides.
//
//   up:   H[r, :]  = MX(gelu(sum_k Xq[perm[r] / k, k] * W1q[e][:, k]))
//   down: Yp[r, :] = sum_f Hq[r, f] * W2q[e][:, f]
//
// for the rows r of expert e's segment [offsets[e], offsets[e+1]).  The
// matrix cores take the codes and the scales as they are stored
// (v_mfma_scale_f32_*_f8f6f4) and accumulate in fp32: nothing is widened in
// memory.  The up-projection's GELU and the quantisation of its result to the
// next product's operand run on the accumulators.
#include "kernels.hpp"
#include "mx.hpp"

namespace moe {
namespace {

// Operand B of the scaled MFMA: its format code is 0 for e4m3, 4 for e2m1.
template <int kFmt> __device__ __forceinline__ constexpr int mx_code() { return kFmt == kMxFp4 ? 4 : 0; }

// 32 weight rows (operand A, e2m1) x 32 token rows (operand B) x 64 of K.
// Lane l holds, of weight row l%32, the 32 elements of K block l/32; of token
// row l%32 the same for e2m1, and for e4m3 the 16 elements l/32 of both
// blocks.  The scales come from lanes l/32 = block for either format.
template <int kFmt>
__device__ __forceinline__ f32x16_t mx_mfma32(i32x8_t w, i32x8_t x, f32x16_t c, int ws, int xs) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 4, mx_code<kFmt>(), 0, ws, 0, xs);
}

__device__ __forceinline__ i32x8_t frag(u32x4_t lo, u32x4_t hi) {
  return i32x8_t{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]),
                 static_cast<int>(hi[0]), static_cast<int>(hi[1]), static_cast<int>(hi[2]), static_cast<int>(hi[3])};
}

// What a product does with 16 consecutive columns of one row, of which this
// lane holds the half `half` of a block of 32 and lane ^ 32 the other half.
template <int kFmt> struct UpOut {
  uint8_t* hq;
  uint8_t* hs;
  __device__ __forceinline__ void store(int64_t row, int N, int col, int half, bool ok, float* v) const {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      v[q] = gelu_tanh_fast(v[q]);
      m = max(m, abs_bits(v[q]));
    }
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
    const uint32_t b = mx_scale_byte<kFmt>(m);
    if (!ok) return;
    mx_store16<kFmt>(hq, row * N + col, v, mx_inv_scale(b), b == 255u);
    if (half == 0) hs[row * (N / kMxBlock) + col / kMxBlock] = static_cast<uint8_t>(b);
  }
};
template <typename T> struct DownOut {
  T* y;
  __device__ __forceinline__ void store(int64_t row, int N, int col, int, bool ok, float* v) const {
    if (!ok) return;
    store8(y + row * N + col, v);
    store8(y + row * N + col + 8, v + 8);
  }
};

// One wave per 32 weight rows x 32 token rows, fragments straight from
// memory.  The weight rows of the tile are taken in the order pi(x) =
// 16*((x>>2)&1) + 4*(x>>3) + (x&3), which gives a lane 16 consecutive output
// columns of its token row.
template <int kFmt, bool kGather, typename Out>
__global__ __launch_bounds__(kWave) void mx_product_direct(MxOperands o, const int32_t* __restrict__ gidx, int gdiv,
                                                           int src_rows, Out out) {
  const int lane = threadIdx.x;
  int t_seg0 = 0, t_seg1 = 0;
  if (lane < o.E) {
    // offsets come from device memory: clamped, every access stays inside the buffers
    t_seg0 = min(max(o.offsets[lane], 0), o.max_rows);
    t_seg1 = min(max(o.offsets[lane + 1], t_seg0), o.max_rows);
  }
  const int t_mt = (t_seg1 - t_seg0 + 31) / 32;
  int t_incl = t_mt;
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const int u = __shfl_up(t_incl, m);
    if (lane >= m) t_incl += u;
  }
  const int ntn = o.N / 32;
  const int64_t tile = blockIdx.x;
  const int e = static_cast<int>(__popcll(__ballot(lane < o.E && static_cast<int64_t>(t_incl) * ntn <= tile)));
  if (e >= o.E) return;
  const int mt_e = __shfl(t_mt, e);
  const int64_t local = tile - static_cast<int64_t>(__shfl(t_incl, e) - mt_e) * ntn;
  const int n0 = static_cast<int>(local / mt_e) * 32;
  const int m0 = __shfl(t_seg0, e) + static_cast<int>(local % mt_e) * 32;
  const int rows = min(32, __shfl(t_seg1, e) - m0);

  const int frow = lane & 31;
  const int half = lane >> 5;
  const int wrow = ((frow >> 2) & 1) * 16 + (frow >> 3) * 4 + (frow & 3);
  const int64_t row = m0 + min(frow, rows - 1);
  int64_t src = row;
  bool live = true;
  if constexpr (kGather) {
    const unsigned u = static_cast<unsigned>(gidx[row]) / static_cast<unsigned>(gdiv);
    live = u < static_cast<unsigned>(src_rows);
    src = live ? u : 0;
  }
  const int64_t xrow_bytes = Mx<kFmt>::bytes(o.K);
  const uint8_t* xp = o.xq + src * xrow_bytes + half * 16;
  const uint8_t* xsp = o.xs + src * (o.K / kMxBlock) + half;
  const int64_t wr = static_cast<int64_t>(e) * o.N + n0 + wrow;
  const uint8_t* wp = o.wq + wr * (o.K / 2) + half * 16;
  const uint8_t* wsp = o.ws + wr * (o.K / kMxBlock) + half;
  const u32x4_t zero = {0u, 0u, 0u, 0u};

  f32x16_t acc;
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = 0.f;
  const int steps = o.K / 64;
  for (int s = 0; s < steps; ++s) {
    const u32x4_t w = ld16(wp + s * 32);
    u32x4_t x0, x1 = zero;
    if constexpr (kFmt == kMxFp4) {
      x0 = ld16(xp + s * 32);
    } else {
      x0 = ld16(xp + s * 64);
      x1 = ld16(xp + s * 64 + 32);
    }
    const int sw = wsp[s * 2];
    const int sx = live ? xsp[s * 2] : 0;
    acc = mx_mfma32<kFmt>(frag(w, zero), frag(live ? x0 : zero, live ? x1 : zero), acc, sw, sx);
  }
  float v[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) v[q] = acc[q];
  out.store(m0 + frow, o.N, n0 + 16 * half, half, frow < rows, v);
}

template <int kFmt, bool kGather, typename Out>
hipError_t launch_product(const MxOperands& o, const int32_t* gidx, int gdiv, int src_rows, const Out& out,
                          hipStream_t stream) {
  const int64_t tiles = (static_cast<int64_t>((o.max_rows + 31) / 32) + o.E) * (o.N / 32);
  if (tiles > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx_product_direct<kFmt, kGather, Out>), dim3(static_cast<unsigned>(tiles)), dim3(kWave), 0,
                     stream, o, gidx, gdiv, src_rows, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_up(int fmt, const MxOperands& o, const int32_t* gidx, int gdiv, int src_rows, uint8_t* hq,
                        uint8_t* hs, hipStream_t stream) {
  if (o.max_rows <= 0) return hipSuccess;
  if (fmt == kMxFp4)
    return launch_product<kMxFp4, true>(o, gidx, gdiv, src_rows, UpOut<kMxFp4>{hq, hs}, stream);
  return launch_product<kMxFp8, true>(o, gidx, gdiv, src_rows, UpOut<kMxFp8>{hq, hs}, stream);
}

hipError_t launch_mx_down(int dtype, int fmt, const MxOperands& o, void* y, hipStream_t stream) {
  if (o.max_rows <= 0) return hipSuccess;
  const int rows = o.max_rows;
  if (dtype == kDtypeBF16) {
    const DownOut<uint16_t> out{static_cast<uint16_t*>(y)};
    return fmt == kMxFp4 ? launch_product<kMxFp4, false>(o, nullptr, 1, rows, out, stream)
                         : launch_product<kMxFp8, false>(o, nullptr, 1, rows, out, stream);
  }
  const DownOut<float> out{static_cast<float*>(y)};
  return fmt == kMxFp4 ? launch_product<kMxFp4, false>(o, nullptr, 1, rows, out, stream)
                       : launch_product<kMxFp8, false>(o, nullptr, 1, rows, out, stream);
}

}  // namespace moe
