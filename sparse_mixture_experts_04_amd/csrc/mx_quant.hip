// Quantisation to the microscaled (MX) formats and back, and the residual's
// addition with the root-mean-square norm that stands before the layer, with
// its outputs for the router (the layer's type) and for the experts (MX).
//
// Quantisation (OCP Microscaling Formats v1.0): for a block of 32 consecutive
// elements, amax = max |v|, scale 2^(floor(log2 amax) - emax), codes = v /
// scale rounded to nearest even and saturated.  Every step is exact but that
// one rounding, so codes and scales are the definition's, bit for bit.
// All three kernels are bound by memory: each element is touched once, and the
// four lanes of a block exchange their maxima in registers.  At 180224 x 2048
// bf16 <-> e2m1, 0.93 GB each way, quantising takes 154 us (6.1 TB/s) and the
// way back 224 us (4.2; 138 where the codes are still in the last-level
// cache); a copy of 4 GiB runs at 4.7.  8 x 3584 takes one launch, 2.5 us.
#include "kernels.hpp"
#include "mx.hpp"

namespace moe {
namespace {

constexpr int kQThreads = 256;

// A block of 32 may not straddle rows (cols is a multiple of 32), so rows
// and columns do not matter: chunk c holds elements 8c .. 8c+7 and blocks are
// groups of 4 chunks.
template <typename T, int kFmt>
__global__ __launch_bounds__(kQThreads) void mx_quantize_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales, int64_t chunks) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kQThreads;
  // chunks is a multiple of 4: the lanes of a block leave the loop together
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; c < chunks; c += stride) {
    float v[8];
    load8(x + c * 8, v);
    const uint32_t b = mx_scale_byte<kFmt>(mx_block_max(v));
    mx_store8<kFmt>(codes, c * 8, v, mx_inv_scale(b), b == 255u);
    if ((c & 3) == 0) scales[c >> 2] = static_cast<uint8_t>(b);
  }
}

// One 16-byte store per thread and so 8 bf16 or 4 f32 values each: a wave's
// stores lie side by side, which non-temporal stores need (f32 with two stores
// per lane, 32 bytes apart: 208 us at 65536 x 2048, against 93).  The values are
// two to eight times the bytes read; through the caches e2m1 to bf16 took 230 us
// at 180224 x 2048 against 224, and the quantisation after it 176 against 154.
template <typename T, int kFmt>
__global__ __launch_bounds__(kQThreads) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  T* __restrict__ x, int64_t chunks) {
  constexpr int kEl = 16 / sizeof(T);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kQThreads;
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; c < chunks; c += stride) {
    float v[kEl];
    mx_load<kFmt, kEl>(codes, c * kEl, v);
    const float s = mx_scale(scales[c >> (kEl == 8 ? 2 : 3)]);
#pragma unroll
    for (int i = 0; i < kEl; ++i) v[i] *= s;
    if constexpr (kEl == 8) {
      st16_nt(x + c * 8, pack8_bf16(v));
    } else {
      st16_nt(x + c * 4, u32x4_t{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                 __float_as_uint(v[3])});
    }
  }
}

// A block's work is one sweep of 256 threads: blocks start in order, so the
// memory in flight stays one moving window.  (A grid of 16 blocks per CU that
// strides over everything left 20 % of the bandwidth unused: 4.9 against
// 6.0 TB/s at 180224 x 2048.)  The kernels' loops serve only sizes past the
// largest grid, 2^32 threads.
int quant_grid(int64_t chunks) {
  const int64_t blocks = (chunks + kQThreads - 1) / kQThreads;
  constexpr int64_t kCap = (int64_t{1} << 32) / kQThreads - 1;
  return static_cast<int>(blocks < kCap ? blocks : kCap);
}

template <typename T>
hipError_t quantize_t(int fmt, const void* x, uint8_t* codes, uint8_t* scales, int64_t chunks, hipStream_t stream) {
  const dim3 grid(quant_grid(chunks));
  if (fmt == kMxFp4)
    hipLaunchKernelGGL((mx_quantize_kernel<T, kMxFp4>), grid, dim3(kQThreads), 0, stream, static_cast<const T*>(x),
                       codes, scales, chunks);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<T, kMxFp8>), grid, dim3(kQThreads), 0, stream, static_cast<const T*>(x),
                       codes, scales, chunks);
  return hipGetLastError();
}

template <typename T>
hipError_t dequantize_t(int fmt, const uint8_t* codes, const uint8_t* scales, void* x, int64_t chunks,
                        hipStream_t stream) {
  const dim3 grid(quant_grid(chunks));
  if (fmt == kMxFp4)
    hipLaunchKernelGGL((mx_dequantize_kernel<T, kMxFp4>), grid, dim3(kQThreads), 0, stream, codes, scales,
                       static_cast<T*>(x), chunks);
  else
    hipLaunchKernelGGL((mx_dequantize_kernel<T, kMxFp8>), grid, dim3(kQThreads), 0, stream, codes, scales,
                       static_cast<T*>(x), chunks);
  return hipGetLastError();
}

// One block per token.  s = x + r is formed in fp32 and kept in registers
// (kNC chunks of 8 elements per thread), so each input is read once.
//   sum = round(s);  n = s * rstd * gamma;  y = round(n);  MX codes of n
// The norm and the codes start from the unrounded s and n: the only roundings
// are the ones of the stored results.  The squares are summed in fp64: fp32
// would overflow to infinity for |s| past 1.8e19, which bf16 holds.
// The bf16 sum, which nothing reads before the layer has run, is stored past
// the caches (16384 x 2048: 48.9 -> 44.4 us, 6.8 TB/s); y and the codes, which
// the router and the experts read next, are not.
// x, r, sum and y may be the same buffer: a thread reads its elements of x and
// r before it writes them anywhere, and nobody else reads them.
template <typename T, int kFmt, int kNC, int kThreads>
__global__ __launch_bounds__(kThreads) void add_rmsnorm_kernel(const T* x, const T* r, const T* __restrict__ gamma,
                                                               float eps, T* sum, T* y, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales, int d) {
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  const int chunks = d / 8;
  const int64_t base = t * d;
  float v[kNC][8];
  double ss = 0.0;
#pragma unroll
  for (int i = 0; i < kNC; ++i) {
    const int c = tid + i * kThreads;
    if (c < chunks) {
      load8(x + base + c * 8, v[i]);
      if (r != nullptr) {
        float w[8];
        load8(r + base + c * 8, w);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[i][q] += w[q];
      }
      if (sum != nullptr) store8_nt(sum + base + c * 8, v[i]);
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fma(static_cast<double>(v[i][q]), static_cast<double>(v[i][q]), ss);
    }
  }
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) ss += __shfl_xor(ss, m);
  if constexpr (kThreads > kWave) {
    __shared__ double part[kThreads / kWave];
    if (tid % kWave == 0) part[tid / kWave] = ss;
    __syncthreads();
    ss = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) ss += part[w];
  }
  const float rstd = static_cast<float>(1.0 / sqrt(ss / d + static_cast<double>(eps)));
#pragma unroll
  for (int i = 0; i < kNC; ++i) {
    const int c = tid + i * kThreads;
    if (c < chunks) {  // chunks is a multiple of 8: the 4 lanes of a block are in or out together
      float g[8];
      load8(gamma + c * 8, g);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[i][q] = v[i][q] * rstd * g[q];
      if (y != nullptr) store8(y + base + c * 8, v[i]);
      if (codes != nullptr) {
        const uint32_t b = mx_scale_byte<kFmt>(mx_block_max(v[i]));
        mx_store8<kFmt>(codes, base + c * 8, v[i], mx_inv_scale(b), b == 255u);
        if ((c & 3) == 0) scales[(base >> 5) + (c >> 2)] = static_cast<uint8_t>(b);
      }
    }
  }
}

template <typename T, int kFmt>
hipError_t rmsnorm_tf(const T* x, const T* r, const T* gamma, float eps, T* sum, T* y, uint8_t* codes,
                      uint8_t* scales, int T_tok, int d, hipStream_t stream) {
  const int chunks = d / 8;
#define MOE_NORM(NC, TH)                                                                                             \
  hipLaunchKernelGGL((add_rmsnorm_kernel<T, kFmt, NC, TH>), dim3(T_tok), dim3(TH), 0, stream, x, r, gamma, eps, sum, \
                     y, codes, scales, d)
  if (chunks <= 64) MOE_NORM(1, 64);
  else if (chunks <= 256) MOE_NORM(1, 256);
  else if (chunks <= 512) MOE_NORM(2, 256);
  else if (chunks <= 1024) MOE_NORM(4, 256);
  else if (chunks <= 4096) MOE_NORM(4, 1024);
  else return hipErrorInvalidValue;
#undef MOE_NORM
  return hipGetLastError();
}

template <typename T>
hipError_t rmsnorm_t(int fmt, const void* x, const void* r, const void* gamma, float eps, void* sum, void* y,
                     uint8_t* codes, uint8_t* scales, int T_tok, int d, hipStream_t stream) {
  const T* xp = static_cast<const T*>(x);
  const T* rp = static_cast<const T*>(r);
  const T* gp = static_cast<const T*>(gamma);
  return fmt == kMxFp4
             ? rmsnorm_tf<T, kMxFp4>(xp, rp, gp, eps, static_cast<T*>(sum), static_cast<T*>(y), codes, scales, T_tok,
                                     d, stream)
             : rmsnorm_tf<T, kMxFp8>(xp, rp, gp, eps, static_cast<T*>(sum), static_cast<T*>(y), codes, scales, T_tok,
                                     d, stream);
}

}  // namespace

hipError_t launch_mx_quantize(int dtype, int fmt, const void* x, void* codes, uint8_t* scales, int64_t n,
                              hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  uint8_t* c = static_cast<uint8_t*>(codes);
  return dtype == kDtypeBF16 ? quantize_t<uint16_t>(fmt, x, c, scales, n / 8, stream)
                             : quantize_t<float>(fmt, x, c, scales, n / 8, stream);
}

hipError_t launch_mx_dequantize(int dtype, int fmt, const void* codes, const uint8_t* scales, void* x, int64_t n,
                                hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  const uint8_t* c = static_cast<const uint8_t*>(codes);
  return dtype == kDtypeBF16 ? dequantize_t<uint16_t>(fmt, c, scales, x, n / 8, stream)
                             : dequantize_t<float>(fmt, c, scales, x, n / 4, stream);
}

hipError_t launch_add_rmsnorm(int dtype, int fmt, const void* x, const void* r, const void* gamma, float eps,
                              void* sum, void* y, void* codes, uint8_t* scales, int T_tok, int d,
                              hipStream_t stream) {
  if (T_tok <= 0) return hipSuccess;
  uint8_t* c = static_cast<uint8_t*>(codes);
  return dtype == kDtypeBF16 ? rmsnorm_t<uint16_t>(fmt, x, r, gamma, eps, sum, y, c, scales, T_tok, d, stream)
                             : rmsnorm_t<float>(fmt, x, r, gamma, eps, sum, y, c, scales, T_tok, d, stream);
}

}  // namespace moe
