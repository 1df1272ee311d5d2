// Device-side helpers of the microscaled (MX) formats: 32 consecutive
// elements share one power-of-two scale (an e8m0 byte b stands for 2^(b-127),
// 255 for NaN) and are held as e2m1 (4 bits, two to a byte, the even element
// in the low nibble) or e4m3 (8 bits) codes.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int kMxBlock = 32;
constexpr int kMxFp4 = 0;  // e2m1: largest value 6 = 1.5 * 2^2
constexpr int kMxFp8 = 1;  // e4m3: largest value 448 = 1.75 * 2^8

typedef int i32x8_t __attribute__((ext_vector_type(8)));

template <int kFmt> struct Mx {
  static constexpr int kEmax = kFmt == kMxFp4 ? 2 : 8;  // exponent of the largest element value
  // bytes of n codes
  static constexpr __host__ __device__ int64_t bytes(int64_t n) { return kFmt == kMxFp4 ? n / 2 : n; }
};

// The bits of |v|: they order finite values by size, with infinities and NaN
// above all of them, so the integer maximum over a block also tells whether
// any element is not finite.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale byte of a block from the largest abs_bits: floor(log2 amax) - emax,
// biased by 127, at least 0 (amax below the normal range has an exponent
// field of 0 and lands there too); 255 if an element is not finite.
template <int kFmt> __device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits) {
  const int b = max(static_cast<int>(amax_bits >> 23) - Mx<kFmt>::kEmax, 0);
  return amax_bits >= 0x7f800000u ? 255u : static_cast<uint32_t>(b);
}

// 2^(127 - b), the factor that takes elements to code range: always a normal
// float (b <= 252), so the product is exact wherever it does not round to
// zero as a code.  0 for a block that is not finite (its codes are 0).
__device__ __forceinline__ float mx_inv_scale(uint32_t b) {
  return b == 255u ? 0.f : __uint_as_float((254u - b) << 23);
}

// 2^(b - 127); NaN for b = 255.
__device__ __forceinline__ float mx_scale(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fc00000u) : b == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// Eight elements to codes, round to nearest even, saturating: 4 bytes of e2m1
// or 8 bytes of e4m3.  bad: the block holds a NaN or an infinity (0 * inf
// would make a NaN code).
__device__ __forceinline__ uint32_t mx_encode8_fp4(const float* v, float inv, bool bad) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0] * inv, v[1] * inv, 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2] * inv, v[3] * inv, 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4] * inv, v[5] * inv, 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6] * inv, v[7] * inv, 1.0f, 3);
  return bad ? 0u : r;
}
// The conversion itself turns values from 464 up into NaN: clamp first.
__device__ __forceinline__ float clamp448(float v) { return __builtin_amdgcn_fmed3f(v, -448.f, 448.f); }
__device__ __forceinline__ uint32_t mx_encode4_fp8(const float* v, float inv, bool bad) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(v[0] * inv), clamp448(v[1] * inv), r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(v[2] * inv), clamp448(v[3] * inv), r, true);
  return bad ? 0u : static_cast<uint32_t>(r);
}

// Stores the codes of 8 consecutive elements, the first of them element `at`
// of the code array (at is a multiple of 8).
template <int kFmt>
__device__ __forceinline__ void mx_store8(uint8_t* codes, int64_t at, const float* v, float inv, bool bad) {
  if constexpr (kFmt == kMxFp4) {
    *reinterpret_cast<uint32_t*>(codes + at / 2) = mx_encode8_fp4(v, inv, bad);
  } else {
    *reinterpret_cast<uint2*>(codes + at) = make_uint2(mx_encode4_fp8(v, inv, bad), mx_encode4_fp8(v + 4, inv, bad));
  }
}

// e2m1 code (4 bits) to fp32: exponent field 0 holds 0 and 0.5, others 2^(f-1) (1 + m/2).
__device__ __forceinline__ float mx_decode_fp4(uint32_t c) {
  const uint32_t mag = c & 7u;
  // 1 and up: exponent field f and mantissa m shifted into place with the exponent rebiased by 126.
  const float v = mag < 2u ? 0.5f * static_cast<float>(mag) : __uint_as_float((mag << 22) + (126u << 23));
  return (c & 8u) ? -v : v;
}

// The 4 e4m3 codes of a dword to fp32.
__device__ __forceinline__ void mx_decode4_fp8(uint32_t r, float* v) {
  const f32x2_t a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(r), false);
  const f32x2_t b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(r), true);
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
}

// 8 or 4 codes, the first of element `at`, to fp32 values (before the scale).
template <int kFmt, int kEl> __device__ __forceinline__ void mx_load(const uint8_t* codes, int64_t at, float* v) {
  static_assert(kEl == 8 || kEl == 4, "");
  if constexpr (kFmt == kMxFp4) {
    uint32_t r;
    if constexpr (kEl == 8) r = *reinterpret_cast<const uint32_t*>(codes + at / 2);
    else r = *reinterpret_cast<const uint16_t*>(codes + at / 2);
#pragma unroll
    for (int i = 0; i < kEl; ++i) v[i] = mx_decode_fp4(r >> (4 * i));
  } else if constexpr (kEl == 8) {
    const uint2 r = *reinterpret_cast<const uint2*>(codes + at);
    mx_decode4_fp8(r.x, v);
    mx_decode4_fp8(r.y, v + 4);
  } else {
    mx_decode4_fp8(*reinterpret_cast<const uint32_t*>(codes + at), v);
  }
}

// 8 consecutive elements of a bf16 or fp32 array (16-byte aligned) to and from fp32.
__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  const u32x4_t r = ld16(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r[i] << 16);
    v[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const u32x4_t a = ld16(p), b = ld16(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = __uint_as_float(a[i]);
    v[4 + i] = __uint_as_float(b[i]);
  }
}
__device__ __forceinline__ u32x4_t pack8_bf16(const float* v) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  return r;
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) { st16(p, pack8_bf16(v)); }
__device__ __forceinline__ void store8(float* p, const float* v) {
  u32x4_t a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_uint(v[i]);
    b[i] = __float_as_uint(v[4 + i]);
  }
  st16(p, a);
  st16(p + 4, b);
}

// For values that nothing reads soon.  fp32 goes through the caches: a lane's
// two stores touch every other 16 bytes, and the caches join them.
__device__ __forceinline__ void store8_nt(uint16_t* p, const float* v) { st16_nt(p, pack8_bf16(v)); }
__device__ __forceinline__ void store8_nt(float* p, const float* v) { store8(p, v); }

// Largest abs_bits over the 4 lanes that hold a block (8 elements each).
__device__ __forceinline__ uint32_t mx_block_max(const float* v) {
  uint32_t m = abs_bits(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, abs_bits(v[i]));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1)));
  m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2)));
  return m;
}

}  // namespace moe
