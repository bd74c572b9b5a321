// The 8-bit block format on the device (gfx950, wave64).
//
// A block is 128 consecutive values of a row.  Its scale is a power of two,
// 2^e with e the smallest integer >= -126 for which the block's largest
// finite magnitude is at most 448 * 2^e (448: the largest e4m3 value), stored
// as the e8m0 byte e + 127.  A code is RNE(x * 2^-e) in e4m3.  Why a power of
// two: e4m3's relative step does not depend on where in its range a value
// lies, so a scale rounded up to a power of two loses range (one bit of
// about 18) and no precision; x * 2^-e is exact, so quantising has exactly one
// rounding and any two implementations agree bit for bit; a decoded value has
// four significant bits, so reading back to bf16 is exact as well; and the
// byte is what the matrix cores take as their block scale.
// Values that are not finite become NaN codes and do not count for e.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_common.h"
#include "sv_host_quant.h"

namespace sv {

constexpr int kLanesPerBlock = 16;                            // lanes that share a block of the format
constexpr int kPerLaneQ = kQuantBlock / kLanesPerBlock;       // 8 values per lane
constexpr uint32_t kInfBits = 0x7f800000u;

// Maximum over the 16 lanes of a DPP row, in every lane of the row.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, (uint32_t)dpp::mov<dpp::kQuadSwap1, 0xf>(0, (int)v));
  v = max(v, (uint32_t)dpp::mov<dpp::kQuadSwap2, 0xf>(0, (int)v));
  v = max(v, (uint32_t)dpp::mov<dpp::kHalfMirror, 0xf>(0, (int)v));
  v = max(v, (uint32_t)dpp::mov<dpp::kMirror, 0xf>(0, (int)v));
  return v;
}

// Scale byte of a block whose largest finite magnitude has the fp32 bits a.
// With |x|max = m * 2^k, 1 <= m < 2, and 448 = 1.75 * 2^8: e = k - 8, or
// k - 7 where m > 1.75; adding 2^21 - 1 to the bits carries into the exponent
// exactly where the mantissa is above 0.75 * 2^23.  Zeros and subnormals end
// at the least byte, 1.
__device__ __forceinline__ int scale_byte(uint32_t a) {
  return max(1, (int)((a + 0x1fffffu) >> 23) - 8);
}

// 2^-e for a scale byte in 1 .. 248.
__device__ __forceinline__ float inverse_scale(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// A lane's eight values of a block to eight codes (value i in byte i).  The
// 16 lanes of a DPP row hold one block and all call this; *byte is the
// block's scale byte.  Magnitudes are compared as integers, where infinities
// and NaN lie above every finite value: a block that has any is gone over
// again with those left out.
__device__ __forceinline__ uint2 quantize8(float (&x)[kPerLaneQ], int* byte) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < kPerLaneQ; ++i) a = max(a, __float_as_uint(x[i]) & 0x7fffffffu);
  a = row16_max(a);
  if (a >= kInfBits) {
    a = 0;
#pragma unroll
    for (int i = 0; i < kPerLaneQ; ++i) {
      const uint32_t b = __float_as_uint(x[i]) & 0x7fffffffu;
      if (b < kInfBits) a = max(a, b);
      else x[i] = __uint_as_float(0x7fc00000u);
    }
    a = row16_max(a);  // the whole DPP row is in this branch: a was the row's maximum
  }
  const int sb = scale_byte(a);
  int lo = 0, hi = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  const float inv = inverse_scale(sb);
  // |x * inv| <= 448, so the conversion's overflow behaviour never matters.
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * inv, x[1] * inv, lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * inv, x[3] * inv, lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * inv, x[5] * inv, hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * inv, x[7] * inv, hi, true);
#endif
  *byte = sb;
  return uint2{(uint32_t)lo, (uint32_t)hi};
}

// Vectors at any address of whole elements: the hardware takes unaligned ones,
// and the compiler makes one access of each of these.
typedef uint32_t u32x4_any2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_any4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any1 __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
template <typename T> struct AnyVector;
template <> struct AnyVector<uint16_t> { typedef u32x4_any2 type; };
template <> struct AnyVector<float> { typedef u32x4_any4 type; };

// 16 bytes at p.  kVec: p is 16-byte aligned.  kStream: nontemporal.
template <typename T, bool kVec, bool kStream>
__device__ __forceinline__ u32x4 load16(const T* p) {
  if constexpr (kVec) return kStream ? stream16(p) : *reinterpret_cast<const u32x4*>(p);
  else return *reinterpret_cast<const typename AnyVector<T>::type*>(p);
}

// Eight consecutive values p[0 .. 7] as float, of which n (possibly <= 0)
// exist: the others are zeros and not read.  kVec: p is 16-byte aligned and n is
// at least 8 or at most 0.
template <typename T, bool kVec, bool kStream = true>
__device__ __forceinline__ void load8(const T* p, int n, float (&x)[kPerLaneQ]) {
  if (n >= kPerLaneQ) {
    if constexpr (sizeof(T) == 2) {
      const u32x4 w = load16<T, kVec, kStream>(p);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[2 * q] = bf16_lo(w[q]), x[2 * q + 1] = bf16_hi(w[q]);
    } else {
      const u32x4 w0 = load16<T, kVec, kStream>(p), w1 = load16<T, kVec, kStream>(p + 4);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] = __uint_as_float(w0[q]), x[4 + q] = __uint_as_float(w1[q]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPerLaneQ; ++i) x[i] = !kVec && i < n ? to_f32(p[i]) : 0.0f;
  }
}

// Eight codes at q.  kVec: 8-byte aligned.
template <bool kVec>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint2 q) {
  if (n >= kPerLaneQ) {
    // Nontemporal: nothing reads them soon, and the lines leave whole (a weight of 128256 x 4096: 265 -> 254 us).
    if (kVec) __builtin_nontemporal_store((uint64_t)q.x | ((uint64_t)q.y << 32), reinterpret_cast<uint64_t*>(p));
    else *reinterpret_cast<u32x2_any*>(p) = u32x2_any{q.x, q.y};
  } else if (!kVec) {
#pragma unroll
    for (int e = 0; e < kPerLaneQ; ++e)
      if (e < n) p[e] = (uint8_t)(e < 4 ? q.x >> (8 * e) : q.y >> (8 * (e - 4)));
  }
}

}  // namespace sv
