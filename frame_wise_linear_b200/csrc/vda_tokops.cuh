// Device helpers of the token operators (layer norm, rotary positions, 8-bit
// checkpoints): typed vector loads and stores, and the 8-bit block format.
//
// 8-bit block format.  A row's elements fall into blocks of 32 (the last one
// may be short).  A block stores e4m3 codes (1 sign, 4 exponent, 3 mantissa
// bits, largest finite 448) and one byte s = e + 127, where e >= -127 is the
// least integer with max |x| <= 448 * 2^e over the block's finite values; a
// code is x * 2^-e rounded to nearest even.  The scale is a power of two, so
// that scaling is exact both ways and an element is rounded once, by at most
// 2^-4 of its value (or 2^-10 * 2^e where that is more: below 2^-6 * 2^e the
// codes are equally spaced); a scale that is not a power of two would win
// nothing back but the last binade of the range.  NaN and infinities become
// NaN and do not count for the scale, so the rest of their block stays.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace vda {
namespace tokops {

constexpr int kBlock = 32;   // elements that share a scale

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <int Bytes>
struct RawOf;
template <> struct RawOf<1> { using type = uint8_t; };
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };

// VE consecutive elements of type T as they are stored: one load or store of
// VE * sizeof(T) bytes (1 to 16), whose address is a multiple of that.
template <typename T, int VE>
struct Pack {
  using Raw = typename RawOf<VE * (int)sizeof(T)>::type;
  union {
    Raw raw;
    T e[VE];
    uint32_t w[(VE * (int)sizeof(T) + 3) / 4];
  };
  __device__ __forceinline__ Pack() {}
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const Raw*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = Raw{}; }
  __device__ __forceinline__ float get(int i) const { return to_f32(e[i]); }
  __device__ __forceinline__ void set(int i, float x) { e[i] = from_f32<T>(x); }
  // Elements i and i + 1 (i even), word by word.
  __device__ __forceinline__ float2 get2(int i) const {
    if constexpr (sizeof(T) == 2)
      return make_float2(__uint_as_float(w[i / 2] << 16), __uint_as_float(w[i / 2] & 0xffff0000u));
    else
      return make_float2(to_f32(e[i]), to_f32(e[i + 1]));
  }
  __device__ __forceinline__ void set2(int i, float2 v) {
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 b = __float22bfloat162_rn(v);
      w[i / 2] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      e[i] = from_f32<T>(v.x);
      e[i + 1] = from_f32<T>(v.y);
    }
  }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// |x| where x is finite, else 0: what an element adds to its block's maximum.
__device__ __forceinline__ float block_mag(float x) { return finite(x) ? fabsf(x) : 0.f; }

// The scale byte of a block whose largest finite magnitude is `top`: top =
// m 2^k (1 <= m < 2) needs e = k - 8 while m <= 1.75 (448 = 1.75 * 2^8), one
// more above.  Subnormal and zero `top` take e = -127.
__device__ __forceinline__ int scale_byte(float top) {
  const uint32_t b = __float_as_uint(top);
  const int s = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return s < 0 ? 0 : s;
}
// 2^(s - 127) and 2^(127 - s), both exact (s = 0: the subnormal 2^-127).
__device__ __forceinline__ float scale_of(int s) { return __uint_as_float(s ? (uint32_t)s << 23 : 0x400000u); }
__device__ __forceinline__ float inv_scale_of(int s) { return __uint_as_float((uint32_t)(254 - s) << 23); }

// Two scaled values to two codes (x in the low byte); NaN stays NaN.
__device__ __forceinline__ uint32_t encode2(float2 v) {
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}
// The same for any values of a block with scale byte s: infinities become NaN,
// and at the largest scale byte, 247, where a scaled value of 248 or more
// would round to 256, which stands for 2^128, 240 is taken, within the same
// half step of 2^-4.
__device__ __forceinline__ uint32_t encode2_any(float2 v, float inv, int s) {
  const float nan = __uint_as_float(0x7fffffffu), most = s >= 247 ? 240.f : 448.f;
  v.x = finite(v.x) ? fminf(fmaxf(v.x * inv, -most), most) : nan;
  v.y = finite(v.y) ? fminf(fmaxf(v.y * inv, -most), most) : nan;
  return encode2(v);
}
// The values of two codes, unscaled (exact).
__device__ __forceinline__ float2 decode2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Two float32 at a time: one instruction each on this architecture.
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Elements i and i + 1 of a vector (i even) plus c: bf16 is added to float32 as
// it is, without being widened first (exact operands, one rounding to float32).
template <typename T, int VE>
__device__ __forceinline__ float2 plus2(const Pack<T, VE>& q, int i, float2 c) {
  if constexpr (sizeof(T) == 2) {
    float2 r;
    asm("add.rn.f32.bf16 %0, %1, %2;" : "=f"(r.x) : "h"((uint16_t)q.w[i / 2]), "f"(c.x));
    asm("add.rn.f32.bf16 %0, %1, %2;" : "=f"(r.y) : "h"((uint16_t)(q.w[i / 2] >> 16)), "f"(c.y));
    return r;
  } else {
    return add2(q.get2(i), c);
  }
}

// The lanes of a group of Lanes neighbours (a power of two up to 32).
template <int Lanes>
__device__ __forceinline__ uint32_t lane_group() {
  return (uint32_t)((1ull << Lanes) - 1) << ((threadIdx.x & 31) / Lanes * Lanes);
}
// The largest of v over a group; `mask`: lanes that are here together, whole groups.
template <int Lanes>
__device__ __forceinline__ float lanes_max(float v, uint32_t mask) {
#pragma unroll
  for (int o = Lanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(mask, v, o));
  return v;
}

// From here up (448 * 2^119: infinity among them) a block takes encode2_any.
constexpr float kLargeTop = 448.f * 0x1p119f;

// VE values to codes, and the block's scale byte, by the 32 / VE neighbouring
// lanes that hold the block (values beyond the row are 0; `mask`: the lanes that
// are here together).  fmaxf passes over NaN, so a block without infinities
// needs no test of its elements; kSmall: there are none, nor values near
// float32's end.
template <int VE, bool kSmall>
__device__ __forceinline__ int encode_block(const float (&x)[VE], Pack<uint8_t, VE>& codes, uint32_t mask) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < VE; ++i) top = fmaxf(top, fabsf(x[i]));
  top = lanes_max<kBlock / VE>(top, mask);
  int s = scale_byte(top);
  uint32_t two[VE > 1 ? VE / 2 : 1];
  if (kSmall || top <= kLargeTop) {
    const float2 inv = both(inv_scale_of(s));
#pragma unroll
    for (int i = 0; i < VE; i += 2) two[i / 2] = encode2(mul2(make_float2(x[i], VE > 1 ? x[i + 1] : 0.f), inv));
  } else {
    top = 0.f;
#pragma unroll
    for (int i = 0; i < VE; ++i) top = fmaxf(top, block_mag(x[i]));
    top = lanes_max<kBlock / VE>(top, lane_group<kBlock / VE>());
    s = scale_byte(top);
#pragma unroll
    for (int i = 0; i < VE; i += 2)
      two[i / 2] = encode2_any(make_float2(x[i], VE > 1 ? x[i + 1] : 0.f), inv_scale_of(s), s);
  }
  if constexpr (VE == 1) codes.e[0] = (uint8_t)two[0];
  if constexpr (VE == 4) codes.raw = two[0] | two[1] << 16;
  if constexpr (VE == 8) codes.raw = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
  return s;
}

// The values of VE neighbouring codes, unscaled (exact), in pairs; one code: in x.
template <int VE>
__device__ __forceinline__ void decode_pairs(const Pack<uint8_t, VE>& c, float2 (&out)[VE > 1 ? VE / 2 : 1]) {
  static_assert(VE == 1 || VE == 4 || VE == 8, "1, 4 or 8 codes");
  if constexpr (VE == 1) {
    out[0] = decode2(c.e[0]);
  } else {
    uint32_t w[VE / 4];
    if constexpr (VE == 4) {
      w[0] = c.raw;
    } else {
      w[0] = c.raw.x;
      w[1] = c.raw.y;
    }
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) {
      out[2 * i] = decode2(w[i] & 0xffffu);
      out[2 * i + 1] = decode2(w[i] >> 16);
    }
  }
}

// Asynchronous copies of 4, 8 or 16 bytes into shared memory, in groups that
// complete in order; both addresses are multiples of the size.
template <int Bytes>
__device__ __forceinline__ void async_copy(void* shared, const void* global) {
  const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(shared));
  if constexpr (Bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(global) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(global), "n"(Bytes) : "memory");
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most N of this thread's groups are still on their way.
template <int N>
__device__ __forceinline__ void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace tokops
}  // namespace vda
