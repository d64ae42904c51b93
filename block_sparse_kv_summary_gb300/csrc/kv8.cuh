// K and V in 8 bits.  A block's 16 tokens of one head are held as codes c and
// one fp32 scale; with m the largest magnitude among its tokens and M the
// type's largest value (127 for int8, 448 for e4m3),
//
//     scale = m / M,    c = nearest(x (M / m)), halfway cases to even,
//
// each operation rounded once, and everything zero where m < 2^-100: there the
// quotients leave the normal numbers, and no logit or output notices.  A block
// with an infinity or a NaN has a scale of NaN and codes of zero, so that all of
// it reads as NaN.
//
// int8 spaces its values evenly below m, which suits coordinates of one size;
// e4m3 keeps four bits of each value, which suits blocks whose coordinates
// differ in size (channels some times wider than the others).
#pragma once

#include <cuda_fp8.h>

#include "compkv_device.cuh"

namespace compkv {

template <int KV>
struct Codes;
template <>
struct Codes<kKvInt8> {
  static constexpr float most = 127.f;
  // four values (|x| <= 127 up to a rounding, which the nearest integer swallows): added to 3 * 2^22, a value is rounded
  // to the nearest integer, halfway cases to even, and stands in the low bits.  One by one: as pairs, ptxas makes one
  // instruction of the addition and the product in front of it, which then rounds once where the definition rounds twice.
  static __device__ __forceinline__ uint32_t pack(float2 a, float2 b) {
    constexpr float magic = 12582912.f;
    a = make_float2(__fadd_rn(a.x, magic), __fadd_rn(a.y, magic));
    b = make_float2(__fadd_rn(b.x, magic), __fadd_rn(b.y, magic));
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  static __device__ __forceinline__ float4 unpack(uint32_t w) {
    const char4 c = *reinterpret_cast<const char4*>(&w);
    return make_float4((float)c.x, (float)c.y, (float)c.z, (float)c.w);
  }
};
template <>
struct Codes<kKvE4m3> {
  static constexpr float most = 448.f;
  static __device__ __forceinline__ uint32_t pack(float2 a, float2 b) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
  }
  static __device__ __forceinline__ float4 unpack(uint32_t w) {
    const float2 a = __half22float2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3));
    const float2 b = __half22float2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3));
    return make_float4(a.x, a.y, b.x, b.y);
  }
};

// A block's scale and the factor of its values, from the bits of its largest magnitude (an infinity or a NaN
// is larger than any number).
struct Scale {
  float scale, inv;
  template <int KV>
  static __device__ __forceinline__ Scale of(uint32_t bits) {
    const float m = __uint_as_float(bits);
    Scale s = {__fdiv_rn(m, Codes<KV>::most), __fdiv_rn(Codes<KV>::most, m)};
    if (m < 0x1p-100f) s = {0.f, 0.f};
    if (bits >= 0x7f800000u) s = {__uint_as_float(0x7fffffffu), 0.f};
    return s;
  }
};

// The tail.  A place that holds tokens of block b or of a later one goes out of date when block b is written; the writer
// empties it.
constexpr int kTails = 3;
// Whether the place is block b's.
__device__ __forceinline__ bool tail_in(int len, int b) { return len > b * kBlock && len <= (b + 1) * kBlock; }
// The place that holds at least the first `lo` tokens of block b of a unit (-1: none).
__device__ __forceinline__ int tail_place(const Kv8Args& c, int unit, int b, int lo) {
  int place = -1;
#pragma unroll
  for (int i = 0; i < kTails; ++i) {
    const int len = __ldcg(c.tail_len + kTails * unit + i);
    if (tail_in(len, b) && len - b * kBlock >= lo) place = i;
  }
  return place;
}
// The keys there; the values stand behind them.
template <int D>
__device__ __forceinline__ __nv_bfloat16* tail_at(const Kv8Args& c, int unit, int place) {
  return c.tail + (int64_t)(kTails * unit + place) * 2 * kBlock * D;
}

}  // namespace compkv
