// rope.cuh -- what the kernels of rope.cu and norm_rope.cu share: elements,
// angles, and the walk over a token's (layer, head) rows.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace ssa {

constexpr int kRopeThreads = 256;

// Two 16-bit elements of a word as floats, and back (one rounding each).
template <typename T> __device__ __forceinline__ float2 unpack(uint32_t w);
template <> __device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <> __device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <typename T> __device__ __forceinline__ uint32_t pack(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float lo, float hi) {
  return pack_bf16(lo, hi);
}
template <> __device__ __forceinline__ uint32_t pack<__half>(float lo, float hi) {
  return pack_f16(lo, hi);
}

__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float x = a, y = b;
  a = x * cs.x - y * cs.y;
  b = y * cs.x + x * cs.y;
}

template <typename T> __device__ __forceinline__ float one_in(T x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same_v<T, __half>) return __half2float(x);
  else return __bfloat162float(x);
}
template <typename T> __device__ __forceinline__ T one_out(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// (cos, sin) of pos * f turns, f a 64-bit fraction
__device__ __forceinline__ float2 turn(uint64_t pos, uint64_t f) {
  const uint64_t ph = pos * f;
  const uint64_t q = (ph + (1ull << 61)) >> 62;             // nearest quarter turn
  const long long r = (long long)(ph - (q << 62));          // the rest, |r| <= 2^61
  float s, c;
  sincospif(__ll2float_rn(r) * 0x1p-63f, &s, &c);
  if (q & 1) { const float t = c; c = -s; s = t; }
  if (q & 2) { c = -c; s = -s; }
  return make_float2(c, s);
}

// One of q and k, as the lanes of a warp walk over its (layer, head) rows.
struct RopeRows {
  RopeTensor x;
  int per_warp;                          // rows of one warp
  int dh;                                // heads of a step of rows_pass rows, modulo x.heads
  int64_t in_step, out_step;             // elements of such a step ...
  int64_t in_wrap, out_wrap;             // ... and more where it runs past the last head
};

// every access of V elements of this tensor is aligned
inline bool aligned(const RopeTensor& x, int V, int esz, int L, int T) {
  const int64_t step[2][3] = {{x.is[0], x.is[1], x.is[2]}, {x.os[0], x.os[1], x.os[2]}};
  const int n[3] = {L, T, x.heads};
  if ((((uintptr_t)x.in | (uintptr_t)x.out) & (size_t)(V * esz - 1)) != 0) return false;
  for (auto& st : step)
    for (int i = 0; i < 3; ++i)
      if (n[i] > 1 && st[i] % V != 0) return false;
  return true;
}

}  // namespace ssa
