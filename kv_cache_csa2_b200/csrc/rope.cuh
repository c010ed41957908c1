// Rows of heads in 16-byte vectors and the position rotation, shared by the
// head norm and the cache append.
//
// A row of D channels is handled by a group of lanes; every lane owns one ITEM,
// two 8-channel vectors.  The items of the rotated channels hold both halves of
// eight rotated pairs (channels i and i + half), so the rotation needs no
// exchange between lanes; interleaved pairs lie inside a vector anyway.  The
// remaining channels form items of two vectors each (the last may hold one).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace csa2 {
namespace rope {

constexpr int kMaxHalf = 256;

struct RopeArgs {
  const float* inv_freq;   // null: no rotation
  int half, offset, interleaved, inverse;
};

template <class T>
struct Num;
template <>
struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float2 up(uint32_t v) {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};
template <>
struct Num<__half> {
  static __device__ __forceinline__ float2 up(uint32_t v) {
    return __half22float2(*reinterpret_cast<__half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t down(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};

template <class T>
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = Num<T>::up(w[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}
template <class T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(Num<T>::down(x[0], x[1]), Num<T>::down(x[2], x[3]), Num<T>::down(x[4], x[5]),
                    Num<T>::down(x[6], x[7]));
}

// cos and sin of pos * f, the product and the reduction to one turn in 64 bits
// (a position of 2^20 times a frequency near 1 has no fraction left in 32 bits),
// each rounded once to f32.
__device__ __forceinline__ float2 angle_of(int32_t pos, float f, int inverse) {
  const double a = static_cast<double>(pos) * static_cast<double>(f);
  const double n = rint(a * 0.15915494309189535);                  // turns
  double r = fma(-n, 6.283185307179586, a);
  r = fma(-n, 2.4492935982947064e-16, r);                          // 2 pi's next bits
  double s, c;
  sincos(r, &s, &c);
  return make_float2(static_cast<float>(c), static_cast<float>(inverse ? -s : s));
}

struct Item {
  int c0, c1;      // first channel of each vector; -1: none
  int freq;        // first pair of c0 (rotated items); -1: not rotated
};

// Items of a row: half / 8 rotated ones, then the rest two vectors at a time.
__host__ __device__ __forceinline__ int items_of(int D, int half) {
  return half / 8 + ((D - 2 * half) / 8 + 1) / 2;
}
__device__ __forceinline__ Item item_at(int i, int D, int half, int offset) {
  Item it;
  const int nr = half >> 3;
  if (i < nr) {
    it.c0 = offset + 8 * i;
    it.c1 = it.c0 + half;
    it.freq = 8 * i;
    return it;
  }
  const int n = (D - 2 * half) >> 3, m = (n + 1) >> 1, j = i - nr;
  const int a = j * 8, b = (j + m) * 8;
  it.freq = -1;
  it.c0 = j < m ? (a < offset ? a : a + 2 * half) : -1;
  it.c1 = j < m && j + m < n ? (b < offset ? b : b + 2 * half) : -1;
  return it;
}

// Turns an item's pairs.  Every product and sum is rounded by itself, so the
// result does not depend on how a compiler contracts them.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
  const float x = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  const float y = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
  a = x;
  b = y;
}
__device__ __forceinline__ void rotate_item(float (&x0)[8], float (&x1)[8], const Item& it, int half,
                                            bool interleaved, const float2* cs) {
  if (it.freq < 0) return;
  if (!interleaved) {
#pragma unroll
    for (int u = 0; u < 8; ++u) turn(x0[u], x1[u], cs[it.freq + u]);
  } else {
    const int f0 = it.freq >> 1, f1 = (it.freq + half) >> 1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      turn(x0[2 * u], x0[2 * u + 1], cs[f0 + u]);
      turn(x1[2 * u], x1[2 * u + 1], cs[f1 + u]);
    }
  }
}

}  // namespace rope
}  // namespace csa2
