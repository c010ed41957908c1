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
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&x)[4]) {
  x[0] = Num<T>::up(v.x);
  x[1] = Num<T>::up(v.y);
  x[2] = Num<T>::up(v.z);
  x[3] = Num<T>::up(v.w);
}
template <class T>
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  return make_uint4(Num<T>::down(x[0].x, x[0].y), Num<T>::down(x[1].x, x[1].y), Num<T>::down(x[2].x, x[2].y),
                    Num<T>::down(x[3].x, x[3].y));
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

// Pairs of f32 in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 w, x, y; mov.b64 {%0, %1}, w;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A token's angles: entry e holds pairs 2 e and 2 e + 1 as (cos, cos, sin, sin), the
// four entries of eight neighbouring pairs spread over four rows of half / 8, so
// that neighbouring lanes read side by side (all in one row, four would share a bank).
__device__ __forceinline__ int angle_slot(int f, int half) { return ((f >> 1) & 3) * (half >> 3) + (f >> 3); }
__device__ __forceinline__ void put_angle(float4* cs, int f, int half, float2 v) {
  float* e = reinterpret_cast<float*>(cs + angle_slot(f, half)) + (f & 1);
  e[0] = v.x;
  e[2] = v.y;
}

// Turns an item's pairs, two at a time.  Every product and sum is rounded by itself;
// the sums are not paired, because the assembler joins a paired product with a
// paired sum that takes it, .rn or not, and then rounds once.
__device__ __forceinline__ void turn2(float2& a, float2& b, const float4& cs) {
  const float2 c = make_float2(cs.x, cs.y), s = make_float2(cs.z, cs.w);
  const float2 ac = mul2(a, c), bs = mul2(b, s), bc = mul2(b, c), as = mul2(a, s);
  a = make_float2(__fsub_rn(ac.x, bs.x), __fsub_rn(ac.y, bs.y));
  b = make_float2(__fadd_rn(bc.x, as.x), __fadd_rn(bc.y, as.y));
}
__device__ __forceinline__ void rotate_item(float2 (&x0)[4], float2 (&x1)[4], const Item& it, int half,
                                            bool interleaved, const float4* cs) {
  if (it.freq < 0) return;
  if (!interleaved) {
#pragma unroll
    for (int u = 0; u < 4; ++u) turn2(x0[u], x1[u], cs[angle_slot(it.freq + 2 * u, half)]);
  } else {
    const int f0 = it.freq >> 1, f1 = (it.freq + half) >> 1;
#pragma unroll
    for (int u = 0; u < 4; u += 2) {
      float2 a = make_float2(x0[u].x, x0[u + 1].x), b = make_float2(x0[u].y, x0[u + 1].y);
      turn2(a, b, cs[angle_slot(f0 + u, half)]);
      x0[u] = make_float2(a.x, b.x);
      x0[u + 1] = make_float2(a.y, b.y);
      a = make_float2(x1[u].x, x1[u + 1].x), b = make_float2(x1[u].y, x1[u + 1].y);
      turn2(a, b, cs[angle_slot(f1 + u, half)]);
      x1[u] = make_float2(a.x, b.x);
      x1[u + 1] = make_float2(a.y, b.y);
    }
  }
}

}  // namespace rope
}  // namespace csa2
