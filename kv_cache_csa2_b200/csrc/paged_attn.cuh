// Device code shared by the paged attention kernels: warp-level matrix
// instructions on 16-bit types, exact FP4 dequantisation, and which tokens a
// tile of query rows sees.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "common.cuh"
#include "paged.h"
#include "rope.cuh"
#include "sm100.cuh"

namespace csa2 {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The reference that weights 2^(s - reference) of a row with maximum m are taken from, so that
// the largest is 2^lift.  From 2^22 on m - lift would round by more than the half step by
// which 2^15 stays finite in f16; there a score's own steps hide what the lift is for.
__device__ __forceinline__ float lifted(float m, float lift) { return fabsf(m) < 4194304.0f ? m - lift : m; }
// Where a reference may lag by 2^8, f16 weights stand 2^7 above its 1, so that they keep 11
// bits down to 2^-21 of it (f16's last step would else be 2^-24); the two together stay finite.
template <class T>
constexpr float lift_of() { return std::is_same<T, __half>::value ? 7.0f : 0.0f; }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}

// c[16 x 8] += a[16 x 16] b[16 x 8], f32 accumulation
template <class T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// E4M3 scale code as a bf16 pair (exact; the NaN code stays NaN)
__device__ __forceinline__ uint32_t scale_pair(uint32_t code) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3);
  const float f = __half2float(*reinterpret_cast<const __half*>(&h));
  return pack_bf16x2(f, f);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// 8 E2M1 codes (one word) times a scale: 8 bf16.  A code's three magnitude bits
// at the top of a bf16's exponent-and-mantissa boundary are the value times
// 2^-126 (subnormals included), so one exact product restores it.
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t scale2) {
  uint32_t o[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t b = (w >> (8 * u)) & 0xffu;
    const uint32_t t = b | (b << 12);
    const uint32_t v = ((t & 0x00070007u) << 6) | ((t & 0x00080008u) << 12);
    o[u] = mul_bf16x2(mul_bf16x2(v, 0x7e807e80u), scale2);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Length of sequence b, clamped to the table's row; the error word notes one
// outside it.
__device__ __forceinline__ int length_of(const PagedView& kv, int b, bool report) {
  const int n = __ldg(kv.lens + b);
  if (n >= 0 && n <= kv.capacity) return n;
  if (report) raise_dev_error(kv.err, DEVERR_BOUNDS);
  return n < 0 ? 0 : static_cast<int>(kv.capacity);
}

// Channel offset of token j of sequence b (head 0), or -1 when its page lies
// outside the pool.
__device__ __forceinline__ int64_t token_row(const PagedView& kv, int b, int j) {
  const int page = __ldg(kv.table + b * kv.table_stride + (j >> kv.page_shift));
  if (page < 0 || page >= kv.n_pages) {
    raise_dev_error(kv.err, DEVERR_BOUNDS);
    return -1;
  }
  return kv.row(page, j & ((1 << kv.page_shift) - 1), 0);
}

// Tokens [0, sinks) and [lo, hi) in one run of `total` slots: what the rows at
// positions pmin .. pmax see together.
struct Seen {
  int lo, ns, total;
  __device__ __forceinline__ Seen(int pmin, int pmax, int window, int sinks) {
    pmin = max(pmin, 0);
    lo = window > 0 && pmin >= window ? pmin + 1 - window : 0;
    ns = min(sinks, lo);
    total = pmax < 0 ? 0 : ns + (pmax + 1 - lo);
  }
  __device__ __forceinline__ int token(int slot) const { return slot < ns ? slot : slot - ns + lo; }
};
// The same for one row, in tiles of 128 tokens aligned to 128: the sinks', then
// those from the window's start on.
struct AlignedTiles {
  int lo, ns, pmax, sink_tiles, first_tile, tiles;
  __device__ __forceinline__ AlignedTiles(int p, int window, int sinks) : pmax(p) {
    const Seen s(p, p, window, sinks);
    lo = s.lo;
    ns = s.ns;
    sink_tiles = (ns + 127) / 128;
    first_tile = max(lo / 128, sink_tiles);
    tiles = s.total == 0 ? 0 : sink_tiles + max(0, p / 128 + 1 - first_tile);
  }
  __device__ __forceinline__ int start(int i) const { return (i < sink_tiles ? i : i - sink_tiles + first_tile) * 128; }
};
// window = 0: no window.  p - j < window as an unsigned difference is safe for
// every p >= j >= 0.
__device__ __forceinline__ bool sees(int p, int j, int window, int sinks) {
  return j <= p && (window <= 0 || p - j < window || j < sinks);
}

// Pairs of f32 in one instruction, each rounded to nearest.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 x, y, z, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};"
      " fma.rn.f32x2 w, x, y, z; mov.b64 {%0, %1}, w;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 x, y, w; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; add.rn.f32x2 w, x, y; mov.b64 {%0, %1}, w;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// One lane of a converged warp.  The products are issued under this instruction's
// predicate rather than a lane test: their operands live in uniform registers, and
// only here does the compiler know that a single lane is active.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{.reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p;}" : "=r"(e));
  return e != 0;
}
// Descriptors are a base plus an offset of their low word (16-byte units of shared memory).
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t bytes) { return base + (bytes >> 4); }
// One box of the cache's tensor map: channels c .. c + 63 of box rows from `slot` on.
__device__ __forceinline__ void tma_load_page(void* dst, const CUtensorMap* map, uint64_t* bar, int c, int head, int slot,
                                              int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(sm100::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(sm100::smem_u32(bar)), "r"(c), "r"(head), "r"(slot), "r"(page)
      : "memory");
}

// The same box into L2 ahead of its load.
__device__ __forceinline__ void tma_prefetch_page(const CUtensorMap* map, int c, int head, int slot, int page) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c), "r"(head), "r"(slot), "r"(page)
               : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

template <class T>
__host__ __device__ constexpr uint32_t idesc_of(int M, int N, bool a_mn, bool b_mn) {
  return std::is_same<T, __half>::value ? sm100::idesc_f16_f32(M, N, a_mn, b_mn) : sm100::idesc_bf16_f32(M, N, a_mn, b_mn);
}

// sm100::mbar_wait for a converged warp, with a short first look and the clock
// read only every 64 looks.  All lanes look: electing one to do it cost 190
// clocks more per wait in the prompt kernel (330 us against 274).
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  const uint64_t t0 = sm100::globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (sm100::mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (sm100::globaltimer_ns() - t0 > 2000000000ull) {
      raise_dev_error(err, DEVERR_TIMEOUT);
      *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  bool ok = true;
  if (!sm100::mbar_try_wait(bar, parity)) ok = wait_slow(bar, parity, abort, err);
  return __all_sync(0xffffffffu, ok);
}

// Whether a phase is over, without waiting.
__device__ __forceinline__ bool phase_over(uint64_t* bar, uint32_t parity) {
  uint32_t r;
  asm volatile("{.reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p;}"
               : "=r"(r)
               : "r"(sm100::smem_u32(bar)), "r"(parity)
               : "memory");
  return r != 0;
}

// A weight of 0 times a value that is not finite is NaN, so in a tile such a value
// reaches rows that do not see its token.  mend_rows finds those rows and computes
// them again one by one; it runs only when an output is not finite although its row
// sum is (a key that is not finite shows in the sum, and only where it is seen).
//
// All threads of the block take part (blockDim.x a multiple of 32), after every
// output is stored.  bad[r] != 0: row r of n_rows wants a look.  Tokens [0, ns) and
// [lo, pmax] are what the block has loaded; one bit each in `bitmap` says which hold
// such a value (more tokens than `capacity` bits: the rows stay as they are).  A row
// that sees one stays as it is; each other row is the f32 softmax over its own tokens.
struct MendRows {
  const uint16_t* q;                 // the sequence's first q row
  int64_t q_token, q_head;
  uint16_t* out;                     // its first output row, [token][Hq][D]
  float scale2;                      // signed scale * log2(e)
  int Hq, G, kvh, r0, base, window, sinks, lo, ns, pmax, b;
};
template <class T, int D>
__device__ __forceinline__ void mend_rows(const MendRows m, const PagedView& kv, const volatile uint8_t* bad, int n_rows,
                                       uint32_t* bitmap, int capacity) {
  constexpr int PER = D / 32;                          // channels per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int slots = m.ns + (m.pmax + 1 - m.lo);
  if (slots > capacity) return;
  for (int i = threadIdx.x; i < (slots + 31) / 32; i += blockDim.x) bitmap[i] = 0;
  __syncthreads();
  auto row_at = [&](const uint8_t* rows, int j) -> const uint16_t* {
    const int64_t r = token_row(kv, m.b, j);
    return r < 0 ? nullptr : reinterpret_cast<const uint16_t*>(rows) + r + m.kvh * kv.head_stride + lane * PER;
  };
  constexpr uint16_t EXP = std::is_same<T, __half>::value ? 0x7c00 : 0x7f80;
  for (int i = warp; i < slots; i += warps) {
    const uint16_t* v = row_at(kv.v, i < m.ns ? i : i - m.ns + m.lo);
    bool odd = false;
    if (v)
      for (int e = 0; e < PER; ++e) odd |= (v[e] & EXP) == EXP;
    if (__any_sync(0xffffffffu, odd) && lane == 0) atomicOr(bitmap + i / 32, 1u << (i % 32));
  }
  __syncthreads();
  for (int r = warp; r < n_rows; r += warps) {
    if (!bad[r]) continue;
    const int tok = (m.r0 + r) / m.G, pos = m.base + tok, head = m.kvh * m.G + (m.r0 + r) % m.G;
    bool reached = false;
    for (int i = lane; i < slots; i += 32) {
      const int j = i < m.ns ? i : i - m.ns + m.lo;
      reached |= sees(pos, j, m.window, m.sinks) && ((bitmap[i / 32] >> (i % 32)) & 1u);
    }
    if (__any_sync(0xffffffffu, reached)) continue;
    float qr[PER], acc[PER], mx = -INFINITY, l = 0.0f;
    const uint16_t* q = m.q + tok * m.q_token + head * m.q_head + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const float2 f = rope::Num<T>::up(q[e]);
      qr[e] = f.x;
      acc[e] = 0.0f;
    }
    for (int i = 0; i < slots; ++i) {
      const int j = i < m.ns ? i : i - m.ns + m.lo;
      if (!sees(pos, j, m.window, m.sinks)) continue;
      const uint16_t* k = row_at(kv.k, j);
      if (!k) continue;
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < PER; ++e) s += qr[e] * rope::Num<T>::up(k[e]).x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= m.scale2;
      const float now = fmaxf(mx, s), ref = now == -INFINITY ? 0.0f : now;
      const float f = exp2_approx(mx - ref), w = exp2_approx(s - ref);
      const uint16_t* v = row_at(kv.v, j);
      mx = now;
      l = l * f + w;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = acc[e] * f + w * rope::Num<T>::up(v[e]).x;
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    uint16_t* o = m.out + (static_cast<int64_t>(tok) * m.Hq + head) * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) o[e] = static_cast<uint16_t>(rope::Num<T>::down(acc[e] * inv, 0.0f) & 0xffffu);
  }
}

}  // namespace paged
}  // namespace csa2
