// Attention of one new token per sequence over a paged cache, rows of 64, 128 or
// 256 channels: up to 16 query heads of one cache head per CTA, the sequence's
// visible tokens cut into chunks over CTAs.
//
// HBM-bound: every cached row is read once and meets 16 query rows.  What counts
// is bytes in flight, so every warp works alone: it streams its own slices of 16
// tokens (32 of FP4 rows) through a private ring in shared memory (cp.async, no block barrier in
// the loop) and keeps its own running maximum, sum and output in registers; the
// 4 warps meet once at the end.  A page lookup runs one slice ahead of its loads.
//   S[16 heads, 16 tokens] = q k^T, P = 2^(S - m), O[16 heads, D] += P v
// with warp-level products: at 16 rows the arithmetic is 16 multiply-adds per
// byte, far below what they deliver.
// Measured: 64 ragged sequences of up to 16384 tokens, 64 heads over 8 x 128, 233 us
// (6.05 TB/s, 0.92 of a plain copy's rate); one sequence of 8192 with its join, 9.0 us.
//
// FP4 rows stay packed in shared memory; a thread's fragment is made of whole code
// words (8 channels of a token), which become f16 pairs in registers by the hardware's
// E2M1 conversion and one product with the scale: a code times a scale has five
// significant bits between 2^-10 and 2^12, exact in f16.  (Integer steps to bf16 cost
// 26 instructions a word against 19.)  The channels of a dot product may come in any
// order as long as q's come in the same one.  q's rows are brought to f16 by a power
// of two that puts their largest value into [1, 2): values down to 2^-14 keep their
// eight bits, a smaller one moves by at most 2^-25, a quarter step of an f32 at the
// largest.  Measured: 64 ragged sequences of up to 32768, window 8192 + 4, 32 heads
// over 4 x 128, 108 us (slices of 16 tokens 122; four CTAs per SM spill, 141).  Bound by
// the instructions of the decoding, not by the 209 MB (32 us).
#include <algorithm>

#include "launchers.h"
#include "paged_attn.cuh"

namespace csa2 {
namespace {
using namespace paged;
using rope::Num;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <int D, bool FP4>
struct Lay {
  static constexpr int KS = FP4 && D <= 128 ? 32 : 16;             // tokens per slice
  static constexpr int ROW = FP4 ? D / 2 + 16 : 2 * D + 16;        // padded row in shared memory
  static constexpr int SC = FP4 ? KS * (D / 16) : 0;               // a slice's scales
  static constexpr int HALF = KS * ROW + SC;                       // keys (or values) of a slice
  static constexpr int STAGES = FP4 ? (D <= 128 ? 3 : 6) : D == 64 ? 6 : D == 128 ? 3 : 2;
  static constexpr int warp_bytes(bool shared) { return STAGES * HALF * (shared ? 1 : 2); }
  static constexpr int MERGE = kWarps * 16 * (D + 4) * 4 + kWarps * 16 * 8;
  static constexpr int bytes(bool shared) {
    return kWarps * warp_bytes(shared) > MERGE ? kWarps * warp_bytes(shared) : MERGE;
  }
};

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_16s(uint32_t dst, const void* src, uint32_t n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint32_t v;
  asm volatile("{.reg .u16 t; ld.shared.u16 t, [%1]; cvt.u32.u16 %0, t;}" : "=r"(v) : "r"(a));
  return v;
}
// The scale of a 16-channel block, `odd` of two neighbouring ones, as an f16 pair.
__device__ __forceinline__ uint32_t scale_f16(uint32_t two, bool odd) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  const uint32_t v = static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
  return __byte_perm(v, v, odd ? 0x3232 : 0x1010);
}
// Byte k of a word (channels 2 k and 2 k + 1) as an f16 pair, times a scale.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int k, uint32_t s2) {
  uint32_t d;
  asm("{.reg .b8 b, x, y, z; mov.b32 {b, x, y, z}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(d) : "r"(w >> (8 * k)));
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&d), *reinterpret_cast<__half2*>(&s2));
  return *reinterpret_cast<const uint32_t*>(&r);
}

struct Params {
  const uint16_t* q;
  int64_t q_token, q_head;
  uint16_t* out;
  float* lse;
  float* part_o;                     // [B * Hq][chunks][D]
  float2* part_ml;                   // [B * Hq][chunks]
  float scale2;                      // scale * log2(e)
  int Hq, G, row_tiles, window, sinks, chunk, chunks;
  PagedView kv;
};

template <class T, int D, bool FP4, bool SHARED>
__global__ void __launch_bounds__(kThreads) paged_decode_kernel(const Params p) {
  using L = Lay<D, FP4>;
  using M = typename std::conditional<FP4, __half, T>::type;       // type of the products
  constexpr int KS = L::KS;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n8 = lane >> 2, c4 = lane & 3;             // fragment coordinates
  const int b = blockIdx.z, chunk = blockIdx.x;
  const int kvh = blockIdx.y / p.row_tiles, h0 = 16 * (blockIdx.y % p.row_tiles);
  const int rows = min(16, p.G - h0);
  pdl_wait();
  const int len = length_of(p.kv, b, threadIdx.x == 0);
  const Seen seen(len - 1, len - 1, p.window, p.sinks);
  const int64_t c0 = static_cast<int64_t>(chunk) * p.chunk;
  if (chunk > 0 && c0 >= seen.total) return;
  const int v0 = static_cast<int>(c0);
  const int v1 = chunk + 1 < p.chunks ? min(seen.total, v0 + p.chunk) : seen.total;
  const int slices = (v1 - v0 + KS - 1) / KS;

  const uint32_t ring = sm100::smem_u32(smem) + warp * L::warp_bytes(SHARED);
  constexpr int STAGE = L::HALF * (SHARED ? 1 : 2);

  // the row (channel offset) of this lane's token in slice s; -1: none
  auto row_of = [&](int s) -> int64_t {
    const int i = v0 + s * KS + (lane & (KS - 1));
    if (s >= slices || i >= v1) return -1;
    const int64_t r = token_row(p.kv, b, seen.token(i));
    return r < 0 ? -1 : r + kvh * p.kv.head_stride;
  };
  // every token of a slice present: one bit per token
  auto issue = [&](int stage, int64_t row) -> uint32_t {
    const uint32_t dst0 = ring + stage * STAGE;
#pragma unroll
    for (int half = 0; half < (SHARED ? 1 : 2); ++half) {
      const uint8_t* src = half ? p.kv.v : p.kv.k;
      const uint32_t dst = dst0 + half * L::HALF;
      constexpr int CH = FP4 ? D / 32 : D / 8;         // 16-byte pieces of a row
#pragma unroll
      for (int i = 0; i < KS * CH / 32; ++i) {
        const int piece = i * 32 + lane, r = piece / CH, c = piece % CH;
        const int64_t at = __shfl_sync(0xffffffffu, row, r);
        cp_async_16s(dst + r * L::ROW + c * 16, src + (at < 0 ? 0 : (FP4 ? at / 2 : at * 2) + c * 16),
                     at < 0 ? 0u : 16u);
      }
      if (FP4) {
        const uint8_t* sc = half ? p.kv.v_scales : p.kv.k_scales;
        constexpr int SB = D / 16;                     // scale bytes of a row: 4, 8 or 16
        constexpr int W = SB / 4;                      // words (4-byte aligned: strides are multiples of 64)
#pragma unroll
        for (int i = 0; i < (KS * W + 31) / 32; ++i) {
          const int piece = i * 32 + lane, r = (piece / W) & (KS - 1), c = piece % W;
          const int64_t at = __shfl_sync(0xffffffffu, row, r);
          if (piece < KS * W)
            cp_async_4(dst + KS * L::ROW + r * SB + c * 4, sc + (at < 0 ? 0 : at / 16 + c * 4), at < 0 ? 0u : 4u);
        }
      }
    }
    return __ballot_sync(0xffffffffu, row >= 0);
  };

  // q fragments.  16-bit rows: the plain order.  FP4: the order of the code words:
  // thread c4 of a group of 32 channels owns channels 8 c4 .. 8 c4 + 7 as the pairs
  // (0,1) (2,3) of the first step and (4,5) (6,7) of the second.
  float scale2[2] = {p.scale2, p.scale2};              // per row of the fragment
  uint32_t qa[D / 16][4];
  {
    const uint16_t* q0 = p.q + b * p.q_token + (kvh * p.G + h0 + min(n8, rows - 1)) * p.q_head;
    const uint16_t* q1 = p.q + b * p.q_token + (kvh * p.G + h0 + min(n8 + 8, rows - 1)) * p.q_head;
    const bool ok0 = n8 < rows, ok1 = n8 + 8 < rows;
    if (!FP4) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        qa[k][0] = ok0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 16) + c4) : 0u;
        qa[k][1] = ok1 ? __ldg(reinterpret_cast<const uint32_t*>(q1 + k * 16) + c4) : 0u;
        qa[k][2] = ok0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 16) + 4 + c4) : 0u;
        qa[k][3] = ok1 ? __ldg(reinterpret_cast<const uint32_t*>(q1 + k * 16) + 4 + c4) : 0u;
      }
    } else {
#pragma unroll
      for (int g = 0; g < D / 32; ++g) {
        uint4 a = make_uint4(0, 0, 0, 0), e = a;
        if (ok0) a = __ldg(reinterpret_cast<const uint4*>(q0 + g * 32) + c4);
        if (ok1) e = __ldg(reinterpret_cast<const uint4*>(q1 + g * 32) + c4);
        qa[2 * g][0] = a.x;
        qa[2 * g][2] = a.y;
        qa[2 * g + 1][0] = a.z;
        qa[2 * g + 1][2] = a.w;
        qa[2 * g][1] = e.x;
        qa[2 * g][3] = e.y;
        qa[2 * g + 1][1] = e.z;
        qa[2 * g + 1][3] = e.w;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t top = 0;                              // largest |bf16| of the row, as bits
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t v = qa[k][u + 2 * x] & 0x7fff7fffu;
            top = max(top, max(v & 0xffffu, v >> 16));
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t eb = min(max(top >> 7, 1u), 253u);            // its biased exponent
        const float down = __uint_as_float((254u - eb) << 23);
        scale2[u] *= __uint_as_float(eb << 23);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float2 f = Num<__nv_bfloat16>::up(qa[k][u + 2 * x]);
            qa[k][u + 2 * x] = Num<__half>::down(f.x * down, f.y * down);
          }
      }
    }
  }

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

  // the ring: STAGES - 1 slices of this warp ahead
  uint32_t present[L::STAGES];
  int64_t row = row_of(warp);
#pragma unroll
  for (int i = 0; i < L::STAGES - 1; ++i) {
    present[i] = issue(i, row);
    sm100::cp_async_commit();
    row = row_of(warp + (i + 1) * kWarps);
  }
  int stage = 0;
  for (int s = warp; s < slices; s += kWarps) {
    // the slice STAGES - 1 ahead goes into the stage that the last turn freed
    sm100::cp_async_wait<L::STAGES - 2>();
    __syncwarp();
    const int ahead = stage + L::STAGES - 1 >= L::STAGES ? stage - 1 : stage + L::STAGES - 1;
    const uint32_t mask_next = issue(ahead, row);
    sm100::cp_async_commit();
    row = row_of(s + L::STAGES * kWarps);
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < L::STAGES; ++i) {
      if (i == stage) mask = present[i];
      if (i == ahead) present[i] = mask_next;
    }
    const uint32_t kb = ring + stage * STAGE, vb = SHARED ? kb : kb + L::HALF;

    constexpr int NT = KS / 8;                         // 8-token tiles of a slice
    float sc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.0f;
    if (!FP4) {
#pragma unroll
      for (int k = 0; k < D / 16; k += 2) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {                 // 8 tokens x 32 channels
          uint32_t bb[4];
          ldsm4(bb, kb + (i * 8 + (lane & 7)) * L::ROW + k * 32 + (lane >> 3) * 16);
          mma16816<M>(sc[i], qa[k], bb[0], bb[1]);
          mma16816<M>(sc[i], qa[k + 1], bb[2], bb[3]);
        }
      }
    } else {
#pragma unroll
      for (int g = 0; g < D / 32; ++g) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int r = i * 8 + n8;
          const uint32_t w = lds32(kb + r * L::ROW + (4 * g + c4) * 4);
          const uint32_t s2 = scale_f16(lds16(kb + KS * L::ROW + r * (D / 16) + 2 * g), c4 >> 1);
          mma16816<M>(sc[i], qa[2 * g], code_pair(w, 0, s2), code_pair(w, 1, s2));
          mma16816<M>(sc[i], qa[2 * g + 1], code_pair(w, 2, s2), code_pair(w, 3, s2));
        }
      }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool ok = (mask >> (i * 8 + c4 * 2 + (e & 1))) & 1u;
        sc[i][e] = ok ? sc[i][e] * scale2[e >> 1] : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], sc[i][e]);
      }
    float alpha[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
      const float mn = fmaxf(m[u], mx[u]);
      const float ref = mn == -INFINITY ? 0.0f : mn;
      alpha[u] = exp2_approx(m[u] - ref);
      m[u] = mn;
      l[u] *= alpha[u];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[i][2 * u + e] = exp2_approx(sc[i][2 * u + e] - ref);
          l[u] += sc[i][2 * u + e];
        }
    }
    uint32_t pa[KS / 16][4];                           // P as the next product's left operand
#pragma unroll
    for (int t = 0; t < KS / 16; ++t) {
      pa[t][0] = Num<M>::down(sc[2 * t][0], sc[2 * t][1]);
      pa[t][1] = Num<M>::down(sc[2 * t][2], sc[2 * t][3]);
      pa[t][2] = Num<M>::down(sc[2 * t + 1][0], sc[2 * t + 1][1]);
      pa[t][3] = Num<M>::down(sc[2 * t + 1][2], sc[2 * t + 1][3]);
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= alpha[0];
        o[i][1] *= alpha[0];
        o[i][2] *= alpha[1];
        o[i][3] *= alpha[1];
      }
    }
#pragma unroll
    for (int t = 0; t < KS / 16; ++t) {
      if (!FP4) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {             // 16 tokens x 16 channels
          uint32_t bb[4];
          ldsm4t(bb, vb + (t * 16 + (lane & 15)) * L::ROW + (i * 16 + (lane >> 4) * 8) * 2);
          mma16816<M>(o[2 * i], pa[t], bb[0], bb[1]);
          mma16816<M>(o[2 * i + 1], pa[t], bb[2], bb[3]);
        }
      } else {
        // word n8 of a group of 64 channels, of tokens 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9
#pragma unroll
        for (int g = 0; g < D / 64; ++g) {
          uint32_t w[4], s2[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = t * 16 + 2 * c4 + (u & 1) + 8 * (u >> 1);
            w[u] = lds32(vb + r * L::ROW + (8 * g + n8) * 4);
            s2[u] = scale_f16(lds16(vb + KS * L::ROW + r * (D / 16) + 4 * g + 2 * (n8 >> 2)), (n8 >> 1) & 1);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {                // channels 2 k and 2 k + 1 of the word
            const uint32_t x0 = code_pair(w[0], k, s2[0]), x1 = code_pair(w[1], k, s2[1]);
            const uint32_t y0 = code_pair(w[2], k, s2[2]), y1 = code_pair(w[3], k, s2[3]);
            mma16816<M>(o[8 * g + 2 * k], pa[t], __byte_perm(x0, x1, 0x5410), __byte_perm(y0, y1, 0x5410));
            mma16816<M>(o[8 * g + 2 * k + 1], pa[t], __byte_perm(x0, x1, 0x7632), __byte_perm(y0, y1, 0x7632));
          }
        }
      }
    }
    stage = stage + 1 == L::STAGES ? 0 : stage + 1;
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
  }
  // the warps meet: O rows padded by 4 floats, then (m, l)
  sm100::cp_async_wait<0>();
  __syncthreads();
  constexpr int PITCH = D + 4;
  float* so = reinterpret_cast<float*>(smem);
  float2* sml = reinterpret_cast<float2*>(so + kWarps * 16 * PITCH);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = n8 + 8 * u;
    float* dst = so + (warp * 16 + r) * PITCH;
    if (!FP4) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(dst + i * 8 + c4 * 2) = make_float2(o[i][2 * u], o[i][2 * u + 1]);
    } else {
      // product i of group g: column n is channel 64 g + 8 n + i
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        dst[(i / 8) * 64 + 16 * c4 + (i % 8)] = o[i][2 * u];
        dst[(i / 8) * 64 + 16 * c4 + 8 + (i % 8)] = o[i][2 * u + 1];
      }
    }
    if (c4 == 0) sml[warp * 16 + r] = make_float2(m[u], l[u]);
  }
  __syncthreads();
  const bool partial = p.chunks > 1 && seen.total > p.chunk;
  constexpr int PER = D / 4;                           // threads per row, four channels each
  for (int i = threadIdx.x; i < rows * PER; i += kThreads) {
    const int r = i / PER, c = i % PER;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sml[w * 16 + r].x);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float lr = 0.0f;
    float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * 16 + r];
      const float f = exp2_approx(ml.x - ref);
      const float4 v = *reinterpret_cast<const float4*>(so + (w * 16 + r) * PITCH + 4 * c);
      lr += f * ml.y;
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
    const int64_t at = static_cast<int64_t>(b) * p.Hq + kvh * p.G + h0 + r;
    if (partial) {
      reinterpret_cast<float4*>(p.part_o + (at * p.chunks + chunk) * D)[c] = acc;
      if (c == 0) p.part_ml[at * p.chunks + chunk] = make_float2(mx, lr);
    } else {
      const float inv = lr > 0.0f ? 1.0f / lr : (lr == 0.0f ? 0.0f : lr);
      *reinterpret_cast<uint2*>(p.out + at * D + 4 * c) =
          make_uint2(Num<T>::down(acc.x * inv, acc.y * inv), Num<T>::down(acc.z * inv, acc.w * inv));
      if (p.lse && c == 0) p.lse[at] = lr == 0.0f ? -INFINITY : (mx + log2f(lr)) * kLn2;
    }
  }
}

template <class T, int D, bool FP4, bool SHARED>
csa2_status run(const Params& p, dim3 grid, cudaStream_t stream) {
  using L = Lay<D, FP4>;
  static PerDevice<int> opted;
  opted.get(+[]() -> int {
    cudaFuncSetAttribute(paged_decode_kernel<T, D, FP4, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         L::bytes(SHARED));
    return 1;
  });
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::bytes(SHARED);
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attribute()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  begin_launch(stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<T, D, FP4, SHARED>, p);
  note_launch(LK_ATTN, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "csa2_paged_decode_attn: launch failed: %s", cudaGetErrorString(e));
  }
  return check_launch("csa2_paged_decode_attn");
}

}  // namespace

bool paged_decode_stream_applies(const PagedAttn& a) { return a.D <= 256; }

csa2_status launch_paged_decode_stream(const PagedAttn& a, int chunk, int chunks, float* part_o, float2* part_ml,
                                       cudaStream_t stream) {
  Params p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_token = a.q_token;
  p.q_head = a.q_head;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.part_o = part_o;
  p.part_ml = part_ml;
  p.scale2 = a.scale * kLog2e;
  p.Hq = a.Hq;
  p.G = a.G;
  p.row_tiles = (a.G + 15) / 16;
  p.window = a.window;
  p.sinks = a.sinks;
  p.chunk = chunk;
  p.chunks = chunks;
  p.kv = a.kv;
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(a.kv.heads * p.row_tiles),
                  static_cast<unsigned>(a.kv.B));
  const bool sh = a.kv.v == a.kv.k;
#define CSA2_STREAM_T(T_, D_, F_) (sh ? run<T_, D_, F_, true>(p, grid, stream) : run<T_, D_, F_, false>(p, grid, stream))
#define CSA2_STREAM(D_)                                                                       \
  if (a.D == D_)                                                                              \
    return a.fmt == CSA2_KV_FP4   ? CSA2_STREAM_T(__nv_bfloat16, D_, true)                    \
           : a.fmt == CSA2_KV_F16 ? CSA2_STREAM_T(__half, D_, false)                          \
                                  : CSA2_STREAM_T(__nv_bfloat16, D_, false);
  CSA2_STREAM(64) CSA2_STREAM(128) CSA2_STREAM(256)
#undef CSA2_STREAM
#undef CSA2_STREAM_T
  return CSA2_ERR_UNSUPPORTED;
}

}  // namespace csa2
