// Attention of one new token per sequence over a paged cache, rows of 64, 128 or
// 256 channels, FP4 rows of 512 too: up to 16 query heads of one cache head per CTA, the
// sequence's visible tokens cut into chunks over CTAs.
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
// (6.05 TB/s, 0.92 of a plain copy's rate; 250 run for seconds, at the power limit's 1570
// MHz); one sequence of 8192 with its join, 8.9 us.
//
// FP4 rows stay packed in shared memory and become f16 in registers by the hardware's
// E2M1 conversion and one product with the scale: a code times a scale has five
// significant bits between 2^-10 and 2^12, exact in f16.  What bounds it is this
// arithmetic (the integer pipe), so the products stand the other way round, with
// columns of 8 heads:
//   S^T[16 tokens, heads] = k q^T,  P^T turned by movmatrix,  O^T[channels, heads] += v^T P
// The channels of a dot product and the rows of an output may come in any order, so a
// thread takes whole runs of a row's codes (16 bytes of keys, 8 of values at 128
// channels, each with its own scales); the value product wants two tokens of a channel
// side by side, and their codes are paired before they are converted.  q's rows are
// brought to f16 by a power of two that puts their largest value into [1, 2): values down to
// 2^-14 keep their eight bits, a smaller one moves by at most 2^-25, a quarter step of
// an f32 at the largest.  Measured: 64 ragged sequences of up to 32768, window 8192 + 4,
// 32 heads over 4 x 128 (209 MB, 32 us at the copy rate): heads as rows 108 us, this way
// 79, chunks of 1024 tokens 74, bytes of a word by the conversion's own operand instead
// of shifts 68, row addresses once for keys and values 65; four CTAs per SM.  Rows of 512
// channels take 8 heads per CTA, so 64 heads decode a row 8 times: 32 sequences of 8192,
// 64 heads over one row 282 us (16-row tiles of paged_attn.cu 653), 8 heads 48 (168).

#include <algorithm>

#include "launchers.h"
#include "paged_attn.cuh"

namespace csa2 {
namespace {
using namespace paged;
using rope::Num;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

template <int D, bool FP4, int HT>
struct Lay {
  static constexpr int ROWS = 8 * HT;                              // query rows of a CTA
  static constexpr int KS = FP4 && D <= 128 ? 32 : 16;             // tokens per slice
  static constexpr int ROW = FP4 ? D / 2 + 16 : 2 * D + 16;        // padded row in shared memory
  static constexpr int SC = FP4 ? KS * (D / 16) : 0;               // a slice's scales
  static constexpr int HALF = KS * ROW + SC;                       // keys (or values) of a slice
  static constexpr int STAGES = FP4 ? (D <= 128 ? (HT == 1 ? 2 : 3) : D == 256 ? 6 : 3) : D == 64 ? 6 : D == 128 ? 3 : 2;
  static constexpr int warp_bytes(bool shared) { return STAGES * HALF * (shared ? 1 : 2); }
  static constexpr int MERGE = kWarps * ROWS * (D + 4) * 4 + kWarps * ROWS * 8;
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
// N words, or N bytes, from shared memory.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], uint32_t a) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(a));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                   : "r"(a + 4 * i));
  }
}
template <int N>
__device__ __forceinline__ uint32_t lds_bytes(uint32_t a) {
  uint32_t v = 0;
  if constexpr (N == 1) asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  if constexpr (N == 2) asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// Two E4M3 scales (the low bytes) as an f16 pair.
__device__ __forceinline__ uint32_t scales_f16(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
// The transpose of an 8 x 8 matrix of 16-bit values, one register a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// The two codes of byte k of a word as an f16 pair, times a pair of scales.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int k, uint32_t s2) {
  uint32_t d;
  if (k == 0) asm("{.reg .b8 b, x, y, z; mov.b32 {b, x, y, z}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(d) : "r"(w));
  if (k == 1) asm("{.reg .b8 b, x, y, z; mov.b32 {x, b, y, z}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(d) : "r"(w));
  if (k == 2) asm("{.reg .b8 b, x, y, z; mov.b32 {x, y, b, z}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(d) : "r"(w));
  if (k == 3) asm("{.reg .b8 b, x, y, z; mov.b32 {x, y, z, b}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(d) : "r"(w));
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

template <class T, int D, bool FP4, bool SHARED, int HT>
__global__ void __launch_bounds__(kThreads, FP4 && D <= 128 && HT == 1 ? 4 : 1) paged_decode_kernel(const Params p) {
  using L = Lay<D, FP4, HT>;
  using M = typename std::conditional<FP4, __half, T>::type;       // type of the products
  // weights in f16 stand 2^15 above the largest's 1, so that they keep 11 bits down to
  // 2^-29 of it (f16's last step would else be 2^-24); sums, outputs and references all
  // count in these lifted units
  constexpr float LIFT = std::is_same<M, __half>::value ? 15.0f : 0.0f;
  constexpr int KS = L::KS;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n8 = lane >> 2, c4 = lane & 3;             // fragment coordinates
  const int b = blockIdx.z, chunk = blockIdx.x;
  const int kvh = blockIdx.y / p.row_tiles, h0 = L::ROWS * (blockIdx.y % p.row_tiles);
  const int rows = min(L::ROWS, p.G - h0);
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
    constexpr int HALVES = SHARED ? 1 : 2;
    constexpr int CH = FP4 ? D / 32 : D / 8;           // 16-byte pieces of a row
#pragma unroll
    for (int i = 0; i < KS * CH / 32; ++i) {
      const int piece = i * 32 + lane, r = piece / CH, c = piece % CH;
      const int64_t at = __shfl_sync(0xffffffffu, row, r);
      const int64_t off = at < 0 ? 0 : (FP4 ? at >> 1 : at * 2) + c * 16;
      const uint32_t n = at < 0 ? 0u : 16u, dst = dst0 + r * L::ROW + c * 16;
#pragma unroll
      for (int half = 0; half < HALVES; ++half) cp_async_16s(dst + half * L::HALF, (half ? p.kv.v : p.kv.k) + off, n);
    }
    if constexpr (FP4) {
      constexpr int SB = D / 16;                       // scale bytes of a row: 4, 8 or 16
      constexpr int W = SB / 4;                        // words (4-byte aligned: strides are multiples of 64)
#pragma unroll
      for (int i = 0; i < (KS * W + 31) / 32; ++i) {
        const int piece = i * 32 + lane, r = (piece / W) & (KS - 1), c = piece % W;
        const int64_t at = __shfl_sync(0xffffffffu, row, r);
        const int64_t off = at < 0 ? 0 : (at >> 4) + c * 4;
        const uint32_t n = at < 0 ? 0u : 4u, dst = dst0 + KS * L::ROW + r * SB + c * 4;
        if (piece < KS * W) {
#pragma unroll
          for (int half = 0; half < HALVES; ++half)
            cp_async_4(dst + half * L::HALF, (half ? p.kv.v_scales : p.kv.k_scales) + off, n);
        }
      }
    }
    return __ballot_sync(0xffffffffu, row >= 0);
  };

  // 16-bit rows: q is the left operand, rows n8 and n8 + 8 of it this thread's.
  // FP4: the right one, columns 8 h + n8; thread c4 of a row owns the D / 4 channels
  // from c4 * D / 4 on, a code word per two steps: its pairs (0,1) (2,3) and (4,5) (6,7).
  constexpr int NW = D / 32;                           // code words of a thread in a key row
  constexpr int W = D / 64;                            // and in a value row
  uint32_t qa[D / 16][4];
  uint32_t qb[HT][2 * NW][2];
  float scale2[HT][2];                                 // per row / column of the scores
#pragma unroll
  for (int h = 0; h < HT; ++h) scale2[h][0] = scale2[h][1] = p.scale2;
  if constexpr (!FP4) {
    const uint16_t* q0 = p.q + b * p.q_token + (kvh * p.G + h0 + min(n8, rows - 1)) * p.q_head;
    const uint16_t* q1 = p.q + b * p.q_token + (kvh * p.G + h0 + min(n8 + 8, rows - 1)) * p.q_head;
    const bool ok0 = n8 < rows, ok1 = n8 + 8 < rows;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      qa[k][0] = ok0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 16) + c4) : 0u;
      qa[k][1] = ok1 ? __ldg(reinterpret_cast<const uint32_t*>(q1 + k * 16) + c4) : 0u;
      qa[k][2] = ok0 ? __ldg(reinterpret_cast<const uint32_t*>(q0 + k * 16) + 4 + c4) : 0u;
      qa[k][3] = ok1 ? __ldg(reinterpret_cast<const uint32_t*>(q1 + k * 16) + 4 + c4) : 0u;
    }
  } else {
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      const int r = 8 * h + n8;
      const uint16_t* q = p.q + b * p.q_token + (kvh * p.G + h0 + min(r, rows - 1)) * p.q_head + c4 * (D / 4);
      uint32_t top = 0;                                // largest |bf16| of the row, as bits
#pragma unroll
      for (int j = 0; j < NW; ++j) {
        uint4 a = make_uint4(0, 0, 0, 0);
        if (r < rows) a = __ldg(reinterpret_cast<const uint4*>(q) + j);
        qb[h][2 * j][0] = a.x;
        qb[h][2 * j][1] = a.y;
        qb[h][2 * j + 1][0] = a.z;
        qb[h][2 * j + 1][1] = a.w;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t v = qb[h][2 * j + x / 2][x & 1] & 0x7fff7fffu;
          top = max(top, max(v & 0xffffu, v >> 16));
        }
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t eb = min(max(top >> 7, 1u), 253u);              // its biased exponent
      const float down = __uint_as_float((254u - eb) << 23);
#pragma unroll
      for (int j = 0; j < 2 * NW; ++j)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 f = Num<__nv_bfloat16>::up(qb[h][j][x]);
          qb[h][j][x] = Num<__half>::down(f.x * down, f.y * down);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e)                      // this thread's columns are heads 2 c4 + e
        scale2[h][e] *= __uint_as_float(__shfl_sync(0xffffffffu, eb, 4 * (2 * c4 + e)) << 23);
    }
  }

  // 16-bit rows: o[n tile of 8 channels], rows n8, n8 + 8.  FP4: o[HT * product + h]
  float o[FP4 ? HT * D / 16 : D / 8][4];
  constexpr int NO = sizeof(o) / sizeof(o[0]);
#pragma unroll
  for (int i = 0; i < NO; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  constexpr int HS = FP4 ? HT : 1;                     // pairs of query rows of a thread
  float m[HS][2], l[HS][2];
#pragma unroll
  for (int h = 0; h < HS; ++h) {
    m[h][0] = m[h][1] = -INFINITY;
    l[h][0] = l[h][1] = 0.0f;
  }

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

    if constexpr (!FP4) {
      constexpr int NT = KS / 8;                       // 8-token tiles of a slice
      float sc[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.0f;
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
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool ok = (mask >> (i * 8 + c4 * 2 + (e & 1))) & 1u;
          sc[i][e] = ok ? sc[i][e] * p.scale2 : -INFINITY;
          mx[e >> 1] = fmaxf(mx[e >> 1], sc[i][e]);
        }
      float alpha[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
        mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
        const float mn = fmaxf(m[0][u], mx[u]);
        const float ref = mn == -INFINITY ? 0.0f : lifted(mn, LIFT);
        alpha[u] = exp2_approx(lifted(m[0][u], LIFT) - ref);
        m[0][u] = mn;
        l[0][u] *= alpha[u];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            sc[i][2 * u + e] = exp2_approx(sc[i][2 * u + e] - ref);
            l[0][u] += sc[i][2 * u + e];
          }
      }
      uint32_t pa[KS / 16][4];                         // P as the next product's left operand
#pragma unroll
      for (int t = 0; t < KS / 16; ++t) {
        pa[t][0] = Num<M>::down(sc[2 * t][0], sc[2 * t][1]);
        pa[t][1] = Num<M>::down(sc[2 * t][2], sc[2 * t][3]);
        pa[t][2] = Num<M>::down(sc[2 * t + 1][0], sc[2 * t + 1][1]);
        pa[t][3] = Num<M>::down(sc[2 * t + 1][2], sc[2 * t + 1][3]);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.0f || alpha[1] != 1.0f)) {
#pragma unroll
        for (int i = 0; i < NO; ++i) {
          o[i][0] *= alpha[0];
          o[i][1] *= alpha[0];
          o[i][2] *= alpha[1];
          o[i][3] *= alpha[1];
        }
      }
#pragma unroll
      for (int t = 0; t < KS / 16; ++t)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {             // 16 tokens x 16 channels
          uint32_t bb[4];
          ldsm4t(bb, vb + (t * 16 + (lane & 15)) * L::ROW + (i * 16 + (lane >> 4) * 8) * 2);
          mma16816<M>(o[2 * i], pa[t], bb[0], bb[1]);
          mma16816<M>(o[2 * i + 1], pa[t], bb[2], bb[3]);
        }
    } else {
      constexpr int MT = KS / 16;                      // 16-token tiles of a slice
      float sc[MT][HT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int h = 0; h < HT; ++h) sc[i][h][0] = sc[i][h][1] = sc[i][h][2] = sc[i][h][3] = 0.0f;
        constexpr int NC = NW < 4 ? NW : 4;            // code words at a time
#pragma unroll
        for (int j0 = 0; j0 < NW; j0 += NC) {
          uint32_t w[2][NC], s2[2];                    // tokens n8 and n8 + 8
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = i * 16 + 8 * u + n8;
            lds_words<NC>(w[u], kb + r * L::ROW + c4 * (D / 8) + 4 * j0);
            s2[u] = scales_f16(lds_bytes<NC / 2>(kb + KS * L::ROW + r * (D / 16) + c4 * (D / 64) + j0 / 2));
          }
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            uint32_t s[2];                             // the scale of word j's block, twice
#pragma unroll
            for (int u = 0; u < 2; ++u) s[u] = __byte_perm(s2[u], 0u, (j / 2) & 1 ? 0x3232 : 0x1010);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t a[4] = {code_pair(w[0][j], 2 * x, s[0]), code_pair(w[1][j], 2 * x, s[1]),
                                     code_pair(w[0][j], 2 * x + 1, s[0]), code_pair(w[1][j], 2 * x + 1, s[1])};
#pragma unroll
              for (int h = 0; h < HT; ++h)
                mma16816<M>(sc[i][h], a, qb[h][2 * (j0 + j) + x][0], qb[h][2 * (j0 + j) + x][1]);
            }
          }
        }
      }
      uint32_t pb[MT][HT][2];                          // P as the next product's right operand
      bool moved = false;
      float alpha[HT][2];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[i][h][e] *= scale2[h][e & 1];
          }
        if (mask != 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!((mask >> (i * 16 + n8 + 8 * (e >> 1))) & 1u)) sc[i][h][e] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) mx[u] = max3(mx[u], sc[i][h][u], sc[i][h][2 + u]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
#pragma unroll
          for (int x = 4; x < 32; x *= 2) mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], x));
          const float mn = fmaxf(m[h][u], mx[u]);
          const float ref = mn == -INFINITY ? 0.0f : lifted(mn, LIFT);
          alpha[h][u] = exp2_approx(lifted(m[h][u], LIFT) - ref);
          moved |= alpha[h][u] != 1.0f;
          m[h][u] = mn;
          l[h][u] *= alpha[h][u];
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sc[i][h][2 * e + u] = exp2_approx(sc[i][h][2 * e + u] - ref);
              l[h][u] += sc[i][h][2 * e + u];
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            pb[i][h][e] = transpose8(Num<M>::down(sc[i][h][2 * e], sc[i][h][2 * e + 1]));
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int i = 0; i < NO; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[i][e] *= alpha[i % HT][e & 1];
      }
      // a thread takes W words (8 W channels) of tokens 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9;
      // the codes of two tokens are paired before they are converted
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        constexpr int WC = W < 4 ? W : 4;              // words at a time
#pragma unroll
        for (int w0 = 0; w0 < W; w0 += WC) {
          constexpr int SN = WC == 4 ? 2 : 1;          // their scale bytes
          uint32_t ev[2][WC], od[2][WC], s[2][SN];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int r = t * 16 + 8 * u + 2 * c4;
            uint32_t x[WC], y[WC];
            lds_words<WC>(x, vb + r * L::ROW + n8 * (4 * W) + 4 * w0);
            lds_words<WC>(y, vb + (r + 1) * L::ROW + n8 * (4 * W) + 4 * w0);
            const uint32_t at = vb + KS * L::ROW + r * (D / 16) + (n8 * W + w0) / 2;
            const uint32_t sx = lds_bytes<SN>(at), sy = lds_bytes<SN>(at + D / 16);
            s[u][0] = scales_f16(__byte_perm(sx, sy, 0x0040));
            if (SN == 2) s[u][SN - 1] = scales_f16(__byte_perm(sx, sy, 0x0051));
#pragma unroll
            for (int j = 0; j < WC; ++j) {
              ev[u][j] = (x[j] & 0x0f0f0f0fu) | ((y[j] << 4) & 0xf0f0f0f0u);
              od[u][j] = ((x[j] >> 4) & 0x0f0f0f0fu) | (y[j] & 0xf0f0f0f0u);
            }
          }
#pragma unroll
          for (int i = 0; i < 4 * WC; ++i) {           // channel i of the lower, of the upper rows
            const int c = W == 1 ? i : i & 7, j = W == 1 ? 0 : 2 * (i / 8), jh = W == 1 ? 0 : j + 1;
            const int kl = c / 2, kh = W == 1 ? 2 + c / 2 : c / 2;
            uint32_t a[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              a[2 * u] = code_pair(c & 1 ? od[u][j] : ev[u][j], kl, s[u][SN == 2 ? i / 8 : 0]);
              a[2 * u + 1] = code_pair(c & 1 ? od[u][jh] : ev[u][jh], kh, s[u][SN == 2 ? i / 8 : 0]);
            }
#pragma unroll
            for (int h = 0; h < HT; ++h) mma16816<M>(o[HT * (4 * w0 + i) + h], a, pb[t][h][0], pb[t][h][1]);
          }
        }
      }
    }
    stage = stage + 1 == L::STAGES ? 0 : stage + 1;
  }
  // the warps meet: O rows padded by 4 floats, then (m, l)
  sm100::cp_async_wait<0>();
  __syncthreads();
  constexpr int PITCH = D + 4;
  float* so = reinterpret_cast<float*>(smem);
  float2* sml = reinterpret_cast<float2*>(so + kWarps * L::ROWS * PITCH);
  if constexpr (!FP4) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = n8 + 8 * u;
      float* dst = so + (warp * L::ROWS + r) * PITCH;
      l[0][u] += __shfl_xor_sync(0xffffffffu, l[0][u], 1);
      l[0][u] += __shfl_xor_sync(0xffffffffu, l[0][u], 2);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(dst + i * 8 + c4 * 2) = make_float2(o[i][2 * u], o[i][2 * u + 1]);
      if (c4 == 0) sml[warp * L::ROWS + r] = make_float2(lifted(m[0][u], LIFT), l[0][u]);
    }
  } else {
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int r = 8 * h + 2 * c4 + u;
        float* dst = so + (warp * L::ROWS + r) * PITCH + n8 * (8 * W);
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[h][u] += __shfl_xor_sync(0xffffffffu, l[h][u], x);
#pragma unroll
        for (int i = 0; i < D / 16; i += 4)            // channels i .. i + 3 of the lower, of the upper rows
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(dst + (W == 1 ? 4 * e : 16 * (i / 8) + 8 * e + (i & 7))) =
                make_float4(o[HT * i + h][2 * e + u], o[HT * (i + 1) + h][2 * e + u], o[HT * (i + 2) + h][2 * e + u],
                            o[HT * (i + 3) + h][2 * e + u]);
        if (n8 == 0) sml[warp * L::ROWS + r] = make_float2(lifted(m[h][u], LIFT), l[h][u]);
      }
  }
  __syncthreads();
  const bool partial = p.chunks > 1 && seen.total > p.chunk;
  constexpr int PER = D / 4;                           // threads per row, four channels each
  for (int i = threadIdx.x; i < rows * PER; i += kThreads) {
    const int r = i / PER, c = i % PER;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sml[w * L::ROWS + r].x);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float lr = 0.0f;
    float4 acc = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * L::ROWS + r];
      const float f = exp2_approx(ml.x - ref);
      const float4 v = *reinterpret_cast<const float4*>(so + (w * L::ROWS + r) * PITCH + 4 * c);
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

template <class T, int D, bool FP4, bool SHARED, int HT>
csa2_status run(const Params& p, dim3 grid, cudaStream_t stream) {
  using L = Lay<D, FP4, HT>;
  static PerDevice<int> opted;
  opted.get(+[]() -> int {
    cudaFuncSetAttribute(paged_decode_kernel<T, D, FP4, SHARED, HT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<T, D, FP4, SHARED, HT>, p);
  note_launch(LK_ATTN, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "csa2_paged_decode_attn: launch failed: %s", cudaGetErrorString(e));
  }
  return check_launch("csa2_paged_decode_attn");
}

}  // namespace

// FP4 rows under up to 8 heads take products of 8 columns; 512 channels have registers
// for no more.  16-bit rows have 16 query rows either way.
int paged_decode_heads(const PagedAttn& a) { return a.fmt == CSA2_KV_FP4 && (a.G <= 8 || a.D == 512) ? 8 : 16; }
bool paged_decode_stream_applies(const PagedAttn& a) { return a.D <= 256 || a.fmt == CSA2_KV_FP4; }

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
  const int ht = paged_decode_heads(a) / 8;
  p.row_tiles = (a.G + 8 * ht - 1) / (8 * ht);
  p.window = a.window;
  p.sinks = a.sinks;
  p.chunk = chunk;
  p.chunks = chunks;
  p.kv = a.kv;
  const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>(a.kv.heads * p.row_tiles),
                  static_cast<unsigned>(a.kv.B));
  const bool sh = a.kv.v == a.kv.k;
#define CSA2_STREAM_T(T_, D_, F_, H_) (sh ? run<T_, D_, F_, true, H_>(p, grid, stream) : run<T_, D_, F_, false, H_>(p, grid, stream))
#define CSA2_STREAM(D_)                                                                       \
  if (a.D == D_)                                                                              \
    return a.fmt == CSA2_KV_FP4   ? (ht == 1 ? CSA2_STREAM_T(__nv_bfloat16, D_, true, 1) : CSA2_STREAM_T(__nv_bfloat16, D_, true, 2)) \
           : a.fmt == CSA2_KV_F16 ? CSA2_STREAM_T(__half, D_, false, 2)                       \
                                  : CSA2_STREAM_T(__nv_bfloat16, D_, false, 2);
  CSA2_STREAM(64) CSA2_STREAM(128) CSA2_STREAM(256)
  if (a.D == 512) return CSA2_STREAM_T(__nv_bfloat16, 512, true, 1);
#undef CSA2_STREAM
#undef CSA2_STREAM_T
  return CSA2_ERR_UNSUPPORTED;
}

}  // namespace csa2
