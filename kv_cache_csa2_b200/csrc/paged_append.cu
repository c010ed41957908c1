// Appending keys and values to a paged cache, the position rotation and the
// packing to FP4 on the way.
// HBM-bound: a row is read once and written once.  A CTA takes a block of
// tokens, as the head norm does (rope.cuh): rows requested, the tokens' angles
// and page addresses computed once for all heads, then the (token, head) rows.
// An FP4 block of 16 channels is the same vector of two neighbouring lanes, so
// its absolute maximum is one shuffle and each lane packs its own 8 codes.
// Measured: 8191 tokens of 8 heads x 128 (keys and values), 14.4 us (4.7 TB/s; 15.5 with
// one row ahead instead of two), about one wave, so the place and angles of a CTA's tokens
// stand at its start in full; 4096 shared rows x 512 into FP4, 9.2 us, of which the rounding to FP4 (150 instructions
// per 16 channels) is the larger part.
#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"
#include "paged.h"
#include "rope.cuh"
#include "sm100.cuh"

namespace csa2 {
namespace {
using namespace rope;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;
constexpr int kStages = 3;

struct Params {
  const uint16_t *k, *v;
  int64_t k_t, k_h, v_t, v_h;
  const int32_t *seq, *pos;
  int64_t T;
  int H, D, items, lanes;            // H = heads of k plus heads of v
  int step_t, step_h;                // a pass's rows in tokens and heads
  int tokens, rows_cta;
  RopeArgs rope;
  PagedView cache;
};

// 8 values of a 16-channel block (the neighbouring lane holds the other 8):
// codes of this lane's half, and the block's scale.
__device__ __forceinline__ uint32_t pack_half_block(const uint4& v, uint32_t* scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t amax = 0;                                  // |bf16| bits order like the values; NaN is passed over
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t lo = w[j] & 0x7fffu, hi = (w[j] >> 16) & 0x7fffu;
    if (lo <= 0x7f80u) amax = max(amax, lo);
    if (hi <= 0x7f80u) amax = max(amax, hi);
  }
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const uint32_t sc = fp4::scale_code_for(__uint_as_float(amax << 16));
  const float s = fp4::e4m3_value(sc);
  uint32_t codes = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t h = (w[j >> 1] >> (16 * (j & 1))) & 0xffffu;
    uint32_t c = s > 0.0f ? fp4::e2m1_code(__uint_as_float((h & 0x7fffu) << 16), s) : 0u;
    c |= (h >> 12) & 8u;
    codes |= c << (4 * j);
  }
  *scale = sc;
  return codes;
}

template <class T, bool FP4>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const Params p) {
  extern __shared__ uint4 smem[];
  float4* cs = reinterpret_cast<float4*>(smem);                    // angles, [tokens][half / 2]
  __shared__ int64_t s_row[kMaxTokens];                            // the token's place (head 0), -1: skip
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.T - t0));
  const int per_pass = kThreads / p.lanes;
  const int sub = threadIdx.x & (p.lanes - 1);
  const int r_end = min(nt * p.H, static_cast<int>(blockIdx.y + 1) * p.rows_cta);
  int r = blockIdx.y * p.rows_cta + threadIdx.x / p.lanes;
  Item it = item_at(sub, p.D, p.rope.half, p.rope.offset);
  if (sub >= p.items) it.c0 = it.c1 = it.freq = -1;
  const int hk = p.cache.heads;

  // a thread's own vectors, kStages - 1 passes ahead
  uint4* ring = smem + p.tokens * (p.rope.half / 2) + threadIdx.x;
  int stage = 0;
  int tl = r / p.H, head = r - tl * p.H, tl_a = tl, head_a = head;
  auto step = [&](int& t, int& h) {                    // the row a pass further
    t += p.step_t;
    h += p.step_h;
    if (h >= p.H) h -= p.H, ++t;
  };
  auto request = [&](int row, int st) {
    const bool live = row < r_end, is_k = !live || head_a < hk;
    const uint16_t* src = is_k ? p.k : p.v;
    if (live) src += (t0 + tl_a) * (is_k ? p.k_t : p.v_t) + (is_k ? head_a : head_a - hk) * (is_k ? p.k_h : p.v_h);
    uint4* dst = ring + st * 2 * kThreads;
    sm100::cp_async_16(dst, src + max(it.c0, 0), live && it.c0 >= 0 ? 16u : 0u);
    sm100::cp_async_16(dst + kThreads, src + max(it.c1, 0), live && it.c1 >= 0 ? 16u : 0u);
    sm100::cp_async_commit();
    step(tl_a, head_a);
  };
  pdl_wait();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) request(r + i * per_pass, i);
  if (threadIdx.x < nt) {
    const int64_t t = t0 + threadIdx.x;
    const int s = __ldg(p.seq + t);
    int64_t row = -1;
    if (s != -1) {
      const int pos = __ldg(p.pos + t);
      bool ok = s >= 0 && s < p.cache.B && pos >= 0 && pos < p.cache.capacity;
      if (ok) {
        const int page = __ldg(p.cache.table + s * p.cache.table_stride + (pos >> p.cache.page_shift));
        ok = page >= 0 && page < p.cache.n_pages;
        if (ok) row = p.cache.row(page, pos & ((1 << p.cache.page_shift) - 1), 0);
      }
      if (!ok) raise_dev_error(p.cache.err, DEVERR_BOUNDS);
    }
    s_row[threadIdx.x] = row;
  }
  if (p.rope.inv_freq) {
    for (int i = threadIdx.x; i < nt * p.rope.half; i += kThreads) {
      const int t = i / p.rope.half, f = i - t * p.rope.half;
      put_angle(cs + t * (p.rope.half / 2), f, p.rope.half,
                angle_of(__ldg(p.pos + t0 + t), __ldg(p.rope.inv_freq + f), p.rope.inverse));
    }
  }
  __syncthreads();
  // all lanes of a warp stay in the loop together (the shuffles need them)
  for (int base = blockIdx.y * p.rows_cta; base < r_end; base += per_pass, r += per_pass) {
    sm100::cp_async_wait<kStages - 2>();
    uint4 a = ring[stage * 2 * kThreads], b = ring[stage * 2 * kThreads + kThreads];
    request(r + (kStages - 1) * per_pass, stage == 0 ? kStages - 1 : stage - 1);
    stage = stage == kStages - 1 ? 0 : stage + 1;
    const bool live = r < r_end, is_k = head < hk;
    const int my_t = tl, my_h = is_k ? head : head - hk;
    step(tl, head);
    if (live && is_k && p.rope.inv_freq && it.freq >= 0) {
      float2 x0[4], x1[4];
      unpack8<T>(a, x0);
      unpack8<T>(b, x1);
      rotate_item(x0, x1, it, p.rope.half, p.rope.interleaved, cs + my_t * (p.rope.half / 2));
      a = pack8<T>(x0);
      b = pack8<T>(x1);
    }
    uint32_t ca = 0, cb = 0, sa = 0, sb = 0;
    if (FP4) {
      ca = pack_half_block(a, &sa);
      cb = pack_half_block(b, &sb);
    }
    const int64_t row0 = live ? s_row[my_t] : -1;
    if (row0 < 0) continue;
    const int64_t row = row0 + my_h * p.cache.head_stride;
    uint8_t* base_p = const_cast<uint8_t*>(is_k ? p.cache.k : p.cache.v);
    if (FP4) {
      uint8_t* scales = const_cast<uint8_t*>(is_k ? p.cache.k_scales : p.cache.v_scales);
      if (it.c0 >= 0) {
        *reinterpret_cast<uint32_t*>(base_p + (row + it.c0) / 2) = ca;
        if ((it.c0 & 15) == 0) scales[(row + it.c0) / 16] = static_cast<uint8_t>(sa);
      }
      if (it.c1 >= 0) {
        *reinterpret_cast<uint32_t*>(base_p + (row + it.c1) / 2) = cb;
        if ((it.c1 & 15) == 0) scales[(row + it.c1) / 16] = static_cast<uint8_t>(sb);
      }
    } else {
      uint16_t* dst = reinterpret_cast<uint16_t*>(base_p) + row;
      if (it.c0 >= 0) *reinterpret_cast<uint4*>(dst + it.c0) = a;
      if (it.c1 >= 0) *reinterpret_cast<uint4*>(dst + it.c1) = b;
    }
  }
  sm100::cp_async_wait<0>();
}

}  // namespace

csa2_status launch_paged_append(csa2_dtype dtype, const HeadRows& k, const HeadRows& v,
                                const int32_t* seq, const int32_t* pos, int64_t T, int D, bool fp4,
                                const RopeArgs& rope, const PagedView& cache, cudaStream_t stream) {
  Params p = {};
  p.k = static_cast<const uint16_t*>(k.data);
  p.v = static_cast<const uint16_t*>(v.data);
  p.k_t = k.token_stride;
  p.k_h = k.head_stride;
  p.v_t = v.token_stride;
  p.v_h = v.head_stride;
  p.seq = seq;
  p.pos = pos;
  p.T = T;
  p.H = k.heads + v.heads;
  p.D = D;
  p.rope = rope;
  p.cache = cache;
  p.items = items_of(D, rope.half);
  p.lanes = 1;
  while (p.lanes < p.items) p.lanes *= 2;
  const int per_pass = kThreads / p.lanes;
  p.step_t = per_pass / p.H;
  p.step_h = per_pass % p.H;
  const int sms = sm_count();
  // tokens per CTA as in the head norm
  p.tokens = kMaxTokens;
  while (p.tokens > 1 && p.tokens * p.H > per_pass && T / p.tokens < 4 * sms) p.tokens /= 2;
  const int64_t gx = (T + p.tokens - 1) / p.tokens;
  const int passes = (p.tokens * p.H + per_pass - 1) / per_pass;
  int ny = 1;
  if (gx < 2 * sms) ny = static_cast<int>(std::min<int64_t>(passes, (2 * sms + gx - 1) / gx));
  p.rows_cta = (passes + ny - 1) / ny * per_pass;
  ny = (p.tokens * p.H + p.rows_cta - 1) / p.rows_cta;
  if (gx > 0x7fffffffLL) return fail(CSA2_ERR_UNSUPPORTED, "csa2_paged_append: too many tokens");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(ny));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.tokens) * rope.half * sizeof(float2) + kStages * 2 * kThreads * 16;
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attribute()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  begin_launch(stream);
  const cudaError_t e =
      fp4 ? cudaLaunchKernelEx(&cfg, paged_append_kernel<__nv_bfloat16, true>, p)
          : dtype == CSA2_F16 ? cudaLaunchKernelEx(&cfg, paged_append_kernel<__half, false>, p)
                              : cudaLaunchKernelEx(&cfg, paged_append_kernel<__nv_bfloat16, false>, p);
  note_launch(LK_OTHER, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "csa2_paged_append: launch failed: %s", cudaGetErrorString(e));
  }
  return check_launch("csa2_paged_append");
}

}  // namespace csa2
