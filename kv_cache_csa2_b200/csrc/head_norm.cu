// RMS norm and position rotation of query and key heads in one pass:
//   y = x * rsqrt(mean(x^2) + eps) * weight, then the rotated pairs turn by
//   positions[t] * inv_freq.
// HBM-bound (each channel is read and written once, two bytes each way).  A CTA
// takes a block of tokens: it requests its first rows, computes the tokens'
// angles once for all heads into shared memory, and then runs over the
// (token, head) rows; a group of lanes holds a row, the norm is a shuffle sum.
// Rows come by cp.async into a thread's own slots, two passes ahead.
// Measured: 8192 tokens of 64 + 8 heads x 128, 52.2 us (5.79 TB/s, 0.88 of the copy rate;
// 57.5 with the next row in registers; on another card 53.9); 4096 of 64 + 1 heads x 512, 98.6
// us (5.53 TB/s; 107.5 with 64-bit offsets and rows in registers; on another card 101.7).  Run
// for seconds, at the power limit's 1760 MHz, 60.5 and 113.  Next to the memory stands instruction
// issue (every product and sum of the rotation rounds by itself); three or five
// CTAs per SM (54.4, 55), a stage more (53.3) and the weights in registers are slower.

#include <algorithm>

#include "common.cuh"
#include "launchers.h"
#include "paged.h"
#include "sm100.cuh"
#include "rope.cuh"

namespace csa2 {
namespace {
using namespace rope;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;
constexpr int kStages = 3;

struct Side {
  const uint16_t* in;
  uint16_t* out;
  const float* weight;               // null: no norm
  int64_t in_t, in_h, out_t, out_h;  // strides in elements
};

struct Params {
  Side q, k;
  const int32_t* positions;
  int64_t T;
  int Hq, H, D, items, lanes;        // H = query plus key heads; lanes per row (power of two)
  int step_t, step_h;                // a pass's rows in tokens and heads
  int tokens, rows_cta;              // tokens per CTA, rows per CTA (grid.y cuts a token's heads)
  float eps, inv_d;
  RopeArgs rope;
};

// The offset of row (t, head) in a side's tensor: 32 bits where a CTA's rows allow it.
template <class O>
__device__ __forceinline__ O offset_of(int t, int64_t st, int head, int64_t sh) {
  return static_cast<O>(t) * static_cast<O>(st) + static_cast<O>(head) * static_cast<O>(sh);
}

__device__ __forceinline__ void scale8(float2 (&x)[4], float inv, const float* w) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w)), b = __ldg(reinterpret_cast<const float4*>(w) + 1);
  const float2 i2 = make_float2(inv, inv);
  x[0] = mul2(mul2(x[0], i2), make_float2(a.x, a.y));
  x[1] = mul2(mul2(x[1], i2), make_float2(a.z, a.w));
  x[2] = mul2(mul2(x[2], i2), make_float2(b.x, b.y));
  x[3] = mul2(mul2(x[3], i2), make_float2(b.z, b.w));
}

// O: the type of offsets among a CTA's rows (64-bit ones cost a quarter of the instructions)
template <class T, class O>
__global__ void __launch_bounds__(kThreads, 4) head_norm_kernel(const Params p) {
  extern __shared__ uint4 smem[];
  float4* cs = reinterpret_cast<float4*>(smem);        // angles, [tokens][half / 2]
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.T - t0));
  const int per_pass = kThreads / p.lanes;
  const int sub = threadIdx.x & (p.lanes - 1);
  const int r_end = min(nt * p.H, static_cast<int>(blockIdx.y + 1) * p.rows_cta);
  int r = blockIdx.y * p.rows_cta + threadIdx.x / p.lanes;
  Item it = item_at(sub, p.D, p.rope.half, p.rope.offset);
  if (sub >= p.items) it.c0 = it.c1 = it.freq = -1;

  const uint16_t *q_in = p.q.in + t0 * p.q.in_t, *k_in = p.k.in + t0 * p.k.in_t;
  uint16_t *q_out = p.q.out + t0 * p.q.out_t, *k_out = p.k.out + t0 * p.k.out_t;
  // a thread's own vectors, kStages - 1 passes ahead
  uint4* ring = smem + p.tokens * (p.rope.half / 2) + threadIdx.x;
  int stage = 0;
  int tl = r / p.H, head = r - tl * p.H, tl_a = tl, head_a = head;
  auto step = [&](int& t, int& h) {                    // the row a pass further
    t += p.step_t;
    h += p.step_h;
    if (h >= p.H) h -= p.H, ++t;
  };
  auto request = [&](int row, int stage) {
    const bool live = row < r_end, q = live ? head_a < p.Hq : p.Hq > 0;
    const uint16_t* src = (q ? q_in : k_in) + (live ? offset_of<O>(tl_a, q ? p.q.in_t : p.k.in_t,
                                                                   q ? head_a : head_a - p.Hq,
                                                                   q ? p.q.in_h : p.k.in_h) : 0);
    uint4* dst = ring + stage * 2 * kThreads;
    sm100::cp_async_16(dst, src + max(it.c0, 0), live && it.c0 >= 0 ? 16u : 0u);
    sm100::cp_async_16(dst + kThreads, src + max(it.c1, 0), live && it.c1 >= 0 ? 16u : 0u);
    sm100::cp_async_commit();
    step(tl_a, head_a);
  };
  pdl_wait();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) request(r + i * per_pass, i);
  if (p.rope.inv_freq) {
    for (int i = threadIdx.x; i < nt * p.rope.half; i += kThreads) {
      const int t = i / p.rope.half, f = i - t * p.rope.half;
      put_angle(cs + t * (p.rope.half / 2), f, p.rope.half,
                angle_of(__ldg(p.positions + t0 + t), __ldg(p.rope.inv_freq + f), p.rope.inverse));
    }
    __syncthreads();
  }
  // all lanes of a warp stay in the loop together (the shuffles need them)
  for (int base = blockIdx.y * p.rows_cta; base < r_end; base += per_pass, r += per_pass) {
    sm100::cp_async_wait<kStages - 2>();
    float2 x0[4], x1[4];
    unpack8<T>(ring[stage * 2 * kThreads], x0);
    unpack8<T>(ring[stage * 2 * kThreads + kThreads], x1);
    request(r + (kStages - 1) * per_pass, stage == 0 ? kStages - 1 : stage - 1);
    stage = stage == kStages - 1 ? 0 : stage + 1;
    const bool live = r < r_end, is_q = head < p.Hq;
    const int my_t = tl, my_h = head;
    const float* w = is_q ? p.q.weight : p.k.weight;
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u) sum += (x0[u].x * x0[u].x + x0[u].y * x0[u].y) + (x1[u].x * x1[u].x + x1[u].y * x1[u].y);
    for (int o = p.lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // a row is read whole by its lanes before any of them stores (the shuffle
    // above), so an output may be its input
    step(tl, head);
    if (!live) continue;
    if (w) {
      const float inv = rsqrtf(sum * p.inv_d + p.eps);
      if (it.c0 >= 0) scale8(x0, inv, w + it.c0);
      if (it.c1 >= 0) scale8(x1, inv, w + it.c1);
    }
    if (p.rope.inv_freq) rotate_item(x0, x1, it, p.rope.half, p.rope.interleaved, cs + my_t * (p.rope.half / 2));
    uint16_t* dst = (is_q ? q_out : k_out) + offset_of<O>(my_t, is_q ? p.q.out_t : p.k.out_t,
                                                          is_q ? my_h : my_h - p.Hq, is_q ? p.q.out_h : p.k.out_h);
    if (it.c0 >= 0) *reinterpret_cast<uint4*>(dst + it.c0) = pack8<T>(x0);
    if (it.c1 >= 0) *reinterpret_cast<uint4*>(dst + it.c1) = pack8<T>(x1);
  }
  sm100::cp_async_wait<0>();
}

Side side_of(const HeadRows& in, const HeadRows& out, const float* weight) {
  return Side{static_cast<const uint16_t*>(in.data), static_cast<uint16_t*>(out.data), weight,
              in.token_stride, in.head_stride, out.token_stride, out.head_stride};
}

}  // namespace

csa2_status launch_head_norm(csa2_dtype dtype, const HeadRows& q, const float* q_weight,
                             const HeadRows& q_out, const HeadRows& k, const float* k_weight,
                             const HeadRows& k_out, int64_t T, int D, float eps,
                             const int32_t* positions, const RopeArgs& rope, cudaStream_t stream) {
  Params p = {};
  p.q = side_of(q, q_out, q_weight);
  p.k = side_of(k, k_out, k_weight);
  p.positions = positions;
  p.T = T;
  p.Hq = q.heads;
  p.H = q.heads + k.heads;
  p.D = D;
  p.eps = eps;
  p.inv_d = static_cast<float>(1.0 / D);
  p.rope = rope;
  p.items = items_of(D, rope.half);
  p.lanes = 1;
  while (p.lanes < p.items) p.lanes *= 2;
  const int per_pass = kThreads / p.lanes;
  p.step_t = per_pass / p.H;
  p.step_h = per_pass % p.H;
  const int sms = sm_count();
  // as many tokens per CTA as still leave four CTAs per SM (or as fill its
  // threads once); with fewer tokens than that, a token's heads are cut over grid.y
  p.tokens = kMaxTokens;
  while (p.tokens > 1 && p.tokens * p.H > per_pass && T / p.tokens < 4 * sms) p.tokens /= 2;
  const int64_t gx = (T + p.tokens - 1) / p.tokens;
  const int passes = (p.tokens * p.H + per_pass - 1) / per_pass;
  int ny = 1;
  if (gx < 2 * sms) ny = static_cast<int>(std::min<int64_t>(passes, (2 * sms + gx - 1) / gx));
  p.rows_cta = (passes + ny - 1) / ny * per_pass;
  ny = (p.tokens * p.H + p.rows_cta - 1) / p.rows_cta;
  if (gx > 0x7fffffffLL) return fail(CSA2_ERR_UNSUPPORTED, "csa2_qk_norm_rope: too many tokens");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(ny));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.tokens) * rope.half * sizeof(float2) + kStages * 2 * kThreads * 16;
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attribute()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  begin_launch(stream);
  int64_t reach = 0;                                   // the largest offset among a CTA's rows
  for (const HeadRows* r : {&q, &q_out, &k, &k_out})
    if (r->heads > 0)
      reach = std::max(reach, p.tokens > 0x7fffffff / (r->token_stride + 1) || r->heads > 0x7fffffff / (r->head_stride + 1)
                                  ? int64_t{1} << 32
                                  : p.tokens * r->token_stride + r->heads * r->head_stride);
  const bool narrow = reach <= 0x7fffffff;
  const cudaError_t e =
      dtype == CSA2_F16
          ? (narrow ? cudaLaunchKernelEx(&cfg, head_norm_kernel<__half, int32_t>, p)
                    : cudaLaunchKernelEx(&cfg, head_norm_kernel<__half, int64_t>, p))
          : (narrow ? cudaLaunchKernelEx(&cfg, head_norm_kernel<__nv_bfloat16, int32_t>, p)
                    : cudaLaunchKernelEx(&cfg, head_norm_kernel<__nv_bfloat16, int64_t>, p));
  note_launch(LK_OTHER, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "csa2_qk_norm_rope: launch failed: %s", cudaGetErrorString(e));
  }
  return check_launch("csa2_qk_norm_rope");
}

}  // namespace csa2
