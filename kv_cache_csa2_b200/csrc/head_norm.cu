// RMS norm and position rotation of query and key heads in one pass:
//   y = x * rsqrt(mean(x^2) + eps) * weight, then the rotated pairs turn by
//   positions[t] * inv_freq.
// HBM-bound (each channel is read and written once, two bytes each way).  A CTA
// takes a block of tokens: it requests its first rows, computes the tokens'
// angles once for all heads into shared memory, and then runs over the
// (token, head) rows; a group of lanes holds a row, the norm is a shuffle sum.
// Measured: 8192 tokens of 64 + 8 heads x 128, 57.5 us (5.25 TB/s); 4096 of 64 + 1 heads
// x 512, 107.5 us (5.08 TB/s).  What bounds it then is instruction issue (77 % of the
// slots: every product and sum of the rotation rounds by itself) and four CTAs of
// 64 registers per SM; weights held in registers cost a CTA and were slower.
#include <algorithm>

#include "common.cuh"
#include "launchers.h"
#include "paged.h"
#include "rope.cuh"

namespace csa2 {
namespace {
using namespace rope;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;

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
  float eps;
  RopeArgs rope;
};

__device__ __forceinline__ void scale8(float2 (&x)[4], float inv, const float* w) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w)), b = __ldg(reinterpret_cast<const float4*>(w) + 1);
  const float2 i2 = make_float2(inv, inv);
  x[0] = mul2(mul2(x[0], i2), make_float2(a.x, a.y));
  x[1] = mul2(mul2(x[1], i2), make_float2(a.z, a.w));
  x[2] = mul2(mul2(x[2], i2), make_float2(b.x, b.y));
  x[3] = mul2(mul2(x[3], i2), make_float2(b.z, b.w));
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4) head_norm_kernel(const Params p) {
  extern __shared__ float4 cs[];                                   // [tokens][half / 2]
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.tokens;
  const int nt = static_cast<int>(min(static_cast<int64_t>(p.tokens), p.T - t0));
  const int per_pass = kThreads / p.lanes;
  const int sub = threadIdx.x & (p.lanes - 1);
  const int r_end = min(nt * p.H, static_cast<int>(blockIdx.y + 1) * p.rows_cta);
  int r = blockIdx.y * p.rows_cta + threadIdx.x / p.lanes;
  Item it = item_at(sub, p.D, p.rope.half, p.rope.offset);
  if (sub >= p.items) it.c0 = it.c1 = it.freq = -1;

  uint4 v0, v1;
  int tl = r / p.H, head = r - tl * p.H;
  auto request = [&](int row) {
    v0 = v1 = make_uint4(0, 0, 0, 0);
    if (row >= r_end) return;
    const uint16_t* src = head < p.Hq ? p.q.in + (t0 + tl) * p.q.in_t + head * p.q.in_h
                                      : p.k.in + (t0 + tl) * p.k.in_t + (head - p.Hq) * p.k.in_h;
    if (it.c0 >= 0) v0 = *reinterpret_cast<const uint4*>(src + it.c0);
    if (it.c1 >= 0) v1 = *reinterpret_cast<const uint4*>(src + it.c1);
  };
  pdl_wait();
  request(r);
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
    float2 x0[4], x1[4];
    unpack8<T>(v0, x0);
    unpack8<T>(v1, x1);
    const bool live = r < r_end, is_q = head < p.Hq;
    const int my_t = tl, my_h = head;
    const float* w = is_q ? p.q.weight : p.k.weight;
    float sum = 0.0f;
#pragma unroll
    for (int u = 0; u < 4; ++u) sum += (x0[u].x * x0[u].x + x0[u].y * x0[u].y) + (x1[u].x * x1[u].x + x1[u].y * x1[u].y);
    for (int o = p.lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // a row is read whole by its lanes before any of them stores (the shuffle
    // above), so an output may be its input
    tl += p.step_t;                                    // the row a pass further
    head += p.step_h;
    if (head >= p.H) head -= p.H, ++tl;
    request(r + per_pass);
    if (!live) continue;
    if (w) {
      const float inv = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
      if (it.c0 >= 0) scale8(x0, inv, w + it.c0);
      if (it.c1 >= 0) scale8(x1, inv, w + it.c1);
    }
    if (p.rope.inv_freq) rotate_item(x0, x1, it, p.rope.half, p.rope.interleaved, cs + my_t * (p.rope.half / 2));
    uint16_t* dst = is_q ? p.q.out + (t0 + my_t) * p.q.out_t + my_h * p.q.out_h
                         : p.k.out + (t0 + my_t) * p.k.out_t + (my_h - p.Hq) * p.k.out_h;
    if (it.c0 >= 0) *reinterpret_cast<uint4*>(dst + it.c0) = pack8<T>(x0);
    if (it.c1 >= 0) *reinterpret_cast<uint4*>(dst + it.c1) = pack8<T>(x1);
  }
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
  cfg.dynamicSmemBytes = static_cast<size_t>(p.tokens) * rope.half * sizeof(float2);
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attribute()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  begin_launch(stream);
  const cudaError_t e = dtype == CSA2_F16 ? cudaLaunchKernelEx(&cfg, head_norm_kernel<__half>, p)
                                          : cudaLaunchKernelEx(&cfg, head_norm_kernel<__nv_bfloat16>, p);
  note_launch(LK_OTHER, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "csa2_qk_norm_rope: launch failed: %s", cudaGetErrorString(e));
  }
  return check_launch("csa2_qk_norm_rope");
}

}  // namespace csa2
