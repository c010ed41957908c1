// Attention over a paged cache on the warp-level matrix instructions: 16 query
// rows (tokens x heads that share a cache head) against tiles of keys.
//
// Each CTA (4 warps) holds 16 rows of q in shared memory and runs over its keys
// in tiles of KT tokens, two tiles in flight: cp.async (16-bit rows) or loads
// and exact dequantisation (FP4) into padded rows.  Per tile every warp scores
// KT / 4 of the tile's keys, the row maxima meet in shared memory, the weights
// go to shared memory in the 16-bit type, and every warp adds D / 4 of the
// output channels.  One pass with the running maximum and sum.
//
// A decode query's tokens are cut into chunks on several CTAs; chunks > 1 write
// (O, m, l) partials that paged_combine_kernel joins in chunk order.
//
// Takes what the kernels of paged_decode.cu, paged_wide.cu and paged_window.cu do not:
// prompts over rows of 256 and 512 channels (FP4, few heads, short windows, pages below 8
// tokens), and single tokens over 16-bit rows of 512 in pages below 8 tokens.
// Latency-bound, as two block barriers per tile stand between the products.  Measured
// (512 tokens behind 1000, 64 heads over one 512-wide row): 237 us, against 113 on
// the tensor cores in paged_wide.cu.
#include <algorithm>

#include "launchers.h"
#include "paged_attn.cuh"

namespace csa2 {
namespace {
using namespace paged;
using rope::Num;

constexpr int kThreads = 128;

struct Params {
  const uint16_t* q;
  int64_t q_token, q_head;
  uint16_t* out;
  float* lse;
  const int32_t* cu_q;               // null: decode (row b is sequence b's token)
  int64_t T;
  float* part_o;                     // [B * Hq][chunks][D]
  float2* part_ml;                   // [B * Hq][chunks]
  float scale2;                      // scale * log2(e)
  int Hq, G, row_tiles, window, sinks, chunk, chunks;
  int aligned;                       // chunks of aligned tiles (paged_wide.cu)
  PagedView kv;
};

template <int D>
constexpr int tile_keys() { return D == 256 ? 64 : 32; }
// whether single tokens come here
template <int D, bool FP4>
constexpr bool decodes() { return D == 512 && !FP4; }

template <int D>
struct Lay {
  static constexpr int KT = tile_keys<D>();
  static constexpr int ROW = 2 * D + 16;               // bytes of a padded row (ldmatrix without conflicts)
  static constexpr int PROW = 2 * KT + 16;
  static constexpr int Q = 0;
  static constexpr int K = Q + 16 * ROW;
  static constexpr int STAGE = KT * ROW;
  static constexpr int bytes(bool shared) { return K + 2 * STAGE * (shared ? 1 : 2) + 16 * PROW + 4 * 16 * 4 + 2 * KT * 8; }
};

template <class T, int D, bool FP4>
__global__ void __launch_bounds__(kThreads) paged_attn_kernel(const Params p) {
  using L = Lay<D>;
  constexpr int KT = L::KT, NK = KT / 4;               // keys per tile, and per warp in the scores
  constexpr int NC = D / 4;                            // channels per warp in the output
  // f16 weights stand 2^15 above the largest's 1 (see paged_decode.cu)
  constexpr float LIFT = std::is_same<T, __half>::value ? 15.0f : 0.0f;
  extern __shared__ __align__(16) uint8_t smem[];
  const bool shared_kv = p.kv.v == p.kv.k;
  uint8_t* sK = smem + L::K;
  uint8_t* sV = shared_kv ? sK : sK + 2 * L::STAGE;
  uint8_t* sP = sV + 2 * L::STAGE;
  float* sRed = reinterpret_cast<float*>(sP + 16 * L::PROW);
  int64_t* sRow = reinterpret_cast<int64_t*>(sRed + 64);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_wait();
  // which rows
  int b, n_b, kvh, chunk = 0;
  int64_t r0, q_row0;
  const bool decode = decodes<D, FP4>() && p.cu_q == nullptr;
  if (decode) {
    b = blockIdx.z;
    n_b = 1;
    kvh = blockIdx.y / p.row_tiles;
    r0 = 16 * (blockIdx.y % p.row_tiles);
    q_row0 = b;
    chunk = blockIdx.x;
  } else {
    kvh = blockIdx.y;
    int64_t tile = blockIdx.x;
    bool found = false;
    b = 0;
    n_b = 0;
    q_row0 = 0;
    r0 = 0;
    for (int s = 0; s < p.kv.B; ++s) {
      const int c0 = __ldg(p.cu_q + s), c1 = __ldg(p.cu_q + s + 1);
      if (c0 < 0 || c1 < c0 || c1 > p.T) {
        if (tid == 0) raise_dev_error(p.kv.err, DEVERR_BOUNDS);
        continue;
      }
      const int64_t tiles = (static_cast<int64_t>(c1 - c0) * p.G + 15) / 16;
      if (tile < tiles) {
        b = s;
        n_b = c1 - c0;
        q_row0 = c0;
        r0 = tile * 16;
        found = true;
        break;
      }
      tile -= tiles;
    }
    if (!found) return;
  }
  const int64_t rows = min(static_cast<int64_t>(16), static_cast<int64_t>(n_b) * p.G - r0);
  const int len = length_of(p.kv, b, tid == 0);
  const int base = len - n_b;                          // position of the first new token
  const int t_first = static_cast<int>(r0 / p.G), t_last = static_cast<int>((r0 + rows - 1) / p.G);
  const Seen seen(base + t_first, base + t_last, p.window, p.sinks);

  // tiles: a decode chunk runs over slots; a prompt over token tiles aligned to
  // KT, so that a row meets its keys in the same tiles wherever a chunk began
  int v0 = 0, v1 = seen.total, tiles, sink_tiles = 0, first_tile = 0;
  if (decode) {
    const int64_t c0 = static_cast<int64_t>(chunk) * p.chunk;
    if (chunk > 0 && c0 >= seen.total) return;
    v0 = static_cast<int>(c0);
    // the last chunk takes what is left of a sequence longer than the bound
    if (chunk + 1 < p.chunks) v1 = min(seen.total, v0 + p.chunk);
    tiles = (v1 - v0 + KT - 1) / KT;
  } else {
    sink_tiles = (seen.ns + KT - 1) / KT;
    first_tile = max(seen.lo / KT, sink_tiles);
    tiles = seen.total == 0 ? 0 : sink_tiles + max(0, (base + t_last) / KT + 1 - first_tile);
  }
  const int pmax = base + t_last;
  auto token_at = [&](int tile, int r) -> int {        // -1: nothing there
    if (decode) {
      const int s = v0 + tile * KT + r;
      return s < v1 ? seen.token(s) : -1;
    }
    const int j = (tile < sink_tiles ? tile : tile - sink_tiles + first_tile) * KT + r;
    return j <= pmax && (j >= seen.lo || j < seen.ns) ? j : -1;
  };

  // q rows (zero past the last)
  for (int i = tid; i < 16 * (D / 8); i += kThreads) {
    const int r = i / (D / 8), c = i % (D / 8);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      const int64_t rr = r0 + r, t = rr / p.G;
      v = __ldg(reinterpret_cast<const uint4*>(p.q + (q_row0 + t) * p.q_token +
                                               (kvh * p.G + (rr - t * p.G)) * p.q_head) + c);
    }
    *reinterpret_cast<uint4*>(smem + r * L::ROW + c * 16) = v;
  }
  // a tile's row offsets (one tile ahead of its loads)
  auto fill_rows = [&](int tile) {
    if (tid < KT) {
      const int j = tile < tiles ? token_at(tile, tid) : -1;
      const int64_t row = j >= 0 ? token_row(p.kv, b, j) : -1;
      sRow[(tile & 1) * KT + tid] = row < 0 ? -1 : row + kvh * p.kv.head_stride;
    }
  };
  auto load = [&](int tile) {
    const int64_t* rowp = sRow + (tile & 1) * KT;
    for (int s = 0; s < (shared_kv ? 1 : 2); ++s) {
      uint8_t* dst = (s ? sV : sK) + (tile & 1) * L::STAGE;
      const uint8_t* src = s ? p.kv.v : p.kv.k;
      if (!FP4) {
        for (int i = tid; i < KT * (D / 8); i += kThreads) {
          const int r = i / (D / 8), c = i % (D / 8);
          const int64_t row = rowp[r];
          sm100::cp_async_16(dst + r * L::ROW + c * 16, src + (row < 0 ? 0 : row * 2 + c * 16), row < 0 ? 0u : 16u);
        }
      } else {
        const uint8_t* sc = s ? p.kv.v_scales : p.kv.k_scales;
        for (int i = tid; i < KT * (D / 32); i += kThreads) {
          const int r = i / (D / 32), c = i % (D / 32);
          const int64_t row = rowp[r];
          uint4 w = make_uint4(0, 0, 0, 0);
          uint32_t s2 = 0;
          if (row >= 0) {
            w = __ldg(reinterpret_cast<const uint4*>(src + row / 2) + c);
            s2 = __ldg(reinterpret_cast<const uint16_t*>(sc + row / 16) + c);
          }
          const uint32_t lo = scale_pair(s2 & 255u), hi = scale_pair(s2 >> 8);
          uint4* o = reinterpret_cast<uint4*>(dst + r * L::ROW + c * 64);
          o[0] = dequant8(w.x, lo);
          o[1] = dequant8(w.y, lo);
          o[2] = dequant8(w.z, hi);
          o[3] = dequant8(w.w, hi);
        }
      }
    }
    sm100::cp_async_commit();
  };

  float o[NC / 8][4];
#pragma unroll
  for (int i = 0; i < NC / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  // this thread's rows of a fragment: lane / 4 and lane / 4 + 8
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  int pos[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = (lane >> 2) + 8 * u;
    pos[u] = r < rows ? base + static_cast<int>((r0 + r) / p.G) : -1;
  }
  const uint32_t q_sm = sm100::smem_u32(smem), p_sm = sm100::smem_u32(sP);

  fill_rows(0);
  __syncthreads();
  if (tiles > 0) load(0);
  for (int t = 0; t < tiles; ++t) {
    fill_rows(t + 1);
    sm100::cp_async_wait<0>();
    __syncthreads();                                   // tile t, and the next tile's rows, are in place
    if (t + 1 < tiles) load(t + 1);
    const uint32_t k_sm = sm100::smem_u32(sK + (t & 1) * L::STAGE), v_sm = sm100::smem_u32(sV + (t & 1) * L::STAGE);
    const int64_t* rowp = sRow + (t & 1) * KT;
    // scores of this warp's keys
    float s[NK / 8][4];
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll 4
    for (int kk = 0; kk < D / 16; kk += 2) {           // 32 channels
      uint32_t a0[4], a1[4];
      ldsm4(a0, q_sm + (lane & 15) * L::ROW + kk * 32 + (lane >> 4) * 16);
      ldsm4(a1, q_sm + (lane & 15) * L::ROW + kk * 32 + 32 + (lane >> 4) * 16);
#pragma unroll
      for (int i = 0; i < NK / 8; ++i) {               // 8 keys x 32 channels
        uint32_t bb[4];
        ldsm4(bb, k_sm + (warp * NK + i * 8 + (lane & 7)) * L::ROW + kk * 32 + (lane >> 3) * 16);
        mma16816<T>(s[i], a0, bb[0], bb[1]);
        mma16816<T>(s[i], a1, bb[2], bb[3]);
      }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < NK / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = warp * NK + i * 8 + (lane & 3) * 2 + (e & 1);
        const int j = token_at(t, r), u = e >> 1;
        const bool ok = j >= 0 && rowp[r] >= 0 && sees(pos[u], j, p.window, p.sinks);
        s[i][e] = ok ? s[i][e] * p.scale2 : -INFINITY;
        mx[u] = fmaxf(mx[u], s[i][e]);
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
      mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
      if ((lane & 3) == 0) sRed[warp * 16 + (lane >> 2) + 8 * u] = mx[u];
    }
    __syncthreads();
    float alpha[2], ref[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = (lane >> 2) + 8 * u;
      const float mn = fmaxf(m[u], fmaxf(fmaxf(sRed[r], sRed[16 + r]), fmaxf(sRed[32 + r], sRed[48 + r])));
      ref[u] = mn == -INFINITY ? 0.0f : lifted(mn, LIFT);          // nothing seen yet: every weight is 0
      alpha[u] = exp2_approx(lifted(m[u], LIFT) - ref[u]);
      m[u] = mn;
      l[u] *= alpha[u];
    }
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float e0 = exp2_approx(s[i][2 * u] - ref[u]), e1 = exp2_approx(s[i][2 * u + 1] - ref[u]);
        l[u] += e0 + e1;
        *reinterpret_cast<uint32_t*>(sP + ((lane >> 2) + 8 * u) * L::PROW + (warp * NK + i * 8 + (lane & 3) * 2) * 2) =
            Num<T>::down(e0, e1);
      }
    }
#pragma unroll
    for (int i = 0; i < NC / 8; ++i) {
      o[i][0] *= alpha[0];
      o[i][1] *= alpha[0];
      o[i][2] *= alpha[1];
      o[i][3] *= alpha[1];
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < KT / 16; ++kk) {
      uint32_t a[4];
      ldsm4(a, p_sm + (lane & 15) * L::PROW + kk * 32 + (lane >> 4) * 16);
#pragma unroll
      for (int i = 0; i < NC / 16; ++i) {              // 16 keys x 16 channels
        uint32_t bb[4];
        ldsm4t(bb, v_sm + (kk * 16 + (lane & 15)) * L::ROW + (warp * NC + i * 16 + (lane >> 4) * 8) * 2);
        mma16816<T>(o[2 * i], a, bb[0], bb[1]);
        mma16816<T>(o[2 * i + 1], a, bb[2], bb[3]);
      }
    }
  }
  // row sums: over the quad, then over the warps
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
    l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
    if ((lane & 3) == 0) sRed[warp * 16 + (lane >> 2) + 8 * u] = l[u];
  }
  __syncthreads();
  const bool partial = decode && p.chunks > 1 && seen.total > p.chunk;
  __shared__ uint8_t bad[16];                          // prompt rows to look at again
  if (tid < 16) bad[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = (lane >> 2) + 8 * u;
    if (r >= rows) continue;
    const float lr = (sRed[r] + sRed[16 + r]) + (sRed[32 + r] + sRed[48 + r]);
    const int64_t rr = r0 + r, t = rr / p.G;
    const int64_t at = (q_row0 + t) * p.Hq + kvh * p.G + (rr - t * p.G);
    if (partial) {
      float* po = p.part_o + (at * p.chunks + chunk) * D;
#pragma unroll
      for (int i = 0; i < NC / 8; ++i)
        *reinterpret_cast<float2*>(po + warp * NC + i * 8 + (lane & 3) * 2) = make_float2(o[i][2 * u], o[i][2 * u + 1]);
      if (warp == 0 && (lane & 3) == 0) p.part_ml[at * p.chunks + chunk] = make_float2(lifted(m[u], LIFT), lr);
    } else {
      const float inv = lr > 0.0f ? 1.0f / lr : (lr == 0.0f ? 0.0f : lr);
      uint16_t* po = p.out + at * D;
      if (!FP4 && !decode && (__float_as_uint(lr) & 0x7f800000u) != 0x7f800000u) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < NC / 8; ++i)
          odd |= (__float_as_uint(o[i][2 * u]) & 0x7f800000u) == 0x7f800000u ||
                 (__float_as_uint(o[i][2 * u + 1]) & 0x7f800000u) == 0x7f800000u;
        if (odd) bad[r] = 1;
      }
#pragma unroll
      for (int i = 0; i < NC / 8; ++i)
        *reinterpret_cast<uint32_t*>(po + warp * NC + i * 8 + (lane & 3) * 2) =
            Num<T>::down(o[i][2 * u] * inv, o[i][2 * u + 1] * inv);
      if (p.lse && warp == 0 && (lane & 3) == 0)
        p.lse[at] = lr == 0.0f ? -INFINITY : (lifted(m[u], LIFT) + log2f(lr)) * kLn2;
    }
  }
  if (!FP4 && !decode) {
    if (__syncthreads_or(tid < rows && bad[tid])) {
      const MendRows m = {p.q + q_row0 * p.q_token, p.q_token, p.q_head, p.out + q_row0 * p.Hq * D, p.scale2, p.Hq, p.G, kvh,
                          static_cast<int>(r0), base, p.window, p.sinks, seen.lo, seen.ns, pmax, b};
      mend_rows<T, D>(m, p.kv, bad, static_cast<int>(rows), reinterpret_cast<uint32_t*>(sK), 2 * L::STAGE * 8);
    }
  }
}

// Joins a decode row's chunks in order: M = max m_i, out = sum 2^(m_i - M) O_i /
// sum 2^(m_i - M) l_i.  One CTA per row; D / 4 threads take four channels each,
// the groups take chunks in turn and meet in shared memory in a fixed order.
template <class T, int D>
__global__ void __launch_bounds__(128) paged_combine_kernel(const Params p) {
  constexpr int PER = D / 4, GROUPS = 128 / PER;
  __shared__ float red[4];
  __shared__ float4 acc_s[GROUPS][PER];
  __shared__ float l_s[GROUPS];
  const int64_t at = blockIdx.x;
  const int b = static_cast<int>(at / p.Hq);
  pdl_wait();
  const int len = length_of(p.kv, b, false);
  int total, per = p.chunk;                            // tokens (or aligned tiles) in all, per chunk
  if (p.aligned) {
    total = AlignedTiles(len - 1, p.window, p.sinks).tiles;
    per /= 128;
  } else {
    total = Seen(len - 1, len - 1, p.window, p.sinks).total;
  }
  if (total <= per) return;                            // written by the only chunk
  const int n = min(p.chunks, (total - 1) / per + 1);
  const float2* ml = p.part_ml + at * p.chunks;
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < n; i += 128) mx = fmaxf(mx, ml[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float ref = mx == -INFINITY ? 0.0f : mx;
  const int g = threadIdx.x / PER, c = threadIdx.x % PER;
  float4 acc = make_float4(0, 0, 0, 0);
  float l = 0.0f;
  const float4* po = reinterpret_cast<const float4*>(p.part_o + at * p.chunks * D) + c;
#pragma unroll 4
  for (int i = g; i < n; i += GROUPS) {
    const float2 x = ml[i];
    const float w = exp2_approx(x.x - ref);
    const float4 v = po[static_cast<int64_t>(i) * PER];
    l += w * x.y;
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
  }
  acc_s[g][c] = acc;
  if (c == 0) l_s[g] = l;
  __syncthreads();
  if (g == 0) {
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      const float4 v = acc_s[i][c];
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
      l += l_s[i];
    }
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
    *reinterpret_cast<uint2*>(p.out + at * D + 4 * c) =
        make_uint2(Num<T>::down(acc.x * inv, acc.y * inv), Num<T>::down(acc.z * inv, acc.w * inv));
    if (p.lse && c == 0) p.lse[at] = l == 0.0f ? -INFINITY : (mx + log2f(l)) * kLn2;
  }
}

Params params_of(const PagedAttn& a) {
  Params p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_token = a.q_token;
  p.q_head = a.q_head;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.scale2 = a.scale * kLog2e;
  p.Hq = a.Hq;
  p.G = a.G;
  p.window = a.window;
  p.sinks = a.sinks;
  p.kv = a.kv;
  p.chunks = 1;
  return p;
}

template <class T, int D>
csa2_status combine(const Params& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.kv.B * static_cast<int64_t>(p.Hq)));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attribute()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  begin_launch(stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_combine_kernel<T, D>, p);
  note_launch(LK_COMBINE, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "paged attention: launch failed: %s", cudaGetErrorString(e));
  }
  return check_launch("paged attention: combine");
}

csa2_status dispatch_combine(const PagedAttn& a, const Params& p, cudaStream_t stream) {
#define CSA2_COMBINE(D_) \
  if (a.D == D_) return a.fmt == CSA2_KV_F16 ? combine<__half, D_>(p, stream) : combine<__nv_bfloat16, D_>(p, stream);
  CSA2_COMBINE(64) CSA2_COMBINE(128) CSA2_COMBINE(256) CSA2_COMBINE(512)
#undef CSA2_COMBINE
  return CSA2_ERR_UNSUPPORTED;
}

template <class T, int D, bool FP4>
csa2_status run(const Params& p, dim3 grid, cudaStream_t stream) {
  using L = Lay<D>;
  static PerDevice<int> opted;
  opted.get(+[]() -> int {
    cudaFuncSetAttribute(paged_attn_kernel<T, D, FP4>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes(false));
    return 1;
  });
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::bytes(p.kv.v == p.kv.k);
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attribute()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  begin_launch(stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_attn_kernel<T, D, FP4>, p);
  note_launch(LK_ATTN, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "paged attention: launch failed: %s", cudaGetErrorString(e));
  }
  return check_launch("paged attention");
}

csa2_status dispatch(const PagedAttn& a, const Params& p, dim3 grid, cudaStream_t stream) {
#define CSA2_PAGED(D_)                                                                            \
  if (a.D == D_)                                                                                  \
    return a.fmt == CSA2_KV_FP4   ? run<__nv_bfloat16, D_, true>(p, grid, stream)        \
           : a.fmt == CSA2_KV_F16 ? run<__half, D_, false>(p, grid, stream)              \
                                  : run<__nv_bfloat16, D_, false>(p, grid, stream);
  CSA2_PAGED(256) CSA2_PAGED(512)
#undef CSA2_PAGED
  return CSA2_ERR_UNSUPPORTED;
}

// Tokens a decode query may see, as a bound.
int64_t seen_bound(const PagedAttn& a, int64_t max_len) {
  const int64_t n = std::min<int64_t>(max_len, a.kv.capacity);
  return a.window > 0 ? std::min<int64_t>(n, static_cast<int64_t>(a.window) + a.sinks) : n;
}

struct Split {
  int chunk, chunks;
};
// The chunk length of a decode launch.
//  - wide rows on the tensor cores: one CTA per SM, so the number of chunks that
//    wastes least, counting a chunk's start and partial output as 4 tiles
//  - else see below
Split split_of(const PagedAttn& a, int64_t max_len, int chunk) {
  const int64_t seen = std::max<int64_t>(1, seen_bound(a, max_len));
  Split s;
  if (paged_wide_applies(a)) {
    const int nh = paged_wide_heads(a);
    const int64_t units = std::max<int64_t>(1, static_cast<int64_t>(a.kv.B) * a.kv.heads * ((a.G + nh - 1) / nh));
    const int64_t tiles = (seen + 127) / 128 + (a.window > 0 ? 2 : 0);
    int64_t per = std::min<int64_t>((static_cast<int64_t>(chunk) + 127) / 128, tiles);
    if (chunk == 0) {
      int64_t best = 0;
      const int sms = sm_count();
      for (int64_t n = 1; n <= std::min<int64_t>(tiles, 4 * sms); ++n) {
        const int64_t len = (tiles + n - 1) / n;
        const int64_t cost = (units * ((tiles + len - 1) / len) + sms - 1) / sms * (len + 4);
        if (best == 0 || cost < best) {
          best = cost;
          per = len;
        }
        if (n * units > 16 * sms) break;
      }
    }
    s.chunk = static_cast<int>(per * 128);
    s.chunks = static_cast<int>((tiles + per - 1) / per);
    return s;
  }
  const int nh = paged_decode_heads(a);
  const int64_t units = static_cast<int64_t>(a.kv.B) * a.kv.heads * ((a.G + nh - 1) / nh);
  int64_t c = chunk;
  if (c == 0) {
    // two CTAs per SM, but no chunk above 2048 tokens, so that long and short
    // sequences side by side even out, and at most 64 chunks to join unless they
    // hold 256 tokens.  Measured (us at chunks of 256 / 1024 / 2048 / 8192): 64
    // ragged sequences up to 16K, 8 cache heads 338 / 243 / 236 / 285; one of 32K, 8
    // heads 46 / 31 / 34 / 108; 64 of 2K, 4 heads 66 / 53 / 49 / 49; one of 8K, one
    // head 9.6 / 17 / 27 / 90 (128: 9.3, 64: 10.3).  FP4 rows under up to 8 heads have
    // four CTAs per SM and half the work per token: 1024 / 2048, 64 ragged of up to 32K
    // behind a window of 8192, 4 heads 73.6 / 79.8; of 8K, 4 heads x 64 32.9 / 37.1; 64
    // of 2K, 4 heads 33.0 / 31.9
    const int64_t n = std::max<int64_t>(1, 2LL * sm_count() / std::max<int64_t>(1, units));
    c = std::max<int64_t>((seen + n - 1) / n, std::min<int64_t>(256, (seen + 63) / 64));
    c = std::min<int64_t>(a.fmt == CSA2_KV_FP4 && a.G <= 8 ? 1024 : 2048, std::max<int64_t>(64, (c + 63) / 64 * 64));
  }
  s.chunk = static_cast<int>(std::min<int64_t>(c, 0x7fffffc0));
  s.chunks = static_cast<int>((seen + s.chunk - 1) / s.chunk);
  return s;
}

}  // namespace

size_t paged_decode_workspace(const PagedAttn& a, int64_t max_len, int chunk) {
  const Split s = split_of(a, max_len, chunk);
  if (s.chunks <= 1) return 0;
  const size_t n = static_cast<size_t>(a.kv.B) * a.Hq * s.chunks;
  return n * a.D * sizeof(float) + n * sizeof(float2);
}

csa2_status launch_paged_decode(const PagedAttn& a, int64_t max_len, int chunk, void* ws, cudaStream_t stream) {
  const Split s = split_of(a, max_len, chunk);
  Params p = params_of(a);
  p.chunk = s.chunk;
  p.chunks = s.chunks;
  p.row_tiles = (a.G + 15) / 16;
  if (s.chunks > 1) {
    p.part_o = static_cast<float*>(ws);
    p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(a.kv.B) * a.Hq * s.chunks * a.D);
  }
  if (paged_wide_applies(a)) {
    p.aligned = 1;
    CSA2_TRY(launch_paged_wide(a, s.chunk, s.chunks, p.part_o, p.part_ml, stream));
  } else if (paged_decode_stream_applies(a)) {
    CSA2_TRY(launch_paged_decode_stream(a, s.chunk, s.chunks, p.part_o, p.part_ml, stream));
  } else {
    const dim3 grid(static_cast<unsigned>(s.chunks), static_cast<unsigned>(a.kv.heads * p.row_tiles),
                    static_cast<unsigned>(a.kv.B));
    CSA2_TRY(dispatch(a, p, grid, stream));
  }
  return s.chunks > 1 ? dispatch_combine(a, p, stream) : CSA2_OK;
}

csa2_status launch_paged_window(const PagedAttn& a, const int32_t* cu_q, int64_t T, cudaStream_t stream) {
  if (paged_window_tc_applies(a)) return launch_paged_window_tc(a, cu_q, T, stream);
  if (paged_wide_prompt_applies(a)) return launch_paged_wide_prompt(a, cu_q, T, stream);
  Params p = params_of(a);
  p.cu_q = cu_q;
  p.T = T;
  p.row_tiles = 1;
  p.chunk = 0x7fffffff;
  // tiles of 16 (token, head) rows: at most one more per sequence than all rows need
  const int64_t tiles = (T * a.G + 15) / 16 + a.kv.B;
  if (tiles > 0x7fffffffLL) return fail(CSA2_ERR_UNSUPPORTED, "csa2_paged_window_attn: too many rows");
  return dispatch(a, p, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(a.kv.heads)), stream);
}

}  // namespace csa2
