// Attention of a prompt chunk over a paged cache on the 5th-generation tensor
// cores, rows of 64 or 128 channels: causal, with a sliding window and sinks.
//
// The query rows of a cache head are (token, head) pairs, head fastest, so that
// the heads that share keys fill a tile together.  A CTA takes two tiles of 128
// rows against tiles of 128 keys (one pass, running maximum and sum):
//   warps 0-3, 4-7  softmax of row tile 0 / 1: one thread per row reads its
//                   scores from TMEM, writes the weights back there as 16-bit
//                   pairs (the next product's left operand), and at the end
//                   divides and stores the output
//   warps 8, 9      issue row tile 0's / 1's S = Q K^T (M=128, N=64, K=D) and
//                   O += P V (M=128, N=D, K=64), half a key tile at a time
//   warps 10-15     bring the key (even warps) and value rows into the 128-byte
//                   swizzled layout.  16-bit rows in pages of at least 8 tokens: one
//                   warp each, a TMA box per lane; value rows of unwanted tokens are
//                   zeroed before the tile is announced (what lies past a sequence's
//                   end may be anything, and a weight of 0 does not silence a NaN).
//                   Smaller pages go row by row by cp.async, FP4 rows are dequantised
//                   on the way, by three warps each.
// The output stays in TMEM; it is rescaled only when a row's maximum has grown
// by more than 2^8 since its last reference (its weights then exceed 1 by at
// most that, which neither type nor the f32 sums mind).
//
// A row tile's scores have two buffers of 64 columns, one per half of a key tile:
// the tensor cores fill one while the softmax works on the other, whose weights
// take the place of its scores.  (With one buffer of 128 columns the softmax stood
// still for both products of every tile: 3950 clocks per key tile, of which 2200
// were softmax.)  Tiles are aligned to 128 tokens, and within a half the blocks of
// 32 tokens that no row of the row tile sees are skipped; neither touches a row's
// sums, so its bits depend on its own tokens only.
//
// Bound: 4 D flops per (row, key) on the tensor cores against one exponential,
// 16 of which an SM does per clock: at D = 128 both take 1024 clocks per pair of
// 128 x 128 tiles.  Measured: 8192 tokens, window 2048 + 4, 32 heads over 4 x 128, 267 us
// (0.77 Pflop/s; 282 us run for seconds, at the power limit's 1850 MHz); the softmax's latency
// per 64 keys (1900 clocks against 1280 of products) is what is left, and TMEM has no room
// for a third row tile.  The launch's 128 registers a thread cost 20 bytes of spill stores
// and 100 to 116 of loads (8 and 32, 12 and 72 or none with FP4 rows).
#include <algorithm>
#include <type_traits>

#include "launchers.h"
#include "paged_attn.cuh"

namespace csa2 {
namespace {
using namespace paged;
using namespace sm100;
using rope::Num;

constexpr int kThreads = 512;
constexpr int KT = 128;                                // keys per tile
constexpr int HT = 64;                                 // keys per half of a tile: one buffer of scores
constexpr int KB = 32;                                 // keys per block
constexpr int RT = 128;                                // rows per row tile
constexpr int kBits = 8;                               // slots of the presence words
constexpr float kLazy = 8.0f;                          // log2 growth of a maximum that O tolerates

template <int D, bool SHARED>
struct Lay {
  static constexpr int BLK = 128 * 128;                // 64 channels of 128 rows
  static constexpr int TILE = D / 64 * BLK;
  static constexpr int KST = SHARED ? 4 : D == 64 ? 3 : 2;
  static constexpr int VST = SHARED ? 0 : D == 64 ? 3 : 2;
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * TILE;
  static constexpr int V = K + KST * TILE;
  static constexpr int BAR = V + VST * TILE;
  static constexpr int NBAR = 2 * KST + 2 * VST + 4 + 4 + 4 + 2 + 1 + 1;
  static constexpr int BITS = BAR + NBAR * 8;
  static constexpr int MISC = BITS + kBits * 4 * 4;
  static constexpr int BAD = MISC + 16;                // rows to look at again
  static constexpr int BYTES = BAD + 2 * RT + 1024;
};

struct Params {
  const uint16_t* q;
  int64_t q_token, q_head;
  uint16_t* out;
  float* lse;
  const int32_t* cu_q;
  int64_t T;
  float scale2;                      // |scale| * log2(e), at least the smallest normal
  uint32_t flip;                     // 0x80008000 for a negative scale: q's signs turn
  int Hq, G, window, sinks;
  int box;                           // rows of a TMA box (0: none)
  int q_tokens;                      // tokens of a row tile's TMA box of q (0: rows are loaded one by one)
  PagedView kv;
};

// A row tile's q rows: channels c .. c + 63 of the G heads of some tokens.
__device__ __forceinline__ void tma_load_q(void* dst, const CUtensorMap* map, uint64_t* bar, int c, int head, int token) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c), "r"(head), "r"(token)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 2^x for a pair on the multiply-add pipe: n = the integer nearest x, f = x - n in
// [-1/2, 1/2], a degree-5 polynomial of least relative error for 2^f (7.5e-8, found
// by reweighted least squares; 2.3e-7 with f32 coefficients and steps), times 2^n.
// x below -126.5, -inf too, gives 0; NaN stays NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 exp2_pair(float2 x) {
  constexpr float kRound = 12582912.0f;                // 1.5 * 2^23: adding it rounds to an integer
  x = make_float2(max_nan(x.x, -127.0f), max_nan(x.y, -127.0f));
  const float2 t = add2(x, make_float2(kRound, kRound));
  const float2 f = fma2(add2(t, make_float2(-kRound, -kRound)), make_float2(-1.0f, -1.0f), x);
  auto c = [](float v) { return make_float2(v, v); };
  float2 y = fma2(f, c(0.001327647129073739f), c(0.009675541892647743f));
  y = fma2(y, f, c(0.05550713092088699f));
  y = fma2(y, f, c(0.24022120237350464f));
  y = fma2(y, f, c(0.6931469440460205f));
  y = fma2(y, f, c(1.0000001192092896f));
  // the low bits of t hold n; n = -127 makes the factor 0
  const float2 s = make_float2(__int_as_float((__float_as_int(t.x) << 23) + 0x3f800000),
                               __int_as_float((__float_as_int(t.y) << 23) + 0x3f800000));
  return rope::mul2(y, s);
}
// Weights of pair i of a block of 32 tokens: kPoly of every 16 pairs on the multiply-
// add pipe, the rest on the exponential unit (8192 tokens, window 2048: 286 us with
// none, 277 / 271 / 281 with 2 / 4 / 8).  Which is which depends on the token's place
// in its block alone.
constexpr int kPoly = 4;
__device__ __forceinline__ float2 weights(int i, float2 x) {
  return i % (16 / kPoly) == 16 / kPoly - 1 ? exp2_pair(x) : make_float2(exp2_approx(x.x), exp2_approx(x.y));
}

// Row tiles of a CTA: the sequence, its rows, and what they see.
struct Work {
  int b, base, n_rows;               // sequence, position of its first new token, rows of this CTA (<= 256)
  int q_row0, r0;                    // first q row of the sequence, first (token, head) row of the CTA
  int sink_tiles, first_tile, tiles; // key tiles: the sinks', then from first_tile on
  int lo, ns, pmax;                  // tokens loaded: [0, ns) and [lo, pmax]

  __device__ __forceinline__ int tile_start(int j) const {
    return (j < sink_tiles ? j : j - sink_tiles + first_tile) * KT;
  }
};

// What the rows of row tile w see together.
struct RowTile {
  int lo, ns, pmax;
  __device__ __forceinline__ RowTile(const Work& k, int w, int G, int window, int sinks) {
    const int rows = min(RT, k.n_rows - w * RT);
    lo = ns = 0;
    pmax = -1;
    if (rows > 0) {
      const int r = k.r0 + w * RT;
      pmax = k.base + (r + rows - 1) / G;
      const Seen s(k.base + r / G, pmax, window, sinks);
      lo = s.lo;
      ns = s.ns;
    }
  }
  // bit c: block c of the tile is seen by some row
  __device__ __forceinline__ uint32_t blocks(const Work& k, int tile) const {
    uint32_t m = 0;
    const int t0 = k.tile_start(tile);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int t = t0 + c * KB;
      if (t <= pmax && (t + KB > lo || t < ns)) m |= 1u << c;
    }
    return m;
  }
};

// The CTA's tile of 256 rows: tile `index` counted from the last sequence's last
// (a prompt's late tiles see most, so they start first).  Every warp scans for
// itself, 32 sequences at a time.
__device__ bool locate(const Params& p, int64_t index, Work& w) {
  const int lane = threadIdx.x & 31;
  auto tiles_of = [&](int s, int& c0, int& c1) -> int64_t {
    if (s >= p.kv.B) return 0;
    c0 = __ldg(p.cu_q + s);
    c1 = __ldg(p.cu_q + s + 1);
    if (c0 < 0 || c1 < c0 || c1 > p.T) {
      if (threadIdx.x < 32) raise_dev_error(p.kv.err, DEVERR_BOUNDS);
      return 0;
    }
    return (static_cast<int64_t>(c1 - c0) * p.G + 2 * RT - 1) / (2 * RT);
  };
  for (int s0 = (p.kv.B - 1) & ~31; s0 >= 0; s0 -= 32) {
    int c0 = 0, c1 = 0;
    const int64_t mine = tiles_of(s0 + lane, c0, c1);
    int64_t upto = mine;                               // tiles of this sequence and the later ones of the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_down_sync(0xffffffffu, upto, o);
      if (lane + o < 32) upto += x;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, index < upto && index >= upto - mine);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int64_t from_end = index - (__shfl_sync(0xffffffffu, upto, src) - __shfl_sync(0xffffffffu, mine, src));
      const int64_t tile = __shfl_sync(0xffffffffu, mine, src) - 1 - from_end;
      c0 = __shfl_sync(0xffffffffu, c0, src);
      c1 = __shfl_sync(0xffffffffu, c1, src);
      w.b = s0 + src;
      w.q_row0 = c0;
      w.r0 = static_cast<int>(tile * 2 * RT);
      w.n_rows = static_cast<int>(min(static_cast<int64_t>(2 * RT), static_cast<int64_t>(c1 - c0) * p.G - w.r0));
      w.base = length_of(p.kv, w.b, threadIdx.x == 0) - (c1 - c0);
      w.pmax = w.base + (w.r0 + w.n_rows - 1) / p.G;
      const Seen s(w.base + w.r0 / p.G, w.pmax, p.window, p.sinks);
      w.lo = s.lo;
      w.ns = s.ns;
      w.sink_tiles = (s.ns + KT - 1) / KT;
      w.first_tile = max(s.lo / KT, w.sink_tiles);
      w.tiles = s.total == 0 ? 0 : w.sink_tiles + max(0, w.pmax / KT + 1 - w.first_tile);
      return true;
    }
    index -= __shfl_sync(0xffffffffu, upto, 0);
  }
  return false;
}

template <class T, int D, bool FP4, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) paged_window_kernel(const Params p, const __grid_constant__ CUtensorMap k_map,
                                                               const __grid_constant__ CUtensorMap v_map,
                                                               const __grid_constant__ CUtensorMap q_map) {
  using L = Lay<D, SHARED>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR);
  uint64_t* k_full = bar;
  uint64_t* k_empty = k_full + L::KST;
  uint64_t* v_full = SHARED ? k_full : k_empty + L::KST;
  uint64_t* v_empty = SHARED ? k_empty : v_full + L::VST;
  uint64_t* s_full = bar + 2 * L::KST + 2 * L::VST;    // [2][2]: row tile, half
  uint64_t* p_full = s_full + 4;                       // [2][2]
  uint64_t* pv_done = p_full + 4;                      // [2][2]
  uint64_t* all_done = pv_done + 4;                    // [2]: every product of the row tile has ended
  uint64_t* q_full = all_done + 2;
  uint64_t* fix_bar = q_full + 1;                      // boxes that need rows zeroed
  constexpr int VS = SHARED ? L::KST : L::VST;
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + L::BITS);       // [kBits][4]: tokens present
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC + 4);
  uint8_t* sK = smem + L::K;
  uint8_t* sV = SHARED ? sK : smem + L::V;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kvh = blockIdx.y;
  pdl_wait();
  Work wk;
  if (!locate(p, blockIdx.x, wk)) return;              // the same answer in every warp

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::KST; ++i) {
      mbar_init(k_full + i, p.box ? 1 : 4);            // TMA: per tile; else per block
      mbar_init(k_empty + i, 2);                       // one per row tile
    }
    for (int i = 0; i < L::VST; ++i) {
      mbar_init(v_full + i, p.box ? 1 : 4);
      mbar_init(v_empty + i, 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(s_full + 2 * i + h, 1);
        mbar_init(p_full + 2 * i + h, 4);
        mbar_init(pv_done + 2 * i + h, 1);
      }
      mbar_init(all_done + i, 1);
    }
    mbar_init(q_full, p.q_tokens ? 1 : 8);
    mbar_init(fix_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t O_COL = 256;                      // S / P of tile w at 128 w, O at 256 + 128 w
  // registers: 128 x 512 threads at launch = 184 x 256 (softmax) + 72 x 256 (the
  // rest); the warps that dequantise FP4 rows need more
  if (warp >= 8) {
    if (FP4)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp > 9) {
      // ------------------------------------------------------------ loaders
      const int half = (warp - 10) & 1, group = (warp - 10) >> 1;       // keys or values; which of three
      const int ring = half ? VS : L::KST;
      const uint8_t* src = half ? p.kv.v : p.kv.k;
      uint8_t* const dst0 = half ? sV : sK;
      uint64_t *const fulls = half ? v_full : k_full, *const empties = half ? v_empty : k_empty;
      auto wait = [&](uint64_t* at, uint32_t parity) {
        return wait_phase(at, parity, abort_flag, p.kv.err);
      };
      auto wanted = [&](int j) { return j <= wk.pmax && (j >= wk.lo || j < wk.ns); };   // seen by some row
      // channel offset of a wanted token, -1 when its page is outside the pool
      auto row_of = [&](int j) -> int64_t {
        const int64_t r = token_row(p.kv, wk.b, j);
        return r < 0 ? -1 : r + kvh * p.kv.head_stride;
      };
      bool ok = true;
      if (SHARED && half == 1) {
        // the keys are the values
      } else if (p.box > 0) {
        // lane i: channels 64 (i % BLKS) of the box of rows (i / BLKS) * p.box of each tile
        constexpr int BLKS = D / 64;
        const int br = lane / BLKS * p.box;
        const bool mine = group == 0 && br < KT;
        auto some = [&](int a, int n) { return a <= wk.pmax && (a + n > wk.lo || a < wk.ns); };
        auto page_of = [&](int tile) -> int {
          if (!mine || tile >= wk.tiles || !some(wk.tile_start(tile) + br, p.box)) return -1;
          const int pg = __ldg(p.kv.table + wk.b * p.kv.table_stride + ((wk.tile_start(tile) + br) >> p.kv.page_shift));
          if (pg >= 0 && pg < p.kv.n_pages) return pg;
          raise_dev_error(p.kv.err, DEVERR_BOUNDS);
          return -1;
        };
        int page = page_of(0);
        uint32_t fixes = 0;                            // tiles with rows to zero so far
        int issued = 0;                                // tiles whose boxes complete on their own barrier
        for (int tile = 0; tile < (group == 0 ? wk.tiles : 0) && ok; ++tile) {
          const int next = page_of(tile + 1);
          const int st = tile % ring, t0 = wk.tile_start(tile), a = t0 + br;
          uint8_t* dst = dst0 + st * L::TILE;
          const bool any = mine && some(a, p.box);
          const bool all = any && ((a >= wk.lo && a + p.box - 1 <= wk.pmax) || a + p.box <= wk.ns);
          const bool lost = any && page < 0;
          const bool box = any && !lost;
          // values: rows to zero, by boxes (what a block of 32 that is seen holds besides wanted rows)
          const bool clean = half == 1 || SHARED;
          const uint32_t boxes = __ballot_sync(0xffffffffu, box);
          uint32_t rows = __ballot_sync(0xffffffffu, clean && mine && !(box && all) && lane % BLKS == 0 &&
                                                         some(a & ~(KB - 1), KB));
          const bool some_lost = __any_sync(0xffffffffu, lost);
          ok = wait(empties + st, ((tile / ring) & 1) ^ 1);
          if (!ok) break;
          if (half == 0 && lane < 4) {
            // tokens present, 32 to a word
            uint32_t here = 0xffffffffu;
            if (some_lost)
              for (int i = 0; i < KB; ++i) {
                const int j = t0 + lane * KB + i;
                if (wanted(j) && row_of(j) < 0) here &= ~(1u << i);
              }
            bits[(tile % kBits) * 4 + lane] = here;
          }
          __syncwarp();
          uint64_t* const bar_at = rows ? fix_bar : fulls + st;
          if (lane == 0) mbar_arrive_expect_tx(bar_at, __popc(boxes) * p.box * 128);
          __syncwarp();
          if (box)
            tma_load_page(dst + (lane % BLKS) * L::BLK + br * 128, half ? &v_map : &k_map, bar_at, (lane % BLKS) * 64, kvh,
                          a & ((1 << p.kv.page_shift) - 1), page);
          __syncwarp();
          if (!rows) issued = tile + 1;
          if (rows) {
            ok = wait(fix_bar, fixes & 1);
            ++fixes;
            if (!ok) break;
            for (; rows; rows &= rows - 1) {
              const int src_lane = __ffs(rows) - 1, r0 = src_lane / BLKS * p.box;
              const bool loaded = (boxes >> src_lane) & 1u;
              for (int r = r0; r < r0 + p.box; ++r)
                if (!loaded || !wanted(t0 + r))
                  if (lane < D / 8)
                    *reinterpret_cast<uint4*>(dst + (lane / 8) * L::BLK + sw128_offset(r, lane % 8)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(fulls + st);
          }
          page = next;
        }
        if (!ok) {
          // copies in flight land before the block's shared memory goes
          volatile int never = 0;
          for (int t = max(0, issued - ring); t < issued; ++t) wait_phase(fulls + t % ring, (t / ring) & 1, &never, p.kv.err);
        }
      } else {
        // block u % 4 of tile u / 4, three warps in turn
        constexpr int CH = FP4 ? D / 32 : D / 8;       // 16-byte pieces of a row
        const int units = 4 * wk.tiles;
        auto lane_row = [&](int u) -> int64_t {
          if (u >= units) return -1;
          const int j = wk.tile_start(u >> 2) + (u & 3) * KB + lane;
          return wanted(j) ? row_of(j) : -1;
        };
        uint64_t* waiting = nullptr;                   // copies issued, not yet announced
        auto announce = [&](int keep) {                // the copies before the last `keep` groups have landed
          if (keep)
            cp_async_wait<1>();
          else
            cp_async_wait<0>();
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(waiting);
          waiting = nullptr;
        };
        int64_t row = lane_row(group);
        for (int u = group; u < units && ok; u += 3) {
          const int tile = u >> 2, r0 = (u & 3) * KB, st = tile % ring;
          const int64_t next = lane_row(u + 3);
          const bool want = wanted(wk.tile_start(tile) + r0 + lane);
          const uint32_t lost = __ballot_sync(0xffffffffu, want && row < 0);
          const bool none = !__any_sync(0xffffffffu, want);              // its columns are never used
          uint8_t* dst = dst0 + st * L::TILE;
          const uint32_t parity = ((tile / ring) & 1) ^ 1;
          if (!FP4) {
            // do not hold back what has landed while the stage is still in use
            if (waiting && !__all_sync(0xffffffffu, mbar_try_wait(empties + st, parity))) announce(0);
            ok = wait(empties + st, parity);
            if (!ok) break;
            if (!none) {
#pragma unroll 8
              for (int i = 0; i < CH; ++i) {
                const int piece = i * 32 + lane, r = piece / CH, c = piece % CH;
                const int64_t at = __shfl_sync(0xffffffffu, row, r);
                cp_async_16(dst + (c / 8) * L::BLK + sw128_offset(r0 + r, c % 8), src + (at < 0 ? 0 : at * 2 + c * 16),
                            at < 0 ? 0u : 16u);
              }
            }
            cp_async_commit();
            if (half == 0 && lane == 0) bits[(tile % kBits) * 4 + (u & 3)] = ~lost;
            if (waiting) announce(1);
            waiting = fulls + st;
          } else {
            const uint8_t* sc = half ? p.kv.v_scales : p.kv.k_scales;
            uint4 w[CH];
            uint32_t s2[CH];
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              const int piece = i * 32 + lane, r = piece / CH, c = piece % CH;
              const int64_t at = __shfl_sync(0xffffffffu, row, r);
              w[i] = make_uint4(0, 0, 0, 0);
              s2[i] = 0;
              if (at >= 0) {
                w[i] = __ldg(reinterpret_cast<const uint4*>(src + at / 2) + c);
                s2[i] = __ldg(reinterpret_cast<const uint16_t*>(sc + at / 16) + c);
              }
            }
            ok = wait(empties + st, parity);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < CH; ++i) {
              const int piece = i * 32 + lane, r = r0 + piece / CH, c = (piece % CH) * 4;
              const uint32_t lo = scale_pair(s2[i] & 255u), hi = scale_pair(s2[i] >> 8);
              uint8_t* d = dst + (c / 8) * L::BLK;
              *reinterpret_cast<uint4*>(d + sw128_offset(r, c % 8)) = dequant8(w[i].x, lo);
              *reinterpret_cast<uint4*>(d + sw128_offset(r, c % 8 + 1)) = dequant8(w[i].y, lo);
              *reinterpret_cast<uint4*>(d + sw128_offset(r, c % 8 + 2)) = dequant8(w[i].z, hi);
              *reinterpret_cast<uint4*>(d + sw128_offset(r, c % 8 + 3)) = dequant8(w[i].w, hi);
            }
            if (half == 0 && lane == 0) bits[(tile % kBits) * 4 + (u & 3)] = ~lost;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(fulls + st);
          }
          row = next;
        }
        if (waiting) announce(0);
      }
    } else {
      // ------------------------------------------------------------ products
      const int w = warp - 8;
      constexpr uint32_t idesc_s = idesc_of<T>(128, HT, false, false), idesc_o = idesc_of<T>(128, D, false, true);
      const RowTile rt(wk, w, p.G, p.window, p.sinks);
      const uint32_t s_at = __shfl_sync(0xffffffffu, tmem, 0) + w * 128, o_at = s_at + O_COL;
      const uint64_t q_desc = desc_kmajor_sw128(smem_u32(smem + L::Q + w * L::TILE)), k_desc = desc_kmajor_sw128(smem_u32(sK));
      const uint64_t v_desc = desc_mnmajor_sw128(smem_u32(sV), L::BLK, 1024);
      uint32_t p_phase = 0;                            // bit h: parity of p_full[w][h]
      uint32_t started = 0;                            // the output has its first product
      auto wait = [&](uint64_t* at, uint32_t parity) {
        return wait_phase(at, parity, abort_flag, p.kv.err);
      };
      auto scores = [&](int j, int h) {                // called by one lane
        const uint64_t bk = desc_at(k_desc, (j % L::KST) * L::TILE + h * HT * 128);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_bf16(s_at + h * HT, desc_at(q_desc, (kk >> 2) * L::BLK + (kk & 3) * 32),
                   desc_at(bk, (kk >> 2) * L::BLK + (kk & 3) * 32), idesc_s, kk != 0);
        mma_commit(s_full + 2 * w + h);
      };
      uint32_t next = wk.tiles > 0 ? rt.blocks(wk, 0) : 0u;
      bool ok = wait(q_full, 0);
      if (wk.tiles > 0 && ok) {
        ok = wait(k_full, 0);
        tc_fence_after();
        if (ok && elect_one()) {
          if (next & 3u) scores(0, 0);
          if (next & 12u) scores(0, 1);
          if (!SHARED) mma_commit(k_empty);
        }
        __syncwarp();
      }
      for (int j = 0; j < wk.tiles && ok; ++j) {
        const uint64_t bv = desc_at(v_desc, (j % VS) * L::TILE);
        const uint32_t act = next;
        const bool more = j + 1 < wk.tiles;
        next = more ? rt.blocks(wk, j + 1) : 0u;
        ok = wait(v_full + j % VS, (j / VS) & 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t mine = (act >> (2 * h)) & 3u;
          if (ok && mine) {
            ok = wait(p_full + 2 * w + h, (p_phase >> h) & 1);
            p_phase ^= 1u << h;
          }
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {              // 16 keys per product, a block at a time
              if (!((mine >> c) & 1u)) continue;
              const int kk = 4 * h + 2 * c;
              mma_ts(o_at, s_at + h * HT + c * 16, desc_at(bv, kk * 2048), idesc_o, started | (c & mine));
              mma_ts(o_at, s_at + h * HT + c * 16 + 8, desc_at(bv, kk * 2048 + 2048), idesc_o, 1u);
            }
            if (mine) mma_commit(pv_done + 2 * w + h);
            if (h == 1) mma_commit(v_empty + j % VS);  // this row tile is past the tile's values
          }
          __syncwarp();
          if (h == 0 && more) {
            ok = wait(k_full + (j + 1) % L::KST, ((j + 1) / L::KST) & 1);
            if (!ok) break;
            tc_fence_after();
          }
          if (elect_one()) {
            if ((next >> (2 * h)) & 3u) scores(j + 1, h);
            if (!SHARED && h == 1 && more) mma_commit(k_empty + (j + 1) % L::KST);
          }
          __syncwarp();
          if (mine) started = 1u;
        }
      }
      // completes once every product issued above has, also when a wait gave up
      if (elect_one()) mma_commit(all_done + w);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    if (FP4)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int w = warp >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;                    // row of the tile = TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_at = tmem + lane_off + w * 128, o_at = tmem + lane_off + O_COL + w * 128;
    const bool live = w * RT + r < wk.n_rows;
    const int rr = wk.r0 + w * RT + r, tok = rr / p.G, head = kvh * p.G + (rr - tok * p.G);
    const int64_t q_at = live ? (static_cast<int64_t>(wk.q_row0) + tok) * p.q_token + head * p.q_head : -1;
    constexpr int CH = D / 8;                          // 16-byte pieces of a row
    if (p.q_tokens) {
      // boxes of whole tokens; rows past the last hold other queries, which nobody reads
      if (threadIdx.x == 0) mbar_arrive_expect_tx(q_full, (wk.n_rows > RT ? 2 : 1) * L::TILE);
      if (threadIdx.x == 0)
        for (int i = 0; i < (wk.n_rows > RT ? 2 : 1) * (D / 64); ++i)
          tma_load_q(smem + L::Q + i * L::BLK, &q_map, q_full, i % (D / 64) * 64, kvh * p.G,
                     wk.q_row0 + wk.r0 / p.G + i / (D / 64) * p.q_tokens);
    } else {
      // the warp's 32 q rows (zero past the last) into the K-major swizzled tile
      uint4 v[CH];
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, q_at, (i * 32 + lane) / CH);
        v[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(p.q + at) + lane % CH) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int row = quad * 32 + (i * 32 + lane) / CH, c = lane % CH;
        v[i].x ^= p.flip;
        v[i].y ^= p.flip;
        v[i].z ^= p.flip;
        v[i].w ^= p.flip;
        *reinterpret_cast<uint4*>(smem + L::Q + w * L::TILE + (c / 8) * L::BLK + sw128_offset(row, c % 8)) = v[i];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const RowTile rt(wk, w, p.G, p.window, p.sinks);
    const int pos = live ? wk.base + tok : -1;
    // tokens [win, pos] and [0, sink_end) are visible
    const int win = p.window > 0 ? pos - p.window + 1 : 0;
    const int sink_end = min(p.sinks, pos + 1);
    constexpr float LIFT = lift_of<T>();
    float m = -INFINITY;                               // the reference (none yet: -inf)
    float2 l = make_float2(0.0f, 0.0f);
    uint32_t phase = 0, pv_phase = 0;                  // bit h: parity of s_full[w][h], of pv_done[w][h]
    int last = 0;                                      // half handed on last
    bool any = false, ok = true;
    // The reference stays while the maximum has not outgrown it; else the output so
    // far is rescaled, once the products of the half handed on last have ended.
    auto refer = [&](float top) -> float {
      const bool grow = top > m + (kLazy + LIFT) || (m == -INFINITY && top > -INFINITY);
      const float now = lifted(top, LIFT);
      if (__any_sync(0xffffffffu, grow)) {
        const bool scale_o = grow && m > -INFINITY;
        if (__any_sync(0xffffffffu, scale_o)) {
          const float f = scale_o ? exp2_approx(m - now) : 1.0f;
          l.x *= f;
          l.y *= f;
          ok = wait_phase(pv_done + 2 * w + last, ((pv_phase >> last) & 1) ^ 1, abort_flag, p.kv.err);
          if (ok) {
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < D / 16; ++i) {
              uint32_t x[16];
              tmem_ld16(o_at + i * 16, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
              tmem_st16(o_at + i * 16, x);
            }
          }
        }
        if (grow) m = now;
      }
      return m == -INFINITY ? 0.0f : m;
    };
    for (int j = 0; j < wk.tiles && ok; ++j) {
      const uint32_t act = rt.blocks(wk, j);
      const int t0 = wk.tile_start(j);
      const volatile uint32_t* here = bits + (j % kBits) * 4;
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint32_t mine = (act >> (2 * h)) & 3u;
        if (mine == 0) continue;
        const int th = t0 + h * HT;
        const uint32_t sh = s_at + h * HT;
        ok = wait_phase(s_full + 2 * w + h, (phase >> h) & 1, abort_flag, p.kv.err);
        if (!ok) break;
        phase ^= 1u << h;
        any = true;
        tc_fence_after();
        const bool plain = mine == 3u && th >= win && th + HT - 1 <= pos && (here[2 * h] & here[2 * h + 1]) == 0xffffffffu;
        if (__all_sync(0xffffffffu, plain)) {
          // every row sees all 64: the scores stay in registers
          float s[HT];
          tmem_ld32(sh, *reinterpret_cast<uint32_t(*)[32]>(s));
          tmem_ld32(sh + KB, *reinterpret_cast<uint32_t(*)[32]>(s + KB));
          tmem_wait_ld();
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < HT - 4; i += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[i + e], s[i + 4 + e]);
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[HT - 4 + e]);
          const float ref = refer(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale2);
          const float2 sc = make_float2(p.scale2, p.scale2), nr = make_float2(-ref, -ref);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = fma2(make_float2(s[c * KB + 2 * i], s[c * KB + 2 * i + 1]), sc, nr);
              const float2 e = weights(i, x);
              l = add2(l, e);
              pk[i] = Num<T>::down(e.x, e.y);
            }
            tmem_st16(sh + c * 16, pk);
          }
        } else {
          // block by block, read twice (the weights of block 1 land on block 0's
          // scores, which have been read)
          auto visible = [&](int c) -> uint32_t {      // bit i: token i of the block
            const int t = th + c * KB;
            auto upto = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
            return ((upto(pos + 1 - t) & ~upto(win - t)) | upto(sink_end - t)) & here[2 * h + c];
          };
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            if (!((mine >> c) & 1u)) continue;
            uint32_t v[KB];
            tmem_ld32(sh + c * KB, v);
            const uint32_t vis = visible(c);
            tmem_wait_ld();
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < KB; ++i)
              mx[i & 1] = fmaxf(mx[i & 1], (vis >> i) & 1u ? __uint_as_float(v[i]) : -INFINITY);
            top = fmaxf(top, fmaxf(mx[0], mx[1]));
          }
          const float ref = refer(top * p.scale2);
          const float2 sc = make_float2(p.scale2, p.scale2), nr = make_float2(-ref, -ref);
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            if (!((mine >> c) & 1u)) continue;
            uint32_t v[KB], pk[16];
            tmem_ld32(sh + c * KB, v);
            const uint32_t vis = visible(c);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 x = fma2(make_float2((vis >> (2 * i)) & 1u ? __uint_as_float(v[2 * i]) : -INFINITY,
                                                (vis >> (2 * i + 1)) & 1u ? __uint_as_float(v[2 * i + 1]) : -INFINITY),
                                    sc, nr);
              const float2 e = weights(i, x);
              l = add2(l, e);
              pk[i] = Num<T>::down(e.x, e.y);
            }
            tmem_st16(sh + c * 16, pk);
          }
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 2 * w + h);
        pv_phase ^= 1u << h;
        last = h;
      }
    }
    if (any && ok) {
      ok = wait_phase(all_done + w, 0, abort_flag, p.kv.err);
      tc_fence_after();
    } else if (ok) {
      // no product has waited for q, which lands where the outputs pass through
      ok = wait_phase(q_full, 0, abort_flag, p.kv.err);
    }
    if (ok) {
      const float sum = l.x + l.y;
      const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
      const int64_t at = (static_cast<int64_t>(wk.q_row0) + tok) * p.Hq + head;
      // through the row tile's q rows, which no product reads any more, so that a
      // warp stores whole rows
      uint8_t* const stage = smem + L::Q + w * L::TILE;
      bool odd = false;                                // an output that is not finite
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        if (any) {
          tmem_ld32(o_at + c * 32, v);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0;
        }
        if (!FP4)
        {
          float2 z = make_float2(0.0f, 0.0f);          // stays 0 for finite values
#pragma unroll
          for (int i = 0; i < 16; ++i)
            z = fma2(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), make_float2(0.0f, 0.0f), z);
          odd |= !(z.x + z.y == 0.0f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = Num<T>::down(__uint_as_float(v[8 * i + 2 * e]) * inv, __uint_as_float(v[8 * i + 2 * e + 1]) * inv);
          *reinterpret_cast<uint4*>(stage + (c / 2) * L::BLK + sw128_offset(r, (c % 2) * 4 + i)) =
              make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
      __syncwarp();
      const int64_t out_at = live ? at * D : -1;
#pragma unroll 4
      for (int i = 0; i < CH; ++i) {
        const int row = quad * 32 + (i * 32 + lane) / CH, c = lane % CH;
        const int64_t to = __shfl_sync(0xffffffffu, out_at, (i * 32 + lane) / CH);
        const uint4 x = *reinterpret_cast<const uint4*>(stage + (c / 8) * L::BLK + sw128_offset(row, c % 8));
        if (to >= 0) reinterpret_cast<uint4*>(p.out + to)[c] = x;
      }
      if (!FP4) smem[L::BAD + w * RT + r] = odd && live && (__float_as_uint(sum) & 0x7f800000u) != 0x7f800000u;
      if (live && p.lse) p.lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
    }
  }
  // every product has completed before TMEM and shared memory go
  volatile int never = 0;                              // also when a wait gave up: the products still end
  wait_phase(all_done, 0, &never, p.kv.err);
  wait_phase(all_done + 1, 0, &never, p.kv.err);
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (!FP4) {
    const bool look = !*abort_flag && threadIdx.x < 2 * RT && smem[L::BAD + threadIdx.x];
    if (__syncthreads_or(look)) {
      // located anew: keeping the work alive to here cost 13 us of 291
      Work again;
      locate(p, blockIdx.x, again);
      const MendRows m = {p.q + static_cast<int64_t>(again.q_row0) * p.q_token, p.q_token, p.q_head,
                          p.out + static_cast<int64_t>(again.q_row0) * p.Hq * D, p.flip ? -p.scale2 : p.scale2, p.Hq, p.G,
                          static_cast<int>(blockIdx.y), again.r0, again.base, p.window, p.sinks, again.lo, again.ns,
                          again.pmax, again.b};
      mend_rows<T, D>(m, p.kv, smem + L::BAD, again.n_rows, reinterpret_cast<uint32_t*>(smem + L::K),
                      (L::KST + L::VST) * L::TILE * 8);
    }
  }
}

template <class T, int D, bool FP4, bool SHARED>
csa2_status run(const Params& p, dim3 grid, const CUtensorMap (&maps)[3], cudaStream_t stream) {
  using L = Lay<D, SHARED>;
  static PerDevice<int> opted;
  opted.get(+[]() -> int {
    cudaFuncSetAttribute(paged_window_kernel<T, D, FP4, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    return 1;
  });
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attribute()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  begin_launch(stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_window_kernel<T, D, FP4, SHARED>, p, maps[0], maps[1], maps[2]);
  note_launch(LK_ATTN, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "csa2_paged_window_attn: launch failed: %s", cudaGetErrorString(e));
  }
  return check_launch("csa2_paged_window_attn");
}

}  // namespace

bool paged_window_tc_applies(const PagedAttn& a) { return a.D == 64 || a.D == 128; }

csa2_status launch_paged_window_tc(const PagedAttn& a, const int32_t* cu_q, int64_t T, cudaStream_t stream) {
  Params p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_token = a.q_token;
  p.q_head = a.q_head;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.cu_q = cu_q;
  p.T = T;
  const float s = a.scale * kLog2e;
  p.flip = s < 0.0f ? 0x80008000u : 0u;
  p.scale2 = std::max(s < 0.0f ? -s : s, 1.1754944e-38f);
  p.Hq = a.Hq;
  p.G = a.G;
  p.window = a.window;
  p.sinks = a.sinks;
  p.kv = a.kv;
  // at most one tile more per sequence than all rows need
  const int64_t tiles = (T * a.G + 2 * RT - 1) / (2 * RT) + a.kv.B;
  if (T * a.G > 0x7fffff00LL || tiles > 0x7fffffffLL) return fail(CSA2_ERR_UNSUPPORTED, "csa2_paged_window_attn: too many rows");
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(a.kv.heads));
  const bool sh = a.kv.v == a.kv.k;
  CUtensorMap maps[3] = {};                            // keys, values, q
  const int page = 1 << a.kv.page_shift;
  if (a.fmt != CSA2_KV_FP4 && page >= 8 && a.kv.n_pages > 0) {
    p.box = std::min(page, 32);
    for (int i = 0; i < (sh ? 1 : 2); ++i)
      CSA2_TRY(make_tensor_map_paged(&maps[i], i ? a.kv.v : a.kv.k, a.D, a.kv.heads, a.kv.head_stride, page,
                                     a.kv.token_stride, a.kv.n_pages, a.kv.page_stride, p.box));
  }
  // q by TMA when a row tile is whole tokens and no signs turn
  if (RT % a.G == 0 && p.flip == 0) {
    p.q_tokens = RT / a.G;
    CSA2_TRY(make_tensor_map_heads(&maps[2], a.q, a.D, a.Hq, a.q_head, T, a.q_token, a.G, p.q_tokens));
  }
#define CSA2_WIN_T(T_, D_, F_) (sh ? run<T_, D_, F_, true>(p, grid, maps, stream) : run<T_, D_, F_, false>(p, grid, maps, stream))
#define CSA2_WIN(D_)                                                                       \
  if (a.D == D_)                                                                           \
    return a.fmt == CSA2_KV_FP4   ? CSA2_WIN_T(__nv_bfloat16, D_, true)                    \
           : a.fmt == CSA2_KV_F16 ? CSA2_WIN_T(__half, D_, false)                          \
                                  : CSA2_WIN_T(__nv_bfloat16, D_, false);
  CSA2_WIN(64) CSA2_WIN(128)
#undef CSA2_WIN
#undef CSA2_WIN_T
  return CSA2_ERR_UNSUPPORTED;
}

}  // namespace csa2
