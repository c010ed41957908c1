// Attention over a paged cache of a token's many query heads per cache head (a shared
// 512-wide row under 64 heads: 128 flops per byte), on the 5th-generation tensor
// cores: one new token per sequence, its keys cut into chunks, or a prompt, one CTA
// per token (all its rows see the same keys).
//
// A CTA takes up to NH query heads of one cache head and a run of key tiles of 128
// tokens.  Keys stand on the M side, heads on the N side, so that a cached row is
// read from shared memory as it lies, as key and as value:
//   S^T[key, head] = K q^T        (M = 128 keys, N = NH, K = D)
//   O^T[channel, head] += V^T P   (M = 128 channels, N = NH, K = 128 keys)
//   warps 0-15      softmax, one thread per key and 16 of the heads (warps 0-3 alone
//                   for up to 16): P = 2^(s - ref) (f16: lifted by 2^7), row sums kept per thread and added
//                   up at the end
//   one warp        issues the products
//   three warps     fill a ring of 8 blocks of 64 channels x 128 keys (16 KiB, TMA
//                   boxes by page); a block of a shared row serves the score and then
//                   the value product and is refilled as soon as its channels are
//                   through.  (One warp took 450 clocks a block to issue.)  The tile
//                   behind is asked into L2 meanwhile.
// A head's reference is its maximum over the first tile that shows it a score above -inf, and
// moves (with a rescaled output in TMEM) only when some score has outgrown it by 2^8, so the steady state
// takes no maximum across keys: one barrier with an OR per tile asks whether any has.
//
// A 128 KiB tile of 512 channels arrives in 5600 clocks at an SM's share of the memory
// rate, but it fills shared memory next to q, so a tile is a chain: value products (1750
// clocks, a pair of blocks free every 440), the next tile's blocks from L2 (3500 at the 37
// bytes a clock an SM gets), the last pair's score products (650), softmax (1000): 6200.
// Measured: 32 sequences of 65536 tokens, 64 heads over one 512-wide row, 441 us (4.9 TB/s);
// without the prefetch into L2 461, with 8 softmax warps 450, half of their exponentials
// on the multiply-add pipe no change.  That is at 1965 MHz: run for seconds, the card is at
// its power limit, the clock at 1640 MHz and the time at 512 us, so clocks bound it.
#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"
#include "launchers.h"
#include "paged_attn.cuh"

namespace csa2 {
namespace {
using namespace paged;
using namespace sm100;
using rope::Num;

constexpr int kLoaders = 3;
constexpr int KT = 128;                                // keys per tile
constexpr int SLOTS = 8;
constexpr int BLK = KT * 128;                          // 64 channels of 128 keys
constexpr int kBits = 8;
constexpr float kLazy = 8.0f;

template <int D, int NH>
struct Lay {
  static constexpr int SW = NH == 64 ? 16 : 4;          // softmax warps
  static constexpr int HW = 16;                        // heads per softmax thread
  static_assert(SW * HW == 4 * NH, "a thread per key and 16 heads");
  static constexpr int THREADS = (SW + 1 + kLoaders) * 32;
  static constexpr int DB = D / 64;                    // blocks per tile of keys (or values)
  static constexpr int QB = NH * 128;                  // 64 channels of q
  static constexpr int RING = 0;
  static constexpr int Q = RING + SLOTS * BLK;
  static constexpr int P = Q + DB * QB;                // [128 keys][64 heads]
  static constexpr int REF = P + BLK;                  // -reference[NH], factor[NH]
  static constexpr int RED = REF + 2 * NH * 4;         // [4][NH]
  static constexpr int BAR = RED + 4 * NH * 4;
  static constexpr int NBAR = 2 * SLOTS + 3 + kLoaders;
  static constexpr int BITS = BAR + NBAR * 8;
  static constexpr int MISC = BITS + kBits * 4 * 4;
  static constexpr int BYTES = MISC + 16 + 1024;
  static_assert(P % 1024 == 0 && Q % 1024 == 0, "swizzled tiles");
};

struct Params {
  const uint16_t* q;
  int64_t q_token, q_head;
  uint16_t* out;
  float* lse;
  float* part_o;                     // [B * Hq][chunks][D]
  float2* part_ml;
  float scale2;                      // |scale| * log2(e), at least the smallest normal
  uint32_t flip;                     // 0x80008000 for a negative scale
  const int32_t* cu_q;               // prompt: [B + 1]; null: decode
  int T;                             // prompt: rows of q
  int Hq, G, row_tiles, window, sinks, chunk, chunks;
  int box;                           // rows of a TMA box
  PagedView kv;
};

// the softmax warps: do any of their N threads have `pred`
template <int N>
__device__ __forceinline__ bool any_of(bool pred) {
  uint32_t r;
  asm volatile(
      "{.reg .pred p, q; setp.ne.b32 p, %1, 0; barrier.cta.red.or.pred q, 1, %2, p; selp.u32 %0, 1, 0, q;}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred)), "n"(N)
      : "memory");
  return r != 0;
}
template <int N>
__device__ __forceinline__ void bar_of() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(N) : "memory");
}

template <class T, int D, int NH, bool SHARED>
__global__ void __launch_bounds__(Lay<D, NH>::THREADS, 1)
    paged_wide_kernel(const Params p, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using L = Lay<D, NH>;
  constexpr int DB = L::DB, SW = L::SW, HW = L::HW;
  constexpr float LIFT = lift_of<T>(), LAG = kLazy + LIFT;         // the largest log2 of a weight
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::BAR);
  uint64_t *const full = bar, *const empty = bar + SLOTS;
  uint64_t *const s_full = bar + 2 * SLOTS, *const p_full = s_full + 1, *const all_done = s_full + 2, *const fix_bars = s_full + 3;
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + L::BITS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC + 4);
  float* ref = reinterpret_cast<float*>(smem + L::REF);
  float* factor = ref + NH;
  float* red = reinterpret_cast<float*>(smem + L::RED);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int b = blockIdx.z, token = blockIdx.z;              // sequence, row of q
  const int chunk = p.cu_q ? 0 : blockIdx.x;
  const int kvh = blockIdx.y / p.row_tiles, h0 = NH * (blockIdx.y % p.row_tiles);
  const int rows = min(NH, p.G - h0);
  pdl_wait();
  int pos;
  if (p.cu_q) {
    // the sequence of this token (late tokens see most and start first)
    token = p.T - 1 - static_cast<int>(blockIdx.x);
    int n = 0, from = 0;
    b = -1;
    for (int s0 = 0; s0 < p.kv.B && b < 0; s0 += 32) {
      int c0 = 0, c1 = 0;
      if (s0 + lane < p.kv.B) {
        c0 = __ldg(p.cu_q + s0 + lane);
        c1 = __ldg(p.cu_q + s0 + lane + 1);
        if (c0 < 0 || c1 < c0 || c1 > p.T) {
          if (warp == 0) raise_dev_error(p.kv.err, DEVERR_BOUNDS);
          c0 = c1 = 0;
        }
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, token >= c0 && token < c1);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = s0 + src;
        from = __shfl_sync(0xffffffffu, c0, src);
        n = __shfl_sync(0xffffffffu, c1, src) - from;
      }
    }
    if (b < 0) return;                                 // a row of no sequence
    pos = length_of(p.kv, b, threadIdx.x == 0) - n + (token - from);
  } else {
    pos = length_of(p.kv, b, threadIdx.x == 0) - 1;
  }
  const AlignedTiles at(pos, p.window, p.sinks);
  const int per = p.chunk / KT;
  const int first = chunk * per;
  if (chunk > 0 && first >= at.tiles) return;
  const int tiles = (chunk + 1 < p.chunks ? min(at.tiles, first + per) : at.tiles) - first;

  if (threadIdx.x == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, SW);
    mbar_init(all_done, 1);
    for (int i = 0; i < kLoaders; ++i) mbar_init(fix_bars + i, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == SW) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp < SW) {
    // q rows (zero past the last) into K-major swizzled blocks
#pragma unroll 8
    for (int i = threadIdx.x; i < NH * (D / 8); i += SW * 32) {
      const int r = i / (D / 8), c = i % (D / 8);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        v = __ldg(reinterpret_cast<const uint4*>(p.q + token * p.q_token + (kvh * p.G + h0 + r) * p.q_head) + c);
        v.x ^= p.flip;
        v.y ^= p.flip;
        v.z ^= p.flip;
        v.w ^= p.flip;
      }
      *reinterpret_cast<uint4*>(smem + L::Q + (c / 8) * L::QB + sw128_offset(r, c % 8)) = v;
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t O_COL = 128;                      // S at column 0, O block db at 128 + 64 db
  auto wait = [&](uint64_t* x, uint32_t parity) { return wait_phase(x, parity, abort_flag, p.kv.err); };

  if (warp > SW) {
    // ------------------------------------------------------------ loader
    // loader lw takes the blocks lw, lw + 3, .. of a tile; lane i: rows i * p.box ..
    const int lw = warp - SW - 1;
    uint64_t* const fix_bar = fix_bars + lw;
    const int br = lane * p.box;
    const bool mine = br < KT;
    auto some = [&](int a, int n) { return a <= at.pmax && (a + n > at.lo || a < at.ns); };
    auto wanted = [&](int j) { return j <= at.pmax && (j >= at.lo || j < at.ns); };
    auto page_of = [&](int tile) -> int {
      if (!mine || tile >= tiles || !some(at.start(first + tile) + br, p.box)) return -1;
      const int pg = __ldg(p.kv.table + b * p.kv.table_stride + ((at.start(first + tile) + br) >> p.kv.page_shift));
      if (pg >= 0 && pg < p.kv.n_pages) return pg;
      raise_dev_error(p.kv.err, DEVERR_BOUNDS);
      return -1;
    };
    int page = page_of(0);
    uint32_t u = 0, issued = 0, fixes = 0;             // blocks of tiles behind, blocks asked for
    bool ok = true;
    for (int tile = 0; tile < tiles && ok; ++tile) {
      const int next = page_of(tile + 1);
      if (next >= 0) {
        // the tile behind goes to L2 while this one fills shared memory
        const int sl = (at.start(first + tile + 1) + br) & ((1 << p.kv.page_shift) - 1);
        for (int i = lw; i < DB; i += kLoaders) {
          tma_prefetch_page(&k_map, i * 64, kvh, sl, next);
          if (!SHARED) tma_prefetch_page(&v_map, i * 64, kvh, sl, next);
        }
      }
      const int t0 = at.start(first + tile), a = t0 + br;
      const bool any = mine && some(a, p.box);
      const bool all = any && ((a >= at.lo && a + p.box - 1 <= at.pmax) || a + p.box <= at.ns);
      const bool box = any && page >= 0;
      const uint32_t boxes = __ballot_sync(0xffffffffu, box);
      const uint32_t zero = __ballot_sync(0xffffffffu, mine && !(box && all));   // boxes with rows to zero
      const bool some_lost = __any_sync(0xffffffffu, any && page < 0);
      const int slot_in_page = a & ((1 << p.kv.page_shift) - 1);
#pragma unroll
      for (int half = 0; half < (SHARED ? 1 : 2); ++half) {
        // values whose unwanted rows are zeroed before their blocks are announced
        const bool fix = zero != 0 && (half == 1 || SHARED);
        for (int i = lw; i < DB && ok; i += kLoaders) {
          const uint32_t st = (u + i) % SLOTS;
          ok = wait(empty + st, (((u + i) / SLOTS) & 1) ^ 1);
          if (!ok) break;
          if (half == 0 && i == 0) {
            // tokens present, 32 to a word
            if (lane < 4) {
              uint32_t here = 0xffffffffu;
              if (some_lost)
                for (int e = 0; e < 32; ++e) {
                  const int j = t0 + lane * 32 + e;
                  if (wanted(j) && token_row(p.kv, b, j) < 0) here &= ~(1u << e);
                }
              bits[(tile % kBits) * 4 + lane] = here;
            }
            __syncwarp();
          }
          uint64_t* const to = fix ? fix_bar : full + st;
          uint8_t* const dst = smem + L::RING + st * BLK;
          if (lane == 0) mbar_arrive_expect_tx(to, __popc(boxes) * p.box * 128);
          __syncwarp();
          if (box) tma_load_page(dst + br * 128, half ? &v_map : &k_map, to, i * 64, kvh, slot_in_page, page);
          __syncwarp();
          if (!fix) {
            issued = u + i + 1;
            continue;
          }
          ok = wait(fix_bar, fixes & 1);
          ++fixes;
          if (!ok) break;
          for (uint32_t z = zero; z; z &= z - 1) {
            const int src = __ffs(z) - 1;
            const bool loaded = (boxes >> src) & 1u;
#pragma unroll 4
            for (int x = lane; x < p.box * 8; x += 32) {
              const int r = src * p.box + x / 8;
              if (!loaded || !wanted(t0 + r))
                *reinterpret_cast<uint4*>(dst + sw128_offset(r, x % 8)) = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + st);
          issued = u + i + 1;
        }
        if (!ok) break;
        u += DB;
      }
      page = next;
    }
    if (!ok) {
      // copies in flight land before the block's shared memory goes
      volatile int never = 0;
      for (uint32_t i = issued > SLOTS ? issued - SLOTS : 0; i < issued; ++i)
        if (i % DB % kLoaders == static_cast<uint32_t>(lw)) wait_phase(full + i % SLOTS, (i / SLOTS) & 1, &never, p.kv.err);
    }
  } else if (warp == SW) {
    // ------------------------------------------------------------ products
    constexpr uint32_t idesc_s = idesc_of<T>(128, NH, false, false), idesc_o = idesc_of<T>(128, NH, true, true);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t q_desc = desc_kmajor_sw128(smem_u32(smem + L::Q)), k_desc = desc_kmajor_sw128(smem_u32(smem + L::RING));
    const uint64_t v_desc = desc_mnmajor_sw128(smem_u32(smem + L::RING), BLK, 1024);
    const uint64_t p_desc = desc_mnmajor_sw128(smem_u32(smem + L::P), BLK, 1024);
    uint32_t u = 0;                                    // blocks taken
    bool ok = true;
    for (int tile = 0; tile < tiles && ok; ++tile) {
      // two blocks at a time.  The two waits cost 206 clocks even for blocks that are
      // there, half of their products' time, so one look at all blocks comes first.
      const uint32_t mine = u + (lane & (DB - 1));
      uint32_t here = 0;
      for (int i = 0; i < DB && ok; i += 2) {
        const uint32_t st = (u + i) % SLOTS, parity = ((u + i) / SLOTS) & 1;
        if (((here >> i) & 3u) != 3u) {
          here = __ballot_sync(0xffffffffu, phase_over(full + mine % SLOTS, (mine / SLOTS) & 1));
          __syncwarp();
          if (((here >> i) & 3u) != 3u) ok = wait(full + st, parity) && wait(full + st + 1, parity);
        }
        tc_fence_after();
        if (ok && elect_one()) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint64_t a = desc_at(k_desc, (st + e) * BLK), q = desc_at(q_desc, (i + e) * L::QB);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_bf16(tm, desc_at(a, kk * 32), desc_at(q, kk * 32), idesc_s, (i | e | kk) != 0);
            if (!SHARED) mma_commit(empty + st + e);
          }
          if (i == DB - 2) mma_commit(s_full);
        }
        __syncwarp();
      }
      if (!SHARED) u += DB;
      ok = ok && wait(p_full, tile & 1);
      for (int db = 0; db < D / 128 && ok; ++db) {
        const uint32_t st = (u + 2 * db) % SLOTS;
        if (!SHARED) ok = wait(full + st, ((u + 2 * db) / SLOTS) & 1) && wait(full + st + 1, ((u + 2 * db) / SLOTS) & 1);
        tc_fence_after();
        if (ok && elect_one()) {
          const uint64_t a = desc_at(v_desc, st * BLK);
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            mma_bf16(tm + O_COL + db * 64, desc_at(a, kk * 2048), desc_at(p_desc, kk * 2048), idesc_o,
                     tile > 0 || kk > 0);
          mma_commit(empty + st);
          mma_commit(empty + st + 1);
        }
        __syncwarp();
      }
      u += DB;
    }
    if (elect_one()) mma_commit(all_done);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and output
    const int key = (warp & 3) * 32 + lane;            // TMEM lane
    const int hb = warp / 4 * HW;                      // first of this thread's heads
    constexpr int N = SW * 32;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lane_off + hb, o_at = tmem + lane_off + O_COL + hb;
    float2 l[HW / 2];
#pragma unroll
    for (int h = 0; h < HW / 2; ++h) l[h] = make_float2(0.0f, 0.0f);
    if (threadIdx.x < NH) ref[threadIdx.x] = 0.0f;     // -reference: none so far
    bar_of<N>();
    const float4* const mine = reinterpret_cast<const float4*>(ref + hb);
    bool ok = true, started = false;                   // started: every head has a reference
    bool set = false;                                  // head threadIdx.x has one
    for (int tile = 0; tile < tiles && ok; ++tile) {
      ok = wait(s_full, tile & 1);
      tc_fence_after();
      float x[HW];
      auto scores = [&]() {
        tmem_ld16(s_at, *reinterpret_cast<uint32_t(*)[16]>(x));
        tmem_wait_ld();
      };
      if (ok) scores();
      const int j = at.start(first + tile) + key;
      const uint32_t here = *reinterpret_cast<volatile uint32_t*>(bits + (tile % kBits) * 4 + (warp & 3));
      const bool seen = ok && j <= at.pmax && (j >= at.lo || j < at.ns) && ((here >> lane) & 1u);
      // x - reference, rounded once, and the largest; a key that is not seen weighs nothing
      const float2 sc = make_float2(p.scale2, p.scale2);
      auto refer = [&]() -> float {
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < HW; h += 4) {
          const float4 r = mine[h / 4];
          const float2 a = fma2(make_float2(x[h], x[h + 1]), sc, make_float2(r.x, r.y));
          const float2 c = fma2(make_float2(x[h + 2], x[h + 3]), sc, make_float2(r.z, r.w));
          x[h] = seen ? a.x : -INFINITY;
          x[h + 1] = seen ? a.y : -INFINITY;
          x[h + 2] = seen ? c.x : -INFINITY;
          x[h + 3] = seen ? c.y : -INFINITY;
          top = max3(top, x[h], x[h + 1]);
          top = max3(top, x[h + 2], x[h + 3]);
        }
        return top;
      };
      const float top = refer();
      if (any_of<N>(!started || !ok || top > LAG)) {
        if (any_of<N>(!ok)) {                          // all leave together
          ok = false;
          break;
        }
        // every head's maximum over the tile; the heads that outgrew their reference, or
        // have none and see a score above -inf, move to it.  The scores are then taken
        // from the new one: what a far reference rounded away is not in x any more.
        scores();
#pragma unroll
        for (int h = 0; h < HW; ++h) {
          const float m = attn::warp_max_f32(seen ? x[h] * p.scale2 : -INFINITY);
          if (lane == 0) red[(warp & 3) * NH + hb + h] = m;
        }
        bar_of<N>();
        if (threadIdx.x < NH) {
          const int h = threadIdx.x;
          const float m = fmaxf(fmaxf(red[h], red[NH + h]), fmaxf(red[2 * NH + h], red[3 * NH + h]));
          const float was = ref[h];
          const bool move = set ? m + was > LAG : m > -INFINITY;
          const float now = -lifted(m, LIFT);
          if (move) ref[h] = now;
          factor[h] = move && set ? exp2_approx(now - was) : 1.0f;  // nothing weighed before: nothing to rescale
          set |= move;
        }
        started = !any_of<N>(threadIdx.x < rows && !set);
        scores();
        refer();
#pragma unroll
        for (int h = 0; h < HW; h += 2) {
          l[h / 2].x *= factor[hb + h];
          l[h / 2].y *= factor[hb + h + 1];
        }
        if (tile > 0) {
          // the value products of the tile before ended before this tile's scores did
#pragma unroll 1
          for (int i = 0; i < D / 128; ++i) {
            const uint32_t to = o_at + i * 64;
            uint32_t v[16];
            tmem_ld16(to, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * factor[hb + e]);
            tmem_st16(to, v);
          }
          tmem_wait_st();
        }
      }
      uint8_t* const prow = smem + L::P;
#pragma unroll
      for (int h = 0; h < HW; h += 8) {
        uint32_t pk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 e = make_float2(exp2_approx(x[h + 2 * i]), exp2_approx(x[h + 2 * i + 1]));
          l[h / 2 + i] = add2(l[h / 2 + i], e);
          pk[i] = Num<T>::down(e.x, e.y);
        }
        *reinterpret_cast<uint4*>(prow + sw128_offset(key, (hb + h) / 8)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
    ok = wait(all_done, 0) && ok;
    tc_fence_after();
    // row sums over the keys, through the ring (every product has ended)
    float* const sums = reinterpret_cast<float*>(smem + L::RING);      // [128][NH + 1]
#pragma unroll
    for (int h = 0; h < HW; h += 2) {
      sums[key * (NH + 1) + hb + h] = l[h / 2].x;
      sums[key * (NH + 1) + hb + h + 1] = l[h / 2].y;
    }
    bar_of<N>();
    if (threadIdx.x < NH) {
      const int h = threadIdx.x;
      float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll 8
      for (int i = 0; i < 128; i += 4) {
        s0 += sums[i * (NH + 1) + h];
        s1 += sums[(i + 1) * (NH + 1) + h];
        s2 += sums[(i + 2) * (NH + 1) + h];
        s3 += sums[(i + 3) * (NH + 1) + h];
      }
      factor[h] = tiles > 0 ? (s0 + s1) + (s2 + s3) : 0.0f;            // l
    }
    bar_of<N>();
    const int64_t row0 = static_cast<int64_t>(token) * p.Hq + kvh * p.G + h0;
    const bool partial = p.chunks > 1 && at.tiles > per;
#pragma unroll 1
    for (int db = 0; db < D / 128 && ok; ++db) {
      uint32_t v[16];
      if (tiles > 0) {
        tmem_ld16(o_at + db * 64, v);
        tmem_wait_ld();
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if (hb + e >= rows) break;
        const float o = tiles > 0 ? __uint_as_float(v[e]) : 0.0f;
        const int64_t row = row0 + hb + e;
        if (partial) {
          p.part_o[(row * p.chunks + chunk) * D + db * 128 + key] = o;
        } else {
          const float s = factor[hb + e];
          const float inv = s > 0.0f ? 1.0f / s : (s == 0.0f ? 0.0f : s);
          p.out[row * D + db * 128 + key] = static_cast<uint16_t>(Num<T>::down(o * inv, 0.0f) & 0xffffu);
        }
      }
    }
    if (threadIdx.x < rows && ok) {
      const int h = threadIdx.x;
      const float s = factor[h], m = -ref[h];
      if (partial)
        p.part_ml[(row0 + h) * p.chunks + chunk] = make_float2(s == 0.0f ? -INFINITY : m, s);
      else if (p.lse)
        p.lse[row0 + h] = s == 0.0f ? -INFINITY : (m + log2f(s)) * kLn2;
    }
  }
  volatile int never = 0;                              // also when a wait gave up: the products still end
  wait_phase(all_done, 0, &never, p.kv.err);
  tc_fence_before();
  __syncthreads();
  if (warp == SW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class T, int D, int NH, bool SHARED>
csa2_status run(const char* fn, const Params& p, dim3 grid, const CUtensorMap (&maps)[2], cudaStream_t stream) {
  using L = Lay<D, NH>;
  static PerDevice<int> opted;
  opted.get(+[]() -> int {
    cudaFuncSetAttribute(paged_wide_kernel<T, D, NH, SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
    return 1;
  });
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(L::THREADS);
  cfg.dynamicSmemBytes = L::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute at[1] = {pdl_attribute()};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  begin_launch(stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_wide_kernel<T, D, NH, SHARED>, p, maps[0], maps[1]);
  note_launch(LK_ATTN, 1, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(CSA2_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  }
  return check_launch(fn);
}

}  // namespace

int paged_wide_heads(const PagedAttn& a) { return a.G <= 16 ? 16 : 64; }

bool paged_wide_applies(const PagedAttn& a) {
  return a.fmt != CSA2_KV_FP4 && a.kv.page_shift >= 3 && a.kv.n_pages > 0 && a.D == 512;
}

// A CTA per token pays when its heads fill most of the 64 and it sees several tiles;
// else the 16-row tiles of paged_attn.cu, which take several tokens at once, are
// faster.  Measured (us, here / there): 512 tokens behind 1000, 64 heads over one
// 512-wide row, window 2048: 113 / 237; 1000 tokens, 64 heads over one 256-wide row:
// 161 / 414; 512 behind 1000, 16 heads over one 512-wide row: 91 / 75; 60 tokens, 64
// heads, window 128: 39 / 26.  The two round differently, so the rule takes what belongs
// to the layer (format, pages, width, heads, window) and not the table's width or a
// batch's lengths: a query's bits stay the same when its table grows.  Short prompts without
// a window pay for that: one of 60 tokens, 64 heads x 512, 23 / 13; 150 tokens 43 / 40; 300
// tokens 68 / 99.
bool paged_wide_prompt_applies(const PagedAttn& a) {
  return a.fmt != CSA2_KV_FP4 && a.kv.page_shift >= 3 && a.kv.n_pages > 0 && (a.D == 512 || a.D == 256) && a.G >= 32 &&
         (a.window == 0 || static_cast<int64_t>(a.window) + a.sinks >= 512);
}

namespace {

csa2_status launch(const char* fn, const PagedAttn& a, Params& p, dim3 grid, cudaStream_t stream) {
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_token = a.q_token;
  p.q_head = a.q_head;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  const float s = a.scale * kLog2e;
  p.flip = s < 0.0f ? 0x80008000u : 0u;
  p.scale2 = std::max(s < 0.0f ? -s : s, 1.1754944e-38f);
  p.Hq = a.Hq;
  p.G = a.G;
  const int nh = paged_wide_heads(a);
  p.row_tiles = (a.G + nh - 1) / nh;
  p.window = a.window;
  p.sinks = a.sinks;
  p.kv = a.kv;
  const bool sh = a.kv.v == a.kv.k;
  const int page = 1 << a.kv.page_shift;
  p.box = std::min(page, KT);
  CUtensorMap maps[2] = {};
  for (int i = 0; i < (sh ? 1 : 2); ++i)
    CSA2_TRY(make_tensor_map_paged(&maps[i], i ? a.kv.v : a.kv.k, a.D, a.kv.heads, a.kv.head_stride, page,
                                   a.kv.token_stride, a.kv.n_pages, a.kv.page_stride, p.box));
  grid.y = static_cast<unsigned>(a.kv.heads * p.row_tiles);
#define CSA2_WIDE_N(T_, D_, N_) (sh ? run<T_, D_, N_, true>(fn, p, grid, maps, stream) : run<T_, D_, N_, false>(fn, p, grid, maps, stream))
  // rows of 256 channels come here as prompts only, which have more than 16 heads
#define CSA2_WIDE(T_) \
  (a.D == 256 ? CSA2_WIDE_N(T_, 256, 64) : nh == 16 ? CSA2_WIDE_N(T_, 512, 16) : CSA2_WIDE_N(T_, 512, 64))
  return a.fmt == CSA2_KV_F16 ? CSA2_WIDE(__half) : CSA2_WIDE(__nv_bfloat16);
#undef CSA2_WIDE
#undef CSA2_WIDE_N
}

}  // namespace

csa2_status launch_paged_wide(const PagedAttn& a, int chunk, int chunks, float* part_o, float2* part_ml,
                              cudaStream_t stream) {
  Params p = {};
  p.part_o = part_o;
  p.part_ml = part_ml;
  p.chunk = chunk;
  p.chunks = chunks;
  return launch("csa2_paged_decode_attn", a, p, dim3(static_cast<unsigned>(chunks), 1, static_cast<unsigned>(a.kv.B)), stream);
}

csa2_status launch_paged_wide_prompt(const PagedAttn& a, const int32_t* cu_q, int64_t T, cudaStream_t stream) {
  Params p = {};
  p.cu_q = cu_q;
  p.T = static_cast<int>(T);
  p.chunk = KT;
  p.chunks = 1;
  return launch("csa2_paged_window_attn", a, p, dim3(static_cast<unsigned>(T)), stream);
}

}  // namespace csa2
