// Steps 3 and 4 over a paged cache, on tensor cores: shared-KV attention of new
// tokens (groups of up to 128 heads, d = 512, bf16) over every visible entry of
// a cache of any length (dense, HCA) or over the selected entries (kSparse,
// CSA), and the window's raw rows, split over the GPU and joined.
//
//   z_i = scale q.r_i,  o = sum_i e^z_i r_i / (e^sink + sum_i e^z_i)
//
// One pass over the rows with a running maximum and sum per head.  A row is
// 1 KB and takes 4 * 128 * 512 operations: at this machine's copy bandwidth
// and matrix rate both need 0.16 ns a row, so neither may wait for the other.
//
// The output of a token (128 heads x 512 dims in fp32) would fill TMEM, so
// two CTAs share a range of rows, each with half of the output's dims:
//
//   S   = Q K^T           all 512 dims, in BOTH CTAs (M = 128 heads, N = 64)
//   O_c += P V[:, D_c]    the CTA's own 256 dims (N = 256)
//
// Computing S twice costs half as much matrix work again, and the rows are
// read twice from L2 (once from HBM), but the CTAs never wait for each other:
// swapping partial logits, as k_attn_pair does, costs about 1.2 us per 64 rows
// here, more than the second S.  What bounds it: per 64 rows a CTA has 1,790
// clocks of MMAs (16 x 48 with A in shared memory, 16 x 32 with A in TMEM, N =
// 64; 4 x 128, N = 256) and 224 KB through shared memory (1,750 clocks); it
// takes about 2,500.  8 ragged sequences of up to 64K rows (230 MB): 97 to 102 us
// over inputs that the L2 does not hold (116 on one box), 91 replayed on one set
// of them; 16 x 1,152 rows: 21.2 us; 32 x 1,152 selected rows: 26.6 us (42 on
// k_attn_pair with paged rows): about 4 us before the first MMA, 1.35 a tile, 5
// to join the parts.  Chunks of a prompt: 1,024 tokens x 1,152 selected rows 0.46
// to 0.52 ms (618 TFLOP/s), 512 tokens x 16,384 rows 2.4 to 2.9 ms (780 TFLOP/s);
// a pair takes 9 to 14 us to go from a token to the next (Q in, O out).
// Fewer heads cost the same: M is 128 whatever the group holds (16 heads: 16 x
// 1,152 rows 23 to 25 us).
//
// Rotated Q is rounded to bf16, as the operand of the product (half a step is
// 2^-8 of each value, what Q came with).
//
// TMEM (512 columns): O [0,256) | S [256,384) two buffers | Q of the own dims
// as bf16 pairs [384,512).  Q of the other dims stays in shared memory (64
// KB, the A operand from there); P overwrites its S as bf16 pairs.  The rest
// of shared memory is a ring of five slots of 32 KB: 64 rows x 256 dims, a
// tile being two of them (the other half's dims first: they are released
// after S, the own dims' after O).
//
// Warps: 0-3 softmax, one head per thread (= TMEM lane), lazy rescale (a
// head's maximum moves only past 2^8); 4-7 fetch, one 64-dim quarter of each
// slot: a whole tile by TMA, a box per page, a tile with fewer than 64 rows
// (or a page outside the pool) row by row with zeros in the missing ones, so
// that what lies behind the last row is never multiplied; 8 issues the MMAs;
// 9 fetches Q's other half.  Selected entries are fetched by 16-byte cp.async,
// zeros in unused places, their numbers read two tiles ahead and their pages
// one (four rows per TMA gather instruction took 3,800 clocks a tile to issue).
// The first fetching warp leaves each tile's valid rows as a mask for the
// softmax.
//
// Split, few tokens: every token gets the same number of pairs, four to one, in
// one cluster, as many as fit the GPU at once, while none takes more than
// kAdFixedTiles tiles above an even share.  A pair knows its tiles from its own
// token's counts, and the cluster joins its parts: each CTA sends the others
// their share of its dims in fp32, with m and l, into their free rings, and
// finishes its own.  32 x 1,152 selected rows 31.1 -> 26.6 us (two pairs), 16 x
// 1,152 rows 23.1 -> 21.2 us (three) against the ranges below.  The exchange is
// 5 us of it: 2.3 for 64 KB a CTA through distributed shared memory (15 bytes a
// clock), 2.7 to add, turn and write; its two barriers 0.2.
//
// Else all tiles (64 rows; a token's window tiles, then its entries') form one
// sequence.  With no more tokens than CTA pairs each pair takes part of ONE
// token: the fewest tiles L per pair for which sum ceil(tiles / L) fits.
// Where that leaves a pair more than kAdSegTiles tiles above the mean, and
// with more tokens than pairs, the sequence is cut into equal ranges instead,
// and a pair goes from token to token.  A token that one pair holds whole is
// finished there; the others' parts are joined by k_attn_dense_join in their
// order: m and l in fp32, O / l in fp16 under a power-of-two scale per head (11
// bits where the bf16 output keeps 8; half the bytes of fp32, which at 2 parts
// per token is what the join spends its time on).
#pragma once
#include "attn_pair.cuh"
#include "common.cuh"
#include "mxfp4.cuh"
#include "sm100.cuh"

namespace csa {

constexpr int kAdTile = 64;
constexpr int kAdSlots = 5;
constexpr int kAdSlotBytes = 32768;    // 64 rows x 256 dims, or 128 heads x 128 dims of Q
constexpr int kAdChunk = 8192;         // 64 rows x 64 dims
constexpr int kAdQChunk = 16384;       // 128 heads x 64 dims
constexpr int kAdThreads = 320;
// tiles that a prefetch to L2 runs ahead (8 ragged sequences to 64K rows: none
// 94.6 us, 2 tiles 91.4, 4 tiles 92.3, 6 tiles 92.9)
constexpr int kAdAhead = 2;
constexpr int kAdMasks = 8;            // more tiles than the ring lets the fetch run ahead
constexpr int kAdSegTiles = 3;         // tiles above the mean at which equal ranges take over
constexpr int kAdFixedTiles = 6;       // what the device's ranges and the join cost, in tiles
constexpr int kAdMaxPairs = 128;       // units a one-token-per-pair plan may hold
constexpr size_t kAdPartHalfs = 2 * (size_t)kApHeads * kApHalf;  // fp16 values of one part
constexpr int kAdMl = 3 * kApHeads;    // m, l, scale per CTA of a part

struct AttnDenseArgs {
  const __nv_bfloat16* q;
  const int* q_pos;
  const __nv_bfloat16* kv;
  PageMap pm;
  const int* n_cmp;  // dense
  const int* idx;    // sparse: [tokens][topk]
  int topk;
  int n_max;
  const __nv_bfloat16* kv_raw;
  const int* raw_pos0;
  const int* n_raw;
  int raw_max;
  const float* sink;
  int Tq, H, groups, units;  // unit: (token, group of 128 heads)
  int fixed;  // pairs per unit in one cluster, or 0: ranges found on the device
  int window, width, stride, rope_dim;
  int pairs, box_rows;
  float scale_log2;  // |scale| log2(e), above 0
  uint32_t flip;     // sign bits that a negative scale turns in Q
  unsigned long long wait_ns;
  __nv_bfloat16* out;
  __half* part_o;  // [2 pairs][2 halves][32 units of 8 dims][128 heads][8]
  float* part_ml;  // [2 pairs][2 halves][3][128]: m (log2), l, scale
  // what to join: per unit (units <= pairs) its first and last pair, else per
  // pair the unit that starts in it and goes on, and that unit's last pair; a
  // unit that one pair holds has the same first and last (or unit -1)
  int2* desc;
  double freq[kApMaxRope / 2];
};

struct AdMisc {
  float cs[kApMaxRope / 2], sn[kApMaxRope / 2];
  uint64_t full[kAdSlots], empty[kAdSlots];
  uint64_t s_full[2], p_full[2], pv_done[2];
  uint64_t q_full, q_free, q_ready, o_free, mma_drain;
  uint64_t mask_full[kAdMasks];
  uint2 mask[kAdMasks];  // valid rows of the tiles in flight
  uint32_t tmem_base;
  int abort_flag;
  int u0, pre0, g0, g1;  // this pair's first unit, that unit's first tile, its range of tiles
  int total;             // tiles of all units
  int last;              // one token per pair: the last pair of the unit (else -1)
  int tmp[40];
  int tl[kAdMaxPairs];
};

constexpr int kAdQOff = kAdSlots * kAdSlotBytes;
constexpr int kAdMiscOff = kAdQOff + 4 * kAdQChunk;
constexpr size_t kAdSmemBytes = (size_t)kAdMiscOff + sizeof(AdMisc) + 1024;
static_assert(kAdSmemBytes <= 232448, "shared memory budget");

// What a unit reads.
struct AdUnit {
  int token, b, t;
  int n_sel, n_win;
  int raw_row;  // row of kv_raw of the first window row
  int win_tiles, tiles;
};

template <bool kSparse>
__device__ __forceinline__ AdUnit ad_unit(const AttnDenseArgs& a, int u) {
  AdUnit x;
  x.token = u / a.groups;
  x.b = x.token / a.Tq;
  x.t = a.q_pos[x.token];
  x.n_sel = kSparse ? a.topk : max(0, min(n_visible(x.t, a.n_cmp[x.b], a.width, a.stride), a.n_max));
  const int rp0 = a.raw_pos0[x.b];
  const int lo = max(max(0, x.t - a.window + 1), rp0);
  const int hi = min(x.t, rp0 + (min(a.n_raw[x.b], a.raw_max) - 1));
  x.n_win = a.window > 0 && hi >= lo ? hi - lo + 1 : 0;
  x.raw_row = x.b * a.raw_max + (lo - rp0);
  x.win_tiles = (x.n_win + kAdTile - 1) / kAdTile;
  x.tiles = max(1, x.win_tiles + (x.n_sel + kAdTile - 1) / kAdTile);
  return x;
}

// 16 dims of a finished head, times inv: the inverse rotation at -t from dim
// rel = 0 on (all of them or none), bf16.
__device__ __forceinline__ void ad_store16(__nv_bfloat16* dst, int rel, const float (&o)[16], float inv,
                                           const AdMisc& sm, bool live) {
  uint32_t w[8];
  if (rel < 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = ap_bf16x2(o[2 * e] * inv, o[2 * e + 1] * inv);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = sm.cs[(rel >> 1) + e] * inv, s = sm.sn[(rel >> 1) + e] * inv;
      w[e] = ap_bf16x2(o[2 * e] * c + o[2 * e + 1] * s, -o[2 * e] * s + o[2 * e + 1] * c);
    }
  }
  if (live) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <bool kSparse>
__global__ void __launch_bounds__(kAdThreads, 1)
    k_attn_dense(const __grid_constant__ AttnDenseArgs a, const __grid_constant__ CUtensorMap tm_q,
                 const __grid_constant__ CUtensorMap tm_kv,
                 const __grid_constant__ CUtensorMap tm_raw) {
  using namespace sm100;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* q_smem = ring + kAdQOff;
  AdMisc& sm = *reinterpret_cast<AdMisc*>(ring + kAdMiscOff);
  const int part = blockIdx.x & 1, pair = blockIdx.x >> 1;
  // the warp index, known to be the same in all lanes
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int dim0 = part * kApHalf, other0 = kApHalf - dim0;
  const int rope0 = kApDim - a.rope_dim;
  const uint64_t wait_ns = a.wait_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kAdSlots; ++s) {
      mbar_init(&sm.full[s], kSparse ? 128 : 4);  // the fetching lanes / warps
      mbar_init(&sm.empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.q_ready, 128);
    mbar_init(&sm.o_free, 128);
    mbar_init(&sm.mma_drain, 1);
    for (int i = 0; i < kAdMasks; ++i) mbar_init(&sm.mask_full[i], 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (a.fixed > 0) {  // the barriers and TMEM are ready
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  griddep_wait();  // the predecessor's writes are visible
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    // Q, on its way to L2 while the ranges are found (an equal share per CTA,
    // in units of 1 KB)
    const long long rows = (long long)a.units / a.groups * a.H;  // of 512 dims
    const long long r0 = rows * blockIdx.x / gridDim.x, r1 = rows * (blockIdx.x + 1) / gridDim.x;
    for (long long r = r0; r < min(r1, r0 + 64); r += 16)
      prefetch_l2(a.q + r * kApDim, (uint32_t)min(16LL, r1 - r) * kApDim * 2);
  }

  // ---- this pair's range of tiles
  int u, pre, g, g1;
  if (a.fixed > 0) {  // every thread finds it by itself
    u = pair / a.fixed;
    const int n = ad_unit<kSparse>(a, u).tiles;
    pre = 0;
    g = n * (pair % a.fixed) / a.fixed;
    g1 = n * (pair % a.fixed + 1) / a.fixed;
  } else {
    const int per = (a.units + kAdThreads - 1) / kAdThreads;  // units per thread
    const int ua = min(a.units, (int)threadIdx.x * per), ub = min(a.units, ua + per);
    int mine = 0;
    for (int u = ua; u < ub; ++u) {
      const int n = ad_unit<kSparse>(a, u).tiles;
      mine += n;
      if (a.units <= a.pairs) sm.tl[u] = n;
    }
    int total = 0;
    const int inc = block_inclusive_scan(mine, sm.tmp, &total);
    bool one = false;  // one token per pair
    int L = 1;
    if (a.units <= a.pairs) {
      for (int tries = 0; tries < 2; ++tries) {
        const int room = tries == 0 ? a.pairs - a.units / 2 : a.pairs - a.units + 1;
        L = (total + room - 1) / room;
        int need = 0;
        for (int u = lane; u < a.units; u += 32) need += (sm.tl[u] + L - 1) / L;
        if (__reduce_add_sync(0xffffffffu, need) <= a.pairs) break;
      }
      one = L <= total / a.pairs + kAdSegTiles;
    }
    if (threadIdx.x == 0) {
      sm.total = total;
      if (!one) sm.last = -1;
    }
    if (one) {
      if (warp == 0) {
        int at = 0, pre = 0, found = 0;
        for (int u0 = 0; u0 < a.units; u0 += 32) {
          const int u = u0 + lane;
          const int tl = u < a.units ? sm.tl[u] : 0;
          const int cnt = (tl + L - 1) / L;
          int ci = cnt, ti = tl;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int c2 = __shfl_up_sync(0xffffffffu, ci, o), t2 = __shfl_up_sync(0xffffffffu, ti, o);
            if (lane >= o) {
              ci += c2;
              ti += t2;
            }
          }
          const int k = pair - (at + ci - cnt);
          if (k >= 0 && k < cnt) {
            const int base = pre + ti - tl;
            sm.u0 = u;
            sm.pre0 = base;
            const int each = tl / cnt, more = tl - each * cnt;
            sm.g0 = base + k * each + min(k, more);
            sm.g1 = sm.g0 + each + (k < more ? 1 : 0);
            sm.last = pair + cnt - 1 - k;
            found = 1;
          }
          at += __shfl_sync(0xffffffffu, ci, 31);
          pre += __shfl_sync(0xffffffffu, ti, 31);
        }
        if (!__any_sync(0xffffffffu, found) && lane == 0) sm.g0 = sm.g1 = sm.u0 = sm.pre0 = 0;
      }
    } else {
      const int g0 = (int)((long long)total * pair / a.pairs);
      const int g1 = (int)((long long)total * (pair + 1) / a.pairs);
      if (threadIdx.x == 0 && g0 == g1) sm.g0 = sm.g1 = sm.u0 = sm.pre0 = 0;
      if (g0 < g1 && g0 >= inc - mine && g0 < inc) {  // the thread whose units hold tile g0
        int pre = inc - mine, u = ua;
        for (; u < ub; ++u) {
          const int n = ad_unit<kSparse>(a, u).tiles;
          if (g0 < pre + n) break;
          pre += n;
        }
        sm.u0 = u;
        sm.pre0 = pre;
        sm.g0 = g0;
        sm.g1 = g1;
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    g1 = sm.g1;
    u = sm.u0;
    pre = sm.pre0;
    g = sm.g0;
  }
  const uint32_t tmem = sm.tmem_base;
  const uint32_t t_o = tmem, t_s = tmem + 256, t_q = tmem + 384;
  volatile int* abortp = &sm.abort_flag;
  const bool have = g1 > g;  // any tiles
  bool ok = true;
  float m_run = -INFINITY, l_run = 0.f;  // softmax warps: of the segment at hand

  if (warp < 4) {
    // ======================= softmax warps
    const int head = warp * 32 + lane;  // of the unit's group = TMEM lane
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    int item = 0;  // ring items passed
    int gt = 0;    // tiles done, over all segments
    int seg = 0;
    bool joined = false;
    for (; g < g1 && ok; ++seg) {
      const AdUnit x = ad_unit<kSparse>(a, u);
      const int tb = g - pre, te = min(x.tiles, g1 - pre);
      const bool first = tb == 0, whole = first && te == x.tiles;
      // ---- RoPE table, then Q: the own dims to TMEM, the other dims in place
      asm volatile("bar.sync 1, 128;" ::: "memory");  // the last segment's table is done with
      // whole warps, also where rope_dim / 2 ends inside one (frequencies past
      // it are 0): the barrier behind wants them converged
      if (warp < kApMaxRope / 64) {
        float c, s;
        rope_cs_reduced(x.t, a.freq[head], &c, &s);
        sm.cs[head] = c;
        sm.sn[head] = s;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      // 8 dims from d of this thread's head, turned where they rotate (small
      // loops below: code that runs once per token is paid for in instruction
      // fetches)
      auto turn8 = [&](uint4 v, int d) -> uint4 {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if (d >= rope0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = ((d - rope0) >> 1) + e;
            const float c = sm.cs[i], sn = sm.sn[i];
            const float2 f = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w[e]));
            w[e] = ap_bf16x2(f.x * c - f.y * sn, f.x * sn + f.y * c);
          }
        }
        return make_uint4(w[0] ^ a.flip, w[1] ^ a.flip, w[2] ^ a.flip, w[3] ^ a.flip);
      };
      if (seg > 0)  // every QK of the last segment has read Q
        ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.q_free, (uint32_t)(seg - 1) & 1u, abortp, wait_ns));
      tc_fence_after();
#pragma unroll 1
      for (int half = 0; half < 2 && ok; ++half) {
        const int slot = (item + half) % kAdSlots;
        ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.full[slot], (uint32_t)((item + half) / kAdSlots) & 1u,
                                               abortp, wait_ns));
        if (!ok) break;
        const uint8_t* blk = ring + slot * kAdSlotBytes;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = *reinterpret_cast<const uint4*>(blk + c * kAdQChunk + ap_swz(head, k));
          const int d = dim0 + half * 128 + c * 64;
          if (d + 64 > rope0 || a.flip != 0u) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = turn8(v[k], d + k * 8);
          }
          uint32_t r[16];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              r[4 * k] = v[4 * h + k].x;
              r[4 * k + 1] = v[4 * h + k].y;
              r[4 * k + 2] = v[4 * h + k].z;
              r[4 * k + 3] = v[4 * h + k].w;
            }
            tmem_st16(t_q + lane_base + (uint32_t)(half * 64 + c * 32 + h * 16), r);
          }
        }
      }
      if (ok && (a.flip != 0u || (other0 + kApHalf > rope0 && a.rope_dim > 0))) {
        ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.q_full, (uint32_t)seg & 1u, abortp, wait_ns));
        if (ok) {
          const int k0 = a.flip != 0u ? 0 : max(0, rope0 - other0) >> 3;
#pragma unroll 1
          for (int k = k0; k < 32; k += 4) {  // (rope0 is a multiple of 32)
            uint4 v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = *reinterpret_cast<const uint4*>(q_smem + (k >> 3) * kAdQChunk + ap_swz(head, (k & 7) + e));
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(q_smem + (k >> 3) * kAdQChunk + ap_swz(head, (k & 7) + e)) =
                  turn8(v[e], other0 + (k + e) * 8);
          }
        }
      }
      tmem_wait_st();
      fence_proxy_async_shared();
      tc_fence_before();
      ok = ap_softmax_all(ok);  // all have read the Q slots
      if (!ok) break;
      if (threadIdx.x == 0) {
        mbar_arrive(&sm.empty[item % kAdSlots]);
        mbar_arrive(&sm.empty[(item + 1) % kAdSlots]);
      }
      mbar_arrive(&sm.q_ready);
      item += 2 + 2 * (te - tb);

      // ---- the tiles
      m_run = -INFINITY;
      l_run = 0.f;
      const int gt0 = gt;
      for (int i = tb; i < te; ++i, ++gt) {
        const int sb = gt & 1;
        ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.s_full[sb], (uint32_t)(gt >> 1) & 1u, abortp, wait_ns));
        ok = ok && __all_sync(0xffffffffu, mbar_wait_fast(&sm.mask_full[gt % kAdMasks],
                                                          (uint32_t)(gt / kAdMasks) & 1u, abortp, wait_ns));
        if (!ok) break;
        tc_fence_after();
        const uint2 vm = sm.mask[gt % kAdMasks];
        float z[64];  // q.k, not scaled
        {
          uint32_t ra[32], rb[32];
          tmem_ld32(t_s + lane_base + (uint32_t)(sb * 64), ra);
          tmem_ld32(t_s + lane_base + (uint32_t)(sb * 64 + 32), rb);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            z[e] = __uint_as_float(ra[e]);
            z[32 + e] = __uint_as_float(rb[e]);
          }
        }
        if ((vm.x & vm.y) != 0xffffffffu) {
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (!((vm.x >> e) & 1u)) z[e] = -INFINITY;
            if (!((vm.y >> e) & 1u)) z[32 + e] = -INFINITY;
          }
        }
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = z[k];
#pragma unroll
        for (int e = 8; e < 64; ++e) mx[e & 7] = fmaxf(mx[e & 7], z[e]);
        const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                               fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * a.scale_log2;
        const bool move = mt > m_run + kApRescaleLog2 || m_run == -INFINITY;
        const float m_new = move ? mt : m_run;
        if (gt > gt0 && __any_sync(0xffffffffu, move && m_run != -INFINITY)) {
          // O holds P V of earlier tiles: wait for the last one, then rescale
          ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.pv_done[(gt - 1) & 1], (uint32_t)((gt - 1) >> 1) & 1u,
                                                 abortp, wait_ns));
          if (!ok) break;
          tc_fence_after();
          const float alpha = (move && m_run != -INFINITY) ? exp2f(m_run - m_new) : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < kApHalf; cc += 32) {
            uint32_t r[32], w16[16];
            tmem_ld32(t_o + lane_base + (uint32_t)cc, r);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) w16[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st16(t_o + lane_base + (uint32_t)cc, w16);
#pragma unroll
            for (int e = 0; e < 16; ++e) w16[e] = __float_as_uint(__uint_as_float(r[16 + e]) * alpha);
            tmem_st16(t_o + lane_base + (uint32_t)cc + 16, w16);
          }
          l_run *= alpha;
        }
        m_run = m_new;
        uint32_t pk[32];
        float ps8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) ps8[k] = 0.f;
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          // the sum in fp32; P in bf16, the operand of the product (half a step
          // is 2^-8 of each weight; the output keeps as many bits)
          const float p0 = ap_ex2(fmaf(z[2 * e], a.scale_log2, neg_m));
          const float p1 = ap_ex2(fmaf(z[2 * e + 1], a.scale_log2, neg_m));
          ps8[e & 7] += p0 + p1;
          pk[e] = ap_bf16x2(p0, p1);
        }
        l_run += ((ps8[0] + ps8[1]) + (ps8[2] + ps8[3])) + ((ps8[4] + ps8[5]) + (ps8[6] + ps8[7]));
        uint32_t w16[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) w16[e] = pk[e];
        tmem_st16(t_s + lane_base + (uint32_t)(sb * 64), w16);
#pragma unroll
        for (int e = 0; e < 16; ++e) w16[e] = pk[16 + e];
        tmem_st16(t_s + lane_base + (uint32_t)(sb * 64 + 16), w16);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sm.p_full[sb]);
      }
      // ---- epilogue
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.pv_done[(gt - 1) & 1], (uint32_t)((gt - 1) >> 1) & 1u,
                                               abortp, wait_ns));
      ok = ap_softmax_all(ok);
      if (!ok) break;
      if (a.fixed > 1) break;  // joined below
      tc_fence_after();
      const int h = (u % a.groups) * kApHeads + head;  // head of the token
      const bool live = h < a.H;
      if (whole) {
        const float sink_l2 = live ? a.sink[h] * 1.4426950408889634f : 0.f;
        const float mm = fmaxf(m_run, sink_l2);
        const float wm = m_run == -INFINITY ? 0.f : exp2f(m_run - mm);
        const float den = l_run * wm + (sink_l2 == -INFINITY ? 0.f : exp2f(sink_l2 - mm));
        const float scl = den > 0.f || den != den ? wm / den : 0.f;
        __nv_bfloat16* orow = a.out + ((size_t)x.token * a.H + (live ? h : 0)) * kApDim + dim0;
#pragma unroll 1
        for (int d = 0; d < kApHalf; d += 16) {
          uint32_t r[2][8];
          tmem_ld8(t_o + lane_base + (uint32_t)d, r[0]);
          tmem_ld8(t_o + lane_base + (uint32_t)d + 8, r[1]);
          tmem_wait_ld8(r[0], r[1]);
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __uint_as_float(r[e >> 3][e & 7]);
          ad_store16(orow + d, dim0 + d - rope0, o, scl, sm, live);
        }
      } else {
        // a part: O / l times a power of two that puts the head's largest
        // value in [2^14, 2^15), in fp16 (11 bits where the output keeps 8)
        const size_t part_i = ((size_t)(2 * pair + (first ? 1 : 0)) * 2 + part);
        const float inv_l = l_run > 0.f ? 1.f / l_run : (l_run != l_run ? l_run : 0.f);
        float top = 0.f;
#pragma unroll 1
        for (int sl = 0; sl < 8; ++sl) {
          uint32_t r[32];
          tmem_ld32(t_o + lane_base + (uint32_t)(sl * 32), r);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) top = fmaxf(top, fabsf(__uint_as_float(r[e]) * inv_l));
        }
        const int field = (int)(__float_as_uint(top) >> 23);
        const int up = field == 0 || field == 255 ? 0 : max(-100, min(100, 127 + 14 - field));
        const float scl = __uint_as_float((uint32_t)(127 + up) << 23);
        float* pml = a.part_ml + part_i * kAdMl;
        pml[head] = m_run;
        pml[kApHeads + head] = l_run;
        pml[2 * kApHeads + head] = __uint_as_float((uint32_t)(127 - up) << 23);
        const float mul = inv_l * scl;
        uint4* po = reinterpret_cast<uint4*>(a.part_o + part_i * (kAdPartHalfs / 2)) + head;
#pragma unroll 1
        for (int sl = 0; sl < 8; ++sl) {
          uint32_t r[32];
          tmem_ld32(t_o + lane_base + (uint32_t)(sl * 32), r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t hv[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 v = __floats2half2_rn(__uint_as_float(r[8 * k + 2 * e]) * mul,
                                                  __uint_as_float(r[8 * k + 2 * e + 1]) * mul);
              hv[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            po[(sl * 4 + k) * kApHeads] = make_uint4(hv[0], hv[1], hv[2], hv[3]);
          }
        }
      }
      tc_fence_before();
      mbar_arrive(&sm.o_free);
      // the join's work list: the pair that holds a unit's first tile writes it
      if (a.fixed == 0 && first && part == 0 && threadIdx.x == 0) {
        // the pair of the unit's last tile: the largest p with total p / pairs <= that tile
        const int last = sm.last >= 0 ? sm.last
                                      : (int)(((long long)(pre + x.tiles) * a.pairs - 1) / sm.total);
        if (a.units <= a.pairs) {
          a.desc[u] = make_int2(pair, last);
        } else if (!whole) {
          a.desc[pair] = make_int2(u, last);
          joined = true;
        }
      }
      g = pre + te;
      pre += x.tiles;
      ++u;
    }
    if (a.units > a.pairs && part == 0 && threadIdx.x == 0 && !joined) a.desc[pair] = make_int2(-1, -1);
  } else if (warp < 8) {
    // ======================= fetching warps: 64-dim quarter q of each slot
    const int q = warp - 4;
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_kv);
      tma_prefetch_desc(&tm_raw);
    }
    int item = 0, gt = 0;
    auto claim = [&](int n) -> bool {
      bool r = true;
      if (lane == 0)
        r = mbar_wait_fast(&sm.empty[n % kAdSlots], ((uint32_t)(n / kAdSlots) & 1u) ^ 1u, abortp, wait_ns);
      return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
    };
    const int subs = kAdTile / a.box_rows;
    while (g < g1 && ok) {
      const AdUnit x = ad_unit<kSparse>(a, u);
      const int tb = g - pre, te = min(x.tiles, g1 - pre);
      // Q's own dims: two slots of 128 heads x 128 dims
      for (int half = 0; half < 2; ++half, ++item) {
        ok = claim(item);
        if (!ok) break;
        const int slot = item % kAdSlots;
        if (lane == 0 && q < 2) {
          mbar_arrive_expect_tx(&sm.full[slot], kAdQChunk);
          tma_load_2d(ring + slot * kAdSlotBytes + q * kAdQChunk, &tm_q, &sm.full[slot],
                      dim0 + half * 128 + q * 64, x.token * a.H + (u % a.groups) * kApHeads);
        } else if (kSparse || lane == 0) {
          mbar_arrive(&sm.full[slot]);
        }
      }
      // selected entries: lane l < 16 has rows 4 l + c of a tile; entry numbers
      // are read two tiles ahead, their table entries one
      const int* sel = kSparse ? a.idx + (long long)x.token * a.topk : nullptr;
      auto load_idx = [&](int i, int (&ix)[4]) {
        const int e = (i - x.win_tiles) * kAdTile + 4 * lane;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          ix[c] = i >= x.win_tiles && i < te && lane < 16 && e + c < a.topk ? sel[e + c] : -1;
      };
      auto load_pages = [&](const int (&ix)[4], int (&pg)[4]) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          pg[c] = ix[c] >= 0 && ix[c] < a.n_max
                      ? a.pm.table[(long long)x.b * a.pm.width + (ix[c] >> a.pm.shift)] : -1;
      };
      int ix0[4], ix1[4], ix2[4], pg0[4], pg1[4];
      // dense: the page table by windows, so that a whole tile waits for no load
      PageWindow pw;
      if (!kSparse && x.n_sel > 0) pw.start(a.pm, x.b, x.n_sel, max(0, tb - x.win_tiles) * kAdTile >> a.pm.shift);
      if (kSparse) {
        load_idx(tb, ix0);
        load_idx(tb + 1, ix1);
        load_pages(ix0, pg0);
      }
      for (int i = tb; i < te && ok; ++i, ++gt) {
        const bool win = i < x.win_tiles;
        const int j0 = (i - x.win_tiles) * kAdTile;
        const int cnt = win ? x.n_win - i * kAdTile : x.n_sel - j0;
        long long box = -1;           // boxes of a whole tile, one lane each
        bool whole = false;
        uint2 vm;
        int rowk[16];                 // kSparse: rows 4 k + lane / 8, -1 where none
        if (kSparse && !win) {
          load_pages(ix1, pg1);
          load_idx(i + 2, ix2);
          uint32_t nib = 0;
          int rows[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const bool in = (unsigned)pg0[c] < (unsigned)a.pm.n_pages;  // -1 where unused
            if (!in && ix0[c] >= 0 && q == 0) report_error(CSA_ERR_DEVICE_BOUNDS);
            rows[c] = in ? (pg0[c] << a.pm.shift) + (ix0[c] & ((1 << a.pm.shift) - 1)) : -1;
            nib |= in ? 1u << c : 0u;
            ix0[c] = ix1[c];
            ix1[c] = ix2[c];
            pg0[c] = pg1[c];
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int r0 = __shfl_sync(0xffffffffu, rows[0], k), r1 = __shfl_sync(0xffffffffu, rows[1], k);
            const int r2 = __shfl_sync(0xffffffffu, rows[2], k), r3 = __shfl_sync(0xffffffffu, rows[3], k);
            rowk[k] = lane < 16 ? (lane < 8 ? r0 : r1) : (lane < 24 ? r2 : r3);
          }
          vm.x = __reduce_or_sync(0xffffffffu, lane < 8 ? nib << (4 * lane) : 0u);
          vm.y = __reduce_or_sync(0xffffffffu, lane >= 8 && lane < 16 ? nib << (4 * (lane - 8)) : 0u);
        } else {
          if (kSparse) {  // keep the look-ahead moving through the window's tiles
            load_pages(ix1, pg1);
            load_idx(i + 2, ix2);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              ix0[c] = ix1[c];
              ix1[c] = ix2[c];
              pg0[c] = pg1[c];
            }
          }
          whole = cnt >= kAdTile;
          if (whole) {
            if (win)
              box = lane == 0 ? (long long)x.raw_row + (long long)i * kAdTile : -1;
            else {
              pw.seek(j0 >> a.pm.shift);
              const int j = j0 + lane * a.box_rows;
              const int pg = pw.at(j >> a.pm.shift);
              if (lane < subs && (unsigned)pg < (unsigned)a.pm.n_pages)
                box = ((long long)pg << a.pm.shift) + (j & ((1 << a.pm.shift) - 1));
              // a tile a few ahead on its way to L2, by one of the pair's CTAs in
              // turn (within the window of the table at hand)
              const int ja = j + kAdAhead * kAdTile;
              if (q == 0 && ((i ^ part) & 1) == 0 &&
                  (j0 + kAdAhead * kAdTile) >> (a.pm.shift + 5) == pw.w) {
                const int pa = pw.at(ja >> a.pm.shift);
                if (lane < subs && ja < x.n_sel && i + kAdAhead < te &&
                    (unsigned)pa < (unsigned)a.pm.n_pages)
                  prefetch_l2(a.kv + (((long long)pa << a.pm.shift) +
                                      (ja & ((1 << a.pm.shift) - 1))) * kApDim,
                              (uint32_t)a.box_rows * kApDim * 2);
              }
            }
            whole = __popc(__ballot_sync(0xffffffffu, box >= 0)) == (win ? 1 : subs);
          }
          vm = make_uint2(0xffffffffu, 0xffffffffu);
          if (!whole) {
            const bool r0 = lane < cnt && (win || page_row(a.pm, x.b, a.n_max, j0 + lane) >= 0);
            const bool r1 = lane + 32 < cnt && (win || page_row(a.pm, x.b, a.n_max, j0 + lane + 32) >= 0);
            vm.x = __ballot_sync(0xffffffffu, r0);
            vm.y = __ballot_sync(0xffffffffu, r1);
            if (kSparse) {
#pragma unroll
              for (int k = 0; k < 16; ++k)
                rowk[k] = 4 * k + (lane >> 3) < cnt ? x.raw_row + i * kAdTile + 4 * k + (lane >> 3) : -1;
            }
          }
        }
        if (q == 0 && lane == 0) {
          sm.mask[gt % kAdMasks] = vm;
          mbar_arrive(&sm.mask_full[gt % kAdMasks]);
        }
#pragma unroll 1
        for (int half = 0; half < 2; ++half, ++item) {
          ok = claim(item);
          if (!ok) break;
          const int slot = item % kAdSlots;
          const int d0 = (half == 0 ? other0 : dim0) + q * 64;
          uint8_t* dst = ring + slot * kAdSlotBytes + q * kAdChunk;
          const int un = lane & 7;
          const uint32_t base = smem_u32(dst);
          if (kSparse && !whole) {
            // lane l copies 16-byte unit l % 8 of rows 4k + l / 8
            const __nv_bfloat16* src = (win ? a.kv_raw : a.kv) + d0 + un * 8;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int r = 4 * k + (lane >> 3);
              cp_async16(base + (uint32_t)(r * 128 + ((un ^ (r & 7)) << 4)),
                         src + (long long)max(rowk[k], 0) * kApDim, rowk[k] >= 0);
            }
            cp_async_arrive(&sm.full[slot]);
          } else if (whole) {
            if (lane == 0)
              mbar_arrive_expect_tx(&sm.full[slot], kAdChunk);
            else if (kSparse)
              mbar_arrive(&sm.full[slot]);
            __syncwarp();
            if (box >= 0)
              tma_load_2d(dst + (win ? 0 : lane * a.box_rows * 128), win ? &tm_raw : &tm_kv,
                          &sm.full[slot], d0, (int)box);
          } else {
            // row by row
#pragma unroll 4
            for (int k = 0; k < 16; ++k) {
              const int r = 4 * k + (lane >> 3);
              const bool in = ((r < 32 ? vm.x : vm.y) >> (r & 31)) & 1u;
              const __nv_bfloat16* src = a.out;  // not read
              if (in)
                src = (win ? a.kv_raw + ((long long)x.raw_row + (long long)i * kAdTile + r) * kApDim
                           : a.kv + page_row(a.pm, x.b, a.n_max, j0 + r) * kApDim) + d0 + un * 8;
              else if (!win && r < cnt && half == 0 && q == 0 && un == 0)
                report_error(CSA_ERR_DEVICE_BOUNDS);
              cp_async16(base + (uint32_t)(r * 128 + ((un ^ (r & 7)) << 4)), src, in);
            }
            cp_async_wait_all();
            fence_proxy_async_shared();  // read by the MMA (async proxy)
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.full[slot]);
          }
        }
      }
      g = pre + te;
      pre += x.tiles;
      ++u;
    }
    // every copy into shared memory lands before the CTA may exit (the last
    // one asked of each slot; an earlier one was used before it)
    cp_async_wait_all();
    __syncwarp();
    if (lane == 0)
      for (int n = max(0, item - kAdSlots); n < item; ++n)
        mbar_drain(&sm.full[n % kAdSlots], (uint32_t)(n / kAdSlots) & 1u, kApDrainNs);
  } else if (warp == 8) {
    // ======================= MMA issuer (the whole warp runs the loop, one
    // elected lane issues)
    constexpr uint32_t id_qk = idesc_bf16_f32(128, kAdTile);
    constexpr uint32_t id_pv = idesc_bf16_f32(128, kApHalf, 0, 1);
    const uint32_t ring_a = smem_u32(ring);
    const uint64_t a0 = sw128_desc(ring_a + kAdQOff, 16, 1024);
    auto wait = [&](uint64_t* bar, int phase) {
      return __all_sync(0xffffffffu, mbar_wait_fast(bar, (uint32_t)phase & 1u, abortp, wait_ns)) != 0;
    };
    int item = 0, gt = 0;
    for (int seg = 0; g < g1 && ok; ++seg) {
      const AdUnit x = ad_unit<kSparse>(a, u);
      const int n = min(x.tiles, g1 - pre) - (g - pre);
      item += 2;  // Q's own dims
      ok = wait(&sm.q_full, seg) &&
           __all_sync(0xffffffffu, mbar_wait_strict(&sm.q_ready, (uint32_t)seg & 1u, abortp, wait_ns));
      for (int i = 0; i <= n && ok; ++i) {
        if (i < n) {  // S(i) = Q K^T
          const uint32_t d = t_s + (uint32_t)(((gt + i) & 1) * 64);
          const int i0 = item + 2 * i, s0 = i0 % kAdSlots, s1 = (i0 + 1) % kAdSlots;
          ok = wait(&sm.full[s0], i0 / kAdSlots);
          if (!ok) break;
          if (kSparse) fence_proxy_async_shared();  // written by cp.async (generic proxy)
          tc_fence_after();
          const uint64_t b0 = sw128_desc(ring_a + s0 * kAdSlotBytes, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 16; ++ks)
              mma_ss(d, a0 + (uint64_t)(((ks >> 2) * kAdQChunk + (ks & 3) * 32) >> 4),
                     b0 + (uint64_t)(((ks >> 2) * kAdChunk + (ks & 3) * 32) >> 4), id_qk, ks != 0);
            tc_commit(&sm.empty[s0]);
          }
          __syncwarp();
          ok = wait(&sm.full[s1], (i0 + 1) / kAdSlots);
          if (!ok) break;
          if (kSparse) fence_proxy_async_shared();
          tc_fence_after();
          const uint64_t b1 = sw128_desc(ring_a + s1 * kAdSlotBytes, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 16; ++ks)
              mma_ts(d, t_q + (uint32_t)((ks >> 2) * 32 + (ks & 3) * 8),
                     b1 + (uint64_t)(((ks >> 2) * kAdChunk + (ks & 3) * 32) >> 4), id_qk, 1u);
            tc_commit(&sm.s_full[(gt + i) & 1]);
            if (i == n - 1) tc_commit(&sm.q_free);
          }
          __syncwarp();
        }
        if (i > 0) {  // O += P(i - 1) V
          const int j = gt + i - 1, sb = j & 1;
          if (i == 1 && seg > 0) ok = wait(&sm.o_free, seg - 1);  // the last segment's O has been read
          ok = ok && wait(&sm.p_full[sb], j >> 1);
          if (!ok) break;
          tc_fence_after();
          const int s1 = (item + 2 * (i - 1) + 1) % kAdSlots;
          const uint64_t v0 = sw128_desc(ring_a + s1 * kAdSlotBytes, kAdChunk, 1024);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < kAdTile / 16; ++ks)
              mma_ts(t_o, t_s + (uint32_t)(sb * 64 + ks * 8), v0 + (uint64_t)((ks * 16 * 128) >> 4), id_pv,
                     (i > 1 || ks > 0) ? 1u : 0u);
            tc_commit(&sm.empty[s1]);
            tc_commit(&sm.pv_done[sb]);
          }
          __syncwarp();
        }
      }
      item += 2 * n;
      gt += n;
      g += n;
      pre += x.tiles;
      ++u;
    }
    // TMEM is freed only after every MMA issued here has landed
    if (elect_one()) {
      tc_commit(&sm.mma_drain);
      mbar_drain(&sm.mma_drain, 0, kApDrainNs);
    }
    __syncwarp();
  } else {
    // ======================= warp 9: Q's other half
    if (lane == 0) {
      int seg = 0, sent = 0;
      for (; g < g1 && ok; ++seg) {
        const AdUnit x = ad_unit<kSparse>(a, u);
        if (seg > 0) ok = mbar_wait_fast(&sm.q_free, (uint32_t)(seg - 1) & 1u, abortp, wait_ns);
        if (!ok) break;
        mbar_arrive_expect_tx(&sm.q_full, 4 * kAdQChunk);
        for (int c = 0; c < 4; ++c)
          tma_load_2d(q_smem + c * kAdQChunk, &tm_q, &sm.q_full, other0 + c * 64,
                      x.token * a.H + (u % a.groups) * kApHeads);
        sent = seg + 1;
        g = pre + min(x.tiles, g1 - pre);
        pre += x.tiles;
        ++u;
      }
      if (sent > 0) mbar_drain(&sm.q_full, (uint32_t)(sent - 1) & 1u, kApDrainNs);
    }
  }
  __syncwarp();
  tc_fence_before();
  if (a.fixed > 1) {
    // The unit's pairs are a cluster: each hands the others their share of its
    // dims, in fp32 and unscaled, with m and l, and finishes its own share.
    // Warps w and w + 4 read the same TMEM lanes and take every other 16 dims.
    // (Small loops: this runs once, and its instructions are fetched as it goes.)
    const int P = a.fixed, k = pair % P, unit = pair / P, head = (warp & 3) * 32 + lane, first = warp >> 2;
    const int h = (unit % a.groups) * kApHeads + head;
    const bool live = h < a.H && warp < 8;
    const float sink_l2 = live ? a.sink[h] * 1.4426950408889634f : 0.f;
    const uint32_t t_head = t_o + ((uint32_t)((warp & 3) * 32) << 16);
    auto share = [&](int r) { return kApHalf / 32 * r / P * 32; };  // first dim of pair r's share
    const int piece = kApHeads * 4 * 32 * ((kApHalf / 32 + P - 1) / P);
    uint8_t* ml = ring + (P - 1) * piece + head * 8;  // + slot * 1 KB
    // a pair without tiles says so by l = -1
    if (warp < kApMaxRope / 64 && !have)
      rope_cs_reduced(a.q_pos[unit / a.groups], a.freq[head], &sm.cs[head], &sm.sn[head]);
    cluster_sync_all();  // the rings are free: every copy and product is done
    tc_fence_after();
    if (warp < 8) {
#pragma unroll 1
      for (int j = 0; j < P; ++j) {
        const int r = (k + 1 + j) % P;  // its slot j is this pair's; slot P - 1 this pair's own
        if (have && j < P - 1) {
          const int d1 = share(r + 1);
          int d = share(r) + first * 16;
          uint32_t dst = mapa(ring + j * piece, (uint32_t)(2 * r + part)) + (uint32_t)(first * 4 * kApHeads + head) * 16;
#pragma unroll 1
          for (; d < d1; d += 32, dst += 8 * kApHeads * 16) {
            uint32_t v[2][8];
            tmem_ld8(t_head + (uint32_t)d, v[0]);
            tmem_ld8(t_head + (uint32_t)d + 8, v[1]);
            tmem_wait_ld8(v[0], v[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              st_cluster_v4(dst + (uint32_t)(e * kApHeads * 16),
                            make_uint4(v[e >> 1][4 * (e & 1)], v[e >> 1][4 * (e & 1) + 1],
                                       v[e >> 1][4 * (e & 1) + 2], v[e >> 1][4 * (e & 1) + 3]));
          }
        }
        if (first == 0)
          st_cluster_v2(mapa(ml + j * kApHeads * 8, (uint32_t)(2 * r + part)), __float_as_uint(m_run),
                        __float_as_uint(have ? l_run : -1.f));
      }
    }
    __syncwarp();
    cluster_sync_all();  // the shares are here; nobody writes into a CTA that has left
    if (warp < 8) {
      float M = sink_l2;
#pragma unroll 1
      for (int j = 0; j < P; ++j) M = fmaxf(M, *reinterpret_cast<const float*>(ml + j * kApHeads * 8));
      M = M == -INFINITY ? 0.f : M;
      float L = ap_ex2(sink_l2 - M), w_own = 0.f;
#pragma unroll 1
      for (int j = 0; j < P; ++j) {
        const float2 x = *reinterpret_cast<const float2*>(ml + j * kApHeads * 8);
        w_own = ap_ex2(x.x - M);  // (slot P - 1 comes last)
        if (!(x.y < 0.f)) L = fmaf(x.y, w_own, L);
      }
      const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
      const int d1 = share(k + 1);
      int d = share(k) + first * 16;
      __nv_bfloat16* dst = a.out + ((size_t)(unit / a.groups) * a.H + (live ? h : 0)) * kApDim + dim0;
      const uint8_t* got = ring + (first * 4 * kApHeads + head) * 16;
#pragma unroll 1
      for (; d < d1; d += 32, got += 8 * kApHeads * 16) {
        float o[16];
        uint32_t v[2][8];
        if (have) {
          tmem_ld8(t_head + (uint32_t)d, v[0]);
          tmem_ld8(t_head + (uint32_t)d + 8, v[1]);
          tmem_wait_ld8(v[0], v[1]);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] = have ? __uint_as_float(v[e >> 3][e & 7]) * w_own : 0.f;
#pragma unroll 1
        for (int j = 0; j < P - 1; ++j) {
          const float2 x = *reinterpret_cast<const float2*>(ml + j * kApHeads * 8);
          if (x.y < 0.f) continue;  // nothing was sent
          const float w = ap_ex2(x.x - M);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 y = *reinterpret_cast<const float4*>(got + j * piece + e * kApHeads * 16);
            o[4 * e] = fmaf(y.x, w, o[4 * e]);
            o[4 * e + 1] = fmaf(y.y, w, o[4 * e + 1]);
            o[4 * e + 2] = fmaf(y.z, w, o[4 * e + 2]);
            o[4 * e + 3] = fmaf(y.w, w, o[4 * e + 3]);
          }
        }
        ad_store16(dst + d, dim0 + d - rope0, o, inv, sm, live);
      }
    }
    __syncwarp();
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a unit that more than one pair holds:
//   M = max(sink, max m_s),  L = 2^(sink - M) + sum l_s 2^(m_s - M)
//   o = sum (l_s 2^(m_s - M) / L) O_s
// A thread takes 16 dims of a head and every K-th part; K lanes share a head and
// join their states by shuffles, all in a fixed order.  K is the largest at
// which the threads are resident at once (a second wave costs as much as the
// first).  No shared memory, so that CTAs can be resident while the attention
// kernel ends (it leaves 1 KB).
template <int K>
__global__ void __launch_bounds__(128, 8) k_attn_dense_join(const __grid_constant__ AttnDenseArgs a) {
  constexpr int kHeads = 128 / K;  // per CTA
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k = lane / (32 / K), step = K;
  const int slab = (int)blockIdx.x / K;  // 16 dims
  const int head = (int)blockIdx.x % K * kHeads + warp * (32 / K) + lane % (32 / K);
  const int half = slab >> 4, u8 = (slab & 15) * 2;  // two units of 8 dims
  const int d0 = half * kApHalf + u8 * 8;
  const int rope0 = kApDim - a.rope_dim;
  const bool by_unit = a.units <= a.pairs;
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int2 ds = __ldcg(a.desc + blockIdx.y);
  const int unit = by_unit ? (int)blockIdx.y : ds.x;
  const int pair0 = by_unit ? ds.x : (int)blockIdx.y;
  // (a launch that gave up may have written no list)
  if (unit < 0 || unit >= a.units) return;
  const int token = unit / a.groups, h = (unit % a.groups) * kApHeads + head;
  const bool live = h < a.H;
  const float sink_l2 = live ? a.sink[h] * 1.4426950408889634f : 0.f;
  const int t = a.q_pos[token];
  if (pair0 < 0 || ds.y <= pair0 || ds.y >= a.pairs) return;  // nothing to join
  const int n = ds.y - pair0 + 1;
  float m = -INFINITY, L = 0.f, o[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.f;
  for (int s0 = k; s0 < n; s0 += 2 * step) {
    float ms[2], ls[2], sc[2];
    uint4 v[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int s = s0 + i * step;
      ms[i] = -INFINITY;
      ls[i] = sc[i] = 0.f;
      v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (s < n) {
        const size_t pi = (size_t)(2 * (pair0 + s) + (s == 0 ? 1 : 0)) * 2 + half;
        const float* ml = a.part_ml + pi * kAdMl + head;
        const uint4* po = reinterpret_cast<const uint4*>(a.part_o + pi * (kAdPartHalfs / 2)) + u8 * kApHeads + head;
        ms[i] = __ldcg(ml);
        ls[i] = __ldcg(ml + kApHeads);
        sc[i] = __ldcg(ml + 2 * kApHeads);
        v[i][0] = __ldcg(po);
        v[i][1] = __ldcg(po + kApHeads);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float mn = fmaxf(m, ms[i]);
      const float old = m == -INFINITY ? 0.f : exp2f(m - mn);
      const float w = ms[i] == -INFINITY ? 0.f : ls[i] * exp2f(ms[i] - mn);
      m = mn;
      L = fmaf(L, old, w);
      const float ws = w * sc[i];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t hv[4] = {v[i][g].x, v[i][g].y, v[i][g].z, v[i][g].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = ap_f16x2_to_f32(hv[e]);
          o[8 * g + 2 * e] = fmaf(f.x, ws, o[8 * g + 2 * e] * old);
          o[8 * g + 2 * e + 1] = fmaf(f.y, ws, o[8 * g + 2 * e + 1] * old);
        }
      }
    }
  }
  // the head's lanes, and the sink
  float M = m;
#pragma unroll
  for (int x = 32 / K; x < 32; x <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
  M = fmaxf(M, sink_l2);
  const float f = m == -INFINITY ? 0.f : exp2f(m - M);
  L *= f;
#pragma unroll
  for (int x = 32 / K; x < 32; x <<= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
  L += sink_l2 == -INFINITY ? 0.f : exp2f(sink_l2 - M);
  const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
  // lane k finishes 16 / K of the dims: the inverse rotation at -t, bf16
  constexpr int kMine = 16 / K;
  float y[kMine];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float v = o[e] * f;
#pragma unroll
    for (int x = 32 / K; x < 32; x <<= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
    if (e / kMine == k) y[e % kMine] = v * inv;
  }
  const int dm = d0 + kMine * k;
#pragma unroll
  for (int e = 0; e < kMine; e += 2) {
    if (dm + e >= rope0) {
      float c, s;
      rope_cs_reduced(t, a.freq[(dm + e - rope0) >> 1], &c, &s);
      const float x0 = y[e], x1 = y[e + 1];
      y[e] = x0 * c + x1 * s;
      y[e + 1] = -x0 * s + x1 * c;
    }
  }
  if (!live) return;
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + ((size_t)token * a.H + h) * kApDim + dm);
  uint32_t w[kMine / 2];
#pragma unroll
  for (int e = 0; e < kMine / 2; ++e) w[e] = ap_bf16x2(y[2 * e], y[2 * e + 1]);
  if (K == 8)
    dst[0] = w[0];
  else if (K == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[kMine / 2 - 1]);
  else
#pragma unroll
    for (int e = 0; e < kMine / 2; e += 4)
      *reinterpret_cast<uint4*>(dst + e) = make_uint4(w[e], w[(e + 1) % (kMine / 2)], w[(e + 2) % (kMine / 2)],
                                                      w[(e + 3) % (kMine / 2)]);
}

}  // namespace csa
