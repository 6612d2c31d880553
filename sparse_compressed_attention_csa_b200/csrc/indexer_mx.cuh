// Step 2a on 4-bit tensor cores: lightning-indexer scores of MXFP4 queries
// (64 heads x 128 dims) and paged MXFP4 keys.
//
//   D[key][h] = sum_c q[h][c] k[key][c]     (tcgen05 kind::mxf4: E2M1 operands,
//               one E8M0 scale per 32 dims, fp32 in TMEM)
//   s[key]    = sum_h w[h] max(0, D[key][h])
//
// A tile is 256 keys, two MMAs' M of 128; a step is one tile and one query
// token, N = 64 heads; the 128 dims are two K steps of 64.  A key is 64 B of
// codes and 4 B of scales: decode streams 68 B per key where the bf16 indexer
// streams 256, and is bound by latency and by HBM; a prefill is bound by the
// epilogue's CUDA-core work, one maximum and half a packed multiply-add per
// key, token and head.  A thread scores two keys (lane l of both halves of the
// tile) at a time, so that a head's weight, read from shared memory by every
// thread, serves twice.
//
// Roles: warps 0 and 4 + 4 PAR fetch the codes of every second tile by TMA,
// one box per page (64-byte swizzle), and their scales by bulk copies; warp 3
// reorders the scales into the rows of 16 B that tcgen05.cp wants (word c of
// row l belongs to key l + 32 c).  Loading them into that order directly was
// slower: 4-byte cp.async held the copying warp up for 1,000 clocks per 128
// keys, loads through registers (a scoreboard shared with the page lookups)
// for 3,300.  Warp 1 copies scales to TMEM and issues the MMAs into a ring of
// three accumulators.  Warp 2 fetches a unit's queries, their scales and the
// head weights, two units deep.  Warps 4.. read the accumulators back, in PAR
// groups of four warps that take steps in turn.
//
// Work: a unit is up to QU query tokens of one sequence.  With at most
// kImMaxPlan units (decode), the units' tiles form one sequence that is cut
// into equal ranges, one per CTA, which every CTA finds for itself from the
// visible counts; so ragged batches load the SMs evenly.  With more units (a
// prefill), CTAs take whole units in turn, back and forth, the last (the
// longest under a causal mask) first.
//
// Measured: 32 x 16,383 keys (38 MB) 14.8 us a call, 2.6 TB/s, over three sets of
// inputs that the L2 nearly holds (18.5 us alone and cold; the bf16 indexer on
// contiguous keys 27 us in the same loop); the plan, the first tile's trip to
// memory and the last tile's epilogue are about half of it.  8,192 causal tokens
// 103 us, 1.33 PFLOP/s; issue slots 56% busy, the accumulators' hand-over between
// MMA and epilogue is the rest.
#pragma once
#include <type_traits>

#include "common.cuh"
#include "mxfp4.cuh"
#include "sm100.cuh"

namespace csa {

constexpr int kImKeys = 256;           // keys per tile
constexpr int kImHalf = 128;           // the MMA's M
constexpr int kImHeads = 64;
constexpr int kImDim = 128;
constexpr int kImRow = kImDim / 2;     // bytes of codes per key or query head
constexpr int kImScales = kImDim / 32;  // scale bytes per key or query head
constexpr int kImBufs = 3;             // accumulators of 128 columns
constexpr int kImSfa = 4;              // key-scale buffers in TMEM, 8 columns each
constexpr int kImMaxPlan = 512;        // units whose tiles are dealt evenly
constexpr uint64_t kImDrainNs = 100000000ull;  // 100 ms for the wind-down waits

template <int QU, int STAGES>
struct IdxMxSmem {
  static constexpr int kGroups = (QU * kImHeads + 127) / 128;  // 128-row scale groups of a unit
  alignas(1024) uint8_t q[2][QU * kImHeads * kImRow];
  alignas(1024) uint8_t keys[STAGES][kImKeys * kImRow];
  alignas(128) uint8_t qs[2][kGroups * 512];
  alignas(128) uint8_t ks[STAGES][2 * 512];  // interleaved, as tcgen05.cp wants them
  alignas(128) uint8_t raw[STAGES][1040];    // in key order, as they are in memory
  alignas(16) float w[2][QU][kImHeads];
  int tiles[kImMaxPlan];
  uint64_t full[STAGES], empty[STAGES], raw_full[STAGES], acc_full[kImBufs], acc_empty[kImBufs];
  uint64_t q_full[2], q_empty[2], mma_drain, scales_over;
  uint32_t tmem_base;
  int abort_flag;
  int scaled;  // tiles whose scales were reordered, once scales_over is complete
  int u0, pre0, g0, g1;  // planned: first unit, its first tile, the CTA's range of tiles
};

struct IdxMxArgs {
  const uint8_t* q_scales;
  const float* w;
  const uint8_t* k_scales;
  PageMap pm;
  const int* q_pos;
  const int* n_cmp;
  int B, Tq, n_max, width, stride;
  int blocks_q;  // units per sequence
  int units;     // blocks_q * B; unit u is block u / B of sequence u % B
  int planned;   // ranges of tiles, else units in turn
  int box_rows;  // key rows per TMA box (256, or the page size below)
  unsigned long long wait_ns;
  float* scores;
};

// max(0, x) of two values (a NaN stays), packed.
__device__ __forceinline__ unsigned long long im_relu2(uint32_t lo, uint32_t hi) {
  unsigned long long r;
  asm("{\n\t.reg .f32 a, b;\n\t"
      "max.NaN.f32 a, %1, 0f00000000;\n\t"
      "max.NaN.f32 b, %2, 0f00000000;\n\t"
      "mov.b64 %0, {a, b};\n\t}"
      : "=l"(r)
      : "f"(__uint_as_float(lo)), "f"(__uint_as_float(hi)));
  return r;
}

// Two fp32 fused multiply-adds in one instruction.
__device__ __forceinline__ unsigned long long im_fma2(unsigned long long a, unsigned long long b,
                                                      unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Columns: accumulators, key scales, query scales of two units.
template <int QU>
struct IdxMxTmem {
  static constexpr int kAcc = kImBufs * 2 * kImHeads;
  static constexpr int kSfb = ((QU * kImHeads + 127) / 128) * 4;
  static_assert(kAcc + kImSfa * 8 + 2 * kSfb <= 512, "TMEM columns");
};

template <int QU, int STAGES, int PAR>
__global__ void __launch_bounds__(160 + 128 * PAR, 1)
    k_index_scores_mx(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ IdxMxArgs a) {
  using namespace sm100;
  using S = IdxMxSmem<QU, STAGES>;
  using T = IdxMxTmem<QU>;
  // a group waits for its step's accumulator by parity, so the step before it
  // in that buffer has to have passed: it comes no later than the group's last
  static_assert(PAR <= kImBufs, "a group would take an older phase for its own");
  extern __shared__ uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                ~static_cast<uintptr_t>(1023));
  // the warp index, known to be the same in all lanes
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint64_t wait_ns = a.wait_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sm.full[s], 2);  // the codes' bytes, the scales
      mbar_init(&sm.empty[s], 1);
      mbar_init(&sm.raw_full[s], 1);
    }
    for (int i = 0; i < kImBufs; ++i) {
      mbar_init(&sm.acc_full[i], 1);
      mbar_init(&sm.acc_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 33);
      mbar_init(&sm.q_empty[i], 4 * PAR + 1);
    }
    mbar_init(&sm.mma_drain, 1);
    mbar_init(&sm.scales_over, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 3) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  griddep_wait();  // inputs written by the predecessor are visible
  griddep_launch_dependents();
  // the page table on its way to L2 while the plan is made (a line per CTA)
  if (a.pm.table != nullptr && warp == 2 && lane == 0) {
    const long long bytes = (long long)a.B * a.pm.width * 4;
    for (int i = 0; i < 4; ++i) {
      const long long at = ((long long)i * gridDim.x + blockIdx.x) * 128;
      if (at < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(a.pm.table) + at));
    }
  }

  // entries visible to the unit's tokens: lane l's own count (l < nq) and
  // the largest; every lane of the warp takes part
  auto unit_nv = [&](int u, int* nq, int* own) {
    const int b = u % a.B, t0 = u / a.B * QU;
    const int n = min(QU, a.Tq - t0);
    int v = 0;
    if (lane < n) v = min(n_visible(a.q_pos[b * a.Tq + t0 + lane], a.n_cmp[b], a.width, a.stride), a.n_max);
    *nq = n;
    *own = v;
    return __reduce_max_sync(0xffffffffu, v);
  };

  if (a.planned && warp == 1) {
    int total = 0;
    for (int u0 = 0; u0 < a.units; u0 += 32) {
      const int u = u0 + lane;
      int nv = 0;
      if (u < a.units) {
        const int b = u % a.B, t0 = u / a.B * QU;
        const int n = min(QU, a.Tq - t0);
        for (int i = 0; i < n; ++i)
          nv = max(nv, min(n_visible(a.q_pos[b * a.Tq + t0 + i], a.n_cmp[b], a.width, a.stride), a.n_max));
        nv = (nv + kImKeys - 1) / kImKeys;
        sm.tiles[u] = nv;
      }
      total += __reduce_add_sync(0xffffffffu, nv);
    }
    __syncwarp();
    const int g0 = (int)((long long)total * blockIdx.x / gridDim.x);
    const int g1 = (int)((long long)total * (blockIdx.x + 1) / gridDim.x);
    if (lane == 0) {
      sm.g0 = g0;
      sm.g1 = g1;
      sm.u0 = sm.pre0 = 0;
    }
    __syncwarp();
    int at = 0;
    for (int u0 = 0; g0 < g1 && u0 < a.units; u0 += 32) {  // the unit that holds tile g0
      const int u = u0 + lane;
      const int tl = u < a.units ? sm.tiles[u] : 0;
      int inc = tl;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      if (g0 >= at + inc - tl && g0 < at + inc) {
        sm.u0 = u;
        sm.pre0 = at + inc - tl;
      }
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const uint32_t t_sfa = tmem + T::kAcc, t_sfb = t_sfa + kImSfa * 8;
  volatile int* abortp = &sm.abort_flag;

  // item k of this CTA: a unit and its tiles [tb, te), possibly none; false
  // past the end
  struct Item {
    int u, b, t0, nq, own, nv, tb, te;
    int next, pre;  // planned: the unit to come and its first tile
  };
  auto item = [&](int k, Item* it) -> bool {
    if (a.planned) {
      if (k == 0) {
        it->next = sm.u0;
        it->pre = sm.pre0;
      }
      if (it->pre >= sm.g1 || sm.g0 >= sm.g1) return false;
      it->u = it->next++;
      const int tl = sm.tiles[it->u];
      it->tb = max(0, sm.g0 - it->pre);
      it->te = min(tl, sm.g1 - it->pre);
      it->pre += tl;
    } else {
      // back and forth over the CTAs, so that their sums are near
      if ((long long)k * gridDim.x >= a.units) return false;
      const int c = (k & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
      it->u = a.units - 1 - (int)((long long)c + (long long)k * gridDim.x);
      it->tb = it->te = 0;
      if (it->u < 0) return true;  // no unit in this turn
    }
    it->b = it->u % a.B;
    it->t0 = it->u / a.B * QU;
    it->nv = unit_nv(it->u, &it->nq, &it->own);
    if (!a.planned) it->te = (it->nv + kImKeys - 1) / kImKeys;
    return true;
  };

  Item it;
  constexpr int kProducer2 = 4 + 4 * PAR;
  if (warp == 0 || warp == kProducer2) {
    // ---------------- key tiles, every second one
    const int turn = warp == 0 ? 0 : 1;
    if (lane == 0) tma_prefetch_desc(&tm_k);
    static_assert(STAGES % 2 == 0, "a stage belongs to one fetching warp");
    const int subs = kImKeys / a.box_rows;  // boxes per tile, at most 32
    int n = 0;                              // tiles requested
    bool ok = true;
    for (int k = 0; ok && item(k, &it); ++k) {
      const bool paged = a.pm.table != nullptr;
      PageWindow pw;
      if (paged && it.tb < it.te) pw.start(a.pm, it.b, it.nv, (it.tb * kImKeys) >> a.pm.shift);
      for (int i = it.tb; i < it.te; ++i, ++n) {
        if ((n & 1) != turn) continue;
        const int s = n % STAGES;
        const int j0 = i * kImKeys;
        const int jb = j0 + lane * a.box_rows;  // first key of box `lane`
        long long box = lane < subs && jb < it.nv ? (long long)it.b * a.n_max + jb : -1;
        if (paged) {
          pw.seek(j0 >> a.pm.shift);
          const int pg = pw.at(jb >> a.pm.shift);
          if (box >= 0)
            box = (unsigned)pg < (unsigned)a.pm.n_pages
                      ? ((long long)pg << a.pm.shift) + (jb & ((1 << a.pm.shift) - 1)) : -1;
        }
        ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.empty[s], ((uint32_t)(n / STAGES) & 1u) ^ 1u, abortp, wait_ns));
        if (!ok) break;
        const unsigned boxes = __ballot_sync(0xffffffffu, box >= 0);
        // scales: a box's are contiguous; contiguous keys start at a multiple
        // of four, and end at the last whole 16 bytes of the array
        long long sc_row = box, sc_bytes = a.box_rows * kImScales;
        if (!paged) {
          sc_row = box & ~3LL;
          sc_bytes = min(1040LL, ((long long)a.B * a.n_max - sc_row) * kImScales & ~15LL);
        }
        if (lane == 0) {
          const uint32_t n_box = (uint32_t)__popc(boxes);
          mbar_arrive_expect_tx(&sm.full[s], n_box * (uint32_t)(a.box_rows * kImRow));
          mbar_arrive_expect_tx(&sm.raw_full[s], n_box * (uint32_t)sc_bytes);
        }
        __syncwarp();
        if (box >= 0) {
          tma_load_2d(sm.keys[s] + lane * a.box_rows * kImRow, &tm_k, &sm.full[s], 0, (int)box);
          if (sc_bytes > 0)
            bulk_load(sm.raw[s] + lane * a.box_rows * kImScales, a.k_scales + sc_row * kImScales,
                      (uint32_t)sc_bytes, &sm.raw_full[s]);
        }
      }
    }
    // every copy into shared memory lands before the CTA may exit: each warp
    // waits for the last tiles that it asked for itself (after a wait that ran
    // out the other may have asked for fewer, or for more).  `full` also counts
    // warp 3: where that left before a tile, its arrival is made up here
    if (lane == 0) {
      auto drain = [](uint64_t* bar, uint32_t parity) {  // (a call is worth 220 clocks)
        return mbar_try_wait(bar, parity) || mbar_drain(bar, parity, kImDrainNs);
      };
      int i0 = max(0, n - STAGES);
      i0 += (i0 & 1) != turn ? 1 : 0;
      for (int i = i0; i < n; i += 2) drain(&sm.raw_full[i % STAGES], (uint32_t)(i / STAGES) & 1u);
      const bool over = drain(&sm.scales_over, 0);
      for (int i = i0; i < n; i += 2) {
        if (over && i >= sm.scaled) mbar_arrive(&sm.full[i % STAGES]);
        drain(&sm.full[i % STAGES], (uint32_t)(i / STAGES) & 1u);
      }
    }
  } else if (warp == 2) {
    // ---------------- queries, their scales and weights
    if (lane == 0) tma_prefetch_desc(&tm_q);
    int n = 0;
    bool ok = true;
    for (int k = 0; ok && item(k, &it); ++k) {
      if (it.te <= it.tb) continue;
      const int qb = n & 1;
      if (lane == 0) ok = mbar_wait_fast(&sm.q_empty[qb], ((uint32_t)(n >> 1) & 1u) ^ 1u, abortp, wait_ns);
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      if (!ok) break;
      const long long row0 = (long long)it.b * a.Tq + it.t0;  // query token
      if (lane == 0) mbar_arrive_expect_tx(&sm.q_full[qb], (uint32_t)(it.nq * kImHeads * kImRow));
      __syncwarp();
      if (lane < it.nq)
        tma_load_2d(sm.q[qb] + lane * kImHeads * kImRow, &tm_q, &sm.q_full[qb], 0,
                    (int)(row0 + lane) * kImHeads);
      const int heads = it.nq * kImHeads;
      const uint32_t ds = smem_u32(sm.qs[qb]);
      const uint8_t* ss = a.q_scales + row0 * kImHeads * kImScales;
      for (int r = lane; r < heads; r += 32)
        cp_async4(ds + (uint32_t)((r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4),
                  ss + (long long)r * kImScales, true);
      const uint32_t dw = smem_u32(sm.w[qb]);
      const float* sw = a.w + row0 * kImHeads;
      for (int i = lane; i < heads / 4; i += 32) cp_async16(dw + 16u * i, sw + 4 * i, true);
      cp_async_arrive(&sm.q_full[qb]);
      ++n;
    }
    cp_async_wait_all();
    __syncwarp();
    if (lane == 0)
      for (int i = max(0, n - 2); i < n; ++i)
        mbar_drain(&sm.q_full[i & 1], (uint32_t)(i >> 1) & 1u, kImDrainNs);
  } else if (warp == 3) {
    // ---------------- key scales from key order to rows of 16 bytes: lane l
    // takes the words of keys l + 32 c
    int n = 0;
    bool ok = true;
    for (int k = 0; ok && item(k, &it); ++k) {
      for (int i = it.tb; i < it.te; ++i, ++n) {
        const int s = n % STAGES;
        ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.raw_full[s], (uint32_t)(n / STAGES) & 1u, abortp, wait_ns));
        if (!ok) break;
        const uint32_t* raw = reinterpret_cast<const uint32_t*>(sm.raw[s]);
        const long long rows = (long long)a.B * a.n_max;
        const long long r0 = (long long)it.b * a.n_max + (long long)i * kImKeys, r4 = r0 & ~3LL;
        const int off = a.pm.table != nullptr ? 0 : (int)(r0 - r4);
        const int got = a.pm.table != nullptr ? kImKeys : (int)min(260LL, (rows - r4) & ~3LL);  // rows copied
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t v[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int at = off + half * kImHalf + lane + 32 * c;
            v[c] = 0u;
            if (at < got)
              v[c] = raw[at];
            else if (r4 + at < rows)  // contiguous keys: the array's last one to three
              v[c] = reinterpret_cast<const uint32_t*>(a.k_scales)[r4 + at];
          }
          *reinterpret_cast<uint4*>(sm.ks[s] + half * 512 + lane * 16) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        fence_proxy_async_shared();  // read by tcgen05.cp (async proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[s]);
      }
    }
    if (lane == 0) {
      sm.scaled = n;
      mbar_arrive(&sm.scales_over);
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (the whole warp runs the loop, one elected
    // lane issues)
    constexpr uint32_t id0 = idesc_mxf4(kImHalf, kImHeads, 0), id1 = idesc_mxf4(kImHalf, kImHeads, 2);
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      return __all_sync(0xffffffffu, mbar_wait_fast(bar, phase & 1u, abortp, wait_ns)) != 0;
    };
    const uint32_t q0 = smem_u32(sm.q[0]), k0 = smem_u32(sm.keys[0]);
    const uint32_t qs0 = smem_u32(sm.qs[0]), ks0 = smem_u32(sm.ks[0]);
    int n = 0, tile = 0, acc = 0;
    uint32_t aph = 0;  // phase of the accumulator ring
    bool ok = true;
    for (int k = 0; ok && item(k, &it); ++k) {
      if (it.te <= it.tb) continue;
      const int qb = n & 1;
      ok = wait(&sm.q_full[qb], (uint32_t)(n >> 1));
      if (!ok) break;
      fence_proxy_async_shared();  // scales came by cp.async (generic proxy)
      tc_fence_after();
      const uint32_t qs = qs0 + (uint32_t)qb * (S::kGroups * 512);
      if (elect_one())
        for (int g = 0; g < (it.nq * kImHeads + 127) / 128; ++g)
          tc_cp_scales(t_sfb + (uint32_t)(qb * T::kSfb + 4 * g), scale_desc(qs + 512u * g));
      __syncwarp();
      const uint32_t q_addr = q0 + (uint32_t)qb * (QU * kImHeads * kImRow);
      for (int i = it.tb; i < it.te && ok; ++i, ++tile) {
        const int s = tile % STAGES;
        ok = wait(&sm.full[s], (uint32_t)(tile / STAGES));
        if (!ok) break;
        tc_fence_after();
        // the buffer's last reader, tile - 4, has finished: at least four
        // steps lie between, and the accumulators have three buffers
        const uint32_t sfa = t_sfa + (uint32_t)((tile % kImSfa) * 8);
        if (elect_one()) {
          tc_cp_scales(sfa, scale_desc(ks0 + 1024u * s));
          tc_cp_scales(sfa + 4, scale_desc(ks0 + 1024u * s + 512u));
        }
        __syncwarp();
        const uint64_t ka = sw64_desc(k0 + (uint32_t)(s * kImKeys * kImRow), 512);
        const bool two = i * kImKeys + kImHalf < it.nv;
        for (int tok = 0; tok < it.nq; ++tok) {
          ok = wait(&sm.acc_empty[acc], aph ^ 1u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * 2 * kImHeads);
          const uint32_t sfb = t_sfb + (uint32_t)(qb * T::kSfb + tok * 2);
          const uint64_t qa = sw64_desc(q_addr + (uint32_t)(tok * kImHeads * kImRow), 512);
          if (elect_one()) {
            mma_mxf4(d, ka, qa, id0, sfa, sfb, 0u);
            mma_mxf4(d, ka + 2, qa + 2, id1, sfa, sfb, 1u);  // 32 bytes on
            if (two) {
              const uint64_t kb = ka + (uint64_t)(kImHalf * kImRow >> 4);
              mma_mxf4(d + kImHeads, kb, qa, id0, sfa + 4, sfb, 0u);
              mma_mxf4(d + kImHeads, kb + 2, qa + 2, id1, sfa + 4, sfb, 1u);
            }
            tc_commit(&sm.acc_full[acc]);
            if (tok == it.nq - 1) {
              tc_commit(&sm.empty[s]);
              if (i == it.te - 1) tc_commit(&sm.q_empty[qb]);
            }
          }
          __syncwarp();
          acc = acc == kImBufs - 1 ? 0 : acc + 1;
          aph ^= acc == 0 ? 1u : 0u;
        }
      }
      ++n;
    }
    if (elect_one()) {  // TMEM is freed only after every MMA and copy has landed
      tc_commit(&sm.mma_drain);
      mbar_drain(&sm.mma_drain, 0, kImDrainNs);
    }
    __syncwarp();
  } else {
    // ---------------- epilogue: group `par` of four warps takes every PAR-th step
    const int par = (warp - 4) >> 2, quarter = warp & 3;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    int n = 0, acc = 0, turn = 0;
    uint32_t aph = 0;
    bool ok = true;
    for (int k = 0; ok && item(k, &it); ++k) {
      if (it.te <= it.tb) continue;
      const int qb = n & 1;
      ok = __all_sync(0xffffffffu, mbar_wait_strict(&sm.q_full[qb], (uint32_t)(n >> 1) & 1u, abortp, wait_ns));
      const bool paged = a.pm.table != nullptr;
      PageWindow pw;
      if (paged) pw.start(a.pm, it.b, it.nv, (it.tb * kImKeys) >> a.pm.shift);
      float* row0 = a.scores + ((long long)it.b * a.Tq + it.t0) * a.n_max;
      for (int i = it.tb; i < it.te && ok; ++i) {
        const int j = i * kImKeys + quarter * 32 + lane;  // and j + 128
        bool in0 = true, in1 = true;
        if (paged) {
          pw.seek((i * kImKeys) >> a.pm.shift);
          in0 = (unsigned)pw.at(j >> a.pm.shift) < (unsigned)a.pm.n_pages;
          in1 = (unsigned)pw.at((j + kImHalf) >> a.pm.shift) < (unsigned)a.pm.n_pages;
          if (par == 0 && ((!in0 && j < it.nv) || (!in1 && j + kImHalf < it.nv)))
            report_error(CSA_ERR_DEVICE_BOUNDS);
        }
        const bool two = i * kImKeys + kImHalf < it.nv;
        for (int tok = 0; tok < it.nq; ++tok) {
          const int me = acc;
          const uint32_t ph = aph;
          const bool mine = turn == par;
          acc = acc == kImBufs - 1 ? 0 : acc + 1;
          aph ^= acc == 0 ? 1u : 0u;
          turn = turn == PAR - 1 ? 0 : turn + 1;
          if (!mine) continue;
          ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.acc_full[me], ph, abortp, wait_ns));
          if (!ok) break;
          tc_fence_after();
          const int nv = __shfl_sync(0xffffffffu, it.own, tok);
          // 8 heads at a time, the next ones on their way; two packed pairs of
          // sums per key, joined at the end; a NaN passes through the maximum
          const uint32_t col = tmem + lane_base + (uint32_t)(me * 2 * kImHeads);
          const ulonglong2* w = reinterpret_cast<const ulonglong2*>(sm.w[qb][tok]);
          unsigned long long x01 = 0ull, x23 = 0ull, y01 = 0ull, y23 = 0ull;
          auto score = [&](auto both) {
            constexpr bool kBoth = decltype(both)::value;
            uint32_t r[2][2][8];
            tmem_ld8(col, r[0][0]);
            if (kBoth) tmem_ld8(col + kImHeads, r[0][1]);
#pragma unroll
            for (int c = 0; c < kImHeads / 8; ++c) {
              uint32_t(&r0)[8] = r[c & 1][0];
              uint32_t(&r1)[8] = r[c & 1][1];
              if (kBoth)
                tmem_wait_ld8(r0, r1);
              else
                tmem_wait_ld8(r0);
              if (c + 1 < kImHeads / 8) {
                tmem_ld8(col + (uint32_t)(8 * (c + 1)), r[(c + 1) & 1][0]);
                if (kBoth) tmem_ld8(col + (uint32_t)(kImHeads + 8 * (c + 1)), r[(c + 1) & 1][1]);
              } else {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.acc_empty[me]);
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const ulonglong2 wh = w[2 * c + h];
                x01 = im_fma2(wh.x, im_relu2(r0[4 * h], r0[4 * h + 1]), x01);
                x23 = im_fma2(wh.y, im_relu2(r0[4 * h + 2], r0[4 * h + 3]), x23);
                if (kBoth) {
                  y01 = im_fma2(wh.x, im_relu2(r1[4 * h], r1[4 * h + 1]), y01);
                  y23 = im_fma2(wh.y, im_relu2(r1[4 * h + 2], r1[4 * h + 3]), y23);
                }
              }
            }
          };
          if (two)
            score(std::true_type{});
          else
            score(std::false_type{});
          auto sum4 = [](unsigned long long p, unsigned long long q) {
            return (__uint_as_float((uint32_t)p) + __uint_as_float((uint32_t)(p >> 32))) +
                   (__uint_as_float((uint32_t)q) + __uint_as_float((uint32_t)(q >> 32)));
          };
          float* row = row0 + (long long)tok * a.n_max + j;
          if (j < nv && in0) row[0] = sum4(x01, x23);
          if (j + kImHalf < nv && in1) row[kImHalf] = sum4(y01, y23);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_empty[qb]);  // the weights have been read
      ++n;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace csa
