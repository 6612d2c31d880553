// Step 2a on 4-bit tensor cores: lightning-indexer scores of MXFP4 queries
// (64 heads x 128 dims) and paged MXFP4 keys.
//
//   D[key][q*64 + h] = sum_c q[q][h][c] k[key][c]   (tcgen05 kind::mxf4: E2M1
//                      operands, one E8M0 scale per 32 dims, fp32 in TMEM)
//   s[q][key]        = sum_h w[q][h] max(0, D)       (one key per thread)
//
// Keys are the MMA's M (128 per tile), NT tokens x 64 heads its N, the 128
// dims two K steps of 64.  A key is 64 B of codes and 4 B of scales: decode
// streams 68 B per key where the bf16 indexer streams 256, and is HBM-bound;
// a prefill is bound by the epilogue (two instructions per key, token and
// head on CUDA cores), so NT = 2 gives it eight warps.
//
// Roles: warp 0 fetches the codes of key tiles into a ring by TMA, one box per
// page (64-byte swizzle), and their scales by bulk copies; warp 3 reorders the
// scales into the rows of 16 B that tcgen05.cp wants (word c of row l belongs
// to key l + 32 c).  Loading them into that order directly was slower: 4-byte
// cp.async held the copying warp up for 1,000 clocks a tile, loads through
// registers (a scoreboard shared with the page lookups) for 3,300.
// Warp 1 (one thread) copies scales to TMEM and issues the MMAs into a ring
// of three accumulators.  Warp 2 fetches a unit's queries, their scales and
// the head weights, two units deep.  Warps 4.. read the accumulators back, in
// groups of four warps: one token of the NT, every PAR-th block.
//
// Work: a unit is up to QU query tokens of one sequence.  With no more units
// than CTAs, the unit's key tiles are dealt to CTAs by a plan that every CTA
// makes for itself from the visible counts: the fewest tiles L per CTA for
// which sum ceil(tiles_u / L) fits the grid, tried at total / (CTAs - units /
// 2) and taken at total / (CTAs - units), which always fits; so ragged
// batches load the SMs evenly.  With more units, CTAs are persistent and take
// units in turn, the last (in a causal prefill, the longest) first.
#pragma once
#include "common.cuh"
#include "mxfp4.cuh"
#include "sm100.cuh"

namespace csa {

constexpr int kImKeys = 128;
constexpr int kImHeads = 64;
constexpr int kImDim = 128;
constexpr int kImRow = kImDim / 2;     // bytes of codes per key or query head
constexpr int kImScales = kImDim / 32;  // scale bytes per key or query head
constexpr int kImBufs = 3;             // accumulators
constexpr int kImSfa = 4;              // key-scale buffers in TMEM
constexpr int kImMaxPlan = 512;        // units a plan may hold
constexpr uint64_t kImDrainNs = 100000000ull;  // 100 ms for the wind-down waits

template <int NT, int QU, int STAGES>
struct IdxMxSmem {
  static constexpr int kN = NT * kImHeads;
  static constexpr int kBlocks = QU / NT;                // MMA N blocks per unit
  static constexpr int kGroups = (QU * kImHeads + 127) / 128;  // 128-row scale groups of a unit
  alignas(1024) uint8_t q[2][QU * kImHeads * kImRow];
  alignas(1024) uint8_t keys[STAGES][kImKeys * kImRow];
  alignas(128) uint8_t qs[2][kGroups * 512];
  alignas(128) uint8_t ks[STAGES][512];   // interleaved, as tcgen05.cp wants them
  alignas(128) uint8_t raw[STAGES][528];  // in key order, as they are in memory
  alignas(16) float w[2][QU][kImHeads];
  int tiles[kImMaxPlan];
  uint64_t full[STAGES], empty[STAGES], raw_full[STAGES], acc_full[kImBufs], acc_empty[kImBufs];
  uint64_t q_full[2], q_empty[2], mma_drain;
  uint32_t tmem_base;
  int abort_flag;
  int plan[3];  // this CTA's unit, first tile and end tile (planned launches)
  int own[QU];  // entries visible to each of that unit's tokens
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
  int planned;   // one planned item per CTA, else units in turn
  int box_rows;  // key rows per TMA box (128, or the page size below)
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
template <int NT, int QU>
struct IdxMxTmem {
  static constexpr int kAcc = kImBufs * NT * kImHeads;
  static constexpr int kSfb = ((QU * kImHeads + 127) / 128) * 4;
  static constexpr int kUsed = kAcc + kImSfa * 4 + 2 * kSfb;
  static constexpr uint32_t kCols = kUsed <= 256 ? 256 : 512;
  static_assert(kUsed <= 512, "TMEM columns");
};

template <int NT, int QU, int STAGES, int PAR, int MINB>
__global__ void __launch_bounds__(160 + 128 * NT * PAR, MINB)
    k_index_scores_mx(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ IdxMxArgs a) {
  using namespace sm100;
  using S = IdxMxSmem<NT, QU, STAGES>;
  using T = IdxMxTmem<NT, QU>;
  constexpr int N = S::kN;
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
      mbar_init(&sm.acc_empty[i], 4 * NT);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 33);
      mbar_init(&sm.q_empty[i], 4 * NT * PAR + 1);
    }
    mbar_init(&sm.mma_drain, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 3) {
    tmem_alloc(&sm.tmem_base, T::kCols);
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
    const int G = (int)gridDim.x;
    int L = 1;
    for (int tries = 0; tries < 2; ++tries) {
      const int room = tries == 0 ? G - a.units / 2 : G - a.units + 1;
      L = max(1, (total + room - 1) / room);
      int need = 0;
      for (int u = lane; u < a.units; u += 32) need += (sm.tiles[u] + L - 1) / L;
      if (__reduce_add_sync(0xffffffffu, need) <= G) break;
    }
    // the unit whose CTAs hold this one, its parts of nearly equal size
    int at = 0, pu = -1, pb = 0, pe = 0;
    for (int u0 = 0; u0 < a.units; u0 += 32) {
      const int u = u0 + lane;
      const int tl = u < a.units ? sm.tiles[u] : 0;
      const int cnt = (tl + L - 1) / L;
      int inc = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      const int part = (int)blockIdx.x - (at + inc - cnt);
      if (part >= 0 && part < cnt) {
        pu = u;
        const int each = tl / cnt, more = tl - each * cnt;
        pb = part * each + min(part, more);
        pe = pb + each + (part < more ? 1 : 0);
      }
      at += __shfl_sync(0xffffffffu, inc, 31);
    }
    const unsigned who = __ballot_sync(0xffffffffu, pu >= 0);
    if (who == 0 ? lane == 0 : pu >= 0) {
      sm.plan[0] = pu;
      sm.plan[1] = pb;
      sm.plan[2] = pe;
    }
    __syncwarp();
    const int u = sm.plan[0];
    if (u >= 0 && lane < QU) {
      const int b = u % a.B, t = u / a.B * QU + lane;
      sm.own[lane] = t < a.Tq ? min(n_visible(a.q_pos[b * a.Tq + t], a.n_cmp[b], a.width, a.stride), a.n_max) : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const uint32_t t_sfa = tmem + T::kAcc, t_sfb = t_sfa + kImSfa * 4;
  volatile int* abortp = &sm.abort_flag;

  // item k of this CTA: a unit and its key tiles [tb, te); false past the end
  struct Item {
    int u, b, t0, nq, own, nv, tb, te;
  };
  auto item = [&](int k, Item* it) -> bool {
    if (a.planned) {
      if (k > 0 || sm.plan[0] < 0) return false;
      it->u = sm.plan[0];
    } else {
      // back and forth over the CTAs, so that their sums are near
      const int c = (k & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x;
      const long long i = (long long)c + (long long)k * gridDim.x;
      if ((long long)k * gridDim.x >= a.units) return false;
      it->u = a.units - 1 - (int)i;
      if (i >= a.units) it->u = -1;
    }
    if (it->u < 0) {  // no unit in this turn
      it->tb = it->te = it->nv = it->nq = it->own = it->b = it->t0 = 0;
      return true;
    }
    it->b = it->u % a.B;
    it->t0 = it->u / a.B * QU;
    if (a.planned) {
      it->nq = min(QU, a.Tq - it->t0);
      it->own = lane < QU ? sm.own[lane] : 0;
      it->nv = __reduce_max_sync(0xffffffffu, it->own);
    } else {
      it->nv = unit_nv(it->u, &it->nq, &it->own);
    }
    it->tb = a.planned ? sm.plan[1] : 0;
    it->te = a.planned ? sm.plan[2] : (it->nv + kImKeys - 1) / kImKeys;
    return true;
  };

  Item it;
  constexpr int kProducer2 = 4 + 4 * NT * PAR;
  if (warp == 0 || warp == kProducer2) {
    // ---------------- key tiles, every second one
    const int turn = warp == 0 ? 0 : 1;
    if (lane == 0) tma_prefetch_desc(&tm_k);
    const int subs = kImKeys / a.box_rows;  // boxes per tile, at most 16
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
          sc_bytes = min(528LL, ((long long)a.B * a.n_max - sc_row) * kImScales & ~15LL);
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
    // every copy into shared memory lands before the CTA may exit
    if (lane == 0 && turn == 0)
      for (int i = max(0, n - STAGES); i < n; ++i) {
        mbar_drain(&sm.raw_full[i % STAGES], (uint32_t)(i / STAGES) & 1u, kImDrainNs);
        mbar_drain(&sm.full[i % STAGES], (uint32_t)(i / STAGES) & 1u, kImDrainNs);
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
        uint32_t v[4];
        if (a.pm.table != nullptr) {
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = raw[lane + 32 * c];
        } else {
          const long long rows = (long long)a.B * a.n_max;
          const long long r0 = (long long)it.b * a.n_max + (long long)i * kImKeys, r4 = r0 & ~3LL;
          const int got = (int)min(132LL, (rows - r4) & ~3LL);  // rows copied
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int at = (int)(r0 - r4) + lane + 32 * c;
            v[c] = 0u;
            if (at < got)
              v[c] = raw[at];
            else if (r4 + at < rows)  // the array's last one to three
              v[c] = reinterpret_cast<const uint32_t*>(a.k_scales)[r4 + at];
          }
        }
        *reinterpret_cast<uint4*>(sm.ks[s] + lane * 16) = make_uint4(v[0], v[1], v[2], v[3]);
        fence_proxy_async_shared();  // read by tcgen05.cp (async proxy)
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[s]);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (the whole warp runs the loop, one elected
    // lane issues)
    constexpr uint32_t id0 = idesc_mxf4(128, N, 0), id1 = idesc_mxf4(128, N, 2);
    auto wait = [&](uint64_t* bar, uint32_t phase) {
      return __all_sync(0xffffffffu, mbar_wait_fast(bar, phase & 1u, abortp, wait_ns)) != 0;
    };
    const uint32_t q0 = smem_u32(sm.q[0]), k0 = smem_u32(sm.keys[0]);
    const uint32_t qs0 = smem_u32(sm.qs[0]), ks0 = smem_u32(sm.ks[0]);
    int n = 0, tile = 0, step = 0;
    bool ok = true;
    for (int k = 0; ok && item(k, &it); ++k) {
      if (it.te <= it.tb) continue;
      const int qb = n & 1;
      const int blocks = (it.nq + NT - 1) / NT;
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
        const uint32_t sfa = t_sfa + (uint32_t)((tile % kImSfa) * 4);
        if (elect_one()) tc_cp_scales(sfa, scale_desc(ks0 + 512u * s));
        __syncwarp();
        const uint64_t ka = sw64_desc(k0 + (uint32_t)(s * kImKeys * kImRow), 512);
        for (int nb = 0; nb < blocks; ++nb, ++step) {
          const int acc = step % kImBufs;
          ok = wait(&sm.acc_empty[acc], (uint32_t)(step / kImBufs) ^ 1u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * N);
          const uint32_t sfb = t_sfb + (uint32_t)(qb * T::kSfb + nb * (N / 32));
          const uint64_t qa = sw64_desc(q_addr + (uint32_t)(nb * N * kImRow), 512);
          if (elect_one()) {
            mma_mxf4(d, ka, qa, id0, sfa, sfb, 0u);
            mma_mxf4(d, ka + 2, qa + 2, id1, sfa, sfb, 1u);  // 32 bytes on
            tc_commit(&sm.acc_full[acc]);
            if (nb == blocks - 1) {
              tc_commit(&sm.empty[s]);
              if (i == it.te - 1) tc_commit(&sm.q_empty[qb]);
            }
          }
          __syncwarp();
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
    // ---------------- epilogue: group g takes token g % NT of every PAR-th
    // block (step % PAR = g / NT)
    const int g = (warp - 4) >> 2, quarter = warp & 3;
    const int tk = g % NT, par = g / NT;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    int n = 0, step = 0;
    bool ok = true;
    for (int k = 0; ok && item(k, &it); ++k) {
      if (it.te <= it.tb) continue;
      const int qb = n & 1;
      const int blocks = (it.nq + NT - 1) / NT;
      ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.q_full[qb], (uint32_t)(n >> 1) & 1u, abortp, wait_ns));
      const bool paged = a.pm.table != nullptr;
      PageWindow pw;
      if (paged) pw.start(a.pm, it.b, it.nv, (it.tb * kImKeys) >> a.pm.shift);
      for (int i = it.tb; i < it.te && ok; ++i) {
        const int j = i * kImKeys + quarter * 32 + lane;
        bool in_pool = true;
        if (paged) {
          pw.seek((i * kImKeys) >> a.pm.shift);
          in_pool = (unsigned)pw.at(j >> a.pm.shift) < (unsigned)a.pm.n_pages;
          if (!in_pool && j < it.nv && g == 0) report_error(CSA_ERR_DEVICE_BOUNDS);
        }
        for (int nb = 0; nb < blocks; ++nb, ++step) {
          if (PAR > 1 && step % PAR != par) continue;
          const int acc = step % kImBufs;
          ok = __all_sync(0xffffffffu, mbar_wait_fast(&sm.acc_full[acc], (uint32_t)(step / kImBufs) & 1u, abortp, wait_ns));
          if (!ok) break;
          tc_fence_after();
          const int tok = nb * NT + tk;
          const int nv = __shfl_sync(0xffffffffu, it.own, tok & 31);  // 0 past nq
          float s[4] = {0.f, 0.f, 0.f, 0.f};
          auto release = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.acc_empty[acc]);
          };
          if (tok < it.nq) {
            // 16 heads at a time, the next ones on their way; four sums in two
            // packed pairs, joined at the end; a NaN passes through the maximum
            const uint32_t col = tmem + lane_base + (uint32_t)(acc * N + tk * kImHeads);
            const ulonglong2* w = reinterpret_cast<const ulonglong2*>(sm.w[qb][tok]);
            uint32_t r[2][16];
            unsigned long long s01 = 0ull, s23 = 0ull;
            tmem_ld16(col, r[0]);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              tmem_wait_ld16(r[c & 1]);
              if (c < 3)
                tmem_ld16(col + (uint32_t)(16 * (c + 1)), r[(c + 1) & 1]);
              else
                release();
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const ulonglong2 wh = w[4 * c + h];
                s01 = im_fma2(wh.x, im_relu2(r[c & 1][4 * h], r[c & 1][4 * h + 1]), s01);
                s23 = im_fma2(wh.y, im_relu2(r[c & 1][4 * h + 2], r[c & 1][4 * h + 3]), s23);
              }
            }
            s[0] = __uint_as_float((uint32_t)s01);
            s[1] = __uint_as_float((uint32_t)(s01 >> 32));
            s[2] = __uint_as_float((uint32_t)s23);
            s[3] = __uint_as_float((uint32_t)(s23 >> 32));
          } else {
            release();
          }
          if (j < nv && in_pool)
            a.scores[((long long)it.b * a.Tq + it.t0 + tok) * a.n_max + j] = (s[0] + s[1]) + (s[2] + s[3]);
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
    tmem_dealloc(tmem, T::kCols);
  }
}

}  // namespace csa
