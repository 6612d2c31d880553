// Shared-KV attention over paged caches, generic shapes (any head count, d
// in 64 .. 1024, bf16 or fp32), CUDA cores, fp32 math: over the selected
// entries (CSA) or every visible entry (HCA) and the window's raw rows.
//
// One CTA of 8 warps per (query token, HG heads, split of the rows).  A warp
// takes every 8th row of its split: lane l holds dims l, l + 32, ... of the
// row once and uses them for HG heads, whose queries and accumulators stay
// in registers (2 HG d / 32 = 64 of them).  The warps' online-softmax states
// are joined in shared memory; with one split the CTA finishes the output,
// else it writes (m, l, acc) in fp32 and k_attn_paged_join combines the
// splits in their order (deterministic).  A NaN logit makes l NaN, and weights
// of 0 in the joins leave it so.  Bound by its multiply-adds and by
// reading each row once per HG heads: 16 x 1,152 rows of 512 in bf16 under 128
// heads took 617 us here, 25 us on the tensor-core kernel that took over d =
// 512 in bf16 (attn_dense.cuh).
#pragma once
#include "common.cuh"
#include "mxfp4.cuh"

namespace csa {

constexpr int kPgWarps = 8;
constexpr int kPgMaxPairs = 512;

struct PagedAttnArgs {
  const void* q;
  const int* q_pos;
  const void* kv;  // pool [n_pages][page][d]
  PageMap pm;
  const int* idx;    // CSA: [B][Tq][topk]
  const int* n_cmp;  // HCA: [B]
  int n_max;         // entries the table can hold
  const void* kv_raw;
  const int* raw_pos0;
  const int* n_raw;
  int raw_max;
  const float* sink;
  int Tq, H, d, rope_dim, topk, window, width, stride, splits;
  float scale;
  void* out;
  float* part;  // splits > 1: [token][head][split][d + 2]: acc, m, l (natural log)
  double freq[kPgMaxPairs];
};

template <int NK>
__device__ __forceinline__ void pg_rotate(float (&v)[NK], const PagedAttnArgs& a, long long pos) {
  const int lane = threadIdx.x & 31;
  const int rope0 = a.d - a.rope_dim;
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    const int c = lane + 32 * k;
    const float other = __shfl_xor_sync(0xffffffffu, v[k], 1);
    if (c >= rope0) {
      float cs, sn;
      rope_cos_sin(pos, a.freq[(c - rope0) >> 1], &cs, &sn);
      v[k] = (c & 1) ? (other * sn + v[k] * cs) : (v[k] * cs - other * sn);
    }
  }
}

// The output of one head from its joined state: the sink's exponential joins
// the denominator, the RoPE dims turn back, one rounding.
template <typename T, int NK>
__device__ __forceinline__ void pg_finish(const PagedAttnArgs& a, int token, int h, float m, float l,
                                          float (&acc)[NK]) {
  const float sink = a.sink[h];
  const float M = fmaxf(sink, m);
  const float wm = m == -INFINITY ? 0.f : expf(m - M);
  const float L = l * wm + (sink == -INFINITY ? 0.f : expf(sink - M));
  const float inv = L > 0.f || L != L ? wm / L : 0.f;  // no row and no sink: 0
#pragma unroll
  for (int k = 0; k < NK; ++k) acc[k] *= inv;
  pg_rotate<NK>(acc, a, -(long long)a.q_pos[token]);
  T* op = static_cast<T*>(a.out) + ((long long)token * a.H + h) * a.d + (threadIdx.x & 31);
#pragma unroll
  for (int k = 0; k < NK; ++k) store(op + 32 * k, acc[k]);
}

template <typename T, bool kHca, int NK, int HG>
__global__ void __launch_bounds__(32 * kPgWarps) k_attn_paged_simt(const __grid_constant__ PagedAttnArgs a) {
  __shared__ float sm_acc[kPgWarps][NK * 32];
  __shared__ float sm_m[kPgWarps][HG], sm_l[kPgWarps][HG];
  const int split = blockIdx.x % a.splits, h0 = blockIdx.x / a.splits * HG;
  const int token = blockIdx.y, b = token / a.Tq;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int t = a.q_pos[token];

  float qv[HG][NK];
#pragma unroll
  for (int g = 0; g < HG; ++g) {
    const int h = min(h0 + g, a.H - 1);
    const T* qp = static_cast<const T*>(a.q) + ((long long)token * a.H + h) * a.d + lane;
#pragma unroll
    for (int k = 0; k < NK; ++k) qv[g][k] = to_f32(qp[32 * k]);
    pg_rotate<NK>(qv[g], a, t);
  }
  const int n_sel = kHca ? max(0, min(n_visible(t, a.n_cmp[b], a.width, a.stride), a.n_max)) : a.topk;
  const int* sel = kHca ? nullptr : a.idx + (long long)token * a.topk;
  const int rp0 = a.raw_pos0[b];
  const int w_lo = max(max(0, t - a.window + 1), rp0);
  const int w_hi = min(t, rp0 + (min(a.n_raw[b], a.raw_max) - 1));
  const int n_win = a.window > 0 && w_hi >= w_lo ? w_hi - w_lo + 1 : 0;
  const long long n_rows = (long long)n_sel + n_win;
  const long long r0 = n_rows * split / a.splits, r1 = n_rows * (split + 1) / a.splits;

  float m[HG], l[HG], acc[HG][NK];
#pragma unroll
  for (int g = 0; g < HG; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int k = 0; k < NK; ++k) acc[g][k] = 0.f;
  }
  for (long long r = r0 + wid; r < r1; r += kPgWarps) {
    const T* src;
    if (r < n_sel) {
      const int j = kHca ? (int)r : sel[r];
      if (j < 0) continue;
      const long long row = j < a.n_max ? page_row(a.pm, b, a.n_max, j) : -1;
      if (row < 0) {
        if (lane == 0) report_error(CSA_ERR_DEVICE_BOUNDS);
        continue;
      }
      src = static_cast<const T*>(a.kv) + row * a.d;
    } else {
      src = static_cast<const T*>(a.kv_raw) +
            ((long long)b * a.raw_max + (w_lo - rp0) + (r - n_sel)) * a.d;
    }
    float rv[NK];
#pragma unroll
    for (int k = 0; k < NK; ++k) rv[k] = to_f32(src[lane + 32 * k]);
#pragma unroll
    for (int g = 0; g < HG; ++g) {
      float dot = 0.f;
#pragma unroll
      for (int k = 0; k < NK; ++k) dot = fmaf(qv[g][k], rv[k], dot);
      const float z = warp_sum(dot) * a.scale;
      const float mn = fmaxf(m[g], z);
      const float alpha = mn == -INFINITY ? 1.f : expf(m[g] - mn);
      // guarded by z itself: the maximum passes a NaN over, the sum keeps it
      const float p = z == -INFINITY ? 0.f : expf(z - mn);
      l[g] = fmaf(l[g], alpha, p);
#pragma unroll
      for (int k = 0; k < NK; ++k) acc[g][k] = fmaf(p, rv[k], acc[g][k] * alpha);
      m[g] = mn;
    }
  }
  if (lane == 0) {
#pragma unroll
    for (int g = 0; g < HG; ++g) {
      sm_m[wid][g] = m[g];
      sm_l[wid][g] = l[g];
    }
  }
#pragma unroll
  for (int g = 0; g < HG; ++g) {
    __syncthreads();  // the last head's sums have been read
#pragma unroll
    for (int k = 0; k < NK; ++k) sm_acc[wid][lane + 32 * k] = acc[g][k];
    __syncthreads();
    if (wid != 0 || h0 + g >= a.H) continue;
    float M = -INFINITY, L = 0.f, o[NK];
    for (int w = 0; w < kPgWarps; ++w) M = fmaxf(M, sm_m[w][g]);
#pragma unroll
    for (int k = 0; k < NK; ++k) o[k] = 0.f;
    for (int w = 0; w < kPgWarps; ++w) {
      const float s = sm_m[w][g] == -INFINITY ? 0.f : expf(sm_m[w][g] - M);
      L = fmaf(sm_l[w][g], s, L);
#pragma unroll
      for (int k = 0; k < NK; ++k) o[k] = fmaf(sm_acc[w][lane + 32 * k], s, o[k]);
    }
    if (a.splits == 1) {
      pg_finish<T, NK>(a, token, h0 + g, M, L, o);
    } else {
      float* part = a.part + (((long long)token * a.H + h0 + g) * a.splits + split) * (a.d + 2);
#pragma unroll
      for (int k = 0; k < NK; ++k) part[lane + 32 * k] = o[k];
      if (lane == 0) {
        part[a.d] = M;
        part[a.d + 1] = L;
      }
    }
  }
}

// One warp per (token, head): the splits joined in their order.
template <typename T, int NK>
__global__ void __launch_bounds__(32) k_attn_paged_join(const __grid_constant__ PagedAttnArgs a) {
  const int h = blockIdx.x, token = blockIdx.y, lane = threadIdx.x;
  const float* part = a.part + ((long long)token * a.H + h) * a.splits * (a.d + 2);
  float M = -INFINITY, L = 0.f, o[NK];
  for (int s = 0; s < a.splits; ++s) M = fmaxf(M, part[(long long)s * (a.d + 2) + a.d]);
#pragma unroll
  for (int k = 0; k < NK; ++k) o[k] = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float* ps = part + (long long)s * (a.d + 2);
    const float ms = ps[a.d];
    const float w = ms == -INFINITY ? 0.f : expf(ms - M);
    L = fmaf(ps[a.d + 1], w, L);
#pragma unroll
    for (int k = 0; k < NK; ++k) o[k] = fmaf(ps[lane + 32 * k], w, o[k]);
  }
  pg_finish<T, NK>(a, token, h, M, L, o);
}

}  // namespace csa
