// RMS norm of every query and key head with the partial RoPE in the same
// pass: for a head row x of token r,
//   y = x / sqrt(mean(x^2) + eps) * weight,
// then the trailing rope_dim dims of y are rotated in interleaved pairs by
// pos[r] * f_i.  Query rows go to a dense array, key rows to the rows of a
// (paged) cache that a slot list names.
//
// HBM-bound: each value is read once and written once.  A group of G lanes
// (a power of two, 16 bytes per lane and vector) holds one head row in
// registers, so the sum of squares is a shuffle reduction and the row is
// rotated and stored from the same registers.  A group takes several heads
// of ONE token: its lanes cover the same dims in each, so the weights and
// the sines and cosines are formed once per group and stay in registers.
// Queries and keys share the launch (the key blocks follow the query
// blocks).  Sums are fp32; the angle is reduced in double precision.
//
// Heads per group: 1 while the rows are few (a decode step's 2,048 heads of
// 128: 4.2 us, a launch and one trip to memory), up to 32 while the groups
// still fill the GPU 16 times: 8,192 tokens x 128 heads of 512 in bf16 take 377
// us, 5.7 TB/s, 87% of the copy rate (388 on one box; 432 us with 8 heads a
// group, 392 with 16; the sines are then formed for fewer groups), 8,192 x 128
// heads of 128 in fp32 176 us (94%), 8,192 x 32 of 512 in fp32, one head at a
// time, 193 us (88%).  Two heads a turn keep two rows in flight and overlap
// their shuffles: 890 -> 426 us together with holding the next rows as loaded
// (16 bytes) instead of converted.
#pragma once
#include "common.cuh"
#include "compress.cuh"
#include "sm100.cuh"

namespace csa {

constexpr int kNormThreads = 256;
constexpr int kNormTable = 64;  // RoPE pairs whose frequencies come with the launch

// One side (queries or keys) of the call.
struct NormSide {
  const void* x;      // row r, head h at x + r * row_stride + h * dim
  long long row_stride;
  const float* weight;  // [dim] (NULL: ones)
  const int32_t* pos;   // [rows] (NULL: no rotation)
  const int32_t* slots;  // [rows] (NULL: row r goes to row r)
  void* out;             // [out_rows][heads][dim]
  int rows, heads, out_rows;
  int hpg;      // heads per group
  int hgroups;  // groups per token
  int blocks;   // CTAs of this side
};

struct NormRopeArgs {
  NormSide side[2];
  int dim, rope_dim;
  int group;  // lanes per head row, a power of two
  float eps;
  RopeSpec rope;  // for pairs past the table
  double freq[kNormTable];
};

// cos / sin of pos * freq to fp32 accuracy: the angle in half turns is
// reduced to [-1, 1] in double precision (error about 1e-16 of it), and what
// rounding it to fp32 drops is put back to first order.
__device__ __forceinline__ void norm_cos_sin(long long pos, double freq, float* c, float* s) {
  const double turns = (double)pos * freq * 0.15915494309189535;
  const double half = 2.0 * (turns - rint(turns));
  const float hi = (float)half, lo = 3.14159265f * (float)(half - (double)hi);
  float sh, ch;
  sincospif(hi, &sh, &ch);
  *s = fmaf(ch, lo, sh);
  *c = fmaf(-sh, lo, ch);
}

__device__ __forceinline__ void norm_values(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void norm_values(uint4 u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x);
  v[1] = __uint_as_float(u.y);
  v[2] = __uint_as_float(u.z);
  v[3] = __uint_as_float(u.w);
}

template <typename T, int NV, int kRows>
__global__ void __launch_bounds__(kNormThreads) k_norm_rope(const __grid_constant__ NormRopeArgs a) {
  constexpr int VEC = 16 / (int)sizeof(T);
  sm100::griddep_wait();
  sm100::griddep_launch_dependents();
  const int which = (int)blockIdx.x >= a.side[0].blocks ? 1 : 0;
  const NormSide& sd = a.side[which];
  const int block = (int)blockIdx.x - (which ? a.side[0].blocks : 0);
  const int G = a.group;
  const int lane = (int)threadIdx.x & (G - 1);
  const long long gid = (long long)block * (kNormThreads / G) + threadIdx.x / G;
  const long long tok = gid / sd.hgroups;
  const int h0 = (int)(gid - tok * sd.hgroups) * sd.hpg;
  // a group past the end still takes part in its warp's shuffles
  const bool live = tok < sd.rows;
  const int row = live ? (int)tok : 0;
  const int nh = live ? min(sd.hpg, sd.heads - h0) : 0;
  long long orow = row;
  bool store_ok = live;
  if (live && sd.slots != nullptr) {
    const int slot = sd.slots[row];
    store_ok = slot >= 0 && slot < sd.out_rows;
    if (!store_ok && slot != -1 && h0 == 0 && lane == 0) report_error(CSA_ERR_DEVICE_BOUNDS);
    orow = store_ok ? slot : 0;
  }
  const int dim = a.dim;
  const int rope0 = dim - a.rope_dim;
  const T* src = static_cast<const T*>(sd.x) + (long long)row * sd.row_stride + (long long)h0 * dim;
  T* dst = static_cast<T*>(sd.out) + (orow * sd.heads + h0) * (long long)dim;

  // kRows heads at a time, the next ones' values in flight as loaded
  uint4 nx[kRows][NV];
  auto fetch = [&](int h) {
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int c0 = (lane + n * G) * VEC;
        nx[r][n] = make_uint4(0u, 0u, 0u, 0u);
        if (h + r < nh && c0 < dim)
          nx[r][n] = __ldg(reinterpret_cast<const uint4*>(src + (long long)(h + r) * dim + c0));
      }
  };
  fetch(0);
  float w[NV][VEC], cs[NV][VEC / 2], sn[NV][VEC / 2];
  const bool rot = sd.pos != nullptr;
  const int pos = rot ? sd.pos[row] : 0;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c0 = (lane + n * G) * VEC;
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
      float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
      if (sd.weight != nullptr && c0 < dim) f = __ldg(reinterpret_cast<const float4*>(sd.weight + c0 + k));
      w[n][k] = f.x;
      w[n][k + 1] = f.y;
      w[n][k + 2] = f.z;
      w[n][k + 3] = f.w;
    }
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      const int c = c0 + 2 * k;
      cs[n][k] = 1.f;
      sn[n][k] = 0.f;
      if (rot && c >= rope0 && c < dim) {
        const int i = (c - rope0) >> 1;
        norm_cos_sin(pos, i < kNormTable ? a.freq[i] : rope_freq(a.rope, i), &cs[n][k], &sn[n][k]);
      }
    }
  }
  const float inv_dim = 1.f / (float)dim;
  // every lane of the warp makes the same number of turns (the shuffles)
  const int turns = sd.hpg;
  for (int h = 0; h < turns; h += kRows) {
    float v[kRows][NV][VEC], ss[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      ss[r] = 0.f;
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        norm_values(nx[r][n], v[r][n]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) ss[r] = fmaf(v[r][n][k], v[r][n][k], ss[r]);
      }
    }
    if (h + kRows < turns) fetch(h + kRows);
    for (int o = G >> 1; o > 0; o >>= 1) {
#pragma unroll
      for (int r = 0; r < kRows; ++r) ss[r] += __shfl_xor_sync(0xffffffffu, ss[r], o);
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float inv = __frsqrt_rn(fmaf(ss[r], inv_dim, a.eps));
#pragma unroll
      for (int n = 0; n < NV; ++n) {
        const int c0 = (lane + n * G) * VEC;
        float y[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) y[k] = v[r][n][k] * inv * w[n][k];
        if (rot && (n + 1) * G * VEC > rope0) {  // some lane's dims turn (the others' by 1)
#pragma unroll
          for (int k = 0; k < VEC; k += 2) {
            const float p = y[k], q = y[k + 1];
            y[k] = p * cs[n][k / 2] - q * sn[n][k / 2];
            y[k + 1] = p * sn[n][k / 2] + q * cs[n][k / 2];
          }
        }
        if (store_ok && h + r < nh && c0 < dim) store16(dst + (long long)(h + r) * dim + c0, y);
      }
    }
  }
}

}  // namespace csa
