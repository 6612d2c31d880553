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
#pragma once
#include "common.cuh"
#include "compress.cuh"
#include "sm100.cuh"

namespace csa {

constexpr int kNormThreads = 256;
constexpr int kNormMaxPairs = 512;  // RoPE pairs in the table (rope_dim <= 1024)

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
  double freq[kNormMaxPairs];
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

template <typename T, int NV>
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

  // the first head's values are in flight while the table is formed
  float v[NV][VEC];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c0 = (lane + n * G) * VEC;
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[n][k] = 0.f;
    if (nh > 0 && c0 < dim) load16(src + c0, v[n]);
  }
  float w[NV][VEC], cs[NV][VEC / 2], sn[NV][VEC / 2];
  const bool rot = sd.pos != nullptr;
  const int pos = rot ? sd.pos[row] : 0;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    const int c0 = (lane + n * G) * VEC;
#pragma unroll
    for (int k = 0; k < VEC; ++k) w[n][k] = sd.weight != nullptr && c0 < dim ? sd.weight[c0 + k] : 1.f;
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      const int c = c0 + 2 * k;
      cs[n][k] = 1.f;
      sn[n][k] = 0.f;
      if (rot && c >= rope0 && c < dim) norm_cos_sin(pos, a.freq[(c - rope0) >> 1], &cs[n][k], &sn[n][k]);
    }
  }
  const float inv_dim = 1.f / (float)dim;
  // every lane of the warp makes the same number of turns (the shuffles)
  const int turns = sd.hpg;
  for (int h = 0; h < turns; ++h) {
    float nx[NV][VEC];
#pragma unroll
    for (int n = 0; n < NV; ++n) {  // the next head's values
      const int c0 = (lane + n * G) * VEC;
#pragma unroll
      for (int k = 0; k < VEC; ++k) nx[n][k] = 0.f;
      if (h + 1 < nh && c0 < dim) load16(src + (h + 1) * dim + c0, nx[n]);
    }
    float ss = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < VEC; ++k) ss = fmaf(v[n][k], v[n][k], ss);
    for (int o = G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float inv = __frsqrt_rn(fmaf(ss, inv_dim, a.eps));
#pragma unroll
    for (int n = 0; n < NV; ++n) {
      const int c0 = (lane + n * G) * VEC;
      float y[VEC];
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k) {
        const float p = v[n][2 * k] * inv * w[n][2 * k];
        const float q = v[n][2 * k + 1] * inv * w[n][2 * k + 1];
        const bool in = rot && c0 + 2 * k >= rope0;
        y[2 * k] = in ? p * cs[n][k] - q * sn[n][k] : p;
        y[2 * k + 1] = in ? p * sn[n][k] + q * cs[n][k] : q;
      }
      if (store_ok && h < nh && c0 < dim) store16(dst + h * dim + c0, y);
    }
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[n][k] = nx[n][k];
  }
}

}  // namespace csa
