// Microscaled 4-bit floating point (OCP Microscaling Formats v1.0, MXFP4):
// blocks of 32 values share a power-of-two scale held as one E8M0 byte, the
// values are E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two
// to a byte, the even dim in the low half.
//
//   scale byte  max(E(max|x|) - 2, 0), E the fp32 exponent field: the scale
//               is 2^(floor(log2 max|x|) - 2), not below 2^-127; 127 (a scale
//               of 1) for a block of zeros; 255 (NaN) for a block that holds
//               an infinity or a NaN, with codes 0
//   code        x / scale to the nearest E2M1 value, ties to the even code,
//               past 6 to 6 (max|x| / scale lies in [4, 8))
//
// x / scale is exact in fp32 (a power of two; a result small enough to lose
// bits rounds to code 0 either way), so the codes depend on no rounding but
// their own.
//
// Quantizer.  A lane takes 8 values (16 bytes of bf16, 32 of fp32), four
// neighbouring lanes a block: two shuffles give the block's maximum, one
// conversion instruction packs each pair of values.  524,256 keys of 128 into
// random rows, values written too: fp32 94 us, 6.1 TB/s, 93% of the copy rate
// (HBM-bound); bf16 63 us, 4.8 TB/s, 74%, with 72% of the issue slots busy: the
// same instructions over half the bytes.  Two such pieces per thread (bf16:
// 66.5 us with one, 78 with four).  The 4-byte scale rows, each a part of a
// 32-byte sector, do not show: fp32 writes the same ones, and nothing is read
// to fill sectors (136 MB read where rows and slots are 136).
#pragma once
#include "common.cuh"
#include "quantize.cuh"

namespace csa {

constexpr int kMxThreads = 256;
constexpr int kMxNaN = 255;

// Eight fp32 values to eight E2M1 codes, the first in the lowest four bits
// (nearest, ties to even, past 6 to 6).
__device__ __forceinline__ uint32_t mx_pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The values of eight codes.
__device__ __forceinline__ void mx_unpack8(uint32_t c, float (&v)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
    v[2 * k] = f.x;
    v[2 * k + 1] = f.y;
  }
}

// The value of a scale byte: 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float mx_scale(int byte) {
  if (byte == kMxNaN) return __int_as_float(0x7fc00000);
  return __int_as_float(byte == 0 ? 0x00400000 : byte << 23);
}

__device__ __forceinline__ void mx_store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void mx_store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Rows [0, n) of d values (row i at rows + i * row_stride) to the codes and
// scales of row slots[i] (i without slots); `values` (nullable) receives the
// values that the codes stand for, row i dense.  i0: first row of this launch.
template <typename T, int PER>
__global__ void __launch_bounds__(kMxThreads)
    k_quantize_mxfp4(const T* __restrict__ rows, long long row_stride, unsigned n, unsigned cpr,
                     const int32_t* __restrict__ slots, long long i0, long long out_rows,
                     uint8_t* __restrict__ codes, uint8_t* __restrict__ scales,
                     T* __restrict__ values) {
  unsigned r[PER], k[PER];
  int slot[PER];
  float v[PER][8];
#pragma unroll
  for (int p = 0; p < PER; ++p) {  // PER chunks of 8 values, all loads first
    const unsigned chunk = (blockIdx.x * PER + p) * kMxThreads + threadIdx.x;
    r[p] = chunk / cpr;
    k[p] = chunk - r[p] * cpr;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[p][e] = 0.f;
    slot[p] = 0;
    if (r[p] < n) {
      load8(rows + (long long)r[p] * row_stride + 8 * k[p], v[p]);
      if (slots != nullptr) slot[p] = slots[i0 + r[p]];
    }
  }
#pragma unroll
  for (int p = 0; p < PER; ++p) {
    // the largest magnitude as an integer: NaN and infinity sort above all
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[p][e]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    if (r[p] >= n) continue;  // the four lanes of a block agree: cpr is a multiple of 4
    const int field = (int)(top >> 23);
    const bool bad = field == 255;
    const int byte = top == 0 ? 127 : (bad ? kMxNaN : max(field - 2, 0));
    const float inv = bad ? 0.f : __int_as_float((254 - byte) << 23);  // 1 / scale
    uint32_t c = 0;
    if (!bad) {
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = v[p][e] * inv;
      c = mx_pack8(q);
    }
    const long long row = i0 + r[p];
    if (values != nullptr) {
      float q[8];
      mx_unpack8(c, q);
      const float s = mx_scale(byte);
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] *= s;
      mx_store8(values + row * (long long)cpr * 8 + 8 * k[p], q);
    }
    long long o = row;
    if (slots != nullptr) {
      if (slot[p] < 0 || slot[p] >= out_rows) {
        if (slot[p] != -1 && k[p] == 0) report_error(CSA_ERR_DEVICE_BOUNDS);
        continue;
      }
      o = slot[p];
    }
    reinterpret_cast<uint32_t*>(codes)[o * cpr + k[p]] = c;
    if ((k[p] & 3) == 0) scales[o * (cpr >> 2) + (k[p] >> 2)] = (uint8_t)byte;
  }
}

// ---------------------------------------------------------------------------
// Paged caches: sequence b's entry j is row page_table[b][j / page] * page +
// j % page of the pool.  A table entry outside the pool is reported and its
// rows are skipped.
struct PageMap {
  const int32_t* table;  // [B][width]; NULL: sequence b's entries are rows b * n_max + j
  int width;             // pages per sequence in the table
  int shift;             // log2 of the page size
  int n_pages;           // pages in the pool
};

// Pool row of entry j of sequence b, -1 when its page is not in the pool.
__device__ __forceinline__ long long page_row(const PageMap& pm, int b, int n_max, int j) {
  if (pm.table == nullptr) return (long long)b * n_max + j;
  const int page = pm.table[(long long)b * pm.width + (j >> pm.shift)];
  if ((unsigned)page >= (unsigned)pm.n_pages) return -1;
  return ((long long)page << pm.shift) + (j & ((1 << pm.shift) - 1));
}

// A warp's view of one sequence's page table: 32 entries, one per lane, and
// the next 32 already asked for, so that walking a sequence in order waits for
// the table once, not at every new line of it.  Entries past the last needed
// page are not read.
struct PageWindow {
  const int32_t* row;  // the sequence's table row
  int last;            // pages that may be read
  int w;               // window held in `cur`
  int cur, nxt;
  __device__ __forceinline__ int load(int win) const {
    const int p = win * 32 + (int)(threadIdx.x & 31);
    return p < last ? row[p] : -1;
  }
  // every lane; n: entries of the sequence that will be looked up; page0: first page
  __device__ __forceinline__ void start(const PageMap& pm, int b, int n, int page0) {
    row = pm.table + (long long)b * pm.width;
    last = (int)(((long long)n + (1 << pm.shift) - 1) >> pm.shift);
    w = page0 >> 5;
    cur = load(w);
    nxt = load(w + 1);
  }
  // every lane: make the window that holds `page` current (pages only rise)
  __device__ __forceinline__ void seek(int page) {
    while (w < (page >> 5)) {
      cur = nxt;
      ++w;
      nxt = load(w + 1);
    }
  }
  // every lane: the table entry of this lane's page, which lies in the window
  __device__ __forceinline__ int at(int page) const { return __shfl_sync(0xffffffffu, cur, page & 31); }
};

// Indexer scores on CUDA cores, any head count and dim: one key per thread,
// the query's dequantized heads and weights in shared memory, 16 heads at a
// time, 32 dims (one scale) of the key in registers.  Bound by its multiply-adds
// and their reads of shared memory: 32 x 16,383 keys under 32 heads of 128, or 64
// of 64, 240 us (18 TFLOP/s).
__global__ void __launch_bounds__(128)
    k_index_scores_mx_simt(const uint8_t* __restrict__ q_codes, const uint8_t* __restrict__ q_scales,
                           const float* __restrict__ w, const uint8_t* __restrict__ k_codes,
                           const uint8_t* __restrict__ k_scales, PageMap pm,
                           const int* __restrict__ q_pos, const int* __restrict__ n_cmp, int Tq,
                           int n_max, int H_I, int d_I, int width, int stride,
                           float* __restrict__ scores) {
  extern __shared__ float smem[];
  float* qs = smem;              // [H_I][d_I]
  float* ws = smem + H_I * d_I;  // [H_I]
  const int b = blockIdx.z, t = blockIdx.y;
  const long long row = (long long)b * Tq + t;
  const int nv = min(n_visible(q_pos[row], n_cmp[b], width, stride), n_max);
  const int j0 = blockIdx.x * 128;
  if (j0 >= nv) return;
  const int chunks = H_I * d_I / 8;
  for (int i = threadIdx.x; i < chunks; i += 128) {
    float v[8];
    mx_unpack8(reinterpret_cast<const uint32_t*>(q_codes)[row * chunks + i], v);
    const float s = mx_scale(q_scales[(row * chunks + i) / 4]);
#pragma unroll
    for (int e = 0; e < 8; ++e) qs[8 * i + e] = v[e] * s;
  }
  for (int i = threadIdx.x; i < H_I; i += 128) ws[i] = w[row * H_I + i];
  __syncthreads();
  const int j = j0 + (int)threadIdx.x;
  if (j >= nv) return;
  const long long kr = page_row(pm, b, n_max, j);
  if (kr < 0) {
    report_error(CSA_ERR_DEVICE_BOUNDS);
    return;
  }
  const uint4* key = reinterpret_cast<const uint4*>(k_codes + kr * (d_I / 2));
  const uint8_t* ksc = k_scales + kr * (d_I / 32);
  float score = 0.f;
  for (int h0 = 0; h0 < H_I; h0 += 16) {
    const int nh = min(16, H_I - h0);
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    for (int kb = 0; kb < d_I / 32; ++kb) {
      const uint4 u = key[kb];
      const float s = mx_scale(ksc[kb]);
      const uint32_t cw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float kv[8];
        mx_unpack8(cw[g], kv);
#pragma unroll
        for (int e = 0; e < 8; ++e) kv[e] *= s;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i < nh) {
            const float* qp = qs + (h0 + i) * d_I + kb * 32 + g * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[i] = fmaf(qp[e], kv[e], acc[i]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < nh) {
        const float r = acc[i] < 0.f ? 0.f : acc[i];  // a NaN stays
        score = fmaf(ws[h0 + i], r, score);
      }
    }
  }
  scores[row * n_max + j] = score;
}

}  // namespace csa
