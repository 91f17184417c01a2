// Shared by the kernels of attention over a paged quantized cache: their
// parameters, the split of a batch into work items, and the rotation of a row
// held by one warp.
#pragma once

#include <cuda_fp16.h>

#include "tq_kernels.h"
#include "tq_sm100.cuh"

namespace tq {

constexpr int kPagedRows = 16;       // query rows (new token x query head of a group) of a work item
constexpr int kPagedMinSplit = 256;  // keys of a work item at least, where a sequence has them

struct PagedParams {
  const void *y;  // 16-bit queries
  int64_t ldy;
  const int32_t *q_start;  // [nseq + 1]
  const int32_t *kv_len;   // [nseq]
  const int32_t *table;    // [nseq][ldt]
  int64_t ldt;
  int64_t total_q;
  int nseq, heads, kv_heads, group, max_new, max_pages, page_size;
  int64_t npages;
  const uint8_t *kcodes, *ksigns, *vcodes;
  const float2 *knorms, *vnorms;
  int bf16;  // queries and output: bf16, else fp16
  float scale;
  uint16_t ck[16], cv[16];  // fp16 centroids
  const uint32_t *kdiag, *vdiag;
  const uint16_t *qjl;  // d x d fp16 (inner-product keys)
  float kappa;
  void *out;
  int64_t ldo;
  int tiles;       // row tiles of a sequence and KV head, at most
  int nsplit;      // key ranges of a sequence, at most
  int target;      // work items wanted
  float *part_o;   // [nseq * kv_heads][max_new * group][nsplit][D], rotated domain
  float2 *part_ml; // same rows: (max, sum) in base 2
  int *splits;     // [nseq]: key ranges in use
};

// Work items of up to 16 rows: one kernel per (D, inner-product keys) file,
// chosen by the code widths of keys and values.
template <int D, bool IP>
tq_status paged_rows_launch(const PagedParams &prm, int wk, int wv, int64_t items, cudaStream_t st);

namespace paged {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float load16(const void *p, int64_t i, int bf16) {
  const uint16_t v = static_cast<const uint16_t *>(p)[i];
  return bf16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ uint16_t store16(float v, int bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// Unnormalized Walsh-Hadamard transform of D values held by one warp, lane l
// having coordinates l * D/32 .. + D/32 - 1.
template <int D>
__device__ __forceinline__ void warp_fwht(float (&v)[D / 32], int lane) {
  constexpr int V = D / 32;
#pragma unroll
  for (int h = 1; h < V; h <<= 1)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (!(i & h)) {
        const float a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float b = __shfl_xor_sync(0xffffffffu, v[i], m);
      v[i] = (lane & m) ? b - v[i] : v[i] + b;
    }
}
template <int D>
__device__ __forceinline__ void warp_signs(float (&v)[D / 32], const uint32_t *words, int lane) {
  constexpr int V = D / 32;
  const uint32_t w = __ldg(words + lane * V / 32) >> (lane * V % 32);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = __uint_as_float(__float_as_uint(v[i]) ^ (((w >> i) & 1u) << 31));
}
// v = R v and v = R^T v, R = H D3 H D2 H D1 d^-1.5
template <int D>
__device__ __forceinline__ void warp_rotate(float (&v)[D / 32], const uint32_t *diag, int lane) {
#pragma unroll
  for (int r = 0; r < 3; ++r) {
    warp_signs<D>(v, diag + r * (D / 32), lane);
    warp_fwht<D>(v, lane);
  }
  const float f = 1.0f / ((float)D * sqrtf((float)D));
#pragma unroll
  for (int i = 0; i < D / 32; ++i) v[i] *= f;
}
template <int D>
__device__ __forceinline__ void warp_rotate_back(float (&v)[D / 32], const uint32_t *diag, int lane) {
#pragma unroll
  for (int r = 2; r >= 0; --r) {
    warp_fwht<D>(v, lane);
    warp_signs<D>(v, diag + r * (D / 32), lane);
  }
  const float f = 1.0f / ((float)D * sqrtf((float)D));
#pragma unroll
  for (int i = 0; i < D / 32; ++i) v[i] *= f;
}

// D/32 consecutive 16-bit values of one row, written by one lane
template <int D>
__device__ __forceinline__ void write_row(void *out, int64_t at, const float (&v)[D / 32], int lane, int bf16) {
  uint16_t h[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) h[i] = store16(v[i], bf16);
  uint16_t *p = static_cast<uint16_t *>(out) + at + lane * (D / 32);
  if constexpr (D == 128)
    *reinterpret_cast<uint2 *>(p) = make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
  else
    *reinterpret_cast<uint32_t *>(p) = h[0] | (uint32_t)h[1] << 16;
}

struct Seq {
  int start, n, len;  // first query token, new tokens, keys that can be read
  int kv;             // keys by kv_len (the causal limit counts from it)
};
__device__ __forceinline__ Seq seq_of(const PagedParams &p, int i) {
  Seq s;
  const int64_t a = min(max((int64_t)__ldg(p.q_start + i), (int64_t)0), p.total_q);
  const int64_t b = min(max((int64_t)__ldg(p.q_start + i + 1), a), p.total_q);
  s.start = (int)a;
  s.n = (int)min(b - a, (int64_t)p.max_new);
  s.kv = max(__ldg(p.kv_len + i), 0);
  s.len = (int)min((int64_t)s.kv, (int64_t)p.max_pages * p.page_size);
  return s;
}

struct Split {
  int keys;   // keys of a range
  int count;  // ranges
};

// The key ranges of a sequence of `len` keys: about `target` work items of
// equal length over the whole batch, at least kPagedMinSplit keys each, at
// most nsplit ranges a sequence, whole multiples of `step` keys.  `work` =
// sum over sequences of keys * row tiles * KV heads.
__device__ __forceinline__ Split split_of(const PagedParams &p, int64_t work, int len, int step) {
  int64_t per = (work + p.target - 1) / p.target;
  per = max(per, (int64_t)kPagedMinSplit);
  per = max(per, (int64_t)(len + p.nsplit - 1) / p.nsplit);
  per = (per + step - 1) / step * step;
  per = min(per, (int64_t)1 << 30);
  Split s;
  s.keys = (int)per;
  s.count = max(1, (int)((len + per - 1) / per));
  return s;
}

}  // namespace paged
}  // namespace tq
