// Shared by the kernels of attention over a paged quantized cache: their
// parameters, how a batch is cut into work, and the rotation of a row held by
// one warp.
#pragma once

#include <cuda_fp16.h>

#include "tq_flash.cuh"
#include "tq_kernels.h"
#include "tq_sm100.cuh"

namespace tq {

// How a batch is cut into work: a sequence's query rows (new token x query
// head of a group, token-major) in blocks of `rows`, each with the keys that
// its last row sees in units of 2^unit keys.  The units of all (sequence, KV
// head, block), in this order, form one line that the kernel's blocks share
// out in equal contiguous runs, whatever the lengths are; a block of rows
// whose units fall to several runs is put together at the end from their
// partial results.  Sequences of more than `above` and at most `upto` rows.
struct PagedCut {
  int rows, unit, above, upto;
  int grid;          // runs
  int least;         // units of a run, at least
  int64_t *first;    // [nseq + 1]: each sequence's first unit (written by the kernel's block 0)
  float *part_o;     // [2 * grid][rows][D]: unnormalized outputs, rotated domain
  float2 *part_ml;   // [2 * grid][rows]: (maximum, sum) in base 2
};

struct PagedParams {
  const void *y;  // 16-bit queries
  int64_t ldy;
  const int32_t *q_start;  // [nseq + 1]
  const int32_t *kv_len;   // [nseq]
  const int32_t *table;    // [nseq][ldt]
  int64_t ldt;
  int64_t total_q;
  int nseq, heads, kv_heads, group, max_new, max_pages, page_size;
  // ceil(2^31 / (page_size / 16)): key / page_size = (key / 16) * 2 * page_magic >> 32 for keys below 2^29 (a page
  // has at most 64 times 16 keys, so the product's excess stays below one)
  uint32_t page_magic;
  __device__ int page_of(int key) const { return (int)__umulhi((uint32_t)key >> 4 << 1, page_magic); }
  int64_t npages;
  const uint8_t *kcodes, *ksigns, *vcodes;
  const float2 *knorms, *vnorms;
  int bf16;  // queries and output: bf16, else fp16
  float scale;
  uint16_t ck[16], cv[16];  // fp16 centroids, in units of kunit and vunit
  float kunit, vunit;
  float ckf[16], cvf[16];   // the same in fp32
  // fp16 centroids of the keys under several factors (many rows, inner-product keys, fp16 queries)
  uint16_t cks[kAttendFactors][8];
  float cks_by[kAttendFactors];
  const uint32_t *kdiag, *vdiag;
  const uint16_t *qjl;  // d x d fp16 (inner-product keys)
  float kappa;
  void *out;
  int64_t ldo;
  // [nseq + 1]: parts of blocks of rows of the sequences before, which the join by parts takes (written by block 0 of
  // the kernel of few rows); null: the join goes by rows
  int64_t *join_first;
  PagedCut few, many;  // for the kernel of few rows and the kernel of many (its grid 0: not launched)
  float *whole;     // [total_q * heads][D]: normalized rows of blocks that one run had whole, rotated domain
  // many: [total_q * heads][D to 3 D] rotated queries, then their projections (inner-product keys), then the
  // rotated queries' low terms (fp16 queries), fp16
  uint16_t *qprep;
  float *qscale;    // many: [total_q * heads] power of two that undoes their scaling
  int *err;
};

// Rows of a block of the kernel of many rows: two query tiles of 128, or one where
// two would leave no room for keys.  low: of fp16 queries
constexpr int paged_tile_rows(int d, bool ip, bool low) { return (ip || low) && d == 128 ? 128 : 256; }

// Few rows: one kernel per (D, inner-product keys) file, chosen by the code
// widths of keys and values.  Many rows: likewise.
template <int D, bool IP>
tq_status paged_rows_launch(const PagedParams &prm, int wk, int wv, cudaStream_t st);
template <int D, bool IP>
tq_status paged_tiles_launch(const PagedParams &prm, int wk, int wv, cudaStream_t st);

namespace paged {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float widen16(uint16_t v, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)v << 16) : __half2float(__ushort_as_half(v));
}
__device__ __forceinline__ float load16(const void *p, int64_t i, int bf16) {
  return widen16(static_cast<const uint16_t *>(p)[i], bf16);
}
__device__ __forceinline__ uint16_t store16(float v, int bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}

// the same with nothing to add to
__device__ __forceinline__ void mma16816_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Parts of a row are added up relative to the largest exponent of weight times
// value norm (flash::Row), where the sum of the weights alone may be as large as
// 2^80 a key and as small as 2^-100.  So a part's sum is multiplied by a root of
// its factor twice, which loses nothing that matters beside the others (a factor
// of 2^-126 or less is 0, and 80 + 100 < 2 * 126).
__device__ __forceinline__ float ex2_half(float x) { return ex2(0.5f * x); }
// Power of two above v (v >= 0), kept where its reciprocal is normal too
__device__ __forceinline__ float pow2_above(float v) {
  const uint32_t e = (__float_as_uint(v) >> 23) + 1u;  // biased exponent, one up
  return __uint_as_float(min(max(e, 2u), 252u) << 23);
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

// The same for a row held by one thread: no data moves between threads, so
// where there are rows for every thread a transform costs a fifth of the
// warp's.  The three rounds are one loop (code of one round: 2 KB at D = 64).
template <int D>
__device__ __forceinline__ void thread_fwht(float (&v)[D]) {
#pragma unroll
  for (int h = 1; h < D; h <<= 1)
#pragma unroll
    for (int i = 0; i < D; ++i)
      if (!(i & h)) {
        const float a = v[i], b = v[i + h];
        v[i] = a + b;
        v[i + h] = a - b;
      }
}
template <int D>
__device__ __forceinline__ void thread_signs(float (&v)[D], const uint32_t *words) {
#pragma unroll
  for (int g = 0; g < D / 32; ++g) {
    const uint32_t w = __ldg(words + g);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      v[32 * g + i] = __uint_as_float(__float_as_uint(v[32 * g + i]) ^ ((w << (31 - i)) & 0x80000000u));
  }
}
template <int D>
__device__ __forceinline__ void thread_rotate(float (&v)[D], const uint32_t *diag) {
#pragma unroll 1
  for (int r = 0; r < 3; ++r) {
    thread_signs<D>(v, diag + r * (D / 32));
    thread_fwht<D>(v);
  }
  const float f = 1.0f / ((float)D * sqrtf((float)D));
#pragma unroll
  for (int i = 0; i < D; ++i) v[i] *= f;
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
  int start, n, len;  // first query token, new tokens (at most max_new), keys that can be read
  // keys that the first new token sees, by kv_len and all new tokens of the
  // sequence, those that max_new or total_q leaves out among them; may be below 1
  int first;
};
__device__ __forceinline__ Seq seq_of(const PagedParams &p, int i) {
  Seq s;
  const int64_t a = min(max((int64_t)__ldg(p.q_start + i), (int64_t)0), p.total_q);
  const int64_t end = __ldg(p.q_start + i + 1), b = min(max(end, a), p.total_q);
  s.start = (int)a;
  s.n = (int)min(b - a, (int64_t)p.max_new);
  const int kv = max(__ldg(p.kv_len + i), 0);
  s.first = (int)(kv - (end - a) + 1);
  s.len = (int)min((int64_t)kv, (int64_t)p.max_pages * p.page_size);
  return s;
}

__device__ __forceinline__ int blocks_of(const PagedParams &p, const PagedCut &c, const Seq &s) {
  const int rows = s.n * p.group;
  return rows > c.above && rows <= c.upto ? (rows + c.rows - 1) / c.rows : 0;
}
// Keys that the last row of block k sees (the first of its rows may see fewer)
__device__ __forceinline__ int seen_by(const PagedParams &p, const PagedCut &c, const Seq &s, int k) {
  const int last = min((k + 1) * c.rows, s.n * p.group) - 1;
  return max(0, min(s.len, s.first + last / p.group));
}
__device__ __forceinline__ int units_of(const PagedParams &p, const PagedCut &c, const Seq &s, int k) {
  return (seen_by(p, c, s, k) + (1 << c.unit) - 1) >> c.unit;
}
__device__ __forceinline__ int64_t head_units(const PagedParams &p, const PagedCut &c, const Seq &s) {
  int64_t u = 0;
  for (int k = 0, n = blocks_of(p, c, s); k < n; ++k) u += units_of(p, c, s, k);
  return u;
}
// a / b of non-negative numbers, nearly always of 32 bits (a 64-bit division takes a microsecond)
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}
__device__ __forceinline__ int64_t run_units(const PagedCut &c, int64_t total) {
  return max(divide(total + c.grid - 1, c.grid), (int64_t)c.least);
}

// Where a run stands: the units [unit, unit + take) of a block of rows.
struct Cursor {
  int seq, head, block, unit, take;
  int units;     // of the block
  int64_t left;  // units of the run from here on
  Seq s;

  __device__ bool whole() const { return take == units; }
  // partial results of a block that this run has in part: a run has at most
  // two such blocks, one that began before it and one that goes on behind it
  __device__ int slot() const { return 2 * (int)blockIdx.x + (unit == 0 ? 1 : 0); }
  __device__ void load(const PagedParams &p, const PagedCut &c) {
    units = units_of(p, c, s, block);
    take = (int)min((int64_t)(units - unit), left);
  }
  // the next block of rows with units; false at the end of the run
  __device__ bool next(const PagedParams &p, const PagedCut &c) {
    left -= take;
    if (left <= 0) return false;
    unit = 0;
    for (;;) {
      if (++block >= blocks_of(p, c, s)) {
        block = 0;
        if (++head >= p.kv_heads) {
          head = 0;
          do {
            if (++seq >= p.nseq) return false;
            s = seq_of(p, seq);
          } while (blocks_of(p, c, s) == 0);
        }
      }
      load(p, c);
      if (units > 0) return true;
    }
  }
};

// The join takes blocks of rows in parts of up to kJoinRows rows
constexpr int kJoinRows = 16;
__device__ __forceinline__ int parts_of(const PagedCut &c) { return (c.rows + kJoinRows - 1) / kJoinRows; }

// Sums of join parts over the sequences, by one warp
__device__ __forceinline__ void sum_parts(const PagedParams &p) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0;
  for (int i0 = 0; i0 < p.nseq; i0 += 32) {
    int64_t n = 0;
    if (i0 + lane < p.nseq) {
      const Seq s = seq_of(p, i0 + lane);
      n = (int64_t)(s.n * p.group <= p.few.upto ? blocks_of(p, p.few, s) * parts_of(p.few)
                                                : blocks_of(p, p.many, s) * parts_of(p.many)) * p.kv_heads;
    }
    int64_t in = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t b = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += b;
    }
    if (i0 + lane < p.nseq) p.join_first[i0 + lane] = total + in - n;
    total += __shfl_sync(0xffffffffu, in, 31);
  }
  if (lane == 0) p.join_first[p.nseq] = total;
}

// The start of this block's run, found by one warp (block 0's also writes
// c.first): sequence, head, block, unit and units of the run; false if there
// is none.
__device__ __forceinline__ bool find_run(const PagedParams &p, const PagedCut &c, int64_t *found) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0;
  for (int i0 = 0; i0 < p.nseq; i0 += 32) {
    const int64_t u = i0 + lane < p.nseq ? head_units(p, c, seq_of(p, i0 + lane)) * p.kv_heads : 0;
    int64_t in = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t b = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += b;
    }
    if (blockIdx.x == 0 && i0 + lane < p.nseq) c.first[i0 + lane] = total + in - u;
    total += __shfl_sync(0xffffffffu, in, 31);
  }
  if (blockIdx.x == 0 && lane == 0) c.first[p.nseq] = total;
  const int64_t per = run_units(c, total), from = per * blockIdx.x;
  if (from >= total) return false;
  int64_t before = 0;
  for (int i0 = 0; i0 < p.nseq; i0 += 32) {
    Seq s{};
    int64_t hu = 0;
    if (i0 + lane < p.nseq) {
      s = seq_of(p, i0 + lane);
      hu = head_units(p, c, s);
    }
    int64_t in = hu * p.kv_heads;
    const int64_t u = in;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t b = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += b;
    }
    const int64_t at = from - (before + in - u);
    if (u > 0 && at >= 0 && at < u) {
      const int64_t head = divide(at, hu);
      int64_t rest = at - head * hu;
      int k = 0;
      for (;; ++k) {
        const int n = units_of(p, c, s, k);
        if (rest < n) break;
        rest -= n;
      }
      found[0] = i0 + lane;
      found[1] = head;
      found[2] = k;
      found[3] = rest;
      found[4] = min(per, total - from);
    }
    before += __shfl_sync(0xffffffffu, in, 31);
    if (before > from) break;
  }
  return true;
}
__device__ __forceinline__ Cursor start_run(const PagedParams &p, const PagedCut &c, const int64_t *found) {
  Cursor u;
  u.seq = (int)found[0];
  u.head = (int)found[1];
  u.block = (int)found[2];
  u.unit = (int)found[3];
  u.left = found[4];
  u.s = seq_of(p, u.seq);
  u.load(p, c);
  return u;
}

}  // namespace paged
}  // namespace tq
