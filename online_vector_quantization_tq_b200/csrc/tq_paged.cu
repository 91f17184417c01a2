// A quantized KV cache kept in pages: storing encoded rows by slot, and
// causal attention of new tokens over the pages (TurboQuant article 4.1.1:
// the cache's keys and values are both quantized).
//
// A page holds page_size tokens of every KV head, head by head: row
// (page * kv_heads + head) * page_size + offset of each packed array.  The
// row layouts are tq_encode's.
//
// Attention.  With the keys' rotation R and the values' rotation Q,
//
//   x_k = scale ||k|| (<R y, c[code_k]> + gamma_k sqrt(pi/2)/d <S R y, +-1_k>)
//   o   = Q^T sum_k softmax_k(x) ||v_k|| c_v[code_k],
//
// the second term of x only for inner-product keys.  The queries are rotated
// once, the output is rotated back once, and in between every packed row is
// read once and expanded into fp16 MMA operands in registers.
#include <algorithm>

#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {

namespace {

using namespace paged;

// ---------------------------------------------------------------- store

struct StoreArray {
  const uint8_t *src;
  uint8_t *dst;
  int row;  // bytes of a row, a multiple of 4 (0: absent)
};
struct StoreParams {
  StoreArray a[6];  // codes, signs, norms of the keys, then of the values
  const int64_t *slots;
  int64_t tokens, slots_total;  // npages * page_size
  int kv_heads, page_size;
  int words;  // 32-bit words of all six rows together
};

// One thread moves one 32-bit word of one (token, head): the six rows of a
// (token, head) are neighbours in the index, so a warp reads whole rows.
__global__ void __launch_bounds__(256) k_paged_store(const StoreParams p) {
  const int64_t n = p.tokens * p.kv_heads * p.words;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = i / p.words;  // token * kv_heads + head
    int w = (int)(i - row * p.words);
    const int64_t token = row / p.kv_heads;
    const int head = (int)(row - token * p.kv_heads);
    const int64_t slot = p.slots[token];
    if (slot < 0 || slot >= p.slots_total) continue;
    const int64_t page = slot / p.page_size;
    const int64_t to = (page * p.kv_heads + head) * p.page_size + (slot - page * p.page_size);
#pragma unroll
    for (int k = 0; k < 6; ++k) {
      const int rw = p.a[k].row >> 2;
      if (w >= 0 && w < rw)
        reinterpret_cast<uint32_t *>(p.a[k].dst + to * p.a[k].row)[w] =
            __ldg(reinterpret_cast<const uint32_t *>(p.a[k].src + row * p.a[k].row) + w);
      w -= rw;
    }
  }
}

// ---------------------------------------------------------------- queries

// Rotated queries (and their projections) of all rows as fp16 operands of the
// kernel of many rows: row (token * heads + head) is R y / U, and for
// inner-product keys S R y / (64 U) behind it, U a power of two above the row's
// largest coordinate, which goes to qscale.  Coordinates stand where the
// expansion of packed codes and signs puts them.  16 rows a block.
template <int D, bool IP>
__global__ void __launch_bounds__(128) k_paged_queries(const __grid_constant__ PagedParams p, int w) {
  constexpr int V = D / 32, DQ = IP ? 2 * D : D;
  __shared__ __align__(16) uint16_t yh[IP ? 16 * D : 1], yl[IP ? 16 * D : 1];
  __shared__ __align__(16) uint16_t stage[16 * DQ];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * 16, total = p.total_q * p.heads;
  float v[4][V];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * warp + i;
    const bool there = row < total;
    const int64_t at = there ? row / p.heads * p.ldy + row % p.heads * D + lane * V : 0;
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] = there ? load16(p.y, at + e, p.bf16) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) warp_rotate<D>(v[i], p.kdiag, lane);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * warp + i;
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) top = fmaxf(top, fabsf(v[i][e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float up = pow2_above(top), down = 1.0f / up;
    if (lane == 0 && row0 + r < total) p.qscale[row0 + r] = up;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int j = lane * V + e;
      const float x = v[i][e] * down;
      const __half hi = __float2half_rn(x);
      stage[r * DQ + (w == 1 ? j / 32 * 32 + 8 * (j % 4) + j % 32 / 4 : j)] = __half_as_ushort(hi);
      if constexpr (IP) {
        yh[r * D + j] = __half_as_ushort(hi);
        yl[r * D + j] = __half_as_ushort(__float2half_rn(x - __half2float(hi)));
      }
    }
  }
  __syncthreads();
  if constexpr (IP) {
    // p = S y~ with y~ as two fp16 terms; warp w has the 8-column tiles w, w + 4, ..
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = warp; t < D / 8; t += 4) {
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      const uint32_t *srow = reinterpret_cast<const uint32_t *>(p.qjl + (t * 8 + r) * D);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t b0 = __ldg(srow + 8 * k + c), b1 = __ldg(srow + 8 * k + c + 4);
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          const uint32_t *ya = reinterpret_cast<const uint32_t *>((term ? yl : yh) + r * D + 16 * k) + c;
          const uint32_t a[4] = {ya[0], ya[8 * (D / 2)], ya[4], ya[8 * (D / 2) + 4]};
          mma16816(acc, a, b0, b1);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = t * 8 + 2 * c + (e & 1), b = j % 32;  // bits k and k + 16 of a word are neighbours
        stage[(r + 8 * (e >> 1)) * DQ + D + j / 32 * 32 + (b < 16 ? 2 * b : 2 * (b - 16) + 1)] =
            __half_as_ushort(__float2half_rn(acc[e] * (1.0f / 64.0f)));
      }
    }
    __syncthreads();
  }
  const int64_t n = min((int64_t)16, total - row0) * (DQ / 8);
  uint4 *to = reinterpret_cast<uint4 *>(p.qprep + row0 * DQ);
  for (int i = tid; i < n; i += 128) to[i] = reinterpret_cast<const uint4 *>(stage)[i];
}

// ---------------------------------------------------------------- join

// Where the result of a token's rows lies: what all heads of it share
struct Place {
  bool there;       // the token belongs to a sequence
  Seq s;
  const PagedCut *c;
  int row0;         // the token's first row in its sequence's KV head
  int64_t units0;   // first unit of KV head 0's block
  int64_t head_units, per;
  int units;        // of the block
};
// By one warp
__device__ __forceinline__ Place find_token(const PagedParams &p, int64_t token) {
  const int lane = threadIdx.x & 31;
  // the last sequence that starts at or before the token
  int lo = 0, hi = p.nseq;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__ldg(p.q_start + mid) <= token)
      lo = mid;
    else
      hi = mid;
  }
  Place f{};
  f.s = seq_of(p, lo);
  f.there = token >= f.s.start && token < f.s.start + f.s.n;
  if (!f.there) return f;
  const PagedCut &c = f.s.n * p.group <= p.few.upto ? p.few : p.many;
  f.c = &c;
  f.row0 = (int)(token - f.s.start) * p.group;
  f.per = run_units(c, __ldg(c.first + p.nseq));
  for (int k = lane, n = blocks_of(p, c, f.s); k < n; k += 32) f.head_units += units_of(p, c, f.s, k);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) f.head_units += __shfl_xor_sync(0xffffffffu, f.head_units, o);
  f.units0 = __ldg(c.first + lo);
  return f;
}

// Output rows from the normalized rows of whole blocks, or from the partial
// results of the runs that share a block (added up in their order), rotated
// back.  A block of threads takes a token's heads, a warp each; or, where rows
// are few and shared by many runs, one row with WARPS warps that take its runs
// in turn, so that their loads overlap.
template <int D, int WARPS>
__global__ void __launch_bounds__(128) k_attend_paged_join(const __grid_constant__ PagedParams p) {
  constexpr int V = D / 32;
  __shared__ float s_v[4][D], s_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token = WARPS == 1 ? blockIdx.x : blockIdx.x / p.heads;
  const Place f = find_token(p, token);
  if (!f.there) return;
  const PagedCut &c = *f.c;
  int block = -1, units = 0;
  int64_t before = 0;  // units of a KV head's blocks before this one
  for (int h = WARPS == 1 ? warp : (int)(blockIdx.x % p.heads); h < p.heads; h += WARPS == 1 ? 4 : p.heads) {
    const int head = h / p.group, row = f.row0 + h % p.group;
    if (row / c.rows != block) {
      block = row / c.rows;
      before = 0;
      for (int k = lane; k < block; k += 32) before += units_of(p, c, f.s, k);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
      units = units_of(p, c, f.s, block);
    }
    float v[V], L = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.f;
    const int64_t u0 = f.units0 + head * f.head_units + before;
    // (units of a call that fit 32 bits, as nearly all do, need no 64-bit division)
    const bool narrow = u0 + units < 0x7fffffff && f.per < 0x7fffffff;
    const int b0 = narrow ? (int)((uint32_t)u0 / (uint32_t)f.per) : (int)(u0 / f.per);
    const int64_t u1 = u0 + max(units, 1) - 1;
    const int b1 = narrow ? (int)((uint32_t)u1 / (uint32_t)f.per) : (int)(u1 / f.per);
    if (units > 0 && b0 == b1) {
      if (WARPS == 1 || warp == 0) {
        const float *from = p.whole + (token * p.heads + h) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = from[e];
        L = 1.f;
      }
    } else if (units > 0) {
      const int in = row % c.rows;
      auto at = [&](int b) { return ((int64_t)2 * b + (b == b0 ? 1 : 0)) * c.rows + in; };
      float M = -INFINITY;
      for (int b = b0 + lane; b <= b1; b += 32) M = fmaxf(M, c.part_ml[at(b)].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll 4
      for (int b = b0 + (WARPS == 1 ? 0 : warp); b <= b1; b += WARPS) {
        const float2 a = c.part_ml[at(b)];
        const float *po = c.part_o + at(b) * D + lane * V;
        float x[V];
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = po[e];
        if (a.y != 0.f) {  // the row sees some of the run's keys
          const float g = a.x == -INFINITY ? 0.f : ex2(a.x - M);
          L = fmaf(g, a.y, L);
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] = fmaf(g, x[e], v[e]);
        }
      }
    }
    if constexpr (WARPS > 1) {
#pragma unroll
      for (int e = 0; e < V; ++e) s_v[warp][lane * V + e] = v[e];
      if (lane == 0) s_l[warp] = L;
      __syncthreads();
      if (warp > 0) return;
      L = s_l[0] + s_l[1] + s_l[2] + s_l[3];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int j = lane * V + e;
        v[e] = s_v[0][j] + s_v[1][j] + s_v[2][j] + s_v[3][j];
      }
    }
    const float inv = L != 0.f ? 1.0f / L : 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] *= inv;
    warp_rotate_back<D>(v, p.vdiag, lane);
    write_row<D>(p.out, token * p.ldo + (int64_t)h * D, v, lane, p.bf16);
  }
}

int device_sms() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 1;
}

// Sequences of more rows go to the kernel of many rows, whose blocks of 128
// or 256 rows cost the same however few of their rows are there.
constexpr int kFewRows = 32;

// Sizes of a call and where its pieces lie in the workspace
struct Plan {
  PagedCut few{}, many{};
  size_t few_o, few_ml, few_first, many_o, many_ml, many_first, whole, qprep, qscale, total;
};

Plan plan_of(const tq_quantizer *qk, int64_t total_q, int64_t nseq, int64_t heads, int64_t kv_heads, int64_t max_new,
             int sms) {
  Plan L{};
  const int d = qk->d;
  const bool ip = qk->m > 0;
  const int64_t most = std::min(max_new, total_q) * (heads / kv_heads);
  const bool many = most > kFewRows;
  // 8 rows a block where that is all there is: twice the warps on an SM
  L.few = PagedCut{most <= 8 ? 8 : 16, 6, 0, many ? kFewRows : 0x7fffffff, sms, 4, nullptr, nullptr, nullptr};
  if (many) L.many = PagedCut{ip && d == 128 ? 128 : 256, 7, kFewRows, 0x7fffffff, sms, 2, nullptr, nullptr, nullptr};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~size_t(255);
    return at;
  };
  auto cut = [&](const PagedCut &c, size_t &o, size_t &ml, size_t &first) {
    o = take((size_t)2 * c.grid * c.rows * d * sizeof(float));
    ml = take((size_t)2 * c.grid * c.rows * sizeof(float2));
    first = take(c.grid ? (size_t)(nseq + 1) * sizeof(int64_t) : 0);
  };
  cut(L.few, L.few_o, L.few_ml, L.few_first);
  cut(L.many, L.many_o, L.many_ml, L.many_first);
  L.whole = take((size_t)total_q * heads * d * sizeof(float));
  L.qprep = take(many ? (size_t)total_q * heads * d * (ip ? 4 : 2) : 0);
  L.qscale = take(many ? (size_t)total_q * heads * sizeof(float) : 0);
  L.total = off + 256;
  return L;
}

template <int D>
tq_status launch_paged(const PagedParams &prm, const tq_quantizer *qk, const tq_quantizer *qv, cudaStream_t st) {
  tq_status rc = TQ_OK;
  const int64_t rows = prm.total_q * prm.heads;
  if (prm.many.grid > 0) {
    const unsigned blocks = (unsigned)((rows + 15) / 16);
    if (qk->m)
      k_paged_queries<D, true><<<blocks, 128, 0, st>>>(prm, qk->w);
    else
      k_paged_queries<D, false><<<blocks, 128, 0, st>>>(prm, qk->w);
    if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
    rc = qk->m ? paged_tiles_launch<D, true>(prm, qk->w, qv->w, st) : paged_tiles_launch<D, false>(prm, qk->w, qv->w, st);
    if (rc != TQ_OK) return rc;
  }
  rc = qk->m ? paged_rows_launch<D, true>(prm, qk->w, qv->w, st) : paged_rows_launch<D, false>(prm, qk->w, qv->w, st);
  if (rc != TQ_OK) return rc;
  if (rows >= 16 * (int64_t)prm.few.grid)
    k_attend_paged_join<D, 1><<<(unsigned)prm.total_q, 128, 0, st>>>(prm);
  else
    k_attend_paged_join<D, 4><<<(unsigned)rows, 128, 0, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace

tq_status paged_store_launch(const tq_quantizer *qk, const tq_quantizer *qv, const tq_rows &krows,
                             const tq_rows &vrows, const int64_t *slots, int64_t tokens, int kv_heads,
                             const tq_rows &kpages, const tq_rows &vpages, int64_t npages, int page_size,
                             cudaStream_t st) {
  StoreParams p{};
  const tq_quantizer *q[2] = {qk, qv};
  const tq_rows *from[2] = {&krows, &vrows}, *to[2] = {&kpages, &vpages};
  for (int i = 0; i < 2; ++i) {
    const int row[3] = {q[i]->w * q[i]->d / 8, q[i]->m / 8, 8};
    const void *src[3] = {from[i]->codes, from[i]->signs, from[i]->norms};
    void *dst[3] = {to[i]->codes, to[i]->signs, to[i]->norms};
    for (int k = 0; k < 3; ++k) {
      p.a[3 * i + k] = {static_cast<const uint8_t *>(src[k]), static_cast<uint8_t *>(dst[k]), row[k]};
      p.words += row[k] / 4;
    }
  }
  p.slots = slots;
  p.tokens = tokens;
  p.slots_total = npages * page_size;
  p.kv_heads = kv_heads;
  p.page_size = page_size;
  const int64_t n = tokens * kv_heads * p.words;
  const int64_t blocks = std::min<int64_t>((n + 255) / 256, 8 * (int64_t)device_sms());
  k_paged_store<<<(unsigned)blocks, 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

bool attend_paged_supported(const tq_quantizer *qk, const tq_quantizer *qv) {
  return qk->rotation == TQ_ROT_HADAMARD && qv->rotation == TQ_ROT_HADAMARD && qk->d == qv->d &&
         (qk->d == 64 || qk->d == 128) && qv->m == 0 && qv->w >= 2 && qv->w <= 4 && qk->w >= 1 && qk->w <= 4;
}

size_t attend_paged_ws_bytes(const tq_quantizer *qk, int64_t total_q, int64_t nseq, int64_t heads, int64_t kv_heads,
                             int64_t max_new) {
  return plan_of(qk, total_q, nseq, heads, kv_heads, max_new, device_sms()).total;
}

tq_status attend_paged_launch(const tq_quantizer *qk, const tq_quantizer *qv, const PagedArgs &a, cudaStream_t st) {
  PagedParams prm{};
  const int64_t group = a.heads / a.kv_heads;
  const Plan L = plan_of(qk, a.total_q, a.nseq, a.heads, a.kv_heads, a.max_new, device_sms());
  if (!a.workspace || a.workspace_bytes < L.total) return TQ_ERR_WORKSPACE;
  if (a.total_q * a.heads > 0x7fffffff) return TQ_ERR_TOO_LARGE;
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(a.workspace) + 255) & ~uintptr_t(255));
  prm.y = a.y;
  prm.ldy = a.ldy;
  prm.q_start = a.q_start;
  prm.kv_len = a.kv_len;
  prm.table = a.table;
  prm.ldt = a.ldt;
  prm.total_q = a.total_q;
  prm.nseq = (int)a.nseq;
  prm.heads = (int)a.heads;
  prm.kv_heads = (int)a.kv_heads;
  prm.group = (int)group;
  prm.max_new = (int)a.max_new;
  prm.max_pages = (int)a.max_pages;
  prm.page_size = a.page_size;
  const uint32_t p16 = (uint32_t)a.page_size / 16;
  prm.page_magic = (uint32_t)((((uint64_t)1 << 31) + p16 - 1) / p16);
  prm.npages = a.npages;
  prm.kcodes = static_cast<const uint8_t *>(a.kpages.codes);
  prm.ksigns = static_cast<const uint8_t *>(a.kpages.signs);
  prm.knorms = reinterpret_cast<const float2 *>(a.kpages.norms);
  prm.vcodes = static_cast<const uint8_t *>(a.vpages.codes);
  prm.vnorms = reinterpret_cast<const float2 *>(a.vpages.norms);
  prm.bf16 = a.dtype == TQ_BF16;
  prm.scale = a.scale;
  for (int i = 0; i < 16; ++i) {
    prm.ck[i] = i < (1 << qk->w) ? double_to_half_bits(qk->centroids[i]) : 0;
    prm.cv[i] = i < (1 << qv->w) ? double_to_half_bits(qv->centroids[i]) : 0;
    prm.ckf[i] = i < (1 << qk->w) ? (float)qk->centroids[i] : 0.f;
    prm.cvf[i] = i < (1 << qv->w) ? (float)qv->centroids[i] : 0.f;
  }
  prm.kdiag = qk->kt.diag_bits;
  prm.vdiag = qv->kt.diag_bits;
  prm.qjl = qk->kt.qjl16;
  prm.kappa = qk->kt.qjl_scale;
  prm.out = a.out;
  prm.ldo = a.ldo;
  prm.few = L.few;
  prm.many = L.many;
  prm.few.first = reinterpret_cast<int64_t *>(base + L.few_first);
  prm.few.part_o = reinterpret_cast<float *>(base + L.few_o);
  prm.few.part_ml = reinterpret_cast<float2 *>(base + L.few_ml);
  prm.many.first = reinterpret_cast<int64_t *>(base + L.many_first);
  prm.many.part_o = reinterpret_cast<float *>(base + L.many_o);
  prm.many.part_ml = reinterpret_cast<float2 *>(base + L.many_ml);
  prm.whole = reinterpret_cast<float *>(base + L.whole);
  prm.qprep = reinterpret_cast<uint16_t *>(base + L.qprep);
  prm.qscale = reinterpret_cast<float *>(base + L.qscale);
  prm.err = qk->d_err;
  return qk->d == 64 ? launch_paged<64>(prm, qk, qv, st) : launch_paged<128>(prm, qk, qv, st);
}

}  // namespace tq
