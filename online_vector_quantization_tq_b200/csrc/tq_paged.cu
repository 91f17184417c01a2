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

// ---------------------------------------------------------------- join

// Joins the key ranges of a row and rotates it back: one block of four warps
// per row, which take the ranges in turn (so that their loads overlap) and
// are added up in the order of the warps.
template <int D>
__global__ void __launch_bounds__(128) k_attend_paged_join(const __grid_constant__ PagedParams p) {
  constexpr int V = D / 32;
  __shared__ float s_v[4][D], s_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t per = (int64_t)p.max_new * p.group;
  const int64_t w = blockIdx.x;
  const int row = (int)(w % per);
  const int head = (int)(w / per % p.kv_heads), seq = (int)(w / per / p.kv_heads);
  const Seq s = seq_of(p, seq);
  if (row >= s.n * p.group) return;
  const int count = p.splits[seq];
  if (count == 1) return;  // written by its work item
  const float2 *ml = p.part_ml + w * p.nsplit;
  const float *po = p.part_o + w * p.nsplit * D + lane * V;
  float M = -INFINITY;
  for (int i = lane; i < count; i += 32) M = fmaxf(M, ml[i].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = 0.f;
#pragma unroll 4
  for (int i = warp; i < count; i += 4) {
    const float2 a = ml[i];
    float b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) b[e] = po[(int64_t)i * D + e];
    if (a.y != 0.f) {  // the row sees some of the range's keys
      const float f = a.x == -INFINITY ? 0.f : ex2(a.x - M);
      L = fmaf(f, a.y, L);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = fmaf(f, b[e], v[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) s_v[warp][lane * V + e] = v[e];
  if (lane == 0) s_l[warp] = L;
  __syncthreads();
  if (warp > 0) return;
  L = s_l[0] + s_l[1] + s_l[2] + s_l[3];
  const float inv = L != 0.f ? 1.0f / L : 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int j = lane * V + e;
    v[e] = (s_v[0][j] + s_v[1][j] + s_v[2][j] + s_v[3][j]) * inv;
  }
  warp_rotate_back<D>(v, p.vdiag, lane);
  write_row<D>(p.out, (int64_t)(s.start + row / p.group) * p.ldo + (int64_t)(head * p.group + row % p.group) * D, v,
               lane, p.bf16);
}

int device_sms() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 1;
}

struct Plan {
  int64_t tiles, nsplit, items, rows;  // rows: of partial results
  int target;
  size_t part_ml, splits, total;  // offsets after part_o
};

Plan plan_of(int d, int64_t nseq, int64_t kv_heads, int64_t group, int64_t max_new, int64_t cap, int sms) {
  Plan L{};
  L.tiles = (max_new * group + kPagedRows - 1) / kPagedRows;
  const int64_t base = nseq * kv_heads * L.tiles;
  // about six work items per resident block (two per SM), so that the blocks
  // that end early find others to run
  L.target = 12 * sms;
  const int64_t want = (L.target + base - 1) / base;
  L.nsplit = std::max<int64_t>(1, std::min<int64_t>(want, (cap + kPagedMinSplit - 1) / kPagedMinSplit));
  L.items = base * L.nsplit;
  L.rows = L.nsplit > 1 ? nseq * kv_heads * max_new * group * L.nsplit : 0;
  size_t off = (size_t)L.rows * d * sizeof(float);
  L.part_ml = off;
  off += (size_t)L.rows * sizeof(float2);
  L.splits = off;
  off += (size_t)nseq * sizeof(int);
  L.total = off + 256;
  return L;
}

template <int D>
tq_status launch_paged(const PagedParams &prm, const tq_quantizer *qk, const tq_quantizer *qv, int64_t items,
                       cudaStream_t st) {
  const tq_status rc = qk->m ? paged_rows_launch<D, true>(prm, qk->w, qv->w, items, st)
                             : paged_rows_launch<D, false>(prm, qk->w, qv->w, items, st);
  if (rc != TQ_OK || prm.nsplit == 1) return rc;
  const int64_t rows = (int64_t)prm.nseq * prm.kv_heads * prm.max_new * prm.group;
  k_attend_paged_join<D><<<(unsigned)rows, 128, 0, st>>>(prm);
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

size_t attend_paged_ws_bytes(const tq_quantizer *qk, int64_t nseq, int64_t heads, int64_t kv_heads, int64_t max_new,
                             int64_t max_pages, int page_size) {
  return plan_of(qk->d, nseq, kv_heads, heads / kv_heads, max_new, max_pages * page_size, device_sms()).total;
}

tq_status attend_paged_launch(const tq_quantizer *qk, const tq_quantizer *qv, const PagedArgs &a, cudaStream_t st) {
  PagedParams prm{};
  const int64_t group = a.heads / a.kv_heads;
  const Plan L = plan_of(qk->d, a.nseq, a.kv_heads, group, a.max_new, a.max_pages * a.page_size, device_sms());
  if (!a.workspace || a.workspace_bytes < L.total) return TQ_ERR_WORKSPACE;
  if (L.items > 0x7fffffff || L.rows > ((int64_t)1 << 40)) return TQ_ERR_TOO_LARGE;
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(a.workspace) + 15) & ~uintptr_t(15));
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
  }
  prm.kdiag = qk->kt.diag_bits;
  prm.vdiag = qv->kt.diag_bits;
  prm.qjl = qk->kt.qjl16;
  prm.kappa = qk->kt.qjl_scale;
  prm.out = a.out;
  prm.ldo = a.ldo;
  prm.tiles = (int)L.tiles;
  prm.nsplit = (int)L.nsplit;
  prm.target = L.target;
  prm.part_o = reinterpret_cast<float *>(base);
  prm.part_ml = reinterpret_cast<float2 *>(base + L.part_ml);
  prm.splits = reinterpret_cast<int *>(base + L.splits);
  return qk->d == 64 ? launch_paged<64>(prm, qk, qv, L.items, st) : launch_paged<128>(prm, qk, qv, L.items, st);
}

}  // namespace tq
