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
#include <atomic>
#include <cstring>
#include <type_traits>

#include "tq_kernels.h"
#include "tq_paged.cuh"

namespace tq {

namespace {

using namespace paged;

// ---------------------------------------------------------------- store

struct StoreArray {
  const uint8_t *src;
  uint8_t *dst;
  int row;   // bytes of a row, a multiple of 4
  int size;  // bytes of a piece: 16, 8 or 4, dividing the row and aligned at both ends
  int all;   // pieces of a token, of all heads
};
struct StoreParams {
  StoreArray a[6];  // codes, signs, norms of the keys, then of the values
  int arrays, pieces;  // pieces of a token, over all arrays and heads
  const int64_t *slots;
  int64_t tokens, slots_total;  // npages * page_size
  int kv_heads, page_size;
};

constexpr int kStorePieces = 4;  // of a lane and token
constexpr int kStoreTokens = 2;  // of a warp in flight
constexpr int kStoreBlocks = 4;  // of an SM (16384 tokens, a launch among others: 17.3 us, with 8 18.4, with 16 22.5)

// A warp takes a token at a time, its lanes the same pieces of every token (up
// to 16 bytes of a row each), so that where a piece lies within a token's rows
// is found once; blockIdx.y takes further pieces of the same tokens.  Bound by the
// latency of slot, load and store (16384 tokens of 8 heads: 17 us with the launch; by
// 4-byte words 54 us).
__global__ void __launch_bounds__(256) k_paged_store(const __grid_constant__ StoreParams p) {
  const int lane = threadIdx.x & 31;
  const uint8_t *src[kStorePieces];
  uint8_t *dst[kStorePieces];
  int row[kStorePieces], size[kStorePieces];
#pragma unroll
  for (int i = 0; i < kStorePieces; ++i) {
    int n = (blockIdx.y * kStorePieces + i) * 32 + lane;
    size[i] = row[i] = 0;
    src[i] = nullptr;
    dst[i] = nullptr;
    int k = 0;  // the array of the piece
    while (k < p.arrays && n >= p.a[k].all) n -= p.a[k++].all;
    if (k < p.arrays) {
      const StoreArray a = p.a[k];
      const int per = a.row / a.size, head = n / per, at = (n - head * per) * a.size;
      size[i] = a.size;
      row[i] = a.row;
      src[i] = a.src + (int64_t)head * a.row + at;
      dst[i] = a.dst + (int64_t)head * p.page_size * a.row + at;
    }
  }
  const int64_t warps = (int64_t)gridDim.x * 8;
  for (int64_t token = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); token < p.tokens; token += kStoreTokens * warps) {
    int64_t slot[kStoreTokens];
    uint4 v[kStoreTokens][kStorePieces];
#pragma unroll
    for (int u = 0; u < kStoreTokens; ++u) {
      slot[u] = token + u * warps < p.tokens ? __ldg(p.slots + token + u * warps) : -1;
      if (slot[u] >= p.slots_total) slot[u] = -1;
    }
#pragma unroll
    for (int u = 0; u < kStoreTokens; ++u) {
      if (slot[u] < 0) continue;
      const int64_t from = (token + u * warps) * p.kv_heads;
#pragma unroll
      for (int i = 0; i < kStorePieces; ++i) {
        const uint8_t *s = src[i] + from * row[i];
        if (size[i] == 16)
          v[u][i] = __ldg(reinterpret_cast<const uint4 *>(s));
        else if (size[i] == 8)
          *reinterpret_cast<uint2 *>(&v[u][i]) = __ldg(reinterpret_cast<const uint2 *>(s));
        else if (size[i] == 4)
          v[u][i].x = __ldg(reinterpret_cast<const uint32_t *>(s));
      }
    }
#pragma unroll
    for (int u = 0; u < kStoreTokens; ++u) {
      if (slot[u] < 0) continue;
      const int64_t page = divide(slot[u], p.page_size);
      const int64_t to = (page * p.kv_heads - page) * p.page_size + slot[u];  // page * heads * page_size + offset
#pragma unroll
      for (int i = 0; i < kStorePieces; ++i) {
        uint8_t *d = dst[i] + to * row[i];
        if (size[i] == 16)
          *reinterpret_cast<uint4 *>(d) = v[u][i];
        else if (size[i] == 8)
          *reinterpret_cast<uint2 *>(d) = *reinterpret_cast<const uint2 *>(&v[u][i]);
        else if (size[i] == 4)
          *reinterpret_cast<uint32_t *>(d) = v[u][i].x;
      }
    }
  }
}

// ---------------------------------------------------------------- queries

// Rotated queries (and their projections) of all rows as fp16 operands of the
// kernel of many rows: row (token * heads + head) is R y / U, and for
// inner-product keys S R y / (64 U) behind it, U a power of two above the row's
// largest coordinate, which goes to qscale; of fp16 queries (LOW) at last what
// the rounding of R y / U left over.  Coordinates stand where the
// expansion of packed codes and signs puts them.  One thread a row, 64 rows a
// block; the projection on the tensor cores, with y~ as two fp16 terms.
// (37000 rows of d = 128 with the projection: 30 us; by a warp a row, 16 rows a
// block, 115 us.)
constexpr int kQueryRows = 64;

template <int D, bool IP, bool LOW>
__global__ void __launch_bounds__(kQueryRows) k_paged_queries(const __grid_constant__ PagedParams p, int w) {
  constexpr int DQ = (1 + IP + LOW) * D, LD = D + 8;  // padded rows: fragments of 8 rows fall into different banks
  __shared__ __align__(16) uint16_t yh[kQueryRows * LD], yl[IP || LOW ? kQueryRows * LD : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row0 = (int64_t)blockIdx.x * kQueryRows, total = p.total_q * p.heads, row = row0 + tid;
  {
    float v[D];
    const int64_t at = row < total ? row / p.heads * p.ldy + row % p.heads * D : -1;
    const uint16_t *from = static_cast<const uint16_t *>(p.y) + at;
    if (at >= 0 && (p.ldy % 8 | (reinterpret_cast<uintptr_t>(p.y) & 15)) == 0) {
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(from) + c);
        const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * c + e] = widen16((uint16_t)(words[e / 2] >> (16 * (e & 1))), p.bf16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < D; ++e) v[e] = at >= 0 ? widen16(from[e], p.bf16) : 0.f;
    }
    thread_rotate<D>(v, p.kdiag);
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < D; ++e) top = fmaxf(top, fabsf(v[e]));
    const float up = pow2_above(top), down = 1.0f / up;
    if (at >= 0) p.qscale[row] = up;
#pragma unroll
    for (int e = 0; e < D; e += 2) {
      const float2 x = make_float2(v[e] * down, v[e + 1] * down);
      const __half2 hi = __floats2half2_rn(x.x, x.y);
      *reinterpret_cast<__half2 *>(yh + tid * LD + e) = hi;
      if constexpr (IP || LOW) {
        const float2 h = __half22float2(hi);
        *reinterpret_cast<__half2 *>(yl + tid * LD + e) = __floats2half2_rn(x.x - h.x, x.y - h.y);
      }
    }
  }
  __syncthreads();
  // 16-byte pieces, neighbours by neighbouring threads
  const int rows = (int)min((int64_t)kQueryRows, total - row0);
  uint4 *to = reinterpret_cast<uint4 *>(p.qprep + row0 * DQ);
  auto put = [&](const uint16_t *part, int at, bool codes) {  // codes: in the order of the codes' operands
    for (int i = tid; i < rows * (D / 8); i += kQueryRows) {
      const int r = i / (D / 8), c = i % (D / 8);
      uint4 x;
      if (!codes || w != 1) {
        x = *reinterpret_cast<const uint4 *>(part + r * LD + c * 8);
      } else {  // one-bit codes: byte 8 (j % 4) + j / 4 of a group is coordinate j
        uint32_t q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int b = (8 * c + 2 * e) % 32;  // coordinates of positions b and b + 1
          const uint16_t *g = part + r * LD + 8 * c / 32 * 32;
          q[e] = g[4 * (b % 8) + b / 8] | (uint32_t)g[4 * (b % 8 + 1) + b / 8] << 16;
        }
        x = make_uint4(q[0], q[1], q[2], q[3]);
      }
      to[r * (DQ / 8) + at / 8 + c] = x;
    }
  };
  put(yh, 0, true);
  if constexpr (LOW) put(yl, (1 + IP) * D, true);
  float acc[IP ? 2 : 1][IP ? D / 8 : 1][4];  // projections of the warp's 32 rows
  if constexpr (IP) {
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < D / 8; ++t) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[m][t][e] = 0.f;
    }
#pragma unroll 1
    for (int k = 0; k < D / 16; ++k) {
      uint32_t a[2][2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          const uint32_t *ya =
              reinterpret_cast<const uint32_t *>((term ? yl : yh) + (32 * warp + 16 * m + r) * LD + 16 * k) + c;
          a[m][term][0] = ya[0], a[m][term][1] = ya[8 * (LD / 2)], a[m][term][2] = ya[4], a[m][term][3] = ya[8 * (LD / 2) + 4];
        }
#pragma unroll
      for (int t = 0; t < D / 8; ++t) {
        const uint32_t *srow = reinterpret_cast<const uint32_t *>(p.qjl + (t * 8 + r) * D) + 8 * k + c;
        const uint32_t b0 = __ldg(srow), b1 = __ldg(srow + 4);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int term = 0; term < 2; ++term) mma16816(acc[m][t], a[m][term], b0, b1);
      }
    }
    __syncthreads();  // the low terms are read: the projections take their place
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int t = 0; t < D / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = t * 8 + 2 * c + (e & 1), b = j % 32;  // bits k and k + 16 of a word are neighbours
          yl[(32 * warp + 16 * m + r + 8 * (e >> 1)) * LD + j / 32 * 32 + (b < 16 ? 2 * b : 2 * (b - 16) + 1)] =
              __half_as_ushort(__float2half_rn(acc[m][t][e] * (1.0f / 64.0f)));
        }
    __syncthreads();
  }
  if constexpr (IP) put(yl, D, false);
}

// ---------------------------------------------------------------- join

// Where the result of a block of rows lies: runs b0 to b1 have part of it (one
// run: its normalized rows are in p.whole)
struct Place {
  int b0, b1;
  bool seen;  // the block has keys
  __device__ int64_t at(const PagedCut &c, int b) const { return ((int64_t)2 * b + (b == b0 ? 1 : 0)) * c.rows; }
};
// (by a warp: a long chunk has thousands of blocks, whose units are added up)
__device__ __forceinline__ Place place_of(const PagedParams &p, const PagedCut &c, const Seq &s, int seq, int head,
                                          int block) {
  Place f{};
  int64_t before = 0, all = 0;
  const int units = units_of(p, c, s, block), blocks = blocks_of(p, c, s);
  if (blocks == 1) {
    all = units;
  } else {
    for (int k = threadIdx.x & 31; k < blocks; k += 32) {
      const int u = units_of(p, c, s, k);
      all += u;
      if (k < block) before += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
  }
  f.seen = units > 0;
  if (!f.seen) return f;
  const int64_t u0 = __ldg(c.first + seq) + head * all + before, u1 = u0 + units - 1;
  const int64_t per = run_units(c, __ldg(c.first + p.nseq));
  f.b0 = (int)divide(u0, per);
  f.b1 = (int)divide(u1, per);
  return f;
}

// Output rows from the normalized rows of whole blocks, or from the partial
// results of the runs that share a block (added up in their order), rotated
// back.  Many rows: a block of threads takes up to 16 rows of one block, whose
// sequence it finds by a search 32 ways in the sums of sum_parts, and whose place once; each warp has two rows and four runs of each in flight.
// (64 rows a block, a run at a time: 92 us for 1024 rows of 17 runs each.)
constexpr int kJoinThreads = 256;

template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_attend_paged_join_many(const __grid_constant__ PagedParams p) {
  constexpr int V = D / 32, N = 2, kWarps = kJoinThreads / 32, kRuns = 4;
  __shared__ int s_item[4];  // sequence (-1: none), KV head, block, part
  __shared__ Place s_place;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (by value, field by field: a reference to either would make every use a load from global memory)
  auto cut_of = [&](const Seq &s) {
    const bool few = s.n * p.group <= p.few.upto;
    PagedCut c;
    c.rows = few ? p.few.rows : p.many.rows;
    c.unit = few ? p.few.unit : p.many.unit;
    c.above = few ? p.few.above : p.many.above;
    c.upto = few ? p.few.upto : p.many.upto;
    c.grid = few ? p.few.grid : p.many.grid;
    c.least = few ? p.few.least : p.many.least;
    c.first = few ? p.few.first : p.many.first;
    c.part_o = few ? p.few.part_o : p.many.part_o;
    c.part_ml = few ? p.few.part_ml : p.many.part_ml;
    return c;
  };
  if (warp == 0) {
    const int64_t *sums = p.join_first;
    int lo = 0, hi = p.nseq;  // sums[lo] <= this block < sums[hi]
    const bool some = blockIdx.x < __ldg(sums + hi);
    while (some && hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, i = lo + step * (lane + 1);
      lo += step * __popc(__ballot_sync(0xffffffffu, i < hi && __ldg(sums + i) <= blockIdx.x));
      hi = min(hi, lo + step);
    }
    if (some) {
      const Seq s = seq_of(p, lo);
      const PagedCut c = cut_of(s);
      const int64_t at = blockIdx.x - __ldg(sums + lo);
      const int per = blocks_of(p, c, s) * parts_of(c), head = (int)divide(at, per), rest = (int)(at - (int64_t)head * per);
      const Place f = place_of(p, c, s, lo, head, rest / parts_of(c));
      if (lane == 0) {
        s_item[1] = head;
        s_item[2] = rest / parts_of(c);
        s_item[3] = rest % parts_of(c);
        s_place = f;
      }
    }
    if (lane == 0) s_item[0] = some ? lo : -1;
  }
  __syncthreads();
  if (s_item[0] < 0) return;
  const Seq s = seq_of(p, s_item[0]);
  const PagedCut c = cut_of(s);
  const Place f = s_place;
  // the part's rows: no more than its block has (24 rows are two parts, of 16 and 8)
  const int head = s_item[1], in0 = s_item[3] * kJoinRows, first = s_item[2] * c.rows + in0;
  const int rows = min(min(kJoinRows, c.rows - in0), s.n * p.group - first);
  for (int r0 = warp; r0 < rows; r0 += N * kWarps) {
    float v[N][V];
    int64_t out[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = min(first + r0 + i * kWarps, first + rows - 1);  // (a row too many repeats the last)
      const int t = row / p.group, h = head * p.group + row - t * p.group;
      out[i] = (int64_t)(s.start + t) * p.heads + h;
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] = 0.f;
    }
    using Vec = typename std::conditional<D == 128, float4, float2>::type;  // a lane's V floats
    auto load = [&](const float *row, float (&x)[V]) {
      const Vec t = __ldg(reinterpret_cast<const Vec *>(row) + lane);
      memcpy(x, &t, sizeof(t));
    };
    if (f.seen && f.b0 == f.b1) {
#pragma unroll
      for (int i = 0; i < N; ++i) load(p.whole + out[i] * D, v[i]);
    } else if (f.seen) {
      float M[N], L[N];
      int64_t in[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        M[i] = -INFINITY;
        L[i] = 0.f;
        in[i] = in0 + min(r0 + i * kWarps, rows - 1);
      }
#pragma unroll 1
      for (int b = f.b0; b <= f.b1; b += kRuns) {
        float2 a[kRuns][N];
        float x[kRuns][N][V];
#pragma unroll
        for (int u = 0; u < kRuns; ++u)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int64_t at = f.at(c, min(b + u, f.b1)) + in[i];
            a[u][i] = __ldg(c.part_ml + at);
            load(c.part_o + at * D, x[u][i]);
            if (b + u > f.b1) a[u][i] = make_float2(-INFINITY, 0.f);
          }
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float top = M[i];
#pragma unroll
          for (int u = 0; u < kRuns; ++u) top = fmaxf(top, a[u][i].x);
          const float old = M[i] == -INFINITY ? 0.f : ex2_half(M[i] - top);
          M[i] = top;
          L[i] = old * L[i] * old;
#pragma unroll
          for (int e = 0; e < V; ++e) v[i][e] *= old * old;
#pragma unroll
          for (int u = 0; u < kRuns; ++u)
            if (a[u][i].y != 0.f) {  // the row sees some of the run's keys
              const float g = a[u][i].x == -INFINITY ? 0.f : ex2_half(a[u][i].x - top);
              L[i] = fmaf(g * a[u][i].y, g, L[i]);
#pragma unroll
              for (int e = 0; e < V; ++e) v[i][e] = fmaf(g * g, x[u][i][e], v[i][e]);
            }
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float inv = L[i] != 0.f ? 1.0f / L[i] : 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) v[i][e] *= inv;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) warp_rotate_back<D>(v[i], p.vdiag, lane);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (r0 + i * kWarps >= rows) break;
      const int64_t token = out[i] / p.heads;
      write_row<D>(p.out, token * p.ldo + (out[i] - token * p.heads) * D, v[i], lane, p.bf16);
    }
  }
}

// Few rows, each perhaps shared by many runs: four warps a row, which take its
// runs in turn, so that their loads overlap, and are added up in the order of
// the warps.
template <int D>
__global__ void __launch_bounds__(128) k_attend_paged_join(const __grid_constant__ PagedParams p) {
  constexpr int V = D / 32;
  __shared__ float s_v[4][D], s_l[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t token = blockIdx.x / p.heads;
  const int h = (int)(blockIdx.x % p.heads);
  int seq = -1;
  for (int i0 = 0; i0 < p.nseq; i0 += 32) {
    const uint32_t m = __ballot_sync(0xffffffffu, i0 + lane < p.nseq && __ldg(p.q_start + i0 + lane) <= token);
    seq += __popc(m);
    if (m != 0xffffffffu) break;
  }
  if (seq < 0) return;
  const Seq s = seq_of(p, seq);
  if (token < s.start || token >= s.start + s.n) return;
  const PagedCut &c = p.few;
  const int row = (int)(token - s.start) * p.group + h % p.group, block = row / c.rows, in = row - block * c.rows;
  const Place f = place_of(p, c, s, seq, h / p.group, block);
  float v[V], L = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = 0.f;
  if (f.seen && f.b0 == f.b1) {
    if (warp == 0) {
      const float *from = p.whole + (token * p.heads + h) * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = from[e];
      L = 1.f;
    }
  } else if (f.seen) {
    float M = -INFINITY;
    for (int b = f.b0 + lane; b <= f.b1; b += 32) M = fmaxf(M, c.part_ml[f.at(c, b) + in].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll 4
    for (int b = f.b0 + warp; b <= f.b1; b += 4) {
      const float2 a = c.part_ml[f.at(c, b) + in];
      const float *po = c.part_o + (f.at(c, b) + in) * D + lane * V;
      float x[V];
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = po[e];
      if (a.y != 0.f) {  // the row sees some of the run's keys
        const float g = a.x == -INFINITY ? 0.f : ex2_half(a.x - M);
        L = fmaf(g * a.y, g, L);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fmaf(g * g, x[e], v[e]);
      }
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
  write_row<D>(p.out, token * p.ldo + (int64_t)h * D, v, lane, p.bf16);
}

// Sequences of more rows go to the kernel of many rows, whose blocks of 128
// or 256 rows cost the same however few of their rows are there (8 sequences
// of 8000 keys and 8 KV heads, d = 128, us by few / by many: 32 rows 84 / 117,
// 64 rows 137 / 120, 96 rows 194 / 124; 40 sequences, 64 rows 580 / 439, 96 rows
// 860 / 450).  Time alone would set the limit near 48; up to 64 rows keep the
// kernel of few, whose bf16 calls' operands are not rounded with their norms.
constexpr int kFewRows = 64;

// Sizes of a call and where its pieces lie in the workspace
struct Plan {
  PagedCut few{}, many{};
  size_t few_o, few_ml, few_first, many_o, many_ml, many_first, join_first, whole, qprep, qscale, total;
};

// f16: of the queries
Plan plan_of(const tq_quantizer *qk, bool f16, int64_t total_q, int64_t nseq, int64_t heads, int64_t kv_heads,
             int64_t max_new, int sms) {
  Plan L{};
  const int d = qk->d;
  const bool ip = qk->m > 0;
  const int64_t most = std::min(max_new, total_q) * (heads / kv_heads);
  const bool many = most > kFewRows;
  // 8 rows a block where that is all there is: more warps on an SM.  24 where
  // two blocks of 16 would expand every key twice (5 drafted tokens of 4 heads,
  // 16 sequences, d = 64); at d = 128 its registers do not suffice.
  const int rows = most <= 8 && !(f16 && d == 128) ? 8 : d == 64 && most > 16 && most <= 24 ? 24 : 16;
  L.few = PagedCut{rows, 6, 0, many ? kFewRows : 0x7fffffff, sms, 4, nullptr, nullptr, nullptr};
  if (many) L.many = PagedCut{paged_tile_rows(d, ip, f16), 7, kFewRows, 0x7fffffff, sms, 2, nullptr, nullptr, nullptr};
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
  L.join_first = take((size_t)(nseq + 1) * sizeof(int64_t));
  L.whole = take((size_t)total_q * heads * d * sizeof(float));
  L.qprep = take(many ? (size_t)total_q * heads * d * 2 * (1 + ip + f16) : 0);
  L.qscale = take(many ? (size_t)total_q * heads * sizeof(float) : 0);
  L.total = off + 256;
  return L;
}

template <int D>
tq_status launch_paged(const PagedParams &prm, const tq_quantizer *qk, const tq_quantizer *qv, cudaStream_t st) {
  tq_status rc = TQ_OK;
  const int64_t rows = prm.total_q * prm.heads;
  if (prm.many.grid > 0) {
    const unsigned blocks = (unsigned)((rows + kQueryRows - 1) / kQueryRows);
    auto kern = qk->m ? (prm.bf16 ? k_paged_queries<D, true, false> : k_paged_queries<D, true, true>)
                      : (prm.bf16 ? k_paged_queries<D, false, false> : k_paged_queries<D, false, true>);
    kern<<<blocks, kQueryRows, 0, st>>>(prm, qk->w);
    if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
    rc = qk->m ? paged_tiles_launch<D, true>(prm, qk->w, qv->w, st) : paged_tiles_launch<D, false>(prm, qk->w, qv->w, st);
    if (rc != TQ_OK) return rc;
  }
  rc = qk->m ? paged_rows_launch<D, true>(prm, qk->w, qv->w, st) : paged_rows_launch<D, false>(prm, qk->w, qv->w, st);
  if (rc != TQ_OK) return rc;
  if (prm.join_first) {
    // parts of blocks of rows: as many as the rows fill, and of one block more per sequence and KV head
    int64_t most = 0;
    for (const PagedCut *c : {&prm.few, &prm.many}) {
      if (c->grid == 0) continue;
      const int64_t parts = (c->rows + kJoinRows - 1) / kJoinRows;
      most = std::max(most, prm.kv_heads * (prm.total_q * prm.group * parts / c->rows + prm.nseq * parts));
    }
    if (most > 0x7fffffff) return TQ_ERR_TOO_LARGE;
    k_attend_paged_join_many<D><<<(unsigned)most, kJoinThreads, 0, st>>>(prm);
  } else {
    k_attend_paged_join<D><<<(unsigned)rows, 128, 0, st>>>(prm);
  }
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
      if (row[k] == 0) continue;
      int size = 16;  // (the cache's arrays are 16-byte aligned)
      while (row[k] % size != 0 || reinterpret_cast<uintptr_t>(src[k]) % size != 0) size /= 2;
      const int all = row[k] / size * kv_heads;
      p.a[p.arrays++] = {static_cast<const uint8_t *>(src[k]), static_cast<uint8_t *>(dst[k]), row[k], size, all};
      p.pieces += all;
    }
  }
  p.slots = slots;
  p.tokens = tokens;
  p.slots_total = npages * page_size;
  p.kv_heads = kv_heads;
  p.page_size = page_size;
  const int64_t blocks = std::min<int64_t>((tokens + 7) / 8, kStoreBlocks * (int64_t)current_sms());
  const dim3 grid((unsigned)blocks, (unsigned)((p.pieces + 32 * kStorePieces - 1) / (32 * kStorePieces)));
  if (grid.y > 65535) return TQ_ERR_TOO_LARGE;
  k_paged_store<<<grid, 256, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

bool attend_paged_supported(const tq_quantizer *qk, const tq_quantizer *qv) {
  return qk->rotation == TQ_ROT_HADAMARD && qv->rotation == TQ_ROT_HADAMARD && qk->d == qv->d &&
         (qk->d == 64 || qk->d == 128) && qv->m == 0 && qv->w >= 2 && qv->w <= 4 && qk->w >= 1 && qk->w <= 4;
}

size_t attend_paged_ws_bytes(const tq_quantizer *qk, int64_t total_q, int64_t nseq, int64_t heads, int64_t kv_heads,
                             int64_t max_new) {
  const int sms = current_sms();
  return std::max(plan_of(qk, false, total_q, nseq, heads, kv_heads, max_new, sms).total,
                  plan_of(qk, true, total_q, nseq, heads, kv_heads, max_new, sms).total);
}

tq_status attend_paged_launch(const tq_quantizer *qk, const tq_quantizer *qv, const PagedArgs &a, cudaStream_t st) {
  PagedParams prm{};
  const int64_t group = a.heads / a.kv_heads;
  const Plan L = plan_of(qk, a.dtype == TQ_F16, a.total_q, a.nseq, a.heads, a.kv_heads, a.max_new, current_sms());
  if (!a.workspace || a.workspace_bytes < L.total) return TQ_ERR_WORKSPACE;
  if (a.total_q * a.heads > 0x7fffffff || a.npages > (int64_t)0xffffffff / (a.kv_heads * a.page_size))
    return TQ_ERR_TOO_LARGE;
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
    prm.ck[i] = i < (1 << qk->w) ? qk->attend_c[i] : 0;
    prm.cv[i] = i < (1 << qv->w) ? qv->attend_c[i] : 0;
    prm.ckf[i] = i < (1 << qk->w) ? (float)qk->centroids[i] : 0.f;
    prm.cvf[i] = i < (1 << qv->w) ? (float)qv->centroids[i] : 0.f;
  }
  std::memcpy(prm.cks, qk->attend_ck, sizeof(prm.cks));
  std::memcpy(prm.cks_by, qk->attend_by, sizeof(prm.cks_by));
  prm.kunit = qk->attend_unit;
  prm.vunit = qv->attend_unit;
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
  if (L.many.grid > 0 || a.total_q * a.heads >= 16 * (int64_t)L.few.grid)
    prm.join_first = reinterpret_cast<int64_t *>(base + L.join_first);
  prm.whole = reinterpret_cast<float *>(base + L.whole);
  prm.qprep = reinterpret_cast<uint16_t *>(base + L.qprep);
  prm.qscale = reinterpret_cast<float *>(base + L.qscale);
  prm.err = qk->d_err;
  return qk->d == 64 ? launch_paged<64>(prm, qk, qv, st) : launch_paged<128>(prm, qk, qv, st);
}

}  // namespace tq
