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
#include <cuda_fp16.h>

#include <algorithm>

#include "tq_kernels.h"
#include "tq_sm100.cuh"

namespace tq {

namespace {

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

// ---------------------------------------------------------------- attention

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = 16;      // query rows (new token x query head of a group) of a work item
constexpr int kBlock = 16;     // keys of a warp's step; a page is a whole number of blocks
constexpr int kStages = 4;     // blocks in flight per warp, the one being used among them
constexpr int kStageBytes = kBlock * (64 + 16 + 8 + 64 + 8);  // the largest rows: d = 128, 4-bit codes, signs
constexpr int kLutBytes = 256 * 256;
constexpr int kMinSplit = 256;  // keys of a work item at least, where a sequence has them

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
  int wk, wv;      // code bits of keys and values
  int bf16;        // queries and output: bf16, else fp16
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

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

// Power of two not below v (v >= 0), kept where its reciprocal is normal too
__device__ __forceinline__ float pow2_above(float v) {
  const uint32_t e = (__float_as_uint(v) >> 23) + 1u;  // biased exponent, one up
  return __uint_as_float(min(max(e, 2u), 252u) << 23);
}

// The codes are turned into "nibble words": eight codes in the eight 4-bit
// fields of a word.  Word J (0..3) of a 32-coordinate group has in nibble n
// the code of coordinate nibble_coord(w, J, n).
__device__ __forceinline__ int nibble_coord(int w, int J, int n) { return w == 1 ? 4 * n + J : 8 * J + n; }

// Word J of the group whose code words start at `g` (shared memory).
__device__ __forceinline__ uint32_t nibble_word(const uint32_t *g, int w, int J) {
  switch (w) {
    case 4: return g[J];
    case 3:
      return J < 3 ? g[J] & 0x77777777u
                   : ((g[0] >> 1) & 0x44444444u) | ((g[1] >> 2) & 0x22222222u) | ((g[2] >> 3) & 0x11111111u);
    case 2: return (g[J >> 1] >> (2 * (J & 1))) & 0x33333333u;
    default: return (g[0] >> J) & 0x11111111u;
  }
}

// Two fp16 centroids for byte i of a nibble word: the table has a 256-byte
// row per byte value, the keys' pair in 32 copies (one per lane, so a warp's
// lookups never meet in a bank) and behind them the values' pair in 32.  The
// address is one byte permute: byte 1 the code pair, byte 0 the lane.
template <int I>
__device__ __forceinline__ uint32_t lookup(const uint8_t *lut, uint32_t word, uint32_t lane4) {
  return *reinterpret_cast<const uint32_t *>(lut + sm100::prmt(word, lane4, 0x6504u | (I << 4)));
}

struct Split {
  int keys;   // keys of a range, a multiple of the block
  int count;  // ranges
};

// The key ranges of a sequence of `len` keys: about `target` work items of
// equal length over the whole batch, at least kMinSplit keys each, at most
// nsplit ranges a sequence.  `work` = sum over sequences of keys * row tiles
// * KV heads.
__device__ __forceinline__ Split split_of(const PagedParams &p, int64_t work, int len) {
  int64_t per = (work + p.target - 1) / p.target;
  per = max(per, (int64_t)kMinSplit);
  per = max(per, (int64_t)(len + p.nsplit - 1) / p.nsplit);
  per = (per + kWarps * kBlock - 1) / (kWarps * kBlock) * (kWarps * kBlock);
  per = min(per, (int64_t)1 << 30);
  Split s;
  s.keys = (int)per;
  s.count = max(1, (int)((len + per - 1) / per));
  return s;
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

template <int D, bool IP>
__global__ void __launch_bounds__(kThreads, 2) k_attend_paged(const __grid_constant__ PagedParams p) {
  constexpr int NW = D / 32;      // nibble words of a key per lane (a quad holds a key)
  constexpr int KS = D / 16;      // MMA steps along the head dimension
  constexpr int NT = D / 8;       // 8-coordinate output tiles
  extern __shared__ __align__(256) uint8_t smem[];
  uint8_t *lut = smem;
  uint8_t *ring = smem + kLutBytes;
  __shared__ float s_f[2][kRows];         // factors of the scaled queries y~ and p
  __shared__ int s_pmax[kRows];
  __shared__ int64_t s_work[kWarps];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows], s_v[kWarps];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  // ---- the work item
  int64_t item = blockIdx.x;
  const int split = (int)(item % p.nsplit);
  item /= p.nsplit;
  const int tile = (int)(item % p.tiles);
  item /= p.tiles;
  const int head = (int)(item % p.kv_heads), seq = (int)(item / p.kv_heads);
  const Seq s = seq_of(p, seq);
  const int rows = s.n * p.group, row0 = tile * kRows;
  if (row0 >= rows) return;
  Split sp{0x40000000, 1};
  if (p.nsplit > 1) {
    int64_t work = 0;
    for (int i = tid; i < p.nseq; i += kThreads) {
      const Seq o = seq_of(p, i);
      work += (int64_t)o.len * ((o.n * p.group + kRows - 1) / kRows) * p.kv_heads;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(0xffffffffu, work, o);
    if (lane == 0) s_work[warp] = work;
    __syncthreads();
    work = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) work += s_work[w];
    sp = split_of(p, work, s.len);
    if (split >= sp.count) return;
    if (split == 0 && tile == 0 && head == 0 && tid == 0) p.splits[seq] = sp.count;
  }
  // keys that the tile's last row sees bound the range; each row has its limit
  const int last_row = min(row0 + kRows, rows) - 1;
  const int hidden = s.kv - s.n + 1;  // a row of new token t sees the keys below hidden + t
  const int seen = min(s.len, hidden + last_row / p.group);
  const int k0 = split * sp.keys, k1 = min((int)min((int64_t)k0 + sp.keys, (int64_t)s.len), seen);
  int lim[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = row0 + r + 8 * h;
    lim[h] = row < rows ? min(hidden + row / p.group, s.len) : 0;
  }
  const int lim_min = min(s.len, hidden + row0 / p.group);

  // ---- the ring: each warp copies its own blocks, kStages - 1 ahead
  const int cbk = p.wk * (D / 8), cbv = p.wv * (D / 8);
  const int off_ks = kBlock * cbk, off_kn = off_ks + (IP ? kBlock * (D / 8) : 0), off_vc = off_kn + kBlock * 8,
            off_vn = off_vc + kBlock * cbv;
  const bool swz = cbv == 64;  // 64-byte value rows: chunk ^= 2 on every second pair of rows (bank conflicts)
  const int32_t *table = p.table + (int64_t)seq * p.ldt;
  const int nblk = k1 > k0 ? (k1 - k0 + kBlock - 1) / kBlock : 0;
  const int mine = nblk > warp ? (nblk - warp + kWarps - 1) / kWarps : 0;  // blocks of this warp
  uint32_t okbits = 0;
  auto page_at = [&](int j) -> int {  // page of the warp's block j
    return j < mine ? __ldg(table + (k0 + (warp + j * kWarps) * kBlock) / p.page_size) : -1;
  };
  auto copy = [&](int j, int page) {
    if (j < mine) {
      const bool ok = page >= 0 && page < p.npages;
      okbits = (okbits & ~(1u << (j & 31))) | ((ok ? 1u : 0u) << (j & 31));
      if (ok) {
        const int key = k0 + (warp + j * kWarps) * kBlock;
        const int64_t row = ((int64_t)page * p.kv_heads + head) * p.page_size + key % p.page_size;
        const uint32_t st = sm100::smem_u32(ring + (j % kStages) * (kWarps * kStageBytes) + warp * kStageBytes);
        for (int i = lane; i < cbk; i += 32) cp_async16(st + i * 16, p.kcodes + row * cbk + i * 16);
        for (int i = lane; i < cbv; i += 32) {
          const int to = swz ? i ^ (((i >> 3) & 1) << 1) : i;
          cp_async16(st + off_vc + to * 16, p.vcodes + row * cbv + i * 16);
        }
        if (IP)
          if (lane < D / 8) cp_async16(st + off_ks + lane * 16, p.ksigns + row * (D / 8) + lane * 16);
        if (lane >= 16) {
          const int i = lane & 7;
          if (lane < 24)
            cp_async16(st + off_kn + i * 16, reinterpret_cast<const uint8_t *>(p.knorms + row) + i * 16);
          else
            cp_async16(st + off_vn + i * 16, reinterpret_cast<const uint8_t *>(p.vnorms + row) + i * 16);
        }
      }
    }
    cp_async_commit();
  };
  int next_page = 0;
#pragma unroll
  for (int j = 0; j < kStages - 1; ++j) copy(j, page_at(j));
  next_page = page_at(kStages - 1);

  // ---- queries: y~ = R y, scaled by a power of two to below 1 as fp16; for
  // inner-product keys also p = S y~ on the tensor cores (y~ as two fp16 terms)
  uint16_t *yh = reinterpret_cast<uint16_t *>(lut);  // [kRows][D], and the low terms, and p (the table comes later)
  uint16_t *yl = yh + kRows * D, *ph = yl + kRows * D;
  if (tid < kRows) s_pmax[tid] = 0;
  for (int i = warp; i < kRows; i += kWarps) {
    float v[D / 32];
    const int row = row0 + i;
    const bool there = row < rows;
    const int token = there ? row / p.group : 0, h = there ? head * p.group + row % p.group : 0;
    const int64_t at = (int64_t)(s.start + token) * p.ldy + (int64_t)h * D + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) v[e] = there ? load16(p.y, at + e, p.bf16) : 0.f;
    warp_rotate<D>(v, p.kdiag, lane);
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float up = pow2_above(top), down = 1.0f / up;
    if (lane == 0) s_f[0][i] = up;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      const float x = v[e] * down;
      const __half hi = __float2half_rn(x);
      yh[i * D + lane * (D / 32) + e] = __half_as_ushort(hi);
      if (IP) yl[i * D + lane * (D / 32) + e] = __half_as_ushort(__float2half_rn(x - __half2float(hi)));
    }
  }
  __syncthreads();
  if constexpr (IP) {
    // p[row][i] = sum_j S[i][j] y~[row][j]; warp w has the 8-column tiles w, w + kWarps, ..
    float acc[NT / kWarps][4];
#pragma unroll
    for (int t = 0; t < NT / kWarps; ++t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
      const uint32_t *srow = reinterpret_cast<const uint32_t *>(p.qjl + ((warp + t * kWarps) * 8 + r) * D);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t b0 = __ldg(srow + 8 * k + c), b1 = __ldg(srow + 8 * k + c + 4);
#pragma unroll
        for (int term = 0; term < 2; ++term) {
          const uint32_t *ya = reinterpret_cast<const uint32_t *>((term ? yl : yh) + r * D + 16 * k) + c;
          const uint32_t a[4] = {ya[0], ya[8 * (D / 2)], ya[4], ya[8 * (D / 2) + 4]};
          mma16816(acc[t], a, b0, b1);
        }
      }
    }
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < NT / kWarps; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], fabsf(acc[t][e]));
#pragma unroll
    for (int h = 0; h < 2; ++h) atomicMax(&s_pmax[r + 8 * h], __float_as_int(top[h]));  // non-negative floats
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float up = pow2_above(__int_as_float(s_pmax[r + 8 * h])), down = 1.0f / up;
      if (warp == 0 && c == 0) s_f[1][r + 8 * h] = up * s_f[0][r + 8 * h];
#pragma unroll
      for (int t = 0; t < NT / kWarps; ++t)
        reinterpret_cast<__half2 *>(ph + (r + 8 * h) * D + (warp + t * kWarps) * 8)[c] =
            __floats2half2_rn(acc[t][2 * h] * down, acc[t][2 * h + 1] * down);
    }
    __syncthreads();
  }
  // the A operands: step k of a lane pairs the coordinates of its nibble word
  // k / 2, bytes 2 (k % 2) and 2 (k % 2) + 1, as the keys' operands do
  uint32_t qa[KS][4], pa[IP ? KS : 1][4];
  {
    const int grp = D == 128 ? c : c >> 1, jo = D == 128 ? 0 : 2 * (c & 1);
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = r + 8 * (e & 1), byte = 2 * (k & 1) + (e >> 1), J = jo + (k >> 1);
        const int j0 = 32 * grp + nibble_coord(p.wk, J, 2 * byte), j1 = 32 * grp + nibble_coord(p.wk, J, 2 * byte + 1);
        qa[k][e] = yh[row * D + j0] | (uint32_t)yh[row * D + j1] << 16;
        if constexpr (IP) {
          const int i = 2 * k + (e >> 1) + (D == 128 ? 0 : 8 * (c & 1));  // sign bits i and i + 16 of the lane's word
          pa[k][e] = ph[row * D + 32 * grp + i] | (uint32_t)ph[row * D + 32 * grp + i + 16] << 16;
        }
      }
  }
  float fy[2], fp[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    fy[h] = s_f[0][r + 8 * h] * (p.scale * 1.4426950408889634f);
    fp[h] = IP ? s_f[1][r + 8 * h] * (p.scale * 1.4426950408889634f * p.kappa) : 0.f;
  }
  __syncthreads();
  for (int i = tid; i < 256 * 16; i += kThreads) {  // 16-byte pieces: 4 copies
    const int byte = i >> 4, part = i & 15;
    const uint16_t *t = part < 8 ? p.ck : p.cv;
    const uint32_t v = t[byte & 15] | (uint32_t)t[byte >> 4] << 16;
    *reinterpret_cast<uint4 *>(lut + byte * 256 + part * 16) = make_uint4(v, v, v, v);
  }
  __syncthreads();

  // ---- main loop
  const uint32_t lane4 = lane * 4;
  float o[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[t][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float vtop = pow2_above(0.f);  // power of two above the value norms seen; the weights carry its inverse
  for (int j = 0; j < mine; ++j) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    copy(j + kStages - 1, next_page);
    next_page = page_at(j + kStages);
    if (!((okbits >> (j & 31)) & 1u)) continue;
    const uint8_t *st = ring + (j % kStages) * (kWarps * kStageBytes) + warp * kStageBytes;
    const int key0 = k0 + (warp + j * kWarps) * kBlock;
    // position 8 i + 2 c + e of a block holds key 8 i + (e ? 4 + (c ^ 1) : c)
    float x[2][4];
    float2 kn[2][2];
    float vn[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = 8 * i + ((r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1);
      const uint32_t *g = reinterpret_cast<const uint32_t *>(st + key * cbk) + (D == 128 ? c : c >> 1) * p.wk;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const uint32_t word = nibble_word(g, p.wk, D == 128 ? w : 2 * (c & 1) + w);
        mma16816(acc, qa[2 * w], lookup<0>(lut, word, lane4), lookup<1>(lut, word, lane4));
        mma16816(acc, qa[2 * w + 1], lookup<2>(lut, word, lane4), lookup<3>(lut, word, lane4));
      }
      float acc2[4] = {0.f, 0.f, 0.f, 0.f};
      if constexpr (IP) {
        uint32_t sw = *reinterpret_cast<const uint32_t *>(st + off_ks + key * (D / 8) + (D == 128 ? c : c >> 1) * 4);
        if (D == 64) sw >>= 8 * (c & 1);
#pragma unroll
        for (int k = 0; k < KS; ++k)
          mma16816(acc2, pa[k], ((sw << (15 - 2 * k)) & 0x80008000u) ^ 0xBC00BC00u,
                   ((sw << (14 - 2 * k)) & 0x80008000u) ^ 0xBC00BC00u);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int kk = 8 * i + (e ? 4 + (c ^ 1) : c);
        kn[i][e] = *reinterpret_cast<const float2 *>(st + off_kn + kk * 8);
        vn[i][e] = *reinterpret_cast<const float *>(st + off_vn + kk * 8);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = acc[2 * h + e] * fy[h];
          x[i][2 * h + e] = kn[i][e].x * (IP ? fmaf(acc2[2 * h + e] * fp[h], kn[i][e].y, a) : a);
        }
      }
    }
    if (key0 + kBlock > lim_min) {  // some row does not see all of the block
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int kk = key0 + 8 * i + (e ? 4 + (c ^ 1) : c);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (kk >= lim[h]) x[i][2 * h + e] = -INFINITY;
          if (kk >= seen) vn[i][e] = 0.f;  // what lies behind the last key may be anything
        }
    }
    // running maxima; O and l are rescaled only when one grows
    float mn[2];
    bool grow = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float t = fmaxf(fmaxf(x[0][2 * h], x[0][2 * h + 1]), fmaxf(x[1][2 * h], x[1][2 * h + 1]));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
      mn[h] = fmaxf(m[h], t);
      grow |= mn[h] > m[h];
    }
    float vt = fmaxf(fmaxf(vn[0][0], vn[0][1]), fmaxf(vn[1][0], vn[1][1]));
    vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 1));
    vt = fmaxf(vt, __shfl_xor_sync(0xffffffffu, vt, 2));
    if (__any_sync(0xffffffffu, grow || vt > vtop)) {
      const float vnew = vt > vtop ? pow2_above(vt) : vtop;
      const float vf = vtop / vnew;
      vtop = vnew;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float f = mn[h] > m[h] ? ex2(m[h] - mn[h]) : 1.f;
        l[h] *= f;
        m[h] = mn[h];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          o[t][2 * h] *= f * vf;
          o[t][2 * h + 1] *= f * vf;
        }
      }
    }
    const float vinv = 1.0f / vtop;
    uint32_t wa[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float base = m[h] == -INFINITY ? 0.f : m[h];  // no key seen so far: every weight is 0
        const float p0 = ex2(x[i][2 * h] - base), p1 = ex2(x[i][2 * h + 1] - base);
        l[h] += p0 + p1;
        const __half2 w2 = __floats2half2_rn(p0 * (vn[i][0] * vinv), p1 * (vn[i][1] * vinv));
        wa[2 * i + h] = *reinterpret_cast<const uint32_t *>(&w2);
      }
    // values: lane (r, c) has coordinates of r for keys of c; the nibbles of
    // two keys are interleaved before the lookup, which then yields a pair
    const int vg = D == 128 ? r >> 1 : r >> 2, vj = D == 128 ? 2 * (r & 1) : r & 3;
#pragma unroll
    for (int w = 0; w < NT / 8; ++w) {
      uint32_t n[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int kk = 8 * i + (e ? 4 + (c ^ 1) : c);
          const int chunk = swz ? vg ^ (((kk >> 1) & 1) << 1) : vg;
          const uint32_t *g = reinterpret_cast<const uint32_t *>(st + off_vc + kk * cbv) + chunk * p.wv;
          n[i][e] = nibble_word(g, p.wv, vj + w);
        }
      uint32_t ev[2], od[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ev[i] = (n[i][0] & 0x0F0F0F0Fu) | ((n[i][1] << 4) & 0xF0F0F0F0u);
        od[i] = ((n[i][0] >> 4) & 0x0F0F0F0Fu) | (n[i][1] & 0xF0F0F0F0u);
      }
      const uint8_t *vl = lut + 128;
      mma16816(o[8 * w + 0], wa, lookup<0>(vl, ev[0], lane4), lookup<0>(vl, ev[1], lane4));
      mma16816(o[8 * w + 1], wa, lookup<0>(vl, od[0], lane4), lookup<0>(vl, od[1], lane4));
      mma16816(o[8 * w + 2], wa, lookup<1>(vl, ev[0], lane4), lookup<1>(vl, ev[1], lane4));
      mma16816(o[8 * w + 3], wa, lookup<1>(vl, od[0], lane4), lookup<1>(vl, od[1], lane4));
      mma16816(o[8 * w + 4], wa, lookup<2>(vl, ev[0], lane4), lookup<2>(vl, ev[1], lane4));
      mma16816(o[8 * w + 5], wa, lookup<2>(vl, od[0], lane4), lookup<2>(vl, od[1], lane4));
      mma16816(o[8 * w + 6], wa, lookup<3>(vl, ev[0], lane4), lookup<3>(vl, ev[1], lane4));
      mma16816(o[8 * w + 7], wa, lookup<3>(vl, od[0], lane4), lookup<3>(vl, od[1], lane4));
    }
    __syncwarp();  // the stage is read before the next copy into it is issued
  }
  cp_async_wait<0>();

  // ---- the warps' results together, in the order of the warps
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (c == 0) {
      s_m[warp][r + 8 * h] = m[h];
      s_l[warp][r + 8 * h] = l[h];
    }
  }
  if (lane == 0) s_v[warp] = vtop;
  __syncthreads();  // every warp is done with the table
  float *so = reinterpret_cast<float *>(lut) + warp * (kRows * D);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int rr = 2 * c + (e & 1);  // the lane group that holds the coordinate's codes
      const int J = (D == 128 ? 2 * (rr & 1) : rr & 3) + (t >> 3);
      const int j = 32 * (D == 128 ? rr >> 1 : rr >> 2) + 8 * J + (t & 7);
      so[(r + 8 * (e >> 1)) * D + j] = o[t][e];
    }
  __syncthreads();
  for (int i = warp; i < kRows; i += kWarps) {
    const int row = row0 + i;
    if (row >= rows) break;
    float M = -INFINITY, L = 0.f, v[D / 32];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][i]);
#pragma unroll
    for (int e = 0; e < D / 32; ++e) v[e] = 0.f;
    // (a row whose maximum is NaN-free -inf saw no key: L stays 0)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w][i] == -INFINITY ? 0.f : ex2(s_m[w][i] - M);
      if (s_l[w][i] != 0.f) {
        L += f * s_l[w][i];
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
          v[e] += f * s_v[w] * reinterpret_cast<float *>(lut)[(w * kRows + i) * D + lane * (D / 32) + e];
      }
    }
    if (sp.count == 1) {
      const float inv = L != 0.f ? 1.0f / L : 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) v[e] *= inv;
      warp_rotate_back<D>(v, p.vdiag, lane);
      const int64_t at = (int64_t)(s.start + row / p.group) * p.ldo + (int64_t)(head * p.group + row % p.group) * D;
      write_row<D>(p.out, at, v, lane, p.bf16);
    } else {
      const int64_t prow = (((int64_t)seq * p.kv_heads + head) * p.max_new * p.group + row) * p.nsplit + split;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) p.part_o[prow * D + lane * (D / 32) + e] = v[e];
      if (lane == 0) p.part_ml[prow] = make_float2(M, L);
    }
  }
}

// Joins the key ranges of a row (one warp per row) and rotates it back.
template <int D>
__global__ void __launch_bounds__(128) k_attend_paged_join(const __grid_constant__ PagedParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t per = (int64_t)p.max_new * p.group;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (int64_t)p.nseq * p.kv_heads * per) return;
  const int row = (int)(w % per);
  const int head = (int)(w / per % p.kv_heads), seq = (int)(w / per / p.kv_heads);
  const Seq s = seq_of(p, seq);
  if (row >= s.n * p.group) return;
  const int count = p.splits[seq];
  if (count == 1) return;  // written by its work item
  const int64_t first = w * p.nsplit;
  float M = -INFINITY;
  for (int i = 0; i < count; ++i) M = fmaxf(M, p.part_ml[first + i].x);
  float L = 0.f, v[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) v[e] = 0.f;
  for (int i = 0; i < count; ++i) {
    const float2 ml = p.part_ml[first + i];
    if (ml.y == 0.f) continue;  // the row sees none of the range's keys
    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
    L += f * ml.y;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) v[e] += f * p.part_o[(first + i) * D + lane * (D / 32) + e];
  }
  const float inv = L != 0.f ? 1.0f / L : 0.f;
#pragma unroll
  for (int e = 0; e < D / 32; ++e) v[e] *= inv;
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
  L.tiles = (max_new * group + kRows - 1) / kRows;
  const int64_t base = nseq * kv_heads * L.tiles;
  // about six work items per resident block (two per SM), so that the blocks
  // that end early find others to run
  L.target = 12 * sms;
  const int64_t want = (L.target + base - 1) / base;
  L.nsplit = std::max<int64_t>(1, std::min<int64_t>(want, (cap + kMinSplit - 1) / kMinSplit));
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

template <int D, bool IP>
tq_status launch_paged(const PagedParams &prm, int64_t items, cudaStream_t st) {
  constexpr int smem = kLutBytes + kStages * kWarps * kStageBytes;
  auto kern = k_attend_paged<D, IP>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  kern<<<(unsigned)items, kThreads, smem, st>>>(prm);
  if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
  if (prm.nsplit > 1) {
    const int64_t rows = (int64_t)prm.nseq * prm.kv_heads * prm.max_new * prm.group;
    k_attend_paged_join<D><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(prm);
    if (cudaGetLastError() != cudaSuccess) return TQ_ERR_CUDA;
  }
  return TQ_OK;
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
  prm.wk = qk->w;
  prm.wv = qv->w;
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
  if (qk->d == 64) return qk->m ? launch_paged<64, true>(prm, L.items, st) : launch_paged<64, false>(prm, L.items, st);
  return qk->m ? launch_paged<128, true>(prm, L.items, st) : launch_paged<128, false>(prm, L.items, st);
}

}  // namespace tq
