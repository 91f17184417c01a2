// Attention of few query rows (up to 8 or 16 to a block) over a sequence's
// pages: the kernel of tq_attend_paged for decoding and other calls with few
// new tokens.  Instantiated in tq_paged_*.cu, one file per head dimension and
// kind of keys.
//
// One block per SM stays for the whole call and works off its run of units
// (PagedCut).  Its warps take the 16-key steps of a block of rows in turn, each
// with a private ring of cp.async copies, a running softmax and an output
// accumulator of its own, and meet at the end of the block of rows.  A step's
// packed codes become the A fragments of mma.sync.m16n8k16 in registers, 16
// keys (or, for the values, 16 coordinates) by 16; the query rows are the 8
// columns of B, so that a decode step's few rows waste little of a product and
// the accumulators stay small enough for 16 warps on an SM.  (Few rows: the
// tensor cores are not the bound, and tcgen05's 128-row tiles would be mostly
// padding.)  Which coordinate or key a fragment position stands for is free as
// long as both operands agree, so a lane's fragment is exactly the codes of one
// 4..16-byte piece of a packed row, and no data moves between lanes but the
// weights, which movmatrix transposes from accumulator to operand.
//
// Two codes become two fp16 centroids by one shared-memory lookup.  A table
// of all 256 code pairs, each in 32 copies, gives every lane its own bank; its
// rows are 256 bytes (keys' pair and values' pair side by side) and it lies at
// a multiple of 64 KB in shared memory, so that a single byte permute forms the
// whole address (a table elsewhere took an addition per lookup: 64 of 520
// instructions of a step).  A byte-table expansion in registers (PRMT) takes
// 2.75 ALU instructions per code against 0.5 here plus half a lookup.
#pragma once

#include "tq_paged.cuh"

namespace tq {

namespace {

using namespace paged;

constexpr int kBlock = 16;  // keys of a warp's step; a page is a whole number of them
constexpr int kLutBytes = 256 * 256;

// Shapes of a variant with NQ groups of 8 query rows.  As many warps as the
// registers allow: 16 of 128; two groups' accumulators at d = 128 need 168 (12
// warps), with the projections' operands 255 (8), and so do three groups'
// (d = 64).
template <int D, bool IP, int WK, int WV, int NQ>
struct Shape {
  static constexpr int kRows = 8 * NQ;
  static constexpr int kWarps = NQ == 1 || (D == 64 && NQ == 2) ? 16 : IP || NQ == 3 ? 8 : 12;
  static constexpr int kThreads = 32 * kWarps;
  // one warp's stage of the ring: the packed rows of kBlock keys
  static constexpr int kRowK = WK * D / 8, kRowV = WV * D / 8, kRowS = IP ? D / 8 : 0;  // bytes of a packed row
  static constexpr int kSigns = kBlock * kRowK;
  static constexpr int kNormK = kSigns + kBlock * kRowS;
  static constexpr int kCodeV = kNormK + kBlock * 8;
  static constexpr int kNormV = kCodeV + kBlock * kRowV;
  static constexpr int kBytes = kNormV + kBlock * 8;
  // The table takes the second 64 KB of the shared window.  The ring lies on
  // both sides of it: in what is left of the first 64 KB (the first kLow bytes
  // of the dynamic memory, which starts below kStart: 1 KB that the system has
  // and this kernel's static arrays), and behind the table, where the
  // queries (y~, its low terms, and p) come first.
  static constexpr int kStart = 4096, kLow = 65536 - kStart;
  static constexpr int kLdq = D + 8;  // elements: 16-byte pieces of 8 rows fall into different banks
  static constexpr int kQueryRows = kRows < 16 ? 16 : (kRows + 15) / 16 * 16;  // whole tiles of the projection's MMA
  static constexpr int kQuery = kQueryRows * kLdq * 2 * (IP ? 3 : 2);
  static constexpr int kLdo = D + 4;                        // floats: accumulators of a warp fall into different banks
  static constexpr int kMerge = kWarps * kRows * kLdo * 4;  // the warps' outputs, over queries and ring
  static constexpr int kHigh = 232448 + 1024 - 131072 - kQuery;  // bytes behind them
  static constexpr int kLowStages = kLow / kBytes, kFit = (kLowStages + kHigh / kBytes) / kWarps;
  // steps in flight, the one being used among them
  static constexpr int kStages = kFit < 4 ? kFit : 4;
  static constexpr int kHighStages = kStages * kWarps > kLowStages ? kStages * kWarps - kLowStages : 0;
  static constexpr int kTail = kHighStages * kBytes > kMerge - kQuery ? kHighStages * kBytes : kMerge - kQuery;
  static constexpr int kEnd = 131072 + kQuery + kTail;  // of the shared window's bytes in use
  static_assert(kStages >= 3 && kTail <= kHigh, "shared memory");
  // 64-byte value rows: 16-byte piece ^= 2 on every second pair of rows, so that four rows fill the banks
  static constexpr bool kSwizzle = kRowV == 64;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 8x8 tile of 16-bit elements, transposed across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Codes are used as "nibble words": eight codes in the eight 4-bit fields of a
// word.  Word J (0..3) of a 32-coordinate group has in nibble n the code of
// coordinate nibble_coord<W>(J, n).
template <int W>
__device__ __forceinline__ int nibble_coord(int J, int n) {
  return W == 1 ? 4 * n + J : 8 * J + n;
}

// N (1, 2 or 4) consecutive nibble words, from word J0 (a multiple of N), of
// the group whose code words start at g.
template <int W, int N>
__device__ __forceinline__ void nibble_words(const uint8_t *g, int J0, uint32_t (&out)[N]) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(g);
  if constexpr (W == 4) {
    if constexpr (N == 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(w);
      out[0] = v.x, out[1] = v.y, out[2] = v.z, out[3] = v.w;
    } else if constexpr (N == 2) {
      const uint2 v = *reinterpret_cast<const uint2 *>(w + J0);
      out[0] = v.x, out[1] = v.y;
    } else {
      out[0] = w[J0];
    }
  } else if constexpr (W == 3) {
    const uint32_t a = w[0], b = w[1], c = w[2];
    const uint32_t last = ((a >> 1) & 0x44444444u) | ((b >> 2) & 0x22222222u) | ((c >> 3) & 0x11111111u);
    if constexpr (N == 4) {
      out[0] = a & 0x77777777u, out[1] = b & 0x77777777u, out[2] = c & 0x77777777u, out[3] = last;
    } else if constexpr (N == 2) {
      out[0] = (J0 ? c : a) & 0x77777777u;
      out[1] = J0 ? last : b & 0x77777777u;
    } else {
      out[0] = J0 == 3 ? last : (J0 == 0 ? a : J0 == 1 ? b : c) & 0x77777777u;
    }
  } else if constexpr (W == 2) {
    if constexpr (N == 4) {
      const uint2 v = *reinterpret_cast<const uint2 *>(w);
      out[0] = v.x & 0x33333333u, out[1] = (v.x >> 2) & 0x33333333u;
      out[2] = v.y & 0x33333333u, out[3] = (v.y >> 2) & 0x33333333u;
    } else if constexpr (N == 2) {
      const uint32_t v = w[J0 >> 1];
      out[0] = v & 0x33333333u, out[1] = (v >> 2) & 0x33333333u;
    } else {
      out[0] = (w[J0 >> 1] >> (2 * (J0 & 1))) & 0x33333333u;
    }
  } else {
    const uint32_t v = w[0] >> J0;
#pragma unroll
    for (int j = 0; j < N; ++j) out[j] = (v >> j) & 0x11111111u;
  }
}

// Two fp16 centroids (of the keys, or AT = 128: of the values) for byte I of a
// nibble word.  The address: byte 0 is the lane's copy, byte 1 the code pair,
// byte 2 the table's 64 KB, all but byte 1 from `lane4`.
template <int I, int AT>
__device__ __forceinline__ uint32_t lookup(uint32_t word, uint32_t lane4) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1+%2];" : "=r"(v) : "r"(sm100::prmt(word, lane4, 0x6504u | (I << 4))), "n"(AT));
  return v;
}
// The same, not to be merged with an earlier one (whose result would have to be kept)
template <int I>
__device__ __forceinline__ uint32_t lookup_again(uint32_t word, uint32_t lane4) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(sm100::prmt(word, lane4, 0x6504u | (I << 4))));
  return v;
}

template <int D, bool IP, int WK, int WV, int NQ>
__global__ void __launch_bounds__((Shape<D, IP, WK, WV, NQ>::kThreads), 1)
k_attend_paged(const __grid_constant__ PagedParams p) {
  using ST = Shape<D, IP, WK, WV, NQ>;
  constexpr int kWarps = ST::kWarps, kThreads = ST::kThreads, kRows = ST::kRows, kStages = ST::kStages;
  constexpr int NW = D / 32;      // nibble words of a key per lane (a quad holds a key)
  constexpr int KS = D / 16;      // MMA steps along the head dimension
  constexpr int MT = D / 16;      // 16-coordinate output tiles
  constexpr int LDQ = ST::kLdq, LDO = ST::kLdo;
  extern __shared__ __align__(256) uint8_t smem[];
  const uint32_t start = sm100::smem_u32(smem);
  uint8_t *lut = smem + (65536 - start);
  uint16_t *yh = reinterpret_cast<uint16_t *>(lut + kLutBytes);  // [kQueryRows][LDQ], then the low terms, and p
  uint16_t *yl = yh + ST::kQueryRows * LDQ, *ph = yl + ST::kQueryRows * LDQ;
  uint8_t *tail = lut + kLutBytes + ST::kQuery;
  __shared__ int64_t s_run[5];
  __shared__ int s_some;
  __shared__ float s_f[2][ST::kQueryRows];  // factors of the scaled queries y~ and p
  __shared__ int s_pmax[ST::kQueryRows];
  __shared__ float s_psum[ST::kQueryRows];
  __shared__ uint16_t s_c[32];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r = lane >> 2, c = lane & 3;
  {
    uint32_t size;
    asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(size));
    if (start > ST::kStart || start + size < ST::kEnd) {  // (not on this architecture: launch_rows sees to it)
      if (tid == 0) atomicCAS(p.err, 0, 131);
      return;
    }
  }
  if (tid < 32) s_c[tid] = tid < 16 ? p.ck[tid] : p.cv[tid - 16];
  // S's fragments of a warp's 8 columns of the projection: loaded long before they are used
  constexpr int PT = D / 8 > kWarps ? D / 8 / kWarps : 1;  // tiles of 8 columns of a warp: warp, warp + kWarps, ..
  uint32_t sb[IP ? PT : 1][IP ? KS : 1][2];
  auto load_projection = [&] {
    if constexpr (IP) {
      if (warp < D / 8) {
#pragma unroll
        for (int t = 0; t < PT; ++t) {
          const uint32_t *srow = reinterpret_cast<const uint32_t *>(p.qjl + ((warp + t * kWarps) * 8 + r) * D) + c;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            sb[t][k][0] = __ldg(srow + 8 * k);
            sb[t][k][1] = __ldg(srow + 8 * k + 4);
          }
        }
      }
    }
  };
  load_projection();
  __syncthreads();
  if (warp == 0) {
    const bool some = find_run(p, p.few, s_run);
    if (lane == 0) s_some = some;
    if (blockIdx.x == 0 && p.join_first) sum_parts(p);
  } else {
    for (int i = tid - 32; i < 256 * 16; i += kThreads - 32) {  // 16-byte pieces: 4 copies
      const int byte = i >> 4, part = i & 15;
      const uint16_t *t = s_c + (part < 8 ? 0 : 16);
      const uint32_t v = t[byte & 15] | (uint32_t)t[byte >> 4] << 16;
      *reinterpret_cast<uint4 *>(lut + byte * 256 + part * 16) = make_uint4(v, v, v, v);
    }
    for (int i = tid - 32; i < ST::kQuery / 16; i += kThreads - 32)
      reinterpret_cast<uint4 *>(yh)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  if (!s_some) return;
  const uint32_t lane4 = lane * 4 | 1u << 8;
  // fp16 results are precise enough to show the rounding of the rotated
  // queries and of the weights to fp16: their low terms are multiplied too, the
  // queries' from shared memory.  (Not by the variant of 8 rows at d = 128,
  // which the code alone made 5 % slower: fp16 queries take the one of 16 rows
  // there.)
  constexpr bool kLow = D == 64 || NQ > 1;
  const bool low = !p.bf16;
  Cursor cur = start_run(p, p.few, s_run);

  for (;;) {
    const Seq s = cur.s;
    const int head = cur.head, rows = s.n * p.group, row0 = cur.block * kRows;
    const int hidden = s.first;  // a row of new token t sees the keys below hidden + t
    const int seen = seen_by(p, p.few, s, cur.block);
    const int k0 = cur.unit << p.few.unit, k1 = min(k0 + (cur.take << p.few.unit), seen);

    // ---- the ring: each warp copies its own steps, kStages - 1 ahead
    const int32_t *table = p.table + (int64_t)cur.seq * p.ldt;
    const uint32_t page_rows = p.kv_heads * p.page_size, head_row = head * p.page_size;
    uint32_t okbits = 0;  // bit i: whether the i-th last copied step has a page
    // stages: [0] the next to be copied into; they move up with every step
    uint32_t stage[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
      const int at = i * kWarps + warp;
      stage[i] = at < ST::kLowStages ? ST::kStart + at * ST::kBytes
                                     : 131072 + ST::kQuery + (at - ST::kLowStages) * ST::kBytes;
    }
    const uint8_t *const kbase = p.kcodes + lane * 16, *const vbase = p.vcodes + lane * 16;
    const uint8_t *const nbase = reinterpret_cast<const uint8_t *>((lane & 8) ? p.vnorms : p.knorms) + (lane & 7) * 16;
    const uint32_t nto = ((lane & 8) ? ST::kNormV : ST::kNormK) + (lane & 7) * 16;
    auto page_at = [&](int key) -> int { return key < k1 ? __ldg(table + p.page_of(key)) : -1; };
    auto copy = [&](int key, int page) {  // of the step that starts at `key`
      const bool ok = page >= 0 && page < p.npages;  // (-1 behind the last key)
      okbits = okbits << 1 | (ok ? 1u : 0u);
      const uint32_t st = stage[0];
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) stage[i] = stage[i + 1];
      stage[kStages - 1] = st;
      if (ok) {
        // (rows of a cache fit 32 bits: the host checks)
        const uint32_t row = (uint32_t)page * page_rows + (head_row + key - p.page_of(key) * p.page_size);
        const uint8_t *kc = kbase + (uint64_t)row * (uint32_t)ST::kRowK, *vc = vbase + (uint64_t)row * (uint32_t)ST::kRowV;
#pragma unroll
        for (int i = 0; i < ST::kRowK; i += 32)  // kBlock rows = kRowK pieces of 16 bytes
          if (i + 32 <= ST::kRowK || lane < ST::kRowK - i) cp_async16(st + (i + lane) * 16, kc + i * 16);
#pragma unroll
        for (int i = 0; i < ST::kRowV; i += 32)
          if (i + 32 <= ST::kRowV || lane < ST::kRowV - i) {
            const int to = ST::kSwizzle ? (i + lane) ^ (((lane >> 3) & 1) << 1) : i + lane;
            cp_async16(st + ST::kCodeV + to * 16, vc + i * 16);
          }
        if (IP && lane < ST::kRowS)
          cp_async16(st + ST::kSigns + lane * 16, p.ksigns + lane * 16 + (uint64_t)row * (uint32_t)ST::kRowS);
        if (lane >= 16) cp_async16(st + nto, nbase + (uint64_t)row * 8u);
      }
      cp_async_commit();
    };
    constexpr int kStep = kWarps * kBlock;
    int ahead = k0 + warp * kBlock;  // first key of the step to be copied next
    {
      int pages[kStages - 1];
#pragma unroll
      for (int j = 0; j < kStages - 1; ++j) pages[j] = page_at(ahead + j * kStep);
#pragma unroll
      for (int j = 0; j < kStages - 1; ++j, ahead += kStep) copy(ahead, pages[j]);
    }
    int next_page = page_at(ahead);

    // ---- queries: y~ = R y, scaled by a power of two to below 1 as fp16; for
    // inner-product keys also p = S y~ on the tensor cores (y~ as two fp16 terms)
    if (IP && tid < ST::kQueryRows) s_pmax[tid] = 0;
#pragma unroll
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
        yh[i * LDQ + lane * (D / 32) + e] = __half_as_ushort(hi);
        yl[i * LDQ + lane * (D / 32) + e] = __half_as_ushort(__float2half_rn(x - __half2float(hi)));
      }
    }
    __syncthreads();
    if constexpr (IP) {
      // p[row][i] = sum_j S[i][j] y~[row][j]
      constexpr int RT = ST::kQueryRows / 16;
      float acc[RT][PT][4];
      if (warp < D / 8) {
#pragma unroll
        for (int u = 0; u < RT; ++u) {
#pragma unroll
          for (int t = 0; t < PT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[u][t][e] = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int term = 0; term < 2; ++term) {
              const uint32_t *ya =
                  reinterpret_cast<const uint32_t *>((term ? yl : yh) + (16 * u + r) * LDQ + 16 * k) + c;
              const uint32_t a[4] = {ya[0], ya[8 * (LDQ / 2)], ya[4], ya[8 * (LDQ / 2) + 4]};
#pragma unroll
              for (int t = 0; t < PT; ++t) mma16816(acc[u][t], a, sb[t][k][0], sb[t][k][1]);
            }
          float top[2] = {0.f, 0.f};
#pragma unroll
          for (int t = 0; t < PT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], fabsf(acc[u][t][e]));
#pragma unroll
          for (int h = 0; h < 2; ++h)
            atomicMax(&s_pmax[16 * u + r + 8 * h], __float_as_int(top[h]));  // non-negative floats
        }
      }
      __syncthreads();
      if (warp < D / 8) {
#pragma unroll
        for (int u = 0; u < RT; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = 16 * u + r + 8 * h;
            const float up = pow2_above(__int_as_float(s_pmax[i])), down = 1.0f / up;
            if (warp == 0 && c == 0) s_f[1][i] = up * s_f[0][i];
#pragma unroll
            for (int t = 0; t < PT; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int j = (warp + t * kWarps) * 8 + 2 * c + e, b = j % 32;  // coordinates k and k + 16 side by side
                ph[i * LDQ + j / 32 * 32 + (b < 16 ? 2 * b : 2 * (b - 16) + 1)] =
                    __half_as_ushort(__float2half_rn(acc[u][t][2 * h + e] * down));
              }
          }
      }
      __syncthreads();
#pragma unroll
      for (int i = warp; i < kRows; i += kWarps) {
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) sum += __half2float(__ushort_as_half(ph[i * LDQ + e * 32 + lane]));
#pragma unroll
        for (int b = 16; b > 0; b >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, b);
        if (lane == 0) s_psum[i] = sum;
      }
      __syncthreads();
    }
    // the four operand registers of nibble word `w` of this lane, from a row of queries
    auto word_of = [&](const uint16_t *row, int w, uint32_t(&v)[4]) {
      const uint16_t *y = row + 32 * (D == 128 ? c : c >> 1);
      const int J = (D == 128 ? 0 : 2 * (c & 1)) + w;
      if constexpr (WK != 1) {  // eight neighbours
        const uint4 x = *reinterpret_cast<const uint4 *>(y + 8 * J);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = y[nibble_coord<WK>(J, 2 * e)] | (uint32_t)y[nibble_coord<WK>(J, 2 * e + 1)] << 16;
      }
    };
    // the B operands (column r: query row r of a group of 8): step k of a lane
    // pairs the coordinates of its nibble word k / 2, bytes 2 (k % 2) and
    // 2 (k % 2) + 1, as the keys' operands do
    uint32_t qb[NQ][KS][2], pb[IP ? NQ : 1][IP ? KS : 1][2];
    {
      const int grp = D == 128 ? c : c >> 1;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int k = 0; k < KS; k += 2) {  // a nibble word
          uint32_t v4[4];
          word_of(yh + (8 * q + r) * LDQ, k >> 1, v4);
          qb[q][k][0] = v4[0], qb[q][k][1] = v4[1], qb[q][k + 1][0] = v4[2], qb[q][k + 1][1] = v4[3];
          if constexpr (IP) {
            // sign bits i and i + 16 of the lane's word, i = 2 k .. 2 k + 3, times 2^15 over the value of the keys'
            // bit (see there): exact, p is below 1
            const int i0 = 2 * k + (D == 128 ? 0 : 8 * (c & 1));
            const uint4 v = *reinterpret_cast<const uint4 *>(ph + (8 * q + r) * LDQ + 32 * grp + 2 * i0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 u = __hmul2(*reinterpret_cast<const __half2 *>(w + e),
                                        __float2half2_rn((float)(1 << (15 - (2 * k + e) % 8))));
              pb[q][k + (e >> 1)][e & 1] = *reinterpret_cast<const uint32_t *>(&u);
            }
          }
        }
    }
    float fy[NQ][2], fp[NQ][2], pc[NQ][2];  // columns 2 c and 2 c + 1 of the accumulators
    int lim[NQ][2];
    const int lim_min = min(s.len, hidden + row0 / p.group);
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 8 * q + 2 * c + e, row = row0 + i;
        fy[q][e] = s_f[0][i] * (p.scale * 1.4426950408889634f * p.kunit);
        // <p, +-1> = 2 <p, bits> - sum p, and the bits' product comes 2^-9 too small
        fp[q][e] = IP ? s_f[1][i] * (p.scale * 1.4426950408889634f * p.kappa) : 0.f;
        pc[q][e] = IP ? -s_psum[i] * fp[q][e] : 0.f;
        fp[q][e] *= 1024.f;
        lim[q][e] = row < rows ? min(hidden + row / p.group, s.len) : s.len;  // (columns of no row are zeros)
      }

    // ---- main loop
    float o[NQ][MT][4];
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[q][t][e] = 0.f;
    // Sums and references.  A reference is a logit and the exponent of a value norm
    // (kNone: no key was seen), the largest sum of the two among the keys that the
    // row sees: what the values are multiplied by, weight times norm, stays below
    // 2^8, and no norm of a key that is hidden or of little weight takes bits from
    // the others'.  (Apart, since beside a large logit the exponent would be lost
    // from the weights, but not from the values.)  O and l are rescaled only when a
    // reference has grown by more than 8.
    constexpr float kNone = -1e30f;
    float l[NQ][2], base[NQ][2], norm[NQ][2];
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[q][e] = base[q][e] = 0.f;
        norm[q][e] = kNone;
      }
    for (int key0 = k0 + warp * kBlock; key0 < k1; key0 += kStep) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      copy(ahead, next_page);
      ahead += kStep;
      next_page = page_at(ahead);
      if (!((okbits >> (kStages - 1)) & 1u)) continue;
      // the step's stage: the one that the next copy will take
      const uint8_t *st = smem + (stage[0] - start);
      // position 8 i + 2 c + e of a step (a row of A, or of B for the values)
      // holds key 8 i + (e ? 4 + (c ^ 1) : c)
      const int kpos = (r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1;
      float x[NQ][2][2];  // [key half][column]
      float vn[2];
      {
        float acc[NQ][4], acc2[IP ? NQ : 1][4];  // codes' part, signs' part
        uint32_t word[2][NW];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          nibble_words<WK, NW>(st + (8 * i + kpos) * ST::kRowK + (D == 128 ? c : c >> 1) * (4 * WK),
                               D == 128 ? 0 : 2 * (c & 1), word[i]);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const uint32_t a[4] = {lookup<0, 0>(word[0][w], lane4), lookup<0, 0>(word[1][w], lane4),
                                 lookup<1, 0>(word[0][w], lane4), lookup<1, 0>(word[1][w], lane4)};
          const uint32_t b[4] = {lookup<2, 0>(word[0][w], lane4), lookup<2, 0>(word[1][w], lane4),
                                 lookup<3, 0>(word[0][w], lane4), lookup<3, 0>(word[1][w], lane4)};
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (w == 0)
              mma16816_new(acc[q], a, qb[q][0][0], qb[q][0][1]);
            else
              mma16816(acc[q], a, qb[q][2 * w][0], qb[q][2 * w][1]);
            mma16816(acc[q], b, qb[q][2 * w + 1][0], qb[q][2 * w + 1][1]);
            if (D == 64 && low) {
              uint32_t l[4];
              word_of(yl + (8 * q + r) * LDQ, w, l);
              mma16816(acc[q], a, l[0], l[1]);
              mma16816(acc[q], b, l[2], l[3]);
            }
          }
        }
        if (D == 128 && kLow && low) {  // (with lookups of its own, which cost the others less)
#pragma unroll
          for (int w = 0; w < NW; ++w) {
            const uint32_t a[4] = {lookup_again<0>(word[0][w], lane4), lookup_again<0>(word[1][w], lane4),
                                   lookup_again<1>(word[0][w], lane4), lookup_again<1>(word[1][w], lane4)};
            const uint32_t b[4] = {lookup_again<2>(word[0][w], lane4), lookup_again<2>(word[1][w], lane4),
                                   lookup_again<3>(word[0][w], lane4), lookup_again<3>(word[1][w], lane4)};
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              uint32_t l[4];
              word_of(yl + (8 * q + r) * LDQ, w, l);
              mma16816(acc[q], a, l[0], l[1]);
              mma16816(acc[q], b, l[2], l[3]);
            }
          }
        }
        if constexpr (IP) {
          uint32_t sw[2], hw[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            sw[i] = *reinterpret_cast<const uint32_t *>(st + ST::kSigns + (8 * i + kpos) * ST::kRowS +
                                                        (D == 128 ? c : c >> 1) * 4);
            if (D == 64) sw[i] >>= 8 * (c & 1);
            hw[i] = sw[i] >> 8;
          }
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            // bits i and i + 16 (i = 2 k, then 2 k + 1) where they stand: as fp16, 2^(i % 8 - 24) or 0
            const uint32_t m0 = 0x00010001u << (2 * k % 8), m1 = 0x00010001u << (2 * k % 8 + 1);
            const uint32_t *w = 2 * k < 8 ? sw : hw;
            const uint32_t a[4] = {w[0] & m0, w[1] & m0, w[0] & m1, w[1] & m1};
#pragma unroll
            for (int q = 0; q < NQ; ++q)
              if (k == 0)
                mma16816_new(acc2[q], a, pb[q][k][0], pb[q][k][1]);
              else
                mma16816(acc2[q], a, pb[q][k][0], pb[q][k][1]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 kn = *reinterpret_cast<const float2 *>(st + ST::kNormK + (8 * i + kpos) * 8);
          vn[i] = fabsf(*reinterpret_cast<const float *>(st + ST::kNormV + (8 * i + kpos) * 8));
          kn.x = fabsf(kn.x);
          // a norm that is not finite makes a NaN of every row that sees its key, and of no other (an infinite one
          // could make a logit of -inf, and its key would drop out)
          if (!(vn[i] + kn.x + (IP ? fabsf(kn.y) : 0.f) < INFINITY)) {
            kn.x = NAN;
            vn[i] = 0.f;
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = acc[q][2 * i + e] * fy[q][e];
              x[q][i][e] = kn.x * (IP ? fmaf(fmaf(acc2[IP ? q : 0][2 * i + e], fp[q][e], pc[q][e]), kn.y, a) : a);
            }
        }
      }
      if (key0 + kBlock > lim_min) {  // some row does not see all of the step
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kk = key0 + 8 * i + kpos;
#pragma unroll
          for (int q = 0; q < NQ; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (kk >= lim[q][e]) x[q][i][e] = -INFINITY;
          if (kk >= seen) vn[i] = 0.f;  // what lies behind the last key may be anything
        }
      }
      const float ve[2] = {flash::norm_exponent(vn[0]) - 8.f, flash::norm_exponent(vn[1]) - 8.f};
      bool grow = false;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          grow |= fmaxf(x[q][0][e] - base[q][e] + ve[0], x[q][1][e] - base[q][e] + ve[1]) > norm[q][e];
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = fmaxf(x[q][0][e], x[q][1][e]);
#pragma unroll
            for (int b = 4; b < 32; b <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, b));
            float n = fmaxf(x[q][0][e] - t + ve[0], x[q][1][e] - t + ve[1]);
#pragma unroll
            for (int b = 4; b < 32; b <<= 1) n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, b));
            n += 8.f;
            const float up = t - base[q][e] + (n - norm[q][e]);
            if (t > -INFINITY && up > 0.f) {
              const float f = ex2(-0.5f * up);
              base[q][e] = t;
              norm[q][e] = n;
              l[q][e] = f * l[q][e] * f;
#pragma unroll
              for (int k = 0; k < MT; ++k) {
                o[q][k][e] *= f * f;
                o[q][k][2 + e] *= f * f;
              }
            }
          }
      }
      uint32_t wb[NQ][2], wl[NQ][2];  // weights, and for fp16 results their low terms
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        float w[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int i = 0; i < 2; ++i) w[i][e] = ex2(x[q][i][e] - base[q][e] - norm[q][e]);
          l[q][e] += w[0][e] + w[1][e];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const __half2 h = __floats2half2_rn(w[i][0] * vn[i], w[i][1] * vn[i]);
          wb[q][i] = transpose8(*reinterpret_cast<const uint32_t *>(&h));
          if (kLow && low) {
            const float2 g = __half22float2(h);
            const __half2 l = __floats2half2_rn(w[i][0] * vn[i] - g.x, w[i][1] * vn[i] - g.y);
            wl[q][i] = transpose8(*reinterpret_cast<const uint32_t *>(&l));
          }
        }
      }
      // values: lane (r, c) has coordinates of r for keys of c; the nibbles of
      // two keys are interleaved before the lookup, which then yields a pair
      const int vg = D == 128 ? r >> 1 : r >> 2, vj = D == 128 ? 2 * (r & 1) : r & 3;
      uint32_t n[2][2][D / 64];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int kk = 8 * i + (e ? 4 + (c ^ 1) : c);
          const int g = ST::kSwizzle ? vg ^ (((kk >> 1) & 1) << 1) : vg;
          nibble_words<WV, D / 64>(st + ST::kCodeV + kk * ST::kRowV + g * (4 * WV), vj, n[i][e]);
        }
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        uint32_t ev[2], od[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          ev[i] = (n[i][0][w] & 0x0F0F0F0Fu) | ((n[i][1][w] << 4) & 0xF0F0F0F0u);
          od[i] = ((n[i][0][w] >> 4) & 0x0F0F0F0Fu) | (n[i][1][w] & 0xF0F0F0F0u);
        }
        const uint32_t a[4][4] = {
            {lookup<0, 128>(ev[0], lane4), lookup<0, 128>(od[0], lane4), lookup<0, 128>(ev[1], lane4), lookup<0, 128>(od[1], lane4)},
            {lookup<1, 128>(ev[0], lane4), lookup<1, 128>(od[0], lane4), lookup<1, 128>(ev[1], lane4), lookup<1, 128>(od[1], lane4)},
            {lookup<2, 128>(ev[0], lane4), lookup<2, 128>(od[0], lane4), lookup<2, 128>(ev[1], lane4), lookup<2, 128>(od[1], lane4)},
            {lookup<3, 128>(ev[0], lane4), lookup<3, 128>(od[0], lane4), lookup<3, 128>(ev[1], lane4), lookup<3, 128>(od[1], lane4)}};
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            mma16816(o[q][4 * w + b], a[b], wb[q][0], wb[q][1]);
            if (kLow && low) mma16816(o[q][4 * w + b], a[b], wl[q][0], wl[q][1]);
          }
      }
      __syncwarp();  // the stage is read before the next copy into it is issued
    }
    cp_async_wait<0>();

    // ---- the warps' results together, in the order of the warps
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int b = 4; b < 32; b <<= 1) l[q][e] += __shfl_xor_sync(0xffffffffu, l[q][e], b);
        if (r == 0) {
          s_m[warp][8 * q + 2 * c + e] = norm[q][e] == kNone ? -INFINITY : base[q][e] + norm[q][e];
          s_l[warp][8 * q + 2 * c + e] = l[q][e];
        }
      }
    __syncthreads();  // every warp is done with the ring
    load_projection();  // (for the next block of rows)
    // coordinate (D / 8) r + i of a row, i = 2 t + (e >> 1), stands at 8 i + r
    float *so = reinterpret_cast<float *>(yh);
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          so[(warp * kRows + 8 * q + 2 * c + (e & 1)) * LDO + 8 * (2 * t + (e >> 1)) + r] = o[q][t][e];
    __syncthreads();
    for (int i = warp; i < kRows; i += kWarps) {
      const int row = row0 + i;
      if (row >= rows) break;
      float M = -INFINITY, L = 0.f, v[D / 32];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][i]);
#pragma unroll
      for (int e = 0; e < D / 32; ++e) v[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_m[w][i] == -INFINITY ? 0.f : ex2_half(s_m[w][i] - M);
        if (s_l[w][i] != 0.f) {  // the row sees some of the warp's keys
          L += f * s_l[w][i] * f;
#pragma unroll
          for (int e = 0; e < D / 32; ++e) v[e] += f * f * p.vunit * so[(w * kRows + i) * LDO + lane * (D / 32) + e];
        }
      }
      float *to;
      if (cur.whole()) {
        const float inv = L != 0.f ? 1.0f / L : 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) v[e] *= inv;
        to = p.whole + ((int64_t)(s.start + row / p.group) * p.heads + head * p.group + row % p.group) * D;
      } else {
        const int64_t at = (int64_t)cur.slot() * kRows + i;
        if (lane == 0) p.few.part_ml[at] = make_float2(M, L);
        to = p.few.part_o + at * D;
      }
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const int at = lane * (D / 32) + e;
        to[(D / 8) * (at & 7) + (at >> 3)] = v[e];
      }
    }
    if (!cur.next(p, p.few)) break;
    __syncthreads();  // the ring and the queries' place are free
  }
}

template <int D, bool IP, int WK, int WV, int NQ>
tq_status launch_rows(const PagedParams &prm, cudaStream_t st) {
  using ST = Shape<D, IP, WK, WV, NQ>;
  auto kern = k_attend_paged<D, IP, WK, WV, NQ>;
  // dynamic memory starts behind the system's 1 KB and the kernel's static arrays (the kernel checks)
  static std::atomic<uint64_t> ready{0};
  static std::atomic<int> dynamic{0};
  const tq_status rc = once_per_device(ready, [&] {
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return false;
    const int n = ST::kEnd - 1024 - (int)fa.sharedSizeBytes;
    dynamic.store(n);
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, n) == cudaSuccess;
  });
  if (rc != TQ_OK) return rc;
  const int smem = dynamic.load();
  kern<<<(unsigned)prm.few.grid, ST::kThreads, smem, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

template <int D, bool IP, int WK, int WV>
tq_status launch_rows_nq(const PagedParams &prm, cudaStream_t st) {
  if constexpr (D == 64) {
    if (prm.few.rows == 24) return launch_rows<D, IP, WK, WV, 3>(prm, st);
  }
  return prm.few.rows == 8 ? launch_rows<D, IP, WK, WV, 1>(prm, st) : launch_rows<D, IP, WK, WV, 2>(prm, st);
}

template <int D, bool IP, int WK>
tq_status launch_rows_wv(const PagedParams &prm, int wv, cudaStream_t st) {
  switch (wv) {
    case 2: return launch_rows_nq<D, IP, WK, 2>(prm, st);
    case 3: return launch_rows_nq<D, IP, WK, 3>(prm, st);
    case 4: return launch_rows_nq<D, IP, WK, 4>(prm, st);
  }
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace

template <int D, bool IP>
tq_status paged_rows_launch(const PagedParams &prm, int wk, int wv, cudaStream_t st) {
  switch (wk) {
    case 1: return launch_rows_wv<D, IP, 1>(prm, wv, st);
    case 2: return launch_rows_wv<D, IP, 2>(prm, wv, st);
    case 3: return launch_rows_wv<D, IP, 3>(prm, wv, st);
    case 4: return launch_rows_wv<D, IP, 4>(prm, wv, st);
  }
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace tq
