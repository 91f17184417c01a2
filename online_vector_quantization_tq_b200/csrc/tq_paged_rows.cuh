// Attention of up to 16 query rows over a range of a sequence's pages: the
// kernel of tq_attend_paged for decoding and other calls with few new tokens.
// Instantiated in tq_paged_*.cu, one file per head dimension and kind of keys.
//
// A block of four warps takes one work item (sequence, KV head, 16 rows, key
// range); two blocks fit on an SM.  The warps take 16-key steps in turn, each
// with a private ring of cp.async copies, a running softmax and an output
// accumulator of its own, and meet only at the end.  A step's packed codes
// become the B fragments of mma.sync.m16n8k16 in registers: which coordinate
// or key a fragment position stands for is free as long as both operands
// agree, so a lane's fragment is exactly the codes of one 4..16-byte piece of
// a packed row, and no data moves between lanes.  (Few rows: the tensor cores
// are not the bound, and tcgen05's 128-row tiles would be mostly padding.)
//
// Two codes become two fp16 centroids by one shared-memory lookup.  A table
// of all 256 code pairs, each in 32 copies, gives every lane its own bank; its
// rows are 256 bytes (keys' pair and values' pair side by side), so a single
// byte permute forms the address.  A byte-table expansion in registers (PRMT)
// takes 2.75 ALU instructions per code against 0.5 here plus half a lookup.
#pragma once

#include "tq_paged.cuh"

namespace tq {

namespace {

using namespace paged;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kRows = kPagedRows;
constexpr int kBlock = 16;  // keys of a warp's step; a page is a whole number of them
constexpr int kLutBytes = 256 * 256;

// One warp's stage of the ring: the packed rows of kBlock keys.
template <int D, bool IP, int WK, int WV>
struct Stage {
  static constexpr int kRowK = WK * D / 8, kRowV = WV * D / 8, kRowS = IP ? D / 8 : 0;  // bytes of a packed row
  static constexpr int kSigns = kBlock * kRowK;
  static constexpr int kNormK = kSigns + kBlock * kRowS;
  static constexpr int kCodeV = kNormK + kBlock * 8;
  static constexpr int kNormV = kCodeV + kBlock * kRowV;
  static constexpr int kBytes = kNormV + kBlock * 8;
  static constexpr int kStages = 4;  // steps in flight, the one being used among them
  static constexpr int kSmem = kLutBytes + kStages * kWarps * kBytes;
  // 64-byte value rows: 16-byte piece ^= 2 on every second pair of rows, so that four rows fill the banks
  static constexpr bool kSwizzle = kRowV == 64;
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

// Power of two above v (v >= 0), kept where its reciprocal is normal too
__device__ __forceinline__ float pow2_above(float v) {
  const uint32_t e = (__float_as_uint(v) >> 23) + 1u;  // biased exponent, one up
  return __uint_as_float(min(max(e, 2u), 252u) << 23);
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

// Two fp16 centroids for byte I of a nibble word: address byte 1 is the code
// pair, byte 0 the lane's copy.
template <int I>
__device__ __forceinline__ uint32_t lookup(const uint8_t *lut, uint32_t word, uint32_t lane4) {
  return *reinterpret_cast<const uint32_t *>(lut + sm100::prmt(word, lane4, 0x6504u | (I << 4)));
}

template <int D, bool IP, int WK, int WV>
__global__ void __launch_bounds__(kThreads, 2) k_attend_paged(const __grid_constant__ PagedParams p) {
  using ST = Stage<D, IP, WK, WV>;
  constexpr int NW = D / 32;      // nibble words of a key per lane (a quad holds a key)
  constexpr int KS = D / 16;      // MMA steps along the head dimension
  constexpr int NT = D / 8;       // 8-coordinate output tiles
  constexpr int kStages = ST::kStages;
  extern __shared__ __align__(256) uint8_t smem[];
  uint8_t *lut = smem;
  uint8_t *ring = smem + kLutBytes;
  __shared__ float s_f[2][kRows];  // factors of the scaled queries y~ and p
  __shared__ int s_pmax[kRows];
  __shared__ int64_t s_work[kWarps];
  __shared__ uint16_t s_c[32];
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
  if (tid < 32) s_c[tid] = tid < 16 ? p.ck[tid] : p.cv[tid - 16];
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
    sp = split_of(p, work, s.len, kWarps * kBlock);
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

  // ---- the ring: each warp copies its own steps, kStages - 1 ahead
  const int32_t *table = p.table + (int64_t)seq * p.ldt;
  const int nblk = k1 > k0 ? (k1 - k0 + kBlock - 1) / kBlock : 0;
  const int mine = nblk > warp ? (nblk - warp + kWarps - 1) / kWarps : 0;  // steps of this warp
  uint32_t okbits = 0;
  auto page_at = [&](int j) -> int {  // page of the warp's step j
    return j < mine ? __ldg(table + (k0 + (warp + j * kWarps) * kBlock) / p.page_size) : -1;
  };
  auto copy = [&](int j, int page) {
    if (j < mine) {
      const bool ok = page >= 0 && page < p.npages;
      okbits = (okbits & ~(1u << (j & 31))) | ((ok ? 1u : 0u) << (j & 31));
      if (ok) {
        const int key = k0 + (warp + j * kWarps) * kBlock;
        const int64_t row = ((int64_t)page * p.kv_heads + head) * p.page_size + key % p.page_size;
        const uint32_t st = sm100::smem_u32(ring + ((j % kStages) * kWarps + warp) * ST::kBytes);
        const uint8_t *kc = p.kcodes + row * ST::kRowK, *vc = p.vcodes + row * ST::kRowV;
#pragma unroll
        for (int i = 0; i < ST::kRowK; i += 32)  // kBlock rows = kRowK pieces of 16 bytes
          if (i + 32 <= ST::kRowK || lane < ST::kRowK - i) cp_async16(st + (i + lane) * 16, kc + (i + lane) * 16);
#pragma unroll
        for (int i = 0; i < ST::kRowV; i += 32)
          if (i + 32 <= ST::kRowV || lane < ST::kRowV - i) {
            const int to = ST::kSwizzle ? (i + lane) ^ (((lane >> 3) & 1) << 1) : i + lane;
            cp_async16(st + ST::kCodeV + to * 16, vc + (i + lane) * 16);
          }
        if (IP && lane < ST::kRowS)
          cp_async16(st + ST::kSigns + lane * 16, p.ksigns + row * ST::kRowS + lane * 16);
        if (lane >= 16) {
          const int i = lane & 7;
          if (lane < 24)
            cp_async16(st + ST::kNormK + i * 16, reinterpret_cast<const uint8_t *>(p.knorms + row) + i * 16);
          else
            cp_async16(st + ST::kNormV + i * 16, reinterpret_cast<const uint8_t *>(p.vnorms + row) + i * 16);
        }
      }
    }
    cp_async_commit();
  };
  {
    int pages[kStages - 1];
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) pages[j] = page_at(j);
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) copy(j, pages[j]);
  }
  int next_page = page_at(kStages - 1);

  // ---- queries: y~ = R y, scaled by a power of two to below 1 as fp16; for
  // inner-product keys also p = S y~ on the tensor cores (y~ as two fp16 terms)
  uint16_t *yh = reinterpret_cast<uint16_t *>(lut);  // [kRows][D], and the low terms, and p (the table comes later)
  uint16_t *yl = yh + kRows * D, *ph = yl + kRows * D;
  if (tid < kRows) s_pmax[tid] = 0;
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
        const int j0 = 32 * grp + nibble_coord<WK>(J, 2 * byte), j1 = 32 * grp + nibble_coord<WK>(J, 2 * byte + 1);
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
#pragma unroll 8
  for (int i = tid; i < 256 * 16; i += kThreads) {  // 16-byte pieces: 4 copies
    const int byte = i >> 4, part = i & 15;
    const uint16_t *t = s_c + (part < 8 ? 0 : 16);
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
    const uint8_t *st = ring + ((j % kStages) * kWarps + warp) * ST::kBytes;
    const int key0 = k0 + (warp + j * kWarps) * kBlock;
    // position 8 i + 2 c + e of a step holds key 8 i + (e ? 4 + (c ^ 1) : c)
    float x[2][4];
    float vn[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int key = 8 * i + ((r & 1) ? 4 + ((r >> 1) ^ 1) : r >> 1);
      uint32_t word[NW];
      nibble_words<WK, NW>(st + key * ST::kRowK + (D == 128 ? c : c >> 1) * (4 * WK), D == 128 ? 0 : 2 * (c & 1), word);
      float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        // two chains of sums: the second holds the signs' part, or half of the codes'
        mma16816(acc, qa[2 * w], lookup<0>(lut, word[w], lane4), lookup<1>(lut, word[w], lane4));
        mma16816(IP ? acc : acc2, qa[2 * w + 1], lookup<2>(lut, word[w], lane4), lookup<3>(lut, word[w], lane4));
      }
      if constexpr (IP) {
        uint32_t sw =
            *reinterpret_cast<const uint32_t *>(st + ST::kSigns + key * ST::kRowS + (D == 128 ? c : c >> 1) * 4);
        if (D == 64) sw >>= 8 * (c & 1);
#pragma unroll
        for (int k = 0; k < KS; ++k)
          mma16816(acc2, pa[k], ((sw << (15 - 2 * k)) & 0x80008000u) ^ 0xBC00BC00u,
                   ((sw << (14 - 2 * k)) & 0x80008000u) ^ 0xBC00BC00u);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int kk = 8 * i + (e ? 4 + (c ^ 1) : c);
        const float2 kn = *reinterpret_cast<const float2 *>(st + ST::kNormK + kk * 8);
        vn[i][e] = *reinterpret_cast<const float *>(st + ST::kNormV + kk * 8);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = (IP ? acc[2 * h + e] : acc[2 * h + e] + acc2[2 * h + e]) * fy[h];
          x[i][2 * h + e] = kn.x * (IP ? fmaf(acc2[2 * h + e] * fp[h], kn.y, a) : a);
        }
      }
    }
    if (key0 + kBlock > lim_min) {  // some row does not see all of the step
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
    uint32_t n[2][2][NT / 8];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int kk = 8 * i + (e ? 4 + (c ^ 1) : c);
        const int g = ST::kSwizzle ? vg ^ (((kk >> 1) & 1) << 1) : vg;
        nibble_words<WV, NT / 8>(st + ST::kCodeV + kk * ST::kRowV + g * (4 * WV), vj, n[i][e]);
      }
#pragma unroll
    for (int w = 0; w < NT / 8; ++w) {
      uint32_t ev[2], od[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ev[i] = (n[i][0][w] & 0x0F0F0F0Fu) | ((n[i][1][w] << 4) & 0xF0F0F0F0u);
        od[i] = ((n[i][0][w] >> 4) & 0x0F0F0F0Fu) | (n[i][1][w] & 0xF0F0F0F0u);
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
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w][i] == -INFINITY ? 0.f : ex2(s_m[w][i] - M);
      if (s_l[w][i] != 0.f) {  // the row sees some of the warp's keys
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

template <int D, bool IP, int WK, int WV>
tq_status launch_rows(const PagedParams &prm, int64_t items, cudaStream_t st) {
  auto kern = k_attend_paged<D, IP, WK, WV>;
  constexpr int smem = Stage<D, IP, WK, WV>::kSmem;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TQ_ERR_CUDA;
  kern<<<(unsigned)items, kThreads, smem, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

template <int D, bool IP, int WK>
tq_status launch_rows_wv(const PagedParams &prm, int wv, int64_t items, cudaStream_t st) {
  switch (wv) {
    case 2: return launch_rows<D, IP, WK, 2>(prm, items, st);
    case 3: return launch_rows<D, IP, WK, 3>(prm, items, st);
    case 4: return launch_rows<D, IP, WK, 4>(prm, items, st);
  }
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace

template <int D, bool IP>
tq_status paged_rows_launch(const PagedParams &prm, int wk, int wv, int64_t items, cudaStream_t st) {
  switch (wk) {
    case 1: return launch_rows_wv<D, IP, 1>(prm, wv, items, st);
    case 2: return launch_rows_wv<D, IP, 2>(prm, wv, items, st);
    case 3: return launch_rows_wv<D, IP, 3>(prm, wv, items, st);
    case 4: return launch_rows_wv<D, IP, 4>(prm, wv, items, st);
  }
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace tq
