// Causal attention of whole prompts on raw 16-bit queries, keys and values
// (packed sequences, grouped heads): what a server runs on a prompt before
// its keys and values are quantized into the cache.
//
//   o_t = sum_{j <= t} softmax_j(scale <q_t, k_j>) v_j,  sequence by sequence
//
// A block (one per SM: it uses all of TMEM) takes two tiles of 128 query rows
// of one sequence and KV head.  A row is a (token, query head of the group)
// pair, so a tile of a group of g heads covers 128 / g tokens (rounded down):
// with grouped heads a short prompt still fills its tiles, the keys behind the
// diagonal that a tile computes for nothing are fewer, and each key tile is
// fetched once for all heads of its group.  The two tiles share the key and
// value tiles and take turns on the tensor cores: while one tile's logits
// pass through its softmax warps, the other's products run.
//
//   warps 0-3, 4-7  softmax of tile 0 and 1 (tq_flash.cuh), and their output
//   warp 8          TMA: queries, then key and value tiles of 128 keys
//   warp 9          tcgen05: S = Q K^T from shared memory, O += P V with P in
//                   TMEM and V (keys x D) as an MN-major operand
//   warps 10-11     the tail of a value tile: see guard_values
//
// Work is handed out longest first (blocks start in the order of their
// index): the number of key tiles grows with the position in the sequence.
// Bound by the tensor cores and, equally, the exponentials.
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "tq_flash.cuh"
#include "tq_kernels.h"
#include "tq_sm100.cuh"

namespace tq {

namespace {

constexpr int kTile = 128;  // query rows of a tile, keys of a tile
constexpr int kStages = 2;  // key tiles and value tiles in flight
constexpr int kPromptThreads = 384;
// Registers move to the softmax: a warpgroup's share, whose sum is no more
// than the block was launched with (launch_prompt checks).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
constexpr int kLoadWarp = 8, kMmaWarp = 9, kGuardWarp = 10;

struct PromptParams {
  const int32_t *cu;  // [nseq + 1]
  int nseq, kv_heads, group, tokens;  // tokens: of a tile
  int64_t total;
  const uint16_t *v;  // for the guard's slow path
  int64_t ldv, ldo;
  float mult;    // |scale| log2(e)
  int negative;  // scale < 0: the products are negated
  void *out;
  int *err;
};

template <int D>
struct PromptSmem {
  static constexpr int kHalf = kTile * 128;        // 128 rows x 64 elements, 128-byte swizzle
  static constexpr int kOne = kHalf * (D / 64);    // one tile of D elements a row
  static constexpr int kQ = 0, kK = 2 * kOne, kV = kK + kStages * kOne;
  static constexpr int kBytes = kV + kStages * kOne + 1024;
};

// Item of a block, longest first.  A sequence of n tokens has ceil(n / 256
// rows) levels; level L sees about L + 1 times the keys of level 0.  Items are
// ordered by falling level, then sequence, then KV head.  Called by one warp.
__device__ bool find_item(const PromptParams &p, int64_t index, int &seq, int &level, int &head, int &start, int &n) {
  const int lane = threadIdx.x & 31;
  head = (int)(index % p.kv_heads);
  const int64_t rank = index / p.kv_heads;
  const int span = 2 * p.tokens;
  auto length = [&](int i) {
    const int64_t a = min(max((int64_t)__ldg(p.cu + i), (int64_t)0), p.total);
    return (int)(min(max((int64_t)__ldg(p.cu + i + 1), a), p.total) - a);
  };
  auto at_least = [&](int L) {  // items per head of level >= L
    int64_t c = 0;
    for (int i = lane; i < p.nseq; i += 32) c += max(0, (length(i) + span - 1) / span - L);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    return c;
  };
  int top = 0;
  for (int i = lane; i < p.nseq; i += 32) top = max(top, (length(i) + span - 1) / span);
  top = __reduce_max_sync(0xffffffffu, top);
  if (rank >= at_least(0)) return false;
  int lo = 0, hi = top;  // at_least(lo) > rank >= at_least(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (at_least(mid) > rank)
      lo = mid;
    else
      hi = mid;
  }
  level = lo;
  int64_t left = rank - at_least(lo + 1);  // which of the sequences that have level lo
  for (int i0 = 0; i0 < p.nseq; i0 += 32) {
    const bool has = i0 + lane < p.nseq && (length(i0 + lane) + span - 1) / span > lo;
    const uint32_t m = __ballot_sync(0xffffffffu, has);
    if (left < __popc(m)) {
      seq = i0 + __fns(m, 0, (int)left + 1);
      start = (int)min(max((int64_t)__ldg(p.cu + seq), (int64_t)0), p.total);
      n = length(seq);
      return true;
    }
    left -= __popc(m);
  }
  return false;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          sm100::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(sm100::smem_u32(bar))
      : "memory");
}

template <bool BF16>
__device__ __forceinline__ bool finite16(uint32_t v) {
  constexpr uint32_t e = BF16 ? 0x7F80u : 0x7C00u;
  return (v & e) != e;
}

// A product with a weight of 0 is a NaN where the value is infinite or NaN.
// So in the tiles that some row does not see whole, rows behind the end of the
// sequence (another sequence's) are cleared, and values that are not finite
// are cleared with *bad set; the rows that do see them add them at the end.
// Rows up to and including `first` are seen by every query row of the block.
template <int D, bool BF16>
__device__ void guard_values(uint8_t *tile, int key0, int first, int n, int *bad) {
  const int t = threadIdx.x - 32 * kGuardWarp;
  bool found = false;
#pragma unroll 4
  for (int i = t; i < kTile * (D / 8); i += 64) {
    const int half = i / (kTile * 8), r = (i / 8) % kTile;
    if (key0 + r <= first) continue;
    uint4 *at = reinterpret_cast<uint4 *>(tile + half * (kTile * 128) + (i % (kTile * 8)) * 16);
    if (key0 + r >= n) {
      *at = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    uint4 v = *at;
    uint32_t *w = &v.x;
    bool dirty = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t keep = (finite16<BF16>(w[k]) ? 0xFFFFu : 0u) | (finite16<BF16>(w[k] >> 16) ? 0xFFFF0000u : 0u);
      dirty |= keep != 0xFFFFFFFFu;
      w[k] &= keep;
    }
    if (dirty) {
      *at = v;
      found = true;
    }
  }
  if (found) *(volatile int *)bad = 1;
  sm100::fence_proxy_async();
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kPromptThreads, 1)
k_attend_prompt(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ PromptParams p) {
  using SM = PromptSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((0u - sm100::smem_u32(smem_raw)) & 1023u);
  __shared__ uint64_t q_full[2], k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], t_full[kStages],
      t_ok[kStages], s_full[2], p_full[2], p_half[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_item[5], s_bad;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == 0) {
    int seq = 0, level = 0, head = 0, start = 0, n = 0;
    const bool some = find_item(p, blockIdx.x, seq, level, head, start, n);
    if (lane == 0) {
      s_item[0] = some;
      s_item[1] = level;
      s_item[2] = head;
      s_item[3] = start;
      s_item[4] = n;
    }
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&q_full[i], 1);
      sm100::mbar_init(&s_full[i], 1);
      sm100::mbar_init(&p_full[i], kTile);
      sm100::mbar_init(&p_half[i], kTile);
    }
    for (int i = 0; i < kStages; ++i) {
      sm100::mbar_init(&k_full[i], 1);
      sm100::mbar_init(&k_empty[i], 1);
      sm100::mbar_init(&v_full[i], 1);
      sm100::mbar_init(&v_empty[i], 1);
      sm100::mbar_init(&t_full[i], 1);
      sm100::mbar_init(&t_ok[i], 64);
    }
    s_abort = 0;
    s_bad = 0;
    sm100::fence_barrier_init();
  } else if (warp == kLoadWarp && lane == 0) {
    sm100::prefetch_tmap(&mq);
    sm100::prefetch_tmap(&mk);
    sm100::prefetch_tmap(&mv);
  }
  __syncthreads();
  if (!s_item[0]) return;
  if (warp == kMmaWarp) {
    sm100::tmem_alloc(&s_tmem, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int head = s_item[2], start = s_item[3], n = s_item[4];
  const int t0 = s_item[1] * 2 * p.tokens;  // the block's first token
  // key tiles of the two query tiles (the second may lie behind the end)
  const int cnt[2] = {(min(t0 + p.tokens, n) + kTile - 1) / kTile,
                      t0 + p.tokens < n ? (min(t0 + 2 * p.tokens, n) + kTile - 1) / kTile : 0};
  const int tiles = max(cnt[0], cnt[1]);
  const int tail = (t0 + 1) / kTile;  // tiles from here on hold keys that some row does not see

  if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp == kLoadWarp) {
    if (lane == 0) {
      const uint32_t qbytes = (uint32_t)p.group * p.tokens * 128 * (D / 64);
      auto load_q = [&](int i) {
        sm100::mbar_expect_tx(&q_full[i], qbytes);
        for (int h = 0; h < D / 64; ++h)
          tma_load_3d(smem + SM::kQ + i * SM::kOne + h * SM::kHalf, &mq, 64 * h, head * p.group,
                      start + t0 + i * p.tokens, &q_full[i]);
      };
      auto load_kv = [&](uint8_t *dst, const CUtensorMap *m, int j, uint64_t *bar) {
        sm100::mbar_expect_tx(bar, SM::kOne);
        for (int h = 0; h < D / 64; ++h) tma_load_3d(dst + h * SM::kHalf, m, 64 * h, head, start + j * kTile, bar);
      };
      int keys = 0, values = 0;  // copies issued
      for (int j = 0; j < tiles; ++j) {
        const int st = j % kStages;
        const uint32_t ph = (uint32_t)((j / kStages - 1) & 1);
        if (j >= kStages && !sm100::mbar_wait_abort(&k_empty[st], ph, &s_abort, p.err, 101)) break;
        load_kv(smem + SM::kK + st * SM::kOne, &mk, j, &k_full[st]);
        ++keys;
        if (j == 0) {
          load_q(0);
          if (cnt[1]) load_q(1);
        }
        if (j >= kStages && !sm100::mbar_wait_abort(&v_empty[st], ph, &s_abort, p.err, 102)) break;
        load_kv(smem + SM::kV + st * SM::kOne, &mv, j, j < tail ? &v_full[st] : &t_full[st]);
        ++values;
      }
      // no copy is in flight when the block ends, whichever role gave up
      for (int i = 0; i < kStages; ++i) {
        const int k = keys - 1 - i, u = values - 1 - i;
        if (k >= 0) sm100::mbar_wait(&k_full[k % kStages], (uint32_t)((k / kStages) & 1), p.err, 113);
        if (u >= tail) sm100::mbar_wait(&t_full[u % kStages], (uint32_t)(((u - tail) / kStages) & 1), p.err, 114);
        if (u >= 0 && u < tail) sm100::mbar_wait(&v_full[u % kStages], (uint32_t)((u / kStages) & 1), p.err, 115);
        if (keys > 0 && cnt[i]) sm100::mbar_wait(&q_full[i], 0, p.err, 116);
      }
    }
  } else if (warp == kMmaWarp) {
    if (sm100::elect_one()) {
      const uint32_t type = BF16 ? sm100::idesc_bf16_f32(kTile, kTile) : sm100::idesc_f16_f32(kTile, kTile);
      const uint32_t iqk = type | (p.negative ? 1u << 13 : 0u);  // negate A
      const uint32_t ipv = (BF16 ? sm100::idesc_bf16_f32(kTile, D) : sm100::idesc_f16_f32(kTile, D)) | (1u << 16);
      const uint32_t base = sm100::smem_u32(smem);
      bool ok = true;
      auto logits = [&](int i, int j) {
        // (a step along the operand advances the descriptor's address field, in units of 16 bytes)
        const uint64_t q = sm100::desc_sw128(base + SM::kQ + i * SM::kOne);
        const uint64_t k = sm100::desc_sw128(base + SM::kK + (j % kStages) * SM::kOne);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks / 4) * SM::kHalf + (ks % 4) * 32) / 16;
          sm100::mma_f16(tmem + kTile * i, q + off, k + off, iqk, ks != 0);
        }
        sm100::mma_commit(&s_full[i]);
      };
      auto output = [&](int i, int j) {
        const uint64_t v = sm100::desc_sw128_mn(base + SM::kV + (j % kStages) * SM::kOne, SM::kHalf, 1024);
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks) {
          if (ks == kTile / 32) {
            ok = sm100::mbar_poll_abort(&p_full[i], (uint32_t)(j & 1), &s_abort, p.err, 117);
            if (!ok) return;
            sm100::tc_fence_after();
          }
          sm100::mma_f16_ts(tmem + 2 * kTile + kTile * i, tmem + kTile * i + 8 * ks, v + ks * (2048 / 16), ipv,
                            (j | ks) != 0);
        }
      };
      ok = sm100::mbar_poll_abort(&k_full[0], 0, &s_abort, p.err, 103);
      for (int i = 0; i < 2 && ok; ++i)
        if (cnt[i]) {
          ok = sm100::mbar_poll_abort(&q_full[i], 0, &s_abort, p.err, 104);
          if (ok) logits(i, 0);
        }
      if (ok) sm100::mma_commit(&k_empty[0]);
      for (int j = 0; j < tiles && ok; ++j) {
        const int st = j % kStages, nx = (j + 1) % kStages;
        bool have_v = false, have_k = false;
        for (int i = 0; i < 2 && ok; ++i) {
          if (j >= cnt[i]) continue;
          ok = sm100::mbar_poll_abort(&p_half[i], (uint32_t)(j & 1), &s_abort, p.err, 105);
          if (ok && !have_v) {
            ok = j < tail ? sm100::mbar_poll_abort(&v_full[st], (uint32_t)((j / kStages) & 1), &s_abort, p.err, 106)
                          : sm100::mbar_poll_abort(&t_ok[(j - tail) % kStages], (uint32_t)(((j - tail) / kStages) & 1),
                                                   &s_abort, p.err, 107);
            have_v = true;
          }
          if (!ok) break;
          sm100::tc_fence_after();
          output(i, j);
          if (!ok) break;
          if (j + 1 < cnt[i]) {
            if (!have_k) ok = sm100::mbar_poll_abort(&k_full[nx], (uint32_t)(((j + 1) / kStages) & 1), &s_abort, p.err, 108);
            have_k = true;
            if (ok) logits(i, j + 1);
          } else {
            sm100::mma_commit(&s_full[i]);  // the tile's output is complete
          }
        }
        if (!ok) break;
        sm100::mma_commit(&v_empty[st]);
        if (j + 1 < tiles) sm100::mma_commit(&k_empty[nx]);
      }
    }
  } else if (warp >= kGuardWarp) {
    // the tail's stage s of t_full is the stage its tile lies in; t_ok counts
    // tail tiles from 0
    for (int j = tail; j < tiles; ++j) {
      const int st = j % kStages, u = j - tail;
      if (!sm100::mbar_wait_abort(&t_full[st], (uint32_t)((u / kStages) & 1), &s_abort, p.err, 109)) break;
      guard_values<D, BF16>(smem + SM::kV + st * SM::kOne, j * kTile, t0, n, &s_bad);
      sm100::mbar_arrive(&t_ok[u % kStages]);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    if (cnt[warp >> 2]) {
    const int i = warp >> 2, r = tid & (kTile - 1);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s = tmem + kTile * i + lanes, o = tmem + 2 * kTile + kTile * i + lanes;
    const int first = t0 + i * p.tokens, token = first + r / p.group;
    flash::Row row;
    bool ok = true;
    for (int j = 0; j < cnt[i]; ++j) {
      ok = sm100::mbar_poll_abort(&s_full[i], (uint32_t)(j & 1), &s_abort, p.err, 110);
      if (!ok) break;
      sm100::tc_fence_after();
      if ((j + 1) * kTile > first + 1)
        flash::softmax_tile<D, BF16, true, 2>(s, o, j == 0, p.mult, token + 1 - j * kTile, row, &p_half[i], &p_full[i]);
      else
        flash::softmax_tile<D, BF16, false, 2>(s, o, j == 0, p.mult, 0, row, &p_half[i], &p_full[i]);
    }
    if (ok) ok = sm100::mbar_poll_abort(&s_full[i], (uint32_t)(cnt[i] & 1), &s_abort, p.err, 111);
    if (ok) {
      sm100::tc_fence_after();
      const float inv = 1.0f / row.sum;
      const bool mine = r < p.tokens * p.group && token < n;
      const bool bad = *(volatile int *)&s_bad != 0;
      uint16_t *to = static_cast<uint16_t *>(p.out) + (int64_t)(start + token) * p.ldo +
                     (int64_t)(head * p.group + r % p.group) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        sm100::tmem_ld32(o + c, v);
        sm100::tmem_wait_ld();
        if (!mine) continue;
        float2 *f = reinterpret_cast<float2 *>(v);
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = flash::mul2(f[k], make_float2(inv, inv));
        if (bad) {  // add what guard_values took out, where this row sees it
          for (int key = t0 + 1; key <= token; ++key) {
            const uint16_t *vr = p.v + (int64_t)(start + key) * p.ldv + (int64_t)head * D + c;
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const uint32_t b = vr[k];
              if (!finite16<BF16>(b)) {
                const float a = BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((uint16_t)b));
                v[k] = __float_as_uint(__uint_as_float(v[k]) + a);
              }
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4 *>(to + c + 8 * k) =
              make_uint4(flash::pack16<BF16>(f[4 * k]), flash::pack16<BF16>(f[4 * k + 1]),
                         flash::pack16<BF16>(f[4 * k + 2]), flash::pack16<BF16>(f[4 * k + 3]));
      }
    }
  }
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (s_abort) {
    // a role gave up: what is in flight is waited for (bounded) before the
    // block's memory is released
    if (warp == kMmaWarp && lane == 0) {
      __shared__ uint64_t last;
      sm100::mbar_init(&last, 1);
      sm100::fence_barrier_init();
      sm100::mma_commit(&last);
      sm100::mbar_wait(&last, 0, p.err, 112);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) sm100::tmem_dealloc(tmem, 512);
}

// [tokens][heads][d] of 16-bit elements, rows ld elements apart, as a tensor map of boxes 64 x bh x bt
bool make_map(CUtensorMap *m, bool bf16, const void *base, int64_t d, int64_t heads, int64_t tokens, int64_t ld, int bh,
              int bt) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)bh, (cuuint32_t)bt}, one[3] = {1, 1, 1};
  return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base),
            dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16>
tq_status launch_prompt(const PromptArgs &a, int *err, cudaStream_t st) {
  const int group = (int)(a.heads / a.kv_heads), tokens = kTile / group;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, BF16, a.y, D, a.heads, a.total, a.ldy, group, tokens) ||
      !make_map(&mk, BF16, a.k, D, a.kv_heads, a.total, a.ldk, 1, kTile) ||
      !make_map(&mv, BF16, a.v, D, a.kv_heads, a.total, a.ldv, 1, kTile))
    return TQ_ERR_CUDA;
  PromptParams p{};
  p.cu = a.cu;
  p.nseq = (int)a.nseq;
  p.kv_heads = (int)a.kv_heads;
  p.group = group;
  p.tokens = tokens;
  p.total = a.total;
  p.v = static_cast<const uint16_t *>(a.v);
  p.ldv = a.ldv;
  p.ldo = a.ldo;
  // 0 would turn a masked logit, -inf, into a NaN
  p.mult = std::min(std::max(std::fabs(a.scale) * 1.4426950408889634f, FLT_MIN), FLT_MAX);
  p.negative = a.scale < 0.f;
  p.out = a.out;
  p.err = err;
  // at most one started span per sequence beside the whole ones
  const int64_t blocks = (a.total / (2 * tokens) + std::min(a.nseq, a.total)) * a.kv_heads;
  if (blocks > 0x7fffffff) return TQ_ERR_TOO_LARGE;
  auto kern = k_attend_prompt<D, BF16>;
  constexpr int smem = PromptSmem<D>::kBytes;
  static std::atomic<uint64_t> ready{0};
  const tq_status rc = once_per_device(ready, [&] {
    cudaFuncAttributes fa;  // (a split of registers beyond what the block holds would wait for ever)
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess &&
           fa.numRegs * kPromptThreads >= 128 * (2 * kSoftmaxRegs + kOtherRegs) &&
           cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
  });
  if (rc != TQ_OK) return rc;
  kern<<<(unsigned)blocks, kPromptThreads, smem, st>>>(mq, mk, mv, p);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace

tq_status attend_prompt_launch(const tq_quantizer *q, const PromptArgs &a, cudaStream_t st) {
  const bool bf16 = a.dtype == TQ_BF16;
  if (q->d == 64) return bf16 ? launch_prompt<64, true>(a, q->d_err, st) : launch_prompt<64, false>(a, q->d_err, st);
  return bf16 ? launch_prompt<128, true>(a, q->d_err, st) : launch_prompt<128, false>(a, q->d_err, st);
}

}  // namespace tq
