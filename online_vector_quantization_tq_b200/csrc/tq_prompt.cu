// Causal attention of whole prompts on raw 16-bit queries, keys and values
// (packed sequences, grouped heads): what a server runs on a prompt before
// its keys and values are quantized into the cache.
//
//   o_t = sum_{j <= t} softmax_j(scale <q_t, k_j>) v_j,  sequence by sequence
//
// A work item is two tiles of 128 query rows of one sequence and KV head.  A
// row is a (token, query head of the group) pair, so a tile of a group of g
// heads covers 128 / g tokens (rounded down): with grouped heads a short prompt
// still fills its tiles, the keys behind the diagonal that a tile computes for
// nothing are fewer, and each key tile is fetched once for all heads of its
// group.  The two tiles share the key and value tiles and take turns on the
// tensor cores: while one tile's logits pass through its softmax warps, the
// other's products run.
//
// One block per SM stays for the whole call (it uses all of TMEM) and takes
// items in turn, longest first and in alternating order from round to round, so
// that the blocks' sums come out nearly equal: the number of key tiles grows
// with the position in the sequence.  Each role goes on to the next item as
// soon as its part of one is done: the next queries and keys are fetched, and
// their logits computed, while the last outputs are written.  (A block per item
// took 332 us instead of 262 on 16 ragged prompts of up to 2011 tokens.)
//
//   warps 0-3, 4-7  softmax of tile 0 and 1 (tq_flash.cuh), and their output
//   warp 8          finds the items; TMA: queries, then key and value tiles of
//                   128 keys
//   warp 9          tcgen05: S = Q K^T from shared memory, O += P V with P in
//                   TMEM and V (keys x D) as an MN-major operand
//   warps 10-11     look at value tiles before they are used: see guard_values
//
// A tile's output has a barrier of its own (o_full): the next item's logits may
// complete s_full before the softmax has come to look at the output.
//
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
// The search for work items (Items): sequences of a group, groups at most, sequences whose levels are kept
constexpr int kGroup = 128, kGroups = 2048, kCached = 4096;
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
  static constexpr int kMost = kV + kStages * kOne, kLevels = kMost + 4 * kGroups;  // of Items
  static constexpr int kBytes = kLevels + 4 * kCached + 1024;
};

// The items, longest first.  A sequence of n tokens has ceil(n / span) levels
// (span: the tokens of two tiles); level L sees about L + 1 times the keys of
// level 0.  Items are ordered by falling level, then sequence, then KV head.
// Used by one warp, which asks for them in this order.  Levels of up to 128
// sequences stay in registers, and an item's level is found by bisection.  Of
// more, in groups of 128, the search goes on from where it found the last item:
// over a call it looks once at each level of the groups that have it.  (512
// prompts of up to 100 tokens: 270 us; bisecting anew for each item 710 us.  Three
// prompts of up to 4100 tokens, whose 228 levels hold few items each: 98 us; by
// walking down the levels 118 us.)  In shared memory: each group's highest level,
// and the levels of the first kCached sequences.

struct Items {
  const int *cached, *most;  // levels, and of each group the highest
  int few[4];                // the levels of up to 128 sequences
  int level, group;          // the place: groups from here on that have `level`
  int64_t before;            // items per head in front of it

  static __device__ int start_of(const PromptParams &p, int i) {
    return (int)min(max((int64_t)__ldg(p.cu + i), (int64_t)0), p.total);
  }
  static __device__ int length(const PromptParams &p, int i) {
    const int a = start_of(p, i);
    return (int)(min(max((int64_t)__ldg(p.cu + i + 1), (int64_t)a), p.total) - a);
  }
  static __device__ int levels_of(const PromptParams &p, int i) {
    const int span = 2 * p.tokens;
    return i < p.nseq ? (length(p, i) + span - 1) / span : 0;
  }
  static __device__ int groups_of(const PromptParams &p) { return (p.nseq + kGroup - 1) / kGroup; }
  // Before the search, by all warps
  static __device__ void prepare(const PromptParams &p, int *cached, int *most, int warp, int warps) {
    const int lane = threadIdx.x & 31;
    for (int g = warp; g < ((groups_of(p) + 31) & ~31); g += warps) {
      int top = 0;
#pragma unroll
      for (int e = 0; e < kGroup / 32; ++e) {
        const int seq = g * kGroup + 32 * e + lane, n = levels_of(p, seq);
        if (seq < kCached) cached[seq] = n;
        top = max(top, n);
      }
      top = (int)__reduce_max_sync(0xffffffffu, (unsigned)top);
      if (lane == 0) most[g] = top;
    }
  }
  // levels of the lane's sequences of group g
  __device__ void load(const PromptParams &p, int g, int (&n)[4]) const {
#pragma unroll
    for (int e = 0; e < kGroup / 32; ++e) {
      const int seq = g * kGroup + 32 * e + (threadIdx.x & 31);
      n[e] = (g + 1) * kGroup <= kCached ? cached[seq] : levels_of(p, seq);
    }
  }
  __device__ Items(const PromptParams &p, const int *levels, const int *tops)
      : cached(levels), most(tops), level(0), group(0), before(0) {
    for (int g = threadIdx.x & 31; g < groups_of(p); g += 32) level = max(level, most[g]);
    level = (int)__reduce_max_sync(0xffffffffu, (unsigned)level) - 1;
    load(p, 0, few);
  }
  // of up to 128 sequences: items per head of a level above L
  __device__ int64_t above(int L) const {
    int64_t c = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) c += __reduce_add_sync(0xffffffffu, (unsigned)max(0, few[e] - L - 1));
    return c;
  }
  // item (level, KV head, first token and length of its sequence), no earlier one than the last; false behind the end
  __device__ bool find(const PromptParams &p, int64_t index, int4 &item) {
    const int64_t rank = index < 0x7fffffff ? (uint32_t)index / (uint32_t)p.kv_heads : index / p.kv_heads;
    item.y = (int)(index - rank * p.kv_heads);
    if (p.nseq <= kGroup) {
      if (rank >= above(-1)) return false;
      int lo = -1;  // above(lo) > rank >= above(level)
      while (level - lo > 1) {
        const int mid = (level + lo) / 2;
        if (above(mid) > rank)
          lo = mid;
        else
          level = mid;
      }
      before = above(level);
    }
    const int lane = threadIdx.x & 31, groups = groups_of(p);
    for (; level >= 0; --level, group = 0)
      while (group < groups) {
        const int g0 = group & ~31;
        const uint32_t have = __ballot_sync(0xffffffffu, g0 + lane >= group && most[g0 + lane] > level);
        if (have == 0) {
          group = g0 + 32;
          continue;
        }
        group = g0 + __ffs(have) - 1;
        int n[4], count = 0;
        if (p.nseq <= kGroup) {
#pragma unroll
          for (int e = 0; e < 4; ++e) n[e] = few[e];
        } else {
          load(p, group, n);
        }
        uint32_t m[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m[e] = __ballot_sync(0xffffffffu, n[e] > level);
          count += __popc(m[e]);
        }
        if (rank >= before + count) {
          before += count;
          ++group;
          continue;
        }
        int left = (int)(rank - before);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (left >= 0 && left < __popc(m[e])) {
            const int seq = group * kGroup + 32 * e + __fns(m[e], 0, left + 1);
            item.x = level;
            item.z = start_of(p, seq);
            item.w = length(p, seq);
          }
          left -= __popc(m[e]);
        }
        return true;
      }
    return false;
  }
};

// What the roles need to know of an item
struct Work {
  int head, start, n;
  int t0;             // first token, in the sequence
  int cnt[2], tiles;  // key tiles of the two query tiles (the second may lie behind the end), the larger
  int tail;           // tiles from here on hold keys that some row does not see
  __device__ Work(const PromptParams &p, int4 item) : head(item.y), start(item.z), n(item.w) {
    t0 = item.x * 2 * p.tokens;
    cnt[0] = (min(t0 + p.tokens, n) + kTile - 1) / kTile;
    cnt[1] = t0 + p.tokens < n ? (min(t0 + 2 * p.tokens, n) + kTile - 1) / kTile : 0;
    tiles = max(cnt[0], cnt[1]);
    tail = (t0 + 1) / kTile;
  }
};

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
// So in the tiles that some row of the item does not see whole, rows behind the end of the
// sequence (another sequence's) are cleared, and values that are not finite
// are cleared with *bad set; the rows that do see them add them at the end.
// Rows up to and including `first` are seen by every query row of the item.
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
  __shared__ uint64_t q_full[2], q_empty[2], k_full[kStages], k_empty[kStages], v_full[kStages], v_ok[kStages],
      v_empty[kStages], s_full[2], p_half[2], p_full[2], o_full[2], item_full[2], item_empty[2];
  __shared__ uint32_t s_tmem;
  __shared__ int4 s_item[2];  // x < 0: no more
  // whether an item's values had to be cleared; the guard is at most two items ahead of the softmax
  __shared__ int s_bad[8];
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  int *levels = reinterpret_cast<int *>(smem + SM::kLevels), *most = reinterpret_cast<int *>(smem + SM::kMost);
  Items::prepare(p, levels, most, kPromptThreads / 32 - 1 - warp, kPromptThreads / 32);
  if (warp == 0 && lane == 0) {
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&q_full[i], 1);
      sm100::mbar_init(&q_empty[i], 1);
      sm100::mbar_init(&s_full[i], 1);
      sm100::mbar_init(&p_half[i], kTile);
      sm100::mbar_init(&p_full[i], kTile);
      sm100::mbar_init(&o_full[i], 1);
      sm100::mbar_init(&item_full[i], 1);
      sm100::mbar_init(&item_empty[i], 2 * kTile + 64 + 1);
    }
    for (int i = 0; i < kStages; ++i) {
      sm100::mbar_init(&k_full[i], 1);
      sm100::mbar_init(&k_empty[i], 1);
      sm100::mbar_init(&v_full[i], 1);
      sm100::mbar_init(&v_ok[i], 64);
      sm100::mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 8; ++i) s_bad[i] = 0;
    s_abort = 0;
    sm100::fence_barrier_init();
  } else if (warp == kLoadWarp && lane == 0) {
    sm100::prefetch_tmap(&mq);
    sm100::prefetch_tmap(&mk);
    sm100::prefetch_tmap(&mv);
  } else if (warp == kMmaWarp) {
    sm100::tmem_alloc(&s_tmem, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = s_tmem;
  // The items of the block as its roles take them: item k is in s_item[k & 1];
  // a tile's position counts the key tiles of all items.
  auto take = [&](int k, int4 &item) {
    if (!sm100::mbar_wait_abort(&item_full[k & 1], (uint32_t)((k >> 1) & 1), &s_abort, p.err, 118)) return false;
    item = s_item[k & 1];
    sm100::mbar_arrive(&item_empty[k & 1]);
    return item.x >= 0;
  };
  auto phase = [](int pos) { return (uint32_t)((pos / kStages) & 1); };

  if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      const uint32_t qbytes = (uint32_t)p.group * p.tokens * 128 * (D / 64);
      Items items(p, levels, most);
      int keys = 0, values = 0, queries[2] = {0, 0};  // copies issued
      for (int k = 0;; ++k) {
        const int64_t round = (int64_t)k * gridDim.x;
        int4 item = make_int4(-1, 0, 0, 0);
        const bool some = items.find(p, round + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x), item);
        if (!some) item.x = -1;
        bool ok = true;
        if (lane == 0) {
          if (k >= 2) ok = sm100::mbar_wait_abort(&item_empty[k & 1], (uint32_t)(((k >> 1) - 1) & 1), &s_abort, p.err, 119);
          if (ok) {
            s_item[k & 1] = item;
            sm100::mbar_arrive(&item_full[k & 1]);
          }
          if (ok && some) {
            const Work w(p, item);
            auto load_kv = [&](uint8_t *dst, const CUtensorMap *m, int j, uint64_t *bar) {
              sm100::mbar_expect_tx(bar, SM::kOne);
              for (int h = 0; h < D / 64; ++h)
                tma_load_3d(dst + h * SM::kHalf, m, 64 * h, w.head, w.start + j * kTile, bar);
            };
            for (int j = 0; j < w.tiles && ok; ++j) {
              const int st = keys % kStages;
              if (keys >= kStages) ok = sm100::mbar_wait_abort(&k_empty[st], phase(keys - kStages), &s_abort, p.err, 101);
              if (!ok) break;
              load_kv(smem + SM::kK + st * SM::kOne, &mk, j, &k_full[st]);
              ++keys;
              for (int i = 0; i < 2 && j == 0 && ok; ++i) {
                if (!w.cnt[i]) continue;
                if (queries[i])
                  ok = sm100::mbar_wait_abort(&q_empty[i], (uint32_t)((queries[i] - 1) & 1), &s_abort, p.err, 120);
                if (!ok) break;
                sm100::mbar_expect_tx(&q_full[i], qbytes);
                for (int h = 0; h < D / 64; ++h)
                  tma_load_3d(smem + SM::kQ + i * SM::kOne + h * SM::kHalf, &mq, 64 * h, w.head * p.group,
                              w.start + w.t0 + i * p.tokens, &q_full[i]);
                ++queries[i];
              }
              if (ok && values >= kStages)
                ok = sm100::mbar_wait_abort(&v_empty[st], phase(values - kStages), &s_abort, p.err, 102);
              if (!ok) break;
              load_kv(smem + SM::kV + st * SM::kOne, &mv, j, &v_full[st]);
              ++values;
            }
          }
        }
        if (!some || __shfl_sync(0xffffffffu, (int)ok, 0) == 0) break;
      }
      // no copy is in flight when the block ends, whichever role gave up
      if (lane == 0)
        for (int i = 1; i <= kStages; ++i) {
          if (keys >= i) sm100::mbar_wait(&k_full[(keys - i) % kStages], phase(keys - i), p.err, 113);
          if (values >= i) sm100::mbar_wait(&v_full[(values - i) % kStages], phase(values - i), p.err, 114);
          if (queries[i - 1]) sm100::mbar_wait(&q_full[i - 1], (uint32_t)((queries[i - 1] - 1) & 1), p.err, 116);
        }
    } else if (warp == kMmaWarp) {
      if (sm100::elect_one()) {
        const uint32_t type = BF16 ? sm100::idesc_bf16_f32(kTile, kTile) : sm100::idesc_f16_f32(kTile, kTile);
        const uint32_t iqk = type | (p.negative ? 1u << 13 : 0u);  // negate A
        const uint32_t ipv = (BF16 ? sm100::idesc_bf16_f32(kTile, D) : sm100::idesc_f16_f32(kTile, D)) | (1u << 16);
        const uint32_t base = sm100::smem_u32(smem);
        int nq[2] = {0, 0}, np[2] = {0, 0};  // uses of q_full, of p_half and p_full so far
        bool ok = true;
        auto logits = [&](int i, int pos, bool last) {
          // (a step along the operand advances the descriptor's address field, in units of 16 bytes)
          const uint64_t q = sm100::desc_sw128(base + SM::kQ + i * SM::kOne);
          const uint64_t k = sm100::desc_sw128(base + SM::kK + (pos % kStages) * SM::kOne);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t off = ((ks / 4) * SM::kHalf + (ks % 4) * 32) / 16;
            sm100::mma_f16(tmem + kTile * i, q + off, k + off, iqk, ks != 0);
          }
          sm100::mma_commit(&s_full[i]);
          if (last) sm100::mma_commit(&q_empty[i]);
        };
        auto output = [&](int i, int pos, bool fresh) {
          const uint64_t v = sm100::desc_sw128_mn(base + SM::kV + (pos % kStages) * SM::kOne, SM::kHalf, 1024);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) {
            if (ks == kTile / 32) {  // the weights' second half
              ok = sm100::mbar_poll_abort(&p_full[i], (uint32_t)(np[i]++ & 1), &s_abort, p.err, 117);
              if (!ok) return;
              sm100::tc_fence_after();
            }
            sm100::mma_f16_ts(tmem + 2 * kTile + kTile * i, tmem + kTile * i + 8 * ks, v + ks * (2048 / 16), ipv,
                              !fresh || ks != 0);
          }
        };
        int4 item;
        for (int k = 0, pos = 0; ok && take(k, item); ++k) {
          const Work w(p, item);
          ok = sm100::mbar_poll_abort(&k_full[pos % kStages], phase(pos), &s_abort, p.err, 103);
          for (int i = 0; i < 2 && ok; ++i)
            if (w.cnt[i]) {
              ok = sm100::mbar_poll_abort(&q_full[i], (uint32_t)(nq[i]++ & 1), &s_abort, p.err, 104);
              if (ok) logits(i, pos, w.cnt[i] == 1);
            }
          if (ok) sm100::mma_commit(&k_empty[pos % kStages]);
          for (int j = 0; j < w.tiles && ok; ++j, ++pos) {
            bool have_v = false, have_k = false;
            for (int i = 0; i < 2 && ok; ++i) {
              if (j >= w.cnt[i]) continue;
              ok = sm100::mbar_poll_abort(&p_half[i], (uint32_t)(np[i] & 1), &s_abort, p.err, 105);
              if (ok && !have_v) ok = sm100::mbar_poll_abort(&v_ok[pos % kStages], phase(pos), &s_abort, p.err, 107);
              have_v = true;
              if (!ok) break;
              sm100::tc_fence_after();
              output(i, pos, j == 0);
              if (!ok) break;
              if (j + 1 < w.cnt[i]) {
                if (!have_k)
                  ok = sm100::mbar_poll_abort(&k_full[(pos + 1) % kStages], phase(pos + 1), &s_abort, p.err, 108);
                have_k = true;
                if (ok) logits(i, pos + 1, j + 2 == w.cnt[i]);
              } else {
                sm100::mma_commit(&o_full[i]);  // the tile's output is complete
              }
            }
            if (!ok) break;
            sm100::mma_commit(&v_empty[pos % kStages]);
            if (j + 1 < w.tiles) sm100::mma_commit(&k_empty[(pos + 1) % kStages]);
          }
        }
      }
    } else {
      int4 item;
      bool ok = true;
      for (int k = 0, pos = 0; ok && take(k, item); ++k) {
        const Work w(p, item);
        if (tid == 32 * kGuardWarp) s_bad[(k + 4) & 7] = 0;
        for (int j = 0; j < w.tiles; ++j, ++pos) {
          const int st = pos % kStages;
          ok = sm100::mbar_wait_abort(&v_full[st], phase(pos), &s_abort, p.err, 109);
          if (!ok) break;
          if (j >= w.tail)
            guard_values<D, BF16>(smem + SM::kV + st * SM::kOne, j * kTile, w.t0, w.n, &s_bad[k & 7]);
          sm100::mbar_arrive(&v_ok[st]);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2, r = tid & (kTile - 1);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s = tmem + kTile * i + lanes, o = tmem + 2 * kTile + kTile * i + lanes;
    int ns = 0, no = 0;  // uses of s_full, of o_full
    int4 item;
    bool ok = true;
    for (int k = 0; ok && take(k, item); ++k) {
      const Work w(p, item);
      const int cnt = i ? w.cnt[1] : w.cnt[0];
      if (!cnt) continue;
      const int first = w.t0 + i * p.tokens, token = first + r / p.group;
      flash::Row row;
      for (int j = 0; j < cnt; ++j) {
        ok = sm100::mbar_poll_abort(&s_full[i], (uint32_t)(ns++ & 1), &s_abort, p.err, 110);
        if (!ok) break;
        sm100::tc_fence_after();
        if ((j + 1) * kTile > first + 1)
          flash::softmax_tile<D, BF16, true, 2>(s, o, j == 0, p.mult, token + 1 - j * kTile, row, &p_half[i],
                                                &p_full[i]);
        else
          flash::softmax_tile<D, BF16, false, 2>(s, o, j == 0, p.mult, 0, row, &p_half[i], &p_full[i]);
      }
      if (ok) ok = sm100::mbar_poll_abort(&o_full[i], (uint32_t)(no++ & 1), &s_abort, p.err, 111);
      if (!ok) break;
      sm100::tc_fence_after();
      const float inv = 1.0f / row.sum;
      const bool mine = r < p.tokens * p.group && token < w.n;
      const bool bad = *(volatile int *)&s_bad[k & 7] != 0;
      uint16_t *to = static_cast<uint16_t *>(p.out) + (int64_t)(w.start + token) * p.ldo +
                     (int64_t)(w.head * p.group + r % p.group) * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        sm100::tmem_ld32(o + c, v);
        sm100::tmem_wait_ld();
        if (!mine) continue;
        float2 *f = reinterpret_cast<float2 *>(v);
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = flash::mul2(f[e], make_float2(inv, inv));
        if (bad) {  // add what guard_values took out, where this row sees it
          for (int key = w.t0 + 1; key <= token; ++key) {
            const uint16_t *vr = p.v + (int64_t)(w.start + key) * p.ldv + (int64_t)w.head * D + c;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t b = vr[e];
              if (!finite16<BF16>(b)) {
                const float x = BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((uint16_t)b));
                v[e] = __float_as_uint(__uint_as_float(v[e]) + x);
              }
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4 *>(to + c + 8 * e) =
              make_uint4(flash::pack16<BF16>(f[4 * e]), flash::pack16<BF16>(f[4 * e + 1]),
                         flash::pack16<BF16>(f[4 * e + 2]), flash::pack16<BF16>(f[4 * e + 3]));
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
  const int64_t most = (a.total / (2 * tokens) + std::min(a.nseq, a.total)) * a.kv_heads;
  const int64_t blocks = std::min<int64_t>(most, current_sms());
  auto kern = k_attend_prompt<D, BF16>;
  constexpr int smem = PromptSmem<D>::kBytes;
  static_assert(smem <= 232448 - 1024, "shared memory");
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
