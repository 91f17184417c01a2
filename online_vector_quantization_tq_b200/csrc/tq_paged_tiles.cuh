// Attention of many query rows over a sequence's pages (chunks of a prompt,
// long drafts): the kernel of tq_attend_paged for sequences of more rows than
// the kernel of few rows should take.  Instantiated in tq_paged_many_*.cu.
//
// As the prompt kernel (tq_flash.cuh has the softmax), with key and value tiles
// that are expanded from the packed pages instead of copied: both products run
// on tcgen05 with fp16 operands.  A row's operand is its centroids times its
// norm, scaled down by a power of two that is above all norms of the tile, and
// that the softmax takes back.  A norm less than 1 / kSpread of its tile's scale
// (which the row may not even see) is scaled by a power of two of its own, and
// the tile's softmax looks at factors per key.  Each thread makes a table of its
// row's 2^w possible values, so that every element is rounded once, and the
// softmax of a tile without such norms meets no factors per key.  (As fp32
// factors of logits and weights the norms make the softmax the bound: see LOW.)
// Inner-product keys are operands of twice the width, [c | +-64 gamma
// sqrt(pi/2)/d] times the norm, against queries [R y | S R y / 64].
//
// fp16 results (LOW) would show the rounding of these operands: their centroids
// are operands under the codebook's common factor, within 2^-13, with the norms as
// fp32 factors of logits and weights, and the rotated queries' low terms are
// multiplied too, as a third part [R y | S R y / 64 | low] of the query tile,
// against the centroids once more.  (Error against 64 bits, 2-norm over 2-norm:
// 3.1e-4, 2.0e-4 of it the result's own rounding, against 1.5e-3 with the others'
// operands; 512 new tokens on 16384 keys 302 us against 228.)  The residual norms
// of inner-product keys stay operands; each key takes the one of 16 common factors
// (and its table of centroids) that brings its residual norm nearest to an fp16
// number, a seventh of what rounding it would cost.  (Keys of 2 bits, whose sign
// bits make the most of a logit: 4.6e-4, with one factor for all 1.15e-3.)
//
// One block per SM works off its run of units (PagedCut; a unit is a tile of
// 128 keys).  Two warpgroups of softmax share the tensor cores:
//   a block of more than 128 rows: each has a tile of 128 of the rows, and
//     both go through the same key tiles;
//   fewer rows (and, at d = 128, inner-product keys and fp16, whose two query
//     tiles would leave no room for keys): both have the same rows, and take the
//     key tiles in turn; their results are added up at the end.
//
//   warps 0-3, 4-7   softmax; they also fetch their queries and put out results
//   warps 8-11       expand keys, one row a thread; norms
//   warps 12-15      expand values, one row a thread
//   warp 16          tcgen05
//
// Between the issuing thread and a softmax warpgroup the barriers alternate: a
// segment's queries (q_full), then per tile its logits (s_full) and its weights
// (p_half, p_full), at last its output (o_full).  Neither side completes a
// barrier's next phase before the other has seen the last one: a warpgroup
// without a tile in a segment neither arrives on q_full nor is waited for, and
// the output has a barrier of its own, since the next segment's logits may
// complete s_full before the warpgroup has come to look at the output.
//
// Keys and values share one ring of slots (a tile of 16-bit rows, 128-byte
// swizzle), in the order in which the products first need them.
#pragma once

#include "tq_expand.cuh"
#include "tq_flash.cuh"
#include "tq_paged.cuh"

namespace tq {

namespace {

using namespace paged;

constexpr int kTile = 128;
constexpr int kTilesThreads = 640;  // warps 17-19 only complete the last warpgroup
// Registers move to the softmax: a warpgroup's share, whose sum is no more
// than the block was launched with (launch_tiles checks).  (512 new tokens on
// 16384 keys, us: 128 / 72 / 72 254, 136 / 72 / 64 247, 136 / 80 / 48 249, these 233.)
constexpr int kSoftmaxRegs = 144, kExpandRegs = 72, kMmaRegs = 48;
constexpr int kKeyWarp = 8, kValueWarp = 12, kMmaWarp = 16;
constexpr float kSpread = 512.f;  // (kept bits: 11 of the largest centroids, 8 or so of the smallest)
constexpr int kNorms = 8;  // tiles whose scales are kept: more than the ring holds

template <int D, bool IP, bool LOW>
struct TileSmem {
  static constexpr int kHalf = kTile * 128;              // 128 rows of 64 elements
  static constexpr int kSlot = kHalf * (D / 64);
  static constexpr int kSlots = D == 64 ? (IP && LOW ? 6 : 8) : (IP && LOW ? 3 : 4);
  static constexpr int kWide = IP ? 2 : 1;               // slots of a key tile
  static constexpr int kParts = kWide + (LOW ? 1 : 0);   // of a query tile
  static constexpr int kQTiles = (IP || LOW) && D == 128 ? 1 : 2;
  static constexpr int kRows = kTile * kQTiles;          // rows of a block
  static constexpr int kQ = 0, kQTile = kSlot * kParts, kRing = kQTiles * kQTile;
  // a factor of each key's logit, below 0 for a key on a bad page, and of its value
  static constexpr int kKeys = kRing + kSlots * kSlot, kValues = kKeys + kNorms * kTile * 4;
  static_assert(kNorms * kTile == flash::kFactors, "where the softmax finds the factors of values");
  static constexpr int kExps = kValues + kNorms * kTile * 4;  // LOW: the values' exponents
  static constexpr int kBytes = kExps + (LOW ? kNorms * kTile * 4 : 0) + 1024;
};

// Ring positions of key and value tiles: `lead` key tiles first (one where both
// warpgroups see every tile, two where they take turns), then a value tile and
// the next key tile by turns.  Keys and values are filled by different warps,
// each of which sees of a slot's barrier only the phase's parity; a phase is
// told from the one before the last because a filler's positions are never
// more than the ring's slots apart, and slots become free in (nearly) the order
// of their positions.  Where every key tile has two of the four slots, starting
// each segment with its own lead would set value tiles five apart: there (and
// with three slots) the order runs on from one segment to the next.
template <int WIDE, bool ON>
struct RingPlan {
  int lead, tiles;
  int base, before;  // position of the segment's first slot; key tiles before the segment
  __device__ int value(int j) const {
    if (ON) return 2 * WIDE + (before + j) * (WIDE + 1);
    return base + min(lead, tiles) * WIDE + j + WIDE * min(j, max(tiles - lead, 0));
  }
  __device__ int key(int j) const {
    if (ON) return before + j < 2 ? (before + j) * WIDE : value(j - 2) + 1;
    return j < lead ? base + j * WIDE : value(j - lead) + 1;
  }
  __device__ void done() {
    base += tiles * (WIDE + 1);
    before += tiles;
  }
};

template <int D, bool IP, bool LOW>
using Ring = RingPlan<TileSmem<D, IP, LOW>::kWide, IP && D == 128>;

// Tiles of a segment, as every role sees them
struct Segment {
  bool turns;     // the warpgroups take key tiles in turn
  int row0, rows; // first row of the block, rows of the sequence
  int hidden, seen;
  int t0, tiles;  // key tiles
};
template <int D, bool IP, bool LOW>
__device__ __forceinline__ Segment segment_of(const PagedParams &p, const Cursor &cur) {
  using SM = TileSmem<D, IP, LOW>;
  Segment g;
  g.rows = cur.s.n * p.group;
  g.row0 = cur.block * SM::kRows;
  g.turns = SM::kQTiles == 1 || g.rows - g.row0 <= kTile;
  g.hidden = cur.s.first;
  g.seen = seen_by(p, p.many, cur.s, cur.block);
  g.t0 = cur.unit;
  g.tiles = cur.take;
  return g;
}
// Key tiles of the segment for warpgroup i (whose first row is row0 + 128 i where they do not take turns)
__device__ __forceinline__ int tiles_of(const PagedParams &p, const Cursor &cur, const Segment &g, int i) {
  if (g.turns) return (g.tiles + 1 - i) / 2;
  const int last = min(g.row0 + kTile * (i + 1), g.rows) - 1;
  const int seen = max(0, min(cur.s.len, g.hidden + last / p.group));
  return min(max((seen + kTile - 1) / kTile - g.t0, 0), g.tiles);
}

// The values of a 32-coordinate group as four 16-byte chunks of row r, from
// chunk 4 g on.  lo, hi: byte tables of the row's values (byte_tables).
// Four-bit codebooks are symmetric, c[15 - i] = -c[i], and their tables hold the
// upper eight values alone: a code below 8 selects by its complement and has
// its sign set, 18 operations for eight codes against 23 with 16-entry tables.
template <int W>
__device__ __forceinline__ void expand_group(uint8_t *tile, int r, int g, const uint32_t *words,
                                             const uint32_t (&tlo)[4], const uint32_t (&thi)[4]) {
  uint32_t lo[8], hi[8];
  if constexpr (W == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t x = words[k], n = ~x & 0x88888888u, up = n << 4;  // n: codes below 8
      const uint32_t sel = (x ^ (n - (n >> 3))) & 0x77777777u;
      lo[2 * k] = sm100::prmt(tlo[0], tlo[1], sel);
      lo[2 * k + 1] = sm100::prmt(tlo[0], tlo[1], sel >> 16);
      hi[2 * k] = sm100::prmt(thi[0], thi[1], sel) | (sm100::prmt(up, n, 0x5140u) & 0x80808080u);
      hi[2 * k + 1] = sm100::prmt(thi[0], thi[1], sel >> 16) | (sm100::prmt(up, n, 0x7362u) & 0x80808080u);
    }
  } else {
    expand_codes<W>(words, tlo, thi, lo, hi);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int chunk = 4 * g + k;
    *reinterpret_cast<uint4 *>(tile + (chunk >> 3) * (kTile * 128) + sm100::sw128_offset(r, chunk & 7)) =
        make_uint4(sm100::prmt(lo[2 * k], hi[2 * k], 0x5140u), sm100::prmt(lo[2 * k], hi[2 * k], 0x7362u),
                   sm100::prmt(lo[2 * k + 1], hi[2 * k + 1], 0x5140u), sm100::prmt(lo[2 * k + 1], hi[2 * k + 1], 0x7362u));
  }
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t *w, const uint8_t *from) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(from) + i / 4);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  } else if constexpr (N % 2 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(from) + i / 2);
      w[i] = v.x, w[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t *>(from) + i);
  }
}

// Byte tables of a row's values: centroids times f, rounded to fp16 (of four-bit
// codes: the upper eight)
template <int W>
__device__ __forceinline__ void byte_tables(const float *c, float f, uint32_t (&lo)[4], uint32_t (&hi)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = hi[i] = 0u;
    if (4 * i < (W == 4 ? 8 : 1 << W)) {
      constexpr int kFirst = W == 4 ? 8 : 0;
      const float2 ff = make_float2(f, f);
      const uint32_t a = flash::pack16<false>(flash::mul2(make_float2(c[kFirst + 4 * i], c[kFirst + 4 * i + 1]), ff));
      const uint32_t b =
          flash::pack16<false>(flash::mul2(make_float2(c[kFirst + 4 * i + 2], c[kFirst + 4 * i + 3]), ff));
      lo[i] = sm100::prmt(a, b, 0x6420u);
      hi[i] = sm100::prmt(a, b, 0x7531u);
    }
  }
}

// The same of up to eight fp16 centroids in a row
__device__ __forceinline__ void byte_tables(uint4 c, uint32_t (&lo)[4], uint32_t (&hi)[4]) {
  lo[0] = sm100::prmt(c.x, c.y, 0x6420u), hi[0] = sm100::prmt(c.x, c.y, 0x7531u);
  lo[1] = sm100::prmt(c.z, c.w, 0x6420u), hi[1] = sm100::prmt(c.z, c.w, 0x7531u);
  lo[2] = lo[3] = hi[2] = hi[3] = 0u;
}

// The same of fp16 centroids as they are
template <int W>
__device__ __forceinline__ void byte_tables(const uint16_t *c, uint32_t (&lo)[4], uint32_t (&hi)[4]) {
  constexpr int kFirst = W == 4 ? 8 : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = hi[i] = 0u;
    if (4 * i < (W == 4 ? 8 : 1 << W)) {
      const uint32_t a = c[kFirst + 4 * i] | (uint32_t)c[kFirst + 4 * i + 1] << 16;
      const uint32_t b = c[kFirst + 4 * i + 2] | (uint32_t)c[kFirst + 4 * i + 3] << 16;
      lo[i] = sm100::prmt(a, b, 0x6420u);
      hi[i] = sm100::prmt(a, b, 0x7531u);
    }
  }
}

// A norm's part in its tile's largest: what is not finite has none
__device__ __forceinline__ float finite_or_0(float v) { return fabsf(v) < INFINITY ? v : 0.f; }
// Power of two above v (v >= 0) that scales a tile's norms, as the bits of a
// float whose reciprocal is normal too; of values no less than 2^-80
// (flash::norm_exponent)
constexpr uint32_t kLeastKey = 2, kLeastValue = 127 - 80;
__device__ __forceinline__ uint32_t scale_bits(float v, uint32_t least) {
  return min(max((__float_as_uint(v) >> 23) + 1u, least), 252u) << 23;
}
__device__ __forceinline__ float inverse_of(uint32_t bits) { return __uint_as_float(0x7F000000u - bits); }
// Whether norm v of a tile scaled by `bits` has a scale of its own
__device__ __forceinline__ bool stands_alone(float v, uint32_t bits) {
  return v > 0.f && v * kSpread < __uint_as_float(bits);
}

template <int D, bool IP, bool LOW, int WK, int WV>
__global__ void __launch_bounds__(kTilesThreads, 1) k_attend_paged_tiles(const __grid_constant__ PagedParams p) {
  using SM = TileSmem<D, IP, LOW>;
  constexpr int DQ = SM::kParts * D;  // elements of a query operand's row
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((0u - sm100::smem_u32(smem_raw)) & 1023u);
  float *s_keys = reinterpret_cast<float *>(smem + SM::kKeys), *s_values = reinterpret_cast<float *>(smem + SM::kValues);
  __shared__ uint64_t full[SM::kSlots], empty[SM::kSlots], q_full[2], s_full[2], p_half[2], p_full[2], o_full[2], merge, merged;
  __shared__ uint32_t s_tmem;
  __shared__ int64_t s_run[5];
  __shared__ int s_some, s_gap[kNorms][4];          // of a warp's keys: 1 some on a bad page, 2 some scaled by themselves
  __shared__ float s_key[kNorms], s_value[kNorms];  // 2^e of a tile's keys, exponent of its values
  __shared__ float s_top[3][2][4];                  // keys' and values' largest norms, of each warp
  __shared__ float2 s_ml[kTile];
  __shared__ uint4 s_codes[IP && LOW ? kAttendFactors : 1];  // the keys' centroids under each factor
  __shared__ float2 s_by[IP && LOW ? kAttendFactors : 1];    // the factor, and what undoes it beside p.kunit
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == 0) {
    const bool some = find_run(p, p.many, s_run);
    if (lane == 0) s_some = some;
  } else if (warp == 1 && lane == 0) {
    for (int i = 0; i < SM::kSlots; ++i) {
      sm100::mbar_init(&full[i], kTile);
      sm100::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      sm100::mbar_init(&q_full[i], kTile);
      sm100::mbar_init(&s_full[i], 1);
      sm100::mbar_init(&p_half[i], kTile);
      sm100::mbar_init(&p_full[i], kTile);
      sm100::mbar_init(&o_full[i], 1);
    }
    sm100::mbar_init(&merge, kTile);
    sm100::mbar_init(&merged, kTile);
    s_abort = 0;
    sm100::fence_barrier_init();
  } else if (IP && LOW && warp == 2 && lane < kAttendFactors) {
    const uint16_t *c = p.cks[lane];
    s_codes[lane] = make_uint4(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16, c[4] | (uint32_t)c[5] << 16,
                               c[6] | (uint32_t)c[7] << 16);
    s_by[lane] = make_float2(p.cks_by[lane], 1.0f / (p.cks_by[lane] * p.kunit));
  }
  __syncthreads();
  if (!s_some) return;
  if (warp == kMmaWarp) {
    sm100::tmem_alloc(&s_tmem, 512);
    sm100::tmem_relinquish();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::tc_fence_after();
  const uint32_t tmem = s_tmem;
  Cursor cur = start_run(p, p.many, s_run);
  Ring<D, IP, LOW> ring{1, 0, 0, 0};
  // the next segment's tiles in the ring
  auto enter = [&](const Segment &g) {
    ring.lead = g.turns ? 2 : 1;
    ring.tiles = g.tiles;
  };

  if (warp >= kKeyWarp && warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kExpandRegs));
    const bool keys = warp < kValueWarp;
    const int r = tid & (kTile - 1);
    uint32_t tlo[4], thi[4];
    auto wait_slot = [&](int at) {
      return at < SM::kSlots ||
             sm100::mbar_wait_abort(&empty[at % SM::kSlots], (uint32_t)((at / SM::kSlots - 1) & 1), &s_abort, p.err, 121);
    };
    // Largest of a norm over the warpgroup's threads, put down before `agree`
    // and read behind it, alternately in two places (a turn is the tile's number
    // in the run: were it counted anew in each segment, the last tile of one and
    // the first of the next could share a place, with no barrier between the
    // read and the write).  agree: whether any of the threads gave up (they have
    // to leave together).
    auto put_top = [&](int what, int turn, float v) {
      v = finite_or_0(v);  // not below 0: ordered as an integer
      const int top = __reduce_max_sync(0xffffffffu, __float_as_int(v));
      if (lane == 0) s_top[what][turn & 1][warp & 3] = __int_as_float(top);
    };
    auto top_of = [&](int what, int turn) {
      const float *t = s_top[what][turn & 1];
      return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
    };
    auto agree = [&](bool mine) { return !sm100::named_barrier_or(keys ? 1 : 2, kTile, !mine); };
    constexpr int kBehind = -2;  // a page index: the key lies behind those that are seen
    if constexpr (LOW) {
      if (keys && !IP)  // (of inner-product keys each has its own)
        byte_tables<WK>(p.ck, tlo, thi);
      if (!keys)
        byte_tables<WV>(p.cv, tlo, thi);
    }
    bool ok = true;
    do {
      const Segment g = segment_of<D, IP, LOW>(p, cur);
      enter(g);
      const int32_t *table = p.table + (int64_t)cur.seq * p.ldt;
      const int64_t page_rows = (int64_t)p.kv_heads * p.page_size, head_row = (int64_t)cur.head * p.page_size;
      // A tile's packed rows are loaded one tile ahead, their page indices two:
      // the loads' latency passes while the tile before is expanded.
      auto page_of = [&](int j) {
        const int key = (g.t0 + j) * kTile + r;
        if (j >= g.tiles || key >= g.seen) return kBehind;
        const int page = __ldg(table + p.page_of(key));
        return page >= 0 && page < p.npages ? page : -1;
      };
      auto row_of = [&](int j, int page) {
        const int key = (g.t0 + j) * kTile + r;
        return page * page_rows + head_row + (key - p.page_of(key) * p.page_size);
      };
      // (each group of 32 coordinates is loaded again as soon as it is used, so
      // that one row of registers is enough)
      constexpr int G = D / 32;
      int page = page_of(1);
      if (keys) {
        uint32_t w[G][WK], sw[IP ? G : 1];
        float2 n = make_float2(0.f, 0.f);
        float v = 0.f;
        {
          const int pg = page_of(0);
          const int64_t row = pg >= 0 ? row_of(0, pg) : 0;
#pragma unroll
          for (int q = 0; q < G; ++q) {
#pragma unroll
            for (int i = 0; i < WK; ++i) w[q][i] = 0u;
            if (pg >= 0) load_words<WK>(w[q], p.kcodes + row * (WK * D / 8) + q * (4 * WK));
          }
          if constexpr (IP) {
#pragma unroll
            for (int q = 0; q < G; ++q) sw[q] = 0u;
            if (pg >= 0) load_words<G>(sw, p.ksigns + row * (D / 8));
          }
          if (pg >= 0) {
            n = __ldg(p.knorms + row);
            n.x = fabsf(n.x);  // (below 0 is for what has no page)
            v = fabsf(__ldg(&p.vnorms[row].x));
          } else if (pg == -1) {
            n.x = -1.f;
          }
        }
        for (int j = 0; j < g.tiles; ++j) {
          const int pg = page;
          const int64_t row = pg >= 0 ? row_of(j + 1, pg) : 0;
          page = page_of(j + 2);
          const int at = ring.key(j), nr = (ring.before + j) % kNorms;
          if constexpr (!LOW) {
            put_top(0, ring.before + j, fmaxf(n.x, 0.f));
            put_top(1, ring.before + j, v);
          }
          ok = agree(wait_slot(at));
          if (!ok) break;
          // a norm that is not finite makes a NaN of every row that sees its key, and of no other
          const bool finite = v + n.x + (IP ? fabsf(n.y) : 0.f) < INFINITY;
          float signs_by;  // value of the sign bits' operand
          if constexpr (LOW) {
            float undo = 1.f;
            if constexpr (IP) {
              // the factor that takes the residual norm nearest to an fp16 number (in steps of fp32)
              const float g = n.y * (64.f * p.kappa);
              uint32_t best = 0xffffffffu;
#pragma unroll
              for (int k = 0; k < kAttendFactors; ++k) {
                const int off = (int)((__float_as_uint(g * p.cks_by[k]) + 0x1000u) & 0x1FFFu) - 0x1000;
                best = min(best, (uint32_t)abs(off) * kAttendFactors + k);
              }
              best %= kAttendFactors;
              byte_tables(s_codes[best], tlo, thi);
              signs_by = g * s_by[best].x;
              undo = s_by[best].y;
            }
            s_keys[nr * kTile + r] = finite ? n.x * undo : NAN;
            s_values[nr * kTile + r] = finite ? v : 0.f;
            reinterpret_cast<float *>(smem + SM::kExps)[nr * kTile + r] = flash::norm_exponent(finite ? v : 0.f);
            const int gap = __any_sync(0xffffffffu, n.x < 0.f);
            if (lane == 0) s_gap[nr][warp - kKeyWarp] = gap;
          } else {
            const uint32_t kscale = scale_bits(top_of(0, ring.before + j), kLeastKey);
            const uint32_t vscale = scale_bits(top_of(1, ring.before + j), kLeastValue);
            uint32_t kown = kscale, vown = vscale;
            if (stands_alone(n.x, kscale)) kown = scale_bits(n.x, kLeastKey);
            if (stands_alone(v, vscale)) vown = scale_bits(v, kLeastValue);
            const float f = finite ? fmaxf(n.x, 0.f) * inverse_of(kown) : NAN;
            byte_tables<WK>(p.ckf, f, tlo, thi);
            signs_by = f * n.y * (64.f * p.kappa);
            s_keys[nr * kTile + r] = n.x < 0.f ? -1.f : __uint_as_float(kown) * inverse_of(kscale);
            s_values[nr * kTile + r] = __uint_as_float(vown);
            const int gap = __any_sync(0xffffffffu, n.x < 0.f) |
                            __any_sync(0xffffffffu, kown != kscale || vown != vscale) << 1;
            if (lane == 0) s_gap[nr][warp - kKeyWarp] = gap;
            if (r == 0) {
              s_key[nr] = __uint_as_float(kscale);
              s_value[nr] = (float)((int)(vscale >> 23) - 127);
            }
          }
          uint8_t *slot = smem + SM::kRing + (at % SM::kSlots) * SM::kSlot;
#pragma unroll
          for (int q = 0; q < G; ++q) {
            expand_group<WK>(slot, r, q, w[q], tlo, thi);
            if (pg >= 0) load_words<WK>(w[q], p.kcodes + row * (WK * D / 8) + q * (4 * WK));
          }
          sm100::fence_proxy_async();
          sm100::mbar_arrive(&full[at % SM::kSlots]);
          if constexpr (IP) {
            ok = agree(wait_slot(at + 1));
            if (!ok) break;
            uint8_t *signs = smem + SM::kRing + ((at + 1) % SM::kSlots) * SM::kSlot;
            const uint32_t h = __half_as_ushort(__float2half_rn(signs_by));
            const uint32_t minus = (h | h << 16) ^ 0x80008000u;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {  // elements 2 k and 2 k + 1 of a group: bits k and k + 16 of its word
              uint32_t e[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] = ((sw[c >> 2] << (15 - (4 * (c & 3) + i))) & 0x80008000u) ^ minus;
              *reinterpret_cast<uint4 *>(signs + (c >> 3) * SM::kHalf + sm100::sw128_offset(r, c & 7)) =
                  make_uint4(e[0], e[1], e[2], e[3]);
            }
            if (pg >= 0) load_words<G>(sw, p.ksigns + row * (D / 8));
            sm100::fence_proxy_async();
            sm100::mbar_arrive(&full[(at + 1) % SM::kSlots]);
          }
          n = make_float2(pg == -1 ? -1.f : 0.f, 0.f);
          v = 0.f;
          if (pg >= 0) {
            n = __ldg(p.knorms + row);
            n.x = fabsf(n.x);
            v = fabsf(__ldg(&p.vnorms[row].x));
          }
        }
      } else {
        uint32_t w[G][WV];
        float v = 0.f;
        {
          const int pg = page_of(0);
          const int64_t row = pg >= 0 ? row_of(0, pg) : 0;
#pragma unroll
          for (int q = 0; q < G; ++q) {
#pragma unroll
            for (int i = 0; i < WV; ++i) w[q][i] = 0u;
            if (pg >= 0) load_words<WV>(w[q], p.vcodes + row * (WV * D / 8) + q * (4 * WV));
          }
          if (!LOW && pg >= 0) v = fabsf(__ldg(&p.vnorms[row].x));
        }
        for (int j = 0; j < g.tiles; ++j) {
          const int pg = page;
          const int64_t row = pg >= 0 ? row_of(j + 1, pg) : 0;
          page = page_of(j + 2);
          const int at = ring.value(j);
          if constexpr (!LOW) put_top(2, ring.before + j, v);
          ok = agree(wait_slot(at));
          if (!ok) break;
          if constexpr (!LOW) {
            uint32_t own = scale_bits(top_of(2, ring.before + j), kLeastValue);  // (as the keys' threads find it)
            if (stands_alone(v, own)) own = scale_bits(v, kLeastValue);
            byte_tables<WV>(p.cvf, finite_or_0(v) * inverse_of(own), tlo, thi);
          }
          uint8_t *slot = smem + SM::kRing + (at % SM::kSlots) * SM::kSlot;
#pragma unroll
          for (int q = 0; q < G; ++q) {
            expand_group<WV>(slot, r, q, w[q], tlo, thi);
            if (pg >= 0) load_words<WV>(w[q], p.vcodes + row * (WV * D / 8) + q * (4 * WV));
          }
          v = 0.f;
          if (!LOW && pg >= 0) v = fabsf(__ldg(&p.vnorms[row].x));
          sm100::fence_proxy_async();
          sm100::mbar_arrive(&full[at % SM::kSlots]);
        }
      }
      ring.done();
    } while (ok && cur.next(p, p.many));
  } else if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == kMmaWarp && sm100::elect_one()) {
      const uint32_t iqk = sm100::idesc_f16_f32(kTile, kTile) | (p.scale < 0.f ? 1u << 13 : 0u);  // negate A
      const uint32_t ipv = sm100::idesc_f16_f32(kTile, D) | (1u << 16);
      const uint32_t base = sm100::smem_u32(smem);
      int nq[2] = {0, 0}, np[2] = {0, 0};  // uses of q_full, of p_half and p_full so far
      bool ok = true;
      auto wait_full = [&](int at) {
        return sm100::mbar_poll_abort(&full[at % SM::kSlots], (uint32_t)((at / SM::kSlots) & 1), &s_abort, p.err, 122);
      };
      do {
        const Segment g = segment_of<D, IP, LOW>(p, cur);
        enter(g);
        const int cnt[2] = {tiles_of(p, cur, g, 0), tiles_of(p, cur, g, 1)};
        auto logits = [&](int i, int j) {  // S_i = Q K_j^T
          // (a step along the operand advances the descriptor's address field, in units of 16 bytes)
          const uint64_t q = sm100::desc_sw128(base + SM::kQ + (g.turns ? 0 : i) * SM::kQTile);
#pragma unroll
          for (int w = 0; w < SM::kWide; ++w) {
            const int at = ring.key(j) + w;
            ok = ok && wait_full(at);
            if (!ok) return;
            const uint64_t k = sm100::desc_sw128(base + SM::kRing + (at % SM::kSlots) * SM::kSlot);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = ((ks / 4) * SM::kHalf + (ks % 4) * 32) / 16;
              sm100::mma_f16(tmem + kTile * i, q + (w * SM::kSlot / 16 + off), k + off, iqk, (w | ks) != 0);
            }
            if constexpr (LOW) {
              if (w == 0)
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                  const uint32_t off = ((ks / 4) * SM::kHalf + (ks % 4) * 32) / 16;
                  sm100::mma_f16(tmem + kTile * i, q + (SM::kWide * SM::kSlot / 16 + off), k + off, iqk, true);
                }
            }
          }
          sm100::mma_commit(&s_full[i]);
        };
        auto free_keys = [&](int j) {
          for (int k = 0; k < SM::kWide; ++k) sm100::mma_commit(&empty[(ring.key(j) + k) % SM::kSlots]);
        };
        auto output = [&](int i, int j, bool fresh) {  // O_i += P_i V_j
          ok = ok && sm100::mbar_poll_abort(&p_half[i], (uint32_t)(np[i] & 1), &s_abort, p.err, 123);
          const int at = ring.value(j);
          ok = ok && wait_full(at);
          if (!ok) return;
          sm100::tc_fence_after();
          const uint64_t v = sm100::desc_sw128_mn(base + SM::kRing + (at % SM::kSlots) * SM::kSlot, SM::kHalf, 1024);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) {
            if (ks == kTile / 32) {  // the weights' second half
              ok = sm100::mbar_poll_abort(&p_full[i], (uint32_t)(np[i]++ & 1), &s_abort, p.err, 130);
              if (!ok) return;
              sm100::tc_fence_after();
            }
            sm100::mma_f16_ts(tmem + 2 * kTile + kTile * i, tmem + kTile * i + 8 * ks, v + ks * (2048 / 16), ipv,
                              !fresh || ks != 0);
          }
        };
        auto free_value = [&](int j) { sm100::mma_commit(&empty[(ring.value(j)) % SM::kSlots]); };
        for (int i = 0; i < (g.turns ? 1 : 2) && ok; ++i)
          if (cnt[i]) ok = sm100::mbar_poll_abort(&q_full[i], (uint32_t)(nq[i]++ & 1), &s_abort, p.err, 124);
        sm100::tc_fence_after();
        if (g.turns) {
          for (int j = 0; j < 2 && j < g.tiles && ok; ++j) {
            logits(j, j);
            if (ok) free_keys(j);
          }
          for (int j = 0; j < g.tiles && ok; ++j) {
            output(j & 1, j, j < 2);
            if (ok) free_value(j);
            if (ok && j + 2 < g.tiles) {
              logits(j & 1, j + 2);
              if (ok) free_keys(j + 2);
            } else if (ok) {
              sm100::mma_commit(&o_full[j & 1]);  // the warpgroup's output is complete
            }
          }
        } else {
          for (int i = 0; i < 2 && ok; ++i)
            if (cnt[i]) logits(i, 0);
          if (ok) free_keys(0);
          for (int j = 0; j < g.tiles && ok; ++j) {
            for (int i = 0; i < 2 && ok; ++i) {
              if (j >= cnt[i]) continue;
              output(i, j, j == 0);
              if (ok && j + 1 < cnt[i])
                logits(i, j + 1);
              else if (ok)
                sm100::mma_commit(&o_full[i]);
            }
            if (ok) free_value(j);
            if (ok && j + 1 < g.tiles) free_keys(j + 1);
          }
        }
        ring.done();
      } while (ok && cur.next(p, p.many));
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int i = warp >> 2, r = tid & (kTile - 1);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t S = tmem + kTile * i + lanes, O = tmem + 2 * kTile + kTile * i + lanes;
    const float unit = fabsf(p.scale) * 1.4426950408889634f * (LOW ? p.kunit : 1.f);
    int ns = 0, no = 0, nm = 0;  // uses of s_full, of o_full, of merge
    bool ok = true;
    do {
      const Segment g = segment_of<D, IP, LOW>(p, cur);
      enter(g);
      const int cnt = tiles_of(p, cur, g, i);
      const int first = g.row0 + (g.turns ? 0 : kTile * i), row = first + r;
      const bool mine = row < g.rows;
      const int64_t at = (int64_t)(cur.s.start + (mine ? row / p.group : 0)) * p.heads + cur.head * p.group +
                         (mine ? row % p.group : 0);
      const float mult = (mine ? __ldg(p.qscale + at) : 1.f) * unit;
      if (cnt && (i == 0 || !g.turns)) {
        uint8_t *q = smem + SM::kQ + i * SM::kQTile;
        const uint4 *from = reinterpret_cast<const uint4 *>(p.qprep + at * DQ);
#pragma unroll 8
        for (int c = 0; c < DQ / 8; ++c)
          *reinterpret_cast<uint4 *>(q + (c >> 3) * SM::kHalf + sm100::sw128_offset(r, c & 7)) =
              mine ? __ldg(from + c) : make_uint4(0u, 0u, 0u, 0u);
        sm100::fence_proxy_async();
        sm100::mbar_arrive(&q_full[i]);
      }
      const int lim = mine ? min(g.hidden + row / p.group, cur.s.len) : cur.s.len;
      const int lim_first = min(g.hidden + first / p.group, cur.s.len);
      flash::Row st;
      for (int n = 0; n < cnt; ++n) {
        const int j = g.turns ? 2 * n + i : n, nr = (ring.before + j) % kNorms;
        ok = sm100::mbar_poll_abort(&s_full[i], (uint32_t)(ns++ & 1), &s_abort, p.err, 125);
        if (!ok) break;
        sm100::tc_fence_after();
        const float *keys = s_keys + nr * kTile;
        const int end = (g.t0 + j + 1) * kTile, see = lim - (end - kTile);
        const int gap = s_gap[nr][0] | s_gap[nr][1] | s_gap[nr][2] | s_gap[nr][3];
        // (a factor of 0 would turn a masked logit, -inf, into a NaN)
        const float m = fminf(fmaxf(LOW ? mult : mult * s_key[nr], 1.17549435e-38f), 3.402823466e38f);
        const float scale = LOW ? 0.f : s_value[nr];
        bool done = false;
        if (gap == 0 && end <= lim_first)
          done = flash::softmax_tile_twice<D, false, LOW>(S, O, n == 0, m, 0, st, keys, scale, &p_half[i], &p_full[i]);
        else if (gap < 2)
          done = flash::softmax_tile_twice<D, true, LOW>(S, O, n == 0, m, see, st, keys, scale, &p_half[i], &p_full[i]);
        if (!done) st = flash::softmax_tile_own<D>(S, O, n == 0, m, see, st, keys, &p_half[i], &p_full[i]);
      }
      if (ok && cnt) ok = sm100::mbar_poll_abort(&o_full[i], (uint32_t)(no++ & 1), &s_abort, p.err, 126);
      if (!ok) break;
      sm100::tc_fence_after();
      float M = st.sum != 0.f ? st.exponent() : -INFINITY, L = st.sum, f0 = 0.f, f1 = 0.f;
      const float back = LOW ? p.vunit : 1.f;  // of the values' operands
      if (L != 0.f) f0 = 1.f;
      if (g.turns) {
        if (i == 1) {
          s_ml[r] = make_float2(M, L);
          sm100::tc_fence_before();
          sm100::mbar_arrive(&merge);
        } else {
          ok = sm100::mbar_poll_abort(&merge, (uint32_t)(nm & 1), &s_abort, p.err, 127);
          if (!ok) break;
          sm100::tc_fence_after();
          const float2 b = s_ml[r];
          const float top = fmaxf(M, b.x);
          const float a0 = L != 0.f ? ex2_half(M - top) : 0.f, a1 = b.y != 0.f ? ex2_half(b.x - top) : 0.f;
          f0 = a0 * a0;
          f1 = a1 * a1;
          L = a0 * L * a0 + a1 * b.y * a1;
          M = top;
        }
      }
      if (i == 0 || !g.turns) {
        const bool whole = cur.whole();
        const int64_t slot = (int64_t)cur.slot() * SM::kRows + (row - g.row0);
        float *to = whole ? p.whole + at * D : p.many.part_o + slot * D;
        if (whole) {
          const float inv = L != 0.f ? 1.0f / L : 0.f;
          f0 *= inv;
          f1 *= inv;
        } else if (mine) {
          p.many.part_ml[slot] = make_float2(M, L);
        }
        f0 *= back;
        f1 *= back;
        const bool other = g.turns && __any_sync(0xffffffffu, f1 != 0.f);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t v[32], b[32];
          sm100::tmem_ld32(O + c, v);
          if (other) sm100::tmem_ld32(O + kTile + c, b);
          sm100::tmem_wait_ld();
          float *x = reinterpret_cast<float *>(v);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] = f0 != 0.f ? x[k] * f0 : 0.f;  // (an output that no product wrote may hold anything)
            if (other && f1 != 0.f) x[k] = fmaf(__uint_as_float(b[k]), f1, x[k]);
          }
          if (mine)
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4 *>(to + c + k) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
        }
      }
      if (g.turns) {
        // the second warpgroup's output is read before its next product
        sm100::tc_fence_before();
        if (i == 0)
          sm100::mbar_arrive(&merged);
        else
          ok = sm100::mbar_poll_abort(&merged, (uint32_t)(nm & 1), &s_abort, p.err, 128);
        ++nm;
      }
      ring.done();
    } while (ok && cur.next(p, p.many));
  }
  sm100::tc_fence_before();
  __syncthreads();
  if (s_abort) {
    // a role gave up: products in flight are waited for (bounded) before the
    // block's memory is released
    __shared__ uint64_t last;
    if (warp == kMmaWarp && lane == 0) {
      sm100::mbar_init(&last, 1);
      sm100::fence_barrier_init();
      sm100::mma_commit(&last);
      sm100::mbar_wait(&last, 0, p.err, 129);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) sm100::tmem_dealloc(tmem, 512);
}

template <int D, bool IP, bool LOW, int WK, int WV>
tq_status launch_tiles(const PagedParams &prm, cudaStream_t st) {
  using SM = TileSmem<D, IP, LOW>;
  auto kern = k_attend_paged_tiles<D, IP, LOW, WK, WV>;
  constexpr int smem = SM::kBytes;
  static_assert(smem <= 232448 - 8192, "shared memory");
  static_assert(SM::kRows == paged_tile_rows(D, IP, LOW), "the plan's blocks of rows");
  static std::atomic<uint64_t> ready{0};
  const tq_status rc = once_per_device(ready, [&] {
    cudaFuncAttributes fa;  // (a split of registers beyond what the block holds would wait for ever)
    return cudaFuncGetAttributes(&fa, kern) == cudaSuccess &&
           fa.numRegs * kTilesThreads >= 128 * (2 * kSoftmaxRegs + 2 * kExpandRegs + kMmaRegs) &&
           cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess;
  });
  if (rc != TQ_OK) return rc;
  kern<<<(unsigned)prm.many.grid, kTilesThreads, smem, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

template <int D, bool IP, int WK, int WV>
tq_status launch_tiles_low(const PagedParams &prm, cudaStream_t st) {
  return prm.bf16 ? launch_tiles<D, IP, false, WK, WV>(prm, st) : launch_tiles<D, IP, true, WK, WV>(prm, st);
}

template <int D, bool IP, int WK>
tq_status launch_tiles_wv(const PagedParams &prm, int wv, cudaStream_t st) {
  switch (wv) {
    case 2: return launch_tiles_low<D, IP, WK, 2>(prm, st);
    case 3: return launch_tiles_low<D, IP, WK, 3>(prm, st);
    case 4: return launch_tiles_low<D, IP, WK, 4>(prm, st);
  }
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace

template <int D, bool IP>
tq_status paged_tiles_launch(const PagedParams &prm, int wk, int wv, cudaStream_t st) {
  switch (wk) {
    case 1: return launch_tiles_wv<D, IP, 1>(prm, wv, st);
    case 2: return launch_tiles_wv<D, IP, 2>(prm, wv, st);
    case 3: return launch_tiles_wv<D, IP, 3>(prm, wv, st);
    case 4: return launch_tiles_wv<D, IP, 4>(prm, wv, st);
  }
  return TQ_ERR_UNSUPPORTED;
}

}  // namespace tq
