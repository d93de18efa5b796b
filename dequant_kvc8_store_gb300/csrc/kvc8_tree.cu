// kvc8_tree.cu -- attention of drafted tokens: draft t of sequence b, query head j of kv head h,
// attends over the sequence's context and over those of its drafts that the mask names.
//   out = sum_p w_p V'[p] / sum_p w_p,  w_p = exp(scale <q, K'[p]>),  K', V' = fp32(code) * scale
//
// A sequence's T drafts times G query heads are T G query rows against the same positions: 4 T G D
// flops for 2 D bytes of codes a position and head, so HBM would bound up to about 150 rows and the
// tensor cores more.  What bounds it in fact is a step's chain: its scores, their maximum, 64 exponentials a
// thread, the weighted values, with the dequantising warps' instructions between (8 heads, D = 128, whole calls):
//   256 sequences of up to 8192 positions, 16 rows, channel scales   674 us, 3.3 TB/s (a step 2500 cycles)
//   64 of 8192, 16 and 64 rows, dynamic scales                       272 and 303 us, 4.1 and 3.7 TB/s
//   2 of 131072, 256 rows, dynamic scales                            323 us, 845 TFLOP/s (2700 cycles, 70% of issue slots)
//   1 of 500, 16 rows (2 heads, D = 64)                              12.3 us: two launches, round trips
//
// tree_kernel: one persistent CTA per SM, a tile of 128 query rows, 128 positions a step.  S = Q
// K'^T and O += P V' are tcgen05.mma (M = 128, fp16, fp32 in tensor memory); Q lies in tensor memory,
// and P replaces S there: both are A operands.  Warps by role:
//   walk        1: what the CTA's next tiles are, and which drafts some row of them sees
//   fetch       2, for the keys and for the values: pages' codes by bulk copies into rings of two steps in shared
//               memory (2 x 131072: 351 us with one warp for both, 311 with two; three steps of keys were no faster)
//   dequantise  16, eight for the keys and eight for the values: codes to K' and V' as fp16, two stages of
//               each in shared memory
//   mma         one lane issues both products
//   softmax     8, two threads per query row, half of a step's positions each: S from tensor memory,
//               one-pass softmax (Milakov and Gimelshein, Online normalizer calculation for softmax,
//               2018), P back; any m cancels in the quotient, so the running maximum moves only when
//               the weights grow by more than 2^8, and O is seldom rescaled.  Warps without a row do
//               nothing
//   rows        4: the next tile's queries into tensor memory, the last one's O out of it
// With at most 64 rows idle softmax warps dequantise as well (given_up, below).
// S and Q are there twice: the scores of a step are made while the softmax works on the step before.  The roles'
// loops are kept short: together they must fit the SM's instruction cache (with 95 KB of code, of which each
// step ran through about 30, a step took 3100 cycles and the warps waited for instructions; it is 68 to 79 now).
//
// The units (sequence, kv head, row tile, step) are numbered in that order and cut into equal shares,
// a CTA's share in a row: ragged lengths need no plan, every CTA adds up the lengths itself.  What a
// CTA has of a tile that it does not hold whole it leaves as a partial (m, l, O), two at most: of the
// first tile of its share and of the last.  merge_kernel joins them.
//
// Every wait on an mbarrier has a limit, after which the kernel reports KVC8_DEV_TIMEOUT and leaves.  The barrier at
// which a row's two softmax warps meet needs none: a warp that leaves early comes to it once more.
#include "kvc8_tcgen05.cuh"

namespace kvc8 {
namespace {

constexpr int kStages = 2;     // steps of K', of V', of S; tiles of Q and O
constexpr int kMaskSlots = 4;  // steps whose valid counts are kept
constexpr int kTiles = 4;      // tiles that are known ahead
constexpr int kMaxCtas = 152;  // SMs of a GB300
constexpr int kMergeThreads = 256;
constexpr uint32_t kWaitTicks = 4000000000u;  // of the SM's clock: about two seconds

// ---- the work -----------------------------------------------------------------------

struct Raw {
    int32_t c0, c1, ctx;
};
struct Seq {
    int32_t b, token, drafts, ctx, len, steps, tiles;  // tiles: of query rows, per kv head
};

__device__ __forceinline__ Raw read_raw(const TreeArgs &p, int b) {
    Raw r{0, 0, 0};
    if (b < p.base.g.num_seqs) {
        r.c0 = p.cu_q_lens == nullptr ? b : ld_nc_s32(p.cu_q_lens + b);
        r.c1 = p.cu_q_lens == nullptr ? b + 1 : ld_nc_s32(p.cu_q_lens + b + 1);
        r.ctx = ld_nc_s32(p.base.context_lengths + b);
    }
    return r;
}
__device__ __forceinline__ bool bad_range(const TreeArgs &p, const Raw &r) {
    return r.c0 < 0 || r.c1 < r.c0 || r.c1 > p.num_tokens || r.c1 - r.c0 > p.max_drafts;
}
__device__ __forceinline__ Seq make_seq(const TreeArgs &p, int b, const Raw &r) {
    Seq s;
    s.b = b;
    s.token = r.c0;
    s.drafts = bad_range(p, r) ? 0 : r.c1 - r.c0;
    s.ctx = max(r.ctx, 0);
    const int64_t cap = (int64_t)p.base.g.max_blocks_per_seq * p.base.g.block_size;
    s.len = (int32_t)min((int64_t)s.ctx + s.drafts, cap);
    s.steps = (int32_t)(((uint32_t)s.len + kCols - 1) / kCols);
    s.tiles = (s.drafts * p.base.group + kRows - 1) / kRows;
    return s;
}
__device__ __forceinline__ uint32_t units_of(const TreeArgs &p, const Seq &s) {
    return s.drafts > 0 ? (uint32_t)s.tiles * (uint32_t)p.base.g.kv_heads * (uint32_t)s.steps : 0u;
}

// `units` cut over `n` CTAs: each takes `per` in a row, the first `more` one more.
struct Cut {
    uint32_t per, more;
    __device__ __forceinline__ Cut(uint32_t units, uint32_t n) : per(units / n), more(units - units / n * n) {}
    __device__ __forceinline__ uint32_t first_of(uint32_t cta) const { return cta * per + min(cta, more); }
    __device__ __forceinline__ uint32_t cta_of(uint32_t unit) const {
        const uint32_t edge = more * (per + 1);
        return unit < edge ? unit / (per + 1) : more + (unit - edge) / per;
    }
};

// A tile of a CTA's share, for the roles.
struct Tile {
    int32_t b, token, ctx, len;  // its sequence
    int32_t rows, row0, head;    // query rows of the sequence, the tile's first, the kv head
    int32_t step, count, steps;  // the share's first step of it and how many of all
};

// ---- the kernel ---------------------------------------------------------------------

template <int D>
struct Layout {
    static constexpr int kSoftmaxWarps = 8, kRowWarps = 4, kDequantWarps = 16;
    static constexpr int kRowWarp = kSoftmaxWarps, kDequantWarp = kRowWarp + kRowWarps;
    static constexpr int kMmaWarp = kDequantWarp + kDequantWarps, kFetchWarp = kMmaWarp + 1, kWalkWarp = kMmaWarp + 2;  // kFetchWarp + 2: the values'
    static constexpr int kThreads = 1024;
    // Registers per thread: a softmax thread holds 64 scores.
    static constexpr int kSoftmaxRegs = 104, kRowRegs = 64, kDequantRegs = 48, kMmaRegs = 48;
    static constexpr int kLaunchRegs = 64;
    static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + kRowWarps * kRowRegs + kDequantWarps * kDequantRegs +
                        4 * kMmaRegs) <= kThreads * kLaunchRegs,
                  "the warpgroups' registers are the block's");
    static constexpr int kTileBytes = kCols * D * 2;  // a K' or V' stage
    static constexpr int kRawBytes = kCols * D;       // a slot of the ring: a step's codes of keys or of values
    static constexpr int kRing = 32 * 1024 / kRawBytes;  // of keys, and as many of values
    static constexpr int kK = 0;
    static constexpr int kV = kStages * kTileBytes;
    static constexpr int kRaw = 2 * kStages * kTileBytes;
    // more than half of an SM's shared memory, so that a CTA has the SM's tensor memory to itself
    static constexpr int kBytes = kRaw + 2 * kRing * kRawBytes + 1024;
    static_assert(kBytes > 116 * 1024, "one CTA per SM");
    static constexpr int kO = kStages * kCols, kQ = kO + D;  // columns of tensor memory: S twice, O, Q twice
    static constexpr int kTmemCols = 512;
    static_assert(kQ + kStages * D / 2 <= kTmemCols, "tensor memory");
};
constexpr int kMaxRing = Layout<64>::kRing;

struct Barriers {
    // s_full: a step's scores, and its K' stage is free; v_free: its weighted values, and its V' stage
    uint64_t k_full[kStages], v_full[kStages], s_full[kStages], p_full[kStages], v_free[kStages];
    uint64_t q_full[kStages], q_free[kStages], o_full, o_free, ml_full, drained;
    // slots of the keys, then of the values: a warp that waits for a slot's next phase has waited for the last, so
    // that the parity tells them apart
    uint64_t raw_full[2 * kMaxRing], raw_free[2 * kMaxRing];
    uint64_t tile_full[kTiles], tile_free[kTiles];
    uint32_t tmem;
    int32_t stop;
    uint32_t sum[Layout<128>::kThreads / 32];
    int32_t start_b;
    uint32_t start_off;
    uint32_t units, first;  // of all CTAs, this one's
    int32_t total;          // units of this CTA
    Tile tile[kTiles];
    // mode 0, with masks: of each tile, the context (word 0, all ones) and the drafts that some row of it sees
    uint32_t seen[kTiles][1 + KVC8_MAX_DRAFTS / 32 + 1];
    float q_scale[kStages][kRows];  // log2 per unit of score, with the query's power of two
    float m[kRows], l[2][kRows];    // l: of each half of the positions
    float top[2][2][kRows];         // a step's largest score of each half, of two steps
    // of what is in the ring: each group of 16's positions that count, a bit each, the keys' (only with the keys) and
    // the values' scales (mode 2: one a group)
    uint32_t filled[2 * kMaxRing];  // how often
    uint4 raw_valid[2 * kMaxRing];
    alignas(16) float raw_ks[kMaxRing][kCols];
    alignas(16) float raw_vs[2 * kMaxRing][kCols];
    uint4 valid[kMaskSlots];  // a step's positions that count, a bit each
    // modes 0 and 2: what was taken out of each group of 16's scales, as powers of two:
    // the keys' 2^e, the values' e
    alignas(16) float k_pow[kMaskSlots][kCols / 16];
    alignas(16) float v_exp[kMaskSlots][kCols / 16];
};

template <int MODE, int D, int QUADS>
struct Tree {
    using L = Layout<D>;
    static constexpr int kRpw = 16;  // positions of a dequantising warp: one group
    using T = CodeTile<MODE, D, kRpw>;
    static_assert(T::kGroups == 1, "a warp's positions lie in one block");

    const TreeArgs &p;
    Barriers &bar;
    const uint32_t base, tmem;  // shared memory, 1 KB aligned
    const int total;            // units of this CTA
    const int lane, warp;

    // (Read again here, by each role for itself, than kept in registers from the kernel's start.)
    __device__ __forceinline__ Tree(const TreeArgs &args, Barriers &b, uint8_t *dyn)
        : p(args), bar(b), base((smem_u32(dyn) + 1023u) & ~1023u), tmem(b.tmem), total(b.total), lane(threadIdx.x & 31),
          warp(threadIdx.x >> 5) {}

    // A whole warp waits and stays converged.  false: the limit ran out here or elsewhere in the CTA.
    __device__ __forceinline__ bool wait(uint64_t &b, uint32_t parity) const {
        const uint32_t at = smem_u32(&b);
        bool ok = mbar_try(at, parity);
        if (!ok) {
            const uint32_t t0 = clock();
            do {
                ok = mbar_try(at, parity);
            } while (!ok && *static_cast<volatile int32_t *>(&bar.stop) == 0 && (uint32_t)clock() - t0 < kWaitTicks);
            if (!ok) *static_cast<volatile int32_t *>(&bar.stop) = 1;
        }
        return __all_sync(0xFFFFFFFFu, ok);
    }
    __device__ __forceinline__ void arrive(uint64_t &b) const {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&b));
    }

    // ---- walk (a warp) ------------------------------------------------------------
    // Which drafts some row of the tile sees.
    __device__ __forceinline__ void find_seen(const Tile &x, uint32_t *seen) const {
        const int first = x.row0 / p.base.group, last = (min(x.rows, x.row0 + kRows) - 1) / p.base.group;
        const uint32_t *mask = reinterpret_cast<const uint32_t *>(p.mask + (int64_t)(x.token + first) * p.mask_words);
#pragma unroll 1
        for (int w = 0; 32 * p.base.group * w < x.rows; ++w) {
            uint32_t any = 0u;
#pragma unroll 1
            for (int t = lane; t <= last - first; t += 32) any |= __ldg(mask + (int64_t)t * 2 * p.mask_words + w);
            any = __reduce_or_sync(0xFFFFFFFFu, any);
            if (lane == 0) seen[1 + w] = any;
        }
        if (lane == 0) seen[0] = 0xFFFFFFFFu;
    }
    __device__ void walk() const {
        int b = bar.start_b;
        Seq s = make_seq(p, b, read_raw(p, b));
        Raw ahead = read_raw(p, b + 1);  // the next sequence's lengths are on their way
        int tile = (int)(bar.start_off / (uint32_t)s.steps);  // kv head * s.tiles + row tile
        int step = (int)(bar.start_off - (uint32_t)tile * (uint32_t)s.steps);
        int left = total;
        for (uint32_t seg = 0; left > 0; ++seg) {
            Tile x;
            x.b = s.b;
            x.token = s.token;
            x.ctx = s.ctx;
            x.len = s.len;
            x.rows = s.drafts * p.base.group;
            x.head = tile / s.tiles;
            x.row0 = (tile - x.head * s.tiles) * kRows;
            x.step = step;
            x.count = min(left, s.steps - step);
            x.steps = s.steps;
            if (!wait(bar.tile_free[seg % kTiles], ((seg / kTiles) & 1u) ^ 1u)) return;
            if (lane == 0) bar.tile[seg % kTiles] = x;
            if (MODE == 0 && p.mask != nullptr) find_seen(x, bar.seen[seg % kTiles]);
            arrive(bar.tile_full[seg % kTiles]);
            if (seg == 0 && lane == 0) {
                TreeShare r;
                r.units = bar.units;
                r.first = bar.first - (uint32_t)step;
                r.steps = x.steps;
                r.token = x.token;
                r.rows = x.rows;
                r.row = x.row0;
                r.head = x.head;
                r.pad = 0;
                p.shares[blockIdx.x] = r;
            }
            left -= x.count;
            step = 0;
            if (++tile == s.tiles * p.base.g.kv_heads && left > 0) {
                tile = 0;
                do {
                    s = make_seq(p, s.b + 1, ahead);
                    ahead = read_raw(p, s.b + 1);
                } while (s.drafts == 0 && s.b + 1 < p.base.g.num_seqs);
            }
        }
    }
    // The share's tile number `seg`, and that a warp needs it no more.
    __device__ __forceinline__ bool enter(uint32_t seg) const { return wait(bar.tile_full[seg % kTiles], (seg / kTiles) & 1u); }
    __device__ __forceinline__ void leave(uint32_t seg) const { arrive(bar.tile_free[seg % kTiles]); }
    __device__ __forceinline__ const Tile &tile(uint32_t seg) const { return bar.tile[seg % kTiles]; }

    // ---- fetch (a warp) ----------------------------------------------------------
    // Lanes 0-7 have a group of 16 positions each: a step's groups may lie in different blocks.  In the loop's
    // turn n, step n is copied, step n + 1 is placed and its scales asked for, and the block ids of step n + 2 are.
    __device__ __forceinline__ void copy(uint32_t dst, const int8_t *src, uint64_t &full, uint32_t bytes) const {
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                     "l"(src), "r"(bytes), "r"(smem_u32(&full))
                     : "memory");
    }
    __device__ void fetch() const {
        const AttnArgs &a = p.base;
        const int grp = lane & 7, bs = a.g.block_size, values = (warp - L::kFetchWarp) / 2;
        const int8_t *cache = values == 0 ? a.k_cache : a.v_cache;
        uint32_t seg = 0;
        int count = 0;                // steps of the tile not asked for yet
        int left = 0, at = 0, head = 0;  // of the step asked for: positions left, slot and entry of the table
        int drafts = INT32_MIN;          // mode 0, with masks: positions of its tile behind the context
        const int32_t *entry = nullptr;
        int32_t blk = 0;
        int64_t row = 0;  // of the step placed: cache row of the group's first position
        uint32_t valid = 0u;  // the positions that count, a bit each
        float4 ks = make_float4(0.0f, 0.0f, 0.0f, 0.0f), vs = ks;  // mode 0: of positions 4 lane .. 4 lane + 3; mode 2: .x, of the group
        int slot = 0;
        uint32_t round = 0;
        bool good = true;
#pragma unroll 1
        for (int n = -2; n < total && good; ++n) {
            if (n >= 0) {
                const int to = values * L::kRing + slot;
                good = wait(bar.raw_free[to], round ^ 1u);
                if (!good) break;
                if (lane < 8) reinterpret_cast<uint16_t *>(&bar.raw_valid[to])[grp] = (uint16_t)valid;
                if (MODE == 0) {
                    if (values == 0) reinterpret_cast<float4 *>(bar.raw_ks[slot])[lane] = ks;
                    reinterpret_cast<float4 *>(bar.raw_vs[to])[lane] = vs;
                } else if (MODE == 2 && lane < 8) {
                    if (values == 0) bar.raw_ks[slot][grp] = ks.x;
                    bar.raw_vs[to][grp] = vs.x;
                }
                const uint32_t groups = __popc(__ballot_sync(0xFFFFFFFFu, lane < 8 && valid != 0u));
                __syncwarp();
                if (lane == 0) {
                    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(&bar.raw_full[to])),
                                 "r"(groups * 16u * D)
                                 : "memory");
                    ++bar.filled[to];
                }
                __syncwarp();
                const bool one = bs % 128 == 0 && groups == 8;  // one block holds the step
                if (one ? lane == 0 : lane < 8 && valid != 0u)
                    copy(base + L::kRaw + to * L::kRawBytes + grp * 16 * D, cache + row * D, bar.raw_full[to], one ? 128 * D : 16 * D);
                if (++slot == L::kRing) {
                    slot = 0;
                    round ^= 1u;
                }
            }
            if (n >= -1 && n + 1 < total) {
                const bool in = blk >= 0 && blk < a.g.num_blocks;
                if (!in && lane < 8 && values == 0) report(a.dev_error, KVC8_DEV_BAD_BLOCK_ID);
                valid = in ? (1u << max(0, min(16, left))) - 1u : 0u;
                if (MODE == 0) {
                    // The scales of drafts that no row of the tile sees, which may be anything, take no part in the
                    // power that 16 scales have in common.  (The tile's place is not taken by another before its rows
                    // are stored, long after this.  64 x 8192, 16 query rows: 268 -> 272 us, with the masks gone through
                    // here instead of by the walk warp 321.)
                    if (drafts > left - 16) {
                        const int bit = min(drafts - left, KVC8_MAX_DRAFTS - 1) + 32;  // of the group's first position
                        const uint32_t *seen = bar.seen[(seg - 1) % kTiles] + bit / 32;
                        valid &= __funnelshift_r(seen[0], seen[1], (uint32_t)bit & 31u);
                    }
                }
                const int64_t page = (int64_t)(in ? blk : 0) * a.g.kv_heads + head;
                row = page * bs + at;
                if (MODE == 0) {
                    const int64_t r = __shfl_sync(0xFFFFFFFFu, row, lane / 4) + lane % 4 * 4;
                    if (__shfl_sync(0xFFFFFFFFu, valid, lane / 4) != 0u) {
                        if (values == 0) ks = ld_ahead_f32x4(a.k_scale + r);
                        vs = ld_ahead_f32x4(a.v_scale + r);
                    }
                } else if (MODE == 2 && valid != 0u) {
                    if (values == 0) ks.x = ld_ahead_f32(a.k_scale + page);
                    vs.x = ld_ahead_f32(a.v_scale + page);
                }
            }
            if (good && n + 2 < total) {
                if (count == 0) {
                    good = enter(seg);
                    if (!good) break;
                    const Tile &x = tile(seg);
                    const int pos = x.step * kCols + grp * 16;
                    left = x.len - pos;
                    if (MODE == 0) drafts = p.mask != nullptr ? x.len - x.ctx : INT32_MIN;
                    head = x.head;
                    at = pos % bs;
                    entry = a.block_table + (int64_t)x.b * a.g.max_blocks_per_seq + pos / bs;
                    count = x.count;
                    leave(seg++);
                } else {
                    left -= kCols;
                    at += kCols % bs;
                    entry += kCols / bs;
                    if (at >= bs) {
                        at -= bs;
                        ++entry;
                    }
                }
                --count;
                blk = left > 0 ? ld_ahead_s32(entry) : 0;
            }
        }
        // nothing is in flight when the CTA ends, not after a wait that ran out either
        __syncwarp();
#pragma unroll 1
        for (int i = values * L::kRing; i < (values + 1) * L::kRing; ++i) {
            const uint32_t t0 = clock();
            while (bar.filled[i] != 0u && !mbar_try(smem_u32(&bar.raw_full[i]), (bar.filled[i] - 1u) & 1u))
                if ((uint32_t)clock() - t0 > kWaitTicks) break;
        }
    }

    // ---- dequantise (a warp has a group of 16 positions) ------------------------------------------------
    // A tile's rows lie in QUADS quarters of tensor memory's lanes, and the softmax warps of a quarter are those with
    // its number as their remainder by 4, which also share a scheduler of the SM.  Where quarters are empty, their idle
    // softmax warps take places of dequantising warps from the schedulers that have softmax to do: three of one scheduler's
    // four (1 quarter), two of each one's four (2 quarters).  64 x 8192 positions, D = 128: 8 rows to a head,
    // dynamic and channel scales, 306 -> 267 and 283 -> 254 us.  Fewer loads unrolled are quicker with two copies
    // of this loop in the instruction cache (285 and 260 us with four), and slower with one (2 x 131072, 256 rows: 320 and 312).
    __device__ __forceinline__ static bool given_up(int place) {
        return QUADS == 1 ? place > 0 && place % 4 == 0 : QUADS == 2 && place % 4 < 2 && place % 8 >= 4;
    }
    // The place that softmax warp w takes, or -1.
    __device__ __forceinline__ static int taken(int w) {
        return QUADS == 1 ? (w < 4 ? 4 * w : -1) : QUADS == 2 ? 4 + (w & 1) + 8 * (w >> 2) : -1;
    }
    __device__ void dequantise(int place) const {
        const int dw = place % 8, values = place / 8;
        const uint32_t src = base + L::kRaw + (uint32_t)((dw * 16 + T::row_in(lane)) * D + T::block_in(lane) * 64 + lane % 4 * 16);
        int slot = values * L::kRing;
        uint32_t round = 0;
#pragma unroll 1
        for (int n = 0; n < total; ++n) {
            const int st = n % kStages;
            if (!wait(bar.raw_full[slot], round)) return;
            const uint32_t valid = reinterpret_cast<const uint16_t *>(&bar.raw_valid[slot])[dw];
            uint32_t scale = 0u;
            int ek = 0, ev = 0;
            if (MODE != 1) {
                float sk = 0.0f, sv = 0.0f;  // positions behind the end may have any scale
                if (MODE == 0 ? (valid >> lane & 1u) != 0u : valid != 0u) {
                    if (values == 0) sk = bar.raw_ks[slot][MODE == 0 ? dw * 16 + lane : dw];
                    sv = bar.raw_vs[slot][MODE == 0 ? dw * 16 + lane : dw];
                }
                // A scale that is no number must not reach the rows that do not see its position,
                // nor the other scales' power: the value counts as zero, and the score as no number.
                // The value scales' power is found twice, by the keys' warps, who hand it to the softmax, and by
                // the values', who divide by it and see no key scale: so it goes by the value scales alone.
                const bool odd_v = (__float_as_uint(sv) & 0x7F800000u) == 0x7F800000u;
                sv = odd_v ? 0.0f : sv;
                scale = T::normal_scale(sv, T::group_top(sv, lane), kLeastValuePower, ev);
                if (values == 0) {
                    const bool odd = odd_v || (__float_as_uint(sk) & 0x7F800000u) == 0x7F800000u;
                    sk = odd ? 0.0f : sk;
                    scale = T::normal_scale(sk, T::group_top(sk, lane), -100, ek);
                    if (odd) scale = 0x7FFF7FFFu;
                }
            }
            if (!wait(values == 0 ? bar.s_full[st] : bar.v_free[st], ((uint32_t)(n / kStages) & 1u) ^ 1u)) return;
            if (values == 0 && lane == 0) {  // (the step that had this place, four before, is through)
                if (MODE != 1) {
                    bar.k_pow[n % kMaskSlots][dw] = __uint_as_float((uint32_t)(127 + ek) << 23);
                    bar.v_exp[n % kMaskSlots][dw] = (float)ev;
                }
                reinterpret_cast<uint16_t *>(&bar.valid[n % kMaskSlots])[dw] = (uint16_t)valid;
            }
            T::template store_each<QUADS == 4 ? 4 : 2>(
                [&](int k) {
                    uint4 c;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(c.x), "=r"(c.y), "=r"(c.z), "=r"(c.w)
                                 : "r"(src + slot * L::kRawBytes + k * T::kRpl * D)
                                 : "memory");
                    return c;
                },
                scale, base + (values == 0 ? L::kK : L::kV) + st * L::kTileBytes, dw, lane);
            fence_async();
            arrive(values == 0 ? bar.k_full[st] : bar.v_full[st]);
            if (lane == 0) mbar_arrive(smem_u32(&bar.raw_free[slot]));
            if (++slot == (values + 1) * L::kRing) {
                slot = values * L::kRing;
                round ^= 1u;
            }
        }
    }

    // ---- products (a warp, one lane issuing) --------------------------------------------------
    __device__ __forceinline__ void qk(int q, int st, uint32_t tm, uint32_t leader) const {
        const uint64_t kd = operand_desc(base + L::kK, 16) + (uint64_t)(st * (L::kTileBytes >> 4));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint64_t at = (uint64_t)(((i / 4) * (kCols * 128) + (i % 4) * 32) >> 4);
            tc_mma_ts(tm + st * kCols, tm + L::kQ + q * (D / 2) + 8 * i, kd + at, instr_desc(kCols, false), i > 0, leader);
        }
    }
    __device__ __forceinline__ void pv(int st, uint32_t tm, bool acc, uint32_t leader) const {
        const uint64_t v = operand_desc(base + L::kV, kCols * 128) + (uint64_t)(st * (L::kTileBytes >> 4));
#pragma unroll
        for (int i = 0; i < kCols / 16; ++i)
            tc_mma_ts(tm + L::kO, tm + st * kCols + 8 * i, v + (uint64_t)(i * (2048 >> 4)), instr_desc(D, true),
                      acc || i > 0, leader);
    }
    __device__ __forceinline__ bool ready(uint64_t &b, uint32_t parity) const {
        return __all_sync(0xFFFFFFFFu, mbar_test(smem_u32(&b), parity));
    }
    // What steers the loop comes from lane 0, so that the compiler keeps it, and with it stages,
    // addresses and descriptors, in uniform registers.
    __device__ __forceinline__ static int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

    // The scores of a step are issued before the weighted values of the step before, so that the softmax has
    // them early, unless they must wait and the values need not: a new tile's queries may be late.
    __device__ bool products_loop(uint32_t leader) const {
        const uint32_t tm = (uint32_t)uniform((int)tmem);
        const int units = uniform(total);
        int s = 0, v = 0;             // steps whose scores and whose weighted values are issued
        int left = 0;                 // steps of the tile whose scores are still to come
        uint32_t q_seg = 0, seg = 0;  // the next tile of the scores, the tile of the weighted values
        bool first = true;            // step v is its tile's first
        uint32_t lasts = 0;           // bit n & 1: step n is its tile's last
#pragma unroll 1
        while (v < units) {
            bool scores = s < units && s < v + 2;
            if (scores && s > v) {  // step v's values could go first: whichever can
                const uint32_t t0 = clock();
                while (true) {
                    scores = ready(bar.k_full[s & 1], (uint32_t)(s >> 1) & 1u) &&
                             (left > 0 || ready(bar.q_full[q_seg & 1u], (q_seg >> 1) & 1u));
                    if (scores || ready(bar.p_full[v & 1], (uint32_t)(v >> 1) & 1u)) break;
                    const bool over = *static_cast<volatile int32_t *>(&bar.stop) != 0 || (uint32_t)clock() - t0 > kWaitTicks;
                    if (__any_sync(0xFFFFFFFFu, over)) {  // all lanes go together, whatever each has read
                        *static_cast<volatile int32_t *>(&bar.stop) = 1;
                        return false;
                    }
                }
            }
            if (scores) {
                const int st = s & 1;
                if (left == 0) {
                    if (!enter(q_seg)) return false;
                    left = uniform(tile(q_seg).count);
                    leave(q_seg);
                    if (!wait(bar.q_full[q_seg & 1u], (q_seg >> 1) & 1u)) return false;
                    ++q_seg;
                }
                if (!wait(bar.k_full[st], (uint32_t)(s >> 1) & 1u)) return false;
                tc_fence_after();
                qk((int)((q_seg - 1) & 1u), st, tm, leader);
                tc_commit(smem_u32(&bar.s_full[st]), leader);
                lasts &= ~(1u << st);
                if (--left == 0) {
                    tc_commit(smem_u32(&bar.q_free[(q_seg - 1) & 1u]), leader);
                    lasts |= 1u << st;
                }
                ++s;
            } else {
                const int st = v & 1;
                if (first && !wait(bar.o_free, (seg & 1u) ^ 1u)) return false;
                if (!wait(bar.v_full[st], (uint32_t)(v >> 1) & 1u)) return false;
                if (!wait(bar.p_full[st], (uint32_t)(v >> 1) & 1u)) return false;
                tc_fence_after();
                pv(st, tm, !first, leader);
                tc_commit(smem_u32(&bar.v_free[st]), leader);
                first = (lasts >> st & 1u) != 0;
                if (first) {
                    tc_commit(smem_u32(&bar.o_full), leader);
                    ++seg;
                }
                ++v;
            }
        }
        return true;
    }
    __device__ void products() const {
        const uint32_t leader = elect_lane();
        products_loop(leader);
        // what was issued is done before the tensor memory is freed
        tc_commit(smem_u32(&bar.drained), leader);
        const uint32_t t0 = clock();
        while (!mbar_try(smem_u32(&bar.drained), 0))
            if ((uint32_t)clock() - t0 > kWaitTicks) break;
    }

    // ---- rows in, rows out (a thread per row of the tile) ------------------------------------------
    // Query rows of a tile, in mode 1 times the channels' key scales: fp16 after a power of two that
    // brings a row's largest value to [1, 2) and goes into its factor.  Eleven bits hold a bf16 value
    // whole (mode 1: round the product eight times finer than bf16); below 2^-14 of the largest they
    // thin out to 2^-25 of it.
    __device__ __forceinline__ void load_rows(const Tile &w, int rw, int buf) const {
        const AttnArgs &a = p.base;
        const int h = w.head, r0 = w.row0 + rw * 32, rows = w.rows;
        if (r0 < rows) {  // uniform in the warp: some row is a query's
            const int r = r0 + lane, t = r / a.group, j = r - t * a.group;
            const uint16_t *q = a.q + (int64_t)(w.token + t) * a.q_seq_stride + (int64_t)(h * a.group + j) * a.q_head_stride;
            const float *ks = a.k_scale + (MODE == 1 ? (int64_t)h * D : 0);
            // chunk i of the row, eight channels
            auto read = [&](int i) { return r < rows ? __ldg(reinterpret_cast<const uint4 *>(q) + i) : make_uint4(0u, 0u, 0u, 0u); };
            auto value = [&](uint32_t wd, int d) {
                float2 y = make_float2(__uint_as_float(wd << 16), __uint_as_float(wd & 0xFFFF0000u));
                if (MODE == 1) {
                    const float2 s = __ldg(reinterpret_cast<const float2 *>(ks + d));
                    y = make_float2(y.x * s.x, y.y * s.y);
                }
                return y;
            };
            // eight chunks in flight: a row does not fit the registers, and is read twice
            float top = 0.0f;
#pragma unroll 1
            for (int i = 0; i < D / 8; i += 8) {
                uint4 x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = read(i + k);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t wd[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 y = value(wd[e], 8 * (i + k) + 2 * e);
                        top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
                    }
                }
            }
            const int ex = power_of(top);
            // (the sign of the softmax's scale goes to the query)
            const float turn = __uint_as_float(((uint32_t)(127 - ex) << 23) | (a.scale_log2 < 0.0f ? 0x80000000u : 0u));
            const uint32_t q_at = tmem + ((uint32_t)(rw * 32) << 16) + L::kQ + buf * (D / 2);
#pragma unroll 1
            for (int i = 0; i < D / 8; i += 8) {
                uint32_t o[2][16];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4 x = read(i + k);
                    uint32_t *to = o[k / 4] + 4 * (k % 4);
                    to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 y = value(o[k][e], 8 * i + 32 * k + 2 * e);
                        o[k][e] = pack_fp16(y.x * turn, y.y * turn);
                    }
                    tc_st16(q_at + 4 * i + 16 * k, o[k]);
                }
            }
            bar.q_scale[buf][rw * 32 + lane] = fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 + ex) << 23);
            tc_wait_st();
        }
        tc_fence_before();
        arrive(bar.q_full[buf]);
    }

    // A tile's O: to the output where the CTA has the whole tile, else a partial.
    __device__ __forceinline__ void store_rows(const Tile &w, int rw, bool whole, uint32_t seg) const {
        const AttnArgs &a = p.base;
        const int h = w.head, row = rw * 32 + lane, r0 = w.row0 + rw * 32, rows = w.rows;
        const uint32_t o_at = tmem + ((uint32_t)(rw * 32) << 16) + L::kO;
        const float *vs = a.v_scale + (MODE == 1 ? (int64_t)h * D : 0);
        if (r0 < rows) {
            const float m = bar.m[row], l = bar.l[0][row] + bar.l[1][row];
            const float inv = !whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
            const int r = r0 + lane, t = r / a.group, j = r - t * a.group;
            uint16_t *dst = a.out + (int64_t)(w.token + t) * a.out_seq_stride + (int64_t)(h * a.group + j) * a.out_head_stride;
            const int64_t slot = (int64_t)(2 * blockIdx.x + (seg > 0 ? 1 : 0)) * kRows + row;
            float *po = a.part_o + (slot - lane) * D + lane * 8;  // 32 rows' eighths in turn
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                float o[32];
                tc_ld32(o, o_at + c);
                tc_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 s = MODE == 1 ? __ldg(reinterpret_cast<const float4 *>(vs + c + i)) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                    o[i] *= s.x * inv, o[i + 1] *= s.y * inv, o[i + 2] *= s.z * inv, o[i + 3] *= s.w * inv;
                }
                if (MODE == 1 && l == 0.0f) {  // no position: zeros, also where a channel's scale is infinite or no number
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.0f;
                }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4 *>(po + (c + i) / 8 * 256 + i % 8) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else if (r < rows) {
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
                    if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            reinterpret_cast<uint4 *>(dst + c)[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                    } else {  // the output may lie on any element
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            dst[c + 2 * i] = (uint16_t)(y[i] & 0xFFFFu);
                            dst[c + 2 * i + 1] = (uint16_t)(y[i] >> 16);
                        }
                    }
                }
            }
            if (!whole) {
                a.part_m[slot] = m;
                a.part_l[slot] = l;
            }
        }
        tc_fence_before();
        arrive(bar.o_free);
    }

    // Turn seg: the queries of tile seg + 1, then O of tile seg.
    __device__ void rows() const {
        const int rw = warp - L::kRowWarp;
        int in_left = total, out_left = total;
#pragma unroll 1
        for (uint32_t in = 0; out_left > 0; ++in) {
            if (in_left > 0) {
                const int buf = (int)(in & 1u);
                if (!enter(in) || !wait(bar.q_free[buf], ((in >> 1) & 1u) ^ 1u)) return;
                tc_fence_after();
                load_rows(tile(in), rw, buf);
                in_left -= tile(in).count;
            }
            if (in == 0) continue;
            const uint32_t seg = in - 1;
            const Tile &x = tile(seg);
            if (!wait(bar.ml_full, seg & 1u) || !wait(bar.o_full, seg & 1u)) return;
            tc_fence_after();
            store_rows(x, rw, x.count == x.steps, seg);
            out_left -= x.count;
            leave(seg);
        }
    }

    // The two softmax warps of 32 rows meet, by a hardware barrier: no limit, but none is needed.  A warp leaves
    // early only once `stop` is set, and then comes to the barrier one last time (leave_pair), whatever the other
    // one has read: if that one still waits here or comes later, it goes on, finds `stop` set and leaves too.
    // What a warp's lanes have read they settle among themselves, so that they go the same way.
    __device__ __forceinline__ bool meet(int quad) const {
        asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
        return __all_sync(0xFFFFFFFFu, *static_cast<volatile int32_t *>(&bar.stop) == 0);
    }
    __device__ __forceinline__ void leave_pair(int quad) const { asm volatile("bar.arrive %0, 64;" ::"r"(1 + quad) : "memory"); }

    // ---- softmax (two threads per query row, 64 of a step's positions each) -----------------------------------
    // 32 bits of a row's mask; drafts before the first are the context.
    __device__ __forceinline__ uint32_t mask_word(const uint32_t *mask, int word) const {
        if (word < 0) return 0xFFFFFFFFu;
        return word < 2 * p.mask_words ? __ldg(mask + word) : 0u;
    }

    // What of 64 positions a row sees; d0: the draft at the first, if not negative.
    __device__ __forceinline__ void visible(uint32_t (&sees)[2], int d0, int t, int token) const {
        if (p.mask == nullptr) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int upto = t - d0 + 1 - 32 * q;  // positions from the word's first on that are seen
                sees[q] = upto >= 32 ? 0xFFFFFFFFu : upto <= 0 ? 0u : (1u << upto) - 1u;
            }
        } else {
            const uint32_t *mask = reinterpret_cast<const uint32_t *>(p.mask + (int64_t)(token + t) * p.mask_words);
            uint32_t lo = mask_word(mask, d0 >> 5);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t hi = mask_word(mask, (d0 >> 5) + q + 1);
                sees[q] = __funnelshift_r(lo, hi, (uint32_t)d0 & 31u);
                lo = hi;
            }
        }
    }

    __device__ void softmax() const {
        if (!softmax_loop()) leave_pair(warp & 3);
    }
    // false: a wait ran out
    __device__ __forceinline__ bool softmax_loop() const {
        const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        int n = 0;
        uint32_t met = 0;  // steps in which the row's two warps met
#pragma unroll 1
        for (uint32_t seg = 0; n < total; ++seg) {
            if (!enter(seg)) return false;
            const Tile &x = tile(seg);
            const int end = n + x.count, buf = (int)(seg & 1u), token = x.token;
            const bool busy = x.row0 + quad * 32 < x.rows;  // uniform in the warp: some row is a query's
            const int t = min(x.row0 + row, x.rows - 1) / p.base.group;
            int d0 = x.step * kCols + half * 64 - x.ctx;  // the draft at the first position, if not negative
            leave(seg);
            if (!wait(bar.q_full[buf], (seg >> 1) & 1u)) return false;
            const float scale = bar.q_scale[buf][row];
            arrive(bar.q_free[buf]);
            float m = -INFINITY, l = 0.0f;
            bool have_o = false;
#pragma unroll 1
            for (; n < end; ++n, d0 += kCols) {
                const int st = n & 1;
                uint32_t sees[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
                if (d0 + 64 > 0 && busy) visible(sees, d0, t, token);  // some position is a draft's
                if (!wait(bar.s_full[st], (uint32_t)(n >> 1) & 1u)) return false;
                tc_fence_after();
                if (busy) {
                    if (!step(tmem + lanes + st * kCols, tmem + lanes + L::kO, quad, half, scale, have_o, n, met & 1u, sees, m, l))
                        return false;
                    ++met;
                }
                have_o = true;
                tc_fence_before();
                arrive(bar.p_full[st]);
            }
            if (!wait(bar.o_free, (seg & 1u) ^ 1u)) return false;
            if (half == 0) bar.m[row] = m;
            bar.l[half][row] = l;
            arrive(bar.ml_full);
        }
        return true;
    }

    // One step of a row's half: S -> P, the running maximum m and the half's sum l.  A group's weights are
    // 2^(score + e - m), e the exponent taken out of its value scales, so that the product
    // with the tile's values is the weight times the value; m bounds score + e, lazily, and is the
    // same in both halves.  fp16 holds such weights (at most 2^15) eight times finer than bf16, and what
    // falls below 2^-21 of the largest to 2^-32 of it.
    // false: a wait ran out.
    __device__ __forceinline__ bool step(uint32_t s_at, uint32_t o_at, int quad, int half, float scale, bool have_o, int n,
                                         uint32_t met, const uint32_t (&sees)[2], float &m, float &l) const {
        const int slot = n % kMaskSlots;
        const uint2 in = reinterpret_cast<const uint2 *>(&bar.valid[slot])[half];
        const uint32_t keep[2] = {in.x & sees[0], in.y & sees[1]};
        float s[2][32];
#pragma unroll
        for (int q = 0; q < 2; ++q) tc_ld32(s[q], s_at + half * 64 + 32 * q);
#pragma unroll
        for (int q = 0; q < 2; ++q) tc_wait_ld(s[q]);
        if (__any_sync(0xFFFFFFFFu, (keep[0] & keep[1]) != 0xFFFFFFFFu)) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if ((keep[q] >> i & 1u) == 0u) s[q][i] = -INFINITY;
            }
        }
        // Each group of 16's factor of the scores and shift.  The factor is never 0, which times the -inf of a position left
        // out would be no number; 2^-126 instead does not show.
        float f[4], g[4];
        if (MODE == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = fmaxf(scale, 0x1p-126f), g[i] = 0.0f;
        } else {
            const float4 k = reinterpret_cast<const float4 *>(bar.k_pow[slot])[half], e = reinterpret_cast<const float4 *>(bar.v_exp[slot])[half];
            const float ks[4] = {k.x, k.y, k.z, k.w}, es[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = fmaxf(scale * ks[i], 0x1p-126f), g[i] = es[i];
        }
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaf(top16(s[i / 2], i % 2 * 16), f[i], g[i]));
        // The halves' larger one; after it both have read S, over which P is written.
        const int row = quad * 32 + lane;
        bar.top[met][half][row] = mx;
        tc_fence_before();
        if (!meet(quad)) return false;
        tc_fence_after();
        mx = fmaxf(mx, bar.top[met][half ^ 1][row]);
        const bool moves = mx > m + (kLift + kLazy) || (m == -INFINITY && mx > m);
        if (__any_sync(0xFFFFFFFFu, moves)) {
            const float c = moves ? ex2(m - (mx - kLift)) : 1.0f;  // 0 where there was nothing yet
            if (moves) m = mx - kLift;
            l *= c;
            if (have_o) {  // once the step before is in it; half of the channels each
                if (!wait(bar.v_free[(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1u)) return false;
                tc_fence_after();
#pragma unroll 1
                for (int d = 0; d < D / 2; d += 16) {
                    float o[16];
                    tc_ld16(o, o_at + half * (D / 2) + d);
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(o[i] * c);
                    tc_st16(o_at + half * (D / 2) + d, y);
                }
            }
        }
        const float neg = m == -INFINITY ? 0.0f : -m;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float2 sum[2];
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                const float fi = f[2 * q + i / 16], gi = g[2 * q + i / 16] + neg;
                float2 y = __ffma2_rn(make_float2(s[q][i], s[q][i + 1]), make_float2(fi, fi), make_float2(gi, gi));
                y = make_float2(ex2(y.x), ex2(y.y));
                sum[i / 16] = i % 16 == 0 ? y : __fadd2_rn(sum[i / 16], y);
                o[i / 2] = pack_fp16(y.x, y.y);
            }
            tc_st16(s_at + half * 32 + 16 * q, o);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float part = sum[i].x + sum[i].y;
                // (times 2^-e)
                l = MODE == 1 ? l + part : fmaf(part, __uint_as_float((uint32_t)(127 - (int)g[2 * q + i]) << 23), l);
            }
        }
        tc_wait_st();
        return true;
    }
};

template <int MODE, int D, int QUADS>
__global__ void __launch_bounds__(Layout<D>::kThreads, 1) tree_kernel(const TreeArgs p) {
    using L = Layout<D>;
    using Roles = Tree<MODE, D, QUADS>;
    constexpr int kSoftmaxWarps = 2 * QUADS;  // that have a row
    extern __shared__ uint8_t dyn[];
    __shared__ Barriers bar;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int B = p.base.g.num_seqs;
    pdl_launch_dependents();
    // This thread's sequences: the units of all, and where they are few, of its one.
    uint32_t mine = 0, one = 0;
    for (int b = threadIdx.x; b < B; b += L::kThreads) {
        const Raw raw = read_raw(p, b);
        const Seq s = make_seq(p, b, raw);
        one = units_of(p, s);
        mine += one;
        if (blockIdx.x == 0) {
            if (bad_range(p, raw) || raw.ctx < 0) report(p.base.dev_error, KVC8_DEV_BAD_LENGTH);
            if ((int64_t)s.ctx + s.drafts > s.len) report(p.base.dev_error, KVC8_DEV_POS_BEYOND_TABLE);
        }
    }
    if (warp == L::kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < kStages; ++i) {
                mbar_init(smem_u32(&bar.k_full[i]), L::kDequantWarps / 2);
                mbar_init(smem_u32(&bar.v_full[i]), L::kDequantWarps / 2);
                mbar_init(smem_u32(&bar.s_full[i]), 1);
                mbar_init(smem_u32(&bar.v_free[i]), 1);
                mbar_init(smem_u32(&bar.p_full[i]), kSoftmaxWarps);
                mbar_init(smem_u32(&bar.q_full[i]), L::kRowWarps);
                mbar_init(smem_u32(&bar.q_free[i]), 1 + kSoftmaxWarps);
            }
            for (int i = 0; i < 2 * L::kRing; ++i) {
                bar.filled[i] = 0u;
                mbar_init(smem_u32(&bar.raw_full[i]), 1);
                mbar_init(smem_u32(&bar.raw_free[i]), L::kDequantWarps / 2);
            }
            for (int i = 0; i < kTiles; ++i) {
                mbar_init(smem_u32(&bar.tile_full[i]), 1);
                mbar_init(smem_u32(&bar.tile_free[i]), kSoftmaxWarps + L::kRowWarps + 3);
            }
            mbar_init(smem_u32(&bar.o_full), 1);
            mbar_init(smem_u32(&bar.o_free), L::kRowWarps);
            mbar_init(smem_u32(&bar.ml_full), kSoftmaxWarps);
            mbar_init(smem_u32(&bar.drained), 1);
            bar.stop = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            fence_async();
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&bar.tmem)),
                     "r"((uint32_t)L::kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    mine = __reduce_add_sync(0xFFFFFFFFu, mine);
    if (lane == 0) bar.sum[warp] = mine;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    static_assert(L::kThreads == 1024, "a lane per warp");
    const uint32_t units = __reduce_add_sync(0xFFFFFFFFu, bar.sum[lane]);
    const Cut cut(units, gridDim.x);
    const uint32_t first = cut.first_of(blockIdx.x);
    const int total = (int)(cut.first_of(blockIdx.x + 1) - first);
    if (total > 0) {
        // the sequence that has unit `first`
        uint32_t before = 0;
        for (int b0 = 0; b0 < B; b0 += L::kThreads) {
            const int b = b0 + threadIdx.x;
            uint32_t u = one;
            if (B > L::kThreads) u = b < B ? units_of(p, make_seq(p, b, read_raw(p, b))) : 0u;
            uint32_t sum = u;
#pragma unroll
            for (int by = 1; by < 32; by <<= 1) {
                const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, sum, by);
                if (lane >= by) sum += o;
            }
            __syncthreads();
            if (lane == 31) bar.sum[warp] = sum;
            __syncthreads();
            const uint32_t others = bar.sum[lane], all = __reduce_add_sync(0xFFFFFFFFu, others);
            sum += before + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? others : 0u);
            if (first < sum && first >= sum - u) {
                bar.start_b = b;
                bar.start_off = first - (sum - u);
            }
            before += all;
            if (before > first) break;
        }
        if (threadIdx.x == 0) {
            bar.units = units;
            bar.first = first;
            bar.total = total;
        }
        __syncthreads();
        if (warp >= L::kMmaWarp) {
            reg_give<L::kMmaRegs>();
            if (warp == L::kMmaWarp) Roles(p, bar, dyn).products();
            if (warp == L::kFetchWarp || warp == L::kFetchWarp + 2) Roles(p, bar, dyn).fetch();
            if (warp == L::kWalkWarp) Roles(p, bar, dyn).walk();
        } else if (warp >= L::kDequantWarp) {
            reg_give<L::kDequantRegs>();
            const int place = warp - L::kDequantWarp;
            if (!Roles::given_up(place)) Roles(p, bar, dyn).dequantise(place);
        } else if (warp >= L::kRowWarp) {
            static_assert(L::kRowRegs == L::kLaunchRegs, "as launched");
            Roles(p, bar, dyn).rows();
        } else {
            reg_take<L::kSoftmaxRegs>();
            if (warp % 4 < QUADS) Roles(p, bar, dyn).softmax();
            else if (Roles::taken(warp) >= 0) Roles(p, bar, dyn).dequantise(Roles::taken(warp));
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    } else if (threadIdx.x == 0) {
        TreeShare r = {};
        r.units = units;
        p.shares[blockIdx.x] = r;
    }
    if (threadIdx.x == 0 && bar.stop != 0) report(p.base.dev_error, KVC8_DEV_TIMEOUT);
    if (warp == L::kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)L::kTmemCols)
                     : "memory");
}

// Joins the partials of a tile that several CTAs share.  Block (c, y): the tile that CTA c begins in and CTA
// c + 1 goes on with, if there is one, and a part of its rows; D / 8 lanes a row, eight channels each; `share` warps
// take a part of the partials each.
template <int D>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const TreeArgs p, int ctas, int share) {
    constexpr int kLanes = D / 8, kWarpRows = 32 / kLanes;
    __shared__ float s_acc[kMergeThreads][9];
    const AttnArgs &a = p.base;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gl = lane % kLanes;
    const int c0 = blockIdx.x, c = c0 + 1, mine = warp % share;
    pdl_wait_prior_grid();
    const TreeShare r = p.shares[c];
    const Cut cut(r.units, (uint32_t)ctas);
    const uint32_t first = cut.first_of(c);
    if (cut.first_of(c + 1) == first || r.first >= first || r.first < cut.first_of(c0)) return;
    const int row = (blockIdx.y * (kMergeThreads / 32) + warp) / share * kWarpRows + lane / kLanes;
    const int rows = min(kRows, r.rows - r.row);
    if (blockIdx.y * (kMergeThreads / 32) / share * kWarpRows >= rows) return;
    const int parts = (int)cut.cta_of(r.first + (uint32_t)r.steps - 1u) - c0 + 1;
    const int at = min(row, rows - 1);
    // partial i: the last one of CTA c0 (its first, if the tile begins with its share), the first ones of the others
    auto slot_of = [&](int i) {
        return (int64_t)(2 * (c0 + i) + (i == 0 && r.first != cut.first_of(c0) ? 1 : 0)) * kRows + at;
    };
    float M = -INFINITY;
    for (int i = gl; i < parts; i += kLanes) M = fmaxf(M, a.part_m[slot_of(i)]);
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, s));
    float sum = 0.0f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    for (int i0 = mine; i0 < parts; i0 += 4 * share) {
        float4 v[4][2];
        float m[4], l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * share;
            v[k][0] = v[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            m[k] = -INFINITY, l[k] = 0.0f;
            if (i < parts) {
                const int64_t slot = slot_of(i);
                const float4 *src = reinterpret_cast<const float4 *>(a.part_o + slot / 32 * 32 * D + gl * 256 + slot % 32 * 8);
                v[k][0] = src[0];
                v[k][1] = src[1];
                m[k] = a.part_m[slot];
                l[k] = a.part_l[slot];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float f = m[k] == -INFINITY ? 0.0f : ex2(m[k] - M);
            sum += f * l[k];
            acc[0] += f * v[k][0].x, acc[1] += f * v[k][0].y, acc[2] += f * v[k][0].z, acc[3] += f * v[k][0].w;
            acc[4] += f * v[k][1].x, acc[5] += f * v[k][1].y, acc[6] += f * v[k][1].z, acc[7] += f * v[k][1].w;
        }
    }
    if (share > 1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_acc[threadIdx.x][e] = acc[e];
        s_acc[threadIdx.x][8] = sum;
        __syncthreads();
        if (mine != 0) return;
        for (int k = 1; k < share; ++k) {
            const float *o = s_acc[threadIdx.x + 32 * k];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += o[e];
            sum += o[8];
        }
    }
    if (row >= rows) return;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int q = r.row + row, t = q / a.group, j = q - t * a.group;
    uint16_t *dst = a.out + (int64_t)(r.token + t) * a.out_seq_stride + (int64_t)(r.head * a.group + j) * a.out_head_stride + gl * 8;
    uint32_t y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dst[2 * e] = (uint16_t)(y[e] & 0xFFFFu);
            dst[2 * e + 1] = (uint16_t)(y[e] >> 16);
        }
    }
}

struct Space {
    size_t m, l, shares, bytes;  // O first
};
Space space(const kvc8_geom &g) {
    constexpr size_t slots = (size_t)2 * kMaxCtas * kRows;
    Space s;
    s.m = slots * g.head_dim * sizeof(float);
    s.l = s.m + slots * sizeof(float);
    s.shares = s.l + slots * sizeof(float);
    s.bytes = align_up(s.shares + kMaxCtas * sizeof(TreeShare), kAlign);
    return s;
}

template <int MODE, int D, int QUADS>
cudaError_t launch_variant(const TreeArgs &p, cudaStream_t stream) {
    using L = Layout<D>;
    auto kern = tree_kernel<MODE, D, QUADS>;
    static std::atomic<uint64_t> prepared{0};  // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < kMaxDevices ? 1ull << dev : 0;
    if ((prepared.load(std::memory_order_relaxed) & bit) == 0) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
        if (e != cudaSuccess) return e;
        // a block launched with fewer registers could never hand out the warpgroups' shares
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, kern);
        if (e != cudaSuccess) return e;
        if (attr.numRegs < L::kLaunchRegs) return cudaErrorInvalidConfiguration;
        prepared.fetch_or(bit, std::memory_order_relaxed);
    }
    const kvc8_geom &g = p.base.g;
    const int64_t tiles = (int64_t)g.num_seqs * g.kv_heads * ((p.max_drafts * p.base.group + kRows - 1) / kRows);
    const int64_t most = tiles * (((int64_t)g.max_blocks_per_seq * g.block_size + kCols - 1) / kCols);
    const int sms = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    const int grid = (int)(most < sms ? most : sms);
    kern<<<(unsigned)grid, L::kThreads, (size_t)L::kBytes, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess || grid == 1) return e;
    // Partials a row has, about: CTAs per tile.  Up to six a warp.
    int share = 1;
    while (share < kMergeThreads / 32 && grid > 6 * share * tiles) share *= 2;
    const int rows = p.max_drafts * p.base.group < kRows ? p.max_drafts * p.base.group : kRows;
    const int per = kMergeThreads / (D / 8) / share;
    return launch_dependent(merge_kernel<D>, dim3((unsigned)(grid - 1), (unsigned)((rows + per - 1) / per)), kMergeThreads,
                            (size_t)0, stream, p, grid, share);
}

// By the most rows that a head can have.
template <int MODE, int D>
cudaError_t launch_rows(const TreeArgs &p, cudaStream_t stream) {
    const int rows = p.max_drafts * p.base.group;
    if (rows <= kRows / 4) return launch_variant<MODE, D, 1>(p, stream);
    if (rows <= kRows / 2) return launch_variant<MODE, D, 2>(p, stream);
    return launch_variant<MODE, D, 4>(p, stream);
}

template <int MODE>
cudaError_t launch_mode(const TreeArgs &p, cudaStream_t stream) {
    return p.base.g.head_dim == 64 ? launch_rows<MODE, 64>(p, stream) : launch_rows<MODE, 128>(p, stream);
}

}  // namespace

size_t tree_workspace_bytes(const kvc8_geom &g) { return space(g).bytes; }

cudaError_t launch_tree(TreeArgs p, void *workspace, cudaStream_t stream) {
    const Space s = space(p.base.g);
    char *ws = static_cast<char *>(workspace);
    p.base.part_o = reinterpret_cast<float *>(ws);
    p.base.part_m = reinterpret_cast<float *>(ws + s.m);
    p.base.part_l = reinterpret_cast<float *>(ws + s.l);
    p.shares = reinterpret_cast<TreeShare *>(ws + s.shares);
    if (p.base.g.quant_mode == 0) return launch_mode<0>(p, stream);
    if (p.base.g.quant_mode == 1) return launch_mode<1>(p, stream);
    return launch_mode<2>(p, stream);
}

}  // namespace kvc8
