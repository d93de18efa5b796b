// kvc8_tree.cu -- attention of drafted tokens: draft t of sequence b, query head j of kv head h,
// attends over the sequence's context and over those of its drafts that the mask names.
//   out = sum_p w_p V'[p] / sum_p w_p,  w_p = exp(scale <q, K'[p]>),  K', V' = fp32(code) * scale
//
// A sequence's T drafts times G query heads are T G query rows against the same positions: 4 T G D
// flops for 2 D bytes of codes a position and head, so HBM bounds up to about 150 rows and the
// tensor cores more.
//
// tree_kernel: one persistent CTA per SM, a tile of 128 query rows, 128 positions a step.  S = Q
// K'^T and O += P V' are tcgen05.mma (M = 128, fp16, fp32 in tensor memory); P replaces S in
// tensor memory and is the second product's A operand.  Warps by role:
//   softmax     4, a thread per query row: S from tensor memory, one-pass softmax (Milakov and
//               Gimelshein, Online normalizer calculation for softmax, 2018), P back; any m cancels
//               in the quotient, so the running maximum moves only when the weights grow by more
//               than 2^8, and O is seldom rescaled.  Warps without a row do nothing
//   rows        4: the next tile's queries into shared memory, the last one's O out of tensor memory
//   dequantise  8: codes from global memory a step ahead in registers, K' and V' as fp16 into a
//               two-stage ring
//   mma         one lane issues both products
// S and O are there twice: the scores of a step are made while the softmax works on the step before,
// and a tile's first products run while the last one's O is written.
//
// The units (sequence, kv head, row tile, step) are numbered in that order and cut into equal shares,
// a CTA's share in a row: ragged lengths need no plan, every CTA adds up the lengths itself.  What a
// CTA has of a tile that it does not hold whole it leaves as a partial (m, l, O), two at most: of the
// first tile of its share and of the last.  merge_kernel joins them.
//
// Every wait has a limit, after which the kernel reports KVC8_DEV_TIMEOUT and leaves.
#include "kvc8_tcgen05.cuh"

namespace kvc8 {
namespace {

constexpr int kStages = 2;     // steps of K', of V', of S; tiles of Q and O
constexpr int kMaskSlots = 4;  // steps whose valid counts are kept
constexpr int kMaxCtas = 152;  // SMs of a GB300
constexpr int kMergeThreads = 256;

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

// A walk over a CTA's share, tile by tile; the next sequence's lengths are on their way.  Each warp has
// its own in shared memory: it is looked at once a tile, and in registers the whole of it would push out what
// a step needs.
struct Walk {
    Seq s;
    Raw ahead;
    int tile, step;  // tile: kv head * s.tiles + row tile; step: the first of it in the share
    __device__ __forceinline__ int head() const { return tile / s.tiles; }
    __device__ __forceinline__ int row0() const { return (tile - tile / s.tiles * s.tiles) * kRows; }
    // By a whole warp, and only where the share goes on: there is a next tile then.
    __device__ __forceinline__ void next_tile(const TreeArgs &p, int lane) {
        __syncwarp();
        if (lane == 0) {
            step = 0;
            if (tile + 1 < s.tiles * p.base.g.kv_heads) {
                ++tile;
            } else {
                tile = 0;
                Seq x = s;
                Raw r = ahead;
                do {
                    x = make_seq(p, x.b + 1, r);
                    r = read_raw(p, x.b + 1);
                } while (x.drafts == 0 && x.b + 1 < p.base.g.num_seqs);
                s = x;
                ahead = r;
            }
        }
        __syncwarp();
    }
};

// ---- the kernel ---------------------------------------------------------------------

template <int D>
struct Layout {
    static constexpr int kSoftmaxWarps = 4, kRowWarps = 4, kDequantWarps = 8;
    static constexpr int kDequantWarp = kSoftmaxWarps + kRowWarps;
    static constexpr int kMmaWarp = kDequantWarp + kDequantWarps;  // three idle warps behind it
    static constexpr int kThreads = 640;
    // Registers per thread: a softmax thread holds a row's 128 scores, a dequantising one two tiles'
    // codes in flight.
    static constexpr int kSoftmaxRegs = 184, kRowRegs = 64, kDequantRegs = 96, kMmaRegs = 40;
    static constexpr int kLaunchRegs = 96;
    static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + kRowWarps * kRowRegs + kDequantWarps * kDequantRegs +
                        4 * kMmaRegs) <= kThreads * kLaunchRegs,
                  "the warpgroups' registers are the block's");
    static constexpr int kTileBytes = kRows * D * 2;  // a Q tile, K' or V' stage
    static constexpr int kQ = 0;
    static constexpr int kK = kStages * kTileBytes;
    static constexpr int kV = 2 * kStages * kTileBytes;
    static constexpr int kEnd = 3 * kStages * kTileBytes;
    // more than half of an SM's shared memory, so that a CTA has the SM's tensor memory to itself
    static constexpr int kBytes = (kEnd > 120 * 1024 ? kEnd : 120 * 1024) + 1024;
    static constexpr int kO = kStages * kCols;  // columns of tensor memory: S twice, then O
    static constexpr int kTmemCols = 512;
};

struct Barriers {
    // s_full: a step's scores, and its K' stage is free; v_free: its weighted values, and its V' stage
    uint64_t k_full[kStages], v_full[kStages], s_full[kStages], p_full[kStages], v_free[kStages];
    uint64_t q_full[kStages], q_free[kStages], o_full[kStages], o_free[kStages], ml_full[kStages], drained;
    uint32_t tmem;
    int32_t stop;
    uint32_t sum[Layout<128>::kThreads / 32];
    int32_t start_b;
    uint32_t start_off;
    int32_t total;  // units of this CTA
    Walk walk[Layout<128>::kMmaWarp + 1], walk_out[4];  // of each warp; of the rows that go out
    float q_scale[kStages][kRows];  // log2 per unit of score, with the query's power of two
    float m[kStages][kRows], l[kStages][kRows];
    uint2 valid[kMaskSlots];  // 8 bytes: valid positions of each group of 16
    // modes 0 and 2: what was taken out of each group of 16's scales, as powers of two:
    // the keys' 2^e, the values' e and 2^-e
    alignas(16) float k_pow[kMaskSlots][kCols / 16];
    alignas(16) float v_exp[kMaskSlots][kCols / 16];
    alignas(16) float v_inv[kMaskSlots][kCols / 16];
};

template <int MODE, int D>
struct Tree {
    using L = Layout<D>;
    static constexpr int kRpw = kCols / L::kDequantWarps;  // positions of a warp: one group of 16
    using T = CodeTile<MODE, D, kRpw>;
    using Codes = typename T::Codes;
    static_assert(T::kGroups == 1, "a warp's positions lie in one block");

    const TreeArgs &p;
    Barriers &bar;
    const uint32_t base, tmem;  // shared memory, 1 KB aligned
    const int total;            // units of this CTA
    Walk &walk;                 // this warp's
    const int lane, warp;

    // (Read again here, by each role for itself, than kept in registers from the kernel's start.)
    __device__ __forceinline__ Tree(const TreeArgs &args, Barriers &b, uint8_t *dyn)
        : p(args), bar(b), base((smem_u32(dyn) + 1023u) & ~1023u), tmem(b.tmem), total(b.total),
          walk(b.walk[threadIdx.x >> 5]), lane(threadIdx.x & 31), warp(threadIdx.x >> 5) {}

    __device__ __forceinline__ bool wait(uint64_t &b, uint32_t parity) const {
        return wait_limited(b, parity, bar.stop, p.base.dev_error);
    }
    // The same for a whole warp, which leaves it converged.
    __device__ __forceinline__ bool wait_warp(uint64_t &b, uint32_t parity) const {
        return __all_sync(0xFFFFFFFFu, wait(b, parity));
    }
    __device__ __forceinline__ void arrive(uint64_t &b) const {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&b));
    }

    // ---- dequantise ------------------------------------------------------------
    // Where a warp's group of 16 positions lies; of the step whose block id is asked for next.
    struct Place {
        int64_t page;       // block * heads + head
        int32_t at, valid;  // first slot in the block; positions before the end
    };
    __device__ __forceinline__ Place place(int32_t blk, int at, int valid, int head) const {
        const bool in = blk >= 0 && blk < p.base.g.num_blocks;
        if (!in && lane == 0) report(p.base.dev_error, KVC8_DEV_BAD_BLOCK_ID);
        return Place{(int64_t)(in ? blk : 0) * p.base.g.kv_heads + head, at, in ? max(0, min(16, valid)) : 0};
    }
    __device__ __forceinline__ void load(const Place &x, const int8_t *cache, Codes &c) const {
        const int8_t *src = cache + (x.page * p.base.g.block_size + x.at + T::row_in(lane)) * D + T::block_in(lane) * 64 + lane % 4 * 16;
        if (x.valid == 16) {
#pragma unroll
            for (int i = 0; i < T::kLoads; ++i) c.c[i] = ld_ahead_16(src + i * T::kRpl * D);
        } else {
#pragma unroll
            for (int i = 0; i < T::kLoads; ++i) {
                c.c[i] = make_uint4(0u, 0u, 0u, 0u);
                if (i * T::kRpl + T::row_in(lane) < x.valid) c.c[i] = ld_ahead_16(src + i * T::kRpl * D);
            }
        }
    }
    // Modes 0 and 2: the scale of position `lane` of the group.
    __device__ __forceinline__ float load_scale(const Place &x, const float *scale) const {
        const int64_t at = MODE == 0 ? x.page * p.base.g.block_size + x.at + lane : x.page;
        return lane < x.valid ? ld_ahead_f32(scale + at) : 0.0f;  // (16 at most)
    }

    __device__ void dequantise() const {
        const AttnArgs &a = p.base;
        const int dw = warp - L::kDequantWarp;
        // of the step whose block id is asked for next: positions left, slot and entry of the table; a
        // step is `jump` blocks and `rest` slots further on
        const int bs = a.g.block_size, jump = kCols / bs, rest = kCols - jump * bs;
        int left = 0, at = 0, head = 0;
        const int32_t *entry = nullptr;
        auto enter = [&]() {
            const int pos = walk.step * kCols + dw * kRpw;
            left = walk.s.len - pos;
            head = walk.head();
            at = pos % bs;
            entry = a.block_table + (int64_t)walk.s.b * a.g.max_blocks_per_seq + pos / bs;
        };
        auto next = [&]() {
            left -= kCols;
            at += rest;
            entry += jump;
            if (at >= bs) {
                at -= bs;
                ++entry;
            }
            if (left + dw * kRpw <= 0) {
                walk.next_tile(p, lane);
                enter();
            }
        };
        auto id = [&]() { return left > 0 ? ld_ahead_s32(entry) : 0; };
        enter();
        Place x = place(id(), at, left, head);
        Codes k, v;
        float sk = 0.0f, sv = 0.0f;
        auto scales = [&]() {
            if (MODE == 1) return;
            sk = load_scale(x, a.k_scale);
            sv = load_scale(x, a.v_scale);
        };
        scales();
        load(x, a.k_cache, k);
        load(x, a.v_cache, v);
        int32_t blk = 0;
        if (total > 1) {
            next();
            blk = id();
        }
        for (int n = 0; n < total; ++n) {
            const int st = n % kStages;
            const uint32_t par = (uint32_t)(n / kStages) & 1u;
            if (!wait_warp(bar.s_full[st], par ^ 1u)) return;
            uint32_t sk_half = 0u, sv_half = 0u;
            if (MODE != 1) {
                // A scale that is no number must not reach the rows that do not see its position,
                // nor the other scales' power: the value counts as zero, and the score as no number.
                const bool odd = (__float_as_uint(sk) & 0x7F800000u) == 0x7F800000u ||
                                 (__float_as_uint(sv) & 0x7F800000u) == 0x7F800000u;
                sk = odd ? 0.0f : sk;
                sv = odd ? 0.0f : sv;
                int ek, ev;
                const uint32_t top_k = T::group_top(sk, lane), top_v = T::group_top(sv, lane);
                sk_half = T::normal_scale(sk, top_k, -100, ek);
                sv_half = T::normal_scale(sv, top_v, kLeastValuePower, ev);
                if (odd) sk_half = 0x7FFF7FFFu;
                if (lane == 0) {
                    bar.k_pow[n % kMaskSlots][dw] = __uint_as_float((uint32_t)(127 + ek) << 23);
                    bar.v_exp[n % kMaskSlots][dw] = (float)ev;
                    bar.v_inv[n % kMaskSlots][dw] = __uint_as_float((uint32_t)(127 - ev) << 23);
                }
            }
            T::store(k, sk_half, base + L::kK + st * L::kTileBytes, dw, lane);
            if (lane == 0) reinterpret_cast<uint8_t *>(&bar.valid[n % kMaskSlots])[dw] = (uint8_t)x.valid;
            fence_async();
            arrive(bar.k_full[st]);
            const bool more = n + 1 < total;
            if (more) {  // the next step's codes, and the block id of the one after
                x = place(blk, at, left, head);
                scales();
                load(x, a.k_cache, k);
                if (n + 2 < total) {
                    next();
                    blk = id();
                }
            }
            if (!wait_warp(bar.v_free[st], par ^ 1u)) return;
            T::store(v, sv_half, base + L::kV + st * L::kTileBytes, dw, lane);
            fence_async();
            arrive(bar.v_full[st]);
            if (more) load(x, a.v_cache, v);
        }
    }

    // ---- products (a warp, one lane issuing) --------------------------------------------------
    __device__ __forceinline__ void qk(int q, int st, uint32_t tm, uint32_t leader) const {
        const uint64_t qd = operand_desc(base + L::kQ, 16) + (uint64_t)(q * (L::kTileBytes >> 4));
        const uint64_t kd = operand_desc(base + L::kK, 16) + (uint64_t)(st * (L::kTileBytes >> 4));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint64_t at = (uint64_t)(((i / 4) * (kRows * 128) + (i % 4) * 32) >> 4);
            tc_mma_ss(tm + st * kCols, qd + at, kd + at, instr_desc(kCols, false), i > 0, leader);
        }
    }
    __device__ __forceinline__ void pv(int o, int st, uint32_t tm, bool acc, uint32_t leader) const {
        const uint64_t v = operand_desc(base + L::kV, kCols * 128) + (uint64_t)(st * (L::kTileBytes >> 4));
#pragma unroll
        for (int i = 0; i < kCols / 16; ++i)
            tc_mma_ts(tm + L::kO + o * D, tm + st * kCols + 8 * i, v + (uint64_t)(i * (2048 >> 4)), instr_desc(D, true),
                      acc || i > 0, leader);
    }
    // What steers the loop comes from lane 0, so that the compiler keeps it, and with it stages,
    // addresses and descriptors, in uniform registers.
    __device__ __forceinline__ static int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

    __device__ bool products_loop(uint32_t leader) const {
        const uint32_t tm = (uint32_t)uniform((int)tmem);
        const int units = uniform(total);
        int left = uniform(walk.s.steps - walk.step);  // steps of the tile from the next scores on
        uint32_t q_seg = 0, seg = 0;             // tile of the next scores, of the next weighted values
        bool q_first = true;
        // Scores of unit n; returns whether it is its tile's last.
        auto scores = [&](int n, bool &ok) {
            const int st = n & 1, q = (int)(q_seg & 1u);
            ok = (!q_first || wait_warp(bar.q_full[q], (q_seg >> 1) & 1u)) && wait_warp(bar.k_full[st], (uint32_t)(n >> 1) & 1u);
            if (!ok) return false;
            tc_fence_after();
            qk(q, st, tm, leader);
            tc_commit(smem_u32(&bar.s_full[st]), leader);
            const bool last = --left == 0 || n + 1 == units;
            q_first = last;
            if (last) {
                tc_commit(smem_u32(&bar.q_free[q]), leader);
                ++q_seg;
                if (n + 1 < units) {
                    walk.next_tile(p, lane);
                    left = uniform(walk.s.steps);
                }
            }
            return last;
        };
        bool ok, first = true, last = scores(0, ok);
        if (!ok) return false;
        for (int n = 0; n < units; ++n) {
            const int st = n & 1, o = (int)(seg & 1u);
            bool next_last = false;
            if (n + 1 < units) {
                next_last = scores(n + 1, ok);
                if (!ok) return false;
            }
            if (first && !wait_warp(bar.o_free[o], ((seg >> 1) & 1u) ^ 1u)) return false;
            if (!wait_warp(bar.v_full[st], (uint32_t)(n >> 1) & 1u)) return false;
            if (!wait_warp(bar.p_full[st], (uint32_t)(n >> 1) & 1u)) return false;
            tc_fence_after();
            pv(o, st, tm, !first, leader);
            tc_commit(smem_u32(&bar.v_free[st]), leader);
            if (last) {
                tc_commit(smem_u32(&bar.o_full[o]), leader);
                ++seg;
            }
            first = last;
            last = next_last;
        }
        return true;
    }
    __device__ void products() const {
        const uint32_t leader = elect_lane();
        products_loop(leader);
        // what was issued is done before the tensor memory is freed
        tc_commit(smem_u32(&bar.drained), leader);
        const long long t0 = clock64();
        while (!mbar_try(smem_u32(&bar.drained), 0))
            if (clock64() - t0 > kWaitCycles) break;
    }

    // ---- rows in, rows out (a warp has 32 rows of the tile) ------------------------------------------
    // Query rows of a tile, in mode 1 times the channels' key scales: fp16 after a power of two that
    // brings a row's largest value to [1, 2) and goes into its factor.  Eleven bits hold a bf16 value
    // whole (mode 1: round the product eight times finer than bf16); below 2^-14 of the largest they
    // thin out to 2^-25 of it.  D / 8 lanes a row, kAhead loads in flight.
    __device__ __forceinline__ void load_rows(const Walk &w, int rw, int buf) const {
        constexpr int kLanes = D / 8, kWarpRows = 32 / kLanes, kAhead = 4;
        const AttnArgs &a = p.base;
        const int h = w.head(), r0 = w.row0() + rw * 32, rows = w.s.drafts * a.group;
        const int c = lane % kLanes;
        const bool flip = a.scale_log2 < 0.0f;  // the sign goes to the query
        float ks[8];
        if (MODE == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) ks[e] = __ldg(a.k_scale + (int64_t)h * D + 8 * c + e);
        }
#pragma unroll 1
        for (int i0 = 0; i0 < 32 / kWarpRows; i0 += kAhead) {
            if (r0 + i0 * kWarpRows >= (rows + 31) / 32 * 32) break;
            uint4 v[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int r = r0 + (i0 + i) * kWarpRows + lane / kLanes;
                v[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) {
                    const int t = r / a.group, j = r - t * a.group;
                    v[i] = __ldg(reinterpret_cast<const uint4 *>(a.q + (int64_t)(w.s.token + t) * a.q_seq_stride +
                                                                 (int64_t)(h * a.group + j) * a.q_head_stride + 8 * c));
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int at = rw * 32 + (i0 + i) * kWarpRows + lane / kLanes;  // row of the tile
                uint32_t wd[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                float y[8], top = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[2 * e] = __uint_as_float(wd[e] << 16);
                    y[2 * e + 1] = __uint_as_float(wd[e] & 0xFFFF0000u);
                    if (MODE == 1) y[2 * e] *= ks[2 * e], y[2 * e + 1] *= ks[2 * e + 1];
                    top = fmaxf(top, fmaxf(fabsf(y[2 * e]), fabsf(y[2 * e + 1])));
                }
#pragma unroll
                for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                const int ex = power_of(top);
                const float turn = __uint_as_float(((uint32_t)(127 - ex) << 23) | (flip ? 0x80000000u : 0u));
#pragma unroll
                for (int e = 0; e < 4; ++e) wd[e] = pack_fp16(y[2 * e] * turn, y[2 * e + 1] * turn);
                const uint32_t dst = base + L::kQ + buf * L::kTileBytes + (uint32_t)at * 128 +
                                     (uint32_t)(c / 8) * (kRows * 128) + (uint32_t)(((c % 8) ^ (at & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(wd[0]), "r"(wd[1]), "r"(wd[2]),
                             "r"(wd[3])
                             : "memory");
                if (c == 0) bar.q_scale[buf][at] = fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 + ex) << 23);
            }
        }
        fence_async();
        arrive(bar.q_full[buf]);
    }

    // A tile's O: to the output where the CTA has the whole tile, else a partial.
    __device__ __forceinline__ void store_rows(const Walk &w, int rw, int buf, bool whole, uint32_t seg) const {
        const AttnArgs &a = p.base;
        const int h = w.head(), row = rw * 32 + lane, r0 = w.row0() + rw * 32, rows = w.s.drafts * a.group;
        if (r0 < rows) {
            const uint32_t o_at = tmem + ((uint32_t)(rw * 32) << 16) + L::kO + buf * D;
            const int r = r0 + lane, t = r / a.group, j = r - t * a.group;
            const float m = bar.m[buf][row], l = bar.l[buf][row];
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint16_t *dst = a.out + (int64_t)(w.s.token + t) * a.out_seq_stride + (int64_t)(h * a.group + j) * a.out_head_stride;
            const int64_t slot = (int64_t)(2 * blockIdx.x + (seg > 0 ? 1 : 0)) * kRows + row;
            float *po = a.part_o + (slot - lane) * D + lane * 8;  // 32 rows' eighths in turn
#pragma unroll
            for (int c = 0; c < D; c += 16) {
                float o[16];
                tc_ld16(o, o_at + c);
                if (MODE == 1) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 sv = __ldg(reinterpret_cast<const float4 *>(a.v_scale + (int64_t)h * D + c + i));
                        o[i] *= sv.x, o[i + 1] *= sv.y, o[i + 2] *= sv.z, o[i + 3] *= sv.w;
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<float4 *>(po + (c + i) / 8 * 256 + i % 8) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else if (r < rows) {
                    uint32_t y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = pack_bf16(o[2 * i] * inv, o[2 * i + 1] * inv);
                    if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
                        reinterpret_cast<uint4 *>(dst + c)[0] = make_uint4(y[0], y[1], y[2], y[3]);
                        reinterpret_cast<uint4 *>(dst + c)[1] = make_uint4(y[4], y[5], y[6], y[7]);
                    } else {  // the output may lie on any element
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
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
        arrive(bar.o_free[buf]);
    }

    __device__ void rows() const {
        const int rw = warp - L::kSoftmaxWarps;
        Walk &in = walk, &out = bar.walk_out[rw];
        int in_left = total, out_left = total;
        uint32_t in_seg = 0;
        auto load_next = [&]() {
            const int buf = (int)(in_seg & 1u);
            if (!wait_warp(bar.q_free[buf], ((in_seg >> 1) & 1u) ^ 1u)) return false;
            load_rows(in, rw, buf);
            in_left -= min(in_left, in.s.steps - in.step);
            if (in_left > 0) in.next_tile(p, lane);
            ++in_seg;
            return true;
        };
        if (!load_next()) return;
        for (uint32_t seg = 0; out_left > 0; ++seg) {
            if (in_left > 0 && !load_next()) return;
            const int count = min(out_left, out.s.steps - out.step), buf = (int)(seg & 1u);
            if (!wait_warp(bar.ml_full[buf], (seg >> 1) & 1u) || !wait_warp(bar.o_full[buf], (seg >> 1) & 1u)) return;
            tc_fence_after();
            store_rows(out, rw, buf, count == out.s.steps, seg);
            out_left -= count;
            if (out_left > 0) out.next_tile(p, lane);
        }
    }

    // ---- softmax (one thread per query row) -----------------------------------
    // 32 bits of a row's mask from draft i on; drafts before the first are the context.
    __device__ __forceinline__ uint32_t mask_word(const uint32_t *mask, int word) const {
        if (word < 0) return 0xFFFFFFFFu;
        return word < 2 * p.mask_words ? __ldg(mask + word) : 0u;
    }

    __device__ void softmax() const {
        const int row = warp * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        int n = 0, left = total;
        for (uint32_t seg = 0; left > 0; ++seg) {
            const int count = min(left, walk.s.steps - walk.step), buf = (int)(seg & 1u);
            const int r0 = walk.row0() + warp * 32, rows = walk.s.drafts * p.base.group;
            const bool busy = r0 < rows;  // uniform in the warp: some row is a query's
            int d0 = walk.step * kCols - walk.s.ctx;  // the draft at a step's first position, if not negative
            const uint32_t o_at = tmem + lanes + L::kO + buf * D;
            float scale = 0.0f, m = -INFINITY, l = 0.0f;
            for (int i = 0; i < count; ++i, ++n, d0 += kCols) {
                const int st = n & 1;
                const bool drafts = d0 + kCols > 0;  // some position is a draft's
                uint32_t sees[4] = {0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu};
                if (drafts && busy) {
                    const int t = min(r0 + lane, rows - 1) / p.base.group;
                    if (p.mask == nullptr) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int upto = t - d0 + 1 - 32 * q;  // positions from the word's first on that are seen
                            sees[q] = upto >= 32 ? 0xFFFFFFFFu : upto <= 0 ? 0u : (1u << upto) - 1u;
                        }
                    } else {
                        const uint32_t *mask = reinterpret_cast<const uint32_t *>(p.mask + (int64_t)(walk.s.token + t) * p.mask_words);
                        uint32_t lo = mask_word(mask, d0 >> 5);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t hi = mask_word(mask, (d0 >> 5) + q + 1);
                            sees[q] = __funnelshift_r(lo, hi, (uint32_t)d0 & 31u);
                            lo = hi;
                        }
                    }
                }
                if (i == 0) {
                    if (!wait_warp(bar.q_full[buf], (seg >> 1) & 1u)) return;
                    scale = bar.q_scale[buf][row];
                    arrive(bar.q_free[buf]);
                }
                if (!wait_warp(bar.s_full[st], (uint32_t)(n >> 1) & 1u)) return;
                tc_fence_after();
                if (busy && !step(tmem + lanes + st * kCols, o_at, scale, i > 0, n, drafts, sees, m, l)) return;
                tc_fence_before();
                arrive(bar.p_full[st]);
            }
            if (!wait_warp(bar.o_free[buf], ((seg >> 1) & 1u) ^ 1u)) return;
            bar.m[buf][row] = m;
            bar.l[buf][row] = l;
            arrive(bar.ml_full[buf]);
            left -= count;
            if (left > 0) walk.next_tile(p, lane);
        }
    }

    // A group's factor of the scores and shift, read again where they are used (a thread
    // has no registers to keep sixteen).  The factor is never 0, which times the -inf of a
    // position left out would be no number; 2^-126 instead does not show.
    __device__ __forceinline__ float2 factor_shift(int slot, int grp, float scale) const {
        if (MODE == 1) return make_float2(fmaxf(scale, 0x1p-126f), 0.0f);
        float f, e;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(smem_u32(&bar.k_pow[slot][grp])));
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(e) : "r"(smem_u32(&bar.v_exp[slot][grp])));
        return make_float2(fmaxf(scale * f, 0x1p-126f), e);
    }

    // One step of a row: S -> P, the running maximum m and sum l.  A group's weights are
    // 2^(score + e - m), e the exponent taken out of its value scales, so that the product
    // with the tile's values is the weight times the value; m bounds score + e, lazily.
    // fp16 holds such weights (at most 2^15) eight times finer than bf16, and what falls
    // below 2^-21 of the largest to 2^-32 of it.
    __device__ __forceinline__ bool step(uint32_t s_at, uint32_t o_at, float scale, bool have_o, int n, bool drafts,
                                         const uint32_t (&sees)[4], float &m, float &l) const {
        const int slot = n % kMaskSlots;
        const uint2 valid = bar.valid[slot];
        float s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tc_ld32(s[q], s_at + 32 * q);
#pragma unroll
        for (int q = 0; q < 4; ++q) tc_wait_ld(s[q]);
        if (drafts || valid.x != 0x10101010u || valid.y != 0x10101010u) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t counts = (q < 2 ? valid.x : valid.y) >> (q % 2 * 16);
                const uint32_t in = ((1u << (counts & 0xFFu)) - 1u) | (((1u << (counts >> 8 & 0xFFu)) - 1u) << 16);
                const uint32_t keep = in & sees[q];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if ((keep >> i & 1u) == 0u) s[q][i] = -INFINITY;
            }
        }
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 fe = factor_shift(slot, 2 * q + i, scale);
                mx = fmaxf(mx, fmaf(top16(s[q], 16 * i), fe.x, fe.y));
            }
        }
        const bool moves = mx > m + (kLift + kLazy) || (m == -INFINITY && mx > m);
        if (__any_sync(0xFFFFFFFFu, moves)) {
            const float c = moves ? ex2(m - (mx - kLift)) : 1.0f;  // 0 where there was nothing yet
            if (moves) m = mx - kLift;
            l *= c;
            if (have_o) {  // once the step before is in it
                if (!wait_warp(bar.v_free[(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1u)) return false;
                tc_fence_after();
#pragma unroll
                for (int d = 0; d < D; d += 16) {
                    float o[16];
                    tc_ld16(o, o_at + d);
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(o[i] * c);
                    tc_st16(o_at + d, y);
                }
            }
        }
        const float neg = m == -INFINITY ? 0.0f : -m;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float2 a = factor_shift(slot, 2 * q, scale), b = factor_shift(slot, 2 * q + 1, scale);
            const float f[2] = {a.x, b.x}, g[2] = {a.y + neg, b.y + neg};
            float2 sum[2];
            uint32_t o[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float2 y = __ffma2_rn(make_float2(s[q][i], s[q][i + 1]), make_float2(f[i / 16], f[i / 16]),
                                      make_float2(g[i / 16], g[i / 16]));
                y = make_float2(ex2(y.x), ex2(y.y));
                sum[i / 16] = i % 16 == 0 ? y : __fadd2_rn(sum[i / 16], y);
                o[i / 2] = pack_fp16(y.x, y.y);
            }
            tc_st16(s_at + 16 * q, o);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float part = sum[i].x + sum[i].y;
                l = MODE == 1 ? l + part : fmaf(part, bar.v_inv[slot][2 * q + i], l);
            }
        }
        tc_wait_st();
        return true;
    }
};

template <int MODE, int D>
__global__ void __launch_bounds__(Layout<D>::kThreads, 1) tree_kernel(const TreeArgs p) {
    using L = Layout<D>;
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
                mbar_init(smem_u32(&bar.k_full[i]), L::kDequantWarps);
                mbar_init(smem_u32(&bar.v_full[i]), L::kDequantWarps);
                mbar_init(smem_u32(&bar.s_full[i]), 1);
                mbar_init(smem_u32(&bar.v_free[i]), 1);
                mbar_init(smem_u32(&bar.p_full[i]), L::kSoftmaxWarps);
                mbar_init(smem_u32(&bar.q_full[i]), L::kRowWarps);
                mbar_init(smem_u32(&bar.q_free[i]), 1 + L::kSoftmaxWarps);
                mbar_init(smem_u32(&bar.o_full[i]), 1);
                mbar_init(smem_u32(&bar.o_free[i]), L::kRowWarps);
                mbar_init(smem_u32(&bar.ml_full[i]), L::kSoftmaxWarps);
            }
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
    uint32_t units = 0;
#pragma unroll
    for (int i = 0; i < L::kThreads / 32; ++i) units += bar.sum[i];
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
            uint32_t all = 0;
#pragma unroll
            for (int i = 0; i < L::kThreads / 32; ++i) {
                if (i < warp) sum += bar.sum[i];
                all += bar.sum[i];
            }
            sum += before;
            if (first < sum && first >= sum - u) {
                bar.start_b = b;
                bar.start_off = first - (sum - u);
            }
            before += all;
            if (before > first) break;
        }
        __syncthreads();
        if (lane == 0) {
            Walk w;
            w.s = make_seq(p, bar.start_b, read_raw(p, bar.start_b));
            w.ahead = read_raw(p, bar.start_b + 1);
            w.tile = (int)(bar.start_off / (uint32_t)w.s.steps);
            w.step = (int)(bar.start_off - (uint32_t)w.tile * (uint32_t)w.s.steps);
            if (warp <= L::kMmaWarp) bar.walk[warp] = w;
            if (warp < L::kRowWarps) bar.walk_out[warp] = w;
            if (warp == L::kMmaWarp) {
                bar.total = total;
                TreeShare r;
                r.units = units;
                r.first = first - (uint32_t)w.step;
                r.steps = w.s.steps;
                r.token = w.s.token;
                r.rows = w.s.drafts * p.base.group;
                r.row = w.row0();
                r.head = w.head();
                r.pad = 0;
                p.shares[blockIdx.x] = r;
            }
        }
        __syncthreads();
        if (warp >= L::kMmaWarp) {
            reg_give<L::kMmaRegs>();
            if (warp == L::kMmaWarp) Tree<MODE, D>(p, bar, dyn).products();
        } else if (warp >= L::kDequantWarp) {
            static_assert(L::kDequantRegs == L::kLaunchRegs, "as launched");
            Tree<MODE, D>(p, bar, dyn).dequantise();
        } else if (warp >= L::kSoftmaxWarps) {
            reg_give<L::kRowRegs>();
            Tree<MODE, D>(p, bar, dyn).rows();
        } else {
            reg_take<L::kSoftmaxRegs>();
            Tree<MODE, D>(p, bar, dyn).softmax();
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

template <int MODE, int D>
cudaError_t launch_variant(const TreeArgs &p, cudaStream_t stream) {
    using L = Layout<D>;
    auto kern = tree_kernel<MODE, D>;
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

template <int MODE>
cudaError_t launch_mode(const TreeArgs &p, cudaStream_t stream) {
    return p.base.g.head_dim == 64 ? launch_variant<MODE, 64>(p, stream) : launch_variant<MODE, 128>(p, stream);
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
