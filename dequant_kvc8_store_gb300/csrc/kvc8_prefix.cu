// kvc8_prefix.cu -- decode attention of a batch whose sequences share a prefix:
// query head j of sequence b attends over the prefix's positions and then over
// its own, in one softmax.
//   out[b][j] = (sum_p w_p V'[p] + sum_p u_p V'_b[p]) / (sum_p w_p + sum_p u_p)
//   w_p = exp(scale <q, K'[p]>), u_p = exp(scale <q, K'_b[p]>)
// with K', V' = fp32(code) * scale; no position at all gives zeros.
//
// The sequences' own positions are kvc8_prefix_own.cu's: splits, each left as a
// partial (m, l, O).  The prefix is one
// matrix product for all sequences: a kv head's R = sequences * group query rows
// against P positions, 4 R P D flops for 2 P D bytes of codes, so for R above
// about 150 rows the tensor cores and not HBM bound it.
//
// prefix_kernel: a CTA holds NT tiles of 128 query rows and walks positions 128 at
// a time.  S = Q K'^T and O += P V' are tcgen05.mma (M = 128, fp16, fp32 in tensor
// memory); P replaces S in tensor memory and is the second product's A operand.
// Warps by role:
//   softmax     4 per tile, one thread per query row: S from tensor memory, one-pass
//               softmax (Milakov and Gimelshein, Online normalizer calculation for
//               softmax, 2018), P back; any m cancels in the quotient, so the running
//               maximum moves only when the weights grow by more than 2^8, and O is
//               seldom rescaled
//   dequantise  codes from global memory a tile ahead in registers, K' and V' as fp16
//               into a two-stage ring in the 128-byte swizzle (K' K-major, V' as the
//               MN-major B operand of the same rows)
//   mma         one lane issues both products; with two tiles one's products run
//               while the other's softmax does
// The (tile, 128 positions) units are cut over the CTAs (at most one per SM), each taking its
// share in a row, within one tile or (all of them) evenly over all tiles.  A CTA leaves one
// partial per tile it touches; CTA i's of tile t is in slot t + i, which no other pair has.
//
// The own positions' kernel starts when all CTAs have started and fills the SMs that have
// none, then those that are done; merge_kernel joins a row's partials of both.  An SM that
// reads own positions alone waits for memory, one that multiplies alone hardly reads any,
// so the two side by side are quicker than one after the other, and how many CTAs the prefix
// gets depends on how many own positions there are: see best_cut.  Measured, own positions
// first and one CTA per SM -> side by side, all SMs to the prefix -> the cut chosen: 10007
// positions x 23 sequences 36.9 -> 26.7 -> 26.3 us; 8192 x 64 62.0 -> 58.8 -> 47.2 (96 CTAs
// of 152 SMs; 45.1 since); 32768 x 256 198.4 -> 193.9 -> 170.6 (96).
//
// What bounds a step (two tiles, D = 128): 2048 cycles of tensor cores, and on the pipe of
// shared memory 1540 cycles of operand reads, 680 of dequantised tiles stored and 560 of other
// accesses; it takes about 3900.  32768 positions x 1024 rows x 8 kv heads, 137 GFLOP: 120 us
// on all SMs, 166 on 96.
//
// Every wait has a limit, after which the kernel reports KVC8_DEV_TIMEOUT and leaves.
#include "kvc8_codes.cuh"
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kRows = 128;      // query rows of a tile
constexpr int kCols = 128;      // positions of a step
constexpr int kStages = 2;      // steps of K' and of V' in shared memory
constexpr int kMaskSlots = 4;   // steps whose valid counts are kept
constexpr int kMaxCtas = 152;   // SMs of a GB300
// The weights are 2^(score - m) with m below the largest score by kLift when it is set, and
// m moves when a score passes it by kLift + kLazy more: the fp16 weights use fp16's range
// up to 2^15, and one of 2^-21 of the row's largest still has all its eleven bits.
constexpr float kLazy = 8.0f, kLift = 7.0f;
// The least exponent taken out of value scales, so that the sum of such weights (up to 2^15)
// times 2^-e over 2^31 positions is finite.  Scales below 2^-74 then lie under fp16's normal
// range: they and their products with a code are off by 2^-85 each, a value by 2^-78.
constexpr int kLeastValuePower = -60;
constexpr long long kWaitCycles = 4000000000ll;  // about two seconds
constexpr int kMergeThreads = 256;
// What else costs time, in steps, about: a CTA's start and end, its change of tile, the own
// positions' kernel after the prefix's.
constexpr int kStart = 4, kTileChange = 3, kOwnLeast = 3;

// ---- PTX ------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// The same without suspending the thread.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The products are issued by one elected lane of a warp that stays converged, so that
// addresses and descriptors are uniform.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(leader)
        : "memory");
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                          uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                          uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
        : "memory");
}
// 32 columns of this thread's row of tensor memory.
__device__ __forceinline__ void tc_ld32(float (&r)[32], uint32_t addr) {
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]),
          "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]),
          "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_ld16(float (&r)[16], uint32_t addr) {
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
          "=r"(u[14]), "=r"(u[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(u[0]),
        "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]), "r"(u[8]),
        "r"(u[9]), "r"(u[10]), "r"(u[11]), "r"(u[12]), "r"(u[13]), "r"(u[14]), "r"(u[15]), "r"(addr)
        : "memory");
}
// The loads before it are done; r takes part so that nothing reads it earlier.
__device__ __forceinline__ void tc_wait_ld(float (&r)[32]) {
    uint32_t *u = reinterpret_cast<uint32_t *>(r);
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(u[0]), "+r"(u[1]), "+r"(u[2]), "+r"(u[3]), "+r"(u[4]), "+r"(u[5]), "+r"(u[6]),
                   "+r"(u[7]), "+r"(u[8]), "+r"(u[9]), "+r"(u[10]), "+r"(u[11]), "+r"(u[12]),
                   "+r"(u[13]), "+r"(u[14]), "+r"(u[15]), "+r"(u[16]), "+r"(u[17]), "+r"(u[18]),
                   "+r"(u[19]), "+r"(u[20]), "+r"(u[21]), "+r"(u[22]), "+r"(u[23]), "+r"(u[24]),
                   "+r"(u[25]), "+r"(u[26]), "+r"(u[27]), "+r"(u[28]), "+r"(u[29]), "+r"(u[30]),
                   "+r"(u[31])
                 :
                 : "memory");
}
// This warpgroup's registers per thread from here on.
template <int N>
__device__ __forceinline__ void reg_give() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_take() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand: 128-byte swizzle, 8 rows of 128 bytes 1 KB apart (sbo),
// 64-channel blocks of an MN-major operand lbo apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// M = 128, fp16 operands, fp32 accumulators; b_mn: B is MN-major.
constexpr uint32_t instr_desc(int n, bool b_mn) {
    return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(kRows >> 4) << 24);
}

// ---- the work's split -------------------------------------------------------------

// Units (tile, step of 128 positions), numbered tile by tile, are cut into shares: of `n`
// CTAs that share `units` of them each takes `per` in a row, the first `more` one more.
// The CTAs are those of one tile, or all of them share all tiles.  All units are fewer than
// 2^31 (larger calls are refused).
struct PrefixWork {
    uint32_t units, per, more, n;
    int32_t steps, len, per_tile;
    __device__ __forceinline__ uint32_t first_of(uint32_t cta) const { return cta * per + min(cta, more); }
    __device__ __forceinline__ uint32_t cta_of(uint32_t unit) const {
        const uint32_t edge = more * (per + 1);
        return unit < edge ? unit / (per + 1) : more + (unit - edge) / per;
    }
};

// The sequences' own positions, in units of 64: this thread's part of what the block adds up
// (modulo 2^32: it only steers the cut).
__device__ __forceinline__ uint32_t own_part(const PrefixArgs &p) {
    const int64_t cap = (int64_t)p.own.g.max_blocks_per_seq * p.own.g.block_size;
    uint32_t n = 0;
    for (int b = threadIdx.x; b < p.own.g.num_seqs; b += blockDim.x)
        n += (uint32_t)(min((int64_t)max(0, __ldg(p.own.context_lengths + b)), cap) + 63) >> 6;
    return n;
}

// The cut with which prefix and own positions are done first, in steps' times, for a prefix that
// fills its table (see prefix_cuts).  The own positions take `own` steps of an SM: on the SMs without a CTA while the prefix lasts,
// then on all, and then not less than kOwnLeast.  Every CTA finds the same; the first leaves it
// in the workspace for the merge.
__device__ __forceinline__ int best_cut(const PrefixArgs &p, uint32_t own_units) {
    const float own = __fmul_rn(__uint2float_rn(own_units), p.own_weight);
    int best = 0;
    float least = INFINITY;
#pragma unroll 1
    for (int i = 0; i < p.cuts; ++i) {
        const float rest = __fadd_rn(own, -p.cut[i].beside);
        const float t = __fadd_rn(p.cut[i].time, rest > 0.0f ? __fadd_rn(rest, p.own_least) : 0.0f);
        if (t < least) {
            least = t;
            best = i;
        }
    }
    return best;
}

__device__ __forceinline__ PrefixWork prefix_work(const PrefixArgs &p, int32_t given, const PrefixCut &cut) {
    PrefixWork w;
    w.per_tile = cut.per_tile;
    const int64_t cap = (int64_t)p.max_prefix_blocks * p.own.g.block_size;
    w.len = (int32_t)max((int64_t)0, min((int64_t)given, cap));
    w.steps = (int32_t)(((uint32_t)w.len + kCols - 1) / kCols);
    w.n = (uint32_t)(cut.per_tile > 0 ? cut.per_tile : cut.ctas);
    w.units = (uint32_t)w.steps * (uint32_t)(cut.per_tile > 0 ? 1 : p.tiles_per_head * p.own.g.kv_heads);
    w.per = w.units / w.n;
    w.more = w.units - w.per * w.n;
    return w;
}

// ---- the kernel ---------------------------------------------------------------------

template <int MODE, int D, int NT>
struct Layout {
    static constexpr int kDequantWarps = NT == 1 ? 8 : 4;
    static constexpr int kSoftmaxWarps = 4 * NT;
    static constexpr int kMmaWarp = kSoftmaxWarps + kDequantWarps;  // three idle warps behind it
    static constexpr int kThreads = 512;
    // The products of a step's first half run while the second half's weights are made.  With
    // two tiles one's products run beside the other's softmax anyway (60000 positions in mode 0,
    // one tile: 66.0 us in halves, 69.2 whole; two tiles, 1024 rows x 32768: 172.3 and 171.0).
    static constexpr bool kHalves = NT == 1;
    // Registers per thread: a softmax thread holds a row's 128 scores; a dequantising one two
    // tiles' codes in flight, and with scales per row or block those too.  (Two tiles, 32768
    // positions x 1024 rows: dynamic scales 221 us with 176 and 120, 235 with 184 and 104; channel
    // scales 172.4 and 171.8.)  Spilled all the same (bytes a thread stored / loaded): two tiles
    // 20 / 36, in mode 1 32 / 44 at D = 128 and none at 64; one tile none, but 24 / 68 in mode 1
    // at D = 64.
    static constexpr bool kScales = MODE != 1 && NT == 2;
    static constexpr int kSoftmaxRegs = kScales ? 176 : 184, kDequantRegs = NT == 1 ? 112 : kScales ? 120 : 104, kMmaRegs = 40;
    static constexpr int kLaunchRegs = 128;
    static_assert(32 * (kSoftmaxWarps * kSoftmaxRegs + kDequantWarps * kDequantRegs + 4 * kMmaRegs) <=
                      kThreads * kLaunchRegs,
                  "the warpgroups' registers are the block's");
    static constexpr int kTileBytes = kRows * D * 2;  // Q tile, K' or V' stage
    static constexpr int kQ = 0;
    static constexpr int kK = NT * kTileBytes;
    static constexpr int kV = kK + kStages * kTileBytes;
    static constexpr int kEnd = kV + kStages * kTileBytes;
    // more than half of an SM's shared memory, so that a CTA has the SM's tensor
    // memory to itself
    static constexpr int kBytes = (kEnd > 120 * 1024 ? kEnd : 120 * 1024) + 1024;
    static constexpr int kTmemCols = NT * (kCols + D) > 256 ? 512 : 256;
};

struct Barriers {
    uint64_t k_full[kStages], k_free[kStages], v_full[kStages], v_free[kStages];
    uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2], drained;
    uint32_t tmem;
    int32_t stop;
    uint32_t own[16];  // own positions, counted by each warp
    uint2 valid[kMaskSlots];  // 8 bytes: valid positions of each group of 16
    // modes 0 and 2: what was taken out of each group of 16's scales, as powers of two:
    // the keys' 2^e, the values' e and 2^-e
    alignas(16) float k_pow[kMaskSlots][kCols / 16];
    alignas(16) float v_exp[kMaskSlots][kCols / 16];
    alignas(16) float v_inv[kMaskSlots][kCols / 16];
};

template <int MODE, int D, int NT>
struct Prefix {
    using L = Layout<MODE, D, NT>;
    const PrefixArgs &p;
    Barriers &bar;
    const uint32_t base;  // shared memory, 1 KB aligned
    const PrefixWork w;
    const int total;         // units of this CTA
    const int tile0, step0;  // the first one's tile and step
    const int lane;

    // false: the limit ran out here or elsewhere in the CTA
    __device__ __forceinline__ bool wait(uint64_t &b, uint32_t parity) const {
        const uint32_t at = smem_u32(&b);
        if (mbar_try(at, parity)) return true;
        const long long t0 = clock64();
        while (!mbar_try(at, parity)) {
            if (*static_cast<volatile int32_t *>(&bar.stop) != 0) return false;
            if (clock64() - t0 > kWaitCycles) {
                *static_cast<volatile int32_t *>(&bar.stop) = 1;
                report(p.own.dev_error, KVC8_DEV_TIMEOUT);
                return false;
            }
        }
        return true;
    }

    // The same for a whole warp, which leaves it converged.
    __device__ __forceinline__ bool wait_warp(uint64_t &b, uint32_t parity) const {
        return __all_sync(0xFFFFFFFFu, wait(b, parity));
    }

    // ---- dequantise ------------------------------------------------------------
    static constexpr int kRpw = kCols / L::kDequantWarps;  // positions of a warp
    static constexpr int kGroups = kRpw / 16;  // a group of 16 positions lies in one block
    static constexpr int kRpl = 512 / D;  // positions of one load (whole lines: 512 bytes)
    static constexpr int kLoads = kRpw / kRpl;

    // Of each load a lane takes 16 codes of a 64-channel block.  D = 64: codes 16 (l % 4)
    // of position l / 4.  D = 128: of every 16 lanes and two positions, lanes 0-3 take the
    // first block of the first, 4-7 the second of the second, 8-11 the first of the
    // second, 12-15 the second of the first, so that the eight lanes of a shared-memory
    // access hold different rows (see store).
    static __device__ __forceinline__ int row_in(int lane) {
        return D == 64 ? lane >> 2 : 2 * (lane >> 4) + (((lane >> 2) ^ (lane >> 3)) & 1);
    }
    static __device__ __forceinline__ int block_in(int lane) { return D == 64 ? 0 : (lane >> 2) & 1; }
    struct Codes {
        uint4 c[kLoads];
    };
    struct Where {
        int64_t row[kGroups];  // cache row of each group's first position
        int64_t blk[kGroups];  // block * heads + head
        int valid[kGroups];
    };
    struct Ids {
        int32_t blk[kGroups], at[kGroups], valid[kGroups];
    };

    // Block ids of a step's groups, requested a step before they are used.
    __device__ __forceinline__ Ids find(int step, int dw) const {
        Ids x;
        const uint32_t bs = (uint32_t)p.own.g.block_size;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int pos = step * kCols + dw * kRpw + 16 * i;
            const uint32_t lb = (uint32_t)pos / bs;
            x.at[i] = pos - (int)(lb * bs);
            x.valid[i] = min(16, w.len - pos);
            x.blk[i] = pos < w.len ? ld_nc_s32(p.prefix_table + lb) : 0;
        }
        return x;
    }
    __device__ __forceinline__ Where place(const Ids &x, int h) const {
        Where o;
        const kvc8_geom &g = p.own.g;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const bool in = x.blk[i] >= 0 && x.blk[i] < g.num_blocks;
            if (!in && lane == 0) report(p.own.dev_error, KVC8_DEV_BAD_BLOCK_ID);
            o.valid[i] = in ? max(0, x.valid[i]) : 0;
            o.blk[i] = (int64_t)(in ? x.blk[i] : 0) * g.kv_heads + h;
            o.row[i] = o.blk[i] * g.block_size + x.at[i];
        }
        return o;
    }

    __device__ __forceinline__ void load(const Where &x, const int8_t *cache, Codes &c) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int pos = i * kRpl, at = pos % 16 + row_in(lane);
            c.c[i] = make_uint4(0u, 0u, 0u, 0u);
            if (at < x.valid[pos / 16])
                c.c[i] = ld_stream_16(cache + (x.row[pos / 16] + at) * D + block_in(lane) * 64 + lane % 4 * 16);
        }
    }
    // Modes 0 and 2: the scale of position `lane` of the warp.
    __device__ __forceinline__ float load_scale(const Where &x, const float *scale) const {
        const bool second = kGroups == 2 && lane >= 16;
        const int64_t row = second ? x.row[kGroups - 1] : x.row[0];
        const int64_t blk = second ? x.blk[kGroups - 1] : x.blk[0];
        const int valid = second ? x.valid[kGroups - 1] : x.valid[0];
        return lane < kRpw && (lane & 15) < valid ? ld_nc_f32(scale + (MODE == 0 ? row + (lane & 15) : blk)) : 0.0f;
    }

    // fp16 pairs (s / 2^e, s / 2^e) of a position's two scales, e the exponent of the largest
    // of its group of 16, so that 127 times it is far inside fp16 whatever the scales' size.
    // Sizes are compared as integers; in mode 2 a group has one scale.  (Two reductions by the
    // whole warp instead of four exchanges: 32768 positions x 1024 rows, mode 0, 241 -> 235
    // us; for the one group of the other layout the exchanges were faster, 65.7 and 67.4.)
    __device__ __forceinline__ static uint32_t group_top(float s, int lane) {
        uint32_t size = __float_as_uint(s) & 0x7FFFFFFFu;
        if (MODE == 2) return size;
        if (kGroups == 1) {
            float top = fabsf(s);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            return __float_as_uint(top);
        }
        const uint32_t a = __reduce_max_sync(0xFFFFFFFFu, lane < 16 ? size : 0u);
        const uint32_t b = __reduce_max_sync(0xFFFFFFFFu, lane < 16 ? 0u : size);
        return lane < 16 ? a : b;
    }
    __device__ __forceinline__ static uint32_t normal_scale(float s, uint32_t top, int least, int &e) {
        e = max(least, power_of(__uint_as_float(top)));
        s *= __uint_as_float((uint32_t)(127 - e) << 23);
        return pack_fp16(s, s);
    }

    // Codes times their scale (modes 0 and 2; mode 1 has the scales in the query and the
    // output) into the swizzled tile, as fp16: the code is exact, the scale and the product
    // are each rounded to eleven bits, eight times finer than the bf16 rows of the gather.
    // 16-byte chunk n of a 128-byte row lies at n ^ (row mod 8): a lane's two places repeat
    // (D = 128: with one bit flipped) from load to load, and the eight lanes of an access,
    // on two neighbouring rows, hit different banks.
    __device__ __forceinline__ void store(const Codes &c, uint32_t scale, uint32_t tile, int dw) const {
        const int n = (lane & 3) * 2, r = row_in(lane);
        const uint32_t at = tile + (uint32_t)(dw * kRpw + r) * 128 + (uint32_t)block_in(lane) * (kCols * 128);
        const uint32_t c0 = (uint32_t)((n ^ r) << 4), c1 = (uint32_t)(((n + 1) ^ r) << 4);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t wd[4] = {c.c[i].x, c.c[i].y, c.c[i].z, c.c[i].w};
            const uint32_t s = MODE == 1 ? 0u : __shfl_sync(0xFFFFFFFFu, scale, i * kRpl + r);
            uint32_t o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                o[e] = codes_fp16(wd[e >> 1] ^ 0x80808080u, (e & 1) ? 0x4342u : 0x4140u);
                if (MODE != 1) o[e] = mul_fp16(o[e], s);
            }
            const uint32_t flip = (uint32_t)(i * kRpl % 8) << 4, row = at + (uint32_t)(i * kRpl * 128);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + (c0 ^ flip)), "r"(o[0]), "r"(o[1]),
                         "r"(o[2]), "r"(o[3])
                         : "memory");
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row + (c1 ^ flip)), "r"(o[4]), "r"(o[5]),
                         "r"(o[6]), "r"(o[7])
                         : "memory");
        }
    }

    __device__ void dequantise(int dw) const {
        const AttnArgs &a = p.own;
        int tile = tile0, step = step0;
        Where x = place(find(step, dw), tile / p.tiles_per_head);
        Codes k, v;
        float sk = 0.0f, sv = 0.0f;
        auto scales = [&]() {
            if (MODE == 1) return;
            sk = load_scale(x, a.k_scale);
            sv = load_scale(x, a.v_scale);
        };
        auto next = [&]() {
            if (++step == w.steps) {
                step = 0;
                ++tile;
            }
        };
        load(x, a.k_cache, k);
        scales();
        load(x, a.v_cache, v);
        next();
        Ids ids = find(step, dw);
        int n = 0;
        for (; n < total; ++n) {
            const int st = n % kStages;
            const uint32_t par = (uint32_t)(n / kStages) & 1u;
            if (!wait_warp(bar.k_free[st], par ^ 1u)) return;
            uint32_t sk_half = 0u, sv_half = 0u;
            if (MODE != 1) {
                int ek, ev;
                const uint32_t top_k = group_top(sk, lane), top_v = group_top(sv, lane);
                sk_half = normal_scale(sk, top_k, -100, ek);
                sv_half = normal_scale(sv, top_v, kLeastValuePower, ev);
                if (lane < kRpw && lane % 16 == 0) {
                    const int grp = dw * kGroups + lane / 16;
                    bar.k_pow[n % kMaskSlots][grp] = __uint_as_float((uint32_t)(127 + ek) << 23);
                    bar.v_exp[n % kMaskSlots][grp] = (float)ev;
                    bar.v_inv[n % kMaskSlots][grp] = __uint_as_float((uint32_t)(127 - ev) << 23);
                }
            }
            store(k, sk_half, base + L::kK + st * L::kTileBytes, dw);
            if (lane == 0) {
                uint8_t *vc = reinterpret_cast<uint8_t *>(&bar.valid[n % kMaskSlots]) + dw * kGroups;
#pragma unroll
                for (int i = 0; i < kGroups; ++i) vc[i] = (uint8_t)x.valid[i];
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar.k_full[st]));
            const bool more = n + 1 < total;
            if (more) {  // the next step's codes, and the block ids of the one after
                x = place(ids, tile / p.tiles_per_head);
                load(x, a.k_cache, k);
                scales();
                next();
                ids = find(step, dw);
            }
            if (!wait_warp(bar.v_free[st], par ^ 1u)) return;
            store(v, sv_half, base + L::kV + st * L::kTileBytes, dw);
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar.v_full[st]));
            if (more) load(x, a.v_cache, v);
        }
    }

    // ---- products (a warp, one lane issuing) --------------------------------------------------
    // Descriptors of the first operand block; a later one is (bytes >> 4) further on.
    // `peek` runs before the last of the eight are issued, while the tensor cores have
    // work: what it finds ready need not be waited for afterwards.
    template <typename Peek>
    __device__ __forceinline__ void qk(int x, int st, uint32_t tmem, uint32_t leader, Peek &&peek) const {
        const uint64_t q = operand_desc(base + L::kQ, 16) + (uint64_t)(x * (L::kTileBytes >> 4));
        const uint64_t k = operand_desc(base + L::kK, 16) + (uint64_t)(st * (L::kTileBytes >> 4));
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            if (i == D / 16 - 3) peek();
            const uint64_t at = (uint64_t)(((i / 4) * (kRows * 128) + (i % 4) * 32) >> 4);
            tc_mma_ss(tmem + x * kCols, q + at, k + at, instr_desc(kCols, false), i > 0, leader);
        }
    }
    // One half of the step's positions.
    template <typename Peek>
    __device__ __forceinline__ void pv(int x, int half, int st, uint32_t tmem, bool acc, uint32_t leader,
                                       Peek &&peek) const {
        const uint64_t v = operand_desc(base + L::kV, kCols * 128) + (uint64_t)(st * (L::kTileBytes >> 4));
#pragma unroll
        for (int j = 0; j < kCols / 32; ++j) {
            const int i = half * (kCols / 32) + j;
            if (j == 1) peek();
            tc_mma_ts(tmem + NT * kCols + x * D, tmem + x * kCols + 8 * i, v + (uint64_t)(i * (2048 >> 4)),
                      instr_desc(D, true), acc || i > 0, leader);
        }
    }
    __device__ __forceinline__ bool ready(uint64_t &b, uint32_t parity) const {
        return __all_sync(0xFFFFFFFFu, mbar_test(smem_u32(&b), parity));
    }

    // The loop's own quantities come from lane 0, so that the compiler keeps them, and
    // with them stages, addresses and descriptors, in uniform registers.
    __device__ __forceinline__ static int uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

    // The weights that a step's products wait for first.
    __device__ __forceinline__ uint64_t &first_p(int x) const { return L::kHalves ? bar.p_half[x] : bar.p_full[x]; }

    __device__ bool products_loop(uint32_t tmem_any, uint32_t leader) const {
        const uint32_t tmem = (uint32_t)uniform((int)tmem_any);
        const int units = uniform(total), steps = uniform(w.steps);
        int in_tile = uniform(step0);  // step of the tile
        uint32_t seg = 0;
        bool first = true, next_p = false, next_v = false;
        for (int i = 0; i < units; ++i) {
            const int st = i & 1, st1 = st ^ 1;  // stages of this step and the next
            const uint32_t par = (uint32_t)(i >> 1) & 1u, par1 = (uint32_t)((i + 1) >> 1) & 1u;
            const bool more = i + 1 < units && in_tile + 1 < steps;  // the next step is of this tile
            bool p_in[2] = {false, false}, k_in = false, v_in = false;
            if (first) {
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    if (!wait_warp(bar.q_full[x], seg & 1u)) return false;
                    if (x == 0 && !wait_warp(bar.k_full[st], par)) return false;
                    tc_fence_after();
                    qk(x, st, tmem, leader, [] {});
                    tc_commit(smem_u32(&bar.s_full[x]), leader);
                    if (x == NT - 1) tc_commit(smem_u32(&bar.k_free[st]), leader);
                }
            } else {
                p_in[0] = next_p;
                v_in = next_v;
            }
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                if (!p_in[x] && !wait_warp(first_p(x), (uint32_t)st)) return false;
                if (x == 0 && !v_in && !wait_warp(bar.v_full[st], par)) return false;
                tc_fence_after();
                bool p_rest = !L::kHalves;
                pv(x, 0, st, tmem, !first, leader, [&]() {
                    if (L::kHalves) p_rest = ready(bar.p_full[x], (uint32_t)st);
                });
                if (!p_rest && !wait_warp(bar.p_full[x], (uint32_t)st)) return false;
                if (L::kHalves) tc_fence_after();
                pv(x, 1, st, tmem, true, leader, [&]() {
                    if (x == 0 && more) k_in = ready(bar.k_full[st1], par1);
                });
                if (x == NT - 1) tc_commit(smem_u32(&bar.v_free[st]), leader);
                if (more) {
                    if (x == 0 && !k_in && !wait_warp(bar.k_full[st1], par1)) return false;
                    tc_fence_after();
                    qk(x, st1, tmem, leader, [&]() {
                        if (x + 1 < NT) {
                            p_in[x + 1] = ready(first_p(x + 1), (uint32_t)st);
                        } else {
                            next_v = ready(bar.v_full[st1], par1);
                            next_p = NT > 1 && ready(first_p(0), (uint32_t)st1);
                        }
                    });
                    tc_commit(smem_u32(&bar.s_full[x]), leader);
                    if (x == NT - 1) tc_commit(smem_u32(&bar.k_free[st1]), leader);
                } else {
                    tc_commit(smem_u32(&bar.o_full[x]), leader);
                }
            }
            first = !more;
            seg += first ? 1 : 0;
            in_tile = first ? 0 : in_tile + 1;
        }
        return true;
    }

    __device__ void products(uint32_t tmem) const {
        const uint32_t leader = elect_lane();
        products_loop(tmem, leader);
        // what was issued is done before the tensor memory is freed
        tc_commit(smem_u32(&bar.drained), leader);
        const long long t0 = clock64();
        while (!mbar_try(smem_u32(&bar.drained), 0))
            if (clock64() - t0 > kWaitCycles) break;
    }

    // ---- softmax (one thread per query row) -----------------------------------
    __device__ void softmax(int warp, uint32_t tmem) const {
        const AttnArgs &a = p.own;
        const int x = warp >> 2, row = (warp & 3) * 32 + lane;  // tile of the CTA, row of the tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + lanes + x * kCols, o_at = tmem + lanes + NT * kCols + x * D;
        const int rows = p.rows;
        const bool flip = a.scale_log2 < 0.0f;  // the sign goes to the query
        int n = 0;
        uint32_t seg = 0;
        int left = total;
        for (int tile = tile0; left > 0; ++tile, ++seg) {
            const int count = min(left, w.steps - (tile == tile0 ? step0 : 0));
            const int h = tile / p.tiles_per_head;
            const int r0 = (tile - h * p.tiles_per_head) * (NT * kRows) + x * kRows + (warp & 3) * 32;
            const int r = r0 + lane;
            const bool busy = r0 < rows;  // uniform in the warp: some row is a query's
            // log2 per unit of score, with the query's power of two
            float scale = fabsf(a.scale_log2);
            load_query(x, row, r, rows, h, flip, scale);
            fence_async();
            tc_fence_before();  // the last segment's O is read
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar.q_full[x]));
            float m = -INFINITY, l = 0.0f;
            for (int t = 0; t < count; ++t, ++n) {
                if (!wait_warp(bar.s_full[x], (uint32_t)n & 1u)) return;
                tc_fence_after();
                auto done = [&](uint64_t &b) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&b));
                };
                if (busy)
                    step(s_at, o_at, scale, t > 0, n % kMaskSlots, m, l, [&]() { done(bar.p_half[x]); });
                else if (L::kHalves)
                    done(bar.p_half[x]);
                done(bar.p_full[x]);
            }
            if (!wait_warp(bar.o_full[x], seg & 1u)) return;
            tc_fence_after();
            if (busy) {
                const int64_t slot = ((int64_t)tile + blockIdx.x) * (NT * kRows) + x * kRows + row;
                float *po = p.part_o + (slot - lane) * D + lane * 8;  // 32 rows' eighths in turn
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tc_ld32(o, o_at + c);
                    tc_wait_ld(o);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float4 y = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                        if (MODE == 1) {
                            const float4 sv = __ldg(reinterpret_cast<const float4 *>(a.v_scale + (int64_t)h * D + c + i));
                            y = make_float4(y.x * sv.x, y.y * sv.y, y.z * sv.z, y.w * sv.w);
                        }
                        *reinterpret_cast<float4 *>(po + (c + i) / 8 * 256 + i % 8) = y;
                    }
                }
                p.part_m[slot] = m;
                p.part_l[slot] = l;
            }
            left -= count;
        }
    }

    // Query row r of head h into row `row` of tile x, in mode 1 times the channels' key
    // scales: fp16 after a power of two that brings the row's largest value to [1, 2)
    // and goes into `scale`.  Eleven bits hold a bf16 value whole (mode 1: round the
    // product eight times finer than bf16); below 2^-14 of the largest they thin out to
    // 2^-25 of it.
    __device__ __forceinline__ void load_query(int x, int row, int r, int rows, int h, bool flip,
                                               float &scale) const {
        const AttnArgs &a = p.own;
        const uint32_t dst = base + L::kQ + x * L::kTileBytes + (uint32_t)row * 128;
        const bool live = r < rows;
        const uint16_t *q = a.q;
        if (live) {
            const int b = r / a.group, j = r - b * a.group;
            q += (int64_t)b * a.q_seq_stride + (int64_t)(h * a.group + j) * a.q_head_stride;
        }
        const float *ks = a.k_scale + (MODE == 1 ? (int64_t)h * D : 0);
        auto value = [&](uint32_t wd, int d) {
            float2 y = make_float2(__uint_as_float(wd << 16), __uint_as_float(wd & 0xFFFF0000u));
            if (MODE == 1) {
                const float2 s = __ldg(reinterpret_cast<const float2 *>(ks + d));
                y = make_float2(y.x * s.x, y.y * s.y);
            }
            return y;
        };
        uint4 v[D / 8];  // the whole row in flight at once
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (live) v[i] = __ldg(reinterpret_cast<const uint4 *>(q) + i);
        }
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            const uint32_t wd[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = value(wd[e], 8 * i + 2 * e);
                top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
        }
        const int ex = power_of(top);
        const float turn = __uint_as_float(((uint32_t)(127 - ex) << 23) | (flip ? 0x80000000u : 0u));
        scale *= __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            uint32_t wd[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 y = value(wd[e], 8 * i + 2 * e);
                wd[e] = pack_fp16(y.x * turn, y.y * turn);
            }
            const uint32_t at = dst + (uint32_t)(i / 8) * (kRows * 128) + (uint32_t)(((i % 8) ^ (row & 7)) << 4);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(wd[0]), "r"(wd[1]), "r"(wd[2]),
                         "r"(wd[3])
                         : "memory");
        }
    }

    // Leaves out positions of the 32 from c on that are behind the end or in a bad block.
    __device__ __forceinline__ void mask(float (&s)[32], int c, int slot) const {
        const uint32_t wd = c < 64 ? bar.valid[slot].x : bar.valid[slot].y;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i % 16 >= (int)((wd >> (((c % 64) / 16 + i / 16) * 8)) & 0xFF)) s[i] = -INFINITY;
    }
    __device__ __forceinline__ static float max3(float a, float b, float c) {
        float r;
        asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
        return r;
    }
    // Largest of a group of 16.
    __device__ __forceinline__ static float top16(const float (&s)[32], int i0) {
        const float t0 = max3(s[i0], s[i0 + 1], s[i0 + 2]), t1 = max3(s[i0 + 3], s[i0 + 4], s[i0 + 5]);
        const float t2 = max3(s[i0 + 6], s[i0 + 7], s[i0 + 8]), t3 = max3(s[i0 + 9], s[i0 + 10], s[i0 + 11]);
        const float t4 = max3(s[i0 + 12], s[i0 + 13], s[i0 + 14]);
        return max3(max3(t0, t1, t2), max3(t3, t4, s[i0 + 15]), -INFINITY);
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
    // Weights of 32 positions from c on into P's columns, each group of 16 with its own
    // factor and shift; returns their sum.
    __device__ __forceinline__ void weights(const float (&s)[32], int c, const float *f, const float *g, uint32_t s_at,
                                            float2 (&sum)[2]) const {
        uint32_t o[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float2 y = __ffma2_rn(make_float2(s[i], s[i + 1]), make_float2(f[i / 16], f[i / 16]),
                                  make_float2(g[i / 16], g[i / 16]));
            y = make_float2(ex2(y.x), ex2(y.y));
            sum[i / 16] = i % 16 == 0 ? y : __fadd2_rn(sum[i / 16], y);
            o[i / 2] = pack_fp16(y.x, y.y);
        }
        tc_st16(s_at + c / 2, o);
    }

    // One step of a row: S -> P, the running maximum m and sum l.  A group's weights are
    // 2^(score + e - m), e the exponent taken out of its value scales, so that the product
    // with the tile's values is the weight times the value; m bounds score + e, lazily.
    // fp16 holds such weights (at most 2^15) eight times finer than bf16, and what falls
    // below 2^-21 of the largest to 2^-32 of it.
    template <typename Half>
    __device__ __forceinline__ void step(uint32_t s_at, uint32_t o_at, float scale, bool have_o, int slot,
                                         float &m, float &l, Half &&half) const {
        const bool whole = bar.valid[slot].x == 0x10101010u && bar.valid[slot].y == 0x10101010u;
        float s[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tc_ld32(s[q], s_at + 32 * q);
#pragma unroll
        for (int q = 0; q < 4; ++q) tc_wait_ld(s[q]);
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (!whole) mask(s[q], 32 * q, slot);
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
            if (have_o) {
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
            weights(s[q], 32 * q, f, g, s_at, sum);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float part = sum[i].x + sum[i].y;
                l = MODE == 1 ? l + part : fmaf(part, bar.v_inv[slot][2 * q + i], l);
            }
            if (L::kHalves && q == 1) {
                tc_wait_st();
                half();
            }
        }
        tc_wait_st();
    }
};

template <int MODE, int D, int NT>
__global__ void __launch_bounds__(Layout<MODE, D, NT>::kThreads, 1) prefix_kernel(const PrefixArgs p) {
    using L = Layout<MODE, D, NT>;
    extern __shared__ uint8_t dyn[];
    __shared__ Barriers bar;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    const int32_t given = __ldg(p.prefix_length);
    const bool choose = p.cuts > 1;
    PrefixWork w;
    uint32_t own = 0;
    if (choose)
        own = own_part(p);
    else
        w = prefix_work(p, given, p.cut[0]);
    if (warp == L::kMmaWarp) {
        if (lane == 0) {
            for (int i = 0; i < kStages; ++i) {
                mbar_init(smem_u32(&bar.k_full[i]), L::kDequantWarps);
                mbar_init(smem_u32(&bar.v_full[i]), L::kDequantWarps);
                mbar_init(smem_u32(&bar.k_free[i]), 1);
                mbar_init(smem_u32(&bar.v_free[i]), 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&bar.q_full[i]), 4);
                mbar_init(smem_u32(&bar.p_half[i]), 4);
                mbar_init(smem_u32(&bar.p_full[i]), 4);
                mbar_init(smem_u32(&bar.s_full[i]), 1);
                mbar_init(smem_u32(&bar.o_full[i]), 1);
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
    if (choose) {
        own = __reduce_add_sync(0xFFFFFFFFu, own);
        if (lane == 0) bar.own[warp] = own;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    if (choose) {
        own = 0;
#pragma unroll
        for (int i = 0; i < L::kThreads / 32; ++i) own += bar.own[i];
        const int best = best_cut(p, own);
        if (blockIdx.x == 0 && threadIdx.x == 0) *p.chosen = best;
        w = prefix_work(p, given, p.cut[best]);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (given < 0) report(p.own.dev_error, KVC8_DEV_BAD_LENGTH);
        if (given > w.len && given >= 0) report(p.own.dev_error, KVC8_DEV_POS_BEYOND_TABLE);
    }
    const uint32_t group = blockIdx.x / w.n, share = blockIdx.x - group * w.n;  // group: the tile, or 0
    const uint32_t groups = w.per_tile > 0 ? (uint32_t)(p.tiles_per_head * p.own.g.kv_heads) : 1u;
    const uint32_t first = w.first_of(share), total = group < groups ? w.first_of(share + 1) - first : 0u;
    if (total > 0) {
        const uint32_t base = (smem_u32(dyn) + 1023u) & ~1023u;
        const uint32_t tile_in = first / (uint32_t)w.steps;
        const Prefix<MODE, D, NT> k{p,
                                    bar,
                                    base,
                                    w,
                                    (int)total,
                                    (int)(group + tile_in),
                                    (int)(first - tile_in * (uint32_t)w.steps),
                                    lane};
        if (warp >= L::kMmaWarp) {
            reg_give<L::kMmaRegs>();
            if (warp == L::kMmaWarp) k.products(tmem);
        } else if (warp >= L::kSoftmaxWarps) {
            reg_give<L::kDequantRegs>();
            k.dequantise(warp - L::kSoftmaxWarps);
        } else {
            reg_take<L::kSoftmaxRegs>();
            k.softmax(warp, tmem);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    }
    if (warp == L::kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)L::kTmemCols)
                     : "memory");
}

// Joins a query row's partials: the prefix's segments and its own positions' splits.
// D / 8 lanes per query row, eight channels each, four partials' loads in flight (eight, with
// half as many warps: 49.3 us instead of 47.2 for 8192 positions x 64 sequences); where
// rows are few and partials many, `share` warps take a part of them each.
template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) merge_kernel(const PrefixArgs p, int rows_per_tile, int share) {
    constexpr int kLanes = D / 8, kWarpRows = 32 / kLanes;
    __shared__ float s_acc[kMergeThreads][9], s_top[kMergeThreads], s_sum[kMergeThreads];
    const AttnArgs &a = p.own;
    const int H = a.g.kv_heads, G = a.group, B = a.g.num_seqs;
    const int lane = threadIdx.x & 31, gl = lane % kLanes;
    // sequences * query heads < 2^30; rows past the end redo the last one and do not store
    const int mine = (threadIdx.x >> 5) % share;  // which of the warps that share these rows
    const int at = (blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5)) / share * kWarpRows + lane / kLanes;
    const int row = min(at, B * H * G - 1);
    const int b = row / (H * G), hj = row - b * (H * G), h = hj / G, j = hj - h * G;
    const int32_t given = __ldg(p.prefix_length);
    const int r = b * G + j, tile = h * p.tiles_per_head + r / rows_per_tile;
    int parts = 0;
    int64_t slot = 0;  // row of the first segment's partial; segments are a tile's rows apart
    auto locate = [&](const PrefixCut &cut) {
        const PrefixWork w = prefix_work(p, given, cut);
        if (w.steps > 0) {
            const uint32_t first = w.per_tile > 0 ? 0u : (uint32_t)(tile * w.steps);
            const int before = tile * w.per_tile;
            const int c0 = before + (int)w.cta_of(first), c1 = before + (int)w.cta_of(first + w.steps - 1);
            parts = c1 - c0 + 1;
            slot = ((int64_t)tile + c0) * rows_per_tile + r % rows_per_tile;
        }
    };
    if (p.cuts == 1) locate(p.cut[0]);
    pdl_wait_prior_grid();
    const int best = p.cuts > 1 ? *p.chosen : 0;  // used after the own positions' partials
    float M = -INFINITY, L = 0.0f, acc[8];  // L: this lane's share
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
    // all partials, `stride` rows apart, of which this warp takes every share-th; o points
    // to this lane's channels of the first.  The rows of a warp have their own counts: all
    // stay for the longest.
    auto join = [&](const float *pm, const float *pl, const float *o, int64_t stride, int all) {
        const int count = (all - mine + share - 1) / share;  // 0 where all <= mine
        pm += mine * stride, pl += mine * stride, o += mine * stride * D;
        stride *= share;
        const int rounds = (__reduce_max_sync(0xFFFFFFFFu, count) + kLanes - 1) / kLanes;
        for (int i0 = 0; i0 < rounds * kLanes; i0 += kLanes) {
            float4 v[4][2];  // four partials, requested before their weights are known
            auto request = [&](int k0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v[k][0] = v[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (i0 + k0 + k < count) {
                        const float4 *src = reinterpret_cast<const float4 *>(o + (i0 + k0 + k) * stride * D);
                        v[k][0] = src[0];
                        v[k][1] = src[1];
                    }
                }
            };
            request(0);
            const bool in = i0 + gl < count;
            const float m = in ? pm[(i0 + gl) * stride] : -INFINITY, l = in ? pl[(i0 + gl) * stride] : 0.0f;
            float n = m;
#pragma unroll
            for (int s = kLanes / 2; s > 0; s >>= 1) n = fmaxf(n, __shfl_xor_sync(0xFFFFFFFFu, n, s));
            n = fmaxf(M, n);
            // no position yet: nothing is added
            const float g = M == -INFINITY ? 0.0f : exp2f(M - n), f = m == -INFINITY ? 0.0f : exp2f(m - n);
            M = n;
            L = L * g + l * f;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= g;
            const int most = __reduce_max_sync(0xFFFFFFFFu, min(kLanes, count - i0));
            for (int k0 = 0; k0 < most; k0 += 4) {
                if (k0 > 0) request(k0);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float fk = __shfl_sync(0xFFFFFFFFu, f, k0 + k, kLanes);
                    acc[0] += fk * v[k][0].x, acc[1] += fk * v[k][0].y, acc[2] += fk * v[k][0].z, acc[3] += fk * v[k][0].w;
                    acc[4] += fk * v[k][1].x, acc[5] += fk * v[k][1].y, acc[6] += fk * v[k][1].z, acc[7] += fk * v[k][1].w;
                }
            }
        }
    };
    const int64_t len = min((int64_t)ld_nc_s32(a.context_lengths + b), (int64_t)a.g.max_blocks_per_seq * a.g.block_size);
    const int own = len > 0 ? (int)((len + kAttnChunk - 1) / kAttnChunk) : 0;  // splits of its own positions
    const int64_t own0 = ((int64_t)b * p.own_splits * H + h) * G + j;
    join(a.part_m + own0, a.part_l + own0, a.part_o + own0 * D + gl * 8, (int64_t)H * G, own);
    if (p.cuts > 1) locate(p.cut[best]);
    join(p.part_m + slot, p.part_l + slot, p.part_o + slot / 32 * 32 * D + gl * 256 + slot % 32 * 8, rows_per_tile, parts);
    if (share > 1) {  // the same in every warp
        s_top[threadIdx.x] = M;
        s_sum[threadIdx.x] = L;
#pragma unroll
        for (int e = 0; e < 8; ++e) s_acc[threadIdx.x][e] = acc[e];
        __syncthreads();
        if (mine == 0) {
            for (int k = 1; k < share; ++k) {
                const int o = threadIdx.x + 32 * k;
                const float n = fmaxf(M, s_top[o]);
                const float g = M == -INFINITY ? 0.0f : exp2f(M - n), f = s_top[o] == -INFINITY ? 0.0f : exp2f(s_top[o] - n);
                M = n;
                L = L * g + s_sum[o] * f;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = acc[e] * g + s_acc[o][e] * f;
            }
        }
    }
#pragma unroll
    for (int s = kLanes / 2; s > 0; s >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, s);
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    if (at != row || mine != 0) return;
    uint16_t *dst = a.out + (int64_t)b * a.out_seq_stride + (int64_t)hj * a.out_head_stride + gl * 8;
    uint32_t y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
    } else {  // the output may lie on any element
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dst[2 * e] = (uint16_t)(y[e] & 0xFFFFu);
            dst[2 * e + 1] = (uint16_t)(y[e] >> 16);
        }
    }
}

// Tiles of 128 query rows that a CTA holds: two, which share a step's dequantised rows, when
// there are more rows than one holds (whole calls, 1024 rows x 32768 positions: 171 us, with
// one tile 255; 161 rows x 10007: 26.4 and 26.7); else one, whose four softmax warps leave
// eight to dequantise (128 rows x 60000 positions, mode 0: 69.5 us, with two tiles 85.4; 32
// rows x 32768, mode 1: 41.1 and 45.1).
int tiles_per_cta(int64_t rows) { return rows > kRows ? 2 : 1; }

struct Space {
    size_t own, o, m, chosen, bytes;  // own partials first, then the prefix's O, m and l
};

Space space(const kvc8_geom &g, int group) {
    const int64_t rows = (int64_t)g.num_seqs * group;
    const int64_t per = (int64_t)tiles_per_cta(rows) * kRows;
    const size_t slots = (size_t)((rows + per - 1) / per * g.kv_heads + kMaxCtas) * (size_t)per;
    Space s;
    s.own = own_workspace_bytes(g, group);
    s.o = s.own;
    s.m = s.o + align_up(slots * g.head_dim * sizeof(float), kAlign);
    s.chosen = s.m + 2 * align_up(slots * sizeof(float), kAlign);
    s.bytes = s.chosen + kAlign;
    return s;
}

// The cuts to choose from: CTAs that stay within a tile, as many as there is room for and
// down to about half as many, and CTAs that share all work.  None has more CTAs than its
// longest share needs.  Returns the most CTAs of one.  The host knows the tables' room and not
// the lengths in them, so a cut's cost is that of a prefix which fills its table.  Behind a
// shorter one own positions seem to fit beside it more often than they do, and the prefix gets
// more SMs than is best (same lengths, table exact -> twice -> eight times as long: 8192 positions x 64
// sequences 45.3 -> 51.7 -> 56.3 us, 10007 x 23 24.9 -> 26.8 -> 35.1, 32768 x 256 172 -> 182 ->
// 189); likewise with cuts == 1, from the room for own positions.  Results do not depend on it.
int prefix_cuts(PrefixArgs &p, int64_t tiles, int64_t steps) {
    const int64_t units = tiles * steps, sms = p.sms;
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    constexpr int kInTile = 5;
    int most = 0;
    p.cuts = 0;
    for (int i = 0; i < kPrefixCuts; ++i) {
        const int64_t room = sms / tiles;
        const int64_t each = i < kInTile ? room - i * up(room, 2 * kInTile) : 0;
        PrefixCut c;
        int64_t longest;
        if (each > 0) {
            longest = up(steps, each);
            c.per_tile = (int32_t)up(steps, longest);
            c.ctas = (int32_t)(tiles * c.per_tile);
        } else {
            longest = up(units, sms - sms * (i < kInTile ? i : i - kInTile) / 8);
            c.per_tile = 0;
            c.ctas = (int32_t)up(units, longest);
            longest += kTileChange;
        }
        c.time = (float)(sms * (kStart + longest));
        c.beside = (float)((sms - c.ctas) * (kStart + longest));
        bool better = true;
        for (int j = 0; j < p.cuts; ++j) better = better && (c.time < p.cut[j].time || c.ctas < p.cut[j].ctas);
        if (!better) continue;
        p.cut[p.cuts++] = c;
        if (c.ctas > most) most = c.ctas;
    }
    // As many own positions as there is room for fit beside the quickest: nothing to choose.
    // (Reading the lengths and choosing takes 1.5 us.)
    int quick = 0;
    for (int i = 1; i < p.cuts; ++i)
        if (p.cut[i].time < p.cut[quick].time) quick = i;
    const int64_t own_most = (int64_t)p.own.g.num_seqs * ((p.own.g.max_blocks_per_seq * (int64_t)p.own.g.block_size + 63) / 64);
    if ((float)own_most * p.own_weight <= p.cut[quick].beside) {
        p.cut[0] = p.cut[quick];
        p.cuts = 1;
        most = p.cut[0].ctas;
    }
    return most;
}

template <int MODE, int D, int NT>
cudaError_t launch_variant(PrefixArgs p, cudaStream_t stream) {
    using L = Layout<MODE, D, NT>;
    auto kern = prefix_kernel<MODE, D, NT>;
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
    p.rows = p.own.g.num_seqs * p.own.group;
    p.tiles_per_head = (p.rows + NT * kRows - 1) / (NT * kRows);
    const int64_t steps = ((int64_t)p.max_prefix_blocks * p.own.g.block_size + kCols - 1) / kCols;
    const int64_t tiles = (int64_t)p.tiles_per_head * p.own.g.kv_heads;
    p.sms = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    // own positions of a kv head that an SM passes in a step's time
    constexpr float kOwnPerStep = NT == 1 ? 130.0f : 220.0f;
    p.own_weight = 64.0f * (float)p.own.g.kv_heads / kOwnPerStep;
    p.own_least = (float)(p.sms * kOwnLeast);
    const int grid = prefix_cuts(p, tiles, steps);
    kern<<<(unsigned)grid, L::kThreads, (size_t)L::kBytes, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_own(p, stream);
    if (e != cudaSuccess) return e;
    // Partials a row has of the prefix, about: CTAs per tile.  Up to six a warp (of 644 rows
    // with 38 partials each the merge took 32 us with one warp per two rows).
    int share = 1;
    while (share < kMergeThreads / 32 && grid > 6 * share * tiles) share *= 2;
    const int64_t all = (int64_t)p.rows * p.own.g.kv_heads, per = kMergeThreads / (D / 8) / share;
    return launch_dependent(merge_kernel<D>, dim3((unsigned)((all + per - 1) / per)), kMergeThreads, (size_t)0, stream, p,
                            NT * kRows, share);
}

template <int MODE>
cudaError_t launch_mode(const PrefixArgs &p, cudaStream_t stream) {
    const bool two = tiles_per_cta((int64_t)p.own.g.num_seqs * p.own.group) == 2;
    if (p.own.g.head_dim == 64)
        return two ? launch_variant<MODE, 64, 2>(p, stream) : launch_variant<MODE, 64, 1>(p, stream);
    return two ? launch_variant<MODE, 128, 2>(p, stream) : launch_variant<MODE, 128, 1>(p, stream);
}

}  // namespace

size_t shared_prefix_workspace_bytes(const kvc8_geom &g, int group) { return space(g, group).bytes; }

cudaError_t launch_shared_prefix(PrefixArgs p, void *workspace, cudaStream_t stream) {
    const Space s = space(p.own.g, p.own.group);
    char *ws = static_cast<char *>(workspace);
    p.part_o = reinterpret_cast<float *>(ws + s.o);
    p.part_m = reinterpret_cast<float *>(ws + s.m);
    p.part_l = reinterpret_cast<float *>(ws + s.m + (s.chosen - s.m) / 2);
    p.chosen = reinterpret_cast<int32_t *>(ws + s.chosen);
    place_own(p, workspace);
    if (p.own.g.quant_mode == 0) return launch_mode<0>(p, stream);
    if (p.own.g.quant_mode == 1) return launch_mode<1>(p, stream);
    return launch_mode<2>(p, stream);
}

}  // namespace kvc8
