// kvc8_rope.cu -- per-head RMS norm and rotary rotation of new queries and
// keys, the keys (and the values) on their way into the int8 or bf16 pages.
//
// With x a head's row of D channels, phi_i = pos * f_i and (a, b) the channels of
// pair i:
//   y = x / sqrt(mean(x^2) + eps) * w                (where a weight is given)
//   (y_a, y_b) <- m (y_a cos phi - y_b sin phi, y_b cos phi + y_a sin phi)
// A query row is rounded to bf16; a key row is rounded to bf16 or quantised,
//   q = clamp(rne(y / s), -127, 127), s = max|y| / 127 or a static scale;
// a value row takes the same path without norm and rotation.
//
// A frequency is a fraction of a turn in 64-bit fixed point, so pos * f mod 2^64
// is the exact phase; its top 32 bits as a signed fraction of half a turn go
// to sincospi.
//
// Work: L lanes hold a row (D / 16 rounded up to a power of two), 16 channels
// each as two pieces of eight, so a warp takes 32 / L rows of one kind (queries,
// keys or values) of a token at a time.  A lane's two pieces hold whole pairs --
// channels [8c, 8c+8) and [R/2 + 8c, +8) in the half layout, any eight neighbours in
// the interleaved one -- so nothing is exchanged but the row sums and maxima.  A unit of
// work is a token, or a part of its row sets where there are fewer tokens than
// warps.  The warp finds its token's slot, computes the R/2 sines and cosines once
// (a lane R/64 of them, handed over in shared memory), folds the norm's weights into
// them, and then spends on a row little more than unpacking, the sum of squares, four
// multiply-adds a pair and packing.  The rows come through a ring in shared memory,
// three sets ahead.
//
// Codes without dividing: with r within 2^-23 of 1/s, every value fl(y/s) can take lies
// between y r (1 - 2^-21) and y r (1 + 2^-21).  Where both ends round to the same integer,
// so does the quotient; else (a value within 2^-20 of a half-integer, mostly an exact tie of
// a value row, 2 in 10^4) the lane divides.
//
// Measured (GB300, 32 query and 8 kv heads of 128): rows alone, 410 MB in 65 us (0.93 of the
// copy rate); into bf16 pages, 480 MB in 77 us; into int8 pages, 829 MB with dynamic scales in
// 147 us (0.83), 827 MB with block scales in 144 (0.84) and with channel scales in 179 (0.68).
// HBM bounds all but the last, which computes a reciprocal and a limit for every channel of
// every row: with 24 query heads, 161 MB in 39 us (0.61), issue slots 49% and DRAM 39% busy,
// so what its 20 warps per SM wait for bounds it.  256 tokens (64 query heads, 10 MB): 9.8 us,
// a launch's latency.  Five CTAs of four warps per SM (96 registers) were faster than
// four or six, although the int8 rows then spill (bytes a thread stored / loaded: dynamic and
// block scales 40 / 40, channel scales 112 / 160; rows and bf16 pages nothing).
#include "kvc8_codes.cuh"
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kRing = 4;  // row sets per warp in shared memory, one fewer in flight
constexpr int kMaxPairs = 128;

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// Where a token goes.
struct Slot {
    int64_t row;  // cache row of (block, head 0, slot); -1: the token is skipped
    int32_t blk;
    int32_t pos;  // its rotary position: as given, or the slot's as an unsigned number
};

// One token per lane: the warp's next 32 tokens are looked up at once.
template <int SINK>
__device__ __forceinline__ Slot find_slot(const RopeArgs &a, int64_t t, bool report_it) {
    Slot s = {0, 0, 0};
    if (SINK != kSinkRows) {
        const int B = a.g.num_seqs, bs = a.g.block_size, MB = a.g.max_blocks_per_seq;
        int64_t first = t, next = t + 1;
        int b = (int)t;
        if (a.cu_q_lens != nullptr) {
            // the last sequence whose first new token is at or before t
            b = 0;
            for (int step = 1 << (31 - __clz(max(B - 1, 1))); step > 0; step >>= 1)
                if (b + step < B && (int64_t)ld_nc_s32(a.cu_q_lens + b + step) <= t) b += step;
            first = ld_nc_s32(a.cu_q_lens + b);
            next = ld_nc_s32(a.cu_q_lens + b + 1);
        }
        const int64_t ctx = ld_nc_s32(a.context_kv_lens + b), pos = ctx + (t - first);
        int32_t err = 0;
        if (!(first <= t && t < next) || ctx < 0) {
            err = KVC8_DEV_BAD_LENGTH;
        } else {
            // 0 <= pos < 2^32: a 32-bit division
            const int64_t lb = (int64_t)((uint32_t)pos / (uint32_t)bs);
            if (lb >= MB) {
                err = KVC8_DEV_POS_BEYOND_TABLE;
            } else {
                s.blk = ld_nc_s32(a.block_table + (int64_t)b * MB + lb);
                if (s.blk < 0 || s.blk >= a.g.num_blocks) err = KVC8_DEV_BAD_BLOCK_ID;
                s.row = (int64_t)s.blk * a.g.kv_heads * bs + (pos - lb * bs);
                s.pos = (int32_t)(uint32_t)pos;
            }
        }
        if (err != 0) {
            if (report_it) report(a.dev_error, err);
            s.row = -1;
            return s;
        }
    }
    if (a.positions != nullptr) s.pos = ld_nc_s32(a.positions + t);
    return s;
}

// cp.async: 16 bytes global -> shared, waited for by the thread that asked, which alone
// reads them.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 ld_shared16(uint32_t p) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}

constexpr float kMagic = 12582912.0f;            // 1.5 * 2^23: adding it rounds to an integer
constexpr float kRecipLo = 0.99999952316284180f;  // 1 - 2^-21
constexpr float kRecipHi = 1.00000047683715820f;  // 1 + 2^-21

// The definition: one division, round half to even, clamp; 0 when s == 0.
__device__ __noinline__ uint32_t codes_divide(float2 y0, float2 y1, float4 s) {
    auto one = [](float a, float b) {
        const int q = b == 0.0f ? 0 : __float2int_rn(__fdiv_rn(a, b));
        return (uint32_t)min(127, max(-127, q)) & 0xFFu;
    };
    return one(y0.x, s.x) | one(y0.y, s.y) << 8 | one(y1.x, s.z) << 16 | one(y1.y, s.w) << 24;
}

// |x| limited to b, with x's sign.
__device__ __forceinline__ float limit(float x, float b) {
    float r;
    asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(b));
    return r;
}

__device__ __forceinline__ bool recip_ok(float s) { return s >= 0x1p-120f && s <= 0x1p+120f; }

// 1/s within 2^-23 of itself (the hardware's approximation), 0 where s has none.
__device__ __forceinline__ float recip(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return recip_ok(s) ? r : 0.0f;
}

// fl(m / 127) without dividing, by Markstein's correction of a quotient (IBM Journal of
// Research and Development 34, 1990): with c = fl(1/127) and q = fl(m c), the remainder
// m - 127 q is exact in a fused multiply-add, and fl(q + remainder c) is the rounded
// quotient.  Small m, whose remainder might not be normal, and an infinite m divide.
__device__ __forceinline__ float over_127(float m) {
    constexpr float c = 1.0f / 127.0f;
    if (!(m >= 0x1p-90f && m < INFINITY)) return __fdiv_rn(m, 127.0f);
    const float q = __fmul_rn(m, c);
    return __fmaf_rn(__fmaf_rn(-127.0f, q, m), c, q);
}

// Four codes of y for reciprocals r of their scales s; LIMIT: |y / s| may pass 127 and is
// cut at fl(127 s), whose code is 127.  `apart` becomes nonzero where the bracket's ends
// disagree.
template <bool LIMIT>
__device__ __forceinline__ uint32_t codes4(float2 y0, float2 y1, float4 s, float4 r, float2 &apart) {
    if (LIMIT) {
        y0 = make_float2(limit(y0.x, __fmul_rn(127.0f, s.x)), limit(y0.y, __fmul_rn(127.0f, s.y)));
        y1 = make_float2(limit(y1.x, __fmul_rn(127.0f, s.z)), limit(y1.y, __fmul_rn(127.0f, s.w)));
    }
    const float2 lo = make_float2(kRecipLo, kRecipLo), hi = make_float2(kRecipHi, kRecipHi);
    const float2 m2 = make_float2(kMagic, kMagic), n1 = make_float2(-1.0f, -1.0f);
    const float2 ra = make_float2(r.x, r.y), rb = make_float2(r.z, r.w);
    const float2 la = __ffma2_rn(y0, __fmul2_rn(ra, lo), m2), ha = __ffma2_rn(y0, __fmul2_rn(ra, hi), m2);
    const float2 lb = __ffma2_rn(y1, __fmul2_rn(rb, lo), m2), hb = __ffma2_rn(y1, __fmul2_rn(rb, hi), m2);
    const float2 da = __ffma2_rn(la, n1, ha), db = __ffma2_rn(lb, n1, hb);  // 0 where the ends agree
    apart = __ffma2_rn(da, da, apart);
    apart = __ffma2_rn(db, db, apart);
    return __byte_perm(__byte_perm(__float_as_uint(la.x), __float_as_uint(la.y), 0x0040),
                       __byte_perm(__float_as_uint(lb.x), __float_as_uint(lb.y), 0x0040), 0x5410);
}

// L lanes per row, 32 / L rows of a set.
template <int SINK, int L>
__global__ void __launch_bounds__(kRopeWarps * 32, 5) rope_kernel(const RopeArgs a, int parts, int per) {
    constexpr int RW = 32 / L;
    constexpr bool kPages = SINK != kSinkRows;
    __shared__ __align__(16) float turn_s[kRopeWarps][2][kMaxPairs];  // m cos, m sin
    // the two pieces of each lane, apart so that an access covers whole rows of banks
    __shared__ uint4 ring_s[kRopeWarps][kRing][2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int H = a.g.kv_heads, D = a.g.head_dim, R = a.rotary_dim, bs = a.g.block_size;
    const int sq = (a.q_heads + RW - 1) / RW, sk = (H + RW - 1) / RW;
    const int sets = sq + sk + (kPages ? sk : 0);  // row sets of a token: queries, keys, values
    const int rl = lane / L, c = lane % L;
    const bool on_c = c < D / 16;
    // This lane's channels, two pieces of eight, neighbouring lanes' side by side so that
    // every access covers whole sectors.  Half layout: lanes c < R/16 take pairs 8c to
    // 8c + 7, the others pass channels behind R; interleaved: the halves of the row.
    const bool half = a.interleaved == 0, turns = half && c < R / 16;
    const int pass = R + 8 * (c - R / 16);
    const int d0 = !half || turns ? 8 * c : pass;
    const int d1 = !half ? D / 2 + 8 * c : turns ? R / 2 + 8 * c : pass + (D - R) / 2;
    const int v0 = 8 * c, v1 = D / 2 + 8 * c;  // of a value row
    const float inv_d = 1.0f / (float)D;
    float *cos_s = turn_s[warp][0], *sin_s = turn_s[warp][1];

    // Units of work (token, part of its row sets): this warp's are u0, u0 + stride, ...
    const int64_t units = a.num_tokens * parts, stride = (int64_t)gridDim.x * kRopeWarps;
    const int64_t u0 = (int64_t)blockIdx.x * kRopeWarps + warp;
    auto token_of = [&](int64_t u) { return parts == 1 ? u : u / parts; };

    // The row sets to come, requested kRing - 1 ahead of the one being worked on, over the
    // ends of kinds, tokens and units alike.  A lane's copies go to its own places, which it
    // alone reads.
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(&ring_s[warp][0][0][lane]);
    const uint16_t *p0 = nullptr;
    int64_t p_step = 0, pu = u0;
    int p_gap = 0;                    // from the first piece to the second
    int p_left = 0;                   // heads of the kind from this lane's row on
    int p_set = 0, p_end = 0;         // the next set to request, the end of its unit
    uint32_t p_slot = 0, r_slot = 0;  // ring places to fill and to read (bytes)
    constexpr uint32_t kSet = 2 * 32 * 16;
    auto begin = [&](int64_t t, int set) {  // the set may lie inside a kind
        const bool q = set < sq, v = set >= sq + sk;
        const int h = (set - (q ? 0 : v ? sq + sk : sq)) * RW + rl;
        const int64_t hs = q ? a.q_head_stride : a.x_head_stride;
        const uint16_t *row = q ? a.q + t * a.q_tok_stride : (v ? a.v : a.k) + t * a.x_tok_stride;
        p0 = row + h * hs + (v ? v0 : d0);
        p_gap = v ? v1 - v0 : d1 - d0;
        p_step = RW * hs;
        p_left = (q ? a.q_heads : H) - h;
    };
    auto pull = [&]() {
        if (pu < units) {
            if (on_c && p_left > 0) {
                cp_async16(ring + p_slot, p0);
                cp_async16(ring + p_slot + 32 * 16, p0 + p_gap);
            }
            p0 += p_step;
            p_left -= RW;
            if (++p_set == p_end) {  // on to the next unit
                pu += stride;
                if (pu < units) {
                    const int64_t tn = token_of(pu);
                    p_set = (int)(pu - tn * parts) * per;
                    p_end = min(sets, p_set + per);
                    begin(tn, p_set);
                }
            } else if (p_set == sq || p_set == sq + sk) {
                begin(token_of(pu), p_set);
            }
        }
        cp_async_commit();
        p_slot = (p_slot + kSet) & (kRing * kSet - 1);
    };
    uint4 x0, x1;
    auto take = [&]() {
        cp_async_wait<kRing - 2>();
        x0 = ld_shared16(ring + r_slot);
        x1 = ld_shared16(ring + r_slot + 32 * 16);
        r_slot = (r_slot + kSet) & (kRing * kSet - 1);
        pull();
    };

    if (u0 >= units) return;
    if (!on_c) {  // no copy lands here: zeros for the row sums and maxima
#pragma unroll
        for (int i = 0; i < kRing; ++i) ring_s[warp][i][0][lane] = ring_s[warp][i][1][lane] = make_uint4(0u, 0u, 0u, 0u);
    }
    p_set = (int)(u0 - token_of(u0) * parts) * per;
    p_end = min(sets, p_set + per);
    begin(token_of(u0), p_set);
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) pull();
    Slot ahead = {0, 0, 0};
    int turn = 0;
    for (int64_t u = u0; u < units; u += stride, ++turn) {
        if ((turn & 31) == 0) {
            const int64_t mine = u + lane * stride;
            if (mine < units) {
                const int64_t tm = token_of(mine);
                ahead = find_slot<SINK>(a, tm, mine == tm * parts);
            }
        }
        Slot slot;
        slot.row = __shfl_sync(0xFFFFFFFFu, ahead.row, turn & 31);
        slot.blk = __shfl_sync(0xFFFFFFFFu, ahead.blk, turn & 31);
        slot.pos = __shfl_sync(0xFFFFFFFFu, ahead.pos, turn & 31);
        const int64_t t = token_of(u);
        const int s0 = (int)(u - t * parts) * per, s1 = min(sets, s0 + per);
        if (kPages && slot.row < 0) {  // uniform in the warp: the token is skipped
            for (int set = s0; set < s1; ++set) take();
            continue;
        }
        if (s0 < sq + sk) {
            __syncwarp();  // the last token's are used up
            const int64_t pos = a.positions != nullptr ? (int64_t)slot.pos : (int64_t)(uint32_t)slot.pos;
            for (int i = lane; i < R / 2; i += 32) {
                const uint64_t phase = (uint64_t)pos * __ldg(a.freqs + i);
                float s, co;
                sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &co);
                cos_s[i] = co * a.factor;
                sin_s[i] = s * a.factor;
            }
            __syncwarp();
        }

        // Queries and keys: row sets [lo, hi) of one kind.  The rotation with the norm's
        // weights folded in, per channel: out = x * own + partner * other.
        auto rotate_sets = [&](int lo, int hi, int first, const uint16_t *w, auto &&sink) {
            if (lo >= hi) return;
            float2 own[8], other[8];
            {
                float2 wt[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) wt[i] = make_float2(1.0f, 1.0f);
                if (w != nullptr && on_c) {
                    const uint4 w0 = __ldg(reinterpret_cast<const uint4 *>(w + d0));
                    const uint4 w1 = __ldg(reinterpret_cast<const uint4 *>(w + d1));
                    const uint32_t wd[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) wt[i] = make_float2(bf16_lo(wd[i]), bf16_hi(wd[i]));
                }
                float co[8], si[8];  // of this lane's pairs, four to a piece if interleaved
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const int pair = half ? 8 * c + i : (i ? d1 : d0) / 2;
                    const bool in = on_c && (half ? turns : (i ? d1 : d0) < R);
                    const float4 c4 = in ? *reinterpret_cast<const float4 *>(cos_s + pair) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
                    const float4 s4 = in ? *reinterpret_cast<const float4 *>(sin_s + pair) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    co[i] = c4.x, co[i + 1] = c4.y, co[i + 2] = c4.z, co[i + 3] = c4.w;
                    si[i] = s4.x, si[i + 1] = s4.y, si[i + 2] = s4.z, si[i + 3] = s4.w;
                }
                if (half) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 c2 = make_float2(co[2 * i], co[2 * i + 1]), s2 = make_float2(si[2 * i], si[2 * i + 1]);
                        own[i] = __fmul2_rn(wt[i], c2);
                        own[4 + i] = __fmul2_rn(wt[4 + i], c2);
                        other[i] = __fmul2_rn(wt[4 + i], make_float2(-s2.x, -s2.y));
                        other[4 + i] = __fmul2_rn(wt[i], s2);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        own[i] = make_float2(wt[i].x * co[i], wt[i].y * co[i]);
                        other[i] = make_float2(-wt[i].y * si[i], wt[i].x * si[i]);
                    }
                }
            }
            for (int set = lo; set < hi; ++set) {
                float2 v[8];
                take();
                {
                    const uint32_t wd[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = make_float2(bf16_lo(wd[i]), bf16_hi(wd[i]));
                }
                if (w != nullptr) {
                    float2 sa = __fmul2_rn(v[0], v[0]), sb = __fmul2_rn(v[1], v[1]);
#pragma unroll
                    for (int i = 2; i < 8; i += 2) {
                        sa = __ffma2_rn(v[i], v[i], sa);
                        sb = __ffma2_rn(v[i + 1], v[i + 1], sb);
                    }
                    sa = __fadd2_rn(sa, sb);
                    float sum = sa.x + sa.y;
#pragma unroll
                    for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    const float inv = rsqrtf(fmaf(sum, inv_d, a.eps));
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __fmul2_rn(v[i], make_float2(inv, inv));
                }
                float2 y[8];
                if (half) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[i] = __ffma2_rn(v[i], own[i], __fmul2_rn(v[4 + i], other[i]));
                        y[4 + i] = __ffma2_rn(v[4 + i], own[4 + i], __fmul2_rn(v[i], other[4 + i]));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        y[i] = __ffma2_rn(v[i], own[i], __fmul2_rn(make_float2(v[i].y, v[i].x), other[i]));
                }
                sink((set - first) * RW + rl, y);
            }
        };
        auto pack_row = [&](uint16_t *dst, const float2 (&y)[8]) {
            *reinterpret_cast<uint4 *>(dst + d0) = make_uint4(pack_bf16(y[0].x, y[0].y), pack_bf16(y[1].x, y[1].y),
                                                              pack_bf16(y[2].x, y[2].y), pack_bf16(y[3].x, y[3].y));
            *reinterpret_cast<uint4 *>(dst + d1) = make_uint4(pack_bf16(y[4].x, y[4].y), pack_bf16(y[5].x, y[5].y),
                                                              pack_bf16(y[6].x, y[6].y), pack_bf16(y[7].x, y[7].y));
        };
        // A row of 16 values a lane into the int8 pages: pieces at channels o0 and o1.
        auto quantise_row = [&](int h, int8_t *cache, float *scl, const float2 (&y)[8], int o0, int o1) {
            const bool on = on_c && h < H;
            const int64_t row = slot.row + (int64_t)h * bs;
            float s_row = 0.0f;
            if (SINK == kSinkDynamic) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(y[i].x), fabsf(y[i].y)));
#pragma unroll
                for (int o = 1; o < L; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                s_row = over_127(m);
                if (on && c == 0) scl[row] = s_row;
            } else if (SINK == kSinkBlock && on) {
                s_row = ld_nc_f32(scl + (int64_t)slot.blk * H + h);
            }
            if (!on) return;
            uint32_t o[4];
            float2 apart = make_float2(0.0f, 0.0f);
            float least = 1.0f;  // 0: some scale has no reciprocal
            if (SINK == kSinkChannel) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float4 s = __ldg(reinterpret_cast<const float4 *>(scl + h * D + (q < 2 ? o0 : o1) + 4 * (q & 1)));
                    const float4 r = make_float4(recip(s.x), recip(s.y), recip(s.z), recip(s.w));
                    least = fminf(fminf(fminf(r.x, r.y), fminf(r.z, r.w)), least);
                    o[q] = codes4<true>(y[2 * q], y[2 * q + 1], s, r, apart);
                }
            } else {
                const float r = recip(s_row);
                least = r;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    o[q] = codes4<SINK != kSinkDynamic>(y[2 * q], y[2 * q + 1], make_float4(s_row, s_row, s_row, s_row),
                                                        make_float4(r, r, r, r), apart);
            }
            if (apart.x + apart.y != 0.0f || least == 0.0f) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float4 s = make_float4(s_row, s_row, s_row, s_row);
                    if (SINK == kSinkChannel)
                        s = __ldg(reinterpret_cast<const float4 *>(scl + h * D + (q < 2 ? o0 : o1) + 4 * (q & 1)));
                    o[q] = codes_divide(y[2 * q], y[2 * q + 1], s);
                }
            }
            int8_t *dst = cache + row * D;
            st_8(dst + o0, o[0], o[1]);
            st_8(dst + o1, o[2], o[3]);
        };

        rotate_sets(s0, min(s1, sq), 0, a.q_weight, [&](int h, const float2 (&y)[8]) {
            if (on_c && h < a.q_heads)
                pack_row(a.q_out + t * a.qo_tok_stride + (int64_t)h * a.qo_head_stride, y);
        });
        rotate_sets(max(s0, sq), min(s1, sq + sk), sq, a.k_weight, [&](int h, const float2 (&y)[8]) {
            if (SINK == kSinkRows) {
                if (on_c && h < H) pack_row(a.k_out + t * a.ko_tok_stride + (int64_t)h * a.ko_head_stride, y);
            } else if (SINK == kSinkBf16) {
                if (on_c && h < H) pack_row(static_cast<uint16_t *>(a.k_cache) + (slot.row + (int64_t)h * bs) * D, y);
            } else {
                quantise_row(h, static_cast<int8_t *>(a.k_cache), a.k_scale, y, d0, d1);
            }
        });
        if (kPages) {
            for (int set = max(s0, sq + sk); set < s1; ++set) {
                const int h = (set - sq - sk) * RW + rl;
                take();
                if (SINK == kSinkBf16) {  // copied bit for bit
                    if (on_c && h < H) {
                        uint16_t *dst = static_cast<uint16_t *>(a.v_cache) + (slot.row + (int64_t)h * bs) * D;
                        *reinterpret_cast<uint4 *>(dst + v0) = x0;
                        *reinterpret_cast<uint4 *>(dst + v1) = x1;
                    }
                } else {
                    const uint32_t wd[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                    float2 y[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = make_float2(bf16_lo(wd[i]), bf16_hi(wd[i]));
                    quantise_row(h, static_cast<int8_t *>(a.v_cache), a.v_scale, y, v0, v1);
                }
            }
        }
    }
}

template <int SINK, int L>
cudaError_t launch_rope_variant(const RopeArgs &a, cudaStream_t stream) {
    auto kern = rope_kernel<SINK, L>;
    static OccupancySlots slots;
    int occ = 0;
    cudaError_t e = occupancy(slots, kern, kRopeWarps * 32, 0, &occ);
    if (e != cudaSuccess) return e;
    constexpr int RW = 32 / L;
    const int64_t sets = (a.q_heads + RW - 1) / RW + (SINK == kSinkRows ? 1 : 2) * (int64_t)((a.g.kv_heads + RW - 1) / RW);
    const int64_t cap = (int64_t)sm_count() * occ;
    // fewer tokens than resident warps: a token's row sets are shared among several
    int64_t parts = cap * kRopeWarps / a.num_tokens;
    parts = parts < 1 ? 1 : parts > sets ? sets : parts;
    const int64_t per = (sets + parts - 1) / parts;
    parts = (sets + per - 1) / per;  // no part is empty
    const int64_t need = (a.num_tokens * parts + kRopeWarps - 1) / kRopeWarps;
    kern<<<(unsigned)(need < cap ? need : cap), kRopeWarps * 32, 0, stream>>>(a, (int)parts, (int)per);
    return cudaGetLastError();
}

template <int SINK>
cudaError_t launch_rope_sink(const RopeArgs &a, cudaStream_t stream) {
    const int C = a.g.head_dim / 16;  // 1..16
    if (C <= 1) return launch_rope_variant<SINK, 1>(a, stream);
    if (C <= 2) return launch_rope_variant<SINK, 2>(a, stream);
    if (C <= 4) return launch_rope_variant<SINK, 4>(a, stream);
    if (C <= 8) return launch_rope_variant<SINK, 8>(a, stream);
    return launch_rope_variant<SINK, 16>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, RopeSink sink, cudaStream_t stream) {
    switch (sink) {
        case kSinkDynamic: return launch_rope_sink<kSinkDynamic>(a, stream);
        case kSinkChannel: return launch_rope_sink<kSinkChannel>(a, stream);
        case kSinkBlock: return launch_rope_sink<kSinkBlock>(a, stream);
        case kSinkBf16: return launch_rope_sink<kSinkBf16>(a, stream);
        case kSinkRows: return launch_rope_sink<kSinkRows>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kvc8
