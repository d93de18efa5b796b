// kvc8_prefix_own.cu -- the own positions of the shared-prefix attention: each
// sequence's queries over its own pages, every split left as a partial (m, l, O) for
// the merge in kvc8_prefix.cu.
//
// A sequence's context is cut into splits of kAttnChunk positions.  A CTA of four warps
// takes every `stride`-th split of a (sequence, kv head), so that no plan of the ragged
// lengths is needed before the launch and the hardware evens out what they differ by; a
// warp walks sub-tiles of 16 positions with mma.sync.m16n8k16:
// S^T = K Q^T and O^T += V^T P^T, positions or channels on M, the group's query heads
// on N, so nothing is padded and codes go from global memory to operands in registers.
//
// What differs is what the codes cost.  HBM bounds this part (2 D bytes and four
// products' worth of work a position), and the issue slots are mostly conversions.  So
// codes are converted exactly and unscaled: to fp16 by one byte permute and one
// subtraction a pair (bf16, for values that a row's scale follows, takes two logic
// operations more).  The scales follow in fp32: a position's key scale and the head's
// factor multiply the score, its value scale the weight, four products each a sub-tile;
// per-channel scales are in the fp16 query and in the output.  A weight alone fits fp16 (see
// kLift), but its product with a row's or block's value scale has the scale's range, so it is
// rounded to bf16, eight bits where fp16 has eleven: the output is off by 0.0020 of its norm
// then, with per-channel scales by 0.0017, which is the output's own rounding to bf16.
// (The prefix's rows have that range taken out sixteen at a time, in shared memory.)
// Any m gives the same quotient of the sums of 2^(score - m) V and 2^(score - m) as long as
// neither over- nor underflows, so the running maximum (Milakov and Gimelshein, Online
// normalizer calculation for softmax, 2018) need not follow every larger score: it moves
// only when the weights grow by more than 2^8, and most sub-tiles reduce and rescale nothing.
// Measured (2048 items of 1 to 1024 positions, 300 MB): 70 us alone, 4.3 TB/s, issue 36%, the
// warps waiting for loads 40% of the time.  Splits of 256, 512 or 1024 positions (217, 202
// and 199 us for the call that took 199 with 2048), a cp.async ring and L2 prefetch did not help.
#include "kvc8_codes.cuh"
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 16;      // positions per warp step
constexpr int kMaxGroup = 8;  // query heads per kv head (mma N)
// The running maximum stays kLift below the largest score when it is set, so that the
// fp16 weights of mode 1 (at most 2^15) keep their eleven bits down to 2^-21 of a row's
// largest, and moves when a score passes it by kLift + kLazy.
constexpr float kLazy = 8.0f, kLift = 7.0f;

template <bool HALF>
__device__ __forceinline__ void mma(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if (HALF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
            "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// N bytes as 16-byte pieces `gap` apart.
template <int N>
__device__ __forceinline__ void load_codes(const void *p, uint32_t *w, int gap = 16) {
    if (N == 8) {
        asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else {
#pragma unroll
        for (int i = 0; i < N / 16; ++i) {
            const uint4 x = ld_stream_16(static_cast<const char *>(p) + gap * i);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
    }
}

// Query heads gid of an item as mma operands: fp16 (mode 1: times the channels' key
// scales) after a power of two that brings a head's largest value to [1, 2); returns
// the factor of head gid's scores, with that power and the softmax scale in it.
template <int MODE, int D>
__device__ __forceinline__ float load_query(const AttnArgs &a, int b, int h, int gid, int tig, uint32_t (&qf)[D / 8]) {
    constexpr int KB = D / 4;
    float2 v[KB / 2];
#pragma unroll
    for (int i = 0; i < KB / 2; ++i) v[i] = make_float2(0.0f, 0.0f);
    float top = 0.0f;
    if (gid < a.group) {
        const uint16_t *qp = a.q + (int64_t)b * a.q_seq_stride + (int64_t)(h * a.group + gid) * a.q_head_stride + tig * 16;
        const float *ks = a.k_scale + (MODE == 1 ? (int64_t)h * D + tig * 16 : 0);
#pragma unroll
        for (int i = 0; i < KB / 8; ++i) {
            const int at = 64 * (i / 2) + 8 * (i % 2);  // as the codes lie (see the loop)
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(qp + at));
            const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float2 y = make_float2(__uint_as_float(wd[e] << 16), __uint_as_float(wd[e] & 0xFFFF0000u));
                if (MODE == 1) {
                    const float2 s = __ldg(reinterpret_cast<const float2 *>(ks + at + 2 * e));
                    y = make_float2(y.x * s.x, y.y * s.y);
                }
                v[4 * i + e] = y;
                top = fmaxf(top, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
        }
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const int ex = power_of(top);
    const float turn = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
    for (int i = 0; i < KB / 2; ++i) qf[i] = pack_fp16(v[i].x * turn, v[i].y * turn);
    return a.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23);
}

template <int MODE, int D>
__global__ void __launch_bounds__(kThreads, 4) own_kernel(const AttnArgs a, int splits, int stride) {
    constexpr int KB = D / 4;   // K code bytes per thread per position
    constexpr int VB = D / 8;   // V code bytes per thread per position
    constexpr int KS = D / 16;  // QK k-steps = PV m-tiles
    constexpr bool kHalfV = MODE == 1;
    const int H = a.g.kv_heads, bs = a.g.block_size, MB = a.g.max_blocks_per_seq, G = a.group;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int gid = lane >> 2, tig = lane & 3;
    __shared__ float s_o[kWarps][kMaxGroup][D];
    __shared__ float s_m[kWarps][kMaxGroup], s_l[kWarps][kMaxGroup];

    pdl_launch_dependents();
    const int b = blockIdx.x / H, h = blockIdx.x - b * H;
    const int64_t cap = (int64_t)MB * bs, raw_len = ld_nc_s32(a.context_lengths + b);
    if (h == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
        if (raw_len < 0) report(a.dev_error, KVC8_DEV_BAD_LENGTH);
        if (raw_len > cap) report(a.dev_error, KVC8_DEV_POS_BEYOND_TABLE);
    }
    const int64_t len = min(raw_len, cap);

    for (int j = blockIdx.y; (int64_t)j * kAttnChunk < len; j += stride) {
        const int64_t item = ((int64_t)b * splits + j) * H + h;
        const int64_t p_begin = (int64_t)j * kAttnChunk;
        const int64_t p_end = min(len, p_begin + kAttnChunk);

        // The warp's sub-tiles of the split are at most 32: a lane fetches the block id of one.
        constexpr int kStride = kWarps * kSub;
        static_assert(kAttnChunk == 32 * kStride, "a lane to a sub-tile");
        const int start = (int)p_begin + warp * kSub, end = (int)p_end;  // lengths are 32-bit
        const int count = start < end ? (int)((uint32_t)(end - start + kStride - 1) / kStride) : 0;
        int32_t ids = 0;
        if (lane < count)
            ids = ld_nc_s32(a.block_table + (int64_t)b * MB + (uint32_t)(start + lane * kStride) / (uint32_t)bs);

        uint32_t qf[KB / 2];
        const float factor = load_query<MODE, D>(a, b, h, gid, tig, qf);
        // the heads of this thread's score columns, 2 tig and 2 tig + 1
        const float f0 = __shfl_sync(0xFFFFFFFFu, factor, 8 * tig), f1 = __shfl_sync(0xFFFFFFFFu, factor, 8 * tig + 4);

        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
        float o[KS][4];
#pragma unroll
        for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

        for (int i = 0; i < count; ++i) {
            const int p0 = start + i * kStride;
            const int32_t blk = __shfl_sync(0xFFFFFFFFu, ids, i);
            if (blk < 0 || blk >= a.g.num_blocks) {
                if (lane == 0) report(a.dev_error, KVC8_DEV_BAD_BLOCK_ID);
                continue;
            }
            const int valid = min(kSub, end - p0);
            const int64_t row0 = ((int64_t)blk * H + h) * bs + (int)((uint32_t)p0 % (uint32_t)bs);
            uint32_t k0[D / 16], k1[D / 16], v[4][D / 32];
            // channels 16 tig and on of each 64: a load covers whole sectors
            const int8_t *kp = a.k_cache + (row0 + gid) * D + tig * 16;
            load_codes<KB>(kp, k0, 64);
            load_codes<KB>(kp + 8 * D, k1, 64);
            const int8_t *vp = a.v_cache + (row0 + 2 * tig) * D + gid * VB;
            load_codes<VB>(vp, v[0]);
            load_codes<VB>(vp + D, v[1]);
            load_codes<VB>(vp + 8 * D, v[2]);
            load_codes<VB>(vp + 9 * D, v[3]);
            const bool va = gid < valid, vb = gid + 8 < valid;
            float ka = 1.0f, kb = 1.0f, sa = 1.0f, sb = 1.0f;  // scales of positions gid and gid + 8
            if (MODE == 0) {
                ka = ld_nc_f32(a.k_scale + row0 + gid);
                kb = ld_nc_f32(a.k_scale + row0 + gid + 8);
                sa = ld_nc_f32(a.v_scale + row0 + gid);
                sb = ld_nc_f32(a.v_scale + row0 + gid + 8);
            } else if (MODE == 2) {
                ka = kb = ld_nc_f32(a.k_scale + (int64_t)blk * H + h);
                sa = sb = ld_nc_f32(a.v_scale + (int64_t)blk * H + h);
            }
            // S^T = K Q^T
            float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                const uint32_t wa = k0[kk] ^ 0x80808080u, wb = k1[kk] ^ 0x80808080u;
                mma<true>(c, codes_fp16(wa, 0x4140u), codes_fp16(wb, 0x4140u), codes_fp16(wa, 0x4342u),
                          codes_fp16(wb, 0x4342u), qf[2 * kk], qf[2 * kk + 1]);
            }
            c[0] = va ? c[0] * (ka * f0) : -INFINITY;
            c[1] = va ? c[1] * (ka * f1) : -INFINITY;
            c[2] = vb ? c[2] * (kb * f0) : -INFINITY;
            c[3] = vb ? c[3] * (kb * f1) : -INFINITY;
            float x0 = fmaxf(c[0], c[2]), x1 = fmaxf(c[1], c[3]);
            if (__any_sync(0xFFFFFFFFu, x0 > m0 + (kLift + kLazy) || x1 > m1 + (kLift + kLazy) || m0 == -INFINITY)) {
                // a column's maximum is that of the lanes with the same tig
#pragma unroll
                for (int sh = 4; sh < 32; sh <<= 1) {
                    x0 = fmaxf(x0, __shfl_xor_sync(0xFFFFFFFFu, x0, sh));
                    x1 = fmaxf(x1, __shfl_xor_sync(0xFFFFFFFFu, x1, sh));
                }
                const float n0 = fmaxf(m0, x0 - kLift), n1 = fmaxf(m1, x1 - kLift);  // finite: valid >= 1
                const float g0 = ex2(m0 - n0), g1 = ex2(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= g0;
                l1 *= g1;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    o[i][0] *= g0, o[i][2] *= g0;
                    o[i][1] *= g1, o[i][3] *= g1;
                }
            }
            float w[4] = {ex2(c[0] - m0), ex2(c[1] - m1), ex2(c[2] - m0), ex2(c[3] - m1)};
            l0 += w[0] + w[2];
            l1 += w[1] + w[3];
            if (MODE != 1) {  // rows behind the end may hold any scale
                w[0] = va ? w[0] * sa : 0.0f, w[1] = va ? w[1] * sa : 0.0f;
                w[2] = vb ? w[2] * sb : 0.0f, w[3] = vb ? w[3] * sb : 0.0f;
            }
            const uint32_t pb0 = transpose8x8(kHalfV ? pack_fp16(w[0], w[1]) : pack_bf16(w[0], w[1]));
            const uint32_t pb1 = transpose8x8(kHalfV ? pack_fp16(w[2], w[3]) : pack_bf16(w[2], w[3]));
            // O^T += V^T P^T; m-tile i: channels gid * VB + 2i and 2i + 1
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const int wd = (2 * i) >> 2;
                const uint32_t lo = (i & 1) ? 0x0602u : 0x0400u, hi = (i & 1) ? 0x0703u : 0x0501u;
                mma<kHalfV>(o[i], codes_of_two<kHalfV>(v[0][wd], v[1][wd], lo), codes_of_two<kHalfV>(v[0][wd], v[1][wd], hi),
                            codes_of_two<kHalfV>(v[2][wd], v[3][wd], lo), codes_of_two<kHalfV>(v[2][wd], v[3][wd], hi),
                            pb0, pb1);
            }
        }
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) {
            l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, sh);
            l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, sh);
        }
        float *so0 = &s_o[warp][2 * tig][gid * VB], *so1 = so0 + D;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            *reinterpret_cast<float2 *>(so0 + 2 * i) = make_float2(o[i][0], o[i][2]);
            *reinterpret_cast<float2 *>(so1 + 2 * i) = make_float2(o[i][1], o[i][3]);
        }
        if (gid == 0) {
            s_m[warp][2 * tig] = m0;
            s_m[warp][2 * tig + 1] = m1;
            s_l[warp][2 * tig] = l0;
            s_l[warp][2 * tig + 1] = l1;
        }
        __syncthreads();
        // join the warps; with no position in the pool the partial is (-inf, 0, 0)
        for (int idx = threadIdx.x; idx < G * D; idx += kThreads) {
            const int hd = idx / D, d = idx - hd * D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][hd]);
            float L = 0.0f, O = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = s_m[w][hd] == -INFINITY ? 0.0f : ex2(s_m[w][hd] - M);
                L += s_l[w][hd] * f;
                O += s_o[w][hd][d] * f;
            }
            if (MODE == 1) O *= __ldg(a.v_scale + (int64_t)h * D + d);
            a.part_o[(item * G + hd) * D + d] = O;
            if (d == 0) {
                a.part_m[item * G + hd] = M;
                a.part_l[item * G + hd] = L;
            }
        }
        __syncthreads();
    }
    // The merge waits for this grid and, through one block's wait, for the prefix's kernel.
    if (blockIdx.x == 0 && blockIdx.y == 0) pdl_wait_prior_grid();
}

int32_t max_splits(const kvc8_geom &g) {
    return (int32_t)(((int64_t)g.max_blocks_per_seq * g.block_size + kAttnChunk - 1) / kAttnChunk);
}

// CTAs of a launch that keep the GPU full and still start and end in no time when the
// tables have room for many more splits than the sequences use.
constexpr int64_t kMaxGrid = 8192;

template <int MODE, int D>
cudaError_t launch_variant(const AttnArgs &a, cudaStream_t stream) {
    const int64_t pairs = (int64_t)a.g.num_seqs * a.g.kv_heads;
    const int splits = max_splits(a.g);
    int64_t stride = kMaxGrid / pairs;
    stride = stride < 1 ? 1 : stride > splits ? splits : stride;
    return launch_dependent(own_kernel<MODE, D>, dim3((unsigned)pairs, (unsigned)stride), kThreads, (size_t)0, stream, a,
                            splits, (int)stride);
}

template <int MODE>
cudaError_t launch_mode(const AttnArgs &a, cudaStream_t stream) {
    if (a.g.head_dim == 64) return launch_variant<MODE, 64>(a, stream);
    return launch_variant<MODE, 128>(a, stream);
}

}  // namespace

// The partials: O, m, l of each (sequence, split, kv head, query head).
size_t own_workspace_bytes(const kvc8_geom &g, int group) {
    const size_t rows = (size_t)g.num_seqs * g.kv_heads * max_splits(g) * group;
    return align_up(sizeof(float) * rows * g.head_dim, kAlign) + 2 * align_up(sizeof(float) * rows, kAlign);
}

void place_own(PrefixArgs &p, void *workspace) {
    AttnArgs &a = p.own;
    const size_t rows = (size_t)a.g.num_seqs * a.g.kv_heads * max_splits(a.g) * a.group;
    char *base = static_cast<char *>(workspace);
    p.own_splits = max_splits(a.g);
    a.part_o = reinterpret_cast<float *>(base);
    base += align_up(sizeof(float) * rows * a.g.head_dim, kAlign);
    a.part_m = reinterpret_cast<float *>(base);
    base += align_up(sizeof(float) * rows, kAlign);
    a.part_l = reinterpret_cast<float *>(base);
}

cudaError_t launch_own(const PrefixArgs &p, cudaStream_t stream) {
    const AttnArgs &a = p.own;
    if (a.g.quant_mode == 0) return launch_mode<0>(a, stream);
    if (a.g.quant_mode == 1) return launch_mode<1>(a, stream);
    return launch_mode<2>(a, stream);
}

}  // namespace kvc8
