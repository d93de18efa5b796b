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
// channels [8c, 8c+8) and [R/2 + 8c, +8) in the half layout, 16 neighbours in the
// interleaved one -- so nothing is exchanged but the row sums and maxima.  A unit of
// work is a token, or a part of its row sets where there are fewer tokens than
// warps.  The warp finds its token's slot, computes the R/2 sines and cosines once
// (a lane R/64 of them, kept in shared memory) and runs through the row sets, the
// next set's loads in flight.
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kRopeWarps = 4;
constexpr int kMaxPairs = 128;

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Where a token goes.
struct Slot {
    int64_t row;  // cache row of (block, head 0, slot); -1: the token is skipped
    int32_t blk;
    int64_t pos;  // its rotary position
};

template <int SINK>
__device__ __forceinline__ Slot find_slot(const RopeArgs &a, int64_t t, int lane, bool report_it) {
    Slot s = {0, 0, 0};
    if (SINK != kSinkRows) {
        const int bs = a.g.block_size, MB = a.g.max_blocks_per_seq;
        TokenSeq q;
        if (a.cu_q_lens != nullptr) {
            q = seq_ctx_of_token(a.cu_q_lens, a.context_kv_lens, a.g.num_seqs, t, lane);
        } else {
            q = {(int)t, t, t + 1, ld_nc_s32(a.context_kv_lens + t)};
        }
        s.pos = q.ctx + (t - q.first);
        int32_t err = 0;
        int64_t lb = 0;
        if (!(q.first <= t && t < q.next) || q.ctx < 0) {
            err = KVC8_DEV_BAD_LENGTH;
        } else {
            // 0 <= pos < 2^32: a 32-bit division
            lb = (int64_t)((uint32_t)s.pos / (uint32_t)bs);
            if (lb >= MB) {
                err = KVC8_DEV_POS_BEYOND_TABLE;
            } else {
                s.blk = ld_nc_s32(a.block_table + (int64_t)q.b * MB + lb);
                if (s.blk < 0 || s.blk >= a.g.num_blocks) err = KVC8_DEV_BAD_BLOCK_ID;
            }
        }
        if (err != 0) {
            if (report_it && lane == 0) report(a.dev_error, err);
            s.row = -1;
            return s;
        }
        s.row = (int64_t)s.blk * a.g.kv_heads * bs + (s.pos - lb * bs);
    }
    if (a.positions != nullptr) s.pos = ld_nc_s32(a.positions + t);
    return s;
}

// L lanes per row, 32 / L rows of a set.
template <int SINK, int L>
__global__ void __launch_bounds__(kRopeWarps * 32, 6) rope_kernel(const RopeArgs a, int parts) {
    constexpr int RW = 32 / L;
    constexpr bool kPages = SINK != kSinkRows;
    __shared__ __align__(16) float turn_s[kRopeWarps][2][kMaxPairs];  // m cos, m sin
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int H = a.g.kv_heads, D = a.g.head_dim, R = a.rotary_dim, bs = a.g.block_size;
    const int sq = (a.q_heads + RW - 1) / RW, sk = (H + RW - 1) / RW;
    const int sets = sq + sk + (kPages ? sk : 0);  // row sets of a token: queries, keys, values
    const int per = (sets + parts - 1) / parts;
    const int rl = lane / L, c = lane % L;
    const bool on_c = c < D / 16;
    // This lane's channels.  Half layout: lanes c < R/16 rotate channels 8c and R/2 + 8c
    // on; the others pass sixteen of the rest.
    const bool turns = c < R / 16;
    const int d0 = turns && !a.interleaved ? 8 * c : 16 * c;
    const int d1 = turns && !a.interleaved ? R / 2 + 8 * c : 16 * c + 8;
    float *cos_s = turn_s[warp][0], *sin_s = turn_s[warp][1];

    const int64_t units = a.num_tokens * parts;
    for (int64_t u = (int64_t)blockIdx.x * kRopeWarps + warp; u < units; u += (int64_t)gridDim.x * kRopeWarps) {
        const int64_t t = u / parts;
        const int part = (int)(u - t * parts);
        const int s0 = part * per, s1 = min(sets, s0 + per);
        if (s0 >= s1) continue;

        auto source = [&](int set, bool &on, int &h, int &kind) -> const uint16_t * {
            kind = set < sq ? 0 : set < sq + sk ? 1 : 2;
            h = (set - (kind == 0 ? 0 : kind == 1 ? sq : sq + sk)) * RW + rl;
            on = on_c && h < (kind == 0 ? a.q_heads : H);
            return kind == 0 ? a.q + t * a.q_tok_stride + (int64_t)h * a.q_head_stride
                             : (kind == 1 ? a.k : a.v) + t * a.x_tok_stride + (int64_t)h * a.x_head_stride;
        };
        bool on;
        int h, kind;
        uint4 x0 = make_uint4(0u, 0u, 0u, 0u), x1 = x0;
        {
            const uint16_t *src = source(s0, on, h, kind);
            if (on) {
                x0 = ld_stream_16(src + (kind == 2 ? 16 * c : d0));
                x1 = ld_stream_16(src + (kind == 2 ? 16 * c + 8 : d1));
            }
        }
        const Slot slot = find_slot<SINK>(a, t, lane, part == 0);
        if (kPages && slot.row < 0) continue;  // uniform in the warp
        __syncwarp();
        if (s0 < sq + sk) {
            for (int i = lane; i < R / 2; i += 32) {
                const uint64_t phase = (uint64_t)slot.pos * __ldg(a.freqs + i);
                float s, co;
                sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &co);
                cos_s[i] = co * a.factor;
                sin_s[i] = s * a.factor;
            }
        }
        __syncwarp();

        for (int set = s0; set < s1; ++set) {
            const bool cur_on = on;
            const int cur_h = h, cur_kind = kind;
            float2 v[8];  // v[0..3]: the first piece, v[4..7]: the second
            {
                const uint32_t wd[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = make_float2(bf16_lo(wd[i]), bf16_hi(wd[i]));
            }
            const uint4 raw0 = x0, raw1 = x1;
            if (set + 1 < s1) {  // the next set's rows
                const uint16_t *src = source(set + 1, on, h, kind);
                x0 = x1 = make_uint4(0u, 0u, 0u, 0u);
                if (on) {
                    x0 = ld_stream_16(src + (kind == 2 ? 16 * c : d0));
                    x1 = ld_stream_16(src + (kind == 2 ? 16 * c + 8 : d1));
                }
            }
            const uint16_t *w = cur_kind == 0 ? a.q_weight : cur_kind == 1 ? a.k_weight : nullptr;
            if (w != nullptr) {
                float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum2 = __ffma2_rn(v[i], v[i], sum2);
                float sum = sum2.x + sum2.y;
#pragma unroll
                for (int o = 1; o < L; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                const float inv = __frcp_rn(__fsqrt_rn(sum / (float)D + a.eps));
                if (on_c) {
                    const uint4 w0 = __ldg(reinterpret_cast<const uint4 *>(w + d0));
                    const uint4 w1 = __ldg(reinterpret_cast<const uint4 *>(w + d1));
                    const uint32_t wd[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = __fmul2_rn(__fmul2_rn(v[i], make_float2(inv, inv)),
                                          make_float2(bf16_lo(wd[i]), bf16_hi(wd[i])));
                }
            }
            if (cur_kind != 2 && turns) {
                // pairs 8c .. 8c + 7 in either layout
                const float4 *cp = reinterpret_cast<const float4 *>(cos_s + 8 * c);
                const float4 *sp = reinterpret_cast<const float4 *>(sin_s + 8 * c);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float4 co = cp[q], si = sp[q];
                    if (!a.interleaved) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 c2 = e ? make_float2(co.z, co.w) : make_float2(co.x, co.y);
                            const float2 s2 = e ? make_float2(si.z, si.w) : make_float2(si.x, si.y);
                            const float2 ya = v[2 * q + e], yb = v[4 + 2 * q + e];
                            const float2 ns = make_float2(-s2.x, -s2.y);
                            v[2 * q + e] = __ffma2_rn(ya, c2, __fmul2_rn(yb, ns));
                            v[4 + 2 * q + e] = __ffma2_rn(yb, c2, __fmul2_rn(ya, s2));
                        }
                    } else {
                        const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 y = v[4 * q + e];
                            v[4 * q + e] = make_float2(fmaf(y.x, cc[e], -(y.y * ss[e])), fmaf(y.y, cc[e], y.x * ss[e]));
                        }
                    }
                }
            }
            // a value row is held as sixteen neighbours
            const int o0 = cur_kind == 2 ? 16 * c : d0, o1 = cur_kind == 2 ? 16 * c + 8 : d1;
            if (cur_kind == 0 || SINK == kSinkRows || SINK == kSinkBf16) {
                uint16_t *dst;
                if (cur_kind == 0) dst = a.q_out + t * a.qo_tok_stride + (int64_t)cur_h * a.qo_head_stride;
                else if (SINK == kSinkRows) dst = a.k_out + t * a.ko_tok_stride + (int64_t)cur_h * a.ko_head_stride;
                else dst = static_cast<uint16_t *>(cur_kind == 1 ? a.k_cache : a.v_cache) +
                           (slot.row + (int64_t)cur_h * bs) * D;
                uint4 y0 = raw0, y1 = raw1;  // values are copied bit for bit
                if (cur_kind != 2) {
                    y0 = make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y),
                                    pack_bf16(v[3].x, v[3].y));
                    y1 = make_uint4(pack_bf16(v[4].x, v[4].y), pack_bf16(v[5].x, v[5].y), pack_bf16(v[6].x, v[6].y),
                                    pack_bf16(v[7].x, v[7].y));
                }
                if (cur_on) {
                    *reinterpret_cast<uint4 *>(dst + o0) = y0;
                    *reinterpret_cast<uint4 *>(dst + o1) = y1;
                }
            } else {
                const int64_t cache_row = slot.row + (int64_t)cur_h * bs;
                int8_t *dst = static_cast<int8_t *>(cur_kind == 1 ? a.k_cache : a.v_cache) + cache_row * D;
                float *scl = cur_kind == 1 ? a.k_scale : a.v_scale;
                float s_row = 0.0f;
                if (SINK == kSinkDynamic) {
                    float m = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
#pragma unroll
                    for (int o = 1; o < L; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                    s_row = __fdiv_rn(m, 127.0f);
                    if (cur_on && c == 0) scl[cache_row] = s_row;
                } else if (SINK == kSinkBlock && cur_on) {
                    s_row = ld_nc_f32(scl + (int64_t)slot.blk * H + cur_h);
                }
                if (cur_on) {
                    uint32_t o[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float y[4] = {v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y};
                        uint32_t pk = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int d = (q < 2 ? o0 : o1) + 4 * (q & 1) + e;
                            const float s = SINK == kSinkChannel ? ld_nc_f32(scl + (int64_t)cur_h * D + d) : s_row;
                            const int code = s == 0.0f ? 0 : __float2int_rn(__fdiv_rn(y[e], s));
                            pk |= (uint32_t)(uint8_t)(int8_t)min(127, max(-127, code)) << (8 * e);
                        }
                        o[q] = pk;
                    }
                    st_8(dst + o0, o[0], o[1]);
                    st_8(dst + o1, o[2], o[3]);
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
    const int64_t need = (a.num_tokens * parts + kRopeWarps - 1) / kRopeWarps;
    kern<<<(unsigned)(need < cap ? need : cap), kRopeWarps * 32, 0, stream>>>(a, (int)parts);
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
