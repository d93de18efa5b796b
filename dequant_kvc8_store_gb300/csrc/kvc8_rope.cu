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
// One warp per row: lane l holds channels l, l + 32, ...; the pairs meet in
// shared memory.
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kMaxD = 256;

__device__ __forceinline__ float bf16_f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ uint16_t f_bf16(float x) {
    unsigned short b;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(x));
    return b;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

template <int SINK>
__global__ void __launch_bounds__(kRopeWarps * 32) rope_kernel(const RopeArgs a) {
    __shared__ float row_s[kRopeWarps][kMaxD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int H = a.g.kv_heads, D = a.g.head_dim, HQ = a.q_heads;
    const int rows = HQ + (SINK == kSinkRows ? 1 : 2) * H;
    const int64_t units = a.num_tokens * rows;
    float *row = row_s[warp];
    for (int64_t u = (int64_t)blockIdx.x * kRopeWarps + warp; u < units;
         u += (int64_t)gridDim.x * kRopeWarps) {
        const int64_t t = u / rows;
        const int r = (int)(u - t * rows);
        const int kind = r < HQ ? 0 : r < HQ + H ? 1 : 2;  // query, key, value
        const int h = kind == 0 ? r : kind == 1 ? r - HQ : r - HQ - H;
        int64_t pos = 0, cache_row = 0;
        int32_t blk = 0;
        if (SINK != kSinkRows) {
            const int bs = a.g.block_size, MB = a.g.max_blocks_per_seq;
            TokenSeq ts;
            if (a.cu_q_lens != nullptr) {
                ts = seq_ctx_of_token(a.cu_q_lens, a.context_kv_lens, a.g.num_seqs, t, lane);
            } else {
                ts = {(int)t, t, t + 1, a.context_kv_lens[t]};
            }
            pos = ts.ctx + (t - ts.first);
            const int64_t lb = pos / bs;
            int32_t err = 0;
            if (!(ts.first <= t && t < ts.next) || ts.ctx < 0) {
                err = KVC8_DEV_BAD_LENGTH;
            } else if (lb >= MB) {
                err = KVC8_DEV_POS_BEYOND_TABLE;
            } else {
                blk = ld_nc_s32(a.block_table + (int64_t)ts.b * MB + lb);
                if (blk < 0 || blk >= a.g.num_blocks) err = KVC8_DEV_BAD_BLOCK_ID;
            }
            if (err != 0) {
                if (lane == 0) report(a.dev_error, err);
                continue;
            }
            cache_row = ((int64_t)blk * H + h) * bs + (pos - lb * bs);
        }
        if (a.positions != nullptr) pos = a.positions[t];
        const uint16_t *src = kind == 0 ? a.q + t * a.q_tok_stride + h * a.q_head_stride
                                        : (kind == 1 ? a.k : a.v) + t * a.x_tok_stride + h * a.x_head_stride;
        const uint16_t *w = kind == 0 ? a.q_weight : kind == 1 ? a.k_weight : nullptr;
        float sum = 0.0f;
        for (int d = lane; d < D; d += 32) {
            const float x = bf16_f(src[d]);
            row[d] = x;
            sum += x * x;
        }
        if (w != nullptr) {
            const float inv = 1.0f / sqrtf(warp_sum(sum) / (float)D + a.eps);
            for (int d = lane; d < D; d += 32) row[d] = row[d] * inv * bf16_f(w[d]);
        }
        __syncwarp();
        if (kind != 2) {
            const int half = a.rotary_dim / 2;
            for (int i = lane; i < half; i += 32) {
                const uint64_t phase = (uint64_t)pos * a.freqs[i];
                float s, c;
                sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
                s *= a.factor;
                c *= a.factor;
                const int da = a.interleaved ? 2 * i : i, db = a.interleaved ? 2 * i + 1 : i + half;
                const float ya = row[da], yb = row[db];
                row[da] = ya * c - yb * s;
                row[db] = yb * c + ya * s;
            }
        }
        __syncwarp();
        if (kind == 0 || SINK == kSinkRows) {
            uint16_t *dst = kind == 0 ? a.q_out + t * a.qo_tok_stride + h * a.qo_head_stride
                                      : a.k_out + t * a.ko_tok_stride + h * a.ko_head_stride;
            for (int d = lane; d < D; d += 32) dst[d] = f_bf16(row[d]);
        } else if (SINK == kSinkBf16) {
            uint16_t *dst = static_cast<uint16_t *>(kind == 1 ? a.k_cache : a.v_cache) + cache_row * D;
            for (int d = lane; d < D; d += 32) dst[d] = f_bf16(row[d]);
        } else {
            int8_t *dst = static_cast<int8_t *>(kind == 1 ? a.k_cache : a.v_cache) + cache_row * D;
            float *scl = kind == 1 ? a.k_scale : a.v_scale;
            float s_row = 0.0f;
            if (SINK == kSinkDynamic) {
                float m = 0.0f;
                for (int d = lane; d < D; d += 32) m = fmaxf(m, fabsf(row[d]));
                s_row = __fdiv_rn(warp_max(m), 127.0f);
                if (lane == 0) scl[cache_row] = s_row;
            } else if (SINK == kSinkBlock) {
                s_row = scl[(int64_t)blk * H + h];
            }
            for (int d = lane; d < D; d += 32) {
                const float s = SINK == kSinkChannel ? scl[(int64_t)h * D + d] : s_row;
                const int q = s == 0.0f ? 0 : __float2int_rn(__fdiv_rn(row[d], s));
                dst[d] = (int8_t)min(127, max(-127, q));
            }
        }
        __syncwarp();
    }
}

template <int SINK>
cudaError_t launch_rope_variant(const RopeArgs &a, cudaStream_t stream) {
    auto kern = rope_kernel<SINK>;
    static OccupancySlots slots;
    int occ = 0;
    cudaError_t e = occupancy(slots, kern, kRopeWarps * 32, 0, &occ);
    if (e != cudaSuccess) return e;
    const int64_t rows = a.q_heads + (SINK == kSinkRows ? 1 : 2) * (int64_t)a.g.kv_heads;
    const int64_t need = (a.num_tokens * rows + kRopeWarps - 1) / kRopeWarps;
    const int64_t cap = (int64_t)sm_count() * occ;
    kern<<<(unsigned)(need < cap ? need : cap), kRopeWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, RopeSink sink, cudaStream_t stream) {
    switch (sink) {
        case kSinkDynamic: return launch_rope_variant<kSinkDynamic>(a, stream);
        case kSinkChannel: return launch_rope_variant<kSinkChannel>(a, stream);
        case kSinkBlock: return launch_rope_variant<kSinkBlock>(a, stream);
        case kSinkBf16: return launch_rope_variant<kSinkBf16>(a, stream);
        case kSinkRows: return launch_rope_variant<kSinkRows>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace kvc8
