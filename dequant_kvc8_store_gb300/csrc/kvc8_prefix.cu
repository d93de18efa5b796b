// kvc8_prefix.cu -- decode attention of a batch whose sequences share a prefix:
// query head j of sequence b attends over the prefix's positions and then over
// its own, in one softmax.
//   out[b][j] = (sum_p w_p V[p] + sum_p u_p V_b[p]) / (sum_p w_p + sum_p u_p)
//   w_p = exp(scale <q, K[p]>), u_p = exp(scale <q, K_b[p]>)
// with K, V = fp32(code) * scale; no position at all gives zeros.
//
// One CTA per (sequence, kv head) walks its prefix and own positions 128 at a
// time with an online softmax: a thread per position for the scores, a thread
// per channel for the weighted sum.
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kTile = 128;
constexpr int kMaxGroup = 8;

template <int MODE, int D>
__global__ void __launch_bounds__(kTile) prefix_kernel(const PrefixArgs p) {
    const AttnArgs &a = p.own;
    const int H = a.g.kv_heads, bs = a.g.block_size, G = a.group;
    const int b = blockIdx.x / H, h = blockIdx.x - b * H;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __shared__ float q_s[kMaxGroup][D];
    __shared__ float w_s[kMaxGroup][kTile];
    __shared__ int64_t row_s[kTile];  // cache row of each position, -1: left out
    __shared__ float sv_s[kTile];
    __shared__ float red[4][kMaxGroup];
    for (int i = tid; i < G * D; i += kTile) {
        const int j = i / D, d = i - j * D;
        q_s[j][d] = __uint_as_float((uint32_t)a.q[(int64_t)b * a.q_seq_stride +
                                                  (int64_t)(h * G + j) * a.q_head_stride + d] << 16);
    }
    __syncthreads();
    float acc[kMaxGroup], m[kMaxGroup], l[kMaxGroup];
#pragma unroll
    for (int j = 0; j < kMaxGroup; ++j) {
        acc[j] = l[j] = 0.0f;
        m[j] = -INFINITY;
    }
    for (int part = 0; part < 2; ++part) {
        const int32_t *table = part == 0 ? p.prefix_table
                                         : a.block_table + (int64_t)b * a.g.max_blocks_per_seq;
        const int64_t cap = (int64_t)(part == 0 ? p.max_prefix_blocks : a.g.max_blocks_per_seq) * bs;
        int64_t len = part == 0 ? p.prefix_length[0] : a.context_lengths[b];
        if (tid == 0 && h == 0) {
            if (len < 0) report(a.dev_error, KVC8_DEV_BAD_LENGTH);
            if (len > cap) report(a.dev_error, KVC8_DEV_POS_BEYOND_TABLE);
        }
        len = min(len, cap);
        for (int64_t p0 = 0; p0 < len; p0 += kTile) {
            const int64_t pos = p0 + tid;
            float s[kMaxGroup];
#pragma unroll
            for (int j = 0; j < kMaxGroup; ++j) s[j] = -INFINITY;
            int64_t row = -1;
            float sv = 0.0f;
            if (pos < len) {
                const int64_t lb = pos / bs;
                const int32_t blk = table[lb];
                if (blk < 0 || blk >= a.g.num_blocks) {
                    report(a.dev_error, KVC8_DEV_BAD_BLOCK_ID);
                } else {
                    row = ((int64_t)blk * H + h) * bs + (pos - lb * bs);
                    const int64_t at = MODE == 0 ? row : (int64_t)blk * H + h;
                    const float sk = MODE == 1 ? 1.0f : a.k_scale[at];
                    sv = MODE == 1 ? 1.0f : a.v_scale[at];
                    float dot[kMaxGroup];
#pragma unroll
                    for (int j = 0; j < kMaxGroup; ++j) dot[j] = 0.0f;
                    for (int d = 0; d < D; ++d) {
                        const float k = (float)a.k_cache[row * D + d] *
                                        (MODE == 1 ? a.k_scale[h * D + d] : sk);
#pragma unroll
                        for (int j = 0; j < kMaxGroup; ++j)
                            if (j < G) dot[j] += q_s[j][d] * k;
                    }
#pragma unroll
                    for (int j = 0; j < kMaxGroup; ++j)
                        if (j < G) s[j] = dot[j] * a.scale_log2;
                }
            }
            __syncthreads();  // the last round's weights are used up
            row_s[tid] = row;
            sv_s[tid] = sv;
#pragma unroll
            for (int j = 0; j < kMaxGroup; ++j) {
                float x = s[j];
                for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
                if (lane == 0) red[warp][j] = x;
            }
            __syncthreads();
            float f[kMaxGroup];
#pragma unroll
            for (int j = 0; j < kMaxGroup; ++j) {
                const float top = fmaxf(fmaxf(red[0][j], red[1][j]), fmaxf(red[2][j], red[3][j]));
                const float n = fmaxf(m[j], top);
                f[j] = n == -INFINITY ? 1.0f : exp2f(m[j] - n);
                m[j] = n;
                w_s[j][tid] = s[j] == -INFINITY ? 0.0f : exp2f(s[j] - n);
                acc[j] *= f[j];
                l[j] *= f[j];
            }
            __syncthreads();
            const int count = (int)min((int64_t)kTile, len - p0);
            for (int i = 0; i < count; ++i) {
                const int64_t r = row_s[i];
                if (r < 0) continue;
                const float v = tid < D ? (float)a.v_cache[r * D + tid] * sv_s[i] : 0.0f;
#pragma unroll
                for (int j = 0; j < kMaxGroup; ++j) {
                    acc[j] += w_s[j][i] * v;
                    l[j] += w_s[j][i];
                }
            }
        }
    }
    if (tid < D) {
        const float sv = MODE == 1 ? a.v_scale[h * D + tid] : 1.0f;
#pragma unroll
        for (int j = 0; j < kMaxGroup; ++j) {
            if (j >= G) continue;
            unsigned short o;
            asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(o) : "f"(l[j] > 0.0f ? acc[j] * sv / l[j] : 0.0f));
            a.out[(int64_t)b * a.out_seq_stride + (int64_t)(h * G + j) * a.out_head_stride + tid] = o;
        }
    }
}

template <int MODE>
cudaError_t launch_mode(const PrefixArgs &p, cudaStream_t stream) {
    const unsigned grid = (unsigned)(p.own.g.num_seqs * p.own.g.kv_heads);
    if (p.own.g.head_dim == 64) prefix_kernel<MODE, 64><<<grid, kTile, 0, stream>>>(p);
    else prefix_kernel<MODE, 128><<<grid, kTile, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t shared_prefix_workspace_bytes(const kvc8_geom &, int, int32_t) { return kAlign; }

cudaError_t launch_shared_prefix(const PrefixArgs &p, void *, cudaStream_t stream) {
    if (p.own.g.quant_mode == 0) return launch_mode<0>(p, stream);
    if (p.own.g.quant_mode == 1) return launch_mode<1>(p, stream);
    return launch_mode<2>(p, stream);
}

}  // namespace kvc8
