// kvc8_tree.cu -- attention of drafted tokens: draft t of sequence b attends over the
// sequence's context and over those of its drafts that the mask names.
//
// A CTA per (sequence, query head), a warp per draft: 32 positions at a time, a lane's
// own position's score, the running maximum and sum, then every lane its channels of the
// values.
#include "kvc8_codes.cuh"
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kWarps = 8;

template <int MODE, int D>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const TreeArgs t) {
    const AttnArgs &a = t.base;
    const int H = a.g.kv_heads, bs = a.g.block_size, MB = a.g.max_blocks_per_seq, Hq = H * a.group;
    const int b = blockIdx.x / Hq, j = blockIdx.x - b * Hq, h = j / a.group;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __shared__ float s_q[kWarps][D];
    const int64_t cap = (int64_t)MB * bs;
    const int64_t c0 = t.cu_q_lens == nullptr ? b : t.cu_q_lens[b], c1 = t.cu_q_lens == nullptr ? b + 1 : t.cu_q_lens[b + 1];
    const bool first = j == 0 && threadIdx.x == 0;
    if (c0 < 0 || c1 < c0 || c1 > t.num_tokens || c1 - c0 > t.max_drafts) {
        if (first) report(a.dev_error, KVC8_DEV_BAD_LENGTH);
        return;
    }
    const int64_t raw = a.context_lengths[b], ctx = raw < 0 ? 0 : raw;
    if (raw < 0 && first) report(a.dev_error, KVC8_DEV_BAD_LENGTH);
    if (ctx + (c1 - c0) > cap && first) report(a.dev_error, KVC8_DEV_POS_BEYOND_TABLE);
    const int64_t len = min(ctx + (c1 - c0), cap);
    for (int64_t n = c0 + warp; n < c1; n += kWarps) {
        const int self = (int)(n - c0);
        for (int d = lane; d < D; d += 32)
            s_q[warp][d] = __uint_as_float((uint32_t)a.q[n * a.q_seq_stride + j * a.q_head_stride + d] << 16);
        __syncwarp();
        float m = -INFINITY, l = 0.0f, o[D / 32];
        for (int i = 0; i < D / 32; ++i) o[i] = 0.0f;
        for (int64_t p0 = 0; p0 < len; p0 += 32) {
            const int64_t p = p0 + lane;
            bool sees = p < len;
            if (sees && p >= ctx) {
                const int i = (int)(p - ctx);
                sees = t.mask == nullptr ? i <= self : (t.mask[n * t.mask_words + i / 64] >> (i % 64) & 1) != 0;
            }
            int32_t blk = 0;
            if (p < len) {
                blk = a.block_table[(int64_t)b * MB + p / bs];
                if (blk < 0 || blk >= a.g.num_blocks) {
                    report(a.dev_error, KVC8_DEV_BAD_BLOCK_ID);
                    sees = false;
                    blk = 0;
                }
            }
            const int64_t row = ((int64_t)blk * H + h) * bs + p % bs;
            float s = -INFINITY, vs = 1.0f;
            if (sees) {
                float dot = 0.0f;
                for (int d = 0; d < D; ++d) {
                    float x = (float)a.k_cache[row * D + d];
                    if (MODE == 1) x *= a.k_scale[h * D + d];
                    dot += s_q[warp][d] * x;
                }
                if (MODE == 0) dot *= a.k_scale[row], vs = a.v_scale[row];
                if (MODE == 2) dot *= a.k_scale[(int64_t)blk * H + h], vs = a.v_scale[(int64_t)blk * H + h];
                s = dot * a.scale_log2;
            }
            float top = s;
            for (int sh = 16; sh > 0; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, sh));
            top = fmaxf(m, top);
            if (top == -INFINITY) continue;
            const float c = m == -INFINITY ? 0.0f : exp2f(m - top);
            const float w = s == -INFINITY ? 0.0f : exp2f(s - top);
            m = top;
            float sum = w;
            for (int sh = 16; sh > 0; sh >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, sh);
            l = l * c + sum;
            for (int i = 0; i < D / 32; ++i) o[i] *= c;
            for (int k = 0; k < 32; ++k) {
                const float wk = __shfl_sync(0xFFFFFFFFu, w * vs, k);
                const int64_t rk = __shfl_sync(0xFFFFFFFFu, row, k);
                const bool in = __shfl_sync(0xFFFFFFFFu, (int)sees, k) != 0;
                if (!in) continue;
                for (int i = 0; i < D / 32; ++i) o[i] += wk * (float)a.v_cache[rk * D + lane + 32 * i];
            }
        }
        uint16_t *dst = a.out + n * a.out_seq_stride + j * a.out_head_stride;
        for (int i = 0; i < D / 32; ++i) {
            float y = l == 0.0f ? 0.0f : o[i] / l;
            if (MODE == 1) y *= a.v_scale[h * D + lane + 32 * i];
            dst[lane + 32 * i] = (uint16_t)(pack_bf16(y, 0.0f) & 0xFFFFu);
        }
        __syncwarp();
    }
}

template <int MODE>
cudaError_t launch_mode(const TreeArgs &t, cudaStream_t stream) {
    const unsigned grid = (unsigned)(t.base.g.num_seqs * t.base.g.kv_heads * t.base.group);
    if (t.base.g.head_dim == 64) tree_kernel<MODE, 64><<<grid, kWarps * 32, 0, stream>>>(t);
    else tree_kernel<MODE, 128><<<grid, kWarps * 32, 0, stream>>>(t);
    return cudaGetLastError();
}

}  // namespace

size_t tree_workspace_bytes(const kvc8_geom &) { return kAlign; }

cudaError_t launch_tree(TreeArgs t, void *, cudaStream_t stream) {
    if (t.base.g.quant_mode == 0) return launch_mode<0>(t, stream);
    if (t.base.g.quant_mode == 1) return launch_mode<1>(t, stream);
    return launch_mode<2>(t, stream);
}

}  // namespace kvc8
