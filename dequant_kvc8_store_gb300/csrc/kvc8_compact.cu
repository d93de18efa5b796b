// kvc8_compact.cu -- the kept drafts' rows move together behind the context: position
// context + accepted[k] to context + k, k ascending, in every head of both caches.
//
// A CTA per sequence.  It checks the whole list and finds each row's places first, then a
// thread takes a unit of bytes of a head's row (mode 0: also one of the rows' scales) through all
// moves in order: up to kBatch of its loads are in flight, and since accepted[k] >= k ascends
// strictly, no row of a later batch is written by an earlier one.  Different threads' bytes
// do not meet.  A unit is 16 bytes, or four codes where they are quantised anew, a division each.
// The work is a few rows per sequence, so latency bounds it: lengths and indices are one round
// trip, block ids another, and a batch's rows a third.  bf16 pages, 256 sequences of 64 drafts
// (16.5 MB): 7.2 us, 2.3 TB/s; int8 pages, 1 sequence of 12 drafts: 5.2 us, 64 of 24: 6.2 us.
// 33 sequences of 9 to 61 drafts with block scales, a division for each code that changes blocks:
// 12.3 us (with a gather that reads the pages back 19; 34 before four codes had a thread).
//
// The time goes by the longest path, eight moves a round trip and as many rounds as a sequence's rows
// have units for its threads: 16, 64 and 256 kept drafts of one sequence (8 heads, D = 128, in a graph)
// take 6.3, 17.6 and 64 us with a row's scales, 4.0, 10.7 and 37 with the channels', 7.6, 21 and 134 with
// a block's, and 4.5, 11.4 and 40 in bf16; 64 such sequences 68, 40, 142 and 51.  A path is as long as a
// draft tree is deep, so several CTAs to a sequence were not tried.
#include <type_traits>

#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kBatch = 8;  // moves in flight
constexpr int kMaxThreads = 512;
static_assert(KVC8_MAX_DRAFTS <= kMaxThreads, "a thread to an index where threads are many");

// Four codes quantised anew for another block's scale.
__device__ __forceinline__ uint32_t requantised(uint32_t w, float from, float to) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int8_t c = (int8_t)(w >> (8 * i));
        const float x = __fmul_rn((float)c, from);
        int q = to == 0.0f ? 0 : __float2int_rn(fminf(fmaxf(__fdiv_rn(x, to), -127.0f), 127.0f));
        r |= (uint32_t)(q & 0xFF) << (8 * i);
    }
    return r;
}

template <bool REQUANT>
__global__ void __launch_bounds__(kMaxThreads) compact_kernel(const CompactArgs a) {
    using Unit = typename std::conditional<REQUANT, uint32_t, uint4>::type;
    __shared__ int32_t s_from[KVC8_MAX_DRAFTS], s_to[KVC8_MAX_DRAFTS];  // block ids; -1: does not move
    __shared__ int32_t s_from_at[KVC8_MAX_DRAFTS], s_to_at[KVC8_MAX_DRAFTS];
    const int b = blockIdx.x, H = a.g.kv_heads;
    const uint32_t bs = (uint32_t)a.g.block_size;
    const int64_t cap = (int64_t)a.g.max_blocks_per_seq * a.g.block_size;
    const int32_t ctx = a.context_kv_lens[b], n = a.num_accepted[b];
    const int32_t *idx = a.accepted + (int64_t)b * a.max_accepted;
    // asked for together with the lengths
    const int mine = threadIdx.x;
    const int32_t first = mine < a.max_accepted ? idx[mine] : 0, before = mine > 0 && mine < a.max_accepted ? idx[mine - 1] : -1;

    bool bad_index = false, beyond = false;
    const bool in_range = ctx >= 0 && n >= 0 && n <= a.max_accepted;
    if (in_range) {
        for (int k = mine; k < n; k += blockDim.x) {
            const int32_t i = k == mine ? first : idx[k];
            if (i < 0 || (k > 0 && i <= (k == mine ? before : idx[k - 1]))) {
                bad_index = true;
            } else if ((int64_t)ctx + i >= cap) {
                beyond = true;
            } else {
                const uint32_t from = (uint32_t)ctx + (uint32_t)i, to = (uint32_t)ctx + (uint32_t)k;
                const uint32_t fb = from / bs, tb = to / bs;
                const int32_t *row = a.block_table + (int64_t)b * a.g.max_blocks_per_seq;
                int32_t f = ld_nc_s32(row + fb), t = ld_nc_s32(row + tb);
                if (i == k) {
                    f = -1;
                } else if (f < 0 || f >= a.g.num_blocks || t < 0 || t >= a.g.num_blocks) {
                    report(a.dev_error, KVC8_DEV_BAD_BLOCK_ID);
                    f = -1;
                }
                s_from[k] = f;
                s_to[k] = t;
                s_from_at[k] = (int32_t)(from - fb * bs);
                s_to_at[k] = (int32_t)(to - tb * bs);
            }
        }
    }
    bad_index = __syncthreads_or(bad_index) != 0;
    beyond = __syncthreads_or(beyond) != 0;
    if (!in_range || bad_index || beyond) {
        if (threadIdx.x == 0) {
            report(a.dev_error, !in_range ? KVC8_DEV_BAD_LENGTH : bad_index ? KVC8_DEV_BAD_INDEX : KVC8_DEV_POS_BEYOND_TABLE);
            if (a.lens_out != nullptr) a.lens_out[b] = ctx;
        }
        return;
    }
    if (threadIdx.x == 0 && a.lens_out != nullptr) a.lens_out[b] = ctx + n;

    const int chunks = a.row_bytes / (int)sizeof(Unit), rows = 2 * H;  // rows: of the keys, then of the values
    for (int u = threadIdx.x; u < rows * chunks; u += blockDim.x) {
        const int r = u / chunks, c = u - r * chunks, h = r < H ? r : r - H;
        char *cache = (r < H ? a.k_cache : a.v_cache) + c * (int)sizeof(Unit);
        const float *scale = r < H ? a.k_scale : a.v_scale;
        for (int k0 = 0; k0 < n; k0 += kBatch) {
            Unit x[kBatch];
            float from[kBatch], to[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int k = k0 + i;
                if (k < n && s_from[k] >= 0) {
                    const int64_t at = (int64_t)s_from[k] * H + h;
                    x[i] = *reinterpret_cast<const Unit *>(cache + (at * bs + s_from_at[k]) * a.row_bytes);
                    if (REQUANT) {
                        from[i] = ld_nc_f32(scale + at);
                        to[i] = ld_nc_f32(scale + (int64_t)s_to[k] * H + h);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int k = k0 + i;
                if (k < n && s_from[k] >= 0) {
                    if constexpr (REQUANT) {
                        if (from[i] != to[i]) x[i] = requantised(x[i], from[i], to[i]);
                    }
                    const int64_t at = ((int64_t)s_to[k] * H + h) * bs + s_to_at[k];
                    *reinterpret_cast<Unit *>(cache + at * a.row_bytes) = x[i];
                }
            }
        }
    }
    if (a.k_scale == nullptr || a.g.quant_mode != 0) return;
    for (int r = threadIdx.x; r < rows; r += blockDim.x) {
        float *scale = r < H ? a.k_scale : a.v_scale;
        const int h = r < H ? r : r - H;
        for (int k = 0; k < n; ++k) {
            if (s_from[k] < 0) continue;
            const float x = scale[((int64_t)s_from[k] * H + h) * bs + s_from_at[k]];
            scale[((int64_t)s_to[k] * H + h) * bs + s_to_at[k]] = x;
        }
    }
}

}  // namespace

cudaError_t launch_compact(const CompactArgs &a, cudaStream_t stream) {
    const bool requant = a.k_scale != nullptr && a.g.quant_mode == 2;
    const int64_t units = (int64_t)2 * a.g.kv_heads * (a.row_bytes / (requant ? 4 : 16));
    const int threads = units >= kMaxThreads ? kMaxThreads : (int)((units + 31) / 32 * 32);
    if (requant) compact_kernel<true><<<(unsigned)a.g.num_seqs, threads, 0, stream>>>(a);
    else compact_kernel<false><<<(unsigned)a.g.num_seqs, threads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvc8
