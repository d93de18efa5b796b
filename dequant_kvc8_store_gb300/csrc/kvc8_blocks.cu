// kvc8_blocks.cu -- block tables and slots from lengths: blocks that sequences give up are
// pushed on the stack of free blocks, those that they need are popped from it, both in the
// order of sequences and of their tables' entries, so that the result is that of a loop over
// the sequences and does not depend on how the work is shared.
//
// Prefix sums over the sequences of what they give, need and add say where each id and each
// slot goes.  A pushed id may be popped in the same call, so all pushes come before all pops:
// one cluster of CTAs does the call, each with the sums of all sequences in its shared memory
// (they are a few bytes per sequence, and cheaper made eight times than exchanged), and its
// barrier orders pushes and pops, and reads of the lengths and the count before what is written
// in their place (so none of these is a read-only load).  A thread then takes one id or slot, finds its sequence by a binary search
// in the sums, and reads and writes whole lines with its neighbours.
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kThreads = 1024;
constexpr int kCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Largest b in [0, n) with sums[b] <= x < sums[n].
template <typename T>
__device__ __forceinline__ int owner(const T *sums, int n, T x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// What a sequence needs, gives up and adds.
struct Change {
    int32_t need, give;
    int64_t add;
};

__device__ __forceinline__ Change plus(const Change &a, const Change &b) {
    return Change{a.need + b.need, a.give + b.give, a.add + b.add};
}
__device__ __forceinline__ Change from_below(const Change &a, int by) {
    Change r;
    r.need = __shfl_up_sync(0xFFFFFFFFu, a.need, by);
    r.give = __shfl_up_sync(0xFFFFFFFFu, a.give, by);
    r.add = __shfl_up_sync(0xFFFFFFFFu, a.add, by);
    return r;
}

__global__ void __launch_bounds__(kThreads, 1) assign_kernel(const AssignArgs a) {
    extern __shared__ int64_t dyn[];
    const int B = a.num_seqs, MB = a.max_blocks_per_seq;
    const uint32_t bs = (uint32_t)a.block_size;
    int64_t *s_add = dyn;                                    // [B + 1] exclusive sums
    int32_t *s_need = reinterpret_cast<int32_t *>(s_add + B + 1);  // [B + 1]
    int32_t *s_give = s_need + B + 1;                              // [B + 1]
    int32_t *s_held = s_give + B + 1;                              // [B]; -1: lengths out of range
    __shared__ Change s_warp[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    const int64_t cap = (int64_t)MB * a.block_size;

    const int32_t given = *a.free_count;
    const int32_t F = min(max(given, 0), a.num_blocks);
    if (given != F && rank == 0 && threadIdx.x == 0) report(a.dev_error, KVC8_DEV_BAD_LENGTH);

    Change before{0, 0, 0};
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        Change c{0, 0, 0};
        if (b < B) {
            const int32_t held = a.held[b], want = a.want[b];
            const bool good = held >= 0 && want >= 0 && held <= cap && want <= cap;
            if (good) {
                const int32_t hb = (int32_t)(((uint32_t)held + bs - 1) / bs), wb = (int32_t)(((uint32_t)want + bs - 1) / bs);
                c.need = max(0, wb - hb);
                c.give = max(0, hb - wb);
            } else if (rank == 0) {
                report(a.dev_error, held < 0 || want < 0 ? KVC8_DEV_BAD_LENGTH : KVC8_DEV_POS_BEYOND_TABLE);
            }
            if (held >= 0 && want > held) c.add = want - held;
            s_held[b] = good ? held : -1;
        }
        Change sum = c;  // inclusive over the warp, then the block
#pragma unroll
        for (int by = 1; by < 32; by <<= 1) {
            const Change o = from_below(sum, by);
            if (lane >= by) sum = plus(sum, o);
        }
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            Change w = s_warp[lane];
#pragma unroll
            for (int by = 1; by < 32; by <<= 1) {
                const Change o = from_below(w, by);
                if (lane >= by) w = plus(w, o);
            }
            s_warp[lane] = w;
        }
        __syncthreads();
        sum = plus(sum, before);
        if (warp > 0) sum = plus(sum, s_warp[warp - 1]);
        if (b < B) {
            s_need[b + 1] = sum.need;
            s_give[b + 1] = sum.give;
            s_add[b + 1] = sum.add;
        }
        before = plus(before, s_warp[kThreads / 32 - 1]);
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        s_need[0] = s_give[0] = 0;
        s_add[0] = 0;
    }
    __syncthreads();

    const uint32_t first = rank * kThreads + threadIdx.x, stride = kCluster * kThreads;
    auto in_pool = [&](int32_t id) {
        if (id < 0 || id >= a.num_blocks) report(a.dev_error, KVC8_DEV_BAD_BLOCK_ID);
    };
    // given up: entry w_b + j of b's row
    const uint32_t R = (uint32_t)before.give;
    for (uint32_t x = first; x < R; x += stride) {
        const int b = owner(s_give, B, (int32_t)x);
        const int32_t hb = (int32_t)(((uint32_t)s_held[b] + bs - 1) / bs);
        const int32_t entry = hb - s_give[b + 1] + (int32_t)x;  // w_b + (x - s_give[b])
        const int32_t id = a.block_table[(int64_t)b * MB + entry];
        in_pool(id);
        if ((int64_t)F + x < a.num_blocks) a.free_blocks[F + x] = id;
        else report(a.dev_error, KVC8_DEV_BAD_LENGTH);
    }
    cluster_barrier();
    const int32_t have = (int32_t)min((int64_t)F + R, (int64_t)a.num_blocks);

    // needed: entry h_b + j of b's row
    for (uint32_t k = first; k < (uint32_t)min(before.need, have); k += stride) {
        const int b = owner(s_need, B, (int32_t)k);
        if (s_need[b + 1] > have) continue;
        const int32_t hb = (int32_t)(((uint32_t)s_held[b] + bs - 1) / bs);
        const int32_t id = a.free_blocks[have - 1 - (int32_t)k];
        in_pool(id);
        a.block_table[(int64_t)b * MB + hb + ((int32_t)k - s_need[b])] = id;
    }
    for (uint32_t b = first; b < (uint32_t)B; b += stride) {
        const bool whole = s_need[b + 1] == s_need[b] || s_need[b + 1] <= have;
        if (!whole && s_need[b] <= have) report(a.dev_error, KVC8_DEV_NO_FREE_BLOCK);
        a.lens_out[b] = whole && s_held[b] >= 0 ? a.want[b] : a.held[b];
    }
    if (rank == 0 && warp == 0) {  // the last sequence that is served says how many were popped
        int32_t taken = 0;
        if (before.need <= have) {
            taken = before.need;
        } else if (B > 0) {
            taken = s_need[owner(s_need, B + 1, have)];
        }
        if (lane == 0) *a.free_count_out = have - taken;
    }
    const int64_t slots = min(before.add, a.slot_rows);
    if (before.add > a.slot_rows && a.slot_map != nullptr && rank == 0 && threadIdx.x == 0)
        report(a.dev_error, KVC8_DEV_OUT_ROW_RANGE);
    for (int64_t t = first; t < slots; t += stride) {
        const int b = owner(s_add, B, t);
        const int32_t held = s_held[b];
        int64_t slot = -1;
        if (held >= 0 && (s_need[b + 1] == s_need[b] || s_need[b + 1] <= have)) {
            const uint32_t p = (uint32_t)held + (uint32_t)(t - s_add[b]), lb = p / bs, hb = ((uint32_t)held + bs - 1) / bs;
            const int32_t id = lb < hb ? a.block_table[(int64_t)b * MB + lb]
                                       : a.free_blocks[have - 1 - (s_need[b] + (int32_t)(lb - hb))];
            slot = (int64_t)id * bs + (p - lb * bs);
        }
        a.slot_map[t] = slot;
    }
}

size_t shared_bytes(int B) { return sizeof(int64_t) * ((size_t)B + 1) + sizeof(int32_t) * (3 * (size_t)B + 2); }

}  // namespace

cudaError_t launch_assign(const AssignArgs &a, cudaStream_t stream) {
    const size_t smem = shared_bytes(a.num_seqs);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, assign_kernel, a);
}

}  // namespace kvc8
