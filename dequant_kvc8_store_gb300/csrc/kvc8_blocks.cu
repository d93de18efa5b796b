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
// in their place (so none of these is a read-only load).  A thread then takes one id or slot,
// finds its sequence by a binary search in the sums, and reads and writes whole lines with its
// neighbours.
//
// Slots follow from the inputs alone: a popped id is looked up where it comes from, in the stack
// below or in the row that gives it up.  So many of them are made by a kernel of their own on all
// SMs, before the cluster changes anything; meanwhile the cluster makes its sums.
//
// Latency bounds all of it: a decode step's 12 KB (256 sequences, 1150 slots) take 5.9 us, of which
// the launch and one round trip for the lengths are most; 16 prompts of 36 696 slots (0.29 MB) 8.2 to
// 9.3 us (7.2 in a graph);
// 4096 sequences with 820 000 slots (6.7 MB, 1 us at the copy rate) 28.7 us (36.3 without the overlap of
// the two launches, 127 before slots had a kernel of their own).
#include "kvc8_internal.cuh"

namespace kvc8 {
namespace {

constexpr int kThreads = 1024, kFewThreads = 256;
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

// What all sequences up to one need, give and add, in shared memory, and the stack before the pops.
struct Sums {
    int64_t *add;              // [B + 1] exclusive
    int32_t *need, *give;      // [B + 1] exclusive
    int32_t *held;             // [B]; -1: lengths out of range
    int32_t F, R, have, need_all;
    int64_t add_all;

    __device__ __forceinline__ uint32_t blocks(int b, uint32_t bs) const { return ((uint32_t)held[b] + bs - 1) / bs; }
    __device__ __forceinline__ bool served(int b) const { return need[b + 1] == need[b] || need[b + 1] <= have; }
};

// By the whole block; `reports`: this block reports what is out of range.
__device__ __forceinline__ Sums add_up(const AssignArgs &a, int64_t *dyn, bool reports) {
    __shared__ Change s_warp[kThreads / 32];
    const int B = a.num_seqs, T = blockDim.x;
    const uint32_t bs = (uint32_t)a.block_size;
    Sums s;
    s.add = dyn;
    s.need = reinterpret_cast<int32_t *>(s.add + B + 1);
    s.give = s.need + B + 1;
    s.held = s.give + B + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t cap = (int64_t)a.max_blocks_per_seq * a.block_size;

    const int32_t given = *a.free_count;
    s.F = min(max(given, 0), a.num_blocks);
    if (given != s.F && reports && threadIdx.x == 0) report(a.dev_error, KVC8_DEV_BAD_LENGTH);
    if (threadIdx.x == 0) {
        s.need[0] = s.give[0] = 0;
        s.add[0] = 0;
    }
    // this thread's sequences in a row: what they change together, then one scan, then each one's sums
    const int per = (B + T - 1) / T, b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
    auto change = [&](int b, bool first) {
        Change c{0, 0, 0};
        const int32_t held = a.held[b], want = a.want[b];
        const bool good = held >= 0 && want >= 0 && held <= cap && want <= cap;
        if (good) {
            const int32_t hb = (int32_t)(((uint32_t)held + bs - 1) / bs), wb = (int32_t)(((uint32_t)want + bs - 1) / bs);
            c.need = max(0, wb - hb);
            c.give = max(0, hb - wb);
        } else if (reports && first) {
            report(a.dev_error, held < 0 || want < 0 ? KVC8_DEV_BAD_LENGTH : KVC8_DEV_POS_BEYOND_TABLE);
        }
        if (held >= 0 && want > held) c.add = want - held;
        s.held[b] = good ? held : -1;
        return c;
    };
    Change sum{0, 0, 0};
    for (int b = b0; b < b1; ++b) sum = plus(sum, change(b, true));
    Change upto = sum;  // inclusive over the warp, then the block
#pragma unroll
    for (int by = 1; by < 32; by <<= 1) {
        const Change o = from_below(upto, by);
        if (lane >= by) upto = plus(upto, o);
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    if (warp == 0) {
        Change w = lane < T / 32 ? s_warp[lane] : Change{0, 0, 0};
#pragma unroll
        for (int by = 1; by < 32; by <<= 1) {
            const Change o = from_below(w, by);
            if (lane >= by) w = plus(w, o);
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    Change before = warp > 0 ? s_warp[warp - 1] : Change{0, 0, 0};
    const Change all = s_warp[kThreads / 32 - 1];
    upto = plus(upto, before);
    Change at{upto.need - sum.need, upto.give - sum.give, upto.add - sum.add};
    for (int b = b0; b < b1; ++b) {
        at = plus(at, per == 1 ? sum : change(b, false));
        s.need[b + 1] = at.need;
        s.give[b + 1] = at.give;
        s.add[b + 1] = at.add;
    }
    __syncthreads();
    s.R = all.give;
    s.have = (int32_t)min((int64_t)s.F + s.R, (int64_t)a.num_blocks);
    s.need_all = all.need;
    s.add_all = all.add;
    return s;
}

// Where there are more slots than threads, kRun in a row to a thread: one search, and one lookup of an id where they lie in
// one block (one slot to a thread is quicker while threads last: the lookups of a run follow one another).
constexpr int kRun = 4;
__device__ __forceinline__ void write_slots(const AssignArgs &a, const Sums &s, int64_t first, int64_t stride) {
    const int B = a.num_seqs;
    const int64_t MB = a.max_blocks_per_seq, slots = min(s.add_all, a.slot_rows);
    const uint32_t bs = (uint32_t)a.block_size;
    const int run = slots <= stride ? 1 : kRun;
    for (int64_t t0 = first * run; t0 < slots; t0 += stride * run) {
        int b = owner(s.add, B, t0), last_b = -1;
        uint32_t last_lb = 0;
        int32_t id = 0;
        const int64_t end = min(t0 + run, slots);
#pragma unroll 1
        for (int64_t t = t0; t < end; ++t) {
            while (t >= s.add[b + 1]) ++b;
            const int32_t held = s.held[b];
            int64_t slot = -1;
            if (held >= 0 && s.served(b)) {
                const uint32_t p = (uint32_t)held + (uint32_t)(t - s.add[b]), lb = p / bs, hb = s.blocks(b, bs);
                if (b != last_b || lb != last_lb) {
                    if (lb < hb) {
                        id = a.block_table[b * MB + lb];
                    } else {  // popped: from the stack as it was, or from the row that gives it up
                        const int32_t at = s.have - 1 - (s.need[b] + (int32_t)(lb - hb));
                        if (at < s.F) {
                            id = a.free_blocks[at];
                        } else {
                            const int g = owner(s.give, B, at - s.F);
                            id = a.block_table[g * MB + (int32_t)s.blocks(g, bs) - s.give[g + 1] + (at - s.F)];
                        }
                    }
                    last_b = b;
                    last_lb = lb;
                }
                slot = (int64_t)id * bs + (p - lb * bs);
            }
            a.slot_map[t] = slot;
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1) slots_kernel(const AssignArgs a) {
    extern __shared__ int64_t dyn[];
    pdl_launch_dependents();
    const Sums s = add_up(a, dyn, false);
    write_slots(a, s, (int64_t)blockIdx.x * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.x);
}

__global__ void __launch_bounds__(kThreads, 1) assign_kernel(const AssignArgs a, int with_slots) {
    extern __shared__ int64_t dyn[];
    const int B = a.num_seqs;
    const int64_t MB = a.max_blocks_per_seq;
    const uint32_t bs = (uint32_t)a.block_size, rank = cluster_rank();
    const Sums s = add_up(a, dyn, rank == 0);
    pdl_wait_prior_grid();  // slots_kernel, which read what is changed from here on
    const uint32_t first = rank * blockDim.x + threadIdx.x, stride = kCluster * blockDim.x;
    auto in_pool = [&](int32_t id) {
        if (id < 0 || id >= a.num_blocks) report(a.dev_error, KVC8_DEV_BAD_BLOCK_ID);
    };
    // given up: entry w_b + j of b's row
    for (uint32_t x = first; x < (uint32_t)s.R; x += stride) {
        const int b = owner(s.give, B, (int32_t)x);
        const int32_t entry = (int32_t)s.blocks(b, bs) - s.give[b + 1] + (int32_t)x;  // w_b + (x - give[b])
        const int32_t id = a.block_table[b * MB + entry];
        in_pool(id);
        if ((int64_t)s.F + x < a.num_blocks) a.free_blocks[s.F + x] = id;
        else report(a.dev_error, KVC8_DEV_BAD_LENGTH);
    }
    cluster_barrier();
    const int32_t have = s.have;
    // needed: entry h_b + j of b's row
    for (uint32_t k = first; k < (uint32_t)min(s.need_all, have); k += stride) {
        const int b = owner(s.need, B, (int32_t)k);
        if (s.need[b + 1] > have) continue;
        const int32_t id = a.free_blocks[have - 1 - (int32_t)k];
        in_pool(id);
        a.block_table[b * MB + (int32_t)s.blocks(b, bs) + ((int32_t)k - s.need[b])] = id;
    }
    for (uint32_t b = first; b < (uint32_t)B; b += stride) {
        const bool whole = s.served(b);
        if (!whole && s.need[b] <= have) report(a.dev_error, KVC8_DEV_NO_FREE_BLOCK);
        a.lens_out[b] = whole && s.held[b] >= 0 ? a.want[b] : a.held[b];
    }
    if (rank == 0 && threadIdx.x == 0) {
        // the last sequence that is served says how many were popped
        int32_t taken = s.need_all;
        if (taken > have) taken = s.need[owner(s.need, B + 1, have)];
        *a.free_count_out = have - taken;
        if (a.slot_map != nullptr && s.add_all > a.slot_rows) report(a.dev_error, KVC8_DEV_OUT_ROW_RANGE);
    }
    if (with_slots != 0) write_slots(a, s, first, stride);
}

size_t shared_bytes(int B) { return sizeof(int64_t) * ((size_t)B + 1) + sizeof(int32_t) * (3 * (size_t)B + 2); }

}  // namespace

// Slots beyond which they are made on all SMs.  us a call in a graph, in the cluster / with a kernel of their own:
//   sequences   4096 slots     16 384        32 768        36 864       131 072       819 200
//          16   4.4 /  6.9    6.3 /  7.1    6.5 /  7.1    8.5 /  7.1   13.4 /  7.1   61.6 / 12.7
//         256   5.0 /  7.4    6.9 /  7.5    7.0 /  7.6    9.4 /  7.6   14.4 /  7.6   67.1 / 14.7
//        4096   9.1 / 12.3   10.8 / 11.3                 13.9 / 11.5   18.9 / 11.4   76.7 / 21.5
// The count is the device's, so the room for slots decides: with much room and few slots the second launch is for
// nothing (256 sequences, 1024 slots, room for a million: 5.2 us, 4.2 with room for 1024).
constexpr int64_t kManySlots = 1 << 15;

// Lets both kernels have the shared memory of the largest batch, once per device: the limit is the function's, not
// the launch's, so a limit of a batch's own size could be lowered by another host thread before its launch.
static cudaError_t prepare_launches() {
    static std::atomic<uint64_t> prepared{0};  // a bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < kMaxDevices ? 1ull << dev : 0;
    if ((prepared.load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
    const int most = (int)shared_bytes(KVC8_ASSIGN_MAX_SEQS);
    e = cudaFuncSetAttribute(assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) prepared.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

cudaError_t launch_assign(const AssignArgs &a, cudaStream_t stream) {
    const size_t smem = shared_bytes(a.num_seqs);
    if (smem > 48 * 1024) {
        const cudaError_t e = prepare_launches();
        if (e != cudaSuccess) return e;
    }
    const bool many_slots = a.slot_map != nullptr && a.slot_rows > kManySlots;
    if (many_slots) {
        const int64_t ctas = (a.slot_rows + kThreads * kRun - 1) / (kThreads * kRun), sms = sm_count();
        slots_kernel<<<(unsigned)(ctas < sms ? ctas : sms), kThreads, smem, stream>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    // Small CTAs start and meet sooner (256 sequences, 1150 slots: 5.8 us with 256 threads, 6.2 with 1024, 8.2 in one CTA),
    // as long as they have a thread to a sequence and to a slot (16 sequences, 32 768 slots, in a graph: 8.5 and 6.5 us).
    const int64_t slots = a.slot_map != nullptr ? a.slot_rows : 0;
    const int threads = a.num_seqs <= kFewThreads && slots <= kFewThreads * kCluster ? kFewThreads : kThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // the sums are made while slots_kernel runs
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = many_slots ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, assign_kernel, a, a.slot_map != nullptr && !many_slots ? 1 : 0);
}

}  // namespace kvc8
