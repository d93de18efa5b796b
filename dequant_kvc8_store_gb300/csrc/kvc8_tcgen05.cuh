// kvc8_tcgen05.cuh -- what the kernels with tcgen05 products (the shared-prefix and the tree
// attention) have in common: barriers, tensor memory and products, operands in the 128-byte
// swizzle, codes and their scales as fp16 operand tiles, and the largest of a row's scores.
#pragma once

#include "kvc8_codes.cuh"
#include "kvc8_internal.cuh"

namespace kvc8 {

constexpr int kRows = 128;  // query rows of a tile
constexpr int kCols = 128;  // positions of a step
// The weights are 2^(score - m) with m below the largest score by kLift when it is set, and
// m moves when a score passes it by kLift + kLazy more: the fp16 weights use fp16's range
// up to 2^15, and one of 2^-21 of the row's largest still has all its eleven bits.
constexpr float kLazy = 8.0f, kLift = 7.0f;
// The least exponent taken out of value scales, so that the sum of such weights (up to 2^15)
// times 2^-e over 2^31 positions is finite.  Scales below 2^-74 then lie under fp16's normal
// range: they and their products with a code are off by 2^-85 each, a value by 2^-78.
constexpr int kLeastValuePower = -60;

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
// Waits have a limit: about two seconds.
constexpr long long kWaitCycles = 4000000000ll;
// false: the limit ran out here or, by `stop`, elsewhere in the CTA.
__device__ __forceinline__ bool wait_limited(uint64_t &b, uint32_t parity, int32_t &stop, int32_t *dev_error) {
    const uint32_t at = smem_u32(&b);
    if (mbar_try(at, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try(at, parity)) {
        if (*static_cast<volatile int32_t *>(&stop) != 0) return false;
        if (clock64() - t0 > kWaitCycles) {
            *static_cast<volatile int32_t *>(&stop) = 1;
            report(dev_error, KVC8_DEV_TIMEOUT);
            return false;
        }
    }
    return true;
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

// ---- loads ahead ----------------------------------------------------------------------

// Loads whose place in the program matters: a step's scales and block ids are asked for steps
// before they are used, and the compiler, free to, moves such a load down to its use.
__device__ __forceinline__ float ld_ahead_f32(const float *p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float4 ld_ahead_f32x4(const float *p) {
    float4 v;
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ int32_t ld_ahead_s32(const int32_t *p) {
    int32_t v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// ---- scores ------------------------------------------------------------------------

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Largest of a group of 16.
__device__ __forceinline__ float top16(const float (&s)[32], int i0) {
    const float t0 = max3(s[i0], s[i0 + 1], s[i0 + 2]), t1 = max3(s[i0 + 3], s[i0 + 4], s[i0 + 5]);
    const float t2 = max3(s[i0 + 6], s[i0 + 7], s[i0 + 8]), t3 = max3(s[i0 + 9], s[i0 + 10], s[i0 + 11]);
    const float t4 = max3(s[i0 + 12], s[i0 + 13], s[i0 + 14]);
    return max3(max3(t0, t1, t2), max3(t3, t4, s[i0 + 15]), -INFINITY);
}

// ---- codes as operand tiles -----------------------------------------------------------

// A dequantising warp's share of a tile of 128 positions: RPW of them, codes from global memory
// to registers in whole lines of 512 bytes, from there as fp16 to shared memory.
template <int MODE, int D, int RPW>
struct CodeTile {
    static constexpr int kGroups = RPW / 16;  // a group of 16 positions lies in one block
    static constexpr int kRpl = 512 / D;      // positions of one load
    static constexpr int kLoads = RPW / kRpl;

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
    __device__ __forceinline__ static void store_load(const uint4 &c, int i, uint32_t scale, uint32_t at, uint32_t c0, uint32_t c1,
                                                      int r) {
        const uint32_t wd[4] = {c.x, c.y, c.z, c.w};
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
    // load(i): the codes of the i-th load; UNROLL of them at once.
    template <int UNROLL, typename Load>
    __device__ __forceinline__ static void store_each(Load &&load, uint32_t scale, uint32_t tile, int dw, int lane) {
        const int n = (lane & 3) * 2, r = row_in(lane);
        const uint32_t at = tile + (uint32_t)(dw * RPW + r) * 128 + (uint32_t)block_in(lane) * (kCols * 128);
        const uint32_t c0 = (uint32_t)((n ^ r) << 4), c1 = (uint32_t)(((n + 1) ^ r) << 4);
#pragma unroll UNROLL
        for (int i = 0; i < kLoads; ++i) store_load(load(i), i, scale, at, c0, c1, r);
    }
    __device__ __forceinline__ static void store(const Codes &c, uint32_t scale, uint32_t tile, int dw, int lane) {
        store_each<kLoads>([&](int i) { return c.c[i]; }, scale, tile, dw, lane);
    }
};

}  // namespace kvc8
