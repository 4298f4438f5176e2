// The 8-bit integer linear layer (formulas and conventions: include/int8_linear.h).
//
// GB300's int8 tensor rate is a small fraction of its float16 rate, but int8 values
// are float16 numbers, their products (at most 2^14) are exact in float32, and so is a
// sum of 1,024 of them (at most 2^24).  So the products run on tcgen05 kind::f16, and
// every 1,024 steps of the contraction the tile's float32 sums, whole numbers, are
// added to int32 registers: the result is the exact integer, whatever the codes.
//
// Weights stay int8 in memory and on the way to the SM.  They are the MMA's rows (Y^T =
// Wq Xq^T): converter warps read a row's bytes from shared memory, turn them into
// float16 in registers and put them into tensor memory, from where tcgen05.mma takes
// its A operand.  A byte becomes a float16 by a byte permutation (0x6400 | b is 1024 + b)
// and one subtraction for two.  Shared memory then carries, per 64 steps of a 128 x 192
// tile per CTA, 8 KB of bytes twice and 12 KB of tokens twice; with the weights as an
// operand in shared memory it would be 56 KB, more than its rate allows in the MMAs' time.
// The tokens are quantized to float16 whole numbers by a kernel in front (2 n d bytes).
//
// Tile: 256 weight rows x up to 192 tokens on a pair of SMs (cta_group::2).  Tensor
// memory: two 192-column sums, so that one is drained under the other's products, and
// two slots of 128 steps of A (more where the tile has fewer tokens).
//
// Many tokens are bound by the tensor pipe: 8,192 at 4,096 x 11,008 take 413 us in a CUDA graph,
// 1,790 TFLOP/s and 0.95 of the burst rate of a library's 16-bit GEMM; called one after the other
// 436 us (0.90), at the power cap.  Up to some 600 the bytes of the weights should bound it, but
// what shows is latency: 37 tokens there take 15.8 us for 6.8 of bytes: 2.6 us until the kernel
// in front lets this one start, 3 until the first stage is converted, 8 for 32 stages at some 500
// cycles each and 2 for the last tile's way out.  (That stage cost does not depend on the rows, so
// that the plan keeps 96 of them and 58 of 76 pairs are at work.)
//
// Few tokens do not pay for the trip through tensor memory: one or two take one pass over
// the weights with dp4a, up to 16 (in small layers 32) one with warp-level MMAs.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "codes8.cuh"
#include "device_ptr.h"
#include "int8_linear.cuh"
#include "int8_linear.h"
#include "int8_schedule.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rows8.cuh"
#include "workspace_order.h"

namespace hk {
namespace {

using namespace i8;

constexpr int kMaxStages = 12;
constexpr uint32_t kRing = 208 * 1024;
// Slots of A in tensor memory hold a stage, 64 columns: two of them, or more where the
// tile has fewer tokens.  (Half stages in twice as many slots cost a wait more each:
// 447 us against 415 for 8,192 tokens at 4,096 x 11,008.)
constexpr int kMaxSlots = 6;
constexpr int kLook = 4;  // stages whose barriers are asked for at once
constexpr uint32_t kSlotCols = kKB / 2;
constexpr uint32_t kTmemCols = 512;
static_assert(2 * kMaxTok + 2 * kSlotCols <= kTmemCols, "two sums and two slots");
// Tiles of up to so many tokens have epilogues of their own, which hold fewer sums.
constexpr int kNarrowTok = 64, kMiddleTok = 128;
constexpr int kNumBarriers = 4 * kMaxStages + kMaxSlots + 6;
// Sixteen tokens' results on their way out, of an epilogue half (four warps).
constexpr uint32_t kStagingBytes = 16 * kMaxRows * 2;
constexpr uint32_t kBarAt = kRing + 2 * 2 * kStagingBytes;  // two buffers for each half
constexpr size_t kSmemBytes = 1024 + kBarAt + 8 * kNumBarriers + 16;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
// Warp 0: weights, 2: tokens, 3: MMAs; from 4 on: converters, in groups of four that take the
// stages in turn; then the epilogue.  (Tiles of up to 96 rows have no converter on the MMAs'
// scheduler: 128 tokens at 4,096 x 4,096 17.5 us, 19.1 with warp 1 for the MMAs.)
constexpr int kGroups = 2, kFirstEpiWarp = 4 + 4 * kGroups, kEpiWarps = 8;
constexpr int kThreads = 32 * (kFirstEpiWarp + kEpiWarps);
constexpr unsigned long long kDrainLimitNs = 1000000000ull;
constexpr unsigned long long kAbortSettleNs = 2000000ull;
constexpr int64_t kPieceInts = kMaxTok * kMaxRows;  // one CTA's sums of a unit of a split tile

struct PairParams : Schedule {
    // float16 codes [n, d], boxes of tok/2 rows x 64; weights [f, d], boxes of rows x 128;
    // results [n, f], boxes of 16 tokens x rows
    CUtensorMap x, w, y;
    int32_t stages;
    int32_t slots;       // of A in tensor memory
    uint32_t acc_cols;   // columns of one sum in tensor memory; the slots follow the second
    uint32_t w_bytes, stage_bytes;  // of a stage; the tokens' two boxes follow the weights
    const float *x_scale, *w_scale;
    int32_t* pieces;    // sums of the units of split tiles
    uint32_t* arrived;  // units of each split tile that have come, per CTA; zero between launches
    uint32_t* status;
    unsigned long long timeout_ns;
};

// True in one lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(p));
    return p != 0;
}

// D (M = 256 across the pair) (+)= A[tensor memory] * B[shared memory], f16, issued by the even CTA.
// The descriptor's low word holds the address, and no sum of addresses leaves it.
__device__ __forceinline__ void umma_f16_pair_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t b_high,
                                                 uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_low), "r"(b_high), "r"(idesc), "r"(accumulate)
        : "memory");
}

// `bytes` of global memory into this CTA's shared memory; counted on its `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t (&a)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
          "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15])
        : "r"(t)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t (&a)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
        "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(a[4]), "r"(a[5]), "r"(a[6]), "r"(a[7]), "r"(a[8]), "r"(a[9]),
        "r"(a[10]), "r"(a[11]), "r"(a[12]), "r"(a[13]), "r"(a[14]), "r"(a[15]), "r"(a[16]), "r"(a[17]), "r"(a[18]),
        "r"(a[19]), "r"(a[20]), "r"(a[21]), "r"(a[22]), "r"(a[23]), "r"(a[24]), "r"(a[25]), "r"(a[26]), "r"(a[27]),
        "r"(a[28]), "r"(a[29]), "r"(a[30]), "r"(a[31])
        : "memory");
}

// Whether the phase with parity `parity` of `bar` has completed by now.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// As mbar_wait, for barriers that have mostly completed when they are asked: without a
// limit of its own a try_wait answers in 16 cycles, with one in 51.
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_soon(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try(bar, parity)) return true;
        if (globaltimer_ns() - t0 >= limit_ns) return false;
    }
}

template <class T>
__device__ __forceinline__ T rounded(float x);
template <>
__device__ __forceinline__ __half rounded<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 rounded<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// The epilogue warps' barrier, and whether any thread came with `x`.
__device__ __forceinline__ bool epi_barrier_any(bool x) {
    uint32_t any;
    __syncwarp();  // lanes may come from a wait one by one
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(static_cast<uint32_t>(x)), "n"(kEpiWarps * 32)
        : "memory");
    return any != 0;
}

// Quantization of a token, as rows8_quantize does it (see rows8.cu): codes are rint of
// the exact quotient x / s.
template <class T>
__device__ __forceinline__ float2 unpack2f(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2f<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2f<__half>(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}

// The largest magnitude of eight values, as float32 bits.
template <class T>
__device__ __forceinline__ uint32_t top_of8(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.u16x2 %0, %1, %2;" : "=r"(top) : "r"(top), "r"(w[i] & 0x7fff7fffu));
    return __float_as_uint(unpack2f<T>(max(top >> 16, top & 0xffffu)).x);
}

struct TokenScale {
    float stored;     // the scale; NaN where a value is not finite
    float up, s, r;   // values and scale are both taken `up` times (2^64 for a small scale), 1/s
};
__device__ __forceinline__ TokenScale token_scale(uint32_t top) {
    TokenScale k;
    const bool finite = top < 0x7f800000u;
    k.s = finite ? __fdiv_rn(__uint_as_float(top), 127.0f) : 0.0f;
    k.stored = finite ? k.s : __uint_as_float(0x7fffffffu);
    k.up = k.s < kLiftBelow ? kLift : 1.0f;
    k.s = __fmul_rn(k.s, k.up);
    k.r = k.s > 0.0f ? __frcp_rn(k.s) : 0.0f;
    return k;
}
__device__ __forceinline__ int token_code(float x, const TokenScale& k) {
    x = __fmul_rn(x, k.up);
    return nearest_code(fminf(fmaxf(__fmul_rn(x, k.r), -127.0f), 127.0f), x, k.s);
}
// Eight codes, as bytes.
template <class T>
__device__ __forceinline__ uint2 codes_of8(const uint4& v, const TokenScale& k) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float2 a = unpack2f<T>(w[2 * i]), b = unpack2f<T>(w[2 * i + 1]);
        const int q0 = token_code(a.x, k), q1 = token_code(a.y, k), q2 = token_code(b.x, k), q3 = token_code(b.y, k);
        out[i] = __byte_perm(__byte_perm(q0, q1, 0x0040), __byte_perm(q2, q3, 0x0040), 0x5410);
    }
    return k.s > 0.0f ? make_uint2(out[0], out[1]) : make_uint2(0u, 0u);
}

// Every wait is bounded.  The launch before this one is the kernel that writes the
// tokens' codes and scales; it waits for all work before it and only then lets this
// one start, so that only what it writes itself has to be waited for here.
// kTok: the most tokens of a tile.
template <class T, int kTok>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    int8_pair_kernel(const __grid_constant__ PairParams p) {
    constexpr int kCols = kTok / 2;  // tokens of an epilogue thread
    static_assert(kCols % 16 == 0, "sixteen tokens at a time");
    // registers of a thread after the split; the launch has 65,536 / threads for each, in eights
    constexpr int kServeRegs = 40, kConvRegs = 80, kEpiRegs = 136;
    static_assert(128 * kServeRegs + 128 * kGroups * kConvRegs + 32 * kEpiWarps * kEpiRegs <=
                      kThreads * (65536 / kThreads / 8 * 8),
                  "registers");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + kBarAt;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + kBarAt + 8 * kNumBarriers);
    auto wfull_bar = [&](int s) { return bar0 + 8u * s; };                      // this CTA's weights have landed
    auto wempty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };      // its converters have read them
    auto xfull_bar = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };   // even CTA: the pair's tokens
    auto done_bar = [&](int s) { return bar0 + 8u * (3 * kMaxStages + s); };    // MMAs have read them, and their slot of A
    auto afull_bar = [&](int s) { return bar0 + 8u * (4 * kMaxStages + s); };   // even CTA: the pair's slot of A
    auto accf_bar = [&](int b) { return bar0 + 8u * (4 * kMaxStages + kMaxSlots + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (4 * kMaxStages + kMaxSlots + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (4 * kMaxStages + kMaxSlots + 4), piece_bar = drain_bar + 8u;
    __shared__ volatile int aborted;
    __shared__ volatile int epi_last;
    __shared__ float4 epi_scales[2][kCols / 4];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
    const unsigned long long limit = p.timeout_ns;

    if (threadIdx.x == 0) {
        const int busy = (p.rows + 31) / 32;  // converter warps of a group that have rows
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(wfull_bar(s), 1);
            mbar_init(wempty_bar(s), static_cast<uint32_t>(busy));
            mbar_init(xfull_bar(s), 1);
            mbar_init(done_bar(s), 1);
        }
        for (int s = 0; s < p.slots; ++s) mbar_init(afull_bar(s), 2 * static_cast<uint32_t>(busy));  // of each CTA
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), 2 * kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        mbar_init(piece_bar, 1);
        aborted = 0;
        fence_barrier_init();
        prefetch_tensormap(&p.w);
        prefetch_tensormap(&p.x);
        prefetch_tensormap(&p.y);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    // through a reduction, so that it lands in a uniform register
    const uint32_t tmem = __reduce_max_sync(~0u, *reinterpret_cast<volatile uint32_t*>(tmem_slot));

    if (warp < 4) {
        setmaxnreg_dec<kServeRegs>();
        if (warp == 0 && lane == 0) {
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            for (int u = pair; ok && u < p.n_units; u += n_pairs) {
                const Unit un = unit_at(p, u);
                const int row = un.f0 + static_cast<int>(rank) * p.rows;
                for (int kb = un.kb0; kb < un.kb1; ++kb) {
                    if (!mbar_wait_soon(wempty_bar(stage), phase ^ 1u, limit)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(wfull_bar(stage), static_cast<uint32_t>(p.rows) * kKB);
                    tma_load_2d(base + stage * p.stage_bytes, &p.w, wfull_bar(stage), kb * kKB, row);
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                atomicOr(p.status, kStatusTimeoutLoad);
                aborted = 1;
            }
        } else if (warp == 2 && lane == 0) {
            bool ok = true;
            int stage = 0;
            uint32_t phase = 0;
            const uint32_t box = static_cast<uint32_t>(p.tok) * 64u;  // tok / 2 rows of 128 bytes
            Unit un = unit_at(p, pair);
            griddep_wait();
            griddep_launch_dependents();
            for (int u = pair; ok && u < p.n_units; u += n_pairs) {
                if (u != pair) un = unit_at(p, u);
                const int row = un.t0 + static_cast<int>(rank) * (p.tok / 2);
                for (int kb = un.kb0; kb < un.kb1; ++kb) {
                    if (!mbar_wait_soon(done_bar(stage), phase ^ 1u, limit)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = base + stage * p.stage_bytes + p.w_bytes;
                    const uint32_t fb = mapa_shared(xfull_bar(stage), 0);
                    if (rank == 0) mbar_arrive_expect_tx(xfull_bar(stage), 4 * box);
                    tma_load_2d_pair(at, &p.x, fb, kb * kKB, row);
                    tma_load_2d_pair(at + box, &p.x, fb, kb * kKB + 64, row);
                    if (++stage == p.stages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) {
                atomicOr(p.status, kStatusTimeoutLoad);
                aborted = 1;
            }
        } else if (warp == 3 && rank == 0) {
            // The whole warp takes every turn, waits and agrees on the outcome, and one
            // elected lane issues: control flow and operands then stay uniform (an MMA
            // every 40 cycles; 74 from code of one lane).
            bool ok = true;
            int stage = 0, ab = 0;
            uint32_t slot = 0, phase = 0, sphase = 0, aphase = 0;
            // float32 sums, float16 operands, both contiguous along the contraction
            const uint32_t idesc = (1u << 4) | ((static_cast<uint32_t>(p.tok) >> 3) << 17) | ((256u >> 4) << 24);
            // descriptors count 16 bytes
            const uint64_t desc = smem_desc_sw128(base + p.w_bytes, 16u, 1024u);
            const uint32_t high = static_cast<uint32_t>(desc >> 32), first = static_cast<uint32_t>(desc);
            const uint32_t next = p.stage_bytes >> 4, half = static_cast<uint32_t>(p.tok) * 4u;
            uint32_t b = first;
            // A barrier's answer takes some 120 cycles, so that of a few stages (no more than
            // there are slots, whose parity would tell of an earlier use) is asked for at once.
            const int look = p.slots < kLook ? p.slots : kLook, ahead = (lane >> 1) < look ? lane >> 1 : 0;
            int known = 0;
            for (int u = pair; ok && u < p.n_units; u += n_pairs) {
                const Unit un = unit_at(p, u);
                for (int c0 = un.kb0; ok && c0 < un.kb1; c0 += kChunk) {
                    ok = warp_came(mbar_wait_soon(acce_bar(ab), aphase ^ 1u, limit));
                    if (!ok) break;
                    const uint32_t acc = tmem + static_cast<uint32_t>(ab) * p.acc_cols;
                    const int c1 = c0 + kChunk < un.kb1 ? c0 + kChunk : un.kb1;
                    for (int kb = c0; kb < c1; ++kb) {
                        const auto four = [&](uint32_t a, uint32_t at, uint32_t add) {
                            umma_f16_pair_ta(acc, a, at, high, idesc, add);
                            umma_f16_pair_ta(acc, a + 8u, at + 2u, high, idesc, 1u);
                            umma_f16_pair_ta(acc, a + 16u, at + 4u, high, idesc, 1u);
                            umma_f16_pair_ta(acc, a + 24u, at + 6u, high, idesc, 1u);
                        };
                        if (kTok == kMaxTok) {
                            ok = warp_came(mbar_wait_soon(xfull_bar(stage), phase, limit) &&
                                           mbar_wait_soon(afull_bar(slot), sphase, limit));
                            if (!ok) break;
                        } else if (known == 0) {
                            // even lanes ask for tokens, odd ones for slots of A, of this stage and those after it
                            int s = stage + ahead, a = static_cast<int>(slot) + ahead;
                            uint32_t sp = phase, ap = sphase;
                            if (s >= p.stages) s -= p.stages, sp ^= 1u;
                            if (a >= p.slots) a -= p.slots, ap ^= 1u;
                            const uint32_t bar = lane & 1 ? afull_bar(a) : xfull_bar(s), parity = lane & 1 ? ap : sp;
                            known = (__ffs(~__ballot_sync(~0u, mbar_test(bar, parity)) | 1 << 2 * look) - 1) >> 1;
                            __syncwarp();  // what each lane saw complete is complete for the lane that issues (a ballot orders nothing)
                            if (known == 0) {
                                ok = warp_came(mbar_wait_soon(xfull_bar(stage), phase, limit) &&
                                               mbar_wait_soon(afull_bar(slot), sphase, limit));
                                if (!ok) break;
                                known = 1;
                            }
                        }
                        --known;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t a = tmem + 2 * p.acc_cols + slot * kSlotCols;
                            four(a, b, kb != c0 ? 1u : 0u);
                            four(a + 32u, b + half, 1u);
                            tc_commit_pair_mc(done_bar(stage), 0x3);
                        }
                        __syncwarp();
                        if (++slot == static_cast<uint32_t>(p.slots)) {
                            slot = 0;
                            sphase ^= 1u;
                        }
                        b += next;
                        if (++stage == p.stages) {
                            stage = 0;
                            phase ^= 1u;
                            b = first;
                        }
                    }
                    if (!ok) break;
                    if (elect_one()) tc_commit_pair_mc(accf_bar(ab), 0x3);
                    __syncwarp();
                    if (++ab == 2) {
                        ab = 0;
                        aphase ^= 1u;
                    }
                }
            }
            if (elect_one()) {
                if (!ok) {
                    atomicOr(p.status, kStatusTimeoutMma);
                    aborted = 1;
                }
                // every MMA issued has completed before the pair's memories are released
                tc_commit_pair_mc(drain_bar, 0x1);
                if (!mbar_wait_soon(drain_bar, 0, kDrainLimitNs)) atomicOr(p.status, kStatusTimeoutDrain);
            }
            __syncwarp();
        }
    } else if (warp < kFirstEpiWarp) {
        // Converters: a thread owns one weight row, in every kGroups-th stage.
        setmaxnreg_dec<kConvRegs>();
        const int h = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const bool some = (warp & 3) * 32 < p.rows, mine = row < p.rows;
        const uint32_t afull0 = mapa_shared(afull_bar(0), 0);
        bool ok = true;
        int stage = h, slot = h, skip = h;
        int before = h - p.slots;  // the stage whose slot of A this one takes over
        uint32_t phase = 0, bphase = 0;
        for (int u = pair; ok && some && u < p.n_units; u += n_pairs) {
            const Unit un = unit_at(p, u);
            int kb = un.kb0 + skip;
            for (; kb < un.kb1; kb += kGroups) {
                bool come = mbar_wait_soon(wfull_bar(stage), phase, limit);
                const uint32_t src = base + stage * p.stage_bytes + row * 128u;
                const auto load = [&](int j) {
                    return mine ? lds128(src + ((j ^ (row & 7)) << 4)) : make_uint4(0, 0, 0, 0);
                };
                const auto widen16 = [](const uint4& v, uint32_t* a) {
                    widen4(v.x, a[0], a[1]);
                    widen4(v.y, a[2], a[3]);
                    widen4(v.z, a[4], a[5]);
                    widen4(v.w, a[6], a[7]);
                };
                uint32_t a[32];
#pragma unroll
                for (int j = 0; j < 4; ++j) widen16(load(j), a + 8 * j);
                if (before >= 0) come = mbar_wait_soon(done_bar(before), bphase, limit) && come;
                // The warp goes on together or not at all: each lane's waits have a clock of their own, and
                // lanes that gave up alone would be waited for below without a limit.  (What was
                // read above after a wait that ran out goes nowhere.  A vote for each wait spills.)
                ok = warp_came(come);
                if (!ok) break;
                tc_fence_after();
                const uint32_t to = tmem + lanes + 2 * p.acc_cols + static_cast<uint32_t>(slot) * kSlotCols;
                tmem_st32(to, a);
#pragma unroll
                for (int j = 0; j < 4; ++j) widen16(load(4 + j), a + 8 * j);
                tmem_st32(to + 32u, a);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_cluster_relaxed(afull0 + 8u * slot);
                    mbar_arrive(wempty_bar(stage));
                }
                slot += kGroups;
                if (slot >= p.slots) slot -= p.slots;
                before += kGroups;
                if (before >= p.stages) {
                    before -= p.stages;
                    bphase ^= 1u;
                }
                stage += kGroups;
                if (stage >= p.stages) {
                    stage -= p.stages;
                    phase ^= 1u;
                }
            }
            skip = kb - un.kb1;
        }
        if (!ok && lane == 0) {
            atomicOr(p.status, kStatusTimeoutLoad);
            aborted = 1;
        }
    } else {
        // Epilogue: a thread owns one weight row (an output channel) and every other
        // sixteen tokens: of the first four warps the even ones, of the others the odd.
        setmaxnreg_inc<kEpiRegs>();
        griddep_wait();
        const int q = warp & 3, row = q * 32 + lane;
        const int group = (warp - kFirstEpiWarp) >> 2, first = group * 16;
        const bool leader = q == 0 && lane == 0;
        const uint32_t buffers = base + kRing + group * (2 * kStagingBytes);
        uint32_t buffer = buffers;
        const uint32_t acce0 = mapa_shared(acce_bar(0), 0);
        const auto half_barrier = [&] {
            __syncwarp();  // the barrier takes whole warps, and lanes may come from a branch of their own
            asm volatile("bar.sync %0, 128;" ::"r"(2 + group) : "memory");
        };
        // A half's four warps write one buffer while the other is on its way.
        const auto begin = [&] {
            if (leader) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            half_barrier();
        };
        const auto end = [&](auto issue) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            half_barrier();
            if (leader) {
                issue();
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            buffer = buffer == buffers ? buffers + kStagingBytes : buffers;
        };
        bool failed = false;
        int ab = 0;
        uint32_t aphase = 0;
        int32_t sum[kCols];
        for (int u = pair; u < p.n_units; u += n_pairs) {
            const Unit un = unit_at(p, u);
#pragma unroll
            for (int c = 0; c < kCols; ++c) sum[c] = 0;
            // the scales, on their way while the sums are made
            const int ch = un.f0 + static_cast<int>(rank) * p.rows;
            const float sw = row < p.rows && ch + row < p.f ? p.w_scale[ch + row] : 0.0f;
            if (row < kCols) {
                const int t = un.t0 + first + 2 * (row & ~15) + (row & 15);
                reinterpret_cast<float*>(epi_scales[group])[row] = t < p.n ? p.x_scale[t] : 0.0f;
            }
            for (int c0 = un.kb0; c0 < un.kb1; c0 += kChunk) {
                // the warps agree on whether a wait ran out, so that all of them pass the
                // same barriers
                failed = epi_barrier_any(failed || !mbar_wait_soon(accf_bar(ab), aphase, limit));
                tc_fence_after();
                if (!failed) {
                    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(ab) * p.acc_cols;
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        const int at = first + 2 * c;
                        if (at < p.tok) {
                            uint32_t v[16];
                            tmem_ld16(acc + at, v);
#pragma unroll
                            for (int i = 0; i < 16; ++i) sum[c + i] += __float2int_rn(__uint_as_float(v[i]));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(acce0 + 8u * ab);
                if (++ab == 2) {
                    ab = 0;
                    aphase ^= 1u;
                }
            }
            // Sixteen tokens' results, from the sums v on.
            const auto finish = [&](int c, const int32_t* v) {
                const int at = first + 2 * c;
                begin();
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 k = epi_scales[group][(c + i) / 4];
                    const float s4[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const T y = rounded<T>(__fmul_rn(__int2float_rn(v[i + j]), __fmul_rn(s4[j], sw)));
                        uint16_t bits;
                        memcpy(&bits, &y, 2);
                        if (row < p.rows)
                            asm volatile("st.shared.b16 [%0], %1;" ::"r"(buffer + ((i + j) * p.rows + row) * 2), "h"(bits)
                                         : "memory");
                    }
                }
                end([&] {
                    if (ch < p.f && un.t0 + at < p.n)
                        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                                         reinterpret_cast<uint64_t>(&p.y)),
                                     "r"(buffer), "r"(ch), "r"(un.t0 + at)
                                     : "memory");
                });
            };
            bool complete = !failed;
            if (un.parts > 1) {
                // pieces: [token / 4][row][4], so that a thread moves 16 bytes at a time
                const auto piece = [&](int k) {
                    return reinterpret_cast<int4*>(p.pieces + (2 * static_cast<int64_t>(un.split * un.parts + k) + rank) * kPieceInts);
                };
                if (!failed) {
                    int4* const to = piece(un.part) + row;
#pragma unroll
                    for (int c = 0; c < kCols; c += 16) {
                        const int at = first + 2 * c;
                        if (at < p.tok) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                __stcg(to + (at + i) / 4 * kMaxRows,
                                       make_int4(sum[c + i], sum[c + i + 1], sum[c + i + 2], sum[c + i + 3]));
                        }
                    }
                    asm volatile("fence.proxy.async;" ::: "memory");  // they will be read by a bulk copy
                    __threadfence();
                }
                epi_barrier_any(false);
                if (warp == kFirstEpiWarp && lane == 0) {
                    uint32_t* const count = p.arrived + 2 * un.split + rank;
                    const bool last = !failed && atomicAdd(count, 1u) == static_cast<uint32_t>(un.parts - 1);
                    if (last) *count = 0;
                    epi_last = last;
                }
                epi_barrier_any(false);
                complete = epi_last != 0;
                // The others' pieces by way of the ring, as many as fit: a pair has at most one
                // unit of a split tile, its last, and all that the ring was filled for has been read.
                const uint32_t bytes = static_cast<uint32_t>(p.tok) * (kMaxRows * 4);
                const int fit = static_cast<int>(kRing / bytes);
                for (int k = 1, round = 0; complete && k < un.parts; k += fit, ++round) {
                    const int many = fit < un.parts - k ? fit : un.parts - k;
                    if (warp == kFirstEpiWarp && lane == 0) {
                        __threadfence();
                        asm volatile("fence.proxy.async;" ::: "memory");
                        mbar_arrive_expect_tx(piece_bar, bytes * static_cast<uint32_t>(many));
                        for (int j = 0; j < many; ++j) {
                            const int from = un.part + k + j < un.parts ? un.part + k + j : un.part + k + j - un.parts;
                            bulk_load(base + j * bytes, piece(from), bytes, piece_bar);
                        }
                    }
                    failed = epi_barrier_any(!mbar_wait_soon(piece_bar, static_cast<uint32_t>(round) & 1u, limit));
                    complete = !failed;
                    if (!complete) break;
                    for (int j = 0; j < many; ++j) {
                        const int4* const from = reinterpret_cast<const int4*>(gbase + j * bytes) + row;
#pragma unroll
                        for (int c = 0; c < kCols; c += 16) {
                            const int at = first + 2 * c;
                            if (at < p.tok) {
#pragma unroll
                                for (int i = 0; i < 16; i += 4) {
                                    const int4 v = from[(at + i) / 4 * kMaxRows];
                                    sum[c + i] += v.x, sum[c + i + 1] += v.y, sum[c + i + 2] += v.z, sum[c + i + 3] += v.w;
                                }
                            }
                        }
                    }
                    epi_barrier_any(false);  // the ring may be written again
                }
                epi_barrier_any(false);  // epi_last may be written again
            }
            if (complete) {
#pragma unroll
                for (int c = 0; c < kCols; c += 16)
                    if (first + 2 * c < p.tok) finish(c, sum + c);
            }
            half_barrier();  // the scales may be written again
        }
        if (leader) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        if (failed && lane == 0) {
            atomicOr(p.status, kStatusTimeoutEpilogue);
            aborted = 1;
        }
    }

    // After a timeout copies still in flight (a CTA cannot watch all of its own: the
    // tokens' count on the even CTA's barrier) get time to land before the memory goes.
    __syncthreads();
    if (aborted != 0) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kAbortSettleNs) __nanosleep(1000);
    }
    __syncwarp();  // each lane has a clock of its own
    tc_fence_before();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

// ------------------------------------------------------------- few tokens
//
// Reading the weights once is what takes time, so every SM takes the same number of weight
// rows and streams them straight into registers, in the order of memory; the part that
// does not fit there is on its way to L2 while the tokens are quantized.  A thread owns
// kGran granules of 16 columns and keeps their codes of all kTok tokens in registers; `wr` warps
// cover a row, and the CTA's warps cover `rp` rows side by side.  Four dp4a a granule
// and token, one warp reduction a row and token (the more granules, the fewer), integer
// adds in shared memory across warps: exact and independent of the order.
// One token at 4,096 x 11,008: 10.3 us, 4.4 TB/s; at 8,192 x 28,672: 39.0 us, 6.0 TB/s (CUDA
// graphs of calls on weights from HBM, as the figures below).

constexpr int kFewThreads = 512, kFewWarps = kFewThreads / 32;
constexpr int kFewAhead = 256 * 1024;  // bytes a CTA asks into L2

struct FewParams {
    const void* x;          // 16-bit activations, or NULL:
    const int8_t* x_codes;  // 8-bit rows
    const float* x_scale;
    const int8_t* w;
    const float* w_scale;
    void* out;
    int32_t n, d, f;
    int32_t wr, rp;      // warps of a row, rows side by side
    int32_t rows;        // rows of a CTA
};

// The codes of the tokens into shared memory, [kTok][d], by all warps: kFewWarps / kTok of
// them take a token.
template <class T, int kTok>
__device__ __forceinline__ void few_quantize(const FewParams& p, int8_t* codes, uint32_t (&tops)[kFewWarps],
                                             float (&scales)[kTok]) {
    constexpr int kEach = kFewWarps / kTok;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int token = warp / kEach, first = (warp - token * kEach) * 32 + lane, granules = p.d >> 3;
    const bool some = token < p.n;
    const uint4* const row = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + static_cast<int64_t>(some ? token : 0) * p.d);
    uint32_t top = 0;
    if (some)
        for (int g = first; g < granules; g += kEach * 32) top = max(top, top_of8<T>(row[g]));
    top = __reduce_max_sync(~0u, top);
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    if (!some) return;
#pragma unroll
    for (int i = 0; i < kEach; ++i) top = max(top, tops[token * kEach + i]);
    const TokenScale k = token_scale(top);
    if (first == 0) scales[token] = k.stored;
    for (int g = first; g < granules; g += kEach * 32)  // from L1 this time
        *reinterpret_cast<uint2*>(codes + static_cast<int64_t>(token) * p.d + 8 * g) = codes_of8<T>(row[g], k);
}

template <class T, int kTok, int kGran>
__global__ void __launch_bounds__(kFewThreads, 1) int8_few_kernel(const __grid_constant__ FewParams p) {
    constexpr int kBatch = 8 / kGran;  // rows a thread has in flight
    extern __shared__ uint4 few_smem[];
    int32_t* const sums = reinterpret_cast<int32_t*>(few_smem);  // [rows][kTok], then the tokens' codes
    int8_t* const codes = reinterpret_cast<int8_t*>(few_smem + (p.rows * kTok + 3) / 4);
    __shared__ uint32_t tops[kFewWarps];
    __shared__ float scales[kTok];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row0 = blockIdx.x * p.rows;
    const int rows = p.f - row0 < p.rows ? p.f - row0 : p.rows;
    const int at = warp / p.wr;                                  // which of the rows side by side
    const int g0 = (warp - at * p.wr) * 32 + lane;               // first granule
    const int gs = p.wr * 32, granules = p.d >> 4;
    const int8_t* const w = p.w + static_cast<int64_t>(row0) * p.d;
    {
        // (may run under the end of the stream's previous kernel: nothing is read by it)
        const int64_t bytes = static_cast<int64_t>(rows) * p.d, from = static_cast<int64_t>(threadIdx.x) * 8192;
        const int64_t to = bytes < kFewAhead ? bytes : kFewAhead;
        if (from < to) prefetch_l2_bulk(w + from, static_cast<uint32_t>(to - from < 8192 ? to - from : 8192));
    }
    for (int i = threadIdx.x; i < rows * kTok; i += kFewThreads) sums[i] = 0;
    griddep_wait();
    griddep_launch_dependents();

    uint4 v[kBatch][kGran];
    const auto fetch = [&](int r0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int j = 0; j < kGran; ++j) {
                const int r = r0 + b * p.rp, g = g0 + j * gs;
                v[b][j] = at < p.rp && r < rows && g < granules
                              ? __ldcg(reinterpret_cast<const uint4*>(w + static_cast<int64_t>(r) * p.d) + g)
                              : make_uint4(0, 0, 0, 0);
            }
    };
    fetch(at);

    if (p.x_codes) {
        if (threadIdx.x < kTok && threadIdx.x < p.n) scales[threadIdx.x] = p.x_scale[threadIdx.x];
    } else {
        few_quantize<T, kTok>(p, codes, tops, scales);
    }
    __syncthreads();
    uint4 code[kTok][kGran];
#pragma unroll
    for (int t = 0; t < kTok; ++t)
#pragma unroll
        for (int j = 0; j < kGran; ++j) {
            const int g = g0 + j * gs;
            const int8_t* const from = (p.x_codes ? p.x_codes : codes) + static_cast<int64_t>(t) * p.d;
            code[t][j] = t < p.n && g < granules ? reinterpret_cast<const uint4*>(from)[g] : make_uint4(0, 0, 0, 0);
        }

    if (at < p.rp) {
        for (int r0 = at; r0 < rows; r0 += kBatch * p.rp) {
            int32_t acc[kBatch][kTok];
#pragma unroll
            for (int b = 0; b < kBatch; ++b)
#pragma unroll
                for (int t = 0; t < kTok; ++t) {
                    int32_t a = 0;
#pragma unroll
                    for (int j = 0; j < kGran; ++j) {
                        a = __dp4a(static_cast<int>(v[b][j].x), static_cast<int>(code[t][j].x), a);
                        a = __dp4a(static_cast<int>(v[b][j].y), static_cast<int>(code[t][j].y), a);
                        a = __dp4a(static_cast<int>(v[b][j].z), static_cast<int>(code[t][j].z), a);
                        a = __dp4a(static_cast<int>(v[b][j].w), static_cast<int>(code[t][j].w), a);
                    }
                    acc[b][t] = a;
                }
            if (r0 + kBatch * p.rp < rows) fetch(r0 + kBatch * p.rp);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int r = r0 + b * p.rp;
                int32_t mine = 0;  // lane t keeps token t's sum
#pragma unroll
                for (int t = 0; t < kTok; ++t) {
                    const int32_t a = __reduce_add_sync(~0u, acc[b][t]);
                    if (lane == t) mine = a;
                }
                if (lane < kTok && r < rows) atomicAdd(&sums[r * kTok + lane], mine);
            }
        }
    }
    __syncthreads();
    // channel by channel, so that a warp writes side by side
    for (int i = threadIdx.x; i < rows * kTok; i += kFewThreads) {
        const int t = i / rows, r = i - t * rows;
        if (t < p.n)
            static_cast<T*>(p.out)[static_cast<int64_t>(t) * p.f + row0 + r] =
                rounded<T>(__fmul_rn(__int2float_rn(sums[r * kTok + t]), __fmul_rn(scales[t], p.w_scale[row0 + r])));
    }
}

// ------------------------------------------------------- up to 32 tokens
//
// The weights are read once here, too, but with more products than dp4a has time for:
// warp-level MMAs (m16n8k16, float16, float32 sums) on weights that go from memory
// straight into registers.  A thread's 16 bytes of a row serve four MMAs: the
// contraction's order within 64 columns is free, so it is the bytes' order (thread t of
// a row has columns 16 t .. 16 t + 15; MMA i takes bytes 4 i .. 4 i + 3), and the tokens'
// values are read in the same order.
//
// All CTAs, two per SM, take the same number of weight rows, kTilesM x 16 of them at a
// time, and a CTA's warps share the columns, 64 at a time in turn: so every weight and every
// token's value is read by one warp of the CTA, once, and needs no place in shared
// memory.  A block's weights are fetched two to six blocks ahead, its tokens one.  What bounds
// it is both ways into the SMs: every CTA reads all tokens' float16 values from L2, which for
// 16 tokens are 39 MB beside 45 MB of weights at 4,096 x 11,008, and 103 MB at 11,008 x 4,096.
// With the tokens' quantization in front, at 4,096 x 11,008: 3 tokens 12.6 us (15.0 on pairs of
// SMs), 8 13.2 (15.1 there), 16 15.4 (15.1); 16 at 2,048 x 2,048 5.6 (9.9), but at 11,008 x 4,096
// 19.1 (17.5).

constexpr int kMidThreads = 256, kMidWarps = kMidThreads / 32;
constexpr int kMidFlush = 1024 / 64;  // blocks whose sums stay below 2^24

struct MidParams {
    const __half* x;  // [n, d] whole numbers
    const float *x_scale, *w_scale;
    const int8_t* w;
    void* out;
    int32_t n, d, f, bf16;
    int32_t rows;  // of a CTA
};

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int kTilesM, int kTilesN>
__global__ void __launch_bounds__(kMidThreads, 2) int8_mid_kernel(const __grid_constant__ MidParams p) {
    constexpr int kPitch = kTilesM * 16 + 4;  // of a token's sums: no bank conflicts
    __shared__ int32_t sums[kMidWarps][kTilesN * 8][kPitch];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int row0 = blockIdx.x * p.rows;
    const int row1 = row0 + p.rows < p.f ? row0 + p.rows : p.f;
    const int blocks = (p.d + 63) / 64;
    bool waited = false;
    for (int r0 = row0; r0 < row1; r0 += kTilesM * 16) {
        constexpr int kDepth = kTilesM > 1 ? 2 : kTilesN <= 2 ? 6 : kTilesN == 3 ? 4 : 2;
        uint4 a[kDepth][kTilesM][2], x[2][kTilesN][2];
        // the i-th block of this warp: pairs of neighbours, so that a line of memory is read at once
        const auto block = [&](int i) { return (i >> 1) * (2 * kMidWarps) + 2 * warp + (i & 1); };
        const auto fetch_w = [&](int kb, uint4 (&to)[kTilesM][2]) {
            const int k = kb * 64 + t * 16;
#pragma unroll
            for (int m = 0; m < kTilesM; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int row = r0 + m * 16 + h * 8 + g;
                    to[m][h] = kb < blocks && k < p.d && row < row1
                                   ? __ldcg(reinterpret_cast<const uint4*>(p.w + static_cast<int64_t>(row) * p.d + k))
                                   : make_uint4(0, 0, 0, 0);
                }
        };
        const auto fetch_x = [&](int kb, uint4 (&to)[kTilesN][2]) {
            const int k = kb * 64 + t * 16;
#pragma unroll
            for (int c = 0; c < kTilesN; ++c) {
                const int token = c * 8 + g;
                to[c][0] = to[c][1] = make_uint4(0, 0, 0, 0);
                if (token < p.n && kb < blocks && k < p.d) {
                    const uint4* const src = reinterpret_cast<const uint4*>(p.x + static_cast<int64_t>(token) * p.d + k);
                    to[c][0] = __ldcg(src);
                    to[c][1] = __ldcg(src + 1);
                }
            }
        };
#pragma unroll
        for (int i = 0; i < kDepth; ++i) fetch_w(block(i), a[i]);  // (complete: see int8_pair_kernel)
        for (int i = lane; i < kTilesN * 8 * kPitch; i += 32) (&sums[warp][0][0])[i] = 0;
        __syncwarp();
        if (!waited) {
            griddep_wait();
            griddep_launch_dependents();
            waited = true;
        }
        fetch_x(block(0), x[0]);
        float acc[kTilesM][kTilesN][4] = {};
        int held = 0;
        const auto settle = [&] {
#pragma unroll
            for (int m = 0; m < kTilesM; ++m)
#pragma unroll
                for (int c = 0; c < kTilesN; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sums[warp][c * 8 + 2 * t + (e & 1)][m * 16 + (e >> 1) * 8 + g] += __float2int_rn(acc[m][c][e]);
                        acc[m][c][e] = 0.0f;
                    }
            held = 0;
        };
        const auto work = [&](int at, uint4 (&w)[kTilesM][2], const uint4 (&b)[kTilesN][2], uint4 (&next)[kTilesN][2]) {
            fetch_x(block(at + 1), next);
#pragma unroll
            for (int m = 0; m < kTilesM; ++m) {
                const uint32_t top[4] = {w[m][0].x, w[m][0].y, w[m][0].z, w[m][0].w};
                const uint32_t low[4] = {w[m][1].x, w[m][1].y, w[m][1].z, w[m][1].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a0, a1, a2, a3;
                    widen4(top[i], a0, a2);
                    widen4(low[i], a1, a3);
#pragma unroll
                    for (int c = 0; c < kTilesN; ++c) {
                        const uint4 v = b[c][i >> 1];
                        mma_f16_16816(acc[m][c], a0, a1, a2, a3, i & 1 ? v.z : v.x, i & 1 ? v.w : v.y);
                    }
                }
            }
            fetch_w(block(at + kDepth), w);
            if (++held == kMidFlush) settle();
        };
        for (int at = 0; block(at) < blocks; at += kDepth) {
#pragma unroll
            for (int i = 0; i < kDepth; ++i)
                if (i == 0 || block(at + i) < blocks) work(at + i, a[i], x[i & 1], x[(i + 1) & 1]);
        }
        settle();
        __syncthreads();
        const int rows = row1 - r0 < kTilesM * 16 ? row1 - r0 : kTilesM * 16;
        for (int i = threadIdx.x; i < rows * p.n; i += kMidThreads) {
            const int c = i / rows, r = i - c * rows;
            int32_t total = 0;
#pragma unroll
            for (int w = 0; w < kMidWarps; ++w) total += sums[w][c][r];
            const float y = __fmul_rn(__int2float_rn(total), __fmul_rn(p.x_scale[c], p.w_scale[r0 + r]));
            const int64_t at = static_cast<int64_t>(c) * p.f + r0 + r;
            if (p.bf16) static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
            else static_cast<__half*>(p.out)[at] = __float2half_rn(y);
        }
        __syncthreads();  // the sums may be written again
    }
}

// ------------------------------------------------------------- host side

hess_status il_fail(hess_status s, const char* fmt, ...) {
    char buf[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

#define IL_TRY(call)                                                                           \
    do {                                                                                       \
        cudaError_t e_ = (call);                                                               \
        if (e_ != cudaSuccess)                                                                 \
            return il_fail(HESS_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));     \
    } while (0)
#define IL_CHECK(expr)                       \
    do {                                     \
        const hess_status st_ = (expr);      \
        if (st_ != HESS_OK) return st_;      \
    } while (0)

bool il_injected(const char* what) {
    const char* f = std::getenv("HESS_FAULT");
    return f && std::strcmp(f, what) == 0;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn il_encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<EncodeTiledFn>(p);
        return static_cast<EncodeTiledFn>(nullptr);
    }();
    return fn;
}

// Row-major [rows, cols], boxes of box_rows x box_cols, zeros past the edges.
hess_status il_encode_as(CUtensorMap* m, const void* ptr, CUtensorMapDataType type, int item, int64_t rows, int64_t cols,
                         int64_t box_rows, int64_t box_cols, CUtensorMapSwizzle swizzle) {
    const EncodeTiledFn fn = il_encode_fn();
    if (!fn) return il_fail(HESS_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    if (il_injected("encode"))
        return il_fail(HESS_ERR_UNSUPPORTED, "injected tensor-map failure (HESS_FAULT=encode)");
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * item)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)}, es[2] = {1u, 1u};
    const CUresult r = fn(m, type, 2, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return il_fail(HESS_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled failed (%d) for [%lld, %lld]",
                       static_cast<int>(r), static_cast<long long>(rows), static_cast<long long>(cols));
    return HESS_OK;
}
// Operands: boxes of 128 bytes a row in the 128-byte swizzle.
hess_status il_encode(CUtensorMap* m, const void* ptr, bool bytes, int64_t rows, int64_t cols, int64_t box_rows) {
    return il_encode_as(m, ptr, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, bytes ? 1 : 2,
                        rows, cols, box_rows, bytes ? 128 : 64, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Results: boxes of 16 tokens x the rows of a CTA, as they lie.
hess_status il_encode_out(CUtensorMap* m, void* ptr, int32_t dtype, int64_t rows, int64_t cols, int64_t box_cols) {
    return il_encode_as(m, ptr, dtype == HESS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                        rows, cols, 16, box_cols, CU_TENSOR_MAP_SWIZZLE_NONE);
}

constexpr size_t kFewSmem = 72 * 1024;  // two tokens of 32,768 codes, and sums

template <class T, int kTok>
auto few_kernel(int gran) -> void (*)(FewParams) {
    return gran == 1 ? int8_few_kernel<T, kTok, 1> : gran == 2 ? int8_few_kernel<T, kTok, 2>
                     : gran == 4 ? int8_few_kernel<T, kTok, 4> : int8_few_kernel<T, kTok, 8>;
}

template <class T>
auto pair_kernel(int tok) -> void (*)(PairParams) {
    return tok <= kNarrowTok ? int8_pair_kernel<T, kNarrowTok> : tok <= kMiddleTok ? int8_pair_kernel<T, kMiddleTok>
                                                                                   : int8_pair_kernel<T, kMaxTok>;
}

// Per-device set-up: shared-memory limits, and how many pairs stay resident.
hess_status il_prepare(int dev, int* pairs, int* sms_out) {
    static std::mutex mu;
    static int count[128] = {}, sm_count[128] = {};
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 128) return il_fail(HESS_ERR_UNSUPPORTED, "device index %d", dev);
    if (!count[dev]) {
        for (int gran : {1, 2, 4, 8})
            for (auto fn : {few_kernel<__nv_bfloat16, 1>(gran), few_kernel<__nv_bfloat16, 2>(gran),
                            few_kernel<__half, 1>(gran), few_kernel<__half, 2>(gran)})
                IL_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kFewSmem)));
        for (int tok : {kNarrowTok, kMiddleTok, kMaxTok})
            for (auto fn : {pair_kernel<__nv_bfloat16>(tok), pair_kernel<__half>(tok)})
                IL_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(kSmemBytes)));
        int sms = 0;
        IL_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
        sm_count[dev] = sms;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(sms & ~1), 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = kSmemBytes;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, pair_kernel<__nv_bfloat16>(kMaxTok), &cfg) != cudaSuccess ||
            clusters <= 0) {
            cudaGetLastError();
            clusters = sms / 2;
        }
        count[dev] = clusters;
    }
    *pairs = count[dev];
    *sms_out = sm_count[dev];
    return HESS_OK;
}

}  // namespace
}  // namespace hk

struct int8_linear_ctx {
    std::mutex mu;
    int device = 0;
    int pairs = 0, ff_pairs = 0, sms = 0;
    int64_t d = 0, f = 0, tokens = 0, train_tokens = 0;
    int32_t dtype = 0;
    void* memory = nullptr;  // holds what follows
    uint16_t* wide = nullptr;       // [tokens, d] float16 codes
    float* x_scale = nullptr;       // [tokens]
    int32_t* pieces = nullptr;      // one per pair
    void* w_restored = nullptr;     // [f, d]
    void* x_restored = nullptr;     // [train_tokens, d]
    float* ff_pieces = nullptr;
    uint32_t* status = nullptr;     // the status word, then the arrival counts
    size_t status_bytes = 0;
    hk::WorkspaceOrder order;  // of the calls that use that memory
    unsigned long long timeout_ns = 2000000000ull;
};

namespace hk {
namespace {

hess_status il_check_device(const int8_linear_ctx* g) {
    int cur = -1;
    IL_TRY(cudaGetDevice(&cur));
    if (cur != g->device)
        return il_fail(HESS_ERR_INVALID, "handle belongs to device %d but device %d is current", g->device, cur);
    return HESS_OK;
}

hess_status il_check(const int8_linear_ctx* g, const void* p, const char* name, int align = 16) {
    if (!p) return il_fail(HESS_ERR_INVALID, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align)
        return il_fail(HESS_ERR_INVALID, "%s is not %d-byte aligned", name, align);
    char why[128];
    if (const char* w = device_ptr_problem(p, g->device, why)) return il_fail(HESS_ERR_INVALID, "%s %s", name, w);
    return HESS_OK;
}

struct IlBuffer {
    const void* p;  // NULL: not there
    int64_t bytes;
    const char* name;
};
hess_status il_apart(const IlBuffer& out, const IlBuffer& in) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p), b = reinterpret_cast<uintptr_t>(in.p);
    if (out.p && in.p && a < b + static_cast<uintptr_t>(in.bytes) && b < a + static_cast<uintptr_t>(out.bytes))
        return il_fail(HESS_ERR_INVALID, "%s overlaps %s", out.name, in.name);
    return HESS_OK;
}

hess_status il_tokens(int64_t n, int64_t most, const char* what) {
    if (n < 0) return il_fail(HESS_ERR_INVALID, "n_tokens < 0");
    if (n > most)
        return il_fail(HESS_ERR_INVALID, "n_tokens %lld exceeds the handle's %s %lld", static_cast<long long>(n), what,
                       static_cast<long long>(most));
    return HESS_OK;
}

template <class Kernel, class Params>
hess_status il_launch(Kernel kernel, const Params& p, int64_t grid, int threads, size_t smem, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    IL_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
    return HESS_OK;
}

// Granules of 16 columns a thread of the few-token kernel takes: as many as there are (the
// fewer warps share a row, the fewer sums meet), unless that leaves more threads idle; 0
// where a row is too wide.  (0.85: one token at 5,120 x 13,824 14.6 us, 16.1 with eight always; at
// 4,096 x 4,096 5.5 us, 5.9 with the fewest idle threads alone.)
int few_granules(int64_t d) {
    const int64_t granules = d / 16;
    int best = 0;
    double most = 0.0;
    for (int g = 1; g <= 8; g *= 2) {
        const int64_t wr = ceil_div(granules, 32 * g);
        if (wr > kFewWarps) continue;
        const double used = static_cast<double>(granules) * (kFewWarps / wr) / (32.0 * g * kFewWarps);
        if (used >= 0.85 * most) {
            best = g;
            if (used > most) most = used;
        }
    }
    return best;
}
// One or two tokens whose codes fit beside each other: with three, the sums of every
// token over a warp cost more than tensor cores do (13.6 us either way at 4,096 x 11,008,
// 18.6 against 15.8 for four at 11,008 x 4,096).
bool is_few(int64_t n, int64_t d) { return n <= 2 && n * d <= int64_t(64) * 1024; }

hess_status forward_few(const int8_linear_ctx* g, const void* X, const int8_t* codes, const float* scale, int64_t n,
                        const int8_t* W, const float* W_scale, void* Y, cudaStream_t s) {
    FewParams p{};
    p.x = X;
    p.x_codes = codes;
    p.x_scale = scale;
    p.w = W;
    p.w_scale = W_scale;
    p.out = Y;
    p.n = static_cast<int32_t>(n);
    p.d = static_cast<int32_t>(g->d);
    p.f = static_cast<int32_t>(g->f);
    const int gran = few_granules(g->d), tok = static_cast<int>(n);
    p.wr = static_cast<int32_t>(ceil_div(g->d, static_cast<int64_t>(gran) * 512));
    p.rp = kFewWarps / p.wr;
    const int64_t ctas = g->f < g->sms ? g->f : g->sms;
    p.rows = static_cast<int32_t>(ceil_div(g->f, ctas));
    const int64_t grid = ceil_div(g->f, p.rows);
    const size_t smem = static_cast<size_t>(ceil_div(static_cast<int64_t>(p.rows) * tok, 4)) * 16 + (X ? tok * g->d : 0);
    const auto kernel = g->dtype == HESS_BF16
                            ? (tok == 1 ? few_kernel<__nv_bfloat16, 1>(gran) : few_kernel<__nv_bfloat16, 2>(gran))
                            : (tok == 1 ? few_kernel<__half, 1>(gran) : few_kernel<__half, 2>(gran));
    if (smem > kFewSmem) return il_fail(HESS_ERR_INTERNAL, "%zu bytes of shared memory", smem);
    return il_launch(kernel, p, grid, kFewThreads, smem, s);
}

// The tokens' codes as float16 whole numbers, into the workspace.
hess_status widen_tokens(const int8_linear_ctx* g, const void* X, const int8_t* codes, int64_t n, cudaStream_t s) {
    if (X)
        IL_TRY(rows8_quantize_launch(X, g->d, n, g->d, g->dtype, 0, nullptr, 0, g->wide, g->d, g->x_scale, s));
    else
        IL_TRY(rows8_restore_launch({codes, g->d, nullptr, n, g->d, 0, g->wide, g->d}, {}, HESS_F16, false, s));
    return HESS_OK;
}

// Row tiles that a warp's registers hold, for up to 8 `tiles_n` tokens.
int mid_tiles(int tiles_n) { return tiles_n <= 2 ? 3 : tiles_n == 3 ? 2 : 1; }

template <int kTilesN>
auto mid_kernel(int tiles_m) -> void (*)(MidParams) {
    if constexpr (kTilesN == 4) return int8_mid_kernel<1, 4>;
    else if constexpr (kTilesN == 3) return tiles_m == 1 ? int8_mid_kernel<1, 3> : int8_mid_kernel<2, 3>;
    else
        return tiles_m == 1   ? int8_mid_kernel<1, kTilesN>
               : tiles_m == 2 ? int8_mid_kernel<2, kTilesN>
                              : int8_mid_kernel<3, kTilesN>;
}

int64_t mid_rows(const int8_linear_ctx* g) { return ceil_div(g->f, 2 * g->sms); }

// From 17 tokens on only small layers, whose rows a CTA takes in one turn: in two turns, or
// over more columns, every CTA's reading of all tokens costs more than the pairs' start
// (24 tokens: 2,048 x 2,048 6.4 us against 10.0, 4,096 x 8,192 13.8 against 14.8, but, by an
// earlier measurement, 8,192 x 2,048 17.5 against 14.3; 32 at 4,096 x 4,096 11.9 against 12.8, at
// 2,560 x 6,912, two turns, 18.4 against 12.4).
bool is_mid(const int8_linear_ctx* g, int64_t n) {
    const int tiles_n = static_cast<int>(ceil_div(n, 8));
    return tiles_n <= 2 || (tiles_n <= 4 && g->d <= 4096 && mid_rows(g) <= 16 * mid_tiles(tiles_n));
}

hess_status forward_mid(int8_linear_ctx* g, const void* X, const int8_t* codes, const float* scale, int64_t n,
                        const int8_t* W, const float* W_scale, void* Y, cudaStream_t s) {
    MidParams p{};
    p.x = reinterpret_cast<const __half*>(g->wide);
    p.x_scale = X ? g->x_scale : scale;
    p.w_scale = W_scale;
    p.w = W;
    p.out = Y;
    p.n = static_cast<int32_t>(n);
    p.d = static_cast<int32_t>(g->d);
    p.f = static_cast<int32_t>(g->f);
    p.bf16 = g->dtype == HESS_BF16;
    p.rows = static_cast<int32_t>(mid_rows(g));
    const int tiles_n = static_cast<int>(ceil_div(n, 8));
    const int64_t tiles = ceil_div(p.rows, 16), turns = ceil_div(tiles, mid_tiles(tiles_n));
    const int tiles_m = static_cast<int>(ceil_div(tiles, turns));
    const auto kernel = tiles_n <= 1   ? mid_kernel<1>(tiles_m)
                        : tiles_n == 2 ? mid_kernel<2>(tiles_m)
                        : tiles_n == 3 ? mid_kernel<3>(tiles_m)
                                       : mid_kernel<4>(tiles_m);
    IL_TRY(g->order.begin(s));
    IL_CHECK(widen_tokens(g, X, codes, n, s));
    const hess_status st = il_launch(kernel, p, ceil_div(g->f, p.rows), kMidThreads, 0, s);
    IL_TRY(g->order.end(s));
    return st;
}

// X in 16 bits, or codes and scale.
hess_status forward(int8_linear_ctx* g, const void* X, const int8_t* codes, const float* scale, int64_t n,
                    const int8_t* W, const float* W_scale, void* Y, cudaStream_t s) {
    IL_TRY(ensure_context());
    if (is_few(n, g->d)) return forward_few(g, X, codes, scale, n, W, W_scale, Y, s);
    if (is_mid(g, n)) return forward_mid(g, X, codes, scale, n, W, W_scale, Y, s);
    PairParams p{};
    p.n = static_cast<int32_t>(n);
    p.d = static_cast<int32_t>(g->d);
    p.f = static_cast<int32_t>(g->f);
    plan(p, g->pairs);
    p.w_bytes = static_cast<uint32_t>((p.rows + 7) / 8 * 8) * kKB;
    p.stage_bytes = p.w_bytes + static_cast<uint32_t>(p.tok) * 128u;
    const int fit = static_cast<int>(kRing / p.stage_bytes);
    p.stages = fit < kMaxStages ? fit : kMaxStages;
    p.acc_cols = static_cast<uint32_t>((p.tok + 31) / 32 * 32);
    const int slots = static_cast<int>((kTmemCols - 2 * p.acc_cols) / kSlotCols);
    p.slots = slots < kMaxSlots ? slots : kMaxSlots;
    if (p.slots >= p.stages) p.slots = p.stages - 1;  // a stage's barrier tells of one use of a slot
    p.x_scale = X ? g->x_scale : scale;
    p.w_scale = W_scale;
    p.pieces = g->pieces;
    p.arrived = g->status + 1;
    p.status = g->status;
    p.timeout_ns = g->timeout_ns;
    IL_CHECK(il_encode(&p.x, g->wide, false, n, g->d, p.tok / 2));
    IL_CHECK(il_encode(&p.w, W, true, g->f, g->d, p.rows));
    IL_CHECK(il_encode_out(&p.y, Y, g->dtype, n, g->f, p.rows));
    IL_TRY(g->order.begin(s));
    IL_CHECK(widen_tokens(g, X, codes, n, s));
    const int pairs = p.n_units < g->pairs ? p.n_units : g->pairs;
    const hess_status st = il_launch(
        g->dtype == HESS_BF16 ? pair_kernel<__nv_bfloat16>(p.tok) : pair_kernel<__half>(p.tok), p, 2 * pairs, kThreads,
        kSmemBytes, s);
    IL_TRY(g->order.end(s));
    return st;
}

void il_free(int8_linear_ctx* g) {
    cudaFree(g->memory);
    g->order.destroy();
}

}  // namespace
}  // namespace hk

using hk::il_fail;

#define IL_EXPORT extern "C" __attribute__((visibility("default")))

IL_EXPORT hess_status int8_linear_create(int64_t d, int64_t f, int64_t tokens, int64_t train_tokens, int32_t dtype,
                                         int8_linear_t* out) {
    if (!out) return il_fail(HESS_ERR_INVALID, "out is NULL");
    *out = nullptr;
    if (d <= 0 || f <= 0) return il_fail(HESS_ERR_INVALID, "d and f must be positive");
    if (tokens < 0 || train_tokens < 0) return il_fail(HESS_ERR_INVALID, "tokens or train_tokens < 0");
    if (d % 16 || f % 8) return il_fail(HESS_ERR_UNSUPPORTED, "d must be a multiple of 16 and f a multiple of 8");
    if (d > 65536 || f > 65536) return il_fail(HESS_ERR_UNSUPPORTED, "d or f exceeds 65536");
    if (tokens > (int64_t(1) << 26) || train_tokens > (int64_t(1) << 26))
        return il_fail(HESS_ERR_UNSUPPORTED, "tokens or train_tokens > 2^26");
    if (dtype == HESS_F32) return il_fail(HESS_ERR_UNSUPPORTED, "int8_linear takes bf16 or f16");
    if (dtype != HESS_BF16 && dtype != HESS_F16) return il_fail(HESS_ERR_INVALID, "unknown dtype %d", dtype);
    if (hk::il_injected("alloc")) return il_fail(HESS_ERR_OOM, "injected allocation failure (HESS_FAULT=alloc)");
    int dev = 0, pairs = 0, sms = 0, ff_pairs = 0, ff_sms = 0;
    IL_TRY(cudaGetDevice(&dev));
    IL_TRY(hk::ensure_context());
    IL_CHECK(hk::il_prepare(dev, &pairs, &sms));
    if (train_tokens > 0) IL_CHECK(hk::ff_resident_pairs(dev, &ff_pairs, &ff_sms));
    int8_linear_ctx* g = new (std::nothrow) int8_linear_ctx();
    if (!g) return il_fail(HESS_ERR_OOM, "host allocation failed");
    g->device = dev;
    g->pairs = pairs;
    g->ff_pairs = ff_pairs;
    g->sms = sms;
    g->d = d;
    g->f = f;
    g->tokens = tokens;
    g->train_tokens = train_tokens;
    g->dtype = dtype;
    const auto round = [](size_t b) { return (b + 255) / 256 * 256; };
    const size_t wide = round(static_cast<size_t>(tokens) * d * 2), x_scale = round(static_cast<size_t>(tokens) * 4);
    const size_t pieces = tokens > 0 ? static_cast<size_t>(pairs) * 2 * hk::kPieceInts * 4 : 0;
    const size_t w_restored = train_tokens > 0 ? round(static_cast<size_t>(f) * d * 2) : 0;
    const size_t x_restored = round(static_cast<size_t>(train_tokens) * d * 2);
    const size_t ff_pieces = static_cast<size_t>(ff_pairs) * hk::kFfPieceBytes;
    g->status_bytes = (1 + 2 * static_cast<size_t>(pairs) + 2 * static_cast<size_t>(ff_pairs)) * 4;
    cudaError_t e = cudaMalloc(&g->memory, wide + x_scale + pieces + w_restored + x_restored + ff_pieces + g->status_bytes);
    if (e == cudaSuccess) {
        uint8_t* m = static_cast<uint8_t*>(g->memory);
        g->wide = reinterpret_cast<uint16_t*>(m);
        g->x_scale = reinterpret_cast<float*>(m += wide);
        g->pieces = reinterpret_cast<int32_t*>(m += x_scale);
        g->w_restored = m += pieces;
        g->x_restored = m += w_restored;
        g->ff_pieces = reinterpret_cast<float*>(m += x_restored);
        g->status = reinterpret_cast<uint32_t*>(m += ff_pieces);
        e = cudaMemset(g->status, 0, g->status_bytes);
    }
    if (e == cudaSuccess) e = g->order.create();
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        const hess_status s = e == cudaErrorMemoryAllocation ? HESS_ERR_OOM : HESS_ERR_CUDA;
        if (s == HESS_ERR_OOM) cudaGetLastError();
        hk::il_free(g);
        delete g;
        return il_fail(s, "int8_linear_create: %s", cudaGetErrorString(e));
    }
    *out = g;
    return HESS_OK;
}

static hess_status il_forward(int8_linear_t g, const void* X, const int8_t* X_codes, const float* X_scale,
                              bool rows8, int64_t n, const int8_t* W_codes, const float* W_scale, void* Y_out,
                              hess_stream_t stream) {
    if (!g) return il_fail(HESS_ERR_INVALID, "handle is NULL");
    IL_CHECK(hk::il_tokens(n, g->tokens, "tokens"));
    if (n == 0) return HESS_OK;
    std::lock_guard<std::mutex> lk(g->mu);
    IL_CHECK(hk::il_check_device(g));
    if (rows8) {
        IL_CHECK(hk::il_check(g, X_codes, "X_codes"));
        IL_CHECK(hk::il_check(g, X_scale, "X_scale", 4));
    } else {
        IL_CHECK(hk::il_check(g, X, "X"));
    }
    IL_CHECK(hk::il_check(g, W_codes, "W_codes"));
    IL_CHECK(hk::il_check(g, W_scale, "W_scale", 4));
    IL_CHECK(hk::il_check(g, Y_out, "Y_out"));
    const hk::IlBuffer y{Y_out, 2 * n * g->f, "Y_out"};
    IL_CHECK(hk::il_apart(y, {X, 2 * n * g->d, "X"}));
    IL_CHECK(hk::il_apart(y, {X_codes, n * g->d, "X_codes"}));
    IL_CHECK(hk::il_apart(y, {X_scale, 4 * n, "X_scale"}));
    IL_CHECK(hk::il_apart(y, {W_codes, g->f * g->d, "W_codes"}));
    IL_CHECK(hk::il_apart(y, {W_scale, 4 * g->f, "W_scale"}));
    return hk::forward(g, X, X_codes, X_scale, n, W_codes, W_scale, Y_out, static_cast<cudaStream_t>(stream));
}

IL_EXPORT hess_status int8_linear_forward(int8_linear_t g, const void* X, int64_t n_tokens, const int8_t* W_codes,
                                          const float* W_scale, void* Y_out, hess_stream_t stream) {
    return il_forward(g, X, nullptr, nullptr, false, n_tokens, W_codes, W_scale, Y_out, stream);
}

IL_EXPORT hess_status int8_linear_forward_rows8(int8_linear_t g, const int8_t* X_codes, const float* X_scale,
                                                int64_t n_tokens, const int8_t* W_codes, const float* W_scale,
                                                void* Y_out, hess_stream_t stream) {
    return il_forward(g, nullptr, X_codes, X_scale, true, n_tokens, W_codes, W_scale, Y_out, stream);
}

IL_EXPORT hess_status int8_linear_backward(int8_linear_t g, const void* dY, int64_t n_tokens, const int8_t* X_codes,
                                           const float* X_scale, int32_t group, const int8_t* W_codes,
                                           const float* W_scale, void* dX_out, void* dW_out, hess_stream_t stream) {
    if (!g) return il_fail(HESS_ERR_INVALID, "handle is NULL");
    IL_CHECK(hk::il_tokens(n_tokens, g->train_tokens, "train_tokens"));
    if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
        return il_fail(HESS_ERR_UNSUPPORTED, "group must be 0, 32, 64, 128 or 256, got %d", group);
    const int64_t n = n_tokens, groups = group ? (g->d + group - 1) / group : 1;
    const bool want_x = dX_out != nullptr && n > 0, want_w = dW_out != nullptr;
    std::lock_guard<std::mutex> lk(g->mu);
    IL_CHECK(hk::il_check_device(g));
    if (want_w && g->train_tokens == 0) return il_fail(HESS_ERR_INVALID, "the handle's train_tokens is 0");
    if (want_x) {
        IL_CHECK(hk::il_check(g, W_codes, "W_codes", 1));
        IL_CHECK(hk::il_check(g, W_scale, "W_scale", 4));
        IL_CHECK(hk::il_check(g, dX_out, "dX_out"));
    }
    if (want_w) {
        if (n > 0) {
            IL_CHECK(hk::il_check(g, X_codes, "X_codes", 1));
            IL_CHECK(hk::il_check(g, X_scale, "X_scale", 4));
        }
        IL_CHECK(hk::il_check(g, dW_out, "dW_out"));
    }
    if (n > 0 && (want_x || want_w)) {
        IL_CHECK(hk::il_check(g, dY, "dY"));
        const hk::IlBuffer out[] = {{dX_out, 2 * n * g->d, "dX_out"}, {dW_out, 2 * g->f * g->d, "dW_out"}};
        for (const hk::IlBuffer& o : out) {
            IL_CHECK(hk::il_apart(o, {dY, 2 * n * g->f, "dY"}));
            IL_CHECK(hk::il_apart(o, {X_codes, n * g->d, "X_codes"}));
            IL_CHECK(hk::il_apart(o, {X_scale, 4 * n * groups, "X_scale"}));
            IL_CHECK(hk::il_apart(o, {W_codes, g->f * g->d, "W_codes"}));
            IL_CHECK(hk::il_apart(o, {W_scale, 4 * g->f, "W_scale"}));
        }
        IL_CHECK(hk::il_apart(out[1], out[0]));
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n == 0) {
        if (want_w) IL_TRY(cudaMemsetAsync(dW_out, 0, static_cast<size_t>(g->f) * g->d * 2, s));
        return HESS_OK;
    }
    if (!want_x && !want_w) return HESS_OK;
    IL_TRY(hk::ensure_context());
    hk::FfSingle a{};
    a.dY = dY;
    a.W = g->w_restored;
    a.X = g->x_restored;
    a.dX = dX_out;
    a.dW = dW_out;
    a.n = n;
    a.d = g->d;
    a.f = g->f;
    a.dtype = g->dtype;
    a.pairs = g->ff_pairs;
    a.pieces = g->ff_pieces;
    a.arrived = g->status + 1 + 2 * g->pairs;
    a.status = g->status;
    a.timeout_ns = g->timeout_ns;
    IL_TRY(g->order.begin(s));
    hk::RestoreRows w{}, x{};
    if (want_x) w = {W_codes, g->d, W_scale, g->f, g->d, 0, g->w_restored, g->d};
    if (want_w) x = {X_codes, g->d, X_scale, n, g->d, group, g->x_restored, g->d};
    IL_TRY(hk::rows8_restore_launch(w, x, g->dtype, true, s));
    const hess_status st = hk::ff_gradients_single(a, s);
    IL_TRY(g->order.end(s));
    return st;
}

IL_EXPORT hess_status int8_linear_sync(int8_linear_t g, hess_stream_t stream) {
    if (!g) return il_fail(HESS_ERR_INVALID, "handle is NULL");
    std::lock_guard<std::mutex> lk(g->mu);
    IL_CHECK(hk::il_check_device(g));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t word = 0;
    IL_TRY(cudaMemcpyAsync(&word, g->status, sizeof(word), cudaMemcpyDeviceToHost, s));
    IL_TRY(cudaStreamSynchronize(s));
    if (word == 0) return HESS_OK;
    // the arrival counts of an interrupted call go with it, when no call on another
    // stream is at them, and before the next call may be
    IL_TRY(g->order.begin(s));
    IL_TRY(cudaMemsetAsync(g->status, 0, g->status_bytes, s));
    IL_TRY(cudaStreamSynchronize(s));
    return il_fail(HESS_ERR_TIMEOUT, "a device-side wait ran out (status 0x%x); results are invalid", word);
}

IL_EXPORT hess_status int8_linear_set_timeout(int8_linear_t g, int64_t ns) {
    if (!g) return il_fail(HESS_ERR_INVALID, "handle is NULL");
    if (ns < 0) return il_fail(HESS_ERR_INVALID, "the limit must not be negative");
    std::lock_guard<std::mutex> lk(g->mu);
    g->timeout_ns = static_cast<unsigned long long>(ns);
    return HESS_OK;
}

IL_EXPORT hess_status int8_linear_destroy(int8_linear_t g) {
    if (!g) return HESS_OK;
    int cur = 0;
    IL_TRY(cudaGetDevice(&cur));
    IL_TRY(cudaSetDevice(g->device));
    const cudaError_t e = cudaDeviceSynchronize();
    hk::il_free(g);
    cudaSetDevice(cur);
    delete g;
    if (e != cudaSuccess) return il_fail(HESS_ERR_CUDA, "int8_linear_destroy: %s", cudaGetErrorString(e));
    return HESS_OK;
}
