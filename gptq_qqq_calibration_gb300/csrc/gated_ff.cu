// Gated feed-forward projections h = act(X Wg^T) * (X Wu^T) and their gradient
// (formulas and conventions: include/gated_ff.h).
//
// Four contractions share one tensor-core loop; what differs is which operand
// is contiguous along the contraction (K-major) and which along its own rows
// (MN-major), and what happens to the finished tile:
//
//   forward   A = X [n, d]   K-major    B = Wg | Wu [f, d] K-major   sum over d
//   dg, du    the same products, then dh joins in the epilogue
//   dX        A = dg, du     K-major    B = Wg, Wu         MN-major  sum over f, twice
//   dWg, dWu  A = dg | du    MN-major   B = X              MN-major  sum over n
//
// Tile: 256 x 256 on a pair of SMs (tcgen05 cta_group::2), the largest one
// instruction covers, so each SM receives 32 KB per 64 steps of the
// contraction for its share of 256 x 256 x 64 products.  In the forward
// product the pair's B halves are 128 rows of Wg (even CTA) and the same 128
// rows of Wu (odd CTA): g and u of a token land in the same tensor-memory
// lane, 128 columns apart, and meet in the epilogue's registers.  Tensor
// memory holds two tiles, so one tile's epilogue runs under the next one's
// products.
//
// Where the tiles do not fill the pairs (a small problem, or the last round of a
// larger one) each is split along its sum: the pieces' fp32 sums go to memory
// and the pair that comes last adds them, in the order of the pieces, and
// finishes the tile.  Nobody waits for another pair.
//
// Every operand box is 64 x 64 elements with the 128-byte swizzle, whichever
// way it is contiguous: boxes stacked in shared memory serve both the K-major
// and the MN-major descriptors, and one tensor map per matrix is enough.
// Edges cost nothing: the copies fill zeros past the end of a matrix.
//
// The tensor cores bound it, and under long loads the board's power: 8,192 tokens
// at 4,096 x 11,008 forward take 844 us (1,750 TFLOP/s, 0.92 of the burst rate of a
// library GEMM), the gradients of 4,096 tokens 1,310 to 1,350 us (1,640 to 1,690).
// ncu (2,048 tokens): tensor pipe 85 % active forward, 94 % in the gradients'
// kernel.  Below some 600 tokens the weights and their gradients are what takes
// time (4 d f bytes each): 256 tokens forward 48 us for 28 us of bytes, as the 86
// tiles of one row of tiles fill the 76 pairs once and an eighth.
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <new>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_ptr.h"
#include "gated_ff.h"
#include "gated_ff_schedule.cuh"
#include "int8_linear.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rows8.cuh"
#include "workspace_order.h"

namespace hk {
namespace {

using namespace ff;

constexpr int kStages = 6;
constexpr uint32_t kBoxBytes = 64 * 64 * 2;
constexpr uint32_t kOperandBytes = 2 * kBoxBytes;  // 128 rows of A, or of B, per CTA
constexpr uint32_t kStageBytes = 2 * kOperandBytes;
constexpr int kEpiWarps = 8;
constexpr int kFirstEpiWarp = 4;
constexpr int kThreads = (kFirstEpiWarp + kEpiWarps) * 32;
constexpr uint32_t kTmemCols = 512;  // two 256-column tiles
constexpr int kNumBarriers = 2 * kStages + 5;
constexpr uint32_t kOutBytes = 128 * 128;  // 128 rows x 64 columns on their way out, for each half of the epilogue
constexpr uint32_t kAfterRing = kStages * kStageBytes + 2 * kOutBytes;
constexpr size_t kSmemBytes = 1024 + kAfterRing + 8 * kNumBarriers + 16;
constexpr unsigned long long kDrainLimitNs = 1000000000ull;
constexpr unsigned long long kAbortSettleNs = 2000000ull;

enum { kMapX, kMapWg, kMapWu, kMapDg, kMapDu, kMapOut0, kMapOut1, kMapOut2, kMaps };

struct FfParams : FfSchedule {
    CUtensorMap maps[kMaps];  // the last three are written: h | dg, du | dX, dWg, dWu
    int32_t act;
    uint32_t fmt;     // operand format of the instruction descriptor: 0 = f16, 1 = bf16
    const void* dh;
    float* pieces;      // 256 x 256 sums of every unit of a split tile
    uint32_t* arrived;  // pieces of each split tile that have come, per CTA; zero between launches
    uint32_t* status;
    unsigned long long timeout_ns;
};
constexpr int kPieceFloats = 256 * 256;

__device__ __forceinline__ uint32_t instr_desc(uint32_t fmt, bool a_mn, bool b_mn) {
    return (1u << 4) | (fmt << 7) | (fmt << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           ((256u >> 3) << 17) | ((256u >> 4) << 24);
}

__device__ __forceinline__ void tmem_ld16(uint32_t t, uint32_t (&a)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
          "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15])
        : "r"(t)
        : "memory");
}
// Waits for the loads above; `a` and `b` pass through so that no use of them moves before the wait.
__device__ __forceinline__ void tmem_wait16(uint32_t (&a)[16], uint32_t (&b)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(a[0]), "+r"(a[1]), "+r"(a[2]), "+r"(a[3]), "+r"(a[4]), "+r"(a[5]), "+r"(a[6]), "+r"(a[7]),
                   "+r"(a[8]), "+r"(a[9]), "+r"(a[10]), "+r"(a[11]), "+r"(a[12]), "+r"(a[13]), "+r"(a[14]),
                   "+r"(a[15])::"memory");
    asm volatile(""
                 : "+r"(b[0]), "+r"(b[1]), "+r"(b[2]), "+r"(b[3]), "+r"(b[4]), "+r"(b[5]), "+r"(b[6]), "+r"(b[7]),
                   "+r"(b[8]), "+r"(b[9]), "+r"(b[10]), "+r"(b[11]), "+r"(b[12]), "+r"(b[13]), "+r"(b[14]),
                   "+r"(b[15])::"memory");
}

template <class T>
struct Half2;
template <>
struct Half2<__nv_bfloat16> {
    static __device__ uint32_t pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        uint32_t w;
        memcpy(&w, &h, 4);
        return w;
    }
    static __device__ float2 unpack(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};
template <>
struct Half2<__half> {
    static __device__ uint32_t pack(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        uint32_t w;
        memcpy(&w, &h, 4);
        return w;
    }
    static __device__ float2 unpack(uint32_t w) {
        __half2 h;
        memcpy(&h, &w, 4);
        return __half22float2(h);
    }
};

// act(g) = g s and act'(g) = s + g s (1 - s) z', with s = 1 / (1 + e^-z):
// z = g for silu; z = 2 sqrt(2/pi) (g + 0.044715 g^3) for gelu, whose
// (1 + tanh(z / 2)) / 2 is the same s.
__device__ __forceinline__ float gate_sigmoid(float g, int act, float& dz) {
    float z = g;
    dz = 1.0f;
    if (act == GATED_FF_GELU_TANH) {
        const float c = 1.5957691216057308f, g2 = g * g;
        z = c * g * fmaf(0.044715f, g2, 1.0f);
        dz = c * fmaf(3.0f * 0.044715f, g2, 1.0f);
    }
    return __fdividef(1.0f, 1.0f + __expf(-z));
}

// The epilogue warps' own barrier.  (Barriers take whole warps: lanes that may come from a
// branch or from a wait one by one meet first.)
__device__ __forceinline__ void epi_barrier() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
}
// The same, and whether any thread came with `x`: every thread gets the same answer.
__device__ __forceinline__ bool epi_barrier_any(bool x) {
    uint32_t any;
    __syncwarp();
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

// 64 columns of 128 rows go out through shared memory and one TMA store, which
// leaves out what lies past the matrix's edges (each thread storing its row's 16
// bytes at a time half-fills 32-byte sectors, and a tile of dW with few tokens
// takes longer to store than to compute).  The four warps of one half of the
// epilogue share a buffer.
struct OutBuffer {
    uint32_t addr;
    int barrier, row;  // this thread's row
    bool leader;
    __device__ void sync() const {
        __syncwarp();
        asm volatile("bar.sync %0, 128;" ::"r"(barrier) : "memory");
    }
    // the buffer's former content has been read
    __device__ void begin() const {
        if (leader) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        sync();
    }
    // eight values from column 8 j on, two to a word, in the 128-byte swizzle
    __device__ void put(int j, uint4 v) const { sts128(addr + row * 128 + ((j ^ (row & 7)) << 4), v); }
    __device__ void end(const CUtensorMap* map, int x, int y, int cols, int rows) const {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        sync();
        if (leader && x < cols && y < rows) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                             reinterpret_cast<uint64_t>(map)),
                         "r"(addr), "r"(x), "r"(y)
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
};

template <class T>
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(Half2<T>::pack(x[0], x[1]), Half2<T>::pack(x[2], x[3]), Half2<T>::pack(x[4], x[5]),
                      Half2<T>::pack(x[6], x[7]));
}

// Epilogue of one tile by the four warps of one half: rows m.. of this CTA's
// 128, half of the columns.  load(c, a, c2, b) gives the finished sums of the
// tile's 16 columns from c on and from c2 on.
template <class T, int kWhat, class Load>
__device__ __forceinline__ void finish_tile(const FfParams& p, const Unit& un, int half, int m, const OutBuffer& out,
                                            Load load) {
    if constexpr (kWhat != kGradients) {
        const int64_t row = static_cast<int64_t>(m) + out.row;
        const bool in = row < p.n;
        const int n0 = un.n0 + half * 64;
        uint4 later[kWhat == kActGrad ? 8 : 1];  // du, until dg has left the buffer
        out.begin();
#pragma unroll
        for (int c = 0; c < 64; c += 16) {
            uint4 dv[2] = {};
            if constexpr (kWhat == kActGrad) {
                const T* const dh = static_cast<const T*>(p.dh) + row * p.f + n0 + c;
                if (in && n0 + c < p.f) dv[0] = *reinterpret_cast<const uint4*>(dh);
                if (in && n0 + c + 8 < p.f) dv[1] = *reinterpret_cast<const uint4*>(dh + 8);
                __syncwarp();  // the sums' loads take whole warps
            }
            uint32_t g[16], u[16];
            load(half * 64 + c, g, 128 + half * 64 + c, u);
            float first[16];
            if constexpr (kWhat == kForward) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float dz;
                    const float gi = __uint_as_float(g[i]);
                    first[i] = gi * gate_sigmoid(gi, p.act, dz) * __uint_as_float(u[i]);
                }
            } else {
                const uint32_t w[8] = {dv[0].x, dv[0].y, dv[0].z, dv[0].w, dv[1].x, dv[1].y, dv[1].z, dv[1].w};
                float du[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 d2 = Half2<T>::unpack(w[i / 2]);
                    const float dh = (i & 1) ? d2.y : d2.x;
                    float dz;
                    const float gi = __uint_as_float(g[i]);
                    const float s = gate_sigmoid(gi, p.act, dz);
                    du[i] = dh * (gi * s);
                    first[i] = dh * __uint_as_float(u[i]) * fmaf(gi * s * (1.0f - s), dz, s);
                }
                later[c / 8] = pack8<T>(du);
                later[c / 8 + 1] = pack8<T>(du + 8);
            }
            out.put(c / 8, pack8<T>(first));
            out.put(c / 8 + 1, pack8<T>(first + 8));
        }
        out.end(&p.maps[kMapOut0], n0, m, p.f, p.n);
        if constexpr (kWhat == kActGrad) {
            out.begin();
#pragma unroll
            for (int j = 0; j < 8; ++j) out.put(j, later[j]);
            out.end(&p.maps[kMapOut1], n0, m, p.f, p.n);
        }
    } else {
        const CUtensorMap* const map = &p.maps[un.kind == 1 ? kMapOut0 : un.which ? kMapOut2 : kMapOut1];
#pragma unroll 1
        for (int n = half * 128; n < half * 128 + 128; n += 64) {
            out.begin();
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
                uint32_t a[16], b[16];
                load(n + c, a, n + c + 16, b);
                float x[32];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] = __uint_as_float(a[i]);
                    x[16 + i] = __uint_as_float(b[i]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) out.put(c / 8 + i, pack8<T>(x + 8 * i));
            }
            out.end(map, un.n0 + n, m, p.d, un.kind == 1 ? p.n : p.f);
        }
    }
}

// Warp roles of both CTAs: warp 0 copies this CTA's operand boxes (its bytes
// count on the even CTA's barrier), warp 1 of the even CTA issues the pair's
// MMAs, warps 4-11 finish tiles.  Every wait is bounded.
template <class T, int kWhat>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gated_ff_kernel(const __grid_constant__ FfParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - raw);
    const uint32_t bar0 = base + kAfterRing;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + kAfterRing + 8 * kNumBarriers);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * kStages + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * kStages + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kStages + 4);
    __shared__ int aborted;
    __shared__ volatile int epi_last;  // of the epilogue warps

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1;
    const int n_pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), 2 * kEpiWarps);
        }
        mbar_init(drain_bar, 1);
        aborted = 0;
        fence_barrier_init();
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
    const unsigned long long limit = p.timeout_ns;
    // Set-up above may overlap the end of the stream's previous kernel; nothing
    // is read or written before that has completed.
    griddep_wait();
    griddep_launch_dependents();

    if (warp == 0 && lane == 0) {
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0;
        for (int i = 0, u; ok && (u = unit_of<kWhat>(p, pair, n_pairs, i)) >= 0; ++i) {
            const Unit un = unit_at<kWhat>(p, u);
            const int m = un.m0 + static_cast<int>(rank) * 128;
            const int n = un.kind == 0 ? un.n0 : un.n0 + static_cast<int>(rank) * 128;
            for (int kb = un.kb0; kb < un.kb1; ++kb) {
                if (!mbar_wait_cluster(empty_bar(stage), phase ^ 1u, limit)) {
                    ok = false;
                    break;
                }
                const uint32_t sA = base + stage * kStageBytes, sB = sA + kOperandBytes;
                const uint32_t fb = mapa_shared(full_bar(stage), 0);
                if (rank == 0) mbar_arrive_expect_tx(full_bar(stage), 2 * kStageBytes);
                int k = kb * kKB;
                if (un.kind == 0) {
                    const CUtensorMap* const w = &p.maps[rank == 0 ? kMapWg : kMapWu];
                    tma_load_2d_pair(sA, &p.maps[kMapX], fb, k, m);
                    tma_load_2d_pair(sA + kBoxBytes, &p.maps[kMapX], fb, k, m + 64);
                    tma_load_2d_pair(sB, w, fb, k, n);
                    tma_load_2d_pair(sB + kBoxBytes, w, fb, k, n + 64);
                } else if (un.kind == 1) {
                    const bool up = kb >= un.half;
                    const CUtensorMap* const a = &p.maps[up ? kMapDu : kMapDg];
                    const CUtensorMap* const w = &p.maps[up ? kMapWu : kMapWg];
                    if (up) k -= un.half * kKB;
                    tma_load_2d_pair(sA, a, fb, k, m);
                    tma_load_2d_pair(sA + kBoxBytes, a, fb, k, m + 64);
                    tma_load_2d_pair(sB, w, fb, n, k);
                    tma_load_2d_pair(sB + kBoxBytes, w, fb, n + 64, k);
                } else {
                    const CUtensorMap* const a = &p.maps[un.which ? kMapDu : kMapDg];
                    tma_load_2d_pair(sA, a, fb, m, k);
                    tma_load_2d_pair(sA + kBoxBytes, a, fb, m + 64, k);
                    tma_load_2d_pair(sB, &p.maps[kMapX], fb, n, k);
                    tma_load_2d_pair(sB + kBoxBytes, &p.maps[kMapX], fb, n + 64, k);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok) {
            atomicOr(p.status, kStatusTimeoutLoad);
            aborted = 1;
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0;
        int ab = 0;
        uint32_t aphase = 0;
        for (int i = 0, u; ok && (u = unit_of<kWhat>(p, pair, n_pairs, i)) >= 0; ++i) {
            const Unit un = unit_at<kWhat>(p, u);
            // K-major: 16 steps are 32 bytes of a row, 8-row groups are 1,024
            // bytes apart.  MN-major: 16 steps are 16 rows of 128 bytes, the
            // second 64 columns are a box further.
            const bool a_mn = un.kind == 2, b_mn = un.kind != 0;
            const uint32_t a_step = a_mn ? 2048u : 32u, b_step = b_mn ? 2048u : 32u;
            const uint32_t a_lbo = a_mn ? kBoxBytes : 16u, b_lbo = b_mn ? kBoxBytes : 16u;
            const uint32_t idesc = instr_desc(p.fmt, a_mn, b_mn);
            if (!mbar_wait_cluster(acce_bar(ab), aphase ^ 1u, limit)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + static_cast<uint32_t>(ab) * 256u;
            for (int kb = un.kb0; kb < un.kb1; ++kb) {
                if (!mbar_wait_cluster(full_bar(stage), phase, limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sA = base + stage * kStageBytes, sB = sA + kOperandBytes;
#pragma unroll
                for (int j = 0; j < kKB / 16; ++j)
                    umma_f16_pair(acc, smem_desc_sw128(sA + j * a_step, a_lbo, 1024u),
                                  smem_desc_sw128(sB + j * b_step, b_lbo, 1024u), idesc,
                                  kb != un.kb0 || j != 0 ? 1u : 0u);
                tc_commit_pair_mc(empty_bar(stage), 0x3);
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            tc_commit_pair_mc(accf_bar(ab), 0x3);
            if (++ab == 2) {
                ab = 0;
                aphase ^= 1u;
            }
        }
        if (!ok) {
            atomicOr(p.status, kStatusTimeoutMma);
            aborted = 1;
        }
        // every MMA issued has completed before the pair's memories are released
        tc_commit_pair_mc(drain_bar, 0x1);
        if (!mbar_wait(drain_bar, 0, kDrainLimitNs)) atomicOr(p.status, kStatusTimeoutDrain);
    } else if (warp >= kFirstEpiWarp) {
        bool failed = false;
        int ab = 0;
        uint32_t aphase = 0;
        const int q = warp & 3, half = (warp - kFirstEpiWarp) >> 2;
        const int r128 = q * 32 + lane;  // row of this CTA's half of the tile
        const OutBuffer out{base + kStages * kStageBytes + half * kOutBytes, 2 + half, r128, q == 0 && lane == 0};
        const uint32_t acce0 = mapa_shared(acce_bar(0), 0);
        for (int i = 0, u; (u = unit_of<kWhat>(p, pair, n_pairs, i)) >= 0; ++i) {
            const Unit un = unit_at<kWhat>(p, u);
            // The warps go on together: they agree on whether a wait ran out (with the
            // barrier itself: a flag read after it might already be the next unit's),
            // so that all of them pass the same barriers below.
            failed = epi_barrier_any(failed || !mbar_wait_cluster(accf_bar(ab), aphase, limit));
            tc_fence_after();
            const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(ab * 256);
            const int m = un.m0 + static_cast<int>(rank) * 128;
            const auto from_tmem = [&](int c, uint32_t (&a)[16], int c2, uint32_t (&b)[16]) {
                tmem_ld16(acc + c, a);
                tmem_ld16(acc + c2, b);
                tmem_wait16(a, b);
            };
            if (un.parts == 1) {
                if (!failed) finish_tile<T, kWhat>(p, un, half, m, out, from_tmem);
            } else {
                // one piece after the other: this CTA's half of it in blocks of four
                // columns, 128 rows of 16 bytes each
                float* const piece0 = p.pieces + static_cast<int64_t>(un.split) * un.parts * kPieceFloats +
                                      rank * (kPieceFloats / 2) + 4 * r128;
                if (!failed) {
                    float* const mine = piece0 + static_cast<int64_t>(un.part) * kPieceFloats;
                    for (int c = half * 128; c < half * 128 + 128; c += 32) {
                        uint32_t a[16], b[16];
                        from_tmem(c, a, c + 16, b);
#pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            __stcg(reinterpret_cast<uint4*>(mine + (c + k) * 128),
                                   make_uint4(a[k], a[k + 1], a[k + 2], a[k + 3]));
                            __stcg(reinterpret_cast<uint4*>(mine + (c + 16 + k) * 128),
                                   make_uint4(b[k], b[k + 1], b[k + 2], b[k + 3]));
                        }
                    }
                    __threadfence();
                }
                epi_barrier();
                if (warp == kFirstEpiWarp && lane == 0) {
                    uint32_t* const count = p.arrived + 2 * un.split + rank;
                    const bool last = !failed && atomicAdd(count, 1u) == static_cast<uint32_t>(un.parts - 1);
                    if (last) *count = 0;
                    epi_last = last;
                }
                epi_barrier();
                if (epi_last) {
                    __threadfence();
                    finish_tile<T, kWhat>(p, un, half, m, out, [&](int c, uint32_t (&a)[16], int c2, uint32_t (&b)[16]) {
                        float x[16] = {}, y[16] = {};
                        for (int k = 0; k < un.parts; ++k) {
                            const float* const piece = piece0 + static_cast<int64_t>(k) * kPieceFloats;
                            float4 v[8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                v[e] = __ldcg(reinterpret_cast<const float4*>(piece + (c + 4 * e) * 128));
                                v[4 + e] = __ldcg(reinterpret_cast<const float4*>(piece + (c2 + 4 * e) * 128));
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                x[4 * e] += v[e].x, x[4 * e + 1] += v[e].y;
                                x[4 * e + 2] += v[e].z, x[4 * e + 3] += v[e].w;
                                y[4 * e] += v[4 + e].x, y[4 * e + 1] += v[4 + e].y;
                                y[4 * e + 2] += v[4 + e].z, y[4 * e + 3] += v[4 + e].w;
                            }
                        }
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            a[e] = __float_as_uint(x[e]);
                            b[e] = __float_as_uint(y[e]);
                        }
                    });
                }
                epi_barrier();  // epi_last may be written again
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(acce0 + 8u * ab);
            if (++ab == 2) {
                ab = 0;
                aphase ^= 1u;
            }
        }
        if (out.leader) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        if (failed && lane == 0) {
            atomicOr(p.status, kStatusTimeoutEpilogue);
            aborted = 1;
        }
    }

    // After a timeout a CTA cannot watch its own copies land (they count on the
    // even CTA's barrier): it gives them time before its memory goes.
    __syncthreads();
    if (*reinterpret_cast<volatile int*>(&aborted) != 0) {
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
// Up to kFewTokens tokens the work is reading the weights once (4 d f bytes for
// 4 n d f operations: memory-bound below some 280 tokens), so the roles turn:
// weight rows are the MMA's rows (R of Wg and the same R of Wu in one operand),
// tokens its columns (N = n rounded up to 16), and each CTA streams its rows
// through a ring of shared memory.  R is any number up to 64, chosen so that every
// SM gets the same number of rows (37 at f = 11,008: 298 tiles; tiles of 64 would
// be 172, one or two per SM), which needs no split of the sums.  The operand's
// unused rows hold what they hold: an MMA row only reaches its own tensor-memory
// lane.
//
// One CTA per SM with a ring of 192 KB, or two with 92 KB where that gives each
// one tile instead of two: they fill each other's start and end, and the next
// launch's first CTAs find room early (one token, 4,096 x 11,008: 33.4 us with one
// CTA per SM, 29.1 with two, 92 % of the weights' bytes at the copy rate; 2,560 x
// 6,912, one tile per SM either way: 14.3 and 14.9 us; 8,192 x 28,672: 137 and 155).

constexpr int kFewTokens = 128;
constexpr uint32_t kFewRing = 192 * 1024, kFewRing2 = 92 * 1024;
constexpr int kFewMaxStages = 16;
constexpr int kFewThreads = 256;  // warps 0: copies, 1: MMAs, 4-7: epilogue
constexpr int kFewNumBarriers = 2 * kFewMaxStages + 5;
// two buffers of g and u: 16 tokens x 64 rows.  It follows the ring: an operand of
// few rows at the ring's end, which is read as 128 rows all the same, ends in it.
constexpr uint32_t kFewExchange = 2 * 2 * 16 * 64 * 4;
static_assert(kFewExchange >= 128 * 128, "the last operand's 128 rows end in the exchange buffers");
constexpr size_t few_smem(uint32_t ring) { return 1024 + ring + kFewExchange + 8 * kFewNumBarriers + 16; }

struct FewParams {
    CUtensorMap maps[3];  // kMapX: n_cols-row boxes; kMapWg, kMapWu: R-row boxes
    int32_t n, f, act;
    int32_t n_cols;       // n rounded up to 16: the MMA's N
    int32_t rows;         // R
    int32_t rows8;        // R rounded up to 8: where Wu's rows begin in the operand
    int32_t stages;
    int32_t stage_bytes;
    uint32_t ring;        // bytes
    int32_t n_kb;         // boxes along d
    int32_t n_tiles;      // ceil(f / R)
    uint32_t fmt;
    void* out;
    uint32_t* status;
    unsigned long long timeout_ns;
};

template <class T>
__global__ void __launch_bounds__(kFewThreads, 2) gated_ff_few_kernel(const __grid_constant__ FewParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* const gbase = smem_raw + (base - raw);
    float* const exch = reinterpret_cast<float*>(gbase + p.ring);
    const uint32_t bar0 = base + p.ring + kFewExchange;
    uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbase + p.ring + kFewExchange + 8 * kFewNumBarriers);
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (kFewMaxStages + s); };
    auto accf_bar = [&](int b) { return bar0 + 8u * (2 * kFewMaxStages + b); };
    auto acce_bar = [&](int b) { return bar0 + 8u * (2 * kFewMaxStages + 2 + b); };
    const uint32_t drain_bar = bar0 + 8u * (2 * kFewMaxStages + 4);
    __shared__ volatile int aborted;  // a wait of some role ran out

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // X's rows come first in a stage (n_cols of them), then Wg's, then Wu's
    const uint32_t x_bytes = static_cast<uint32_t>(p.n_cols) * 128u;
    const uint32_t u_at = x_bytes + static_cast<uint32_t>(p.rows8) * 128u;
    const uint32_t stage_bytes = static_cast<uint32_t>(p.stage_bytes);
    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(accf_bar(b), 1);
            mbar_init(acce_bar(b), 4);
        }
        mbar_init(drain_bar, 1);
        aborted = 0;
        fence_barrier_init();
        for (int m = 0; m < 3; ++m) prefetch_tensormap(&p.maps[m]);
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), 2 * kFewTokens);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
    const unsigned long long limit = p.timeout_ns;

    if (warp == 0 && lane == 0) {
        // Set-up above, and the first ring of weights on its way to L2 (which
        // later writes to them would update), may overlap the end of the
        // stream's previous kernel; nothing is read before that has completed.
        int kb0 = 0, t0 = blockIdx.x;
        for (int s = 0; s < p.stages && t0 < p.n_tiles; ++s) {
            tma_prefetch_2d(&p.maps[kMapWg], kb0 * kKB, t0 * p.rows);
            tma_prefetch_2d(&p.maps[kMapWu], kb0 * kKB, t0 * p.rows);
            if (++kb0 == p.n_kb) {
                kb0 = 0;
                t0 += gridDim.x;
            }
        }
        griddep_wait();
        griddep_launch_dependents();
        bool ok = true;
        int stage = 0;
        uint32_t phase = 0;
        for (int t = blockIdx.x; ok && t < p.n_tiles; t += gridDim.x) {
            for (int kb = 0; kb < p.n_kb; ++kb) {
                if (!mbar_wait(empty_bar(stage), phase ^ 1u, limit)) {
                    ok = false;
                    break;
                }
                const uint32_t at = base + stage * stage_bytes;
                mbar_arrive_expect_tx(full_bar(stage), x_bytes + 2u * 128u * static_cast<uint32_t>(p.rows));
                tma_load_2d(at + x_bytes, &p.maps[kMapWg], full_bar(stage), kb * kKB, t * p.rows);
                tma_load_2d(at + u_at, &p.maps[kMapWu], full_bar(stage), kb * kKB, t * p.rows);
                tma_load_2d(at, &p.maps[kMapX], full_bar(stage), kb * kKB, 0);
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
    } else if (warp == 1 && lane == 0) {
        bool ok = true;
        int stage = 0, ab = 0;
        uint32_t phase = 0, aphase = 0;
        const uint32_t idesc = (1u << 4) | (p.fmt << 7) | (p.fmt << 10) |
                               ((static_cast<uint32_t>(p.n_cols) >> 3) << 17) | ((128u >> 4) << 24);
        griddep_wait();
        for (int t = blockIdx.x; ok && t < p.n_tiles; t += gridDim.x) {
            if (!mbar_wait(acce_bar(ab), aphase ^ 1u, limit)) {
                ok = false;
                break;
            }
            tc_fence_after();
            for (int kb = 0; kb < p.n_kb; ++kb) {
                if (!mbar_wait(full_bar(stage), phase, limit)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t sB = base + stage * stage_bytes, sA = sB + x_bytes;
#pragma unroll
                for (int j = 0; j < kKB / 16; ++j)
                    umma_f16(tmem + ab * kFewTokens, smem_desc_sw128(sA + j * 32u, 16u, 1024u),
                             smem_desc_sw128(sB + j * 32u, 16u, 1024u), idesc, (kb | j) != 0 ? 1u : 0u);
                tc_commit(empty_bar(stage));
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (!ok) break;
            tc_commit(accf_bar(ab));
            if (++ab == 2) {
                ab = 0;
                aphase ^= 1u;
            }
        }
        if (!ok) {
            atomicOr(p.status, kStatusTimeoutMma);
            aborted = 1;
        }
        tc_commit(drain_bar);
        if (!mbar_wait(drain_bar, 0, kDrainLimitNs)) atomicOr(p.status, kStatusTimeoutDrain);
    } else if (warp >= 4) {
        // Lanes r < R hold g of weight row r, lanes rows8 + r its u.  They meet in
        // shared memory, 16 tokens at a time; each thread then finishes one row
        // of eight tokens.
        griddep_wait();
        const int q = warp - 4, l = q * 32 + lane;
        const int at = l < p.rows ? l : l >= p.rows8 && l < p.rows8 + p.rows ? 16 * 64 + l - p.rows8 : -1;
        const int r = l & 63, c8 = (l >> 6) * 8;
        int ab = 0, buf = 0;
        uint32_t aphase = 0;
        for (int t = blockIdx.x; t < p.n_tiles; t += gridDim.x) {
            const bool ok = warp_came(aborted == 0 && mbar_wait(accf_bar(ab), aphase, limit));
            if (!ok && lane == 0) {
                atomicOr(p.status, kStatusTimeoutEpilogue);
                aborted = 1;
            }
            tc_fence_after();
            const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(ab * kFewTokens);
            const int row = t * p.rows + r;
            const bool mine = ok && r < p.rows && row < p.f;
            // every epilogue warp takes every turn: they meet at a barrier in each
            for (int c = 0; c < p.n_cols; c += 16) {
                uint32_t a[16];
                __syncwarp();  // lanes come from the wait, or from their results, one by one
                tmem_ld16(acc + c, a);
                tmem_wait16(a, a);
                float* const ex = exch + buf * (2 * 16 * 64);
                buf ^= 1;
                if (at >= 0) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) ex[at + i * 64] = __uint_as_float(a[i]);
                }
                __syncwarp();
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (mine && c + c8 < p.n) {
                    uint16_t h[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float dz;
                        const float g = ex[(c8 + i) * 64 + r];
                        h[i] = static_cast<uint16_t>(
                            Half2<T>::pack(g * gate_sigmoid(g, p.act, dz) * ex[16 * 64 + (c8 + i) * 64 + r], 0.0f));
                    }
                    uint16_t* const out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(c + c8) * p.f + row;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (c + c8 + i < p.n) out[static_cast<int64_t>(i) * p.f] = h[i];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce_bar(ab));
            if (++ab == 2) {
                ab = 0;
                aphase ^= 1u;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (aborted != 0) {  // copies still in flight land before the memory goes
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < kAbortSettleNs) __nanosleep(1000);
    }
    __syncwarp();  // each lane has a clock of its own
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kFewTokens);
    }
}

// ------------------------------------------------------------- host side

hess_status ff_fail(hess_status s, const char* fmt, ...) {
    char buf[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

#define FF_TRY(call)                                                                           \
    do {                                                                                       \
        cudaError_t e_ = (call);                                                               \
        if (e_ != cudaSuccess)                                                                 \
            return ff_fail(HESS_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));     \
    } while (0)

bool ff_injected(const char* what) {
    const char* f = std::getenv("HESS_FAULT");
    return f && std::strcmp(f, what) == 0;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn ff_encode_fn() {
    static EncodeTiledFn fn = [] {
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

// Row-major [rows, cols] of 16-bit elements, boxes of box_rows x 64, zeros past the edges.
hess_status ff_encode(CUtensorMap* m, const void* ptr, int32_t dtype, int64_t rows, int64_t cols,
                      uint32_t box_rows = 64) {
    EncodeTiledFn fn = ff_encode_fn();
    if (!fn) return ff_fail(HESS_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    if (ff_injected("encode"))
        return ff_fail(HESS_ERR_UNSUPPORTED, "injected tensor-map failure (HESS_FAULT=encode)");
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2u};
    const cuuint32_t box[2] = {64u, box_rows}, es[2] = {1u, 1u};
    const CUresult r = fn(m, dtype == HESS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          2, const_cast<void*>(ptr), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return ff_fail(HESS_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled failed (%d) for [%lld, %lld]",
                       static_cast<int>(r), static_cast<long long>(rows), static_cast<long long>(cols));
    return HESS_OK;
}

// Per-device set-up: shared-memory limits, and how many pairs stay resident.
hess_status ff_prepare(int dev, int* pairs, int* sms_out) {
    static std::mutex mu;
    static int count[128] = {}, sm_count[128] = {};
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 128) return ff_fail(HESS_ERR_UNSUPPORTED, "device index %d", dev);
    if (!count[dev]) {
        for (auto fn : {gated_ff_kernel<__nv_bfloat16, kForward>, gated_ff_kernel<__nv_bfloat16, kActGrad>,
                        gated_ff_kernel<__nv_bfloat16, kGradients>, gated_ff_kernel<__half, kForward>,
                        gated_ff_kernel<__half, kActGrad>, gated_ff_kernel<__half, kGradients>})
            FF_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kSmemBytes)));
        for (auto fn : {gated_ff_few_kernel<__nv_bfloat16>, gated_ff_few_kernel<__half>})
            FF_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(few_smem(kFewRing))));
        int sms = 0;
        FF_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
        sm_count[dev] = sms;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(sms & ~1), 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = kSmemBytes;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, gated_ff_kernel<__nv_bfloat16, kForward>, &cfg) != cudaSuccess ||
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

// The status word, then two arrival counts for every tile that may be split (at
// most one per pair).
size_t status_bytes(int pairs) { return (1 + 2 * static_cast<size_t>(pairs)) * sizeof(uint32_t); }

}  // namespace
}  // namespace hk

struct gated_ff_ctx {
    std::mutex mu;
    int device = 0;
    int pairs = 0, sms = 0;
    int64_t d = 0, f = 0, train_tokens = 0;
    int32_t dtype = 0, act = 0;
    void* memory = nullptr;   // holds the next four
    float* pieces = nullptr;  // one per pair
    void* dg = nullptr;       // [train_tokens, f] each
    void* du = nullptr;
    uint32_t* status = nullptr;
    void* restored = nullptr;  // X^ [train_tokens, d] of gated_ff_backward_rows8, once it is reserved
    hk::WorkspaceOrder order;  // of the calls that use that memory
    unsigned long long timeout_ns = 2000000000ull;
};

namespace hk {
namespace {

hess_status ff_check_device(const gated_ff_ctx* g) {
    int cur = -1;
    FF_TRY(cudaGetDevice(&cur));
    if (cur != g->device)
        return ff_fail(HESS_ERR_INVALID, "handle belongs to device %d but device %d is current", g->device, cur);
    return HESS_OK;
}

hess_status ff_check(const gated_ff_ctx* g, const void* p, const char* name) {
    if (!p) return ff_fail(HESS_ERR_INVALID, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % 16) return ff_fail(HESS_ERR_INVALID, "%s is not 16-byte aligned", name);
    char why[128];
    if (const char* w = device_ptr_problem(p, g->device, why)) return ff_fail(HESS_ERR_INVALID, "%s %s", name, w);
    return HESS_OK;
}

struct FfBuffer {
    const void* p;  // nullptr: not there
    int64_t elements;
    const char* name;
};
// Outputs share no memory with inputs or with each other: some CTAs read while
// others write.
template <size_t kIn, size_t kOut>
hess_status ff_apart(const FfBuffer (&in)[kIn], const FfBuffer (&out)[kOut]) {
    const auto meet = [](const FfBuffer& a, const FfBuffer& b) {
        const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
        return a.p && b.p && a0 < b0 + 2 * static_cast<uintptr_t>(b.elements) &&
               b0 < a0 + 2 * static_cast<uintptr_t>(a.elements);
    };
    for (size_t o = 0; o < kOut; ++o) {
        for (size_t i = 0; i < kIn; ++i)
            if (meet(out[o], in[i])) return ff_fail(HESS_ERR_INVALID, "%s overlaps %s", out[o].name, in[i].name);
        for (size_t i = 0; i < o; ++i)
            if (meet(out[o], out[i])) return ff_fail(HESS_ERR_INVALID, "%s overlaps %s", out[o].name, out[i].name);
    }
    return HESS_OK;
}

#define FF_CHECK(expr)                       \
    do {                                     \
        const hess_status st_ = (expr);      \
        if (st_ != HESS_OK) return st_;      \
    } while (0)

void ff_params(FfParams& p, const gated_ff_ctx* g, int64_t n) {
    p.n = static_cast<int32_t>(n);
    p.d = static_cast<int32_t>(g->d);
    p.f = static_cast<int32_t>(g->f);
    p.act = g->act;
    p.fmt = g->dtype == HESS_BF16 ? 1u : 0u;
    p.pieces = g->pieces;
    p.arrived = g->status + 1;
    p.status = g->status;
    p.timeout_ns = g->timeout_ns;
}

// Launches so that the kernel's set-up may run while the stream's previous
// kernel ends (each kernel here waits for that one's completion by itself).
template <class Kernel, class Params>
hess_status ff_launch(Kernel kernel, const Params& p, int64_t grid, int threads, size_t smem, cudaStream_t s) {
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
    FF_TRY(cudaLaunchKernelEx(&cfg, kernel, p));
    return HESS_OK;
}

template <int kWhat>
hess_status ff_launch_resident(int resident, int32_t dtype, const FfParams& p, cudaStream_t s) {
    const int pairs = p.n_units < resident ? p.n_units : resident;
    return ff_launch(dtype == HESS_BF16 ? gated_ff_kernel<__nv_bfloat16, kWhat> : gated_ff_kernel<__half, kWhat>, p,
                     2 * pairs, kThreads, kSmemBytes, s);
}
template <int kWhat>
hess_status ff_launch_pairs(const gated_ff_ctx* g, const FfParams& p, cudaStream_t s) {
    return ff_launch_resident<kWhat>(g->pairs, g->dtype, p, s);
}

// The handle's workspace has one user at a time.
hess_status ff_begin(gated_ff_ctx* g, cudaStream_t s) {
    FF_TRY(g->order.begin(s));
    return HESS_OK;
}
hess_status ff_end(gated_ff_ctx* g, cudaStream_t s) {
    FF_TRY(g->order.end(s));
    return HESS_OK;
}

hess_status ff_forward_few(const gated_ff_ctx* g, const void* X, int64_t n, const void* Wg, const void* Wu, void* H,
                           cudaStream_t s) {
    FewParams p{};
    p.n = static_cast<int32_t>(n);
    p.f = static_cast<int32_t>(g->f);
    p.act = g->act;
    p.n_cols = static_cast<int32_t>(ceil_div(n, 16) * 16);
    // two CTAs per SM where one would have two tiles, and the ring still holds enough of them
    const bool two = n <= 64 && g->f > int64_t(64) * g->sms && g->f <= int64_t(128) * g->sms;
    const int64_t ctas = two ? 2 * g->sms : g->sms;
    p.ring = two ? kFewRing2 : kFewRing;
    // the fewest rows on the CTA that has most (counted as tiles of R), then the fewest tiles
    int64_t best = 0;
    for (int64_t R = 8; R <= 64; ++R) {
        const int64_t most = ceil_div(ceil_div(g->f, R), ctas) * R;
        if (best == 0 || most <= best) {
            best = most;
            p.rows = static_cast<int32_t>(R);
        }
    }
    p.rows8 = (p.rows + 7) / 8 * 8;
    p.stage_bytes = 128 * p.n_cols + 256 * p.rows8;
    p.stage_bytes = (p.stage_bytes + 1023) / 1024 * 1024;
    const int fit = static_cast<int>(p.ring) / p.stage_bytes;
    p.stages = fit < kFewMaxStages ? fit : kFewMaxStages;
    p.n_kb = static_cast<int32_t>(ceil_div(g->d, kKB));
    p.n_tiles = static_cast<int32_t>(ceil_div(g->f, p.rows));
    p.fmt = g->dtype == HESS_BF16 ? 1u : 0u;
    p.out = H;
    p.status = g->status;
    p.timeout_ns = g->timeout_ns;
    FF_CHECK(ff_encode(&p.maps[kMapX], X, g->dtype, n, g->d, static_cast<uint32_t>(p.n_cols)));
    FF_CHECK(ff_encode(&p.maps[kMapWg], Wg, g->dtype, g->f, g->d, static_cast<uint32_t>(p.rows)));
    FF_CHECK(ff_encode(&p.maps[kMapWu], Wu, g->dtype, g->f, g->d, static_cast<uint32_t>(p.rows)));
    return ff_launch(g->dtype == HESS_BF16 ? gated_ff_few_kernel<__nv_bfloat16> : gated_ff_few_kernel<__half>, p,
                     p.n_tiles < ctas ? p.n_tiles : ctas, kFewThreads, few_smem(p.ring), s);
}

hess_status ff_tokens(int64_t n) {
    if (n < 0) return ff_fail(HESS_ERR_INVALID, "n_tokens < 0");
    if (n > (int64_t(1) << 26)) return ff_fail(HESS_ERR_UNSUPPORTED, "n_tokens > 2^26");
    return HESS_OK;
}

void ff_free(gated_ff_ctx* g) {
    cudaFree(g->memory);
    cudaFree(g->restored);
    g->order.destroy();
}

}  // namespace

hess_status ff_resident_pairs(int dev, int* pairs, int* sms) { return ff_prepare(dev, pairs, sms); }

hess_status ff_gradients_single(const FfSingle& a, cudaStream_t s) {
    FfParams p{};
    p.n = static_cast<int32_t>(a.n);
    p.d = static_cast<int32_t>(a.d);
    p.f = static_cast<int32_t>(a.f);
    p.single = 1;
    p.fmt = a.dtype == HESS_BF16 ? 1u : 0u;
    p.pieces = a.pieces;
    p.arrived = a.arrived;
    p.status = a.status;
    p.timeout_ns = a.timeout_ns;
    FF_CHECK(ff_encode(&p.maps[kMapDg], a.dY, a.dtype, a.n, a.f));
    if (a.dX) {
        FF_CHECK(ff_encode(&p.maps[kMapWg], a.W, a.dtype, a.f, a.d));
        FF_CHECK(ff_encode(&p.maps[kMapOut0], a.dX, a.dtype, a.n, a.d, 128));
    }
    if (a.dW) {
        FF_CHECK(ff_encode(&p.maps[kMapX], a.X, a.dtype, a.n, a.d));
        FF_CHECK(ff_encode(&p.maps[kMapOut1], a.dW, a.dtype, a.f, a.d, 128));
    }
    plan_gradients(p, a.pairs, a.dX != nullptr, a.dW != nullptr);
    return ff_launch_resident<kGradients>(a.pairs, a.dtype, p, s);
}

}  // namespace hk

using hk::ff_fail;

#define FF_EXPORT extern "C" __attribute__((visibility("default")))

FF_EXPORT hess_status gated_ff_create(int64_t d, int64_t f, int64_t train_tokens, int32_t dtype, int32_t act,
                                      gated_ff_t* out) {
    if (!out) return ff_fail(HESS_ERR_INVALID, "out is NULL");
    *out = nullptr;
    if (d <= 0 || f <= 0) return ff_fail(HESS_ERR_INVALID, "d and f must be positive");
    if (train_tokens < 0) return ff_fail(HESS_ERR_INVALID, "train_tokens < 0");
    if (d % 8 || f % 8) return ff_fail(HESS_ERR_UNSUPPORTED, "d and f must be multiples of 8");
    if (d > 65536 || f > 65536) return ff_fail(HESS_ERR_UNSUPPORTED, "d or f exceeds 65536");
    if (train_tokens > (int64_t(1) << 26)) return ff_fail(HESS_ERR_UNSUPPORTED, "train_tokens > 2^26");
    if (dtype == HESS_F32) return ff_fail(HESS_ERR_UNSUPPORTED, "gated_ff takes bf16 or f16");
    if (dtype != HESS_BF16 && dtype != HESS_F16) return ff_fail(HESS_ERR_INVALID, "unknown dtype %d", dtype);
    if (act != GATED_FF_SILU && act != GATED_FF_GELU_TANH)
        return ff_fail(HESS_ERR_INVALID, "unknown activation %d", act);
    if (hk::ff_injected("alloc")) return ff_fail(HESS_ERR_OOM, "injected allocation failure (HESS_FAULT=alloc)");
    int dev = 0, pairs = 0, sms = 0;
    FF_TRY(cudaGetDevice(&dev));
    FF_TRY(hk::ensure_context());
    FF_CHECK(hk::ff_prepare(dev, &pairs, &sms));
    gated_ff_ctx* g = new (std::nothrow) gated_ff_ctx();
    if (!g) return ff_fail(HESS_ERR_OOM, "host allocation failed");
    g->device = dev;
    g->pairs = pairs;
    g->sms = sms;
    g->d = d;
    g->f = f;
    g->train_tokens = train_tokens;
    g->dtype = dtype;
    g->act = act;
    // one allocation: the split tiles' pieces, dg and du, the status word and the counts
    const size_t pieces = static_cast<size_t>(pairs) * hk::kPieceFloats * sizeof(float);
    const size_t half = (static_cast<size_t>(train_tokens) * static_cast<size_t>(f) * 2 + 255) / 256 * 256;
    cudaError_t e = cudaMalloc(&g->memory, pieces + 2 * half + hk::status_bytes(pairs));
    if (e == cudaSuccess) {
        uint8_t* const m = static_cast<uint8_t*>(g->memory);
        g->pieces = reinterpret_cast<float*>(m);
        g->dg = m + pieces;
        g->du = m + pieces + half;
        g->status = reinterpret_cast<uint32_t*>(m + pieces + 2 * half);
        e = cudaMemset(g->status, 0, hk::status_bytes(pairs));
    }
    if (e == cudaSuccess) e = g->order.create();
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        const hess_status s = e == cudaErrorMemoryAllocation ? HESS_ERR_OOM : HESS_ERR_CUDA;
        if (s == HESS_ERR_OOM) cudaGetLastError();
        hk::ff_free(g);
        delete g;
        return ff_fail(s, "gated_ff_create: %s", cudaGetErrorString(e));
    }
    *out = g;
    return HESS_OK;
}

FF_EXPORT hess_status gated_ff_forward(gated_ff_t g, const void* X, int64_t n_tokens, const void* W_gate,
                                       const void* W_up, void* H_out, hess_stream_t stream) {
    if (!g) return ff_fail(HESS_ERR_INVALID, "handle is NULL");
    FF_CHECK(hk::ff_tokens(n_tokens));
    if (n_tokens == 0) return HESS_OK;
    std::lock_guard<std::mutex> lk(g->mu);
    FF_CHECK(hk::ff_check_device(g));
    FF_CHECK(hk::ff_check(g, X, "X"));
    FF_CHECK(hk::ff_check(g, W_gate, "W_gate"));
    FF_CHECK(hk::ff_check(g, W_up, "W_up"));
    FF_CHECK(hk::ff_check(g, H_out, "H_out"));
    const hk::FfBuffer in[] = {{X, n_tokens * g->d, "X"}, {W_gate, g->f * g->d, "W_gate"}, {W_up, g->f * g->d, "W_up"}};
    const hk::FfBuffer result[] = {{H_out, n_tokens * g->f, "H_out"}};
    FF_CHECK(hk::ff_apart(in, result));
    FF_TRY(hk::ensure_context());
    if (n_tokens <= hk::kFewTokens)
        return hk::ff_forward_few(g, X, n_tokens, W_gate, W_up, H_out, static_cast<cudaStream_t>(stream));
    hk::FfParams p{};
    hk::ff_params(p, g, n_tokens);
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapX], X, g->dtype, n_tokens, g->d));
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapWg], W_gate, g->dtype, g->f, g->d));
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapWu], W_up, g->dtype, g->f, g->d));
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapOut0], H_out, g->dtype, n_tokens, g->f, 128));
    hk::plan_projections(p, g->pairs);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.parts == 1) return hk::ff_launch_pairs<hk::kForward>(g, p, s);
    FF_CHECK(hk::ff_begin(g, s));
    FF_CHECK(hk::ff_launch_pairs<hk::kForward>(g, p, s));
    return hk::ff_end(g, s);
}

// 8-bit rows in the place of X.
struct FfKept {
    const int8_t* codes;
    const float* scale;
    int32_t group;
};

static hess_status ff_backward(gated_ff_t g, const void* X, const FfKept* kept, int64_t n_tokens, const void* W_gate,
                               const void* W_up, const void* dH, void* dX_out, void* dW_gate_out, void* dW_up_out,
                               hess_stream_t stream) {
    if (!g) return ff_fail(HESS_ERR_INVALID, "handle is NULL");
    FF_CHECK(hk::ff_tokens(n_tokens));
    if (kept && kept->group != 0 && kept->group != 32 && kept->group != 64 && kept->group != 128 && kept->group != 256)
        return ff_fail(HESS_ERR_UNSUPPORTED, "group must be 0, 32, 64, 128 or 256, got %d", kept->group);
    if ((dW_gate_out == nullptr) != (dW_up_out == nullptr))
        return ff_fail(HESS_ERR_INVALID, "dW_gate_out and dW_up_out must both be given or both be NULL");
    std::lock_guard<std::mutex> lk(g->mu);
    if (n_tokens > g->train_tokens)
        return ff_fail(HESS_ERR_INVALID, "n_tokens %lld exceeds the handle's train_tokens %lld",
                           static_cast<long long>(n_tokens), static_cast<long long>(g->train_tokens));
    FF_CHECK(hk::ff_check_device(g));
    if (kept) {
        if (!g->restored) return ff_fail(HESS_ERR_INVALID, "gated_ff_reserve_rows8 has not been called");
        if (n_tokens > 0) {
            char why[128];
            if (!kept->codes || !kept->scale) return ff_fail(HESS_ERR_INVALID, "X_codes or X_scale is NULL");
            if (reinterpret_cast<uintptr_t>(kept->scale) % 4)
                return ff_fail(HESS_ERR_INVALID, "X_scale is not aligned to its element");
            if (const char* w = hk::device_ptr_problem(kept->codes, g->device, why))
                return ff_fail(HESS_ERR_INVALID, "X_codes %s", w);
            if (const char* w = hk::device_ptr_problem(kept->scale, g->device, why))
                return ff_fail(HESS_ERR_INVALID, "X_scale %s", w);
        }
        X = g->restored;
    }
    const bool want_x = dX_out != nullptr && n_tokens > 0, want_w = dW_gate_out != nullptr;
    if (n_tokens > 0) {
        if (!kept) FF_CHECK(hk::ff_check(g, X, "X"));
        FF_CHECK(hk::ff_check(g, W_gate, "W_gate"));
        FF_CHECK(hk::ff_check(g, W_up, "W_up"));
        FF_CHECK(hk::ff_check(g, dH, "dH"));
    }
    if (want_x) FF_CHECK(hk::ff_check(g, dX_out, "dX_out"));
    if (want_w) {
        FF_CHECK(hk::ff_check(g, dW_gate_out, "dW_gate_out"));
        FF_CHECK(hk::ff_check(g, dW_up_out, "dW_up_out"));
    }
    const int64_t weights = g->f * g->d;
    // sizes in elements of two bytes
    const int64_t groups = kept && kept->group ? (g->d + kept->group - 1) / kept->group : 1;
    const void* const x_in = kept ? kept->codes : X;
    const void* const scale_in = kept ? kept->scale : nullptr;
    const int64_t x_size = kept ? (n_tokens * g->d + 1) / 2 : n_tokens * g->d;
    const hk::FfBuffer in[] = {{x_in, x_size, kept ? "X_codes" : "X"}, {scale_in, 2 * n_tokens * groups, "X_scale"},
                               {W_gate, weights, "W_gate"}, {W_up, weights, "W_up"}, {dH, n_tokens * g->f, "dH"}};
    const hk::FfBuffer result[] = {{dX_out, n_tokens * g->d, "dX_out"}, {dW_gate_out, weights, "dW_gate_out"},
                                   {dW_up_out, weights, "dW_up_out"}};
    if (n_tokens > 0) FF_CHECK(hk::ff_apart(in, result));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n_tokens == 0) {
        if (want_w) {
            const size_t bytes = static_cast<size_t>(g->f) * static_cast<size_t>(g->d) * 2;
            FF_TRY(cudaMemsetAsync(dW_gate_out, 0, bytes, s));
            FF_TRY(cudaMemsetAsync(dW_up_out, 0, bytes, s));
        }
        return HESS_OK;
    }
    if (!want_x && !want_w) return HESS_OK;
    FF_TRY(hk::ensure_context());
    hk::FfParams p{};
    hk::ff_params(p, g, n_tokens);
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapX], X, g->dtype, n_tokens, g->d));
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapWg], W_gate, g->dtype, g->f, g->d));
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapWu], W_up, g->dtype, g->f, g->d));
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapDg], g->dg, g->dtype, n_tokens, g->f));
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapDu], g->du, g->dtype, n_tokens, g->f));
    p.dh = dH;
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapOut0], g->dg, g->dtype, n_tokens, g->f, 128));
    FF_CHECK(hk::ff_encode(&p.maps[hk::kMapOut1], g->du, g->dtype, n_tokens, g->f, 128));
    hk::plan_projections(p, g->pairs);
    hk::FfParams q = p;  // of the second launch; nothing is enqueued before both are complete
    if (want_x) FF_CHECK(hk::ff_encode(&q.maps[hk::kMapOut0], dX_out, g->dtype, n_tokens, g->d, 128));
    if (want_w) {
        FF_CHECK(hk::ff_encode(&q.maps[hk::kMapOut1], dW_gate_out, g->dtype, g->f, g->d, 128));
        FF_CHECK(hk::ff_encode(&q.maps[hk::kMapOut2], dW_up_out, g->dtype, g->f, g->d, 128));
    }
    hk::plan_gradients(q, g->pairs, want_x, want_w);
    FF_CHECK(hk::ff_begin(g, s));
    if (kept)
        FF_TRY(hk::rows8_restore_launch({kept->codes, g->d, kept->scale, n_tokens, g->d, kept->group, g->restored, g->d},
                                        {}, g->dtype, true, s));
    FF_CHECK(hk::ff_launch_pairs<hk::kActGrad>(g, p, s));
    const hess_status st = hk::ff_launch_pairs<hk::kGradients>(g, q, s);
    FF_CHECK(hk::ff_end(g, s));
    return st;
}

FF_EXPORT hess_status gated_ff_backward(gated_ff_t g, const void* X, int64_t n_tokens, const void* W_gate,
                                        const void* W_up, const void* dH, void* dX_out, void* dW_gate_out,
                                        void* dW_up_out, hess_stream_t stream) {
    return ff_backward(g, X, nullptr, n_tokens, W_gate, W_up, dH, dX_out, dW_gate_out, dW_up_out, stream);
}

FF_EXPORT hess_status gated_ff_reserve_rows8(gated_ff_t g) {
    if (!g) return ff_fail(HESS_ERR_INVALID, "handle is NULL");
    std::lock_guard<std::mutex> lk(g->mu);
    FF_CHECK(hk::ff_check_device(g));
    if (g->restored) return HESS_OK;
    if (g->train_tokens == 0) return ff_fail(HESS_ERR_INVALID, "the handle's train_tokens is 0");
    if (hk::ff_injected("alloc")) return ff_fail(HESS_ERR_OOM, "injected allocation failure (HESS_FAULT=alloc)");
    const cudaError_t e = cudaMalloc(&g->restored, static_cast<size_t>(g->train_tokens) * static_cast<size_t>(g->d) * 2);
    if (e == cudaSuccess) return HESS_OK;
    g->restored = nullptr;
    if (e == cudaErrorMemoryAllocation) cudaGetLastError();
    return ff_fail(e == cudaErrorMemoryAllocation ? HESS_ERR_OOM : HESS_ERR_CUDA, "gated_ff_reserve_rows8: %s",
                   cudaGetErrorString(e));
}

FF_EXPORT hess_status gated_ff_backward_rows8(gated_ff_t g, const int8_t* X_codes, const float* X_scale, int32_t group,
                                              int64_t n_tokens, const void* W_gate, const void* W_up, const void* dH,
                                              void* dX_out, void* dW_gate_out, void* dW_up_out,
                                              hess_stream_t stream) {
    const FfKept kept{X_codes, X_scale, group};
    return ff_backward(g, nullptr, &kept, n_tokens, W_gate, W_up, dH, dX_out, dW_gate_out, dW_up_out, stream);
}

FF_EXPORT hess_status gated_ff_sync(gated_ff_t g, hess_stream_t stream) {
    if (!g) return ff_fail(HESS_ERR_INVALID, "handle is NULL");
    std::lock_guard<std::mutex> lk(g->mu);
    FF_CHECK(hk::ff_check_device(g));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t word = 0;
    FF_TRY(cudaMemcpyAsync(&word, g->status, sizeof(word), cudaMemcpyDeviceToHost, s));
    FF_TRY(cudaStreamSynchronize(s));
    if (word == 0) return HESS_OK;
    // the arrival counts of an interrupted call go with it, when no call on another
    // stream is at them, and before the next call may be
    FF_CHECK(hk::ff_begin(g, s));
    FF_TRY(cudaMemsetAsync(g->status, 0, hk::status_bytes(g->pairs), s));
    FF_TRY(cudaStreamSynchronize(s));
    return ff_fail(HESS_ERR_TIMEOUT, "a device-side wait ran out (status 0x%x); results are invalid", word);
}

FF_EXPORT hess_status gated_ff_set_timeout(gated_ff_t g, int64_t ns) {
    if (!g) return ff_fail(HESS_ERR_INVALID, "handle is NULL");
    if (ns < 0) return ff_fail(HESS_ERR_INVALID, "the limit must not be negative");
    std::lock_guard<std::mutex> lk(g->mu);
    g->timeout_ns = static_cast<unsigned long long>(ns);
    return HESS_OK;
}

FF_EXPORT hess_status gated_ff_destroy(gated_ff_t g) {
    if (!g) return HESS_OK;
    int cur = 0;
    FF_TRY(cudaGetDevice(&cur));
    FF_TRY(cudaSetDevice(g->device));
    const cudaError_t e = cudaDeviceSynchronize();
    hk::ff_free(g);
    cudaSetDevice(cur);
    delete g;
    if (e != cudaSuccess) return ff_fail(HESS_ERR_CUDA, "gated_ff_destroy: %s", cudaGetErrorString(e));
    return HESS_OK;
}
