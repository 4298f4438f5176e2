// Distillation loss from a teacher's top logits, its gradient, and both in one
// pass (formulas and conventions: include/distill.h).
//
// The work is a stream over the student's logits: read them once, write the
// gradient once, a few operations per element.  The loss needs a row's sum of
// exponentials before the first gradient can be written, so a row stays on
// chip in between: a cluster of CTAs shares it, each CTA keeping its slice in
// shared memory, and the slices' maxima and sums meet through distributed
// shared memory.
//
// Exponentials are 2^(s k2 - M2) with k2 = log2(e) / tau and M2 = max(s) k2,
// one FMA and one ex2 per element.  The listed columns are taken out of the
// slice (overwritten with -inf) before the sums, so that the mass outside the
// list is summed directly instead of as a difference, and has a reference of
// its own.  With S_o, M2o of the other columns and S, M2 of the whole row:
//     q_j = 2^(s_j k2 - M2) / S
//     d loss / d s_j = w tau 2^(s_j k2 - M2o) (2^(M2o - M2) / S - p_r / S_o)
// for columns outside the list, w tau (q_j - p_j) for those in it.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_ptr.h"
#include "distill.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace hk {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kNegInf = -INFINITY;

struct DistillArgs {
    const void* logits;
    int64_t ld;
    int64_t rows;
    int32_t vocab;
    int32_t top;
    const void* top_logits;
    const void* top_index;
    int32_t top_dtype;
    int32_t index_bytes;
    const float* lse;
    const float* weights;
    const float* grad;  // backward only
    double inv_tau;
    float tau;
    float inv_hi, inv_lo;  // 1 / tau as the sum of two floats
    float k2;              // log2(e) / tau, rounded
    float k2_slip;         // 1 / tau - k2 ln 2: what that rounding leaves out
    float* loss;
    float* stats;
    void* dlogits;
    int64_t ldd;
    int32_t slice;  // 16-byte granules of a row per CTA
    int32_t chunk;  // granules a CTA holds in shared memory
};

// ---------------------------------------------------------------- elements

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <class T>
struct Elem;

template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kPer = 8;
    static __device__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
    static __device__ void unpack(const uint4& v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ uint4 pack(const float (&x)[8]) {
        uint4 v;
        uint32_t* w = &v.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            memcpy(w + i, &h, 4);
        }
        return v;
    }
    static __device__ float max_of(const uint4& v) {
        __nv_bfloat162 h[4];
        memcpy(h, &v, 16);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
};

template <>
struct Elem<__half> {
    static constexpr int kPer = 8;
    static __device__ float to_f(__half v) { return __half2float(v); }
    static __device__ __half from_f(float v) { return __float2half_rn(v); }
    static __device__ void unpack(const uint4& v, float (&x)[8]) {
        __half2 h[4];
        memcpy(h, &v, 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    static __device__ uint4 pack(const float (&x)[8]) {
        __half2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        uint4 v;
        memcpy(&v, h, 16);
        return v;
    }
    static __device__ float max_of(const uint4& v) {
        __half2 h[4];
        memcpy(h, &v, 16);
        const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
};

template <>
struct Elem<float> {
    static constexpr int kPer = 4;
    static __device__ float to_f(float v) { return v; }
    static __device__ float from_f(float v) { return v; }
    static __device__ void unpack(const uint4& v, float (&x)[4]) { memcpy(x, &v, 16); }
    static __device__ uint4 pack(const float (&x)[4]) {
        uint4 v;
        memcpy(&v, x, 16);
        return v;
    }
    static __device__ float max_of(const uint4& v) {
        float x[4];
        memcpy(x, &v, 16);
        return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    }
};

__device__ __forceinline__ float load_top(const DistillArgs& a, int64_t i) {
    if (a.top_dtype == HESS_F32) return static_cast<const float*>(a.top_logits)[i];
    if (a.top_dtype == HESS_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(a.top_logits)[i]);
    return __half2float(static_cast<const __half*>(a.top_logits)[i]);
}

__device__ __forceinline__ int64_t load_index(const DistillArgs& a, int64_t i) {
    return a.index_bytes == 8 ? static_cast<const int64_t*>(a.top_index)[i]
                              : static_cast<int64_t>(static_cast<const int32_t*>(a.top_index)[i]);
}

// exp(t / tau - base) for a teacher logit; base is the teacher's log-sum
// (`full`) or, times 1 / tau, the largest listed logit.  The argument is
// rounded relative to itself, not to t / tau.
__device__ __forceinline__ float teacher_exp(const DistillArgs& a, float t, float base, bool full) {
    const float d = full ? t : t - base;
    const float x = fmaf(d, a.inv_hi, full ? -base : 0.0f);
    return expf(fmaf(d, a.inv_lo, x));
}

// Natural logarithm to about 2^-25 of the mantissa's own: the exponent's part
// is added in fp64, so a large result carries no larger error.
__device__ __forceinline__ double log_wide(float x) {
    if (!(x > 0.0f) || x == INFINITY) return static_cast<double>(logf(x));
    int e;
    float m = frexpf(x, &e);
    if (m < 0.70710678f) {
        m *= 2.0f;
        e -= 1;
    }
    return static_cast<double>(logf(m)) + static_cast<double>(e) * kLn2;
}

// 2^(a - b) with b >= a; 0 when a is -inf (whatever b is).
__device__ __forceinline__ float rescale(float a, float b) { return a == kNegInf ? 0.0f : ex2(a - b); }

// A row of logits as 16-byte granules of memory: granule g, element e is
// column g * kPer + e - off.  The first and the last granule may hold
// neighbours' elements.
template <class T>
struct RowView {
    const T* row;
    int off;  // elements between the granule boundary and the row's start
    int n;    // granules
    __device__ RowView(const void* base, int64_t ld, int64_t r, int vocab) {
        row = static_cast<const T*>(base) + r * ld;
        off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        n = (off + vocab + Elem<T>::kPer - 1) / Elem<T>::kPer;
    }
    __device__ const T* granule(int g) const { return row - off + static_cast<int64_t>(g) * Elem<T>::kPer; }
    __device__ bool whole(int g, int vocab) const {
        return (g > 0 || off == 0) && (g + 1) * Elem<T>::kPer - off <= vocab;
    }
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// Starts the copies of granules [g0, g1) of the row into `buf`; elements of
// the edge granules that belong to other rows are set to -inf.
template <class T>
__device__ __forceinline__ void load_chunk(const RowView<T>& v, int vocab, int g0, int g1, uint4* buf) {
    const uint32_t dst = smem_u32(buf);
    for (int g = g0 + threadIdx.x; g < g1; g += kThreads) {
        if (v.whole(g, vocab)) {
            cp_async16(dst + (g - g0) * 16u, v.granule(g));
        } else {
            T* const e = reinterpret_cast<T*>(buf + (g - g0));
            for (int i = 0; i < Elem<T>::kPer; ++i) {
                const int j = g * Elem<T>::kPer + i - v.off;
                e[i] = j >= 0 && j < vocab ? v.row[j] : Elem<T>::from_f(kNegInf);
            }
        }
    }
}

// Writes one granule of gradients; `vec` when the output row has the logits
// row's alignment and the granule lies inside the row.
template <class T>
__device__ __forceinline__ void store_granule(T* out_row, int g, int off, int vocab, bool vec,
                                              const float (&x)[Elem<T>::kPer]) {
    const int j0 = g * Elem<T>::kPer - off;
    if (vec) {
        *reinterpret_cast<uint4*>(out_row + j0) = Elem<T>::pack(x);
    } else {
        for (int i = 0; i < Elem<T>::kPer; ++i)
            if (j0 + i >= 0 && j0 + i < vocab) out_row[j0 + i] = Elem<T>::from_f(x[i]);
    }
}

template <class T>
__device__ __forceinline__ void zero_slice(const RowView<T>& v, T* out_row, int vocab, bool same, int g0, int g1) {
    float z[Elem<T>::kPer] = {};
    for (int g = g0 + threadIdx.x; g < g1; g += kThreads)
        store_granule<T>(out_row, g, v.off, vocab, same && v.whole(g, vocab), z);
}

template <class V, class Op>
__device__ __forceinline__ V warp_reduce(V x, Op op) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

struct MaxOp {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct AddOp {
    __device__ float operator()(float a, float b) const { return a + b; }
};

// Sum of float pairs (hi, lo) over a warp: every addition keeps its error.
__device__ __forceinline__ void warp_sum_pairs(float& hi, float& lo) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, hi, o), l = __shfl_xor_sync(0xffffffffu, lo, o);
        float e;
        hi = two_sum_f32(hi, h, e);
        lo += l + e;
    }
}

// What the warp that reads the teacher's list leaves for the others.
struct Shared {
    int live, bad;
    float tm, m_top;     // largest listed logit, teacher's and student's
    float p_hi, p_lo;    // sum of the list's exponentials
    float p_inv;
    float a;             // sum of p (t - s) / tau
    float2 part[kMaxCluster * kWarps];  // (maximum, sum) of every warp of the cluster's slices
    float2 top[kMaxCluster];            // (sum over the listed columns, their number) of every slice
};

__host__ __device__ constexpr size_t align16(size_t n) { return (n + 15) & ~size_t(15); }
// Dynamic shared memory: the chunk, then four arrays of `top` words.
size_t row_smem(int chunk, int top) { return size_t(chunk) * 16 + align16(size_t(top) * 4) * 4; }

// The teacher's list of a row, by one warp: columns, exponentials and the
// student's logits there (they are read here, before any gradient is stored).
template <class T>
__device__ __forceinline__ void read_list(const DistillArgs& a, int64_t row, const T* logits, int* s_idx,
                                          float* s_p, float* s_s, Shared& sh) {
    constexpr int kBatch = 4;  // loads in flight per lane
    const int K = a.top, lane = threadIdx.x & 31;
    bool any = false, bad = false;
    float tm = kNegInf, mt = kNegInf;
    for (int k0 = lane; k0 < K; k0 += 32 * kBatch) {
        int64_t j[kBatch];
        float t[kBatch], s[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = k0 + 32 * i;
            j[i] = k < K ? load_index(a, row * K + k) : -1;
            t[i] = k < K ? load_top(a, row * K + k) : kNegInf;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (t[i] == kNegInf) j[i] = -1;
            if (j[i] >= a.vocab) {
                bad = true;
                j[i] = -1;
            }
            s[i] = j[i] >= 0 ? Elem<T>::to_f(logits[j[i]]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int k = k0 + 32 * i;
            if (k >= K) break;
            s_idx[k] = j[i] >= 0 ? static_cast<int>(j[i]) : -1;
            s_p[k] = t[i];
            s_s[k] = s[i];
            if (j[i] >= 0) {
                any = true;
                tm = fmaxf(tm, t[i]);
                mt = fmaxf(mt, s[i]);
            }
        }
    }
    tm = warp_reduce(tm, MaxOp());
    mt = warp_reduce(mt, MaxOp());
    const bool full = a.lse != nullptr;
    const float base = full ? a.lse[row] : tm;
    float hi = 0.0f, lo = 0.0f, sum = 0.0f;
    for (int k = lane; k < K; k += 32) {
        float e = 0.0f;
        if (s_idx[k] >= 0) {
            const float t = s_p[k], s = s_s[k];
            e = teacher_exp(a, t, base, full);
            if (e != 0.0f)
                sum += s == kNegInf ? INFINITY : e * fmaf(s, a.k2_slip, fmaf(t - s, a.inv_hi, (t - s) * a.inv_lo));
            float err;
            hi = two_sum_f32(hi, e, err);
            lo += err;
        }
        s_p[k] = e;
    }
    warp_sum_pairs(hi, lo);
    sum = warp_reduce(sum, AddOp());
    const float p_inv = full ? 1.0f : 1.0f / (hi + lo);
    __syncwarp();
    if (!full)
        for (int k = lane; k < K; k += 32) s_p[k] *= p_inv;
    any = __any_sync(0xffffffffu, any);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        sh.live = any || bad;
        sh.bad = bad;
        sh.tm = tm;
        sh.m_top = mt;
        sh.p_hi = hi;
        sh.p_lo = lo;
        sh.p_inv = p_inv;
        sh.a = sum;
    }
    __syncwarp();
}

// Takes the listed columns out of a chunk, by one warp: s_lead gets the mass
// of a column at its first slot and -1 at others, and the student's
// exponentials there are summed.  Each slot first writes its number into the
// chunk: one that reads another's back shares its column.
template <class T>
__device__ __forceinline__ void take_out(const DistillArgs& a, T* e, int j0, int j1, int j_base, const int* s_idx,
                                         const float* s_p, const float* s_s, float* s_lead, float m2_top,
                                         float& sum_top, float& listed) {
    const int K = a.top, lane = threadIdx.x & 31;
    for (int k = lane; k < K; k += 32) {
        const int j = s_idx[k];
        if (j < j0 || j >= j1) continue;
        const uint16_t tag = static_cast<uint16_t>(k);
        memcpy(&e[j - j_base], &tag, 2);
    }
    __syncwarp();
    bool twice = false;
    for (int k = lane; k < K; k += 32) {
        const int j = s_idx[k];
        if (j < j0 || j >= j1) continue;
        uint16_t tag;
        memcpy(&tag, &e[j - j_base], 2);
        twice |= tag != k;
    }
    twice = __any_sync(0xffffffffu, twice);
    for (int k = lane; k < K; k += 32) {
        const int j = s_idx[k];
        if (j < j0 || j >= j1) continue;
        e[j - j_base] = Elem<T>::from_f(kNegInf);
        float p = s_p[k];
        bool first = true;
        if (twice) {  // rare: a column's first slot takes the sum over its slots
            p = 0.0f;
            for (int l = 0; l < K; ++l) {
                if (s_idx[l] != j) continue;
                first = first && l >= k;
                p += s_p[l];
            }
        }
        s_lead[k] = first ? p : -1.0f;
        if (first) {
            sum_top += m2_top == kNegInf ? 0.0f : ex2(fmaf(s_s[k], a.k2, -m2_top));
            listed += 1.0f;
        }
    }
}

// One row per cluster.
template <class T, bool kGrad>
__global__ void __launch_bounds__(kThreads) distill_row_kernel(const DistillArgs a) {
    constexpr int kPer = Elem<T>::kPer;
    extern __shared__ uint4 buf[];
    __shared__ Shared sh;
    const int K = a.top;
    const size_t kstep = align16(size_t(K) * 4) / 4;
    int* const s_idx = reinterpret_cast<int*>(buf + a.chunk);   // column, -1 for an empty slot
    float* const s_p = reinterpret_cast<float*>(s_idx) + kstep;  // p
    float* const s_s = s_p + kstep;                              // student logit
    float* const s_lead = s_s + kstep;                           // p of the column at its first slot, else -1

    uint32_t C;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
    const uint32_t rank = cluster_ctarank();
    const int64_t row = blockIdx.x / C;
    const RowView<T> v(a.logits, a.ld, row, a.vocab);
    const int g_lo = min(v.n, static_cast<int>(rank) * a.slice), g_hi = min(v.n, g_lo + a.slice);
    T* const out = kGrad ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
    const bool same = kGrad && ((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T)) == static_cast<unsigned>(v.off);
    const float w = a.weights ? a.weights[row] : 1.0f;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n_chunks = max(1, (g_hi - g_lo + a.chunk - 1) / a.chunk);

    bool live = w != 0.0f;
    if (live) {
        load_chunk<T>(v, a.vocab, g_lo, min(g_hi, g_lo + a.chunk), buf);
        if (warp == 0) read_list<T>(a, row, v.row, s_idx, s_p, s_s, sh);
        cp_async_wait();
        __syncthreads();
        live = sh.live != 0;
    }
    if (!live) {
        if (kGrad) zero_slice<T>(v, out, a.vocab, same, g_lo, g_hi);
        if (rank == 0 && tid < DISTILL_STATS) {
            if (tid == 0) a.loss[row] = 0.0f;
            if (!kGrad) a.stats[row * DISTILL_STATS + tid] = 0.0f;
        }
        return;  // the whole cluster leaves here, as all of it read the same row
    }
    const float m2_top = sh.m_top * a.k2;  // reference of the listed columns (all slices use this one)

    // ---- maximum and sum of this thread's part of the slice
    float m2 = kNegInf, sum = 0.0f, sum_top = 0.0f, listed = 0.0f;
    for (int c = 0; c < n_chunks; ++c) {
        const int g0 = g_lo + c * a.chunk, n = max(0, min(g_hi, g0 + a.chunk) - g0);
        if (c > 0) {
            __syncthreads();  // the chunk before is no longer read
            load_chunk<T>(v, a.vocab, g0, g0 + n, buf);
            cp_async_wait();
            __syncthreads();
        }
        if (warp == 0) {
            const int j_base = g0 * kPer - v.off;
            take_out<T>(a, reinterpret_cast<T*>(buf), max(j_base, 0), j_base + n * kPer, j_base, s_idx, s_p, s_s,
                        s_lead, m2_top, sum_top, listed);
        }
        __syncthreads();
        float m = kNegInf;
        for (int g = tid; g < n; g += kThreads) m = fmaxf(m, Elem<T>::max_of(buf[g]));
        m *= a.k2;
        if (m > m2) {
            sum *= rescale(m2, m);
            m2 = m;
        }
        const float ref = m2 == kNegInf ? 0.0f : m2;
        for (int g = tid; g < n; g += kThreads) {
            float x[kPer];
            Elem<T>::unpack(buf[g], x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) sum += ex2(fmaf(x[i], a.k2, -ref));
        }
    }

    // ---- the row's sums: every warp's pair goes to every CTA of the cluster
    {
        const float mw = warp_reduce(m2, MaxOp());
        sum = warp_reduce(sum * rescale(m2, mw), AddOp());
        if (warp == 0) {
            sum_top = warp_reduce(sum_top, AddOp());
            listed = warp_reduce(listed, AddOp());
        }
        if (lane < static_cast<int>(C)) {
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                             mapa_shared(smem_u32(&sh.part[rank * kWarps + warp]), lane)),
                         "f"(mw), "f"(sum)
                         : "memory");
            if (warp == 0)
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                                 mapa_shared(smem_u32(&sh.top[rank]), lane)),
                             "f"(sum_top), "f"(listed)
                             : "memory");
        }
    }
    cluster_sync_all();
    float m2o = kNegInf, s_o = 0.0f, s_t = 0.0f;
    listed = 0.0f;
    for (uint32_t i = lane; i < C * kWarps; i += 32) m2o = fmaxf(m2o, sh.part[i].x);
    m2o = warp_reduce(m2o, MaxOp());
    for (uint32_t i = lane; i < C * kWarps; i += 32) s_o += sh.part[i].y * rescale(sh.part[i].x, m2o);
    s_o = warp_reduce(s_o, AddOp());
    for (uint32_t r = 0; r < C; ++r) {
        s_t += sh.top[r].x;
        listed += sh.top[r].y;
    }
    const float M2 = fmaxf(m2o, m2_top);
    const float f_o = rescale(m2o, M2);
    const float S = s_o * f_o + s_t * rescale(m2_top, M2);
    const float inv_S = sh.bad ? NAN : 1.0f / S;
    // the teacher's mass outside its list; none where the list names every column
    float p_r = a.lse ? (1.0f - sh.p_hi) - sh.p_lo : 0.0f;
    if (p_r < 0.0f || listed >= static_cast<float>(a.vocab)) p_r = 0.0f;
    float B = f_o * inv_S;
    if (p_r > 0.0f && s_o > 0.0f) B -= p_r / s_o;
    const float ref_o = m2o == kNegInf ? 0.0f : m2o;

    // ---- the loss, by one thread (a few fp64 operations a row: that pipe is slow)
    if (rank == 0 && tid == kThreads - 32) {
        const double ln_sum = static_cast<double>(M2) * kLn2 + log_wide(S);  // of the student
        double L;
        if (a.lse) {
            const double P = static_cast<double>(sh.p_hi) + static_cast<double>(sh.p_lo);
            L = static_cast<double>(sh.a) + P * (ln_sum - static_cast<double>(a.lse[row]));
        } else {
            L = static_cast<double>(sh.a * sh.p_inv) + ln_sum - static_cast<double>(sh.tm) * a.inv_tau -
                log_wide(sh.p_hi + sh.p_lo);
        }
        if (p_r != 0.0f)
            L += static_cast<double>(p_r) *
                 (log_wide(p_r) - (static_cast<double>(m2o) * kLn2 + log_wide(s_o) - ln_sum));
        if (sh.bad) L = NAN;
        a.loss[row] = static_cast<float>(static_cast<double>(w * a.tau * a.tau) * L);
        if (!kGrad) {
            float4* const st = reinterpret_cast<float4*>(a.stats + row * DISTILL_STATS);
            st[0] = make_float4(M2, inv_S, ref_o, B);
            st[1] = make_float4(sh.tm, sh.p_inv, 1.0f, 0.0f);
        }
    }
    if constexpr (kGrad) {
        const float gs = w * a.tau, mul = gs * B;
        for (int c = n_chunks - 1; c >= 0; --c) {
            const int g0 = g_lo + c * a.chunk, g1 = min(g_hi, g0 + a.chunk);
            if (c != n_chunks - 1) {
                __syncthreads();
                load_chunk<T>(v, a.vocab, g0, g1, buf);
                cp_async_wait();
                __syncthreads();
            }
            for (int g = g0 + tid; g < g1; g += kThreads) {
                float x[kPer];
                Elem<T>::unpack(buf[g - g0], x);
#pragma unroll
                for (int i = 0; i < kPer; ++i) x[i] = ex2(fmaf(x[i], a.k2, -ref_o)) * mul;
                store_granule<T>(out, g, v.off, a.vocab, same && v.whole(g, a.vocab), x);
            }
        }
        __syncthreads();
        const int j0 = max(0, g_lo * kPer - v.off), j1 = min(a.vocab, g_hi * kPer - v.off);
        for (int k = tid; k < K; k += kThreads) {
            const int j = s_idx[k];
            if (j >= j0 && j < j1 && !(s_lead[k] < 0.0f))
                out[j] = Elem<T>::from_f(gs * (ex2(fmaf(s_s[k], a.k2, -M2)) * inv_S - s_lead[k]));
        }
    }
}

// Gradient from saved statistics: one CTA per slice of a row, no exchange.
constexpr int kInFlight = 4;                       // granules a thread loads at a time
constexpr int kBwdSlice = kThreads * kInFlight * 2;  // granules per CTA

template <class T>
__global__ void __launch_bounds__(kThreads) distill_backward_kernel(const DistillArgs a, int n_slices) {
    constexpr int kPer = Elem<T>::kPer;
    __shared__ int s_j[DISTILL_MAX_TOP];
    __shared__ float s_p[DISTILL_MAX_TOP], s_s[DISTILL_MAX_TOP];
    __shared__ int s_n;
    __shared__ int s_slot[DISTILL_MAX_TOP];
    const int64_t row = blockIdx.x / n_slices;
    const int part = static_cast<int>(blockIdx.x % n_slices);
    const RowView<T> v(a.logits, a.ld, row, a.vocab);
    const int g_lo = part * kBwdSlice, g_hi = min(v.n, g_lo + kBwdSlice);
    if (g_lo >= g_hi) return;
    T* const out = static_cast<T*>(a.dlogits) + row * a.ldd;
    const bool same = ((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T)) == static_cast<unsigned>(v.off);
    const float w = a.weights ? a.weights[row] : 1.0f;
    const float4 st0 = *reinterpret_cast<const float4*>(a.stats + row * DISTILL_STATS);
    const float4 st1 = *reinterpret_cast<const float4*>(a.stats + row * DISTILL_STATS + 4);
    const int tid = threadIdx.x;
    if (w == 0.0f || st1.z == 0.0f) {
        zero_slice<T>(v, out, a.vocab, same, g_lo, g_hi);
        return;
    }
    const float M2 = st0.x, inv_S = st0.y, ref_o = st0.z;
    const float gs = w * a.tau * (a.grad ? a.grad[row] : 1.0f), mul = gs * st0.w;
    // this slice's part of the list; the student's logits there are read
    // before any gradient is stored (dlogits may be logits)
    if (tid == 0) s_n = 0;
    __syncthreads();
    const int j0 = max(0, g_lo * kPer - v.off), j1 = min(a.vocab, g_hi * kPer - v.off);
    const bool full = a.lse != nullptr;
    const float base = full ? a.lse[row] : st1.x;
    for (int k = tid; k < a.top; k += kThreads) {
        const int64_t j = load_index(a, row * a.top + k);
        if (j < j0 || j >= j1) continue;
        const float t = load_top(a, row * a.top + k);
        if (t == kNegInf) continue;
        const int n = atomicAdd(&s_n, 1);
        s_j[n] = static_cast<int>(j);
        s_slot[n] = k;
        s_s[n] = Elem<T>::to_f(v.row[j]);
        s_p[n] = teacher_exp(a, t, base, full) * st1.y;
    }
    __syncthreads();
    for (int g = g_lo + tid; g < g_hi; g += kThreads * kInFlight) {
        uint4 b[kInFlight];
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int gg = g + i * kThreads;
            if (gg < g_hi && v.whole(gg, a.vocab)) b[i] = *reinterpret_cast<const uint4*>(v.granule(gg));
        }
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int gg = g + i * kThreads;
            if (gg >= g_hi) break;
            float x[kPer];
            const bool whole = v.whole(gg, a.vocab);
            if (whole) {
                Elem<T>::unpack(b[i], x);
            } else {
                for (int e = 0; e < kPer; ++e) {
                    const int j = gg * kPer + e - v.off;
                    x[e] = j >= 0 && j < a.vocab ? Elem<T>::to_f(v.row[j]) : 0.0f;
                }
            }
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[e] = ex2(fmaf(x[e], a.k2, -ref_o)) * mul;
            store_granule<T>(out, gg, v.off, a.vocab, same && whole, x);
        }
    }
    __syncthreads();
    const int n = s_n;
    for (int i = tid; i < n; i += kThreads) {
        // a column listed more than once: its first slot writes the sum, taken
        // in the order of the slots
        const int j = s_j[i];
        bool first = true, twice = false;
        for (int l = 0; l < n; ++l) {
            if (l == i || s_j[l] != j) continue;
            twice = true;
            first = first && s_slot[l] > s_slot[i];
        }
        if (!first) continue;
        float p = s_p[i];
        if (twice) {
            p = 0.0f;
            for (int after = -1;;) {
                int best = -1;
                for (int l = 0; l < n; ++l)
                    if (s_j[l] == j && s_slot[l] > after && (best < 0 || s_slot[l] < s_slot[best])) best = l;
                if (best < 0) break;
                p += s_p[best];
                after = s_slot[best];
            }
        }
        out[j] = Elem<T>::from_f(gs * (ex2(fmaf(s_s[i], a.k2, -M2)) * inv_S - p));
    }
}

// ------------------------------------------------------------- host side

hess_status ds_fail(hess_status s, const char* fmt, ...) {
    char buf[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

#define DS_TRY(call)                                                                           \
    do {                                                                                       \
        cudaError_t e_ = (call);                                                               \
        if (e_ != cudaSuccess)                                                                 \
            return ds_fail(HESS_ERR_CUDA, "%s failed: %s", #call, cudaGetErrorString(e_));     \
    } while (0)

size_t elem_size(int32_t dtype) { return dtype == HESS_F32 ? 4 : 2; }
bool known(int32_t dtype) { return dtype == HESS_BF16 || dtype == HESS_F16 || dtype == HESS_F32; }

// Checks shared by the three calls; fills `a`.
hess_status ds_args(DistillArgs& a, const void* logits, int64_t ld, int64_t rows, int64_t vocab, int32_t dtype,
                    const void* top_logits, int32_t top_dtype, const void* top_index, int32_t index_bytes,
                    int64_t top, const float* lse, const float* weights, double temperature) {
    if (rows < 0) return ds_fail(HESS_ERR_INVALID, "rows < 0");
    if (vocab < 1) return ds_fail(HESS_ERR_INVALID, "vocab must be positive");
    if (vocab > (int64_t(1) << 30)) return ds_fail(HESS_ERR_UNSUPPORTED, "vocab > 2^30");
    if (rows > (int64_t(1) << 27)) return ds_fail(HESS_ERR_UNSUPPORTED, "rows > 2^27");
    if (!known(dtype)) return ds_fail(HESS_ERR_INVALID, "unknown dtype %d", dtype);
    if (!known(top_dtype)) return ds_fail(HESS_ERR_INVALID, "unknown top_dtype %d", top_dtype);
    if (index_bytes != 4 && index_bytes != 8)
        return ds_fail(HESS_ERR_INVALID, "index_bytes must be 4 or 8 (got %d)", index_bytes);
    if (ld < vocab) return ds_fail(HESS_ERR_INVALID, "ld < vocab");
    if (top < 1) return ds_fail(HESS_ERR_INVALID, "top must be positive");
    if (top > DISTILL_MAX_TOP) return ds_fail(HESS_ERR_UNSUPPORTED, "top > %d", DISTILL_MAX_TOP);
    if (!(temperature >= 1e-3 && temperature <= 1e3))
        return ds_fail(HESS_ERR_INVALID, "temperature must be in [1e-3, 1e3]");
    if (rows > 0) {
        if (!logits) return ds_fail(HESS_ERR_INVALID, "logits is NULL");
        if (!top_logits || !top_index) return ds_fail(HESS_ERR_INVALID, "top_logits or top_index is NULL");
        const uintptr_t lp = reinterpret_cast<uintptr_t>(logits), tp = reinterpret_cast<uintptr_t>(top_logits);
        if (lp % elem_size(dtype) || tp % elem_size(top_dtype) ||
            reinterpret_cast<uintptr_t>(top_index) % static_cast<unsigned>(index_bytes) ||
            reinterpret_cast<uintptr_t>(lse) % 4 || reinterpret_cast<uintptr_t>(weights) % 4)
            return ds_fail(HESS_ERR_INVALID, "a pointer is not aligned to its element");
    }
    a = DistillArgs{};
    a.logits = logits;
    a.ld = ld;
    a.rows = rows;
    a.vocab = static_cast<int32_t>(vocab);
    a.top = static_cast<int32_t>(top);
    a.top_logits = top_logits;
    a.top_index = top_index;
    a.top_dtype = top_dtype;
    a.index_bytes = index_bytes;
    a.lse = lse;
    a.weights = weights;
    a.inv_tau = 1.0 / temperature;
    a.tau = static_cast<float>(temperature);
    a.inv_hi = static_cast<float>(a.inv_tau);
    a.inv_lo = static_cast<float>(a.inv_tau - static_cast<double>(a.inv_hi));
    a.k2 = static_cast<float>(1.0 / (temperature * kLn2));
    a.k2_slip = static_cast<float>(a.inv_tau - static_cast<double>(a.k2) * kLn2);
    return HESS_OK;
}

hess_status ds_buffers(const DistillArgs& a, int* dev_out) {
    int dev = 0;
    DS_TRY(cudaGetDevice(&dev));
    const struct {
        const void* p;
        const char* name;
    } bufs[] = {{a.logits, "logits"}, {a.top_logits, "top_logits"}, {a.top_index, "top_index"},
                {a.lse, "teacher_lse"}, {a.weights, "weights"}, {a.grad, "grad"}, {a.loss, "loss"},
                {a.stats, "stats"}, {a.dlogits, "dlogits"}};
    for (const auto& b : bufs) {
        char why[128];
        if (!b.p) continue;
        if (const char* w = device_ptr_problem(b.p, dev, why)) return ds_fail(HESS_ERR_INVALID, "%s %s", b.name, w);
    }
    *dev_out = dev;
    return HESS_OK;
}

hess_status ds_output(const DistillArgs& a, int32_t dtype, bool want_grad) {
    if (want_grad && a.rows > 0) {
        if (!a.dlogits) return ds_fail(HESS_ERR_INVALID, "dlogits is NULL");
        if (reinterpret_cast<uintptr_t>(a.dlogits) % elem_size(dtype))
            return ds_fail(HESS_ERR_INVALID, "a pointer is not aligned to its element");
    }
    if (want_grad) {
        if (a.ldd < a.vocab) return ds_fail(HESS_ERR_INVALID, "ldd < vocab");
        if (a.rows > 0) {
            const uintptr_t s0 = reinterpret_cast<uintptr_t>(a.logits), d0 = reinterpret_cast<uintptr_t>(a.dlogits);
            const size_t es = elem_size(dtype);
            const uintptr_t s1 = s0 + ((a.rows - 1) * a.ld + a.vocab) * es;
            const uintptr_t d1 = d0 + ((a.rows - 1) * a.ldd + a.vocab) * es;
            const bool in_place = s0 == d0 && a.ld == a.ldd;
            if (!in_place && s0 < d1 && d0 < s1)
                return ds_fail(HESS_ERR_INVALID, "dlogits overlaps logits without being logits");
        }
    }
    return HESS_OK;
}

constexpr size_t kMaxDynamic = 220 * 1024;

hess_status ds_prepare(int dev, int* sms) {
    static std::mutex mu;
    static int count[128] = {};
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 128) return ds_fail(HESS_ERR_UNSUPPORTED, "device index %d", dev);
    if (!count[dev]) {
        for (auto fn : {distill_row_kernel<__nv_bfloat16, false>, distill_row_kernel<__nv_bfloat16, true>,
                        distill_row_kernel<__half, false>, distill_row_kernel<__half, true>,
                        distill_row_kernel<float, false>, distill_row_kernel<float, true>})
            DS_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kMaxDynamic)));
        int n = 0;
        DS_TRY(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
        count[dev] = n;
    }
    *sms = count[dev];
    return HESS_OK;
}

template <bool kGrad>
hess_status launch_rows(DistillArgs& a, int32_t dtype, cudaStream_t s) {
    int dev = 0, sms = 0;
    hess_status st = ds_buffers(a, &dev);
    if (st != HESS_OK) return st;
    st = ds_prepare(dev, &sms);
    if (st != HESS_OK) return st;
    const int per = static_cast<int>(16 / elem_size(dtype));
    const int granules = static_cast<int>((static_cast<int64_t>(a.vocab) + 2 * (per - 1)) / per);
    // CTAs per row: one, until its slice fits in what is left of shared memory
    // with three CTAs on an SM (64 KB each).
    int C = 1;
    while (C < kMaxCluster && (granules + C - 1) / C > 4096) C *= 2;
    a.slice = (granules + C - 1) / C;
    a.chunk = a.slice < 12288 ? a.slice : 12288;
    const size_t smem = row_smem(a.chunk, a.top);
    auto fn = dtype == HESS_BF16 ? distill_row_kernel<__nv_bfloat16, kGrad>
              : dtype == HESS_F16 ? distill_row_kernel<__half, kGrad> : distill_row_kernel<float, kGrad>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * C), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(C);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    DS_TRY(cudaLaunchKernelEx(&cfg, fn, a));
    return HESS_OK;
}

}  // namespace
}  // namespace hk

#define DS_EXPORT extern "C" __attribute__((visibility("default")))

DS_EXPORT hess_status distill_forward(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int32_t dtype,
                                      const void* top_logits, int32_t top_dtype, const void* top_index,
                                      int32_t index_bytes, int64_t top, const float* teacher_lse,
                                      const float* weights, double temperature, float* loss, float* stats,
                                      hess_stream_t stream) {
    hk::DistillArgs a;
    hess_status st = hk::ds_args(a, logits, ld, rows, vocab, dtype, top_logits, top_dtype, top_index, index_bytes,
                                 top, teacher_lse, weights, temperature);
    if (st != HESS_OK) return st;
    if (rows == 0) return HESS_OK;
    if (!loss || !stats) return hk::ds_fail(HESS_ERR_INVALID, "loss or stats is NULL");
    if (reinterpret_cast<uintptr_t>(loss) % 4 || reinterpret_cast<uintptr_t>(stats) % 16)
        return hk::ds_fail(HESS_ERR_INVALID, "loss must be 4-byte and stats 16-byte aligned");
    a.loss = loss;
    a.stats = stats;
    return hk::launch_rows<false>(a, dtype, static_cast<cudaStream_t>(stream));
}

DS_EXPORT hess_status distill_step(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int32_t dtype,
                                   const void* top_logits, int32_t top_dtype, const void* top_index,
                                   int32_t index_bytes, int64_t top, const float* teacher_lse,
                                   const float* weights, double temperature, float* loss, void* dlogits,
                                   int64_t ldd, hess_stream_t stream) {
    hk::DistillArgs a;
    hess_status st = hk::ds_args(a, logits, ld, rows, vocab, dtype, top_logits, top_dtype, top_index, index_bytes,
                                 top, teacher_lse, weights, temperature);
    if (st != HESS_OK) return st;
    a.loss = loss;
    a.dlogits = dlogits;
    a.ldd = ldd;
    st = hk::ds_output(a, dtype, true);
    if (st != HESS_OK) return st;
    if (rows == 0) return HESS_OK;
    if (!loss || reinterpret_cast<uintptr_t>(loss) % 4)
        return hk::ds_fail(HESS_ERR_INVALID, "loss is NULL or not 4-byte aligned");
    return hk::launch_rows<true>(a, dtype, static_cast<cudaStream_t>(stream));
}

DS_EXPORT hess_status distill_backward(const void* logits, int64_t ld, int64_t rows, int64_t vocab, int32_t dtype,
                                       const void* top_logits, int32_t top_dtype, const void* top_index,
                                       int32_t index_bytes, int64_t top, const float* teacher_lse,
                                       const float* weights, double temperature, const float* stats,
                                       const float* grad, void* dlogits, int64_t ldd, hess_stream_t stream) {
    hk::DistillArgs a;
    hess_status st = hk::ds_args(a, logits, ld, rows, vocab, dtype, top_logits, top_dtype, top_index, index_bytes,
                                 top, teacher_lse, weights, temperature);
    if (st != HESS_OK) return st;
    a.stats = const_cast<float*>(stats);
    a.grad = grad;
    a.dlogits = dlogits;
    a.ldd = ldd;
    st = hk::ds_output(a, dtype, true);
    if (st != HESS_OK) return st;
    if (rows == 0) return HESS_OK;
    if (!stats || reinterpret_cast<uintptr_t>(stats) % 16 || reinterpret_cast<uintptr_t>(grad) % 4)
        return hk::ds_fail(HESS_ERR_INVALID, "stats is NULL or not 16-byte aligned, or grad not 4-byte aligned");
    int dev = 0;
    st = hk::ds_buffers(a, &dev);
    if (st != HESS_OK) return st;
    const int per = static_cast<int>(16 / hk::elem_size(dtype));
    const int64_t granules = (vocab + 2 * (per - 1)) / per;
    const int n_slices = static_cast<int>((granules + hk::kBwdSlice - 1) / hk::kBwdSlice);
    if (rows * n_slices > 0x7fffffffll) return hk::ds_fail(HESS_ERR_UNSUPPORTED, "rows * vocab is too large");
    const unsigned grid = static_cast<unsigned>(rows * n_slices);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == HESS_BF16)
        hk::distill_backward_kernel<__nv_bfloat16><<<grid, hk::kThreads, 0, s>>>(a, n_slices);
    else if (dtype == HESS_F16)
        hk::distill_backward_kernel<__half><<<grid, hk::kThreads, 0, s>>>(a, n_slices);
    else
        hk::distill_backward_kernel<float><<<grid, hk::kThreads, 0, s>>>(a, n_slices);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return hk::ds_fail(HESS_ERR_CUDA, "distill_backward: %s", cudaGetErrorString(e));
    return HESS_OK;
}
