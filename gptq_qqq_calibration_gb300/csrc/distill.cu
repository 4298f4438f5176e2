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
// distill_stream_kernel does this for a stream of rows with one CTA per SM
// that never waits for memory it could have asked for earlier: its buffers
// hold several rows' slices, each filled by one bulk copy; a warp per buffer
// reads the teacher's list meanwhile; and the compute warps take the sums of
// row i + 1 before they write row i's gradient, so that the exchange between
// the CTAs of a cluster hides behind it.  Rows too long for two slices per SM
// go to distill_row_kernel, one cluster per row, its slice in pieces.
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
    int32_t chunk;  // distill_row_kernel: granules a CTA holds in shared memory
    int32_t n_buf;  // distill_stream_kernel: slices a CTA holds
    int32_t n_list;  // and lists
};

// ---------------------------------------------------------------- elements

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a * b + c on two fp32 values at once.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t both(float x) { return pack2(__float_as_uint(x), __float_as_uint(x)); }

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

// Running sum hi + lo of fp32 terms and products that keeps its rounding
// errors, for the handful of terms of a row's loss that are large next to it.
struct Pair {
    float hi = 0.0f, lo = 0.0f;
    __device__ void add(float x) {
        float e;
        hi = two_sum_f32(hi, x, e);
        lo += e;
    }
    __device__ void add_product(float a, float b) {
        const float p = __fmul_rn(a, b);
        add(p);
        lo += __fmaf_rn(a, b, -p);
    }
    __device__ void add(const Pair& q) {
        add(q.hi);
        lo += q.lo;
    }
    // x ln 2
    __device__ void add_ln2(float x) {
        constexpr float h = static_cast<float>(kLn2);
        add_product(x, h);
        lo += x * static_cast<float>(kLn2 - static_cast<double>(h));
    }
    // sign * ln(x) for a normal x: its exponent's part exactly, its mantissa's
    // (at most ln 2 / 2) by logf
    __device__ void add_log(float x, float sign) {
        int e = static_cast<int>(__float_as_uint(x) >> 23) - 127;
        float m = __uint_as_float((__float_as_uint(x) & 0x7fffffu) | 0x3f800000u);
        if (m > 1.41421356f) {
            m *= 0.5f;
            e += 1;
        }
        add_ln2(sign * static_cast<float>(e));
        add(sign * logf(m));
    }
    __device__ float value() const { return hi + lo; }
};

// 2^(a - b) with b >= a; 0 when a is -inf (whatever b is).
__device__ __forceinline__ float rescale(float a, float b) { return a == kNegInf ? 0.0f : ex2(a - b); }

__device__ __forceinline__ void st_cluster_f32x2(uint32_t addr, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
// Two floats to a CTA of the cluster, counted as 8 bytes on its barrier, whose
// phase so covers them.  (A plain store and an arrive with release would have
// to wait, 2,300 cycles here, for this thread's earlier global stores too.)
__device__ __forceinline__ void send_f32x2(uint32_t addr, float x, float y, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr),
                 "f"(x), "f"(y), "r"(bar)
                 : "memory");
}

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
__device__ __forceinline__ void zero_slice(const RowView<T>& v, T* out_row, int vocab, bool same, int g0, int g1,
                                           int t, int n_threads) {
    float z[Elem<T>::kPer] = {};
    for (int g = g0 + t; g < g1; g += n_threads)
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

// What the warp that reads the teacher's list leaves for the others.
struct ListInfo {
    int live, bad;
    float w;             // the row's weight
    float tm, m_top;     // largest listed logit, teacher's and student's
    float p_hi, p_lo;    // sum of the list's exponentials
    float p_inv;
    float a;             // sum of p (t - s) / tau
    float lse;           // the teacher's, when given
};

template <class T>
__device__ __forceinline__ void add_exps(const uint4& v, uint64_t kk, uint64_t ref, uint64_t& s0, uint64_t& s1) {
    constexpr int kPer = Elem<T>::kPer;
    float x[kPer];
    Elem<T>::unpack(v, x);
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
        float u0, u1, v0, v1;
        unpack2(fma2(pack2(__float_as_uint(x[i]), __float_as_uint(x[i + 1])), kk, ref), u0, u1);
        unpack2(fma2(pack2(__float_as_uint(x[i + 2]), __float_as_uint(x[i + 3])), kk, ref), v0, v1);
        s0 = add2(s0, pack2(__float_as_uint(ex2(u0)), __float_as_uint(ex2(u1))));
        s1 = add2(s1, pack2(__float_as_uint(ex2(v0)), __float_as_uint(ex2(v1))));
    }
}

// Sum of 2^(x k2 - m2) over this thread's granules t, t + n_threads, ... of a slice.
template <class T>
__device__ __forceinline__ float exp_sum(const uint4* buf, int n, int t, int n_threads, float k2, float m2) {
    const uint64_t kk = both(k2), ref = both(-m2);
    uint64_t s0 = 0, s1 = 0;
    int g = t;
    for (; g + 3 * n_threads < n; g += 4 * n_threads) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = buf[g + i * n_threads];
#pragma unroll
        for (int i = 0; i < 4; ++i) add_exps<T>(v[i], kk, ref, s0, s1);
    }
    for (; g < n; g += n_threads) add_exps<T>(buf[g], kk, ref, s0, s1);
    float a, b;
    unpack2(add2(s0, s1), a, b);
    return a + b;
}

// Reference and sum of a warp's share of a slice (its lanes are threads t of
// n_threads), the same in every lane.  One pass suffices when the listed
// columns' maximum `guess` is a fair reference for the others, as it nearly
// always is: a sum that neither overflows nor comes near underflow is as exact
// with one reference as with another.  Otherwise the share's own maximum is
// taken first.
template <class T>
__device__ __forceinline__ void slice_sums(const uint4* buf, int n, int t, int n_threads, float k2, float guess,
                                           float& m2, float& sum) {
    m2 = guess;
    sum = 0.0f;
    if (fabsf(guess) < 1e30f) sum = warp_reduce(exp_sum<T>(buf, n, t, n_threads, k2, guess), AddOp());
    if (sum > 1e-12f && sum < 1e30f) return;
    float m = kNegInf;
    for (int g = t; g < n; g += n_threads) m = fmaxf(m, Elem<T>::max_of(buf[g]));
    m2 = warp_reduce(m, MaxOp()) * k2;
    sum = warp_reduce(exp_sum<T>(buf, n, t, n_threads, k2, m2 == kNegInf ? 0.0f : m2), AddOp());
}

// The sums of a whole row, from its slices' parts; every lane gets them.
struct RowSums {
    float M2, S, inv_S;   // reference and sum of the whole row
    float m2o, s_o;       // of the columns outside the list
    float ref_o, B;       // gradient outside the list: w tau B 2^(s k2 - ref_o)
    float p_r;            // the teacher's mass outside its list
};
__device__ __forceinline__ RowSums row_sums(const DistillArgs& a, const ListInfo& info, const float2* part, int n_part,
                                            const float2* top, int n_top) {
    const int lane = threadIdx.x & 31;
    RowSums r;
    r.m2o = kNegInf;
    r.s_o = 0.0f;
    for (int i = lane; i < n_part; i += 32) r.m2o = fmaxf(r.m2o, part[i].x);
    r.m2o = warp_reduce(r.m2o, MaxOp());
    for (int i = lane; i < n_part; i += 32) r.s_o += part[i].y * rescale(part[i].x, r.m2o);
    r.s_o = warp_reduce(r.s_o, AddOp());
    float s_t = 0.0f, listed = 0.0f;
    for (int i = 0; i < n_top; ++i) {
        s_t += top[i].x;
        listed += top[i].y;
    }
    const float m2_top = info.m_top * a.k2;
    r.M2 = fmaxf(r.m2o, m2_top);
    const float f_o = rescale(r.m2o, r.M2);
    r.S = r.s_o * f_o + s_t * rescale(m2_top, r.M2);
    r.inv_S = info.bad ? NAN : 1.0f / r.S;
    r.p_r = a.lse ? (1.0f - info.p_hi) - info.p_lo : 0.0f;
    // none where the list names every column
    if (r.p_r < 0.0f || listed >= static_cast<float>(a.vocab)) r.p_r = 0.0f;
    r.B = f_o * r.inv_S;
    if (r.p_r > 0.0f && r.s_o > 0.0f) r.B -= r.p_r / r.s_o;
    r.ref_o = r.m2o == kNegInf ? 0.0f : r.m2o;
    return r;
}

// The row's loss.  Its terms cancel (a log-sum of 20 against logits of 20 for a
// loss of 0.1), so they are summed with their rounding errors; fp64 would do,
// but one dependent chain of it takes 4,800 cycles here against some 500.
__device__ __forceinline__ float row_loss(const DistillArgs& a, const ListInfo& info, const RowSums& r) {
    if (info.bad) return NAN;
    const float scale = info.w * a.tau * a.tau;
    constexpr float ln2 = static_cast<float>(kLn2);
    const bool full = a.lse != nullptr;
    // infinities and NaN, which the pairs do not carry
    const float ln_s = r.M2 * ln2 + logf(r.S);
    const float rest = r.p_r != 0.0f ? r.p_r * (logf(r.p_r) - (r.m2o * ln2 + logf(r.s_o) - ln_s)) : 0.0f;
    const float plain = (full ? info.a + info.p_hi * (ln_s - info.lse)
                              : info.a * info.p_inv + ln_s - info.tm * a.inv_hi - logf(info.p_hi)) + rest;
    if (!(fabsf(plain) < INFINITY)) return scale * plain;
    Pair ln_sum;  // log of the student's sum of exponentials
    ln_sum.add_ln2(r.M2);
    ln_sum.add_log(r.S, 1.0f);
    Pair L;
    if (full) {
        Pair d = ln_sum;
        d.add(-info.lse);
        L.add(info.a);
        L.add_product(info.p_hi, d.hi);
        L.lo += info.p_hi * d.lo + info.p_lo * d.hi;
        if (r.p_r != 0.0f) {
            Pair g = ln_sum;
            g.add_ln2(-r.m2o);
            g.add_log(r.s_o, -1.0f);
            g.add_log(r.p_r, 1.0f);
            L.add_product(r.p_r, g.hi);
            L.lo += r.p_r * g.lo;
        }
    } else {
        L.add(info.a * info.p_inv);
        L.add(ln_sum);
        L.add_product(-info.tm, a.inv_hi);
        L.lo -= info.tm * a.inv_lo;
        L.add_log(info.p_hi + info.p_lo, -1.0f);
    }
    return scale * L.value();
}
__device__ __forceinline__ void store_stats(const DistillArgs& a, int64_t row, const ListInfo& info,
                                            const RowSums& r) {
    float4* const st = reinterpret_cast<float4*>(a.stats + row * DISTILL_STATS);
    st[0] = make_float4(r.M2, r.inv_S, r.ref_o, r.B);
    st[1] = make_float4(info.tm, info.p_inv, 1.0f, 0.0f);
}
__device__ __forceinline__ void store_dead(const DistillArgs& a, int64_t row, bool stats) {
    a.loss[row] = 0.0f;
    if (stats) {
        float4* const st = reinterpret_cast<float4*>(a.stats + row * DISTILL_STATS);
        st[0] = st[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
}

template <class T>
__device__ __forceinline__ void slice_grads(const uint4& v, uint64_t kk, uint64_t ref, uint64_t mul,
                                            float (&x)[Elem<T>::kPer]) {
    Elem<T>::unpack(v, x);
#pragma unroll
    for (int i = 0; i < Elem<T>::kPer; i += 2) {
        float u0, u1;
        unpack2(fma2(pack2(__float_as_uint(x[i]), __float_as_uint(x[i + 1])), kk, ref), u0, u1);
        const uint64_t p = fma2(pack2(__float_as_uint(ex2(u0)), __float_as_uint(ex2(u1))), mul, 0ull);
        unpack2(p, x[i], x[i + 1]);
    }
}

// Gradient of granules [g0, g1) outside the list, from the slice at `buf`
// (granule g0 first), by thread t of n_threads.
template <class T>
__device__ __forceinline__ void write_slice(const DistillArgs& a, const RowView<T>& v, const uint4* buf, T* out,
                                            bool same, int g0, int g1, int t, int n_threads, float ref_o, float mul) {
    constexpr int kPer = Elem<T>::kPer;
    const uint64_t kk = both(a.k2), ref = both(-ref_o), mm = both(mul);
    float x[kPer];
    if (!same) {  // the output rows start at another place of a granule: element by element
        for (int g = g0 + t; g < g1; g += n_threads) {
            slice_grads<T>(buf[g - g0], kk, ref, mm, x);
            store_granule<T>(out, g, v.off, a.vocab, false, x);
        }
        return;
    }
    const int ga = g0 < g1 && !v.whole(g0, a.vocab) ? g0 + 1 : g0;
    const int gb = g1 > ga && !v.whole(g1 - 1, a.vocab) ? g1 - 1 : g1;
    uint4* const o = reinterpret_cast<uint4*>(out - v.off) + g0;
    int g = ga - g0 + t;
    const int n = gb - g0;
    for (; g + 3 * n_threads < n; g += 4 * n_threads) {
        uint4 b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = buf[g + i * n_threads];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            slice_grads<T>(b[i], kk, ref, mm, x);
            o[g + i * n_threads] = Elem<T>::pack(x);
        }
    }
    for (; g < n; g += n_threads) {
        slice_grads<T>(buf[g], kk, ref, mm, x);
        o[g] = Elem<T>::pack(x);
    }
    for (int e : {ga > g0 ? g0 : -1, gb < g1 ? gb : -1}) {  // granules shared with a neighbouring row
        if (e < 0 || t >= kPer) continue;
        slice_grads<T>(buf[e - g0], kk, ref, mm, x);
        const int j = e * kPer + t - v.off;
        float mine = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine = t == i ? x[i] : mine;
        if (j >= 0 && j < a.vocab) out[j] = Elem<T>::from_f(mine);
    }
}

__host__ __device__ constexpr size_t align16(size_t n) { return (n + 15) & ~size_t(15); }
// Dynamic shared memory of distill_row_kernel: the chunk, then three arrays of
// `top` words.
size_t row_smem(int chunk, int top) { return size_t(chunk) * 16 + align16(size_t(top) * 4) * 3; }

// The first entries of a row's list and the row's scalars, asked for ahead: as
// they lie in memory, because converting one would wait for it.
constexpr int kAhead = 4;  // entries a lane
struct ListAhead {
    uint32_t j_lo[kAhead], j_hi[kAhead];
    uint32_t t[kAhead];
    float w, lse;
};
__device__ __forceinline__ void ask_entry(const DistillArgs& a, int64_t i, bool in, uint32_t& j_lo, uint32_t& j_hi,
                                          uint32_t& t) {
    j_lo = j_hi = 0xffffffffu;  // -1: an empty slot
    t = 0;
    if (!in) return;
    if (a.index_bytes == 8) {
        j_lo = static_cast<const uint32_t*>(a.top_index)[2 * i];
        j_hi = static_cast<const uint32_t*>(a.top_index)[2 * i + 1];
    } else {
        j_lo = static_cast<const uint32_t*>(a.top_index)[i];
    }
    if (a.top_dtype == HESS_F32)
        t = static_cast<const uint32_t*>(a.top_logits)[i];
    else
        t = static_cast<const uint16_t*>(a.top_logits)[i];
}
__device__ __forceinline__ int64_t entry_index(const DistillArgs& a, uint32_t lo, uint32_t hi) {
    return a.index_bytes == 8 ? static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo)
                              : static_cast<int64_t>(static_cast<int32_t>(lo));
}
__device__ __forceinline__ float entry_logit(const DistillArgs& a, uint32_t t) {
    if (a.top_dtype == HESS_F32) return __uint_as_float(t);
    if (a.top_dtype == HESS_BF16) return __uint_as_float(t << 16);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(t)));
}
__device__ __forceinline__ void ask_list(const DistillArgs& a, int64_t row, ListAhead& l) {
    const int lane = threadIdx.x & 31;
    l.w = a.weights ? a.weights[row] : 1.0f;
    l.lse = a.lse ? a.lse[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int k = lane + 32 * i;
        ask_entry(a, row * a.top + k, k < a.top, l.j_lo[i], l.j_hi[i], l.t[i]);
    }
}

// The teacher's list of a row, by one warp: columns, exponentials and the
// student's logits there (they are read here, before any gradient is stored).
template <class T>
__device__ __forceinline__ void read_list(const DistillArgs& a, int64_t row, const T* logits, const ListAhead& ahead,
                                          int* s_idx, float* s_p, float* s_s, ListInfo& info) {
    const int K = a.top, lane = threadIdx.x & 31;
    bool any = false, bad = false;
    float tm = kNegInf, mt = kNegInf;
    ListAhead l = ahead;
    for (int k0 = lane;;) {
        int j[kAhead];
        float t[kAhead], s[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t at = entry_index(a, l.j_lo[i], l.j_hi[i]);
            t[i] = entry_logit(a, l.t[i]);
            const bool held = at >= 0 && t[i] != kNegInf;
            bad |= held && at >= a.vocab;
            j[i] = held && at < a.vocab ? static_cast<int>(at) : -1;
            s[i] = j[i] >= 0 ? Elem<T>::to_f(logits[j[i]]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = k0 + 32 * i;
            if (k >= K) break;
            s_idx[k] = j[i];
            s_p[k] = t[i];
            s_s[k] = s[i];
            if (j[i] >= 0) {
                any = true;
                tm = fmaxf(tm, t[i]);
                mt = fmaxf(mt, s[i]);
            }
        }
        k0 += 32 * kAhead;
        if (k0 - lane >= K) break;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            ask_entry(a, row * K + k0 + 32 * i, k0 + 32 * i < K, l.j_lo[i], l.j_hi[i], l.t[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
    }
    const bool full = a.lse != nullptr;
    const float base = full ? ahead.lse : tm;
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
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float h = __shfl_xor_sync(0xffffffffu, hi, o), q = __shfl_xor_sync(0xffffffffu, lo, o);
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        float e;
        hi = two_sum_f32(hi, h, e);
        lo += q + e;
    }
    const float p_inv = full ? 1.0f : 1.0f / (hi + lo);
    if (!full)
        for (int k = lane; k < K; k += 32) s_p[k] *= p_inv;
    any = __any_sync(0xffffffffu, any);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) info = ListInfo{any || bad, bad, ahead.w, tm, mt, hi, lo, p_inv, sum, base};
    __syncwarp();
}

// Takes the listed columns [j0, j1) out of a chunk, by one warp, and sums the
// student's exponentials there.  Each slot first writes its number into the
// chunk: one that reads another's back shares its column.  Afterwards the
// first slot of a column holds the p of all its slots, the others -1.
template <class T>
__device__ __forceinline__ void take_out(const DistillArgs& a, T* e, int j0, int j1, int j_base, const int* s_idx,
                                         float* s_p, const float* s_s, float m2_top, float& sum_top, float& listed) {
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
    if (__any_sync(0xffffffffu, twice)) {
        // rare: for every slot that lost its column to another, the column's
        // first slot gets the sum (lanes over the slots) and the others -1
        for (int k0 = 0; k0 < K; k0 += 32) {
            const int mine = k0 + lane < K ? s_idx[k0 + lane] : -1;
            bool lost = false;
            if (mine >= j0 && mine < j1) {
                uint16_t tag;
                memcpy(&tag, &e[mine - j_base], 2);
                lost = tag != k0 + lane;
            }
            for (uint32_t todo = __ballot_sync(0xffffffffu, lost); todo; todo &= todo - 1) {
                const int j = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
                float p = 0.0f;
                int first = K;
                for (int l = lane; l < K; l += 32)
                    if (s_idx[l] == j) {
                        if (!(s_p[l] < 0.0f)) p += s_p[l];
                        first = min(first, l);
                    }
                p = warp_reduce(p, AddOp());
                first = __reduce_min_sync(0xffffffffu, first);
                for (int l = lane; l < K; l += 32)
                    if (s_idx[l] == j) s_p[l] = l == first ? p : -1.0f;
                __syncwarp();
            }
        }
    }
    for (int k = lane; k < K; k += 32) {
        const int j = s_idx[k];
        if (j < j0 || j >= j1) continue;
        e[j - j_base] = Elem<T>::from_f(kNegInf);
        if (!(s_p[k] < 0.0f)) {
            sum_top += m2_top == kNegInf ? 0.0f : ex2(fmaf(s_s[k], a.k2, -m2_top));
            listed += 1.0f;
        }
    }
}

// Gradients of the listed columns [j0, j1), by thread t of n_threads.
template <class T>
__device__ __forceinline__ void write_listed(const DistillArgs& a, T* out, int j0, int j1, const int* s_idx,
                                             const float* s_p, const float* s_s, int t, int n_threads, float gs,
                                             const RowSums& r) {
    for (int k = t; k < a.top; k += n_threads) {
        const int j = s_idx[k];
        if (j >= j0 && j < j1 && !(s_p[k] < 0.0f))
            out[j] = Elem<T>::from_f(gs * (ex2(fmaf(s_s[k], a.k2, -r.M2)) * r.inv_S - s_p[k]));
    }
}

// One row per cluster, each CTA's slice in pieces of a.chunk granules: for rows
// too long for distill_stream_kernel.
template <class T, bool kGrad>
__global__ void __launch_bounds__(kThreads) distill_row_kernel(const DistillArgs a) {
    constexpr int kPer = Elem<T>::kPer;
    extern __shared__ uint4 buf[];
    __shared__ ListInfo info;
    __shared__ float2 part[kMaxCluster * kWarps];  // (maximum, sum) of every warp of the cluster
    __shared__ float2 top[kMaxCluster];            // (sum over the listed columns, their number) of every slice
    const size_t kstep = align16(size_t(a.top) * 4) / 4;
    int* const s_idx = reinterpret_cast<int*>(buf + a.chunk);    // column, -1 for an empty slot
    float* const s_p = reinterpret_cast<float*>(s_idx) + kstep;  // p
    float* const s_s = s_p + kstep;                              // student logit

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
        if (warp == 0) {
            ListAhead ahead;
            ask_list(a, row, ahead);
            read_list<T>(a, row, v.row, ahead, s_idx, s_p, s_s, info);
        }
        cp_async_wait();
        __syncthreads();
        live = info.live != 0;
    }
    if (!live) {
        if (kGrad) zero_slice<T>(v, out, a.vocab, same, g_lo, g_hi, tid, kThreads);
        if (rank == 0 && tid == 0) store_dead(a, row, !kGrad);
        return;  // the whole cluster leaves here, as all of it read the same row
    }
    const float m2_top = info.m_top * a.k2;  // reference of the listed columns (all slices use this one)
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
                        m2_top, sum_top, listed);
        }
        __syncthreads();
        float mc, sc;
        slice_sums<T>(buf, n, tid, kThreads, a.k2, m2_top, mc, sc);
        const float m = fmaxf(m2, mc);
        sum = sum * rescale(m2, m) + sc * rescale(mc, m);
        m2 = m;
    }

    // every warp's pair goes to every CTA of the cluster
    if (warp == 0) {
        sum_top = warp_reduce(sum_top, AddOp());
        listed = warp_reduce(listed, AddOp());
    }
    if (lane < static_cast<int>(C)) {
        st_cluster_f32x2(mapa_shared(smem_u32(&part[rank * kWarps + warp]), lane), m2, sum);
        if (warp == 0) st_cluster_f32x2(mapa_shared(smem_u32(&top[rank]), lane), sum_top, listed);
    }
    cluster_sync_all();
    const RowSums r = row_sums(a, info, part, static_cast<int>(C) * kWarps, top, static_cast<int>(C));
    if (rank == 0 && tid == kThreads - 32) {
        a.loss[row] = row_loss(a, info, r);
        if (!kGrad) store_stats(a, row, info, r);
    }
    if constexpr (kGrad) {
        const float gs = w * a.tau;
        for (int c = n_chunks - 1; c >= 0; --c) {
            const int g0 = g_lo + c * a.chunk, g1 = min(g_hi, g0 + a.chunk);
            if (c != n_chunks - 1) {
                __syncthreads();
                load_chunk<T>(v, a.vocab, g0, g1, buf);
                cp_async_wait();
                __syncthreads();
            }
            write_slice<T>(a, v, buf, out, same, g0, g1, tid, kThreads, r.ref_o, gs * r.B);
        }
        __syncthreads();
        write_listed<T>(a, out, max(0, g_lo * kPer - v.off), min(a.vocab, g_hi * kPer - v.off), s_idx, s_p, s_s, tid,
                        kThreads, gs, r);
    }
}

// ---------------------------------------------------- a stream of rows

constexpr int kListWarps = 8;
constexpr int kStreamWarps = 16;  // compute warps
constexpr int kFirstCompute = kListWarps + 1;
constexpr int kStreamThreads = (kFirstCompute + kStreamWarps) * 32;
constexpr int kComputeThreads = kStreamWarps * 32;
constexpr int kMaxBuffers = 8;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

// Shared-memory layout of distill_stream_kernel (byte offsets): n_buf slices,
// n_list rows' lists, 2 n_list slots of the exchange.
struct StreamLayout {
    size_t lists, parts, tops, info, bars, bytes;
    __host__ __device__ StreamLayout(int n_buf, int n_list, int slice, int top, int C) {
        const int slots = 2 * n_list;
        lists = static_cast<size_t>(n_buf) * slice * 16;
        parts = lists + static_cast<size_t>(n_list) * 3 * align16(static_cast<size_t>(top) * 4);
        tops = parts + static_cast<size_t>(slots) * C * kStreamWarps * 8;
        info = tops + static_cast<size_t>(slots) * C * 8;
        bars = align16(info + static_cast<size_t>(n_list) * sizeof(ListInfo));
        bytes = bars + static_cast<size_t>(n_buf + 3 * n_list + slots) * 8;
    }
};

// Rows cluster, cluster + n_clusters, ...; row number i of them uses buffer
// i mod n_buf, list i mod n_list and exchange slot i mod 2 n_list.
//   producer warp: asks for row i's slice as soon as its buffer is free;
//   list warp i mod n_list: reads row i's list (well before its slice is there),
//     takes the listed columns out of the landed slice and hands it over
//     ("ready"); later computes the loss (CTA 0 of the cluster);
//   compute warps: sums of row i + 1 (sent to every CTA of the cluster, which
//     counts them on the row's exchange barrier), then row i's gradient.
// A wait goes by the parity of a barrier's phase, so every barrier has waiters
// that see each of its phases: one that a list warp waits on belongs to the
// list, not to the buffer, which other rows pass through in between.
// An exchange slot is free again in time: a CTA sends row j only after its list
// warp has seen row j - n_list exchanged, which needs every CTA's list warp on
// that row, and so done with row j - 2 n_list, and every CTA's compute warps
// past the gradient of row j - n_list - 2.
// Every wait is bounded.  After one that runs out the CTA waits no more but
// goes through the motions, sending NaN, so that nobody waits for it for long:
// the rows concerned get a NaN loss.
template <class T, bool kGrad>
__global__ void __launch_bounds__(kStreamThreads, 1) distill_stream_kernel(const DistillArgs a) {
    constexpr int kPer = Elem<T>::kPer;
    extern __shared__ uint4 buf0[];
    __shared__ volatile int failed;
    uint32_t C;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
    const uint32_t rank = cluster_ctarank();
    const int n_buf = a.n_buf, n_list = a.n_list, slots = 2 * n_list;
    uint8_t* const base = reinterpret_cast<uint8_t*>(buf0);
    const StreamLayout lay(n_buf, n_list, a.slice, a.top, static_cast<int>(C));
    const size_t kstep = align16(size_t(a.top) * 4) / 4;
    float2* const parts = reinterpret_cast<float2*>(base + lay.parts);
    float2* const tops = reinterpret_cast<float2*>(base + lay.tops);
    ListInfo* const infos = reinterpret_cast<ListInfo*>(base + lay.info);
    const uint32_t bars = smem_u32(base + lay.bars);
    auto empty_bar = [&](int b) { return bars + 8u * b; };
    auto full_bar = [&](int l) { return bars + 8u * (n_buf + l); };
    auto ready_bar = [&](int l) { return bars + 8u * (n_buf + n_list + l); };
    auto done_bar = [&](int l) { return bars + 8u * (n_buf + 2 * n_list + l); };
    auto x_bar = [&](int s) { return bars + 8u * (n_buf + 3 * n_list + s); };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int b = 0; b < n_buf; ++b) mbar_init(empty_bar(b), kStreamWarps);
        for (int l = 0; l < n_list; ++l) {
            mbar_init(full_bar(l), 1);
            mbar_init(ready_bar(l), 1);
            mbar_init(done_bar(l), kStreamWarps);
        }
        for (int s = 0; s < slots; ++s) mbar_init(x_bar(s), 1);
        failed = 0;
        fence_barrier_init();
    }
    cluster_sync_all();

    const int64_t cluster = blockIdx.x / C, n_clusters = gridDim.x / C;
    const int n_it = static_cast<int>((a.rows - cluster + n_clusters - 1) / n_clusters);
    // this CTA's slice of a row, and the granules of it that hold no other row's elements
    auto slice_of = [&](const RowView<T>& v, int& g_lo, int& g_hi) {
        g_lo = min(v.n, static_cast<int>(rank) * a.slice);
        g_hi = min(v.n, g_lo + a.slice);
    };
    auto inner = [&](const RowView<T>& v, int g_lo, int g_hi, int& ga, int& gb) {
        ga = g_lo < g_hi && !v.whole(g_lo, a.vocab) ? g_lo + 1 : g_lo;
        gb = g_hi > ga && !v.whole(g_hi - 1, a.vocab) ? g_hi - 1 : g_hi;
    };

    if (warp == kListWarps) {
        if (lane == 0) {
            int b = 0, l = 0;
            uint32_t phase = 1;
            float w = a.weights ? a.weights[cluster] : 1.0f;
            for (int it = 0; it < n_it; ++it) {
                const int64_t row = cluster + it * n_clusters;
                if (failed != 0 || !mbar_wait(empty_bar(b), phase, kWaitLimitNs)) {
                    failed = 1;
                    break;
                }
                if (w != 0.0f) {
                    const RowView<T> v(a.logits, a.ld, row, a.vocab);
                    int g_lo, g_hi, ga, gb;
                    slice_of(v, g_lo, g_hi);
                    inner(v, g_lo, g_hi, ga, gb);
                    const uint32_t bytes = gb > ga ? static_cast<uint32_t>(gb - ga) * 16u : 0u;
                    // what the warps wrote into the buffer comes before the copy
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive_expect_tx(full_bar(l), bytes);
                    if (bytes)
                        asm volatile(
                            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                            ::"r"(smem_u32(buf0 + static_cast<size_t>(b) * a.slice + (ga - g_lo))),
                            "l"(v.granule(ga)), "r"(bytes), "r"(full_bar(l))
                            : "memory");
                } else {
                    mbar_arrive(full_bar(l));
                }
                if (it + 1 < n_it && a.weights) w = a.weights[row + n_clusters];
                if (++b == n_buf) {
                    b = 0;
                    phase ^= 1u;
                }
                if (++l == n_list) l = 0;
            }
        }
    } else if (warp < n_list) {
        const int l = warp;
        int* const s_idx = reinterpret_cast<int*>(base + lay.lists) + static_cast<size_t>(l) * 3 * kstep;
        float* const s_p = reinterpret_cast<float*>(s_idx) + kstep;
        float* const s_s = s_p + kstep;
        ListInfo& info = infos[l];
        uint32_t done_phase = 0, full_phase = 0;
        ListAhead ahead;
        if (l < n_it) ask_list(a, cluster + l * n_clusters, ahead);
        for (int it = l; it < n_it; it += n_list) {
            const int64_t row = cluster + it * n_clusters;
            const int slot = it % slots, b = it % n_buf;
            bool ok = failed == 0;
            // every warp of the cluster will send 8 bytes, every list warp 8 more
            if (lane == 0) mbar_arrive_expect_tx(x_bar(slot), C * (kStreamWarps + 1) * 8u);
            float sum_top = 0.0f, listed = 0.0f;
            if (ok && ahead.w != 0.0f) {
                const RowView<T> v(a.logits, a.ld, row, a.vocab);
                int g_lo, g_hi, ga, gb;
                slice_of(v, g_lo, g_hi);
                inner(v, g_lo, g_hi, ga, gb);
                read_list<T>(a, row, v.row, ahead, s_idx, s_p, s_s, info);
                // the next row's list is on its way while this row is waited for
                if (it + n_list < n_it) ask_list(a, row + n_list * n_clusters, ahead);
                ok = mbar_wait(full_bar(l), full_phase, kWaitLimitNs);
                if (ok && info.live) {
                    uint4* const buf = buf0 + static_cast<size_t>(b) * a.slice;
                    for (int g : {ga > g_lo ? g_lo : -1, gb < g_hi ? gb : -1}) {
                        if (g < 0 || lane >= kPer) continue;
                        const int j = g * kPer + lane - v.off;
                        reinterpret_cast<T*>(buf + (g - g_lo))[lane] =
                            j >= 0 && j < a.vocab ? v.row[j] : Elem<T>::from_f(kNegInf);
                    }
                    __syncwarp();
                    const int j_base = g_lo * kPer - v.off;
                    take_out<T>(a, reinterpret_cast<T*>(buf), max(j_base, 0), j_base + (g_hi - g_lo) * kPer, j_base,
                                s_idx, s_p, s_s, info.m_top * a.k2, sum_top, listed);
                }
            } else {
                if (it + n_list < n_it) ask_list(a, row + n_list * n_clusters, ahead);
                ok = ok && mbar_wait(full_bar(l), full_phase, kWaitLimitNs);
                if (lane == 0) info.live = 0;
            }
            full_phase ^= 1u;
            if (!ok) {
                failed = 1;
                sum_top = NAN;  // the row becomes NaN in every CTA
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(ready_bar(l));
            sum_top = warp_reduce(sum_top, AddOp());
            listed = warp_reduce(listed, AddOp());
            if (lane < static_cast<int>(C))
                send_f32x2(mapa_shared(smem_u32(&tops[slot * C + rank]), lane), sum_top, listed,
                           mapa_shared(x_bar(slot), lane));
            ok = ok && mbar_wait_cluster(x_bar(slot), static_cast<uint32_t>(it / slots) & 1u, kWaitLimitNs);
            if (!ok) failed = 1;
            const bool live = ok && info.live;
            RowSums r{};
            if (live && (kGrad || rank == 0))
                r = row_sums(a, info, parts + slot * C * kStreamWarps, static_cast<int>(C) * kStreamWarps,
                             tops + slot * C, static_cast<int>(C));
            if (rank == 0) {
                if (!ok) {
                    if (lane == 0) a.loss[row] = NAN;
                } else if (!live) {
                    if (lane == 0) store_dead(a, row, !kGrad);
                } else {
                    const float loss = row_loss(a, info, r);
                    if (lane == 0) {
                        a.loss[row] = loss;
                        if (!kGrad) store_stats(a, row, info, r);
                    }
                }
            }
            // the compute warps are done with the row: the listed columns' values
            // go over the zeros they stored there, and the list is free
            if (!mbar_wait(done_bar(l), done_phase, failed != 0 ? 0ull : kWaitLimitNs)) failed = 1;
            done_phase ^= 1u;
            if constexpr (kGrad) {
                if (live && failed == 0) {
                    const RowView<T> v(a.logits, a.ld, row, a.vocab);
                    int g_lo, g_hi;
                    slice_of(v, g_lo, g_hi);
                    write_listed<T>(a, static_cast<T*>(a.dlogits) + row * a.ldd, max(0, g_lo * kPer - v.off),
                                    min(a.vocab, g_hi * kPer - v.off), s_idx, s_p, s_s, lane, 32, info.w * a.tau, r);
                }
            }
            __syncwarp();
        }
    } else if (warp >= kFirstCompute) {
        const int t = tid - kFirstCompute * 32, cw = warp - kFirstCompute;
        // it runs one ahead of the row whose gradient is written
        int b = 0, l = 0, slot = 0, pb = 0, pl = 0, pslot = 0;
        uint32_t ready_phase = 0, x_phase = 0;
        for (int it = 0; it < n_it + (kGrad ? 1 : 0); ++it) {
            if (it < n_it) {
                const int64_t row = cluster + it * n_clusters;
                const bool ok = failed == 0 && mbar_wait(ready_bar(l), ready_phase, kWaitLimitNs);
                float m2 = kNegInf, sum = 0.0f;
                if (ok && infos[l].live) {
                    const RowView<T> v(a.logits, a.ld, row, a.vocab);
                    const int g_lo = min(v.n, static_cast<int>(rank) * a.slice), g_hi = min(v.n, g_lo + a.slice);
                    slice_sums<T>(buf0 + static_cast<size_t>(b) * a.slice, g_hi - g_lo, t, kComputeThreads, a.k2,
                                  infos[l].m_top * a.k2, m2, sum);
                }
                if (!ok) {
                    failed = 1;
                    sum = NAN;
                }
                if (lane < static_cast<int>(C))
                    send_f32x2(mapa_shared(smem_u32(&parts[(slot * C + rank) * kStreamWarps + cw]), lane), m2, sum,
                               mapa_shared(x_bar(slot), lane));
                if (!kGrad) {
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(empty_bar(b));
                        mbar_arrive(done_bar(l));
                    }
                }
                if (++b == n_buf) b = 0;
                if (++l == n_list) {
                    l = 0;
                    ready_phase ^= 1u;
                }
                if (++slot == slots) slot = 0;
            }
            if constexpr (kGrad) {
                if (it > 0) {
                    const int64_t row = cluster + (it - 1) * n_clusters;
                    const ListInfo& info = infos[pl];
                    const RowView<T> v(a.logits, a.ld, row, a.vocab);
                    const int g_lo = min(v.n, static_cast<int>(rank) * a.slice), g_hi = min(v.n, g_lo + a.slice);
                    T* const out = static_cast<T*>(a.dlogits) + row * a.ldd;
                    const bool same =
                        ((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T)) == static_cast<unsigned>(v.off);
                    const bool ok = failed == 0 && mbar_wait_cluster(x_bar(pslot), x_phase, kWaitLimitNs);
                    if (!ok) failed = 1;
                    if (ok && info.live != 0) {
                        const RowSums r = row_sums(a, info, parts + pslot * C * kStreamWarps,
                                                   static_cast<int>(C) * kStreamWarps, tops + pslot * C,
                                                   static_cast<int>(C));
                        write_slice<T>(a, v, buf0 + static_cast<size_t>(pb) * a.slice, out, same, g_lo, g_hi, t,
                                       kComputeThreads, r.ref_o, info.w * a.tau * r.B);
                    } else if (ok) {
                        zero_slice<T>(v, out, a.vocab, same, g_lo, g_hi, t, kComputeThreads);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(empty_bar(pb));
                        mbar_arrive(done_bar(pl));
                    }
                    if (++pb == n_buf) pb = 0;
                    if (++pl == n_list) pl = 0;
                    if (++pslot == slots) {
                        pslot = 0;
                        x_phase ^= 1u;
                    }
                }
            }
        }
    }
    // no CTA leaves while another may still send to it
    cluster_sync_all();
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
        zero_slice<T>(v, out, a.vocab, same, g_lo, g_hi, tid, kThreads);
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

constexpr size_t kMaxDynamic = 226 * 1024;
constexpr size_t kMaxDynamicRow = 220 * 1024;

template <class T, bool kGrad>
struct Kernels {
    static constexpr auto stream = distill_stream_kernel<T, kGrad>;
    static constexpr auto row = distill_row_kernel<T, kGrad>;
};

cudaLaunchConfig_t cluster_config(unsigned grid, int threads, size_t smem, int C, cudaStream_t s,
                                  cudaLaunchAttribute* attr) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = static_cast<unsigned>(C);
    attr->val.clusterDim.y = 1;
    attr->val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

// Per-device set-up: shared-memory limits, and how many clusters of each size
// can be resident with one CTA per SM.
struct DeviceInfo {
    bool ready = false;
    int clusters[kMaxCluster + 1] = {};
};
hess_status ds_prepare(int dev, const DeviceInfo** out) {
    static std::mutex mu;
    static DeviceInfo infos[128];
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 128) return ds_fail(HESS_ERR_UNSUPPORTED, "device index %d", dev);
    DeviceInfo& d = infos[dev];
    if (!d.ready) {
        for (auto fn : {Kernels<__nv_bfloat16, false>::row, Kernels<__nv_bfloat16, true>::row,
                        Kernels<__half, false>::row, Kernels<__half, true>::row, Kernels<float, false>::row,
                        Kernels<float, true>::row})
            DS_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kMaxDynamicRow)));
        for (auto fn : {Kernels<__nv_bfloat16, false>::stream, Kernels<__nv_bfloat16, true>::stream,
                        Kernels<__half, false>::stream, Kernels<__half, true>::stream,
                        Kernels<float, false>::stream, Kernels<float, true>::stream})
            DS_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kMaxDynamic)));
        int sms = 0;
        DS_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
        for (int C = 1; C <= kMaxCluster; C *= 2) {
            cudaLaunchAttribute attr;
            cudaLaunchConfig_t cfg = cluster_config(static_cast<unsigned>(sms / C * C), kStreamThreads, kMaxDynamic,
                                                    C, nullptr, &attr);
            int n = 0;
            DS_TRY(cudaOccupancyMaxActiveClusters(&n, Kernels<__nv_bfloat16, true>::stream, &cfg));
            d.clusters[C] = n;
        }
        d.ready = true;
    }
    *out = &d;
    return HESS_OK;
}

template <class T, bool kGrad>
hess_status launch_typed(DistillArgs& a, const DeviceInfo& d, cudaStream_t s) {
    constexpr int per = Elem<T>::kPer;
    const int granules = static_cast<int>((static_cast<int64_t>(a.vocab) + 2 * (per - 1)) / per);
    cudaLaunchAttribute attr;
    // long lists take their room from the slices: fewer of them at a time
    const int n_list = a.top <= 128 ? kListWarps : kListWarps / 2;
    // CTAs per row: the fewest with which two slices fit an SM; more when there
    // are not enough rows for the SMs, down to slices of 2 KB.
    for (int C = 1; C <= kMaxCluster; C *= 2) {
        if (d.clusters[C] < 1) break;
        const int slice = (granules + C - 1) / C;
        if (StreamLayout(2, n_list, slice, a.top, C).bytes > kMaxDynamic) continue;
        if (2 * C <= kMaxCluster && a.rows <= d.clusters[2 * C] && slice >= 256) continue;
        const int64_t clusters = a.rows < d.clusters[C] ? a.rows : d.clusters[C];
        const int64_t per_cluster = (a.rows + clusters - 1) / clusters;
        int n_buf = 2;
        while (n_buf < kMaxBuffers && n_buf < per_cluster &&
               StreamLayout(n_buf + 1, n_list, slice, a.top, C).bytes <= kMaxDynamic)
            ++n_buf;
        a.slice = slice;
        a.n_buf = n_buf;
        a.n_list = n_list;
        const cudaLaunchConfig_t cfg =
            cluster_config(static_cast<unsigned>(clusters * C), kStreamThreads,
                           StreamLayout(n_buf, n_list, slice, a.top, C).bytes, C, s, &attr);
        DS_TRY(cudaLaunchKernelEx(&cfg, Kernels<T, kGrad>::stream, a));
        return HESS_OK;
    }
    const int C = kMaxCluster;
    a.slice = (granules + C - 1) / C;
    a.chunk = a.slice < 12288 ? a.slice : 12288;
    const cudaLaunchConfig_t cfg = cluster_config(static_cast<unsigned>(a.rows * C), kThreads,
                                                  row_smem(a.chunk, a.top), C, s, &attr);
    DS_TRY(cudaLaunchKernelEx(&cfg, Kernels<T, kGrad>::row, a));
    return HESS_OK;
}

template <bool kGrad>
hess_status launch_rows(DistillArgs& a, int32_t dtype, cudaStream_t s) {
    int dev = 0;
    hess_status st = ds_buffers(a, &dev);
    if (st != HESS_OK) return st;
    const DeviceInfo* d = nullptr;
    st = ds_prepare(dev, &d);
    if (st != HESS_OK) return st;
    if (dtype == HESS_BF16) return launch_typed<__nv_bfloat16, kGrad>(a, *d, s);
    if (dtype == HESS_F16) return launch_typed<__half, kGrad>(a, *d, s);
    return launch_typed<float, kGrad>(a, *d, s);
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
