// Distillation loss from a teacher's top logits, its gradient, and both in one
// pass (formulas and conventions: include/distill.h).
//
// The work is a stream over the student's logits: read them once, write the
// gradient once, a few operations per element.  The loss needs a row's sum of
// exponentials before the first gradient can be written, so the logits are
// needed twice: a CTA (or a cluster of CTAs) takes one row, sums it straight from
// memory, and reads it again, from L2, for the gradient.  The L2 holds what is in
// flight (launch_typed) as long as the gradient's stores leave it first, which
// they are marked to do.
//
// Memory bounds it.  8,192 rows of 128,000 bf16 logits, an eighth of them without
// weight: the loss alone takes 266 us, the rate of a copy of the bytes it reads;
// loss and gradient 688 us, 83 % of that rate (ncu: 5.2 TB/s, a tenth of the
// logits read twice); the gradient from saved statistics 604 us, 95 %.  What the
// step lacks is the start of a row, two loads of DRAM one after the other, and the
// meeting of its warps, which only other CTAs hide.  Keeping the rows in shared
// memory instead (a cluster per row, bulk copies, a warp for each list) was built
// too: its phases wait for one another inside each SM, and the step took 821 us.
//
// Exponentials are 2^(s k2 - M2) with k2 = log2(e) / tau and M2 = max(s) k2,
// one FMA and one ex2 per element.  The listed columns are left out of the
// sums (a bit for each column, looked at once per 16 bytes), so that the mass
// outside the list is summed directly instead of as a difference, and has a
// reference of its own.  With S_o, M2o of the other columns and S, M2 of the whole row:
//     q_j = 2^(s_j k2 - M2) / S
//     d loss / d s_j = w tau 2^(s_j k2 - M2o) (2^(M2o - M2) / S - p_r / S_o)
// for columns outside the list, w tau (q_j - p_j) for those in it.  Where the list
// holds at most half of either mass, P of the teacher's and Q of the student's, both
// are nearly one outside it, and their roundings would outweigh what differs; there
// the same is taken from the masses inside:
//     log(p_r / q_r) = log1p(-P) - log1p(-Q),    1 / S - p_r / S_o = (P - Q) / S_o
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

constexpr int kMaxThreads = 512;
constexpr int kMaxWarps = kMaxThreads / 32;
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
    int32_t slice;     // 16-byte granules of a row per CTA, a multiple of kSegment
    int32_t segments;  // of a row, at most
    int32_t ahead;     // rows in work at a time, about
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

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float x) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(x) : "memory");
}
__device__ __forceinline__ void st_cluster_f32x2(uint32_t addr, float x, float y) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
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

// What a row's list comes to.
struct ListInfo {
    int bad;
    float w;             // the row's weight
    float tm, m_top;     // largest listed logit, teacher's and student's
    float p_hi, p_lo;    // sum of the list's exponentials
    float p_inv;
    float a;             // sum of p (t - s) / tau
    float lse;           // the teacher's, when given
};

// A slice of a row: granules [lo, hi), of which [a, b) hold no other row's
// elements, and the bits of its listed columns (bit 0: element 0 of granule lo).
template <class T>
struct Slice {
    int lo, hi, a, b;
    const uint8_t* listed;
    __device__ Slice(const RowView<T>& v, int vocab, int rank, int per_cta, const uint8_t* bits) : listed(bits) {
        lo = min(v.n, rank * per_cta);
        hi = min(v.n, lo + per_cta);
        a = lo < hi && !v.whole(lo, vocab) ? lo + 1 : lo;
        b = hi > a && !v.whole(hi - 1, vocab) ? hi - 1 : hi;
    }
    // bits of granule g, the first element lowest
    __device__ uint32_t bits(int g) const {
        const uint32_t i = static_cast<uint32_t>(g - lo);
        if (Elem<T>::kPer == 8) return listed[i];
        return (listed[i >> 1] >> ((i & 1u) * 4u)) & 15u;
    }
};

// Loads of 16 bytes that stay in L2 for the second pass, or leave it first.
template <bool kKeep>
__device__ __forceinline__ uint4 load_granule(const void* p) {
    if constexpr (kKeep)
        return __ldcg(static_cast<const uint4*>(p));
    else
        return __ldcs(static_cast<const uint4*>(p));
}

template <class T, bool kFull>
__device__ __forceinline__ void add_exps(const uint4& v, uint32_t bits, uint64_t kk, uint64_t ref, uint64_t& s0,
                                         uint64_t& s1) {
    constexpr int kPer = Elem<T>::kPer;
    float x[kPer];
    Elem<T>::unpack(v, x);
    if (kFull && bits) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = bits >> i & 1u ? kNegInf : x[i];
    }
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
        float u0, u1, v0, v1;
        unpack2(fma2(pack2(__float_as_uint(x[i]), __float_as_uint(x[i + 1])), kk, ref), u0, u1);
        unpack2(fma2(pack2(__float_as_uint(x[i + 2]), __float_as_uint(x[i + 3])), kk, ref), v0, v1);
        s0 = add2(s0, pack2(__float_as_uint(ex2(u0)), __float_as_uint(ex2(u1))));
        s1 = add2(s1, pack2(__float_as_uint(ex2(v0)), __float_as_uint(ex2(v1))));
    }
}

// Column of element `i` of an edge granule of the slice (which = 0: the first,
// 1: the last), or -1 where there is none or it is another row's.
template <class T>
__device__ __forceinline__ int edge_column(const RowView<T>& v, const Slice<T>& sl, int vocab, int which, int i) {
    const int g = which == 0 ? (sl.a > sl.lo ? sl.lo : -1) : (sl.b < sl.hi ? sl.b : -1);
    if (g < 0 || i >= Elem<T>::kPer) return -1;
    const int j = g * Elem<T>::kPer + i - v.off;
    return j >= 0 && j < vocab ? j : -1;
}

// A row is summed in segments of 256 granules, eight a lane, one warp each; the
// segments' sums are added in a fixed order.  So a row's bits do not depend on
// how many CTAs and threads it is given, and not on the rows beside it.
constexpr int kSegment = 256;

// Granule g for the sums: whole, or with -inf in the place of other rows' elements.
template <class T, bool kKeep>
__device__ __forceinline__ uint4 any_granule(const RowView<T>& v, const Slice<T>& sl, int vocab, int g) {
    if (g >= sl.a && g < sl.b) return load_granule<kKeep>(v.granule(g));
    float x[Elem<T>::kPer];
#pragma unroll
    for (int k = 0; k < Elem<T>::kPer; ++k) {
        const int j = g * Elem<T>::kPer + k - v.off;
        x[k] = g < sl.hi && j >= 0 && j < vocab ? Elem<T>::to_f(v.row[j]) : kNegInf;
    }
    return Elem<T>::pack(x);
}
template <class T, bool kFull>
__device__ __forceinline__ uint32_t any_bits(const Slice<T>& sl, int g) {
    return kFull && g < sl.hi ? sl.bits(g) : 0u;
}

// Sum of the segment from granule g0 on with reference m2, in every lane.
template <class T, bool kFull, bool kKeep>
__device__ __forceinline__ float segment_sum(const RowView<T>& v, const Slice<T>& sl, int vocab, int g0, float k2,
                                             float m2) {
    const uint64_t kk = both(k2), ref = both(-m2);
    const int lane = threadIdx.x & 31;
    uint64_t s0 = 0, s1 = 0;
    if (g0 >= sl.a && g0 + kSegment <= sl.b) {
#pragma unroll 1
        for (int g = g0 + lane; g < g0 + kSegment; g += 128) {
            uint4 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = load_granule<kKeep>(v.granule(g + 32 * i));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                add_exps<T, kFull>(b[i], kFull ? sl.bits(g + 32 * i) : 0u, kk, ref, s0, s1);
        }
    } else {  // the row's first or last; the same order
#pragma unroll 1
        for (int g = g0 + lane; g < g0 + kSegment; g += 32)
            add_exps<T, kFull>(any_granule<T, kKeep>(v, sl, vocab, g), any_bits<T, kFull>(sl, g), kk, ref, s0, s1);
    }
    float x, y;
    unpack2(add2(s0, s1), x, y);
    return warp_reduce(x + y, AddOp());
}

// The segment's own maximum, times k2.
template <class T, bool kFull>
__device__ __noinline__ float segment_max(const RowView<T>& v, const Slice<T>& sl, int vocab, int g0, float k2) {
    float m = kNegInf;
#pragma unroll 1
    for (int g = g0 + static_cast<int>(threadIdx.x & 31); g < g0 + kSegment; g += 32) {
        float x[Elem<T>::kPer];
        Elem<T>::unpack(any_granule<T, true>(v, sl, vocab, g), x);
        const uint32_t bits = any_bits<T, kFull>(sl, g);
#pragma unroll
        for (int k = 0; k < Elem<T>::kPer; ++k) m = fmaxf(m, bits >> k & 1u ? kNegInf : x[k]);
    }
    return warp_reduce(m, MaxOp()) * k2;
}

// Reference and sum of a segment.  The listed columns' maximum `guess` nearly
// always is a fair reference for the others: a sum that neither overflows nor
// comes near underflow is as exact with one reference as with another.
// Otherwise the segment's own maximum is taken.
template <class T, bool kFull, bool kKeep>
__device__ __forceinline__ float2 segment(const RowView<T>& v, const Slice<T>& sl, int vocab, int g0, float k2,
                                          float guess) {
    float m2 = fabsf(guess) < 1e30f ? guess : 0.0f;
    float sum = segment_sum<T, kFull, kKeep>(v, sl, vocab, g0, k2, m2);
    if (!(sum > 1e-27f && sum < 1e30f)) {
        m2 = segment_max<T, kFull>(v, sl, vocab, g0, k2);
        sum = segment_sum<T, kFull, kKeep>(v, sl, vocab, g0, k2, m2 == kNegInf ? 0.0f : m2);
    }
    return make_float2(m2, sum);
}

// The sums of a whole row; every lane gets them.
struct RowSums {
    float M2, S, inv_S;   // reference and sum of the whole row
    float m2o, s_o;       // of the columns outside the list (with kFull; else the same)
    float ref_o, B;       // gradient outside the list: w tau B 2^(s k2 - ref_o)
    float p_r;            // the teacher's mass outside its list
    float Q;              // the student's mass inside the list
    bool small;           // the list holds at most half of either mass
};
// part: (reference, sum) of every segment; s_exp, with kFull: the student's
// exponential of every listed column, -1 for a slot that stands for none.
template <bool kFull>
__device__ __forceinline__ RowSums row_sums(const DistillArgs& a, const ListInfo& info, const float2* part, int n_part,
                                            const float* s_exp) {
    const int lane = threadIdx.x & 31;
    RowSums r;
    r.m2o = kNegInf;
    r.s_o = 0.0f;
    for (int i = lane; i < n_part; i += 32) r.m2o = fmaxf(r.m2o, part[i].x);
    r.m2o = warp_reduce(r.m2o, MaxOp());
    for (int i = lane; i < n_part; i += 32) r.s_o += part[i].y * rescale(part[i].x, r.m2o);
    r.s_o = warp_reduce(r.s_o, AddOp());
    r.M2 = r.m2o;
    r.S = r.s_o;
    r.p_r = r.Q = 0.0f;
    r.small = false;
    float f_o = 1.0f;
    if (kFull) {
        float s_t = 0.0f;
        int listed = 0;
        for (int k = lane; k < a.top; k += 32)
            if (!(s_exp[k] < 0.0f)) {
                s_t += s_exp[k];
                ++listed;
            }
        s_t = warp_reduce(s_t, AddOp());
        listed = __reduce_add_sync(0xffffffffu, listed);
        const float m2_top = info.m_top * a.k2;
        r.M2 = fmaxf(r.m2o, m2_top);
        f_o = rescale(r.m2o, r.M2);
        s_t *= rescale(m2_top, r.M2);
        r.S = r.s_o * f_o + s_t;
        r.Q = s_t / r.S;
        r.p_r = (1.0f - info.p_hi) - info.p_lo;
        // none where the list names every column
        if (r.p_r < 0.0f || listed >= a.vocab) r.p_r = 0.0f;
        r.small = r.p_r >= 0.5f && r.Q <= 0.5f;
    }
    r.inv_S = info.bad ? NAN : 1.0f / r.S;
    r.B = f_o * r.inv_S;
    if (r.small)
        r.B = (info.p_hi - r.Q + info.p_lo) / r.s_o + (info.bad ? NAN : 0.0f);
    else if (r.p_r > 0.0f && r.s_o > 0.0f)
        r.B -= r.p_r / r.s_o;
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
        if (r.small) {
            L.add(r.p_r * (log1pf(-(info.p_hi + info.p_lo)) - log1pf(-r.Q)));
        } else if (r.p_r != 0.0f) {
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

// Gradients of a slice as if no column were listed; where the output row starts
// at another place of a 16-byte granule than the logits' row (!same), element
// by element.
template <class T>
__device__ __forceinline__ void write_slice(const DistillArgs& a, const RowView<T>& v, const Slice<T>& sl, T* out,
                                            bool same, float ref_o, float mul) {
    constexpr int kPer = Elem<T>::kPer;
    const uint64_t kk = both(a.k2), ref = both(-ref_o), mm = both(mul);
    const int nt = blockDim.x, t = threadIdx.x;
    float x[kPer];
    int g = sl.a + t;
    if (same) {
        uint4* const o = reinterpret_cast<uint4*>(out - v.off);
        for (; g + 3 * nt < sl.b; g += 4 * nt) {
            uint4 b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) b[i] = load_granule<false>(v.granule(g + i * nt));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                slice_grads<T>(b[i], kk, ref, mm, x);
                __stcs(o + g + i * nt, Elem<T>::pack(x));
            }
        }
    }
    for (; g < sl.b; g += nt) {
        slice_grads<T>(load_granule<false>(v.granule(g)), kk, ref, mm, x);
        store_granule<T>(out, g, v.off, a.vocab, same, x);
    }
    for (int e = 0; e < 2; ++e) {  // granules shared with a neighbouring row
        const int j = edge_column(v, sl, a.vocab, e, t);
        if (j >= 0) out[j] = Elem<T>::from_f(ex2(fmaf(Elem<T>::to_f(v.row[j]), a.k2, -ref_o)) * mul);
    }
}

// Dynamic shared memory: the bits of a slice's listed columns, the sums of the
// whole row's segments, and kListArrays arrays of `top` words.
constexpr int kListArrays = 5;
__host__ __device__ constexpr size_t align16(size_t n) { return (n + 15) & ~size_t(15); }
__host__ __device__ constexpr size_t bit_bytes(int slice) { return align16(static_cast<size_t>(slice)); }
__host__ __device__ constexpr size_t part_bytes(int segments) { return align16(static_cast<size_t>(segments) * 8); }
__host__ __device__ constexpr size_t list_bytes(int top) { return align16(static_cast<size_t>(top) * 4); }
size_t dynamic_bytes(int slice, int segments, int top) {
    return bit_bytes(slice) + part_bytes(segments) + kListArrays * list_bytes(top);
}

// One row per cluster; kFull: the teacher's log-sum is given.
template <class T, bool kGrad, bool kFull>
__global__ void __launch_bounds__(kMaxThreads, 3) distill_kernel(const DistillArgs a) {
    constexpr int kPer = Elem<T>::kPer;
    extern __shared__ uint4 dyn[];
    __shared__ float w_tm[kMaxWarps], w_mt[kMaxWarps];
    __shared__ int w_flags[kMaxWarps];
    __shared__ int next_segment;
    __shared__ ListInfo info;
    const int K = a.top, tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, n_warps = nt >> 5;
    uint8_t* const base = reinterpret_cast<uint8_t*>(dyn);
    uint32_t* const bits = reinterpret_cast<uint32_t*>(base);
    float2* const part = reinterpret_cast<float2*>(base + bit_bytes(a.slice));
    const size_t step = list_bytes(K) / 4;
    int* const s_idx = reinterpret_cast<int*>(base + bit_bytes(a.slice) + part_bytes(a.segments));
    float* const s_p = reinterpret_cast<float*>(s_idx) + step;  // p before its normalisation
    float* const s_s = s_p + step;                              // the student's logit
    float* const s_lead = s_s + step;                           // the column's p, or -1 where another slot has it
    float* const s_exp = s_lead + step;                         // the student's exponential, or -1

    uint32_t C;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
    const uint32_t rank = cluster_ctarank();
    const int64_t row = blockIdx.x / C;
    const RowView<T> v(a.logits, a.ld, row, a.vocab);
    const Slice<T> sl(v, a.vocab, static_cast<int>(rank), a.slice, reinterpret_cast<const uint8_t*>(bits));
    T* const out = kGrad ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
    const bool same = kGrad && ((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T)) == static_cast<unsigned>(v.off);
    // The row's scalars and the first entries of its list come together, and with
    // them the list of a row that will be worked on when this one is done, which
    // then finds it in L2 (loads of DRAM take 2 to 4 us while others stream).
    const float w = a.weights ? a.weights[row] : 1.0f;
    const float lse = kFull ? a.lse[row] : 0.0f;
    const int64_t j_first = tid < K ? load_index(a, row * K + tid) : -1;
    const float t_first = tid < K ? load_top(a, row * K + tid) : kNegInf;
    const int64_t later = row + a.ahead;
    uint32_t j_later = 0xffffffffu;
    if (later < a.rows && tid < K) {
        const int64_t i = later * K + tid;
        j_later = static_cast<const uint32_t*>(a.top_index)[a.index_bytes == 8 ? 2 * i : i];
        prefetch_l2(static_cast<const uint8_t*>(a.top_logits) + i * (a.top_dtype == HESS_F32 ? 4 : 2));
    }
    for (int i = tid; i < static_cast<int>(bit_bytes(a.slice) / 16); i += nt) dyn[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) next_segment = 0;
    __syncthreads();

    // ---- the teacher's list, the bits of its columns, and the student's logits there
    const int j_base = sl.lo * kPer - v.off, j0 = max(j_base, 0), j1 = min(a.vocab, sl.hi * kPer - v.off);
    float tm = kNegInf, mt = kNegInf;
    {
        bool any = false, bad = false, twice = false;
        if (w != 0.0f) {
            // The slice sets out for L2 while the list is worked on (8,192 x
            // 128,000 bf16: 772 -> 730 us; without the gradient it only gets in the
            // way of the loads).
            if (kGrad && lane == 0) {
                const int per = (sl.b - sl.a + n_warps - 1) / n_warps;
                const int g0 = sl.a + warp * per, g1 = min(sl.b, g0 + per);
                if (g0 < g1) prefetch_l2_bulk(v.granule(g0), static_cast<uint32_t>(g1 - g0) * 16u);
            }
            for (int k = tid; k < K; k += nt) {
                const int64_t j = k == tid ? j_first : load_index(a, row * K + k);
                const float t = k == tid ? t_first : load_top(a, row * K + k);
                const bool held = j >= 0 && t != kNegInf;
                const bool in = held && j < a.vocab;
                bad |= held && !in;
                any |= held;
                s_idx[k] = in ? static_cast<int>(j) : -1;
                s_p[k] = t;
                s_exp[k] = -1.0f;
                if (in) {
                    const float s = Elem<T>::to_f(v.row[j]);
                    if (j >= j0 && j < j1) {
                        const uint32_t bit = static_cast<uint32_t>(static_cast<int>(j) - j_base);
                        twice |= (atomicOr(bits + (bit >> 5), 1u << (bit & 31u)) >> (bit & 31u) & 1u) != 0;
                    }
                    s_s[k] = s;
                    tm = fmaxf(tm, t);
                    mt = fmaxf(mt, s);
                }
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        }
        const int flags = __reduce_or_sync(0xffffffffu, (any ? 1u : 0u) | (bad ? 2u : 0u) | (twice ? 4u : 0u));
        if (lane == 0) {
            w_tm[warp] = tm;
            w_mt[warp] = mt;
            w_flags[warp] = flags;
        }
    }
    __syncthreads();
    int flags = 0;
    for (int i = 0; i < n_warps; ++i) {
        tm = fmaxf(tm, w_tm[i]);
        mt = fmaxf(mt, w_mt[i]);
        flags |= w_flags[i];
    }
    if (!flags) {  // no weight or no list: the whole cluster leaves here
        if (kGrad) zero_slice<T>(v, out, a.vocab, same, sl.lo, sl.hi, tid, nt);
        if (rank == 0 && tid == 0) store_dead(a, row, !kGrad);
        return;
    }
    // the other CTAs may write here from now on (they wait for it below)
    if (C > 1) cluster_arrive();
    const float m2_top = mt * a.k2;
    if (warp == n_warps - 1) {
        // ---- the last warp: p, the list's sums, and the student's exponentials
        // at the listed columns, while the others begin with the segments
        ListInfo q{(flags & 2) != 0, w, tm, mt, 0.0f, 0.0f, 1.0f, 0.0f, lse};
        for (int k = lane; k < K; k += 32) {
            float e = 0.0f;
            if (s_idx[k] >= 0) {
                const float t = s_p[k], s = s_s[k];
                e = teacher_exp(a, t, kFull ? lse : tm, kFull);
                if (e != 0.0f)
                    q.a += s == kNegInf ? INFINITY : e * fmaf(s, a.k2_slip, fmaf(t - s, a.inv_hi, (t - s) * a.inv_lo));
                float err;
                q.p_hi = two_sum_f32(q.p_hi, e, err);
                q.p_lo += err;
            }
            s_p[k] = e;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, q.p_hi, o), l = __shfl_xor_sync(0xffffffffu, q.p_lo, o);
            q.a += __shfl_xor_sync(0xffffffffu, q.a, o);
            float e;
            q.p_hi = two_sum_f32(q.p_hi, h, e);
            q.p_lo += l + e;
        }
        if (!kFull) q.p_inv = 1.0f / (q.p_hi + q.p_lo);
        if (lane == 0) info = q;
        __syncwarp();
    }
    if (C > 1) cluster_wait();
    if (warp == n_warps - 1) {
        // A column's p at its first slot; the others, if it is listed more than
        // once, stand back.  The exponentials go to every CTA of the cluster.
        for (int k = lane; k < K; k += 32) {
            const int j = s_idx[k];
            if (j < j0 || j >= j1) continue;
            float p = s_p[k];
            if (flags & 4) {
                p = 0.0f;
                for (int l = 0; l < K && p >= 0.0f; ++l)
                    if (s_idx[l] == j) p = l < k ? -1.0f : p + s_p[l];
            }
            s_lead[k] = p < 0.0f ? p : p * info.p_inv;
            if (kFull && !(p < 0.0f)) {
                const float e = m2_top == kNegInf ? 0.0f : ex2(fmaf(s_s[k], a.k2, -m2_top));
                for (uint32_t r = 0; r < C; ++r) st_cluster_f32(mapa_shared(smem_u32(s_exp + k), r), e);
            }
        }
        __syncwarp();
    }

    // ---- the sums of the slice's segments, which go to every CTA of the cluster
    for (;;) {
        int i = 0;
        if (lane == 0) i = atomicAdd(&next_segment, 1);
        const int g0 = sl.lo + __shfl_sync(0xffffffffu, i, 0) * kSegment;
        if (g0 >= sl.hi) break;
        const float2 q = segment<T, kFull, kGrad>(v, sl, a.vocab, g0, a.k2, m2_top);
        if (lane < static_cast<int>(C))
            st_cluster_f32x2(mapa_shared(smem_u32(part + g0 / kSegment), lane), q.x, q.y);
    }
    if (j_later < static_cast<uint32_t>(a.vocab))
        prefetch_l2(static_cast<const T*>(a.logits) + later * a.ld + j_later);
    if (C == 1)
        __syncthreads();
    else
        cluster_sync_all();
    const RowSums r = row_sums<kFull>(a, info, part, (v.n + kSegment - 1) / kSegment, s_exp);
    if (rank == 0 && warp == n_warps - 1) {
        const float loss = row_loss(a, info, r);
        if (lane == 0) {
            a.loss[row] = loss;
            if (!kGrad) store_stats(a, row, info, r);
        }
    }
    if constexpr (kGrad) {
        const float gs = w * a.tau;
        write_slice<T>(a, v, sl, out, same, r.ref_o, gs * r.B);
        __syncthreads();  // the listed columns' values go over what was just stored there
        for (int k = tid; k < K; k += nt) {
            const int j = s_idx[k];
            if (j >= j0 && j < j1 && !(s_lead[k] < 0.0f))
                out[j] = Elem<T>::from_f(gs * (ex2(fmaf(s_s[k], a.k2, -r.M2)) * r.inv_S - s_lead[k]));
        }
    }
}

// Gradient from saved statistics: one CTA per slice of a row, no exchange.
// A stream without reuse: 4,096 x 65,536 bf16 176 us, 83 % of a copy of its bytes
// (186 us with 256 threads a CTA; 8,192 x 4,000: 43 against 72 us).
constexpr int kBwdThreads = 128;
constexpr int kInFlight = 4;                            // granules a thread loads at a time
constexpr int kBwdSlice = kBwdThreads * kInFlight * 2;  // granules per CTA

template <class T>
__global__ void __launch_bounds__(kBwdThreads) distill_backward_kernel(const DistillArgs a, int n_slices) {
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
        zero_slice<T>(v, out, a.vocab, same, g_lo, g_hi, tid, kBwdThreads);
        return;
    }
    const float M2 = st0.x, inv_S = st0.y, ref_o = st0.z;
    const float gs = w * a.tau * (a.grad ? a.grad[row] : 1.0f), mul = gs * st0.w;
    // the first loads are on their way while the list is read
    uint4 b[kInFlight];
    const auto load = [&](int g) {
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int gg = g + i * kBwdThreads;
            if (gg < g_hi && v.whole(gg, a.vocab)) b[i] = load_granule<false>(v.granule(gg));
        }
    };
    load(g_lo + tid);
    // this slice's part of the list; the student's logits there are read
    // before any gradient is stored (dlogits may be logits)
    if (tid == 0) s_n = 0;
    __syncthreads();
    const int j0 = max(0, g_lo * kPer - v.off), j1 = min(a.vocab, g_hi * kPer - v.off);
    const bool full = a.lse != nullptr;
    const float base = full ? a.lse[row] : st1.x;
    for (int k = tid; k < a.top; k += kBwdThreads) {
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
    for (int g = g_lo + tid; g < g_hi; g += kBwdThreads * kInFlight) {
        if (g != g_lo + tid) load(g);
#pragma unroll
        for (int i = 0; i < kInFlight; ++i) {
            const int gg = g + i * kBwdThreads;
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
    for (int i = tid; i < n; i += kBwdThreads) {
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
    if (vocab > (int64_t(1) << 22)) return ds_fail(HESS_ERR_UNSUPPORTED, "vocab > 2^22");
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
            const bool in_place = s0 == d0 && (a.ld == a.ldd || a.rows == 1);
            // rows of one stride may lie between each other, as columns of one buffer
            const uintptr_t stride = a.ld * es, width = a.vocab * es;
            const uintptr_t shift = (d0 > s0 ? d0 - s0 : stride - (s0 - d0) % stride) % stride;
            const bool between = a.ld == a.ldd && shift >= width && shift + width <= stride;
            if (!in_place && !between && s0 < d1 && d0 < s1)
                return ds_fail(HESS_ERR_INVALID, "dlogits overlaps logits without being logits");
        }
    }
    return HESS_OK;
}

constexpr size_t kMaxDynamic = 220 * 1024;

template <class T, bool kGrad>
hess_status launch_typed(DistillArgs& a, int sms, cudaStream_t s) {
    constexpr int per = Elem<T>::kPer;
    const int granules = static_cast<int>((static_cast<int64_t>(a.vocab) + 2 * (per - 1)) / per);
    // CTAs per row and threads per CTA (the kernels' registers leave an SM 1,536
    // threads; figures: bf16 rows with an eighth without weight, in steady state).
    // With the gradient the slices in flight should fill L2 and no more, 72 MB: they
    // are read again from there.  One CTA a row while its 512 threads keep to that,
    // else twice the fewest that do, and as few threads as do (8,192 x 128,000: 687
    // us with 4 CTAs of 256 threads a row, 707 with 2 of 512, 805 with 2 of 384,
    // 902 with 1 of 512; 4,096 x 100,000: 290 us with 4 of 192, 318 with 2 of 512;
    // 4,096 x 65,536: 184 us with 1 of 512, 198 with 2 of 256).
    // Without it one CTA, and small ones, which hide each other's start (8,192 x
    // 128,000: 266 us with 256 threads, 291 with 512, 313 with 128; 4,096 x 65,536:
    // 72 us with 128, 76 with 256, 98 with 512).  Rows between those two widths go
    // with the wider ones: 128 threads are 7 % faster there for many of them (8,192 x
    // 96,000: 201 against 214) up to some 12,000 granules (8,192 x 112,000: 286
    // against 244), but slower where 256 make one wave (904 x 96,000: 42 against 29).
    a.segments = (granules + kSegment - 1) / kSegment;
    const auto slice_at = [&](int c) { return (a.segments + c - 1) / c * kSegment; };
    const auto fits = [&](int c) { return dynamic_bytes(slice_at(c), a.segments, a.top) <= kMaxDynamic; };
    const double in_flight = 72e6;
    int C = 1, threads = slice_at(1) > 8448 ? 256 : 128;
    if (kGrad) {
        while (C < kMaxCluster && 3.0 * sms * 16.0 * slice_at(C) > in_flight) C *= 2;
        if (C > 1 && C < kMaxCluster) C *= 2;
        int per_sm = 12;  // CTAs of floor(1536 / per_sm) threads, where that is just how many fit
        while (per_sm > 3 && (per_sm * (16.0 * sms) * slice_at(C) > in_flight ||
                              1536 / (1536 / per_sm / 32 * 32) != per_sm))
            --per_sm;
        threads = 1536 / per_sm / 32 * 32;
    }
    while (C < kMaxCluster && !fits(C)) C *= 2;
    // Few rows: more CTAs for each while half of the threads would be idle; and
    // smaller ones where one wave of them then does for two (301 x 50,257 f32 with
    // gradient, 2 CTAs a row: 29.6 us with 384 threads, 40 with 512; from three
    // waves to two it is a loss, 512 x 128,000 bf16: 65 against 60 us).  Not where
    // a thread would walk more than 110 granules: too few loads are then in flight
    // (the loss, one wave against two; 87 granules, 1,150 x 128,000 bf16: 45 and 55
    // us; 104, 1,350 rows of it: 52 and 60; 100, 1,500 x 50,257 f32: 46 and 49; but
    // 130, 1,700 x 128,000 bf16: 82 and 67; 124, 1,150 x 94,364 f32: 87 and 75).
    const int64_t room = int64_t(1536) * sms;
    while (C < kMaxCluster && 2 * a.rows * C * threads <= room && granules >= 512 * C) C *= 2;
    const int64_t ctas = a.rows * C, slots = int64_t(1536 / threads) * sms;
    if (ctas > slots && ctas <= 2 * slots) {
        const int64_t t = 1536 / ((ctas + sms - 1) / sms) / 32 * 32;
        if (t >= 128 && 2 * t >= threads && slice_at(C) <= 110 * t) threads = static_cast<int>(t);
    }
    // not reached: the widest vocabulary in f32, 8 CTAs and the longest list take 185 KB
    if (!fits(C))
        return ds_fail(HESS_ERR_UNSUPPORTED, "vocab %d is too wide for the bits of its columns", a.vocab);
    a.slice = slice_at(C);
    a.ahead = static_cast<int32_t>(room / (int64_t(C) * threads));
    const size_t smem = dynamic_bytes(a.slice, a.segments, a.top);
    auto fn = a.lse ? distill_kernel<T, kGrad, true> : distill_kernel<T, kGrad, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.rows * C), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(C);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = C > 1 ? 1 : 0;
    DS_TRY(cudaLaunchKernelEx(&cfg, fn, a));
    return HESS_OK;
}

template <class T>
cudaError_t allow_shared() {
    for (auto fn : {distill_kernel<T, false, false>, distill_kernel<T, false, true>, distill_kernel<T, true, false>,
                    distill_kernel<T, true, true>}) {
        const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kMaxDynamic));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

hess_status ds_prepare(int dev, int* sms) {
    static std::mutex mu;
    static int count[128] = {};
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 0 || dev >= 128) return ds_fail(HESS_ERR_UNSUPPORTED, "device index %d", dev);
    if (!count[dev]) {
        DS_TRY(allow_shared<__nv_bfloat16>());
        DS_TRY(allow_shared<__half>());
        DS_TRY(allow_shared<float>());
        int n = 0;
        DS_TRY(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
        count[dev] = n;
    }
    *sms = count[dev];
    return HESS_OK;
}

template <bool kGrad>
hess_status launch_rows(DistillArgs& a, int32_t dtype, cudaStream_t s) {
    int dev = 0;
    hess_status st = ds_buffers(a, &dev);
    if (st != HESS_OK) return st;
    int sms = 0;
    st = ds_prepare(dev, &sms);
    if (st != HESS_OK) return st;
    if (dtype == HESS_BF16) return launch_typed<__nv_bfloat16, kGrad>(a, sms, s);
    if (dtype == HESS_F16) return launch_typed<__half, kGrad>(a, sms, s);
    return launch_typed<float, kGrad>(a, sms, s);
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
        hk::distill_backward_kernel<__nv_bfloat16><<<grid, hk::kBwdThreads, 0, s>>>(a, n_slices);
    else if (dtype == HESS_F16)
        hk::distill_backward_kernel<__half><<<grid, hk::kBwdThreads, 0, s>>>(a, n_slices);
    else
        hk::distill_backward_kernel<float><<<grid, hk::kBwdThreads, 0, s>>>(a, n_slices);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return hk::ds_fail(HESS_ERR_CUDA, "distill_backward: %s", cudaGetErrorString(e));
    return HESS_OK;
}
