// 8-bit rows: int8 codes with a scale per row or per group of columns
// (formulas and conventions: include/rows8.h).
//
// The unit of work is a segment: 256 columns of one row, eight per lane of a warp.
// A group of 32 .. 256 columns lies inside a segment, so its maximum is a few
// shuffles; a whole row's segments are held in the registers of one CTA and its
// maximum meets in shared memory, so that the values are read once either way.
// Where rows start on 16 bytes and d is a multiple of 8 a lane owns eight columns
// side by side (16-byte accesses); otherwise it owns columns 32 apart, which keeps a
// warp's accesses contiguous at any alignment.
//
// The whole number nearest to the exact quotient x / s is wanted.  x (1/s) differs from
// the quotient by less than 2^-15 for |x / s| <= 127.5, so both round to the same whole
// number unless the product lies that close to a half: only then is it looked at more
// closely (1 value in 10^4), and the kernel stays at the memory's pace.
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_ptr.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rows8.cuh"
#include "rows8.h"

namespace hk {
namespace {

constexpr int kSegment = 256;
constexpr int kItemSegments = 4;  // segments one warp has in flight

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Column of a lane's element e within a segment.
template <bool kVec>
__device__ __forceinline__ int column(int lane, int e) {
    return kVec ? lane * 8 + e : e * 32 + lane;
}

// A lane's eight values of the segment that begins at column c0; zeros past d.
template <class T, bool kVec>
struct Raw {
    union {
        uint4 q[sizeof(T) / 2];
        T v[8];
    };
    __device__ Raw() {}
    __device__ __forceinline__ void load(const T* row, int64_t c0, int64_t d, int lane) {
        if constexpr (kVec) {
            const int64_t c = c0 + lane * 8;
            if (c < d) {
#pragma unroll
                for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
                    q[i] = __ldcs(reinterpret_cast<const uint4*>(row + c) + i);
            } else {
#pragma unroll
                for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) q[i] = make_uint4(0, 0, 0, 0);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t c = c0 + column<false>(lane, e);
                v[e] = c < d ? row[c] : from_f32<T>(0.0f);
            }
        }
    }
};

// |x| as bits: ordered like the values, infinity and NaN above all of them.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

struct Scale {
    float s;     // as it is stored
    float t, r;  // what the values are divided by, and its reciprocal
    int how;     // 0: codes are 0, 1: s is a normal number, 2: s is subnormal
};
__device__ __forceinline__ Scale scale_of(uint32_t top) {
    Scale k;
    k.t = k.r = 1.0f;
    k.how = 0;
    if (top >= 0x7f800000u) {
        k.s = __uint_as_float(0x7fffffffu);
        return k;
    }
    k.s = __fdiv_rn(__uint_as_float(top), 127.0f);
    if (k.s == 0.0f) return k;
    // a subnormal scale and its values are both taken 2^64 times (exactly)
    k.how = k.s < 1.17549435e-38f ? 2 : 1;
    k.t = k.how == 2 ? __fmul_rn(k.s, 18446744073709551616.0f) : k.s;
    k.r = __frcp_rn(k.t);
    return k;
}

constexpr float kNearHalf = 0.5f - 1.0f / 32768.0f;

// rint(x / s) of the exact quotient.  Near a half the sign of x - (half) s, which a
// fused multiply-add gives exactly, says on which side of it the quotient lies.
__device__ __forceinline__ int encode1(float x, const Scale& k) {
    if (k.how == 0) return 0;
    if (k.how == 2) x = __fmul_rn(x, 18446744073709551616.0f);
    const float t = fminf(fmaxf(__fmul_rn(x, k.r), -127.0f), 127.0f);
    float q = rintf(t);
    if (fabsf(__fsub_rn(t, q)) > kNearHalf) {
        const float lo = floorf(t);
        const float e = __fmaf_rn(-__fadd_rn(lo, 0.5f), k.t, x);
        if (e != 0.0f) q = e > 0.0f ? __fadd_rn(lo, 1.0f) : lo;
        else q = rintf(__fadd_rn(lo, 0.5f));
    }
    return static_cast<int>(q);
}

// Eight codes in the low bytes of eight words.
__device__ __forceinline__ void encode8(const float (&x)[8], const Scale& k, int (&q)[8]) {
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number, half to even
    if (k.how == 1) {
        float far = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float t = __fmul_rn(x[e], k.r);
            const float y = __fadd_rn(t, kMagic);
            far = fmaxf(far, fabsf(__fsub_rn(t, __fsub_rn(y, kMagic))));
            q[e] = __float_as_int(y);
        }
        if (far <= kNearHalf) return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = encode1(x[e], k);
}

__device__ __forceinline__ uint32_t pack_bytes(int a, int b, int c, int d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The low bytes of two words as float16 whole numbers: 1024 + (q + 128) has the
// byte q ^ 0x80 at its low end.
__device__ __forceinline__ uint32_t wide2(int a, int b) {
    const uint32_t w = __byte_perm(a, b, 0x3430) & 0x00ff00ffu;  // a's and b's low byte, 16 bits each
    const uint32_t biased = w ^ 0x64806480u;
    __half2 h;
    memcpy(&h, &biased, 4);
    h = __hsub2(h, __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    uint32_t out;
    memcpy(&out, &h, 4);
    return out;
}

// Codes as bytes, or as float16 whole numbers.
template <bool kVec>
__device__ __forceinline__ void store8(int8_t* codes, __half* wide, int64_t c0, int64_t d, int lane, const int (&q)[8]) {
    if constexpr (kVec) {
        const int64_t c = c0 + lane * 8;
        if (c >= d) return;
        if (codes) {
            const uint2 w = make_uint2(pack_bytes(q[0], q[1], q[2], q[3]), pack_bytes(q[4], q[5], q[6], q[7]));
            *reinterpret_cast<uint2*>(codes + c) = w;
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = wide2(q[2 * i], q[2 * i + 1]);
            *reinterpret_cast<uint4*>(wide + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t c = c0 + column<false>(lane, e);
            if (c < d) {
                if (codes) codes[c] = static_cast<int8_t>(q[e]);
                else wide[c] = __ushort_as_half(static_cast<unsigned short>(wide2(q[e], 0)));
            }
        }
    }
}

// item / items, without a 64-bit division where 32 bits do.
__device__ __forceinline__ int64_t row_of(int64_t item, int32_t items) {
    if (item < 0x100000000ll) return static_cast<uint32_t>(item) / static_cast<uint32_t>(items);
    return item / items;
}

struct QuantizeParams {
    const void* x;
    int64_t ldx, n, d, ldc, ldw;
    int32_t group;    // group kernel: 32 .. 256, or 256 for whole rows of at most 256 columns
    int32_t shift;    // its logarithm
    int64_t groups;   // scales of a row
    int32_t items;    // group kernel: items of kItemSegments segments in a row
    int32_t held;     // row kernel: columns that a pass of the CTA covers
    int8_t* codes;
    __half* wide;
    float* scale;
};

// Scales per group: one warp takes kItemSegments segments of a row.
template <class T, bool kVec>
__global__ void __launch_bounds__(256) rows8_group_kernel(const __grid_constant__ QuantizeParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t r = row_of(item, p.items);
    if (r >= p.n) return;
    const int64_t c00 = (item - r * p.items) * (kItemSegments * kSegment);
    const T* const row = static_cast<const T*>(p.x) + r * p.ldx;
    Raw<T, kVec> raw[kItemSegments];
#pragma unroll
    for (int i = 0; i < kItemSegments; ++i) raw[i].load(row, c00 + i * kSegment, p.d, lane);
#pragma unroll
    for (int i = 0; i < kItemSegments; ++i) {
        const int64_t c0 = c00 + i * kSegment;
        if (c0 >= p.d) return;
        float x[8];
        int q[8];
        int8_t* const codes = p.codes ? p.codes + r * p.ldc : nullptr;
        __half* const wide = p.codes ? nullptr : p.wide + r * p.ldw;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = to_f32(raw[i].v[e]);
        if constexpr (kVec) {
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, magnitude(x[e]));
            for (int o = p.group >> 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
            const Scale k = scale_of(top);
            const int64_t c = c0 + lane * 8;
            if (c < p.d && (lane & ((p.group >> 3) - 1)) == 0) p.scale[r * p.groups + (c >> p.shift)] = k.s;
            encode8(x, k, q);
        } else {
            // a group is group / 32 elements of every lane
            const int each = p.group >> 5;
            uint32_t top[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) top[e] = __reduce_max_sync(~0u, magnitude(x[e]));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                uint32_t t = 0;
#pragma unroll
                for (int o = 0; o < 8; ++o)
                    if (o / each == e / each) t = max(t, top[o]);
                const Scale k = scale_of(t);
                const int64_t c = c0 + e * 32;
                if (lane == 0 && e % each == 0 && c < p.d) p.scale[r * p.groups + (c >> p.shift)] = k.s;
                q[e] = encode1(x[e], k);
            }
        }
        store8<kVec>(codes, wide, c0, p.d, lane, q);
    }
}

// One scale per row: a CTA takes one row, kHeld segments per warp in registers.
// Rows longer than that are read twice (the second time mostly from L2).
template <class T, bool kVec, int kHeld>
__global__ void __launch_bounds__(512) rows8_row_kernel(const __grid_constant__ QuantizeParams p) {
    griddep_wait();
    griddep_launch_dependents();
    __shared__ uint32_t tops[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = blockIdx.x;
    const T* const row = static_cast<const T*>(p.x) + r * p.ldx;
    int8_t* const codes = p.codes ? p.codes + r * p.ldc : nullptr;
    __half* const wide = p.codes ? nullptr : p.wide + r * p.ldw;
    Raw<T, kVec> raw[kHeld];
    uint32_t top = 0;
    for (int64_t c00 = warp * (kHeld * kSegment); c00 < p.d; c00 += p.held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) raw[i].load(row, c00 + i * kSegment, p.d, lane);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, magnitude(to_f32(raw[i].v[e])));
    }
    top = __reduce_max_sync(~0u, top);
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = lane < static_cast<int>(blockDim.x >> 5) ? tops[lane] : 0u;
    top = __reduce_max_sync(~0u, top);
    const Scale k = scale_of(top);
    if (threadIdx.x == 0) p.scale[r] = k.s;
    for (int64_t c00 = warp * (kHeld * kSegment); c00 < p.d; c00 += p.held) {
        if (p.held < p.d) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) raw[i].load(row, c00 + i * kSegment, p.d, lane);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int64_t c0 = c00 + i * kSegment;
            if (c0 >= p.d) break;
            float x[8];
            int q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = to_f32(raw[i].v[e]);
            encode8(x, k, q);
            store8<kVec>(codes, wide, c0, p.d, lane, q);
        }
    }
}

struct RestoreParams {
    const int8_t* codes;
    const float* scale;  // NULL: 1
    int64_t ldc, n, d, ldx;
    int32_t shift;   // log2(group); whole rows: 63
    int64_t groups;  // scales of a row
    int32_t items;   // items of kItemSegments segments in a row
    void* x;
};

// A byte as a float: 2^23 + (q + 128) has the byte q ^ 0x80 at its low end.
__device__ __forceinline__ float byte_to_f32(uint32_t biased, uint32_t which) {
    return __fsub_rn(__uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7440 + which)), 8388736.0f);
}

template <class T, bool kVec>
__global__ void __launch_bounds__(256) rows8_restore_kernel(const __grid_constant__ RestoreParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t r = row_of(item, p.items);
    if (r >= p.n) return;
    const int64_t c00 = (item - r * p.items) * (kItemSegments * kSegment);
    const int8_t* const codes = p.codes + r * p.ldc;
    const float* const scale = p.scale ? p.scale + r * p.groups : nullptr;
    T* const out = static_cast<T*>(p.x) + r * p.ldx;
    if constexpr (kVec) {
        uint2 w[kItemSegments];
        float s[kItemSegments];
#pragma unroll
        for (int i = 0; i < kItemSegments; ++i) {
            const int64_t c = c00 + i * kSegment + lane * 8;
            const bool in = c < p.d;
            w[i] = in ? __ldcs(reinterpret_cast<const uint2*>(codes + c)) : make_uint2(0, 0);
            s[i] = in && scale ? scale[c >> p.shift] : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < kItemSegments; ++i) {
            const int64_t c = c00 + i * kSegment + lane * 8;
            if (c >= p.d) return;
            const uint32_t a = w[i].x ^ 0x80808080u, b = w[i].y ^ 0x80808080u;
            union {
                uint4 q[sizeof(T) / 2];
                T v[8];
            } y;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y.v[e] = from_f32<T>(__fmul_rn(byte_to_f32(a, e), s[i]));
                y.v[4 + e] = from_f32<T>(__fmul_rn(byte_to_f32(b, e), s[i]));
            }
#pragma unroll
            for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j) reinterpret_cast<uint4*>(out + c)[j] = y.q[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kItemSegments; ++i) {
            int8_t q[8];
            float s[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t c = c00 + i * kSegment + column<false>(lane, e);
                q[e] = c < p.d ? codes[c] : int8_t(0);
                s[e] = c < p.d && scale ? scale[c >> p.shift] : 1.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int64_t c = c00 + i * kSegment + column<false>(lane, e);
                if (c < p.d) out[c] = from_f32<T>(__fmul_rn(static_cast<float>(q[e]), s[e]));
            }
        }
    }
}

int log2_of(int32_t group) {
    int k = 0;
    while ((1 << k) < group) ++k;
    return k;
}

template <class Kernel, class Params>
cudaError_t rows_launch(Kernel kernel, const Params& p, int64_t grid, int threads, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

bool aligned(const void* p, int64_t stride_bytes, int to) {
    return reinterpret_cast<uintptr_t>(p) % to == 0 && stride_bytes % to == 0;
}

template <class T, bool kVec>
cudaError_t quantize_as(QuantizeParams& p, cudaStream_t s) {
    if (p.group != 0 || p.d <= kSegment) {
        if (p.group == 0) p.group = kSegment;
        p.shift = log2_of(p.group);
        p.items = static_cast<int32_t>((p.d + kItemSegments * kSegment - 1) / (kItemSegments * kSegment));
        return rows_launch(rows8_group_kernel<T, kVec>, p, (p.n * p.items + 7) / 8, 256, s);
    }
    // Few rows are spread over more warps each, so that a row takes one round trip to
    // memory and little work after it; many rows get smaller CTAs.
    const int64_t segments = (p.d + kSegment - 1) / kSegment;
    const int64_t held = p.n <= 512 ? (segments + 15) / 16 : 4;
    const int h = held <= 1 ? 1 : held <= 2 ? 2 : 4;
    int64_t warps = (segments + h - 1) / h;
    if (warps > 16) warps = 16;
    p.held = static_cast<int32_t>(warps * h * kSegment);
    const auto kernel = h == 1 ? rows8_row_kernel<T, kVec, 1> : h == 2 ? rows8_row_kernel<T, kVec, 2>
                                                                       : rows8_row_kernel<T, kVec, 4>;
    return rows_launch(kernel, p, p.n, static_cast<int>(warps) * 32, s);
}

template <class T>
cudaError_t quantize_of(QuantizeParams& p, cudaStream_t s) {
    const bool vec = p.d % 8 == 0 && aligned(p.x, p.ldx * static_cast<int64_t>(sizeof(T)), 16) &&
                     (p.codes ? aligned(p.codes, p.ldc, 8) : aligned(p.wide, p.ldw * 2, 16));
    return vec ? quantize_as<T, true>(p, s) : quantize_as<T, false>(p, s);
}

template <class T>
cudaError_t restore_of(RestoreParams& p, cudaStream_t s) {
    const bool vec = p.d % 8 == 0 && aligned(p.codes, p.ldc, 8) &&
                     aligned(p.x, p.ldx * static_cast<int64_t>(sizeof(T)), 16);
    return rows_launch(vec ? rows8_restore_kernel<T, true> : rows8_restore_kernel<T, false>, p,
                       (p.n * p.items + 7) / 8, 256, s);
}

hess_status rows_fail(hess_status s, const char* fmt, ...) {
    char buf[384];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return s;
}

int item_bytes(int32_t dtype) { return dtype == HESS_F32 ? 4 : 2; }

struct RowsBuffer {
    const void* p;
    int64_t bytes;
    int align;
    const char* name;
};

hess_status check_sizes(int64_t n, int64_t d, int64_t ldx, int64_t ldc, int32_t dtype, int32_t group) {
    if (n < 0) return rows_fail(HESS_ERR_INVALID, "n_rows < 0");
    if (d <= 0) return rows_fail(HESS_ERR_INVALID, "d must be positive");
    if (ldx < d || ldc < d) return rows_fail(HESS_ERR_INVALID, "a row stride is less than d");
    if (dtype != HESS_BF16 && dtype != HESS_F16 && dtype != HESS_F32)
        return rows_fail(HESS_ERR_INVALID, "unknown dtype %d", dtype);
    if (group < 0) return rows_fail(HESS_ERR_INVALID, "group < 0");
    if (group != 0 && group != 32 && group != 64 && group != 128 && group != 256)
        return rows_fail(HESS_ERR_UNSUPPORTED, "group must be 0, 32, 64, 128 or 256, got %d", group);
    if (n > 0x7fffffff) return rows_fail(HESS_ERR_UNSUPPORTED, "n_rows exceeds 2^31 - 1");
    if (d > (int64_t(1) << 24)) return rows_fail(HESS_ERR_UNSUPPORTED, "d exceeds 2^24");
    // strides that keep every offset inside 64 bits, and a grid inside its limit
    if (ldx > (int64_t(1) << 28) || ldc > (int64_t(1) << 28))
        return rows_fail(HESS_ERR_UNSUPPORTED, "a row stride exceeds 2^28");
    if (n * ((d + kItemSegments * kSegment - 1) / (kItemSegments * kSegment)) > int64_t(8) * 0x7fffffff)
        return rows_fail(HESS_ERR_UNSUPPORTED, "n_rows * d is too large");
    return HESS_OK;
}

hess_status check_buffers(const RowsBuffer (&b)[3]) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return rows_fail(HESS_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    for (const RowsBuffer& x : b) {
        if (!x.p) return rows_fail(HESS_ERR_INVALID, "%s is NULL", x.name);
        if (reinterpret_cast<uintptr_t>(x.p) % x.align)
            return rows_fail(HESS_ERR_INVALID, "%s is not aligned to its element", x.name);
        char why[128];
        if (const char* w = device_ptr_problem(x.p, dev, why)) return rows_fail(HESS_ERR_INVALID, "%s %s", x.name, w);
    }
    return HESS_OK;
}

// Whether two buffers, from their first byte to their last, share one.
bool meet(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(b_bytes) && b0 < a0 + static_cast<uintptr_t>(a_bytes);
}

}  // namespace

cudaError_t rows8_quantize_launch(const void* X, int64_t ldx, int64_t n, int64_t d, int32_t dtype, int32_t group,
                                  int8_t* codes, int64_t ldc, uint16_t* wide, int64_t ldw, float* scale,
                                  cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    QuantizeParams p{};
    p.x = X;
    p.ldx = ldx;
    p.n = n;
    p.d = d;
    p.ldc = ldc;
    p.ldw = ldw;
    p.group = group;
    p.groups = group ? (d + group - 1) / group : 1;
    p.codes = codes;
    p.wide = reinterpret_cast<__half*>(wide);
    p.scale = scale;
    if (dtype == HESS_BF16) return quantize_of<__nv_bfloat16>(p, s);
    if (dtype == HESS_F16) return quantize_of<__half>(p, s);
    return quantize_of<float>(p, s);
}

cudaError_t rows8_restore_launch(const int8_t* codes, int64_t ldc, const float* scale, int64_t n, int64_t d,
                                 int32_t group, void* X, int64_t ldx, int32_t dtype, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    RestoreParams p{};
    p.codes = codes;
    p.scale = scale;
    p.ldc = ldc;
    p.n = n;
    p.d = d;
    p.ldx = ldx;
    p.shift = group ? log2_of(group) : 63;
    p.groups = group ? (d + group - 1) / group : 1;
    p.items = static_cast<int32_t>((d + kItemSegments * kSegment - 1) / (kItemSegments * kSegment));
    p.x = X;
    if (dtype == HESS_BF16) return restore_of<__nv_bfloat16>(p, s);
    if (dtype == HESS_F16) return restore_of<__half>(p, s);
    return restore_of<float>(p, s);
}

}  // namespace hk

using hk::rows_fail;

#define ROWS_EXPORT extern "C" __attribute__((visibility("default")))
#define ROWS_CHECK(expr)                \
    do {                                \
        const hess_status st_ = (expr); \
        if (st_ != HESS_OK) return st_; \
    } while (0)

ROWS_EXPORT hess_status rows8_quantize(const void* X, int64_t ldx, int64_t n_rows, int64_t d, int32_t dtype,
                                       int32_t group, int8_t* codes_out, int64_t ldc, float* scale_out,
                                       hess_stream_t stream) {
    ROWS_CHECK(hk::check_sizes(n_rows, d, ldx, ldc, dtype, group));
    if (n_rows == 0) return HESS_OK;
    const int item = hk::item_bytes(dtype);
    const int64_t scales = 4 * n_rows * (group ? (d + group - 1) / group : 1);
    ROWS_CHECK(hk::check_buffers({{X, 0, item, "X"}, {codes_out, 0, 1, "codes_out"}, {scale_out, 0, 4, "scale_out"}}));
    const int64_t x_bytes = ((n_rows - 1) * ldx + d) * item, c_bytes = (n_rows - 1) * ldc + d;
    if (hk::meet(X, x_bytes, codes_out, c_bytes)) return rows_fail(HESS_ERR_INVALID, "codes_out overlaps X");
    if (hk::meet(X, x_bytes, scale_out, scales)) return rows_fail(HESS_ERR_INVALID, "scale_out overlaps X");
    if (hk::meet(codes_out, c_bytes, scale_out, scales))
        return rows_fail(HESS_ERR_INVALID, "scale_out overlaps codes_out");
    const cudaError_t e = hk::rows8_quantize_launch(X, ldx, n_rows, d, dtype, group, codes_out, ldc, nullptr, 0,
                                                    scale_out, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rows_fail(HESS_ERR_CUDA, "rows8_quantize: %s", cudaGetErrorString(e));
    return HESS_OK;
}

ROWS_EXPORT hess_status rows8_restore(const int8_t* codes, int64_t ldc, const float* scale, int64_t n_rows, int64_t d,
                                      int32_t group, void* X_out, int64_t ldx, int32_t dtype, hess_stream_t stream) {
    ROWS_CHECK(hk::check_sizes(n_rows, d, ldx, ldc, dtype, group));
    if (n_rows == 0) return HESS_OK;
    const int item = hk::item_bytes(dtype);
    const int64_t scales = 4 * n_rows * (group ? (d + group - 1) / group : 1);
    ROWS_CHECK(hk::check_buffers({{codes, 0, 1, "codes"}, {scale, 0, 4, "scale"}, {X_out, 0, item, "X_out"}}));
    const int64_t x_bytes = ((n_rows - 1) * ldx + d) * item;
    if (hk::meet(X_out, x_bytes, codes, (n_rows - 1) * ldc + d))
        return rows_fail(HESS_ERR_INVALID, "X_out overlaps codes");
    if (hk::meet(X_out, x_bytes, scale, scales)) return rows_fail(HESS_ERR_INVALID, "X_out overlaps scale");
    const cudaError_t e = hk::rows8_restore_launch(codes, ldc, scale, n_rows, d, group, X_out, ldx, dtype,
                                                   static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rows_fail(HESS_ERR_CUDA, "rows8_restore: %s", cudaGetErrorString(e));
    return HESS_OK;
}
