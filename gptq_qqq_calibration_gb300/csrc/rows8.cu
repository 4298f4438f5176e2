// 8-bit rows: int8 codes with a scale per row or per group of columns
// (formulas and conventions: include/rows8.h).
//
// The unit of work is a segment: 256 columns of one row, eight per lane of a warp (512
// and sixteen where rows allow it).  A group of 32 .. 256 columns lies inside a segment,
// so its maximum is a few shuffles; a whole row is held by one CTA, in registers or, where
// there are many rows, in shared memory, and its maximum meets in shared memory, so
// that the values are read once either way.  A lane's columns come in runs of V side by
// side, 32 V columns apart: V is 16 or 8 where rows are multiples of 16 bytes, 4 or 2 where
// they are of less, else 1, which keeps a warp's accesses contiguous at any alignment.
//
// The whole number nearest to the exact quotient x / s is wanted, and the memory's pace
// leaves some ten instructions a value.  A multiply-add that adds 1.5 * 2^23 rounds a
// product to a whole number.  What it must not do is put a quotient near a half on the
// wrong side:
//   * 16-bit values.  With p significant bits in x and a, 127 x / a is a half itself or
//     1 / (254 * 2^p) >= 2^-19 of itself away from one.  So only halves matter, where x / s lies
//     above or below by the rounding of s = a / 127: the multiplier is taken 2^-21 above
//     or below 1/s, to the side of that rounding (a row whose s needs none and is no
//     power of two is divided value by value).
//   * 32-bit values.  One multiplier below 1/s and one above it: where both products round
//     alike that is the code, and where they do not (1 value in 10^5) the exact sign of
//     the remainder at the half between them decides.
//
// Bytes bound all of it (times in CUDA graphs): 16,384 x 11,008 bf16 take 92 us with a scale per
// 128 columns, 89 with one per row and 79 back (floor 80 at the copy rate of 6,781 GB/s),
// 32,768 x 4,096 fp32 101 and 98 us (floor 99).  Rows that are no multiples of 16 bytes cost more
// instructions: 16,383 x 8,191 bf16 96 us per 32 columns, 71 per row and 70 back (floor 59).
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "codes8.cuh"
#include "device_ptr.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "rows8.cuh"
#include "rows8.h"

namespace hk {
namespace {

constexpr int kSegment = 256;
// Values of a lane in a segment, and columns of a segment, for runs of V.
__host__ __device__ constexpr int lane_values(int v) { return v > 8 ? v : 8; }
__host__ __device__ constexpr int segment_columns(int v) { return 32 * lane_values(v); }
constexpr int kItemSegments = 4;  // segments one warp has in flight

template <class T>
__device__ __forceinline__ float2 pair_f32(uint32_t w);  // two 16-bit values
template <>
__device__ __forceinline__ float2 pair_f32<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 pair_f32<__half>(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}

// Column of a lane's element e within a segment.
template <int V>
__device__ __forceinline__ int column(int lane, int e) {
    return (e / V) * (32 * V) + lane * V + e % V;
}

// V elements of 16 or 32 bits from an address aligned to all of them (or, beyond 16
// bytes, to 16), as words.
template <int kBytes>
__device__ __forceinline__ void load_words(const void* p, uint32_t* w) {
    if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
            const uint4 v = __ldcs(static_cast<const uint4*>(p) + i);
            w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
        }
    } else if constexpr (kBytes == 8) {
        const uint2 v = __ldcs(static_cast<const uint2*>(p));
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = __ldcs(static_cast<const uint32_t*>(p));
    }
}

// A lane's values of a segment: words of two 16-bit values or of one of 32 bits; zeros
// past the row's end.
template <class T, int V>
struct Raw {
    static constexpr int kWords = lane_values(V) * sizeof(T) / 4;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T* row, int c0, int d, int lane) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
        for (int e = 0; e < lane_values(V); e += V) {
            const int c = c0 + column<V>(lane, e);
            if (c < d) {  // d is a multiple of V
                if constexpr (V > 1) {
                    load_words<V * sizeof(T)>(row + c, w + e * sizeof(T) / 4);
                } else if constexpr (sizeof(T) == 4) {
                    w[e] = __float_as_uint(__ldcs(reinterpret_cast<const float*>(row) + c));
                } else {
                    const uint32_t h = __ldcs(reinterpret_cast<const unsigned short*>(row) + c);
                    w[e / 2] |= e & 1 ? h << 16 : h;
                }
            }
        }
    }
    __device__ __forceinline__ float value(int e) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(w[e]);
        } else {
            const float2 f = pair_f32<T>(w[e / 2]);
            return e & 1 ? f.y : f.x;
        }
    }
    // The largest magnitude of the values of run r, as float32 bits.  Bits without the sign
    // are ordered like the values, infinity and NaN above all of them.
    __device__ __forceinline__ uint32_t top(int r) const {
        uint32_t t = 0;
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = r * V; e < r * V + V; ++e) t = max(t, w[e] & 0x7fffffffu);
        } else {
            if constexpr (V > 1) {
#pragma unroll
                for (int i = r * V / 2; i < (r + 1) * V / 2; ++i) asm("max.u16x2 %0, %1, %2;" : "=r"(t) : "r"(t), "r"(w[i] & 0x7fff7fffu));
                t = max(t >> 16, t & 0xffffu);
            } else {
                t = (r & 1 ? w[r / 2] >> 16 : w[r / 2]) & 0x7fffu;
            }
            t = __float_as_uint(pair_f32<T>(t).x);
        }
        return t;
    }
};

// The scale of a maximum, and what the values are multiplied by.
struct Scale {
    float s, lo, hi;  // 16-bit values: lo alone
    bool plain;       // codes by the multipliers; otherwise by `code_of`
};

template <class T>
__device__ __forceinline__ Scale scale_of(uint32_t top) {
    Scale k;
    const float t = __uint_as_float(top);
    // From 2^-100 on no step is subnormal, and t c, corrected by its remainder, is t / 127
    // correctly rounded: a quotient by a divisor known beforehand (Brisebarre, Muller and
    // Raina, 2004), for every significand (tests/test_gpu_rows8_scales.py).
    if (top - 0x0d800000u < 0x7f800000u - 0x0d800000u) {
        const float c = 1.0f / 127.0f;
        constexpr float kBelow = 1.0f - 1.0f / 2097152.0f, kAbove = 1.0f + 1.0f / 2097152.0f;
        const float q = __fmul_rn(t, c);
        k.s = __fmaf_rn(__fmaf_rn(-127.0f, q, t), c, q);
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(k.s));  // within 2^-23
        k.plain = true;
        if constexpr (sizeof(T) == 4) {
            k.lo = __fmul_rn(r, kBelow);  // within 2^-20 below 1/s,
            k.hi = __fmul_rn(r, kAbove);  // and above
        } else {
            const float left = __fmaf_rn(-127.0f, k.s, t);  // exact
            k.lo = __fmul_rn(r, left > 0.0f ? kAbove : kBelow);
            k.hi = 0.0f;
            if (left == 0.0f) {
                // s is t / 127 itself, and halves go to the even code: right where 1/s is exact
                k.lo = __uint_as_float(0x7f000000u - __float_as_uint(k.s));
                k.plain = (__float_as_uint(k.s) & 0x7fffffu) == 0;
            }
        }
        return k;
    }
    k.s = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __fdiv_rn(t, 127.0f);
    k.lo = k.hi = 0.0f;
    k.plain = top == 0;
    return k;
}

// rint(x / s) of the exact quotient, by a division.
__device__ __forceinline__ int code_of(float x, float s) {
    if (!(s > 0.0f)) return 0;  // 0 or NaN
    if (s < kLiftBelow) {
        s = __fmul_rn(s, kLift);
        x = __fmul_rn(x, kLift);
    }
    return nearest_code(fminf(fmaxf(__fdiv_rn(x, s), -127.0f), 127.0f), x, s);
}

__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number

// The code of x where its two products round to a and z, neighbours (as bits of kMagic + q).
__device__ __forceinline__ uint32_t between(float x, float s, uint32_t a, uint32_t z) {
    const float fa = __fsub_rn(__uint_as_float(a), kMagic), fz = __fsub_rn(__uint_as_float(z), kMagic);
    const float e = __fmaf_rn(-0.5f * __fadd_rn(fa, fz), s, x);  // exact in sign
    if (e == 0.0f) return a & 1 ? z : a;
    return e > 0.0f ? max(a, z) : min(a, z);
}

// The codes of run r, in order, as bytes of `out` (V / 4 words, or one for V = 1).
template <class T, int V>
__device__ __forceinline__ void encode(const Raw<T, V>& raw, int r, const Scale& k, uint32_t* out) {
    uint32_t a[V];
    if constexpr (V > 1) {
        const uint64_t lo = pack2(__float_as_uint(k.lo), __float_as_uint(k.lo));
        const uint64_t hi = pack2(__float_as_uint(k.hi), __float_as_uint(k.hi));
        const uint64_t m = pack2(__float_as_uint(kMagic), __float_as_uint(kMagic));
        uint32_t z[V], differ = 0;
#pragma unroll
        for (int e = 0; e < V; e += 2) {  // two multiply-adds at a time
            const uint64_t x = pack2(__float_as_uint(raw.value(r * V + e)), __float_as_uint(raw.value(r * V + e + 1)));
            uint64_t y;
            asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(x), "l"(lo), "l"(m));
            a[e] = static_cast<uint32_t>(y), a[e + 1] = static_cast<uint32_t>(y >> 32);
            if constexpr (sizeof(T) == 4) {
                asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(x), "l"(hi), "l"(m));
                z[e] = static_cast<uint32_t>(y), z[e + 1] = static_cast<uint32_t>(y >> 32);
                differ |= (a[e] ^ z[e]) | (a[e + 1] ^ z[e + 1]);
            }
        }
        if constexpr (sizeof(T) == 4) {
            if (differ != 0) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (a[e] != z[e]) a[e] = between(raw.value(r * V + e), k.s, a[e], z[e]);
            }
        }
    } else {
        const float x = raw.value(r);
        a[0] = __float_as_uint(__fmaf_rn(x, k.lo, kMagic));
        if constexpr (sizeof(T) == 4) {
            const uint32_t z = __float_as_uint(__fmaf_rn(x, k.hi, kMagic));
            if (a[0] != z) a[0] = between(x, k.s, a[0], z);
        }
    }
    if (!k.plain) {
#pragma unroll
        for (int e = 0; e < V; ++e) a[e] = static_cast<uint32_t>(code_of(raw.value(r * V + e), k.s));
    }
    if constexpr (V == 1) {
        out[0] = a[0];
    } else if constexpr (V == 2) {
        out[0] = __byte_perm(a[0], a[1], 0x0040);
    } else {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) out[i] = pack_bytes(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
    }
}

// The codes of one run at column c, as bytes or as float16 whole numbers (those in runs of
// eight or sixteen only).
template <int V>
__device__ __forceinline__ void store(int8_t* codes, __half* wide, int c, const uint32_t* q) {
    if constexpr (V == 1) {
        codes[c] = static_cast<int8_t>(q[0]);
    } else if constexpr (V == 2) {
        *reinterpret_cast<unsigned short*>(codes + c) = static_cast<unsigned short>(q[0]);
    } else if constexpr (V == 4) {
        *reinterpret_cast<uint32_t*>(codes + c) = q[0];
    } else if (codes) {
        if constexpr (V == 16) *reinterpret_cast<uint4*>(codes + c) = make_uint4(q[0], q[1], q[2], q[3]);
        else *reinterpret_cast<uint2*>(codes + c) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 8; ++i) {
            uint4 w;
            widen4(q[2 * i], w.x, w.y);
            widen4(q[2 * i + 1], w.z, w.w);
            reinterpret_cast<uint4*>(wide + c)[i] = w;
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
    int64_t ldx, n, ldc, ldw;
    int32_t d;
    int32_t group;    // group kernels: 32 .. 256, or 256 for whole rows of at most 256 columns
    int32_t shift;    // its logarithm
    int64_t groups;   // scales of a row
    int32_t items;    // group kernel: segments of a row
    int32_t held;     // row kernel: columns that a pass of the CTA covers
    int8_t* codes;
    __half* wide;
    float* scale;
};

// Scales per group.  Warps walk the segments of all rows, with the next one on its way
// from memory under the one at work.
template <class T, int V, int kGroup>
__device__ __forceinline__ void encode_segment(const QuantizeParams& p, const Raw<T, V>& raw, int64_t r, int c0, int lane) {
    static_assert(V >= 8 && kGroup >= 32 && kGroup <= 32 * V, "a lane's run is all it has, and lies in one group");
    uint32_t top = raw.top(0);
#pragma unroll
    for (int o = kGroup / V / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
    int8_t* const codes = p.codes ? p.codes + r * p.ldc : nullptr;
    __half* const wide = p.codes ? nullptr : p.wide + r * p.ldw;
    const Scale s = scale_of<T>(top);
    const int c = c0 + lane * V;
    if (c < p.d) {
        if ((c & (kGroup - 1)) == 0) p.scale[r * p.groups + (c >> p.shift)] = s.s;
        uint32_t q[V / 4];
        encode<T, V>(raw, 0, s, q);
        store<V>(codes, wide, c, q);
    }
}

// Segment `index` of all rows, walked by `step` segments at a time.
struct Walk {
    int64_t r;
    int32_t c;  // segment of the row
    __device__ __forceinline__ Walk(int64_t index, int32_t segments) {
        r = row_of(index, segments);
        c = static_cast<int32_t>(index - r * segments);
    }
    __device__ __forceinline__ void add(const Walk& step, int32_t segments) {
        r += step.r;
        c += step.c;
        if (c >= segments) {
            c -= segments;
            ++r;
        }
    }
};

constexpr int kGroupWarps = 8, kGroupCtas = 4;

template <class T, int V, int kGroup>
__global__ void __launch_bounds__(kGroupWarps * 32, kGroupCtas)
    rows8_group_kernel(const __grid_constant__ QuantizeParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * kGroupWarps + (threadIdx.x >> 5);
    const Walk step(static_cast<int64_t>(gridDim.x) * kGroupWarps, p.items);
    Walk at(warp, p.items);
    const auto fetch = [&](Raw<T, V>& raw, const Walk& w) {
        if (w.r < p.n) raw.load(static_cast<const T*>(p.x) + w.r * p.ldx, w.c * segment_columns(V), p.d, lane);
    };
    Walk next = at;
    Raw<T, V> a, b;
    fetch(a, at);
    // two segments a turn, each fetched while the other is at work
#pragma unroll 1
    while (at.r < p.n) {
        next.add(step, p.items);
        fetch(b, next);
        encode_segment<T, V, kGroup>(p, a, at.r, at.c * segment_columns(V), lane);
        at = next;
        if (at.r >= p.n) return;
        next.add(step, p.items);
        fetch(a, next);
        encode_segment<T, V, kGroup>(p, b, at.r, at.c * segment_columns(V), lane);
        at = next;
    }
}

// The same for rows that are no multiples of 16 bytes.  Loads and stores keep a warp's
// accesses side by side, in runs of V values; in between the values change lanes through
// shared memory, so that a lane has sixteen neighbours and with them one scale.  (With a
// scale for every run: 301 us against 97 for 16,383 x 8,191 bf16 in groups of 32.)
template <class T, int V>
__global__ void __launch_bounds__(kGroupWarps * 32, 3) rows8_odd_kernel(const __grid_constant__ QuantizeParams p) {
    constexpr int kSeg = 512;
    __shared__ __align__(16) T values[kGroupWarps][kSeg];
    __shared__ __align__(16) int8_t results[kGroupWarps][kSeg];
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    T* const mine = values[w];
    int8_t* const out = results[w];
    const Walk step(static_cast<int64_t>(gridDim.x) * kGroupWarps, p.items);
    const auto fetch = [&](uint32_t (&to)[16 / V][V * sizeof(T) < 4 ? 1 : V * sizeof(T) / 4], const Walk& at) {
        const T* const row = static_cast<const T*>(p.x) + at.r * p.ldx;
#pragma unroll
        for (int i = 0; i < 16 / V; ++i) {
            const int c = at.c * kSeg + i * (32 * V) + lane * V;
            const bool in = at.r < p.n && c < p.d;
            if constexpr (V * sizeof(T) >= 4) {
                if (in) load_words<V * sizeof(T)>(row + c, to[i]);
                else
#pragma unroll
                    for (int k = 0; k < static_cast<int>(V * sizeof(T) / 4); ++k) to[i][k] = 0;
            } else {
                to[i][0] = in ? __ldcs(reinterpret_cast<const unsigned short*>(row) + c) : 0u;
            }
        }
    };
    Walk at(static_cast<int64_t>(blockIdx.x) * kGroupWarps + w, p.items);
    uint32_t held[16 / V][V * sizeof(T) < 4 ? 1 : V * sizeof(T) / 4];
    fetch(held, at);
#pragma unroll 1
    while (at.r < p.n) {
#pragma unroll
        for (int i = 0; i < 16 / V; ++i) {
            T* const to = mine + i * (32 * V) + lane * V;
            if constexpr (V * sizeof(T) < 4) {
                *reinterpret_cast<unsigned short*>(to) = static_cast<unsigned short>(held[i][0]);
            } else {
#pragma unroll
                for (int k = 0; k < static_cast<int>(V * sizeof(T) / 4); ++k) reinterpret_cast<uint32_t*>(to)[k] = held[i][k];
            }
        }
        const Walk here = at;
        at.add(step, p.items);
        fetch(held, at);
        __syncwarp();
        Raw<T, 16> raw;
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(T)); ++k) {
            const uint4 v = reinterpret_cast<const uint4*>(mine + lane * 16)[k];
            raw.w[4 * k] = v.x, raw.w[4 * k + 1] = v.y, raw.w[4 * k + 2] = v.z, raw.w[4 * k + 3] = v.w;
        }
        uint32_t top = raw.top(0);
        for (int o = p.group >> 5; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
        const Scale s = scale_of<T>(top);
        const int c = here.c * kSeg + lane * 16;
        if (c < p.d && (c & (p.group - 1)) == 0) p.scale[here.r * p.groups + (c >> p.shift)] = s.s;
        uint32_t q[4];
        encode<T, 16>(raw, 0, s, q);
        *reinterpret_cast<uint4*>(out + lane * 16) = make_uint4(q[0], q[1], q[2], q[3]);
        __syncwarp();
        int8_t* const codes = p.codes + here.r * p.ldc;
#pragma unroll
        for (int i = 0; i < 16 / V; ++i) {
            const int from = i * (32 * V) + lane * V, to = here.c * kSeg + from;
            if (to < p.d) {
                if constexpr (V == 1) codes[to] = out[from];
                else if constexpr (V == 2) *reinterpret_cast<unsigned short*>(codes + to) = *reinterpret_cast<const unsigned short*>(out + from);
                else *reinterpret_cast<uint32_t*>(codes + to) = *reinterpret_cast<const uint32_t*>(out + from);
            }
        }
        __syncwarp();
    }
}

// One scale per row: a CTA takes one row, kHeld segments per warp in registers.
// Rows longer than that are read twice (the second time mostly from L2).  Two large
// CTAs per SM, so that one loads while the other works.
constexpr int kRowWarps = 24;
template <class T, int V, int kHeld>
__global__ void __launch_bounds__(kRowWarps * 32, 2) rows8_row_kernel(const __grid_constant__ QuantizeParams p) {
    constexpr int kRuns = 8 / V;
    griddep_wait();
    griddep_launch_dependents();
    __shared__ uint32_t tops[kRowWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r = blockIdx.x;
    const T* const row = static_cast<const T*>(p.x) + r * p.ldx;
    int8_t* const codes = p.codes ? p.codes + r * p.ldc : nullptr;
    __half* const wide = p.codes ? nullptr : p.wide + r * p.ldw;
    Raw<T, V> raw[kHeld];
    uint32_t top = 0;
    for (int c00 = warp * (kHeld * kSegment); c00 < p.d; c00 += p.held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) raw[i].load(row, c00 + i * kSegment, p.d, lane);
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
#pragma unroll
            for (int k = 0; k < kRuns; ++k) top = max(top, raw[i].top(k));
    }
    top = __reduce_max_sync(~0u, top);
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = lane < static_cast<int>(blockDim.x >> 5) ? tops[lane] : 0u;
    top = __reduce_max_sync(~0u, top);
    const Scale s = scale_of<T>(top);
    if (threadIdx.x == 0) p.scale[r] = s.s;
    for (int c00 = warp * (kHeld * kSegment); c00 < p.d; c00 += p.held) {
        if (p.held < p.d) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i) raw[i].load(row, c00 + i * kSegment, p.d, lane);
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
#pragma unroll
            for (int k = 0; k < kRuns; ++k) {
                const int c = c00 + i * kSegment + column<V>(lane, k * V);
                if (c < p.d) {
                    uint32_t q[V > 4 ? 2 : 1];
                    encode<T, V>(raw[i], k, s, q);
                    store<V>(codes, wide, c, q);
                }
            }
    }
}

// One scale per row, rows of at most kShort segments: a warp holds one.
constexpr int kShort = 4;

template <class T, int V>
__global__ void __launch_bounds__(kGroupWarps * 32, 3) rows8_short_kernel(const __grid_constant__ QuantizeParams p) {
    constexpr int kRuns = lane_values(V) / V;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGroupWarps;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * kGroupWarps + (threadIdx.x >> 5); r < p.n; r += step) {
        const T* const row = static_cast<const T*>(p.x) + r * p.ldx;
        Raw<T, V> raw[kShort];
#pragma unroll
        for (int i = 0; i < kShort; ++i) raw[i].load(row, i * segment_columns(V), p.d, lane);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kShort; ++i)
#pragma unroll
            for (int k = 0; k < kRuns; ++k) top = max(top, raw[i].top(k));
        const Scale s = scale_of<T>(__reduce_max_sync(~0u, top));
        if (lane == 0) p.scale[r] = s.s;
        int8_t* const codes = p.codes ? p.codes + r * p.ldc : nullptr;
        __half* const wide = p.codes ? nullptr : p.wide + r * p.ldw;
#pragma unroll
        for (int i = 0; i < kShort; ++i)
#pragma unroll
            for (int k = 0; k < kRuns; ++k) {
                const int c = i * segment_columns(V) + column<V>(lane, k * V);
                if (c < p.d) {
                    uint32_t q[V > 4 ? V / 4 : 1];
                    encode<T, V>(raw[i], k, s, q);
                    store<V>(codes, wide, c, q);
                }
            }
    }
}

// One scale per row, many rows of 16-bit values: a CTA walks rows, with the next one on
// its way into shared memory under the one at work.  A thread copies, and later reads,
// the same granules of eight values, so only the maxima have to meet.  (Rows in
// registers cost every warp its start and its scale for two segments of a row: 124 us
// against 90 for 16,384 x 11,008 bf16.)
// kAny: rows without gaps that start anywhere.  Granules are the matrix's, so that those of
// values and those of codes fall together; a row's first and last one it shares with its
// neighbours.  (16,383 x 8,191 bf16: 74 us; in runs that the rows' starts allow 127.)
constexpr int kStreamThreads = 128;

template <class T, bool kAny>
__global__ void __launch_bounds__(kStreamThreads) rows8_stream_kernel(const __grid_constant__ QuantizeParams p) {
    extern __shared__ uint4 buffers[];  // two rows
    __shared__ uint32_t tops[2][kStreamThreads / 32];
    const int held = kAny ? (p.d >> 3) + 2 : p.d >> 3;  // granules of a buffer
    const auto before = [&](int64_t r) { return kAny ? static_cast<int>((r * p.d) & 7) : 0; };
    const auto granules_of = [&](int64_t r) { return kAny ? (before(r) + p.d + 7) >> 3 : p.d >> 3; };
    griddep_wait();
    griddep_launch_dependents();
    const auto fetch = [&](int64_t r, int b) {
        if (r < p.n) {
            const int granules = granules_of(r);
            const int64_t start = kAny ? r * p.d - before(r) : r * p.ldx;
            const uint4* const src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + start);
            const uint32_t dst = smem_u32(buffers + b * held);
            for (int g = threadIdx.x; g < granules; g += kStreamThreads) {
                if constexpr (kAny) {  // nothing behind the matrix is read
                    const int64_t left = p.n * p.d - start - 8 * static_cast<int64_t>(g);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * g), "l"(src + g),
                                 "r"(left < 8 ? static_cast<uint32_t>(2 * left) : 16u)
                                 : "memory");
                } else {
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + 16 * g), "l"(src + g) : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(blockIdx.x, 0);
    int b = 0;
#pragma unroll 1
    for (int64_t r = blockIdx.x; r < p.n; r += gridDim.x, b ^= 1) {
        fetch(r + gridDim.x, b ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        const uint4* const row = buffers + b * held;
        const int granules = granules_of(r), first = before(r), last = first + p.d;
        Raw<T, 8> raw;
        uint32_t top = 0;
#pragma unroll 4
        for (int g = threadIdx.x; g < granules; g += kStreamThreads) {
            const uint4 v = row[g];
            raw.w[0] = v.x, raw.w[1] = v.y, raw.w[2] = v.z, raw.w[3] = v.w;
            if (kAny && (g == 0 || g == granules - 1)) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (8 * g + k < first || 8 * g + k >= last) raw.w[k / 2] &= k & 1 ? 0x0000ffffu : 0xffff0000u;
            }
            top = max(top, raw.top(0));
        }
        top = __reduce_max_sync(~0u, top);
        if ((threadIdx.x & 31) == 0) tops[b][threadIdx.x >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kStreamThreads / 32; ++i) top = max(top, tops[b][i]);
        const Scale s = scale_of<T>(top);
        if (threadIdx.x == 0) p.scale[r] = s.s;
        int8_t* const codes = kAny ? p.codes + (r * p.d - first) : p.codes ? p.codes + r * p.ldc : nullptr;
        __half* const wide = p.codes ? nullptr : p.wide + r * p.ldw;
#pragma unroll 2
        for (int g = threadIdx.x; g < granules; g += kStreamThreads) {
            const uint4 v = row[g];
            raw.w[0] = v.x, raw.w[1] = v.y, raw.w[2] = v.z, raw.w[3] = v.w;
            uint32_t q[2];
            encode<T, 8>(raw, 0, s, q);
            if (kAny && (g == 0 || g == granules - 1)) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (8 * g + k >= first && 8 * g + k < last)
                        codes[8 * g + k] = static_cast<int8_t>(q[k / 4] >> (8 * (k % 4)));
            } else {
                store<8>(codes, wide, 8 * g, q);
            }
        }
    }
}

struct RestoreJob {
    const int8_t* codes;
    const float* scale;  // NULL: 1
    int64_t ldc, n, ldx;
    int32_t d;
    int32_t shift;   // log2(group); whole rows: 31
    int64_t groups;  // scales of a row
    int32_t items;   // items of kItemSegments segments in a row
    void* x;
};
struct RestoreParams {
    RestoreJob job[2];
    int64_t first;   // blocks of the first job
    int32_t early;   // the next kernel may start before this one's inputs are there
};

// A byte as a float: 2^23 + (q + 128) has the byte q ^ 0x80 at its low end.
__device__ __forceinline__ float byte_to_f32(uint32_t biased, uint32_t which) {
    return __fsub_rn(__uint_as_float(__byte_perm(biased, 0x4b000000u, 0x7440 + which)), 8388736.0f);
}

template <class T>
__device__ __forceinline__ uint32_t two_of(float a, float b);  // as 16-bit values
template <>
__device__ __forceinline__ uint32_t two_of<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
template <>
__device__ __forceinline__ uint32_t two_of<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}

// V values of one run at `out`.
template <class T, int V>
__device__ __forceinline__ void put(T* out, const float (&x)[V]) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 1) {
            *reinterpret_cast<float*>(out) = x[0];
        } else if constexpr (V == 2) {
            *reinterpret_cast<float2*>(out) = make_float2(x[0], x[1]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + i) =
                    make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        }
    } else if constexpr (V == 1) {
        *reinterpret_cast<unsigned short*>(out) = static_cast<unsigned short>(two_of<T>(x[0], 0.0f));
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = two_of<T>(x[2 * i], x[2 * i + 1]);
        if constexpr (V == 2) *reinterpret_cast<uint32_t*>(out) = w[0];
        else if constexpr (V == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <class T, int V>
__global__ void __launch_bounds__(256) rows8_restore_kernel(const __grid_constant__ RestoreParams all) {
    constexpr int kRuns = 8 / V;
    if (all.early) griddep_launch_dependents();
    griddep_wait();
    if (!all.early) griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const bool second = blockIdx.x >= all.first;
    const RestoreJob p = second ? all.job[1] : all.job[0];
    const int64_t block = second ? blockIdx.x - all.first : blockIdx.x;
    const int64_t item = block * 8 + (threadIdx.x >> 5);
    const int64_t r = row_of(item, p.items);
    if (r >= p.n) return;
    const int c00 = static_cast<int>(item - r * p.items) * (kItemSegments * kSegment);
    const int8_t* const codes = p.codes + r * p.ldc;
    const float* const scale = p.scale ? p.scale + r * p.groups : nullptr;
    T* const out = static_cast<T*>(p.x) + r * p.ldx;
    uint32_t w[kItemSegments][kRuns][V > 4 ? 2 : 1];
    float s[kItemSegments][kRuns];
#pragma unroll
    for (int i = 0; i < kItemSegments; ++i)
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
            const int c = c00 + i * kSegment + column<V>(lane, k * V);
            const bool in = c < p.d;
            if constexpr (V == 8) {
                const uint2 v = in ? __ldcs(reinterpret_cast<const uint2*>(codes + c)) : make_uint2(0, 0);
                w[i][k][0] = v.x, w[i][k][1] = v.y;
            } else if constexpr (V == 4) {
                w[i][k][0] = in ? __ldcs(reinterpret_cast<const uint32_t*>(codes + c)) : 0u;
            } else if constexpr (V == 2) {
                w[i][k][0] = in ? __ldcs(reinterpret_cast<const unsigned short*>(codes + c)) : 0u;
            } else {
                w[i][k][0] = in ? __ldcs(reinterpret_cast<const unsigned char*>(codes + c)) : 0u;
            }
            s[i][k] = in && scale ? scale[c >> p.shift] : 1.0f;
        }
#pragma unroll
    for (int i = 0; i < kItemSegments; ++i)
#pragma unroll
        for (int k = 0; k < kRuns; ++k) {
            const int c = c00 + i * kSegment + column<V>(lane, k * V);
            if (c < p.d) {
                float x[V];
#pragma unroll
                for (int e = 0; e < V; ++e)
                    x[e] = __fmul_rn(byte_to_f32(w[i][k][e / 4] ^ 0x80808080u, e % 4), s[i][k]);
                put<T, V>(out + c, x);
            }
        }
}

// Rows without gaps that are short or start anywhere: the matrix as one run of values, eight a
// lane, which rows' and groups' ends may cut.  16,383 x 8,191 bf16 take 70 us, 131,072 x 200
// f16 16 (rows one by one, in runs that their starts allow: 151 and 28; where those are four
// values that is the faster way: 16,384 x 8,188 f16 67 us against 71 here).
struct FlatParams {
    const int8_t* codes;
    const float* scale;
    void* x;
    int64_t total, groups;
    int32_t d, shift;
};

template <class T>
__global__ void __launch_bounds__(256) rows8_restore_flat_kernel(const __grid_constant__ FlatParams p) {
    constexpr int kEach = 4;  // runs of a thread
    griddep_wait();
    griddep_launch_dependents();
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (256 * kEach) + threadIdx.x) * 8;
    T* const out = static_cast<T*>(p.x);
    uint2 w[kEach];
    float s0[kEach], s1[kEach];
    int cut[kEach];
    bool plain[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t e = first + i * (256 * 8);
        plain[i] = e + 8 <= p.total;
        if (!plain[i]) continue;
        w[i] = __ldcs(reinterpret_cast<const uint2*>(p.codes + e));
        const int64_t r = row_of(e, p.d);
        const int c = static_cast<int>(e - r * p.d);
        const float* const at = p.scale + r * p.groups + (c >> p.shift);
        // the columns of this scale and of the next one, which is the next in memory
        const auto span = [&](int from) {
            const uint32_t end = (static_cast<uint32_t>(from) | ((1u << p.shift) - 1u)) + 1u;
            return static_cast<int>(end < static_cast<uint32_t>(p.d) ? end : p.d) - from;
        };
        cut[i] = span(c);
        s0[i] = *at;
        s1[i] = cut[i] < 8 ? at[1] : 0.0f;
        if (cut[i] < 8) plain[i] = cut[i] + span(c + cut[i] < p.d ? c + cut[i] : 0) >= 8;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t e = first + i * (256 * 8);
        if (plain[i]) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = __fmul_rn(byte_to_f32((k < 4 ? w[i].x : w[i].y) ^ 0x80808080u, k % 4), k < cut[i] ? s0[i] : s1[i]);
            put<T, 8>(out + e, x);
        } else {  // the last values, or a third scale
            for (int64_t k = e; k < e + 8 && k < p.total; ++k) {
                const int64_t r = row_of(k, p.d);
                const float x[1] = {__fmul_rn(static_cast<float>(p.codes[k]),
                                              p.scale[r * p.groups + (static_cast<int>(k - r * p.d) >> p.shift)])};
                put<T, 1>(out + k, x);
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
cudaError_t rows_launch(Kernel kernel, const Params& p, int64_t grid, int threads, cudaStream_t s, size_t smem = 0) {
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
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

bool aligned(const void* p, int64_t stride_bytes, int to) {
    return reinterpret_cast<uintptr_t>(p) % to == 0 && stride_bytes % to == 0;
}

constexpr int kStreamSmem = 100 * 1024;  // two rows of at most 25,600 values

// The current device's SMs, after its first call also with the stream kernels' shared memory.
cudaError_t prepare(int* sms) {
    static std::mutex mu;
    static int count[128] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    if (!count[dev]) {
        for (auto fn : {rows8_stream_kernel<__nv_bfloat16, false>, rows8_stream_kernel<__half, false>,
                        rows8_stream_kernel<__nv_bfloat16, true>, rows8_stream_kernel<__half, true>})
            if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem)) != cudaSuccess)
                return e;
        if ((e = cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    }
    *sms = count[dev];
    return cudaSuccess;
}

template <class Kernel>
cudaError_t launch_walk(Kernel kernel, const QuantizeParams& p, int ctas_per_sm, cudaStream_t s) {
    int sms = 0;
    const cudaError_t e = prepare(&sms);
    if (e != cudaSuccess) return e;
    const int64_t all = (p.n * p.items + kGroupWarps - 1) / kGroupWarps;
    const int64_t fit = static_cast<int64_t>(sms) * ctas_per_sm;
    return rows_launch(kernel, p, all < fit ? all : fit, kGroupWarps * 32, s);
}

template <class Kernel>
cudaError_t launch_stream(Kernel kernel, const QuantizeParams& p, size_t smem, cudaStream_t s) {
    int sms = 0, per_sm = 0;
    cudaError_t e = prepare(&sms);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kStreamThreads, smem);
    if (e != cudaSuccess) return e;
    const int64_t fit = static_cast<int64_t>(sms) * (per_sm < 1 ? 1 : per_sm);
    return rows_launch(kernel, p, p.n < fit ? p.n : fit, kStreamThreads, s, smem);
}

// A scale for every row of more than 256 values.  Few rows are spread over more warps
// each, so that a row takes one round trip to memory and little work after it; many go one
// to a warp, or through shared memory.  The border of 512 rows lies between those of narrow
// rows and of wide 16-bit ones (few / many, us): 1,024 fp32 columns 1.68 / 1.90 at 512 rows, 2.68 / 2.15
// at 1,024; 4,096 bf16 1.46 / 1.59 at 64, 2.21 / 1.74 at 256, 5.39 / 3.85 at 1,024; 16,384 bf16 4.15 / 4.34
// at 256, 6.11 / 6.24 at 512, 17.4 / 16.5 at 2,048; 4,100 bf16 1.83 / 2.29 at 256, 6.31 / 4.36 at 1,024.
template <class T, int V>
cudaError_t quantize_rows(QuantizeParams& p, cudaStream_t s) {
    if (p.d <= kShort * kSegment && p.n > 512) {
        int sms = 0;
        const cudaError_t e = prepare(&sms);
        if (e != cudaSuccess) return e;
        const int64_t all = (p.n + kGroupWarps - 1) / kGroupWarps, fit = static_cast<int64_t>(sms) * 6;
        return rows_launch(rows8_short_kernel<T, V>, p, all < fit ? all : fit, kGroupWarps * 32, s);
    }
    if constexpr (V == 8 && sizeof(T) == 2) {
        if (p.n > 512 && 4 * static_cast<size_t>(p.d) <= kStreamSmem)
            return launch_stream(rows8_stream_kernel<T, false>, p, 4 * static_cast<size_t>(p.d), s);
    }
    const int segments = (p.d + kSegment - 1) / kSegment;
    const int h = p.n <= 512 && segments <= kRowWarps ? 1 : segments <= 2 * kRowWarps || sizeof(T) == 4 ? 2 : 4;
    int warps = (segments + h - 1) / h;
    if (warps > kRowWarps) warps = kRowWarps;
    p.held = warps * h * kSegment;
    if (h == 1) return rows_launch(rows8_row_kernel<T, V, 1>, p, p.n, warps * 32, s);
    if constexpr (sizeof(T) == 2) {
        if (h == 4) return rows_launch(rows8_row_kernel<T, V, 4>, p, p.n, warps * 32, s);
    }
    return rows_launch(rows8_row_kernel<T, V, 2>, p, p.n, warps * 32, s);
}

template <class T, int V>
cudaError_t quantize_as(QuantizeParams& p, cudaStream_t s) {
    if (p.group != 0 || p.d <= kSegment) {
        if (p.group == 0) p.group = kSegment;
        p.shift = log2_of(p.group);
        if constexpr (V >= 8) {
            p.items = (p.d + segment_columns(V) - 1) / segment_columns(V);
            return launch_walk(p.group == 32    ? rows8_group_kernel<T, V, 32>
                               : p.group == 64  ? rows8_group_kernel<T, V, 64>
                               : p.group == 128 ? rows8_group_kernel<T, V, 128>
                                                : rows8_group_kernel<T, V, 256>,
                               p, kGroupCtas, s);
        } else {
            p.items = (p.d + 511) / 512;
            return launch_walk(rows8_odd_kernel<T, V>, p, 6, s);
        }
    }
    if constexpr (V == 16) {
        return quantize_as<T, 8>(p, s);
    } else {
        return quantize_rows<T, V>(p, s);
    }
}

// The widest run that rows of both matrices allow, and, with `spread`, that gives every lane one.
int run_of(int most, bool spread, int32_t d, const void* x, int64_t x_row, int x_item, const void* q, int64_t q_row, int q_item) {
    for (int v : {16, 8, 4, 2})
        if (v <= most && (v <= 4 || !spread || 32 * v <= d) && d % v == 0 && aligned(x, x_row * x_item, v * x_item < 16 ? v * x_item : 16) &&
            aligned(q, q_row * q_item, v * q_item < 16 ? v * q_item : 16))
            return v;
    return 1;
}

template <class T>
cudaError_t quantize_of(QuantizeParams& p, cudaStream_t s) {
    const int most = sizeof(T) == 2 ? 16 : 8;
    const int v = p.codes ? run_of(most, true, p.d, p.x, p.ldx, sizeof(T), p.codes, p.ldc, 1)
                          : run_of(most, false, p.d, p.x, p.ldx, sizeof(T), p.wide, p.ldw, 2);
    if (!p.codes && v < 8) return cudaErrorInvalidValue;  // float16 codes leave in runs of at least eight
    if constexpr (sizeof(T) == 2) {
        if (v == 16) return quantize_as<T, 16>(p, s);
        const size_t smem = 2 * 16 * static_cast<size_t>((p.d >> 3) + 2);
        if (v < 8 && p.group == 0 && p.codes && p.ldx == p.d && p.ldc == p.d && p.d > kShort * kSegment && p.n > 512 &&
            smem <= kStreamSmem && aligned(p.x, 0, 16) && aligned(p.codes, 0, 8))
            return launch_stream(rows8_stream_kernel<T, true>, p, smem, s);
    }
    return v == 8   ? quantize_as<T, 8>(p, s)
           : v == 4 ? quantize_as<T, 4>(p, s)
           : v == 2 ? quantize_as<T, 2>(p, s)
                    : quantize_as<T, 1>(p, s);
}

template <class T>
cudaError_t restore_of(RestoreParams& p, cudaStream_t s) {
    // 16 bytes of output a lane
    int v = sizeof(T) == 2 ? 8 : 4;
    const RestoreJob& only = p.job[0];
    if (only.n > 0 && p.job[1].n == 0 && only.scale && only.ldx == only.d && only.ldc == only.d && only.d >= 16 &&
        aligned(only.x, 0, 16) && aligned(only.codes, 0, 8) &&
        (only.d < 2 * kSegment ||
         run_of(v, true, only.d, only.x, only.ldx, sizeof(T), only.codes, only.ldc, 1) < (sizeof(T) == 2 ? 4 : 2))) {
        const FlatParams f{only.codes, only.scale, only.x, only.n * only.d, only.groups, only.d, only.shift};
        return rows_launch(rows8_restore_flat_kernel<T>, f, (f.total + 256 * 4 * 8 - 1) / (256 * 4 * 8), 256, s);
    }
    int64_t blocks = 0;
    for (RestoreJob& j : p.job) {
        if (j.n == 0) continue;
        v = run_of(v, true, j.d, j.x, j.ldx, sizeof(T), j.codes, j.ldc, 1);
        blocks += (j.n * j.items + 7) / 8;
    }
    p.first = (p.job[0].n * p.job[0].items + 7) / 8;
    if (blocks == 0) return cudaSuccess;
    if constexpr (sizeof(T) == 4)
        return rows_launch(v == 4   ? rows8_restore_kernel<T, 4>
                           : v == 2 ? rows8_restore_kernel<T, 2>
                                    : rows8_restore_kernel<T, 1>,
                           p, blocks, 256, s);
    return rows_launch(v == 8   ? rows8_restore_kernel<T, 8>
                       : v == 4 ? rows8_restore_kernel<T, 4>
                       : v == 2 ? rows8_restore_kernel<T, 2>
                                : rows8_restore_kernel<T, 1>,
                       p, blocks, 256, s);
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

// Rows that follow each other without a gap, and whose groups end with the row, are as well
// fewer and longer rows: n, d and group become those, and no lane is left without values at a
// row's end (131,072 x 128 bf16 with a scale per row: 9.6 us and 9.0 back; one by one 41 and 26).
// Above 2^30 values they are joined by powers of two, which an odd number of rows does not allow.
static void join_rows(int64_t& n, int64_t& d, int32_t& group, int64_t& ldx, int64_t& ldc) {
    constexpr int64_t kMost = int64_t(1) << 30;  // columns are counted in 32 bits
    const int32_t whole = group ? group : d >= 32 && d <= 256 && (d & (d - 1)) == 0 ? static_cast<int32_t>(d) : 0;
    if (n < 2 || ldx != d || ldc != d || whole == 0 || d % whole) return;
    int64_t k = n;
    if (n * d > kMost)
        for (k = 1; n % (2 * k) == 0 && 2 * k * d <= kMost;) k *= 2;
    if (k == 1) return;
    n /= k;
    d *= k;
    ldx = ldc = d;
    group = whole;
}

cudaError_t rows8_quantize_launch(const void* X, int64_t ldx, int64_t n, int64_t d, int32_t dtype, int32_t group,
                                  int8_t* codes, int64_t ldc, uint16_t* wide, int64_t ldw, float* scale,
                                  cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    if (codes) join_rows(n, d, group, ldx, ldc);
    QuantizeParams p{};
    p.x = X;
    p.ldx = ldx;
    p.n = n;
    p.d = static_cast<int32_t>(d);
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

cudaError_t rows8_restore_launch(const RestoreRows& a, const RestoreRows& b, int32_t dtype, bool early, cudaStream_t s) {
    RestoreParams p{};
    const RestoreRows* const rows[2] = {&a, &b};
    for (int i = 0; i < 2; ++i) {
        RestoreRows r = *rows[i];
        RestoreJob& j = p.job[i];
        j.n = r.n;
        if (r.n == 0) continue;
        join_rows(r.n, r.d, r.group, r.ldx, r.ldc);
        j.n = r.n;
        j.codes = r.codes;
        j.scale = r.scale;
        j.ldc = r.ldc;
        j.d = static_cast<int32_t>(r.d);
        j.ldx = r.ldx;
        j.shift = r.group ? log2_of(r.group) : 31;
        j.groups = r.group ? (r.d + r.group - 1) / r.group : 1;
        j.items = static_cast<int32_t>((r.d + kItemSegments * kSegment - 1) / (kItemSegments * kSegment));
        j.x = r.x;
    }
    p.early = early ? 1 : 0;
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
    const cudaError_t e = hk::rows8_restore_launch({codes, ldc, scale, n_rows, d, group, X_out, ldx}, {}, dtype, false,
                                                   static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return rows_fail(HESS_ERR_CUDA, "rows8_restore: %s", cudaGetErrorString(e));
    return HESS_OK;
}
