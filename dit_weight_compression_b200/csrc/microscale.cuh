// microscale.cuh -- device functions shared by the 4-bit quantiser (fp4.cu) and the quantised
// key/value cache (cache.cu): loading eight neighbouring elements, block scales, E2M1 codes.
//
// Everything here rounds the exact quotient v / q.  That holds in fp32 because every scale q has
// at most four significant bits (a power of two, or an E4M3 value times a power of two): the border
// between two codes, m * q with m of three bits, is then a float itself.
//   * q a power of two: v / q is a float, nothing is rounded before the code.
//   * fp32 elements, other q: the correctly rounded quotient (Markstein: an approximate quotient, its
//     exact remainder, one correction) falls on a border only if v does, because two different
//     floats differ by more than that rounding (2^-24 relative).
//   * bf16 and fp16 elements, other q: v has at most 11 bits, so v / q is on a border m or at least
//     m * 2^-11 >= 2^-13 away from it.  One fma, v * (1/q) + 384, rounds to a multiple of 2^-15:
//     the reciprocal's error (2^-22) cannot take a value over a border, and borders come out exact.
// The elements go in pairs through the packed fp32 instructions, and the largest of 16-bit elements is
// found on their bits, two at a time: a block costs about 7 instructions an element less than one by
// one, and the quantiser is bound by its loads instead of by issue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "entropack.h"

namespace ep {
namespace ms {

constexpr uint32_t kFullMask = 0xffffffffu;

// A dependent launch's first step: everything before this kernel in its stream has finished, and the next
// kernel may be set up from here on (it waits in the same way before it touches memory).
__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;\n griddepcontrol.launch_dependents;" ::: "memory");
}

template <int DT>
struct Elem;
template <>
struct Elem<EP_BF16> { using T = __nv_bfloat16; };
template <>
struct Elem<EP_FP16> { using T = __half; };
template <>
struct Elem<EP_F32> { using T = float; };

// Eight neighbouring elements as loaded.
template <int DT>
struct Raw8 { uint32_t w[DT == EP_F32 ? 8 : 4]; };

template <int DT>
__device__ __forceinline__ Raw8<DT> zero_raw8() {
    Raw8<DT> r;
#pragma unroll
    for (uint32_t& w : r.w) w = 0;
    return r;
}

// n (0 to 8) elements from p on, zeros behind them.  `width`: the alignment of p in bytes, 16, 8 or 4;
// anything less goes element by element.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const typename Elem<DT>::T* p, int n, int width) {
    constexpr int W = DT == EP_F32 ? 8 : 4;
    Raw8<DT> r = zero_raw8<DT>();
    if (n <= 0) return r;
    if (n == 8 && width == 16) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 u = reinterpret_cast<const uint4*>(p)[i];
            r.w[4 * i] = u.x, r.w[4 * i + 1] = u.y, r.w[4 * i + 2] = u.z, r.w[4 * i + 3] = u.w;
        }
    } else if (n == 8 && width == 8) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            const uint2 u = reinterpret_cast<const uint2*>(p)[i];
            r.w[2 * i] = u.x, r.w[2 * i + 1] = u.y;
        }
    } else if (n == 8 && width == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                if constexpr (DT == EP_F32) r.w[j] = reinterpret_cast<const uint32_t*>(p)[j];
                else r.w[j / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j % 2));
            }
    }
    return r;
}

// 32 bytes of elements (16 or 8) at any address: the aligned 16-byte granules that hold them, all loaded
// before the first is used, and then shifted into place.  Nothing outside [lo, hi), the matrix from its
// first element to its last, is read: a granule that reaches over either end goes element by element.
template <int DT>
__device__ __noinline__ uint4 load_granule_parts(uintptr_t at, uintptr_t lo, uintptr_t hi) {
    uint32_t w[4] = {0, 0, 0, 0};
    constexpr int kSize = sizeof(typename Elem<DT>::T);
#pragma unroll
    for (int b = 0; b < 16; b += kSize)
        if (at + b >= lo && at + b < hi) {
            if constexpr (kSize == 4) w[b / 4] = *reinterpret_cast<const uint32_t*>(at + b);
            else w[b / 4] |= uint32_t(*reinterpret_cast<const uint16_t*>(at + b)) << (8 * (b % 4));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int DT>
struct Piece {
    uint32_t w[12];
    // n: elements wanted, 0 to 32 / size.
    __device__ __forceinline__ void load(const typename Elem<DT>::T* p, int n, uintptr_t lo, uintptr_t hi) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p), first = at & ~uintptr_t(15);
        const uintptr_t end = n > 0 ? at + n * sizeof(*p) : first;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            uint4 u = make_uint4(0, 0, 0, 0);
            const uintptr_t g = first + 16 * i;
            if (g < end) u = g >= lo && g + 16 <= hi ? *reinterpret_cast<const uint4*>(g) : load_granule_parts<DT>(g, lo, hi);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    }
    // The elements, zeros from the n-th on, as chunks of 8.
    __device__ __forceinline__ void take(const typename Elem<DT>::T* p, int n, Raw8<DT>* v) {
        const uint32_t s = uint32_t(reinterpret_cast<uintptr_t>(p)) & 15u;
#pragma unroll
        for (int i = 0; i < 10; ++i) w[i] = s & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 9; ++i) w[i] = s & 4 ? w[i + 1] : w[i];
        if constexpr (DT != EP_F32)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = s & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
        constexpr int kWords = DT == EP_F32 ? 8 : 4, kPer = DT == EP_F32 ? 1 : 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t keep = n >= kPer * (i + 1) ? 0xffffffffu : kPer == 2 && n == 2 * i + 1 ? 0xffffu : 0u;
            v[i / kWords].w[i % kWords] = w[i] & keep;
        }
    }
};

// Elements 2i and 2i + 1 as floats.
template <int DT>
__device__ __forceinline__ float2 pair(const Raw8<DT>& r, int i) {
    if constexpr (DT == EP_F32) return make_float2(__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1]));
    else if constexpr (DT == EP_BF16) return make_float2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
}

// The largest |v| as the bits of its own type without the sign, which are in the order of the values;
// a NaN or an infinity is at least kInf.
template <int DT>
struct AbsBits {
    static constexpr uint32_t kInf = DT == EP_F32 ? 0x7f800000u : DT == EP_BF16 ? 0x7f80u : 0x7c00u;
};
template <int DT>
__device__ __forceinline__ uint32_t abs_max8(const Raw8<DT>& r) {
    if constexpr (DT == EP_F32) {
        uint32_t m = 0;
#pragma unroll
        for (uint32_t w : r.w) m = max(m, w & 0x7fffffffu);
        return m;
    } else {
        uint32_t m = __vmaxu2(__vmaxu2(r.w[0] & 0x7fff7fffu, r.w[1] & 0x7fff7fffu),
                              __vmaxu2(r.w[2] & 0x7fff7fffu, r.w[3] & 0x7fff7fffu));
        return max(m & 0xffffu, m >> 16);
    }
}
template <int DT>
__device__ __forceinline__ float abs_value(uint32_t bits) {
    if constexpr (DT == EP_F32) return __uint_as_float(bits);
    else if constexpr (DT == EP_BF16) return __uint_as_float(bits << 16);
    else return __half2float(__ushort_as_half(uint16_t(bits)));
}
// The largest of LANES neighbouring lanes (a power of two), in each of them.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
    return m;
}

// Two floats at a time.
__device__ __forceinline__ unsigned long long as_u64(float2 v) {
    return static_cast<unsigned long long>(__float_as_uint(v.x)) | (static_cast<unsigned long long>(__float_as_uint(v.y)) << 32);
}
__device__ __forceinline__ float2 as_float2(unsigned long long v) {
    return make_float2(__uint_as_float(uint32_t(v)), __uint_as_float(uint32_t(v >> 32)));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_float2(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)));
    return as_float2(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
    return as_float2(d);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// floor(log2 x) of a normal x; at most -127 for smaller ones.
__device__ __forceinline__ int log2_floor(float x) { return (__float_as_int(x) >> 23) - 127; }

// The tensor scale: the smallest power of two with amax <= 2688 g, 2688 = 1.3125 * 2^11 = 6 * 448.
__device__ __forceinline__ float tensor_scale_of(float amax) {
    const int m = __float_as_int(amax) & 0x7fffff;
    const int k = log2_floor(amax) - 11 + (m > 0x280000 ? 1 : 0);
    return pow2f(min(max(k, -100), 117));
}

__device__ __forceinline__ uint32_t e4m3_of(float v) {  // nearest, saturating
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(v));
    return r & 0xffu;
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(two)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Block scale bytes and what they stand for.
template <bool NV>
__device__ __forceinline__ float scale_value(uint32_t byte) {
    if constexpr (NV) return e4m3x2_value(byte & 0x7fu).x;
    return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

// 1 / q, within one unit in the last place, and then (for a q of few bits) correctly rounded.
__device__ __forceinline__ float reciprocal_near(float q) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(q));
    return y;
}
__device__ __forceinline__ float reciprocal(float q) {
    const float y = reciprocal_near(q);
    return __fmaf_rn(y, __fmaf_rn(-q, y, 1.0f), y);
}

struct Block {
    uint32_t byte;  // the stored scale
    float q, inv;   // element = E2M1(v / q); inv = 1 / q, 0 where every element is 0
    float amax;
};
// The scale of a block from the bits of its largest element.
template <int DT, bool NV>
__device__ __forceinline__ Block block_scale(uint32_t amax_bits, float g, float g_inv) {
    Block b;
    b.amax = abs_value<DT>(amax_bits);
    const bool fine = amax_bits < AbsBits<DT>::kInf;
    if constexpr (NV) {
        // amax / 6: for 16-bit elements the product with fl(1/6) is exact where it is on a border of
        // two E4M3 values and far closer than the next element elsewhere; fp32 is corrected
        constexpr float kSixth = 1.0f / 6.0f;
        float t = b.amax * kSixth;
        if constexpr (DT == EP_F32) t = __fmaf_rn(__fmaf_rn(-6.0f, t, b.amax), kSixth, t);
        b.byte = e4m3_of(t * g_inv);
        b.q = e4m3x2_value(b.byte).x * g;
        b.inv = !fine || b.q == 0.0f ? 0.0f : DT == EP_F32 ? reciprocal(b.q) : reciprocal_near(b.q);
        if (!fine) b.byte = 0x7f;
    } else {
        const int e = max(log2_floor(b.amax) - 2, -127);
        b.byte = fine ? uint32_t(e + 127) : 255u;
        b.q = 1.0f;  // not used
        b.inv = fine ? pow2f(-e) : 0.0f;
    }
    return b;
}

__device__ __forceinline__ uint32_t e2m1_pack8(const float2* x) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
    return r;
}

// Eight elements of one block as eight codes, the first in the lowest four bits.
template <int DT, bool NV>
__device__ __forceinline__ uint32_t quantize8(const Raw8<DT>& r, const Block& b) {
    float2 x[4];
    const float2 inv = both(b.inv);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = pair<DT>(r, i);
        if constexpr (!NV) {
            x[i] = mul2(v, inv);
        } else if constexpr (DT != EP_F32) {
            x[i] = add2(fma2(v, inv, both(384.0f)), both(-384.0f));
        } else {
            x[i] = mul2(v, inv);
            x[i] = fma2(fma2(x[i], both(-b.q), v), inv, x[i]);
        }
    }
    if constexpr (NV && DT == EP_F32)  // far above the block's range (a tensor scale given too small)
        if (b.amax > 8.0f * b.q) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = pair<DT>(r, i);
                x[i] = make_float2(__fdiv_rn(v.x, b.q), __fdiv_rn(v.y, b.q));
            }
        }
    return b.inv == 0.0f ? 0u : e2m1_pack8(x);  // q = 0, or a NaN block
}

// The values of eight codes.
__device__ __forceinline__ void e2m1_values8(uint32_t codes, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t h;
        asm("{\n .reg .b8 a;\n cvt.u8.u32 a, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}" : "=r"(h) : "r"((codes >> (8 * i)) & 0xffu));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t r;
    if constexpr (DT == EP_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
// Eight values as they are stored.
template <int DT>
__device__ __forceinline__ Raw8<DT> pack8(const float* v) {
    Raw8<DT> r;
#pragma unroll
    for (int i = 0; i < (DT == EP_F32 ? 8 : 4); ++i) {
        if constexpr (DT == EP_F32) r.w[i] = __float_as_uint(v[i]);
        else r.w[i] = pack2<DT>(v[2 * i], v[2 * i + 1]);
    }
    return r;
}
// The first n of eight values to p, which is aligned to `width` bytes as for load_raw8.
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, int n, int width, const float* v) {
    constexpr int W = DT == EP_F32 ? 8 : 4;
    const Raw8<DT> packed = pack8<DT>(v);
    const uint32_t* w = packed.w;
    if (n == 8 && width == 16) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if (n == 8 && width == 8) {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) reinterpret_cast<uint2*>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
    } else if (n == 8 && width == 4) {
#pragma unroll
        for (int i = 0; i < W; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) {
                if constexpr (DT == EP_F32) reinterpret_cast<uint32_t*>(p)[j] = w[j];
                else reinterpret_cast<uint16_t*>(p)[j] = uint16_t(w[j / 2] >> (16 * (j % 2)));
            }
    }
}

}  // namespace ms

// ---- host side -----------------------------------------------------------------------------------
namespace op {

inline int elem_bytes(int dtype) { return dtype == EP_BF16 || dtype == EP_FP16 ? 2 : dtype == EP_F32 ? 4 : 0; }
inline bool is_fp4(int format) { return format == EP_MXFP4 || format == EP_NVFP4; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t fp4_row_bytes(int64_t cols) { return 16 * div_up(cols, 32); }
inline int64_t fp4_blocks(int format, int64_t cols) { return div_up(cols, format == EP_MXFP4 ? 32 : 16); }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
// The widest access, 16, 8 or 4 bytes, that fits a pointer and strides (in bytes); else 1.
inline int access_width(const void* p, int64_t stride, int64_t stride2 = 0) {
    for (int w : {16, 8, 4})
        if (aligned(p, size_t(w)) && stride % w == 0 && stride2 % w == 0) return w;
    return 1;
}

// Launch as a programmatic dependent: the kernel may be set up while the one before it in the
// stream still runs, and waits for it in wait_for_stream().
// `cluster`: blocks of a cluster (1: none).
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = unsigned(cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
    return launch_clusters(kernel, grid, block, smem, 1, st, std::forward<Args>(args)...);
}

}  // namespace op
}  // namespace ep
