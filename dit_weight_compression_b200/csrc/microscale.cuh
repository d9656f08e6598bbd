// microscale.cuh -- device functions shared by the 4-bit quantiser (fp4.cu) and the quantised
// key/value cache (cache.cu): loading eight neighbouring elements, block scales, E2M1 codes.
//
// Everything here rounds the exact quotient v / q.  That holds in fp32 because every scale q has
// at most four significant bits (a power of two, or an E4M3 value times a power of two): the border
// between two codes, m * q with m of three bits, is then a float itself.
//   * q a power of two: v / q is a float, nothing is rounded before the code.
//   * fp32 elements, other q: the IEEE quotient falls on a border only if v does, because two
//     different floats differ by more than the division's rounding (2^-24 relative).
//   * bf16 and fp16 elements, other q: v has at most 11 bits, so v / q is on a border m or at least
//     m * 2^-11 >= 2^-13 away from it.  One fma, v * (1/q) + 384, rounds to a multiple of 2^-15:
//     the reciprocal's error (2^-24) cannot take a value over a border, and borders come out exact.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "entropack.h"

namespace ep {
namespace ms {

constexpr uint32_t kFullMask = 0xffffffffu;

// A dependent launch's first step: everything before this kernel in its stream has finished.
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int DT>
struct Elem;
template <>
struct Elem<EP_BF16> { using T = __nv_bfloat16; };
template <>
struct Elem<EP_FP16> { using T = __half; };
template <>
struct Elem<EP_F32> { using T = float; };

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }

// Eight neighbouring elements as loaded, and as floats.
template <int DT>
struct Raw8 { uint4 u[DT == EP_F32 ? 2 : 1]; };

template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const typename Elem<DT>::T* p) {
    Raw8<DT> r;
#pragma unroll
    for (int i = 0; i < (DT == EP_F32 ? 2 : 1); ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}

template <int DT>
__device__ __forceinline__ void raw_to_float8(const Raw8<DT>& r, float* v) {
    if constexpr (DT == EP_F32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[4 * i] = __uint_as_float(r.u[i].x);
            v[4 * i + 1] = __uint_as_float(r.u[i].y);
            v[4 * i + 2] = __uint_as_float(r.u[i].z);
            v[4 * i + 3] = __uint_as_float(r.u[i].w);
        }
    } else {
        const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == EP_BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                v[2 * i] = f.x;
                v[2 * i + 1] = f.y;
            }
        }
    }
}

// The first n (0 to 8) of eight elements, one by one; zeros behind them.
template <int DT>
__device__ __forceinline__ void load_some(const typename Elem<DT>::T* p, int n, float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? to_float(p[j]) : 0.0f;
}

// max(a, |b|), NaN if either is.
__device__ __forceinline__ float max_abs(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(fabsf(b)));
    return d;
}
__device__ __forceinline__ float abs_max8(const float* v) {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max_abs(m, v[j]);
    return m;
}
// The largest of `lanes` neighbouring lanes (a power of two), in each of them.
__device__ __forceinline__ float lanes_max(float m, int lanes) {
    for (int o = 1; o < lanes; o <<= 1) m = max_abs(m, __shfl_xor_sync(kFullMask, m, o));
    return m;
}
__device__ __forceinline__ bool is_finite(float amax) { return amax < __int_as_float(0x7f800000); }
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

struct Block {
    uint32_t byte;  // the stored scale
    float q, inv;   // element = E2M1(v / q); inv = 1 / q (0 where every element is 0)
};
template <bool NV>
__device__ __forceinline__ Block block_scale(float amax, float g, float g_inv) {
    Block b;
    if constexpr (NV) {
        b.byte = e4m3_of(__fdiv_rn(amax, 6.0f) * g_inv);
        b.q = e4m3x2_value(b.byte).x * g;
        b.inv = b.q > 0.0f ? __frcp_rn(b.q) : 0.0f;
        if (!is_finite(amax)) b.byte = 0x7f;
    } else {
        const int e = max(log2_floor(amax) - 2, -127);
        b.byte = uint32_t(e + 127);
        b.q = 1.0f;  // not used
        b.inv = pow2f(-e);
        if (!is_finite(amax)) b.byte = 255;
    }
    if (!is_finite(amax)) b.inv = 0.0f;
    return b;
}

__device__ __forceinline__ uint32_t e2m1_pack8(const float* x) {
    uint32_t r;
    asm("{\n .reg .b8 a, b, c, d;\n"
        " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
        " mov.b32 %0, {a, b, c, d};\n}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

// Eight elements of one block as eight codes, the first in the lowest four bits.
template <int DT, bool NV>
__device__ __forceinline__ uint32_t quantize8(const float* v, const Block& b) {
    if (b.inv == 0.0f) return 0;  // q = 0, or a NaN block
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if constexpr (!NV) x[j] = v[j] * b.inv;
        else if constexpr (DT == EP_F32) x[j] = __fdiv_rn(v[j], b.q);
        else x[j] = __fadd_rn(__fmaf_rn(v[j], b.inv, 384.0f), -384.0f);
    }
    return e2m1_pack8(x);
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

// Eight floats to eight neighbouring elements, at once (16-byte aligned) or the first n one by one.
template <int DT>
__device__ __forceinline__ typename Elem<DT>::T from_float(float v) {
    if constexpr (DT == EP_BF16) return __float2bfloat16_rn(v);
    else if constexpr (DT == EP_FP16) return __float2half_rn(v);
    else return v;
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t r;
    if constexpr (DT == EP_BF16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
template <int DT>
__device__ __forceinline__ void store8(typename Elem<DT>::T* p, const float* v) {
    if constexpr (DT == EP_F32) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                                                  pack2<DT>(v[6], v[7]));
    }
}
template <int DT>
__device__ __forceinline__ void store_some(typename Elem<DT>::T* p, int n, const float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) p[j] = from_float<DT>(v[j]);
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

// Launch as a programmatic dependent: the kernel may be set up while the one before it in the
// stream still runs, and waits for it in wait_for_stream().
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

}  // namespace op
}  // namespace ep
