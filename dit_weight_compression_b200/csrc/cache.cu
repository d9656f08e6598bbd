// cache.cu -- the quantised key/value cache: ep_cache_write and ep_cache_read.  The formats are
// defined in entropack.h; the 4-bit block arithmetic is in microscale.cuh.
#include <algorithm>
#include <string>

#include "blob.h"
#include "microscale.cuh"
#include "ops.h"

namespace ep {
namespace {

using namespace ms;

// Two variants of each kernel.  The common one serves rows of up to 256 elements in whole eights, 16-byte
// aligned outside the cache: a lane has 16 elements, so that the row's addresses, maximum and scale, which
// cost as much as 8 elements, are shared by more (for 8 elements 228 -> 130 instructions of a lane in an
// int8 write, 138 -> 73 in an fp8 read; copying at the memory's rate leaves time for 133).
// The other serves every head up to 1024 elements, 8 a lane, at any alignment.
constexpr int kThreads = 256;
constexpr int kMaxHeadDim = 1024;
constexpr int kMaxFastDim = 256;
constexpr int kLaunchTokens = 65536; // tokens of one write launch
constexpr int kMaxWriteTokens = 64;  // most tokens of one block of a write
constexpr int kAloneTokens = 1024;   // up to so many tokens a write looks for repeated slots itself
constexpr int kMendThreads = 1024;
constexpr int kMendTokens = 512;     // tokens of one block of mend_kernel
constexpr int kTableBits = 11;       // hash table of their slots
constexpr int kTable = 1 << kTableBits;
constexpr int kMaxReadTokens = 64;   // most tokens of one block of a read
constexpr int kSharedSeqs = 1024;    // sequence starts that a read searches in shared memory

struct CacheView {
    uint8_t* data;
    uint8_t* scales;
    int64_t row_bytes;
    int64_t scale_bytes;  // of one row: 4, or one a block
    void* heads;          // source or output rows
    int64_t token_stride, head_stride;
    int head_dim;
    int width;            // alignment of its rows for load_raw8 and store8
};

struct WriteArgs {
    CacheView c[2];
    const int64_t* slots;
    int64_t n_slots;      // n_pages * page_size
    int64_t tokens;       // of this launch
    int n, heads;         // caches, and heads of each
    float heads_inv;
    int per_block;        // tokens of one block
    bool alone;           // drop repeated slots here: no mend_kernel follows
};

struct ReadArgs {
    CacheView c[2];
    const int32_t* page_table;
    int64_t table_stride, pages_per_seq, n_pages, tokens;
    const int32_t* cu_seqlens;
    int n_seqs, page_size;
    int n, heads;         // caches, and heads of each
    float heads_inv;
    int per_block;        // tokens of one block
};

// r / d for 0 <= r <= 2^20 and d_inv = 1.0f / d: (r + 1/2) / d is at least 1 / (2 d) away from an integer,
// more than the product's rounding.
__device__ __forceinline__ int quotient(int r, float d_inv) { return int((float(r) + 0.5f) * d_inv); }

// ---- writing -----------------------------------------------------------------------------------

// The smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8), at least 2^-100.
__device__ __forceinline__ int e4m3_row_exponent(float amax) {
    const int m = __float_as_int(amax) & 0x7fffff;
    return max(log2_floor(amax) - 8 + (m > 0x600000 ? 1 : 0), -100);
}

// The integer nearest v / s, ties to even: a candidate from the reciprocal, at most one off, and the
// exact remainder v - n s (it is a multiple of the smaller of the two units in the last place and
// not much above s, so the fma does not round it) to settle the border.
__device__ __forceinline__ int nearest_quotient(float v, float s, float inv) {
    const float n = rintf(v * inv);
    const float r = __fmaf_rn(-n, s, v), h = 0.5f * s;
    int i = int(n);
    if (r > h || (r == h && (i & 1))) ++i;
    if (r < -h || (r == -h && (i & 1))) --i;
    return i;
}

// Eight int8 payload bytes.  Candidates from the reciprocal in pairs, rounded by adding 1.5 * 2^23 (the
// integer is then the sum's low byte); only if a remainder is within 2^-20 of half a step, or above
// it, the elements are settled one by one.
template <int DT>
__device__ __forceinline__ uint2 int8_payload(const Raw8<DT>& v, float s, float inv) {
    constexpr float kMagic = 12582912.0f;
    float2 y[4];
    float worst = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = pair<DT>(v, i);
        y[i] = fma2(x, both(inv), both(kMagic));
        const float2 r = fma2(add2(y[i], both(-kMagic)), both(-s), x);
        worst = fmaxf(worst, fmaxf(fabsf(r.x), fabsf(r.y)));
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __byte_perm(__byte_perm(__float_as_uint(y[2 * i].x), __float_as_uint(y[2 * i].y), 0x0040),
                           __byte_perm(__float_as_uint(y[2 * i + 1].x), __float_as_uint(y[2 * i + 1].y), 0x0040), 0x5410);
    if (worst >= 0.5f * s * (1.0f - 0x1p-20f)) {
        w[0] = w[1] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 x = pair<DT>(v, j / 2);
            w[j / 4] |= uint32_t(nearest_quotient(j % 2 ? x.y : x.x, s, inv) & 0xff) << (8 * (j % 4));
        }
    }
    return make_uint2(w[0], w[1]);
}
template <int DT>
__device__ __forceinline__ uint2 e4m3_payload(const Raw8<DT>& v, float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint16_t lo, hi;
        const float2 a = mul2(pair<DT>(v, 2 * i), both(inv)), b = mul2(pair<DT>(v, 2 * i + 1), both(inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
        w[i] = uint32_t(lo) | (uint32_t(hi) << 16);
    }
    return make_uint2(w[0], w[1]);
}

// Scale and reciprocal of an 8-bit row from the bits of its largest element: payload = v * inv, rounded;
// inv = 0 where the payload is zeros.  int8: s is the product with the float nearest 1/127, as torch divides by a
// constant on a GPU, so that rows quantised there in elementary operations get the same scale and, with the
// payload nearest v / s, the same integers.  It is at most a unit in the last place from the rounded amax / 127.
template <int DT, int FMT>
__device__ __forceinline__ void row_scale(uint32_t bits, float& s, float& inv) {
    const bool fine = bits < AbsBits<DT>::kInf;
    const float amax = abs_value<DT>(bits);
    if constexpr (FMT == EP_FP8_E4M3) {
        const int e = e4m3_row_exponent(amax);
        s = pow2f(e);
        inv = pow2f(-e);
    } else {
        s = amax >= 0x1p-100f ? __fmul_rn(amax, 1.0f / 127.0f) : 0.0f;
        inv = s > 0.0f ? reciprocal_near(s) : 0.0f;
    }
    if (!fine) s = __int_as_float(0x7fc00000), inv = 0.0f;
}
template <int DT, int FMT>
__device__ __forceinline__ uint2 payload8(const Raw8<DT>& v, float s, float inv) {
    if (inv == 0.0f) return make_uint2(0, 0);
    if constexpr (FMT == EP_FP8_E4M3) return e4m3_payload<DT>(v, inv);
    else return int8_payload<DT>(v, s, inv);
}

// When a launch names a slot more than once, payload and scale have to come from one token, the last.
// (Launches of one call follow each other, so that between launches the later wins.)  A write of few
// tokens drops the others itself: every block compares its slots with all that come after.  For many
// tokens that wait before the first store costs more than it brings (9 of 33 us for 16384), so the write
// does not look, and mend_kernel, which finds the slots while the write's last blocks run, writes those
// tokens once more.

// Where a block's tokens go: their slots, -1 for one that is skipped.  All threads; ends with a barrier.
__device__ __forceinline__ void find_slots(const WriteArgs& a, int64_t t0, int n, int64_t* slot, int* dropped) {
    if (int(threadIdx.x) < n) {
        const int64_t s = a.slots[t0 + threadIdx.x];
        slot[threadIdx.x] = s >= 0 && s < a.n_slots ? s : -1;
        dropped[threadIdx.x] = 0;
    }
    __syncthreads();
    if (!a.alone) return;
    for (int64_t j0 = t0 + 1 + threadIdx.x; j0 < a.tokens; j0 += 4 * kThreads) {
        int64_t s[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) s[u] = j0 + u * kThreads < a.tokens ? a.slots[j0 + u * kThreads] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            for (int i = 0; i < n; ++i)
                if (s[u] >= 0 && slot[i] == s[u] && t0 + i < j0 + u * kThreads) dropped[i] = 1;
    }
    __syncthreads();
    if (int(threadIdx.x) < n && dropped[threadIdx.x]) slot[threadIdx.x] = -1;
    __syncthreads();
}

// A block takes a few tokens, all heads of one cache; rows go in batches of LANES lanes a row, whose loads
// are all on their way before the first is used, those of the first batch before the slots are looked up.
template <int DT, int FMT, int LANES>
__global__ void __launch_bounds__(kThreads, DT == EP_F32 ? 3 : 4) cache_write_kernel(const __grid_constant__ WriteArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int kBatch = DT == EP_F32 ? 2 : 4, kStep = kThreads / LANES;
    constexpr bool kFp4 = FMT == EP_MXFP4 || FMT == EP_NVFP4;
    __shared__ int64_t slot[kMaxWriteTokens];
    __shared__ int dropped[kMaxWriteTokens];
    wait_for_stream();
    const int64_t t0 = int64_t(blockIdx.x) * a.per_block;
    const int n = int(min(int64_t(a.per_block), a.tokens - t0));
    const CacheView& c = a.c[blockIdx.y];
    const int rows = n * a.heads;
    const T* src = static_cast<const T*>(c.heads) + t0 * c.token_stride;
    const int sub = threadIdx.x / LANES, lane = threadIdx.x % LANES;
    // 4-bit: sixteen neighbours, of one block; 8-bit: twice eight, so that lanes touch neighbouring bytes
    const int e = (kFp4 ? 16 : 8) * lane, e2 = e + (kFp4 ? 8 : 8 * LANES);
    Raw8<DT> v[kBatch][2];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int r = base + u * kStep + sub, i = quotient(r, a.heads_inv), h = r - i * a.heads;
            const bool in = r < rows;
            const T* p = src + i * c.token_stride + h * c.head_stride;
            v[u][0] = load_raw8<DT>(p + e, in && e < c.head_dim ? 8 : 0, 16);
            v[u][1] = load_raw8<DT>(p + e2, in && e2 < c.head_dim ? 8 : 0, 16);
        }
    };
    load(0);
    find_slots(a, t0, n, slot, dropped);
    // every lane of a warp stays in the loop: rows past the end are zeros and not written
    for (int base = 0; base < rows;) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (base + u * kStep >= rows) break;
            const int r = base + u * kStep + sub;
            const bool in = r < rows;
            const int i = in ? quotient(r, a.heads_inv) : 0, h = r - i * a.heads;
            const int64_t to = in ? slot[i] : -1, row = to * a.heads + h;
            const bool live = to >= 0 && e < c.head_dim;
            uint32_t bits = max(abs_max8<DT>(v[u][0]), abs_max8<DT>(v[u][1]));
            if constexpr (kFp4) {
                constexpr bool NV = FMT == EP_NVFP4;
                const Block b = block_scale<DT, NV>(lanes_max<NV ? 1 : 2>(bits), 1.0f, 1.0f);
                const uint2 w = make_uint2(quantize8<DT, NV>(v[u][0], b), quantize8<DT, NV>(v[u][1], b));
                // the lane past an odd number of sixteens writes the row's padding
                if (to >= 0 && 8 * lane < int(c.row_bytes)) {
                    *reinterpret_cast<uint2*>(c.data + row * c.row_bytes + 8 * lane) = w;
                    if (live && (NV || lane % 2 == 0)) c.scales[row * c.scale_bytes + (NV ? lane : lane / 2)] = uint8_t(b.byte);
                }
            } else {
                bits = lanes_max<LANES>(bits);
                float s, inv;
                row_scale<DT, FMT>(bits, s, inv);
                if (live) {
                    uint8_t* data = c.data + row * c.row_bytes;
                    *reinterpret_cast<uint2*>(data + e) = payload8<DT, FMT>(v[u][0], s, inv);
                    if (e2 < c.head_dim) *reinterpret_cast<uint2*>(data + e2) = payload8<DT, FMT>(v[u][1], s, inv);
                    if (lane == 0) reinterpret_cast<float*>(c.scales)[row] = s;
                }
            }
        }
        base += kBatch * kStep;
        if (base < rows) load(base);
    }
}

// One row of any head by a warp, 4 chunks of 8 elements a lane, at any alignment.
template <int DT, int FMT>
__device__ __forceinline__ void write_any_row(const CacheView& c, const typename Elem<DT>::T* src, int64_t row) {
    constexpr int NC = kMaxHeadDim / 256;
    const int lane = threadIdx.x % 32;
    uint8_t* data = c.data + row * c.row_bytes;
    Raw8<DT> v[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) v[k] = load_raw8<DT>(src + 8 * (lane + 32 * k), min(8, c.head_dim - 8 * (lane + 32 * k)), c.width);
    if constexpr (FMT == EP_FP8_E4M3 || FMT == EP_INT8) {
        uint32_t bits = 0;
#pragma unroll
        for (int k = 0; k < NC; ++k) bits = max(bits, abs_max8<DT>(v[k]));
        float s, inv;
        row_scale<DT, FMT>(lanes_max<32>(bits), s, inv);
        if (lane == 0) reinterpret_cast<float*>(c.scales)[row] = s;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int at = 8 * (lane + 32 * k);
            if (at >= c.head_dim) break;
            const uint2 w = payload8<DT, FMT>(v[k], s, inv);
            if (c.head_dim % 8 == 0) {
                *reinterpret_cast<uint2*>(data + at) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at + j < c.head_dim) data[at + j] = uint8_t((j < 4 ? w.x : w.y) >> (8 * (j % 4)));
            }
        }
    } else {
        constexpr bool NV = FMT == EP_NVFP4;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            const int chunk = lane + 32 * k;
            const Block b = block_scale<DT, NV>(lanes_max<NV ? 2 : 4>(abs_max8<DT>(v[k])), 1.0f, 1.0f);
            const uint32_t codes = quantize8<DT, NV>(v[k], b);
            if (4 * chunk >= int(c.row_bytes)) continue;
            *reinterpret_cast<uint32_t*>(data + 4 * chunk) = codes;
            if (chunk % (NV ? 2 : 4) == 0 && 8 * chunk < c.head_dim)
                c.scales[row * c.scale_bytes + chunk / (NV ? 2 : 4)] = uint8_t(b.byte);
        }
    }
}

// cache_write_kernel for any head: a warp a row.
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) cache_write_any_kernel(const __grid_constant__ WriteArgs a) {
    using T = typename Elem<DT>::T;
    __shared__ int64_t slot[kMaxWriteTokens];
    __shared__ int dropped[kMaxWriteTokens];
    wait_for_stream();
    const int64_t t0 = int64_t(blockIdx.x) * a.per_block;
    const int n = int(min(int64_t(a.per_block), a.tokens - t0));
    find_slots(a, t0, n, slot, dropped);
    const CacheView& c = a.c[blockIdx.y];
    for (int r = threadIdx.x / 32; r < n * a.heads; r += kThreads / 32) {
        const int i = quotient(r, a.heads_inv), h = r - i * a.heads;
        if (slot[i] >= 0)
            write_any_row<DT, FMT>(c, static_cast<const T*>(c.heads) + (t0 + i) * c.token_stride + h * c.head_stride,
                                   slot[i] * a.heads + h);
    }
}

// After a write that did not look: each block puts the slots of 512 tokens into a hash table, looks up all
// slots of the launch, and writes those of its tokens again that come last of several to a slot.  A slot has one
// entry, the last of the block's tokens that name it, however many do: with an entry for each, 65536 tokens of
// which half name one slot (padding in a slot of its own) took 3 ms, walking chains of equal entries.
__device__ __forceinline__ uint32_t slot_hash(int64_t s) {
    return ((uint32_t(s) ^ uint32_t(uint64_t(s) >> 32)) * 2654435761u) >> (32 - kTableBits);
}
template <int DT, int FMT>
__global__ void __launch_bounds__(kMendThreads) mend_kernel(const __grid_constant__ WriteArgs a) {
    using T = typename Elem<DT>::T;
    static_assert(kMendThreads >= kMendTokens && 2 * kMendTokens <= kTable, "a thread for each token, and room in the table");
    __shared__ int64_t slot[kMendTokens];
    __shared__ int earlier[kMendTokens], later[kMendTokens], table[kTable], any;
    const int64_t t0 = int64_t(blockIdx.x) * kMendTokens;
    const int n = int(min(int64_t(kMendTokens), a.tokens - t0));
    // The slots are read before the write is waited for: the write itself started only when everything
    // before it was done, and does not change them.  (From L2: nothing older is taken.)
    int64_t own = -1;
    if (int(threadIdx.x) < n) {
        own = __ldcg(a.slots + t0 + threadIdx.x);
        if (own >= a.n_slots) own = -1;
        slot[threadIdx.x] = own;
        earlier[threadIdx.x] = later[threadIdx.x] = 0;
    }
    for (int i = threadIdx.x; i < kTable; i += kMendThreads) table[i] = -1;
    if (threadIdx.x == 0) any = 0;
    __syncthreads();
    if (own >= 0)
        for (uint32_t h = slot_hash(own);; h = (h + 1) % kTable) {
            const int i = atomicCAS(&table[h], -1, int(threadIdx.x));
            if (i == -1) break;
            if (slot[i] == own) {  // an entry keeps its slot, whichever token it names
                atomicMax(&table[h], int(threadIdx.x));
                break;
            }
        }
    __syncthreads();
    for (int64_t j0 = threadIdx.x; j0 < a.tokens; j0 += 8 * kMendThreads) {
        int64_t s[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) s[u] = j0 + u * kMendThreads < a.tokens ? __ldcg(a.slots + j0 + u * kMendThreads) : -1;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (s[u] < 0) continue;
            const int64_t j = j0 + u * kMendThreads - t0;
            int i;
            for (uint32_t h = slot_hash(s[u]); (i = table[h]) != -1 && slot[i] != s[u]; h = (h + 1) % kTable) {}
            if (i != -1 && j != i) (j < i ? earlier : later)[i] = any = 1;
        }
    }
    __syncthreads();
    wait_for_stream();
    if (!any) return;
    for (int r = threadIdx.x / 32; r < a.n * n * a.heads; r += kMendThreads / 32) {
        const int i = r / (a.n * a.heads), rest = r - i * a.n * a.heads, ci = rest / a.heads, h = rest - ci * a.heads;
        const CacheView& c = a.c[ci];
        if (earlier[i] && !later[i])
            write_any_row<DT, FMT>(c, static_cast<const T*>(c.heads) + (t0 + i) * c.token_stride + h * c.head_stride,
                                   slot[i] * a.heads + h);
    }
}

// ---- reading -----------------------------------------------------------------------------------

// The values of 8 payload elements: two words, or one of the 4-bit formats.
template <int FMT>
__device__ __forceinline__ void values8(uint32_t lo, uint32_t hi, float s, float* v) {
    if constexpr (FMT == EP_FP8_E4M3 || FMT == EP_INT8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t two = ((j < 2 ? lo : hi) >> (16 * (j % 2))) & 0xffffu;
            const float2 f = FMT == EP_FP8_E4M3 ? e4m3x2_value(two)
                                                : make_float2(float(int8_t(two & 0xff)), float(int8_t(two >> 8)));
            const float2 p = mul2(f, both(s));
            v[2 * j] = p.x;
            v[2 * j + 1] = p.y;
        }
    } else {
        e2m1_values8(lo, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= s;
    }
}

// The last sequence that starts at or before token t.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int n_seqs, int64_t t) {
    int lo = 0, hi = n_seqs;  // cu[lo] <= t < cu[hi], if t is in any sequence
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (int64_t(cu[mid]) <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The slots of a block's tokens: -1 for one without a valid page (zeros), -2 past the sequences.  All
// threads; ends with a barrier.
__device__ __forceinline__ void find_pages(const ReadArgs& a, int64_t t0, int n, int32_t* starts, int64_t* slot) {
    const bool shared = a.n_seqs <= kSharedSeqs;
    if (shared) {
        for (int i = threadIdx.x; i <= a.n_seqs; i += kThreads) starts[i] = a.cu_seqlens[i];
        __syncthreads();
    }
    if (int(threadIdx.x) < n) {
        const int32_t* cu = shared ? starts : a.cu_seqlens;
        const int64_t t = t0 + threadIdx.x;
        int64_t s = -2;
        const int seq = sequence_of(cu, a.n_seqs, t);
        const int64_t pos = t - cu[seq];
        if (pos >= 0 && t < cu[seq + 1]) {  // the position fits 32 bits: tokens do
            s = -1;
            const uint32_t p = uint32_t(pos) / uint32_t(a.page_size);
            if (int64_t(p) < a.pages_per_seq) {
                const int64_t page = a.page_table[seq * a.table_stride + p];
                if (page >= 0 && page < a.n_pages) s = page * a.page_size + (uint32_t(pos) - p * uint32_t(a.page_size));
            }
        }
        slot[threadIdx.x] = s;
    }
    __syncthreads();
}

// A block takes up to 64 tokens, all heads of all outputs: finds their slots, then reads rows of LANES
// lanes in batches, whose loads are all on their way before the first is used.
template <int DT, int FMT, int LANES>
__global__ void __launch_bounds__(kThreads, 4) cache_read_kernel(const __grid_constant__ ReadArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int kBatch = 4, kStep = kThreads / LANES;
    constexpr bool kFp4 = FMT == EP_MXFP4 || FMT == EP_NVFP4;
    __shared__ int32_t starts[kSharedSeqs + 1];
    __shared__ int64_t slot[kMaxReadTokens];
    wait_for_stream();
    const int64_t t0 = int64_t(blockIdx.x) * a.per_block;
    const int n = int(min(int64_t(a.per_block), a.tokens - t0));
    find_pages(a, t0, n, starts, slot);
    const int rows = n * a.heads, all = a.n * rows, lane = threadIdx.x % LANES;
    for (int base = threadIdx.x / LANES; base < all; base += kBatch * kStep) {
        uint2 q[kBatch][2];  // chunks `lane` and `lane + LANES` of 8 elements
        float s[kBatch][kFp4 ? 2 : 1];
        T* dst[kBatch];
        bool second[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            int r = base + u * kStep;
            const bool in = r < all;
            const int ci = r >= rows && in ? 1 : 0;
            r = in ? r - (ci ? rows : 0) : 0;
            const int t = quotient(r, a.heads_inv), h = r - t * a.heads;
            const CacheView& c = a.c[ci];
            const int64_t from = slot[t], row = from * a.heads + h;
            dst[u] = in && from != -2 && 8 * lane < c.head_dim
                         ? static_cast<T*>(c.heads) + (t0 + t) * c.token_stride + h * c.head_stride + 8 * lane
                         : nullptr;
            second[u] = 8 * (lane + LANES) < c.head_dim;
            q[u][0] = q[u][1] = make_uint2(0, 0);
            s[u][0] = s[u][kFp4 ? 1 : 0] = 0.0f;
            if (dst[u] && from >= 0) {
                const uint8_t* p = c.data + row * c.row_bytes;
                if constexpr (kFp4) {
                    constexpr int kPer = FMT == EP_NVFP4 ? 2 : 4;  // chunks of a block
                    const uint8_t* sc = c.scales + row * c.scale_bytes;
                    q[u][0].x = reinterpret_cast<const uint32_t*>(p)[lane];
                    s[u][0] = scale_value<FMT == EP_NVFP4>(sc[lane / kPer]);
                    if (second[u]) {
                        q[u][1].x = reinterpret_cast<const uint32_t*>(p)[lane + LANES];
                        s[u][1] = scale_value<FMT == EP_NVFP4>(sc[(lane + LANES) / kPer]);
                    }
                } else {
                    q[u][0] = reinterpret_cast<const uint2*>(p)[lane];
                    if (second[u]) q[u][1] = reinterpret_cast<const uint2*>(p)[lane + LANES];
                    s[u][0] = reinterpret_cast<const float*>(c.scales)[row];
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (!dst[u]) continue;
            float v[8];
            values8<FMT>(q[u][0].x, q[u][0].y, s[u][0], v);
            store8<DT>(dst[u], 8, 16, v);
            if (second[u]) {
                values8<FMT>(q[u][1].x, q[u][1].y, s[u][kFp4 ? 1 : 0], v);
                store8<DT>(dst[u] + 8 * LANES, 8, 16, v);
            }
        }
    }
}

// The same for any head: a warp a row, 8 elements a lane, at any alignment.
template <int DT, int FMT>
__global__ void __launch_bounds__(kThreads) cache_read_any_kernel(const __grid_constant__ ReadArgs a) {
    using T = typename Elem<DT>::T;
    __shared__ int32_t starts[kSharedSeqs + 1];
    __shared__ int64_t slot[kMaxReadTokens];
    wait_for_stream();
    const int64_t t0 = int64_t(blockIdx.x) * a.per_block;
    const int n = int(min(int64_t(a.per_block), a.tokens - t0));
    find_pages(a, t0, n, starts, slot);
    const int rows = n * a.heads, lane = threadIdx.x % 32;
    for (int r = threadIdx.x / 32; r < a.n * rows; r += kThreads / 32) {
        const int ci = r >= rows, t = quotient(r - ci * rows, a.heads_inv), h = r - ci * rows - t * a.heads;
        const CacheView& c = a.c[ci];
        const int64_t from = slot[t], row = from * a.heads + h;
        if (from == -2) continue;
        T* dst = static_cast<T*>(c.heads) + (t0 + t) * c.token_stride + h * c.head_stride;
        const uint8_t* data = c.data + row * c.row_bytes;
        for (int e = 8 * lane; e < c.head_dim; e += 256) {
            const int m = min(8, c.head_dim - e);
            uint32_t w[2] = {0, 0};
            float s = 0.0f, v[8];
            if (from >= 0) {
                if constexpr (FMT == EP_MXFP4 || FMT == EP_NVFP4) {
                    w[0] = *reinterpret_cast<const uint32_t*>(data + e / 2);
                    s = scale_value<FMT == EP_NVFP4>(c.scales[row * c.scale_bytes + e / (FMT == EP_NVFP4 ? 16 : 32)]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < m) w[j / 4] |= uint32_t(data[e + j]) << (8 * (j % 4));
                    s = reinterpret_cast<const float*>(c.scales)[row];
                }
            }
            values8<FMT>(w[0], w[1], s, v);
            store8<DT>(dst + e, m, c.width, v);
        }
    }
}

// ---- host side -----------------------------------------------------------------------------------
// What serves a call: the lanes of a row at 16 elements each, or 0 for any head.
int lanes_of(const CacheView* c, int n) {
    int dim = 0;
    for (int i = 0; i < n; ++i) {
        if (c[i].head_dim % 8 != 0 || c[i].head_dim > kMaxFastDim || c[i].width != 16) return 0;
        dim = std::max(dim, c[i].head_dim);
    }
    return dim <= 64 ? 4 : dim <= 128 ? 8 : 16;
}

template <int DT, int FMT>
cudaError_t launch_write(const WriteArgs& w, int lanes, dim3 grid, cudaStream_t st) {
    const auto kernel = lanes == 4   ? cache_write_kernel<DT, FMT, 4>
                        : lanes == 8 ? cache_write_kernel<DT, FMT, 8>
                        : lanes == 16 ? cache_write_kernel<DT, FMT, 16>
                                      : cache_write_any_kernel<DT, FMT>;
    const cudaError_t e = op::launch(kernel, grid, dim3(kThreads), 0, st, w);
    if (e != cudaSuccess || w.alone) return e;
    return op::launch(mend_kernel<DT, FMT>, dim3(unsigned(op::div_up(w.tokens, kMendTokens))), dim3(kMendThreads), 0, st, w);
}
template <int DT>
cudaError_t write_as(int fmt, const WriteArgs& w, int lanes, dim3 grid, cudaStream_t st) {
    switch (fmt) {
        case EP_FP8_E4M3: return launch_write<DT, EP_FP8_E4M3>(w, lanes, grid, st);
        case EP_INT8: return launch_write<DT, EP_INT8>(w, lanes, grid, st);
        case EP_MXFP4: return launch_write<DT, EP_MXFP4>(w, lanes, grid, st);
        default: return launch_write<DT, EP_NVFP4>(w, lanes, grid, st);
    }
}
template <int DT, int FMT>
cudaError_t launch_read(const ReadArgs& r, int lanes, dim3 grid, cudaStream_t st) {
    const auto kernel = lanes == 4   ? cache_read_kernel<DT, FMT, 4>
                        : lanes == 8 ? cache_read_kernel<DT, FMT, 8>
                        : lanes == 16 ? cache_read_kernel<DT, FMT, 16>
                                      : cache_read_any_kernel<DT, FMT>;
    return op::launch(kernel, grid, dim3(kThreads), 0, st, r);
}
template <int DT>
cudaError_t read_as(int fmt, const ReadArgs& r, int lanes, dim3 grid, cudaStream_t st) {
    switch (fmt) {
        case EP_FP8_E4M3: return launch_read<DT, EP_FP8_E4M3>(r, lanes, grid, st);
        case EP_INT8: return launch_read<DT, EP_INT8>(r, lanes, grid, st);
        case EP_MXFP4: return launch_read<DT, EP_MXFP4>(r, lanes, grid, st);
        default: return launch_read<DT, EP_NVFP4>(r, lanes, grid, st);
    }
}

// Checks caches and the tensors that go with them, and fills the views the kernels read.
int make_views(const ep_cache* caches, const ep_heads* h, int n, const char* who, CacheView* out) {
    const std::string w(who);
    for (int i = 0; i < n; ++i) {
        const ep_cache& c = caches[i];
        const ep_heads& x = h[i];
        const bool fp4 = op::is_fp4(c.format);
        if (!fp4 && c.format != EP_FP8_E4M3 && c.format != EP_INT8) return set_error(EP_ERR_DTYPE, w + ": unsupported cache format");
        const int es = op::elem_bytes(x.dtype);
        if (es == 0) return set_error(EP_ERR_DTYPE, w + ": heads must be EP_BF16, EP_FP16 or EP_F32");
        if (c.n_pages < 0 || c.page_size < 1 || c.heads < 1 || c.head_dim < 1 || c.head_dim > kMaxHeadDim || c.heads > 4096 ||
            c.n_pages > (int64_t(1) << 40) / c.page_size)
            return set_error(EP_ERR_SHAPE, w + ": cache geometry out of range");
        if (x.tokens < 0 || x.tokens > 0x7fffffff || x.heads != c.heads || x.head_dim != c.head_dim)
            return set_error(EP_ERR_SHAPE, w + ": heads do not match the cache");
        if (c.format != caches[0].format || c.n_pages != caches[0].n_pages || c.page_size != caches[0].page_size ||
            c.heads != caches[0].heads || x.tokens != h[0].tokens)
            return set_error(EP_ERR_SHAPE, w + ": the caches of one call differ in geometry");
        if (x.dtype != h[0].dtype) return set_error(EP_ERR_DTYPE, w + ": the heads of one call differ in type");
        if (x.token_stride < 0 || x.head_stride < 0) return set_error(EP_ERR_ARG, w + ": negative stride");
        if (c.n_pages > 0 && (!c.data || !c.scales || !op::aligned(c.data, 16) || !op::aligned(c.scales, fp4 ? 1 : 4)))
            return set_error(EP_ERR_ARG, w + ": cache data or scales are NULL or misaligned");
        if (x.tokens > 0 && (!x.data || !op::aligned(x.data, size_t(es))))
            return set_error(EP_ERR_ARG, w + ": heads are NULL or misaligned");
        CacheView& v = out[i];
        v.data = static_cast<uint8_t*>(c.data);
        v.scales = static_cast<uint8_t*>(c.scales);
        v.row_bytes = fp4 ? op::fp4_row_bytes(c.head_dim) : c.head_dim;
        v.scale_bytes = fp4 ? op::fp4_blocks(c.format, c.head_dim) : 4;
        v.heads = x.data;
        v.token_stride = x.token_stride;
        v.head_stride = x.head_stride;
        v.head_dim = c.head_dim;
        v.width = op::access_width(x.data, x.token_stride * es, x.head_stride * es);
    }
    return EP_OK;
}

// Whether two caches (of make_views) have bytes in common: a write's blocks for one would race with the other's.
bool share_bytes(const ep_cache* c, const CacheView* v) {
    struct Range { uintptr_t at, end; } r[2][2];
    for (int i = 0; i < 2; ++i) {
        const uintptr_t rows = uintptr_t(c[i].n_pages) * uintptr_t(c[i].page_size) * uintptr_t(c[i].heads);
        const uintptr_t data = reinterpret_cast<uintptr_t>(c[i].data), scales = reinterpret_cast<uintptr_t>(c[i].scales);
        r[i][0] = {data, data + rows * uintptr_t(v[i].row_bytes)};
        r[i][1] = {scales, scales + rows * uintptr_t(v[i].scale_bytes)};
    }
    for (const Range& x : r[0])
        for (const Range& y : r[1])
            if (x.at < y.end && y.at < x.end) return true;
    return false;
}

// Whether the rows lie apart: a token's heads within its stride, or a head's tokens within its own.
bool rows_apart(const ep_heads& h) {
    const int64_t t = h.tokens - 1, n = h.heads - 1, d = h.head_dim;
    const auto nested = [d](int64_t few, int64_t inner, int64_t many, int64_t outer) {  // few + 1 rows, inner apart, and so on
        return (few <= 0 || inner >= d) && (many <= 0 || (outer >= d && (few <= 0 || (outer - d) / few >= inner)));
    };
    return nested(n, h.head_stride, t, h.token_stride) || nested(t, h.token_stride, n, h.head_stride);
}

// The current device, which must be the caches' and heads' own.
int device_of(const ep_cache* caches, const ep_heads* h, int n, const char* who, int& sms) {
    int dev = 0;
    const int rc = op::current_device(dev, sms);
    if (rc != EP_OK) return rc;
    for (int i = 0; i < n; ++i)
        if (caches[i].device != dev || h[i].device != dev)
            return set_error(EP_ERR_ARG, std::string(who) + ": a tensor is not on the current device");
    return EP_OK;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_cache_write(const ep_cache* caches, const ep_heads* src, int n, const int64_t* slots, void* stream) {
    clear_error();
    if (!caches || !src || n < 1 || n > 2) return set_error(EP_ERR_ARG, "ep_cache_write: NULL argument, or not one or two caches");
    int sms = 0;
    WriteArgs w = {};
    int rc = make_views(caches, src, n, "ep_cache_write", w.c);
    if (rc != EP_OK) return rc;
    const int64_t tokens = src[0].tokens;
    if (tokens > 0 && (!slots || !op::aligned(slots, 8))) return set_error(EP_ERR_ARG, "ep_cache_write: slots are NULL or misaligned");
    if (n == 2 && share_bytes(caches, w.c)) return set_error(EP_ERR_ARG, "ep_cache_write: the two caches share memory");
    rc = device_of(caches, src, n, "ep_cache_write", sms);
    if (rc != EP_OK || tokens == 0 || caches[0].n_pages == 0) return rc;
    const int lanes = lanes_of(w.c, n);
    const int es = op::elem_bytes(src[0].dtype);
    w.n_slots = caches[0].n_pages * caches[0].page_size;
    w.n = n;
    w.heads = caches[0].heads;
    w.heads_inv = 1.0f / float(w.heads);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    for (int64_t t0 = 0; t0 < tokens; t0 += kLaunchTokens) {
        WriteArgs part = w;
        part.slots = slots + t0;
        part.tokens = std::min<int64_t>(kLaunchTokens, tokens - t0);
        for (int i = 0; i < n; ++i)
            part.c[i].heads = static_cast<uint8_t*>(w.c[i].heads) + t0 * w.c[i].token_stride * es;
        // a block's rows are one batch of its threads (16384 tokens of 8 heads of 128, int8: 26.9 us with these 16
        // tokens a block, 29.8 with 8, 27.5 with 32); few tokens are spread over the SMs
        const int batch = 4 * kThreads / std::max(lanes, 4) / w.heads;
        part.per_block = int(std::max<int64_t>(1, std::min<int64_t>({kMaxWriteTokens, batch, op::div_up(part.tokens, 2 * sms)})));
        part.alone = part.tokens <= kAloneTokens;
        const dim3 grid(unsigned(op::div_up(part.tokens, part.per_block)), unsigned(n));
        const cudaError_t e = src[0].dtype == EP_BF16   ? write_as<EP_BF16>(caches[0].format, part, lanes, grid, st)
                              : src[0].dtype == EP_FP16 ? write_as<EP_FP16>(caches[0].format, part, lanes, grid, st)
                                                        : write_as<EP_F32>(caches[0].format, part, lanes, grid, st);
        if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_cache_write: ") + cudaGetErrorString(e));
    }
    return EP_OK;
}

extern "C" int ep_cache_read(const ep_cache* caches, const ep_heads* out, int n, const int32_t* page_table, int64_t table_stride,
                             int64_t pages_per_seq, int n_seqs, const int32_t* cu_seqlens, void* stream) {
    clear_error();
    if (!caches || !out || n < 1 || n > 2) return set_error(EP_ERR_ARG, "ep_cache_read: NULL argument, or not one or two caches");
    int sms = 0;
    ReadArgs r = {};
    int rc = make_views(caches, out, n, "ep_cache_read", r.c);
    if (rc != EP_OK) return rc;
    if (n_seqs < 0 || pages_per_seq < 0 || table_stride < pages_per_seq)
        return set_error(EP_ERR_ARG, "ep_cache_read: bad sequence count or page table");
    if (!cu_seqlens || !op::aligned(cu_seqlens, 4) || (n_seqs > 0 && pages_per_seq > 0 && (!page_table || !op::aligned(page_table, 4))))
        return set_error(EP_ERR_ARG, "ep_cache_read: page_table or cu_seqlens is NULL or misaligned");
    for (int i = 0; i < n; ++i)
        if (!rows_apart(out[i])) return set_error(EP_ERR_ARG, "ep_cache_read: rows of out overlap");
    if (n == 2 && out[0].tokens > 0 && out[0].data == out[1].data)
        return set_error(EP_ERR_ARG, "ep_cache_read: the two outputs are one");
    rc = device_of(caches, out, n, "ep_cache_read", sms);
    if (rc != EP_OK || n_seqs == 0 || out[0].tokens == 0) return rc;
    r.page_table = page_table;
    r.table_stride = table_stride;
    r.pages_per_seq = pages_per_seq;
    r.n_pages = caches[0].n_pages;
    r.tokens = out[0].tokens;
    r.cu_seqlens = cu_seqlens;
    r.n_seqs = n_seqs;
    r.page_size = caches[0].page_size;
    r.heads = caches[0].heads;
    r.heads_inv = 1.0f / float(r.heads);
    r.n = n;
    // few tokens are spread over the SMs
    r.per_block = int(std::max<int64_t>(1, std::min<int64_t>(kMaxReadTokens, op::div_up(r.tokens, 4 * sms))));
    const dim3 grid(unsigned(op::div_up(r.tokens, r.per_block)));
    const int lanes = lanes_of(r.c, n);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = out[0].dtype == EP_BF16   ? read_as<EP_BF16>(caches[0].format, r, lanes, grid, st)
                          : out[0].dtype == EP_FP16 ? read_as<EP_FP16>(caches[0].format, r, lanes, grid, st)
                                                    : read_as<EP_F32>(caches[0].format, r, lanes, grid, st);
    if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_cache_read: ") + cudaGetErrorString(e));
    return EP_OK;
}
