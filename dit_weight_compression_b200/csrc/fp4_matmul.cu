// fp4_matmul.cu -- ep_fp4_matmul: out = a * transpose(b) + bias for two microscaled 4-bit matrices,
// on the block-scaled 4-bit tensor cores.
#include <algorithm>
#include <atomic>
#include <string>

#include "blob.h"
#include "fp4_shape.h"
#include "microscale.cuh"
#include "ops.h"
#include "tcgen05.cuh"

namespace ep {
namespace {

using namespace tc;

constexpr int kStepK = 256;     // elements of K a pipeline stage holds: 128 bytes of a row
constexpr int kThreads = 192;   // warp 0 copies, warp 1 issues products, warps 2 to 5 read the sums

// Sticky word of products that gave up a wait, read and cleared by ep_op_status.
__device__ uint32_t ep_op_status_word;

struct MatmulArgs {
    const uint8_t* a_scales;
    const uint8_t* b_scales;
    const float* ga;
    const float* gb;
    const void* bias;
    void* out;
    int64_t stride;            // of out's rows
    int64_t rows, cols;        // of out
    int scale_tiles;           // 512-byte scale tiles along K
    int steps;                 // stages along K
    int k64;                   // products of 64 along K
    int n_tiles;               // tiles of 128 rows of b
    int out_dtype;
    int width;                 // alignment of out's rows: 16, 8 or 4 bytes, or 1 for their elements'
    int gives_up;              // 0, or one more than the tile that acts as if a wait for its copies had run out
    uint32_t tries;            // limit of the waits of one role for another
};

// Tile sizes, stage layout and tensor memory columns of a variant with tiles of NT tokens.
template <int NT, bool NV>
struct Geo {
    static constexpr int kScaleTiles = NV ? 4 : 2;            // scale tiles of 128 rows x one stage
    static constexpr int kB = 128 * 128, kA = NT * 128;       // bytes of the operands' stage tiles
    static constexpr int kS = kScaleTiles * 512;              // and of each one's scales
    static constexpr int kStage = kB + kA + 2 * kS;
    static constexpr int kBudget = 113 * 1024 - 2048;         // two CTAs share an SM
    static constexpr int kStages = kBudget / kStage;
    static constexpr int kSum = NT < 32 ? 32 : NT;            // accumulator columns
    static constexpr int kScaleCols = 8 * kScaleTiles;        // of one stage
    static constexpr int kColumns = 256;
    static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + 256;
    static_assert(kStages >= 3, "a pipeline of at least three stages");
    static_assert(kSum + kStages * kScaleCols <= kColumns, "tensor memory");
    static_assert(kStage % 1024 == 0, "swizzled tiles start on 1024-byte boundaries");
    static_assert(kStages * kStage >= 128 * NT * 4, "partial sums fit the stages");
};

__device__ __forceinline__ float bias_at(const MatmulArgs& a, int64_t n) {
    if (!a.bias) return 0.0f;
    if (a.out_dtype == EP_F32) return static_cast<const float*>(a.bias)[n];
    if (a.out_dtype == EP_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[n]);
    return __half2float(static_cast<const __half*>(a.bias)[n]);
}

// Two factors of the product of the tensor scales, which need not be a float itself (two of 2^64, or a subnormal
// one beside a large one): a power of two is moved from the larger to the smaller until both are about the
// product's square root, or, where the smaller is subnormal, both at most 1.  A sum times the product, formed as
// (sum * x) * y, then passes through a number between the sum and the result, so that the first step neither
// overflows nor loses bits where the whole does not.  (y is brought below the normal floats only by products
// under 2^-250, whose results are 0: sums of NVFP4 stay below 2^53, and MXFP4's scale is 1.)
__device__ __forceinline__ float2 tensor_scales(float ga, float gb) {
    const bool ordered = fabsf(ga) <= fabsf(gb);
    const float x = ordered ? ga : gb, y = ordered ? gb : ga;
    const int d = min((ms::log2_floor(fabsf(y)) - ms::log2_floor(fabsf(x))) / 2, 126);
    return make_float2(x * ms::pow2f(d), y * ms::pow2f(-d));
}

// The first n of four neighbouring elements of row i from column j (a multiple of 4) on.
__device__ __forceinline__ void store4(const MatmulArgs& a, int64_t i, int64_t j, int n, const float* v) {
    const int64_t at = i * a.stride + j;
    if (a.out_dtype == EP_F32) {
        float* o = static_cast<float*>(a.out) + at;
        if (n == 4 && a.width == 16) {
            *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < n) o[k] = v[k];
        }
        return;
    }
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        w[k] = a.out_dtype == EP_BF16 ? ms::pack2<EP_BF16>(v[2 * k], v[2 * k + 1]) : ms::pack2<EP_FP16>(v[2 * k], v[2 * k + 1]);
    uint16_t* o = static_cast<uint16_t*>(a.out) + at;
    if (n == 4 && a.width >= 8) {
        *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < n) o[k] = uint16_t(w[k / 2] >> (16 * (k % 2)));
    }
}

// ---- short products -------------------------------------------------------------------------------
// One cluster per tile of 128 rows of b (the tensor core's lanes, so that few tokens do not leave them
// idle) x NT tokens; its CTAs share the stages along K and then the tile's tokens: each adds up its share
// of tokens over all CTAs' partial sums, in rank order, and writes runs of 128 outputs.  Two CTAs share an
// SM: the copies of one go on while the other starts or ends.  Bound by the reading of b: 1 x 28672 x 8192
// nvfp4 23 us, 5.7 TB/s; all sizes take 3.4 to 3.8 us and their bytes at about 6.5 TB/s.
template <int NT, bool NV>
__global__ void __launch_bounds__(kThreads, 2) fp4_split_kernel(const __grid_constant__ CUtensorMap b_map,
                                                                 const __grid_constant__ CUtensorMap a_map,
                                                                 const __grid_constant__ MatmulArgs a) {
    using G = Geo<NT, NV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const uint32_t base = smem_addr(smem);
    const uint32_t bars = base + G::kStages * G::kStage;  // full, empty of each stage; done; the TMEM address
    auto full = [&](int s) { return bars + 8 * s; };
    auto empty = [&](int s) { return bars + 8 * (G::kStages + s); };
    const uint32_t done = bars + 16 * G::kStages, slot = done + 8, lost = slot + 4;
    const int warp = int(uniform(threadIdx.x / 32)), lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank(), ranks = cluster_ranks();
    const int tile = int(blockIdx.x / ranks);
    const int n0 = (tile % a.n_tiles) * 128, m0 = (tile / a.n_tiles) * NT;
    const int k0 = int(int64_t(a.steps) * rank / ranks), steps = int(int64_t(a.steps) * (rank + 1) / ranks) - k0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        bar_init(done, 1);
        store_u32(lost, 0);
        prefetch_map(&b_map);
        prefetch_map(&a_map);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc(slot, G::kColumns);
    fence_before();
    __syncthreads();
    fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));
    tmem = uniform(tmem);
    // The weights' first two stages on their way to L2 while the kernel that makes the activations ends (one
    // token quantised and 28672 x 8192: 25.5 -> 25.0 us in all; with five stages the product alone loses up
    // to 0.6 us to asking twice).
    if (warp == 0 && elect_one())
        for (int it = 0; it < min(steps, 2); ++it) {
            const int k = k0 + it;
            prefetch_2d(&b_map, 128 * k, n0);
            prefetch_bulk(a.b_scales + (int64_t(n0 / 128) * a.scale_tiles + int64_t(k) * G::kScaleTiles) * 512,
                          512 * min(G::kScaleTiles, a.scale_tiles - k * G::kScaleTiles));
        }
    __syncwarp();
    ms::wait_for_stream();

    bool ok = true;
    if (warp == 0) {
        const bool leader = elect_one();
        int issued = 0;
        for (int it = 0; it < steps; ++it) {
            const int s = it % G::kStages, k = k0 + it;
            if (it >= G::kStages && !(ok = bar_wait(empty(s), (it / G::kStages - 1) & 1))) break;
            const int bytes = 512 * min(G::kScaleTiles, a.scale_tiles - k * G::kScaleTiles);
            const uint32_t st = base + s * G::kStage;
            const int64_t at = int64_t(k) * G::kScaleTiles;
            if (leader) {
                bar_expect(full(s), G::kB + G::kA + 2 * bytes);
                tma_2d(st, &b_map, 128 * k, n0, full(s));
                bulk_copy(st + G::kB + G::kA, a.b_scales + (int64_t(n0 / 128) * a.scale_tiles + at) * 512, bytes, full(s));
                tma_2d(st + G::kB, &a_map, 128 * k, m0, full(s));
                bulk_copy(st + G::kB + G::kA + G::kS, a.a_scales + (int64_t(m0 / 128) * a.scale_tiles + at) * 512, bytes, full(s));
            }
            issued = it + 1;
        }
        // nothing may still be on its way into this CTA's memory when it leaves
        for (int it = max(0, issued - G::kStages); it < issued; ++it) ok &= bar_wait(full(it % G::kStages), (it / G::kStages) & 1);
    } else if (warp == 1) {
        const bool leader = elect_one();
        for (int it = 0; it < steps; ++it) {
            const int s = it % G::kStages;
            if (!(ok = bar_wait(full(s), (it / G::kStages) & 1))) break;
            fence_after();
            const uint32_t st = base + s * G::kStage;
            const uint32_t sb = tmem + G::kSum + s * G::kScaleCols, sa = sb + 4 * G::kScaleTiles;
            const uint32_t db = operand_low(st), da = operand_low(st + G::kB), ds = scale_low(st + G::kB + G::kA);
            const int products = min(4, a.k64 - 4 * (k0 + it)), tiles = NV ? products : (products + 1) / 2;
            if (leader) {
#pragma unroll
                for (int t = 0; t < G::kScaleTiles; ++t)
                    if (t < tiles) {
                        copy_scales(sb + 4 * t, desc(ds + 32 * t, kScaleHigh));
                        copy_scales(sa + 4 * t, desc(ds + (G::kS >> 4) + 32 * t, kScaleHigh));
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < products) {
                        const int t = NV ? j : j / 2;
                        mma_fp4<NV>(tmem, desc(db + 2 * j, kOperandHigh), desc(da + 2 * j, kOperandHigh), mma_fp4_idesc<NV>(NT, j % 2),
                                    sb + 4 * t, sa + 4 * t, it > 0 || j > 0);
                    }
                commit(empty(s));
            }
        }
        if (leader) commit(done);
        if (a.gives_up == tile + 1 && rank == ranks - 1) ok = false;
    }
    __syncwarp();
    // every warp: the sums are ready, and no copy or product uses the stages any more
    ok &= bar_wait(done, 0);
    fence_after();
    if (!ok) store_u32(lost, 1);  // some of these sums are not whole

    const float ga = *a.ga, gb = *a.gb;
    float* part = reinterpret_cast<float*>(smem);  // [token][row of b]
    if (warp >= 2) {
        const int row = (warp % 4) * 32 + lane;
        for (int c = 0; c < NT; c += 16) {
            uint32_t r[16];
            tmem_load16(tmem + (uint32_t(warp % 4) << 21) + c, r);
            tmem_wait_load();
#pragma unroll
            for (int j = 0; j < 16; ++j) part[(c + j) * 128 + row] = __uint_as_float(r[j]);
        }
    }
    fence_before();
    __syncwarp();
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    const uint32_t missing = uint32_t(lane) < ranks ? peer_load_u32(lost, uint32_t(lane)) : 0;  // of each CTA
    const float2 g = tensor_scales(ga, gb);
    const int c0 = NT * int(rank) / int(ranks), c1 = NT * (int(rank) + 1) / int(ranks);
    const int64_t col = int64_t(n0) + 4 * lane;
    const int n = int(max(int64_t(0), min(int64_t(4), a.cols - col)));
    float bias[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) bias[j] = j < n ? bias_at(a, col + j) : 0.0f;
    for (int c = c0 + warp; c < c1 && int64_t(m0) + c < a.rows; c += kThreads / 32) {
        float v[4] = {};
        for (uint32_t r = 0; r < ranks; ++r) {
            const float4 f = peer_load4(base + 4 * (c * 128 + 4 * lane), r);
            v[0] += f.x;
            v[1] += f.y;
            v[2] += f.z;
            v[3] += f.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fmaf_rn(v[j] * g.x, g.y, bias[j]);
        // a tile with a part missing is not written (asked here, where the loads of the sums have covered the answer's way)
        if (!__any_sync(ms::kFullMask, missing) && n > 0) store4(a, int64_t(m0) + c, col, n, v);
    }
    __syncwarp();
    if (ranks > 1) cluster_sync();  // no CTA leaves while another reads its sums
    else __syncthreads();
    fence_after();
    if (!ok) atomicOr(&ep_op_status_word, 1u);
    if (warp == 2) tmem_free(tmem, G::kColumns);
}

// ---- long products ---------------------------------------------------------------------------------
// Persistent pairs of CTAs, each pair on tiles of 256 x 256: a CTA holds 128 rows of a (the tensor core's
// lanes) and half of the tile's rows of b, so that of every operand byte brought to an SM twice as much is
// used as by a CTA alone.  Warp 0 copies, warp 1 of the first CTA issues products for both, warps 2 to 9
// take the sums: they read all of them into registers, give the accumulator back, and write while the next
// tile's products run.  (Tensor memory: 256 columns of sums leave 256 for scales, so the accumulator is
// single; handing it back before it is read, which is wrong, would save nothing measurable.)
// 8192 x 28672 x 8192 nvfp4: 677 to 687 us in bursts of three, 5.6 PFLOP/s.  Its copies from L2 bind it (without
// them 4096 x 9472 x 8192 takes 23% less), then the board's power: in loops of a second the clock falls and
// the large product takes 790 to 820 us.
template <bool NV>
struct PairGeo {
    static constexpr int kScaleTiles = NV ? 4 : 2;
    static constexpr int kOperand = 128 * 128;                 // a's rows, and as much of b
    static constexpr int kAS = kScaleTiles * 512, kBS = 2 * kScaleTiles * 512;
    static constexpr int kStage = 2 * kOperand + kAS + kBS;
    static constexpr int kStages = 5;
    static constexpr int kScaleCols = 4 * kScaleTiles * 3;
    static constexpr int kOut = 4096;                          // a reading warp's outputs on their way
    static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + 8 * kOut + 256;
    static constexpr int kThreads = 320;
    static_assert(256 + kStages * kScaleCols <= 512, "tensor memory");
    static_assert(kSmem <= 227 * 1024, "shared memory");
};

struct PairArgs {
    MatmulArgs m;
    int a_tiles, b_tiles;     // tiles of 256 rows
    int group;                // tiles of a taken together before the next tiles of b
};

// A warp's 32 rows x 128 bytes of outputs, one row a lane in registers, to memory: through 4 KB of shared
// memory (16-byte pieces, exclusive-ored with the row against bank conflicts), so that the lanes write
// neighbouring bytes of a row.  A lane storing its own row's 16 bytes took 7 us of a 256 x 256 bf16 tile;
// this way it is 3 to 4, which the next tile's products hide from about 2048 columns of K on.
__device__ __forceinline__ void store_rows(const MatmulArgs& m, uint32_t buf, int lane, int64_t row0, int64_t col, const uint32_t* w) {
    const int size = m.out_dtype == EP_F32 ? 4 : 2, per = 128 / size;  // columns
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + 128 * lane + 16 * (i ^ (lane & 7))), "r"(w[4 * i]),
                     "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                     : "memory");
    __syncwarp();
    const int rows = int(max(int64_t(0), min(int64_t(32), m.rows - row0))), cols = int(max(int64_t(0), min(int64_t(per), m.cols - col)));
    uint8_t* out = static_cast<uint8_t*>(m.out) + (row0 * m.stride + col) * size;
    if (m.width == 16 && cols == per) {
        const int c = lane % 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + lane / 8;
            uint4 u;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                         : "r"(buf + 128 * r + 16 * (c ^ (r & 7))));
            if (r < rows) *reinterpret_cast<uint4*>(out + r * m.stride * size + 16 * c) = u;
        }
        return;
    }
    // rows that start anywhere, or the last columns
    for (int r = 0; r < rows; ++r) {
        const uint32_t line = buf + 128 * r;
        if (size == 4 || (m.width >= 4 && cols % 2 == 0)) {
            uint32_t u;
            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(u) : "r"(line + 16 * ((lane / 4) ^ (r & 7)) + 4 * (lane % 4)));
            if (4 * lane < cols * size) *reinterpret_cast<uint32_t*>(out + r * m.stride * size + 4 * lane) = u;
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int c = lane + 32 * e;
                uint16_t u;
                asm volatile("ld.shared.b16 %0, [%1];" : "=h"(u) : "r"(line + 16 * ((c / 8) ^ (r & 7)) + 2 * (c % 8)));
                if (c < cols) *reinterpret_cast<uint16_t*>(out + r * m.stride * size + 2 * c) = u;
            }
        }
    }
}

// The t-th tile: columns of `group` tiles of a, so that what runs at one time shares operands in L2.
__device__ __forceinline__ void pair_tile(const PairArgs& a, int t, int& ta, int& tb) {
    const int per = a.group * a.b_tiles, g = t / per, rows = min(a.group, a.a_tiles - g * a.group), r = t - g * per;
    tb = r / rows;
    ta = g * a.group + (r - tb * rows);
}

template <bool NV>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairGeo<NV>::kThreads, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap b_map,
                    const __grid_constant__ CUtensorMap as_map, const __grid_constant__ CUtensorMap bs_map,
                    const __grid_constant__ PairArgs args) {
    using G = PairGeo<NV>;
    const MatmulArgs& m = args.m;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    const uint32_t out_bufs = base + G::kStages * G::kStage, bars = out_bufs + 8 * G::kOut;
    auto full = [&](int s) { return bars + 8 * s; };  // used in the first CTA
    auto empty = [&](int s) { return bars + 8 * (G::kStages + s); };
    const uint32_t summed = bars + 16 * G::kStages, taken = summed + 8, drained = taken + 8, slot = drained + 8;
    const int warp = int(uniform(threadIdx.x / 32)), lane = threadIdx.x % 32;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x / 2, pairs = gridDim.x / 2, tiles = args.a_tiles * args.b_tiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < G::kStages; ++s) {
            bar_init(full(s), 1);
            bar_init(empty(s), 1);
        }
        bar_init(summed, 1);
        bar_init(taken, 16);  // the 8 reading warps of both CTAs
        bar_init(drained, 1);
        prefetch_map(&a_map);
        prefetch_map(&b_map);
        prefetch_map(&as_map);
        prefetch_map(&bs_map);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tmem_alloc_pair(slot, 512);
    fence_before();
    __syncthreads();
    cluster_sync();
    fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));
    tmem = uniform(tmem);
    ms::wait_for_stream();

    bool ok = true;
    if (warp == 0) {
        const bool leader = elect_one();
        const uint32_t first = uniform(first_cta(bars));
        int it = 0;
        for (int t = pair; t < tiles && ok; t += pairs) {
            int ta, tb;
            pair_tile(args, t, ta, tb);
            const int a_row = 256 * ta + 128 * int(rank), b_row = 256 * tb + 128 * int(rank);
            const int a_scales = (2 * ta + int(rank)) * m.scale_tiles, b_scales = 2 * tb * m.scale_tiles;
            for (int k = 0; k < m.steps; ++k, ++it) {
                const int s = it % G::kStages;
                if (it >= G::kStages && !(ok = bar_wait(empty(s), (it / G::kStages - 1) & 1, m.tries))) break;
                const uint32_t st = base + s * G::kStage;
                if (leader) {
                    if (rank == 0) bar_expect(full(s), 2 * G::kStage);
                    tma_2d_pair(st, &a_map, 128 * k, a_row, first + 8 * s);
                    tma_2d_pair(st + G::kOperand, &b_map, 128 * k, b_row, first + 8 * s);
                    tma_2d_pair(st + 2 * G::kOperand, &as_map, 0, a_scales + G::kScaleTiles * k, first + 8 * s);
                    tma_2d_pair(st + 2 * G::kOperand + G::kAS, &bs_map, 0, b_scales + G::kScaleTiles * k, first + 8 * s);
                    tma_2d_pair(st + 2 * G::kOperand + 2 * G::kAS, &bs_map, 0, b_scales + m.scale_tiles + G::kScaleTiles * k, first + 8 * s);
                }
            }
        }
        // nothing may still be on its way into this CTA's memory when it leaves: every stage that was
        // filled has been used (both CTAs see that), or on giving up at least arrived (the first does)
        for (int i = max(0, it - G::kStages); i < it; ++i) {
            if (rank == 0) ok &= bar_wait(full(i % G::kStages), (i / G::kStages) & 1);
            if (ok) ok &= bar_wait(empty(i % G::kStages), (i / G::kStages) & 1);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const bool leader = elect_one();
            int it = 0, n = 0;
            for (int t = pair; t < tiles && ok; t += pairs, ++n) {
                if (n > 0 && !(ok = bar_wait(taken, (n - 1) & 1, m.tries))) break;
                fence_after();
                for (int k = 0; k < m.steps; ++k, ++it) {
                    const int s = it % G::kStages;
                    if (!(ok = bar_wait(full(s), (it / G::kStages) & 1, m.tries))) break;
                    fence_after();
                    const uint32_t st = base + s * G::kStage;
                    const uint32_t sa = tmem + 256 + s * G::kScaleCols, sb = sa + 4 * G::kScaleTiles;
                    const uint32_t da = operand_low(st), db = operand_low(st + G::kOperand), ds = scale_low(st + 2 * G::kOperand);
                    const int products = min(4, m.k64 - 4 * k), scales = NV ? products : (products + 1) / 2;
                    if (leader) {
#pragma unroll
                        for (int j = 0; j < G::kScaleTiles; ++j)
                            if (j < scales) {
                                copy_scales<2>(sa + 4 * j, desc(ds + 32 * j, kScaleHigh));
                                copy_scales<2>(sb + 8 * j, desc(ds + (G::kAS >> 4) + 32 * j, kScaleHigh));
                                copy_scales<2>(sb + 8 * j + 4, desc(ds + (2 * G::kAS >> 4) + 32 * j, kScaleHigh));
                            }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (j < products)
                                mma_fp4<NV, 2>(tmem, desc(da + 2 * j, kOperandHigh), desc(db + 2 * j, kOperandHigh),
                                               mma_fp4_idesc<NV, 2>(256, j % 2), sa + 4 * (NV ? j : j / 2), sb + 8 * (NV ? j : j / 2),
                                               k > 0 || j > 0);
                        commit_pair(empty(s));
                    }
                }
                if (m.gives_up == t + 1) ok = false;
                if (!ok) break;  // sums of which a part is missing are not handed on: the readers give up as well
                if (leader) commit_pair(summed);
            }
            if (!ok) {  // the products on their way end before anything is taken down
                if (leader) commit_pair(drained);
                __syncwarp();
                bar_wait(drained, 0);
            }
        }
    } else {
        const float2 g = tensor_scales(*m.ga, *m.gb);
        const int quarter = warp % 4, half = (warp - 2) / 4;  // 32 lanes x 128 columns a warp
        int n = 0;
        for (int t = pair; t < tiles; t += pairs, ++n) {
            int ta, tb;
            pair_tile(args, t, ta, tb);
            if (!(ok = bar_wait(summed, n & 1, m.tries))) break;
            fence_after();
            uint32_t r[8][16];
#pragma unroll
            for (int c = 0; c < 8; ++c) tmem_load16(tmem + (uint32_t(quarter) << 21) + 128 * half + 16 * c, r[c]);
            tmem_wait_load();
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive_cluster(first_cta(taken));
            const int64_t row0 = int64_t(256) * ta + 128 * int(rank) + 32 * quarter, col = int64_t(256) * tb + 128 * half;
            const uint32_t buf = out_bufs + (warp - 2) * G::kOut;
            if (m.bias) {  // the warp's 128 columns', through its buffer
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int c = 32 * j + lane;
                    const float v = col + c < m.cols ? bias_at(m, col + c) : 0.0f;
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(buf + 4 * c), "f"(v) : "memory");
                }
                __syncwarp();
#pragma unroll
                for (int c = 0; c < 128; c += 4) {
                    float v[4];
                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                                 : "r"(buf + 4 * c));
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        r[c / 16][c % 16 + j] = __float_as_uint(__fmaf_rn(__uint_as_float(r[c / 16][c % 16 + j]) * g.x, g.y, v[j]));
                }
            } else {
#pragma unroll
                for (int c = 0; c < 128; ++c) r[c / 16][c % 16] = __float_as_uint(__uint_as_float(r[c / 16][c % 16]) * g.x * g.y);
            }
            if (m.out_dtype == EP_F32) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (col + 32 * c < m.cols) store_rows(m, buf, lane, row0, col + 32 * c, &r[2 * c][0]);
            } else {
#pragma unroll
                for (int c = 0; c < 64; ++c) {
                    const float lo = __uint_as_float(r[c / 8][2 * (c % 8)]), hi = __uint_as_float(r[c / 8][2 * (c % 8) + 1]);
                    r[c / 16][c % 16] = m.out_dtype == EP_BF16 ? ms::pack2<EP_BF16>(lo, hi) : ms::pack2<EP_FP16>(lo, hi);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (col + 64 * c < m.cols) store_rows(m, buf, lane, row0, col + 64 * c, &r[2 * c][0]);
            }
        }
    }
    __syncwarp();
    if (!ok) atomicOr(&ep_op_status_word, 1u);
    fence_before();
    cluster_sync();  // no CTA leaves while the other still uses its memory or barriers
    fence_after();
    if (warp == 2) tmem_free_pair(tmem, 512);
}

// A product without columns: out is the bias, or zero.
__global__ void __launch_bounds__(256) bias_kernel(const MatmulArgs a, int64_t rows, int64_t cols) {
    ms::wait_for_stream();
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < rows * cols; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / cols, c = i - r * cols;
        const float v = bias_at(a, c);
        const int64_t at = r * a.stride + c;
        if (a.out_dtype == EP_F32) static_cast<float*>(a.out)[at] = v;
        else if (a.out_dtype == EP_BF16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
        else static_cast<__half*>(a.out)[at] = __float2half_rn(v);
    }
}

// A wait that can only give up: a barrier that nothing arrives on.
__global__ void __launch_bounds__(32) wait_probe_kernel(uint32_t tries) {
    __shared__ __align__(8) uint64_t bar;
    ms::wait_for_stream();
    if (threadIdx.x == 0) bar_init(smem_addr(&bar), 1);
    __syncthreads();
    if (!bar_wait(smem_addr(&bar), 0, tries)) atomicOr(&ep_op_status_word, 1u);
}

// ---- host side -------------------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return EncodeTiled(nullptr);
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// Packed rows in boxes of 128 bytes x `box_rows`, swizzled; what lies outside reads as zeros.
bool operand_map(CUtensorMap* map, const ep_fp4_tensor* t, int box_rows) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t row = cuuint64_t(op::fp4_row_bytes(t->cols));
    const cuuint64_t dims[2] = {row, cuuint64_t(t->rows)}, strides[1] = {row};
    const cuuint32_t box[2] = {128, cuuint32_t(box_rows)}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, t->data, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of `split` CTAs of a variant that fit the device at one time (looked up once; 0: none does), after
// setting its kernel's shared memory.
template <int NT, bool NV>
cudaError_t clusters_of(int dev, int split, int& clusters) {
    static std::atomic<int> known[kMaxDevices][fp4::kMaxSplit + 1];
    clusters = known[dev][split].load(std::memory_order_relaxed);
    if (clusters > 0) return cudaSuccess;
    const auto kernel = fp4_split_kernel<NT, NV>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(Geo<NT, NV>::kSmem));
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(split));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Geo<NT, NV>::kSmem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = unsigned(split);
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg);
    }
    if (e == cudaSuccess) known[dev][split].store(clusters, std::memory_order_relaxed);
    return e;
}

// Scale tiles of 512 bytes, `box` of them at a time.
bool scale_map(CUtensorMap* map, const ep_fp4_tensor* t, int scale_tiles, int box) {
    const EncodeTiled fn = encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[2] = {128, cuuint64_t(op::div_up(t->rows, 128)) * cuuint64_t(scale_tiles)}, strides[1] = {512};
    const cuuint32_t size[2] = {128, cuuint32_t(box)}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, t->scales, dims, strides, size, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pairs of CTAs that fit the device at one time (looked up once; 0: none does), after setting the kernel's shared memory.
template <bool NV>
cudaError_t pairs_of(int dev, int& pairs) {
    static std::atomic<int> known[kMaxDevices];
    pairs = known[dev].load(std::memory_order_relaxed);
    if (pairs > 0) return cudaSuccess;
    const auto kernel = fp4_pair_kernel<NV>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(PairGeo<NV>::kSmem));
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(PairGeo<NV>::kThreads);
        cfg.dynamicSmemBytes = PairGeo<NV>::kSmem;
        e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
    }
    if (e == cudaSuccess) known[dev].store(pairs, std::memory_order_relaxed);
    return e;
}

template <bool NV>
int run_pairs(const ep_fp4_tensor* a, const ep_fp4_tensor* b, const MatmulArgs& args, int pairs, cudaStream_t st) {
    CUtensorMap a_map, b_map, as_map, bs_map;
    if (!operand_map(&a_map, a, 128) || !operand_map(&b_map, b, 128) ||
        !scale_map(&as_map, a, args.scale_tiles, PairGeo<NV>::kScaleTiles) ||
        !scale_map(&bs_map, b, args.scale_tiles, PairGeo<NV>::kScaleTiles))
        return set_error(EP_ERR_CUDA, "ep_fp4_matmul: tensor map");
    PairArgs p = {args};
    p.a_tiles = int(op::div_up(a->rows, 256));
    p.b_tiles = int(op::div_up(b->rows, 256));
    // as many tiles of a as keep within about a quarter of L2; b's are then read from memory once for every
    // `group` of them (8192 x 28672 x 8192: 745 us with 4, 710 with 8, 691 with 16, 694 with 32)
    p.group = int(std::max<int64_t>(4, std::min<int64_t>(16, (int64_t(32) << 20) / (256 * op::fp4_row_bytes(a->cols)))));
    if (int64_t(p.a_tiles) * p.b_tiles > 0x7fffffff) return set_error(EP_ERR_SHAPE, "ep_fp4_matmul: too many tiles");
    const cudaError_t e = op::launch(fp4_pair_kernel<NV>, dim3(unsigned(2 * std::min(pairs, p.a_tiles * p.b_tiles))),
                                     dim3(PairGeo<NV>::kThreads), PairGeo<NV>::kSmem, st, a_map, b_map, as_map, bs_map, p);
    if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_fp4_matmul: ") + cudaGetErrorString(e));
    return EP_OK;
}

template <int NT, bool NV>
cudaError_t split_of(int dev, int64_t tiles, int steps, int& split) {
    return fp4::split_of(tiles, steps, [dev](int n, int& clusters) { return clusters_of<NT, NV>(dev, n, clusters); },
                         cudaErrorInvalidConfiguration, split);
}

template <int NT, bool NV>
int run_split(const ep_fp4_tensor* a, const ep_fp4_tensor* b, const MatmulArgs& args, int dev, cudaStream_t st) {
    using G = Geo<NT, NV>;
    CUtensorMap b_map, a_map;
    if (!operand_map(&b_map, b, 128) || !operand_map(&a_map, a, NT)) return set_error(EP_ERR_CUDA, "ep_fp4_matmul: tensor map");
    const int64_t tiles = int64_t(args.n_tiles) * op::div_up(a->rows, NT);
    int split = 1;
    cudaError_t e = split_of<NT, NV>(dev, tiles, args.steps, split);
    const int64_t grid = tiles * split;
    if (grid > 0x7fffffff) return set_error(EP_ERR_SHAPE, "ep_fp4_matmul: too many tiles");
    if (e == cudaSuccess) {
        e = op::launch_clusters(fp4_split_kernel<NT, NV>, dim3(unsigned(grid)), dim3(kThreads), G::kSmem, split, st, b_map, a_map, args);
    }
    if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_fp4_matmul: ") + cudaGetErrorString(e));
    return EP_OK;
}

template <bool NV>
int matmul(const ep_fp4_tensor* a, const ep_fp4_tensor* b, const MatmulArgs& args, int dev, cudaStream_t st) {
    const int64_t m = a->rows;
    if (m <= 16) return run_split<16, NV>(a, b, args, dev, st);
    if (m <= 32) return run_split<32, NV>(a, b, args, dev, st);
    if (m <= 64) return run_split<64, NV>(a, b, args, dev, st);
    // More than 128 tokens go in pairs, unless there are so few outputs that each tile's sum along K is
    // worth sharing among three CTAs or more (200 tokens, 2048 outputs of 8192: 7.7 us so, 14.1 in pairs;
    // 256, 4096 of 4096: 8.9 and 9.8; 384, which can share by two only: 10.5 and 10.0; 130, 28672 of 1024:
    // 13.9 and 10.1).
    // Without room for a pair of CTAs (a part of a GPU) every product is a short one.
    int split = fp4::kMaxSplit, pairs = 0;
    if (m > 128) {
        cudaError_t e = split_of<128, NV>(dev, int64_t(args.n_tiles) * op::div_up(m, 128), args.steps, split);
        if (e == cudaSuccess && split < 3) e = pairs_of<NV>(dev, pairs);
        if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_fp4_matmul: ") + cudaGetErrorString(e));
    }
    if (pairs == 0) return run_split<128, NV>(a, b, args, dev, st);
    return run_pairs<NV>(a, b, args, pairs, st);
}

}  // namespace
}  // namespace ep

using namespace ep;

namespace {

int product(const ep_fp4_tensor* a, const ep_fp4_tensor* b, const void* bias, const ep_tensor* out, int gives_up, uint32_t tries, void* stream) {
    clear_error();
    if (!a || !b || !out) return set_error(EP_ERR_ARG, "ep_fp4_matmul: NULL argument");
    int rc = op::check_fp4(a, "ep_fp4_matmul");
    if (rc == EP_OK) rc = op::check_fp4(b, "ep_fp4_matmul");
    if (rc != EP_OK) return rc;
    if (a->format != b->format) return set_error(EP_ERR_DTYPE, "ep_fp4_matmul: the operands differ in format");
    if (a->cols != b->cols) return set_error(EP_ERR_SHAPE, "ep_fp4_matmul: the operands differ in columns");
    const int es = op::elem_bytes(out->dtype);
    if (es == 0) return set_error(EP_ERR_DTYPE, "ep_fp4_matmul: the output must be EP_BF16, EP_FP16 or EP_F32");
    if (out->rows != a->rows || out->cols != b->rows) return set_error(EP_ERR_SHAPE, "ep_fp4_matmul: output shape");
    if (bias && !op::aligned(bias, size_t(es))) return set_error(EP_ERR_ARG, "ep_fp4_matmul: the bias is misaligned");
    const bool empty = out->rows == 0 || out->cols == 0;
    if (!empty && (!out->data || !op::aligned(out->data, size_t(es)) || out->row_stride < out->cols))
        return set_error(EP_ERR_ARG, "ep_fp4_matmul: bad output pointer or row stride");
    int dev = 0, sms = 0;
    rc = op::current_device(dev, sms);
    if (rc != EP_OK) return rc;
    if (a->device != dev || b->device != dev || out->device != dev)
        return set_error(EP_ERR_ARG, "ep_fp4_matmul: a tensor is not on the current device");
    if (empty) return EP_OK;
    MatmulArgs args = {};
    args.gives_up = gives_up;
    args.tries = tries;
    args.ga = a->tensor_scale;
    args.gb = b->tensor_scale;
    args.bias = bias;
    args.out = out->data;
    args.stride = out->row_stride;
    args.out_dtype = out->dtype;
    args.rows = out->rows;
    args.cols = out->cols;
    args.a_scales = static_cast<const uint8_t*>(a->scales);
    args.b_scales = static_cast<const uint8_t*>(b->scales);
    args.n_tiles = int(op::div_up(b->rows, 128));
    args.width = op::access_width(out->data, out->row_stride * es);
    args.steps = int(op::div_up(a->cols, kStepK));
    args.k64 = int(op::div_up(a->cols, 64));
    args.scale_tiles = int(op::div_up(op::fp4_blocks(a->format, a->cols), 4));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->cols == 0) {
        const int64_t n = out->rows * out->cols;
        const cudaError_t e =
            op::launch(bias_kernel, dim3(unsigned(std::min<int64_t>(op::div_up(n, 256), 8 * sms))), dim3(256), 0, st, args, out->rows, out->cols);
        if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_fp4_matmul: ") + cudaGetErrorString(e));
        return EP_OK;
    }
    return a->format == EP_NVFP4 ? matmul<true>(a, b, args, dev, st) : matmul<false>(a, b, args, dev, st);
}

}  // namespace

extern "C" int ep_fp4_matmul(const ep_fp4_tensor* a, const ep_fp4_tensor* b, const void* bias, const ep_tensor* out, void* stream) {
    return product(a, b, bias, out, 0, kWaitTries, stream);
}

extern "C" int ep_fp4_matmul_probe(const ep_fp4_tensor* a, const ep_fp4_tensor* b, const ep_tensor* out, int tile, uint32_t wait_tries,
                                   void* stream) {
    if (tile < 0 || tile == 0x7fffffff || wait_tries == 0) {
        clear_error();
        return set_error(EP_ERR_ARG, "ep_fp4_matmul_probe: bad tile or zero limit");
    }
    return product(a, b, nullptr, out, tile + 1, wait_tries, stream);
}

extern "C" int ep_op_wait_probe(uint32_t wait_tries, void* stream) {
    clear_error();
    if (wait_tries == 0) return set_error(EP_ERR_ARG, "ep_op_wait_probe: zero limit");
    const cudaError_t e = op::launch(wait_probe_kernel, dim3(1), dim3(32), 0, static_cast<cudaStream_t>(stream), wait_tries);
    if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_op_wait_probe: ") + cudaGetErrorString(e));
    return EP_OK;
}

extern "C" int ep_op_status(void* stream) {
    clear_error();
    uint32_t word = 0;
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, ep_op_status_word, sizeof(word));
    const uint32_t zero = 0;
    if (e == cudaSuccess && word) e = cudaMemcpyToSymbol(ep_op_status_word, &zero, sizeof(zero));
    if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_op_status: ") + cudaGetErrorString(e));
    if (word) return set_error(EP_ERR_CUDA, "a 4-bit product gave up waiting; its output is incomplete");
    return EP_OK;
}
