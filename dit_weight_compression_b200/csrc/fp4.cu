// fp4.cu -- the microscaled 4-bit container: ep_fp4_sizes, ep_fp4_quantize, ep_fp4_dequantize and
// ep_decompress_fp4.  The formats are defined in entropack.h, their arithmetic in microscale.cuh.
#include <algorithm>
#include <cmath>
#include <string>

#include "blob.h"
#include "microscale.cuh"
#include "ops.h"

namespace ep {
namespace {

using namespace ms;

constexpr int kTileRows = 128;   // a block handles 128 rows x 128 columns: whole 512-byte scale
constexpr int kTileCols = 128;   // tiles (two for blocks of 16), written at once
constexpr int kThreads = 256;
constexpr int kPassRows = kThreads / (kTileCols / 8);  // dequantising: 16 threads a row, 8 elements each
constexpr int kPasses = kTileRows / kPassRows;
constexpr int kMaxPartials = EP_FP4_SCALE_FLOATS - 1;

// How the rows of a dense matrix lie: 16-byte aligned and whole (in sixteens, or eights when written); at
// least 8-byte aligned; anywhere.
enum Rows { kWhole, kEven, kAnywhere };

struct QuantArgs {
    const void* x;
    int64_t stride, rows, cols;
    uint8_t* data;
    uint8_t* scales;
    float* tensor_scale;
    int64_t row_bytes;
    int col_tiles;    // blocks side by side
    int scale_tiles;  // 512-byte scale tiles side by side
    float fixed;      // > 0: the tensor scale
    int partials;     // > 0: its maxima are in tensor_scale[1 ..]; 0 and no fixed scale: each block
                      // looks at all of x
    int width;        // alignment of the rows for load_raw8
    int start_width;  // and of the first element
    bool backwards;   // take the last rows first
};

// The largest finite |v| of eight, as bits.
template <int DT>
__device__ __forceinline__ uint32_t finite_max8(const Raw8<DT>& r) {
    uint32_t m = abs_max8(r);
    if (m >= AbsBits<DT>::kInf) {
        m = 0;
        constexpr uint32_t kMask = DT == EP_F32 ? 0x7fffffffu : 0x7fffu;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t w = (DT == EP_F32 ? r.w[j] : r.w[j / 2] >> (16 * (j % 2))) & kMask;
            if (w < AbsBits<DT>::kInf) m = max(m, w);
        }
    }
    return m;
}

// The largest of a block's threads, in all of them.
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* smem) {
    m = lanes_max<32>(m);
    if (threadIdx.x % 32 == 0) smem[threadIdx.x / 32] = m;
    __syncthreads();
    return lanes_max<kThreads / 32>(smem[threadIdx.x % (kThreads / 32)]);
}

// The largest finite |v| of chunks of eight elements `first`, `first + step`, ... of x; four in flight.
template <int DT>
__device__ __forceinline__ uint32_t max_of_chunks(const QuantArgs& a, int64_t first, int64_t step) {
    using T = typename Elem<DT>::T;
    const T* x = static_cast<const T*>(a.x);
    const bool flat = a.stride == a.cols;  // rows without gaps are one row
    const int64_t cols = flat ? a.rows * a.cols : a.cols, per_row = (cols + 7) / 8, n = (flat ? 1 : a.rows) * per_row;
    const int width = flat ? a.start_width : a.width;
    uint32_t m = 0;
    int64_t i = first;
    if (flat && width == 16) {  // whole chunks: nothing to check, nothing to divide
        const int64_t whole = cols / 8;
        const T* p = x + 8 * first;
        for (; i + 3 * step < whole; i += 4 * step, p += 32 * step) {
            Raw8<DT> r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = load_raw8<DT>(p + 8 * k * step, 8, 16);
#pragma unroll
            for (int k = 0; k < 4; ++k) m = max(m, finite_max8<DT>(r[k]));
        }
    }
    for (; i < n; i += step) {
        const int64_t row = flat ? 0 : i / per_row, c = 8 * (i - row * per_row);
        m = max(m, finite_max8<DT>(load_raw8<DT>(x + row * a.stride + c, int(min(int64_t(8), cols - c)), width)));
    }
    return m;
}

// First pass over x for a tensor scale: block i's maximum goes to tensor_scale[1 + i].  Bound by memory
// (5.6 TB/s of 8192 x 11008 bf16).
template <int DT>
__global__ void __launch_bounds__(kThreads, DT == EP_F32 ? 4 : 6) amax_kernel(const QuantArgs a) {
    using T = typename Elem<DT>::T;
    __shared__ uint32_t smem[kThreads / 32];
    wait_for_stream();
    uint32_t m = 0;
    if (a.stride == a.cols) {
        m = max_of_chunks<DT>(a, int64_t(blockIdx.x) * kThreads + threadIdx.x, int64_t(gridDim.x) * kThreads);
    } else {  // rows apart: runs of a row, so that a division serves four loads of the block
        constexpr int kRun = 4 * 8 * kThreads;
        const int64_t runs = (a.cols + kRun - 1) / kRun;
        for (int64_t u = blockIdx.x; u < a.rows * runs; u += gridDim.x) {
            const int64_t row = u / runs, c = (u - row * runs) * kRun + 8 * int(threadIdx.x);
            const T* p = static_cast<const T*>(a.x) + row * a.stride + c;
            Raw8<DT> r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                r[k] = load_raw8<DT>(p + 8 * k * kThreads, int(max(int64_t(0), min(int64_t(8), a.cols - c - 8 * k * kThreads))), a.width);
#pragma unroll
            for (int k = 0; k < 4; ++k) m = max(m, finite_max8<DT>(r[k]));
        }
    }
    m = block_max(m, smem);
    if (threadIdx.x == 0) a.tensor_scale[1 + blockIdx.x] = abs_value<DT>(m);
}

// One pass: a block reads its 128 x 128 elements, forms the block scales among neighbouring threads and
// writes their codes and its scale tiles.  A thread has 16 neighbours of 16-bit elements (with 8, a scale
// was formed 2 or 4 times over and issue took as long as the memory: 100 instructions for 8 elements and
// 73 us for 8192 x 16384 bf16; now 65 and 52), but 8 of fp32 (16 are 64 bytes, too far from one thread
// to the next: 40 us for 4096 x 11008, 36 with 8).
template <int DT, bool NV, int ROWS>
__global__ void __launch_bounds__(kThreads, NV && DT == EP_F32 ? 3 : 4) quantize_kernel(const __grid_constant__ QuantArgs a) {
    using T = typename Elem<DT>::T;
    constexpr int kC = DT == EP_F32 ? 1 : 2;                        // chunks of 8 elements a thread
    constexpr int kParts = kTileCols / (8 * kC);                    // threads a row
    constexpr int kRows = kThreads / kParts, kSteps = kTileRows / kRows;
    constexpr int kBatch = ROWS != kAnywhere ? 4 : 2;                            // steps in flight
    constexpr int kOwners = (NV ? 16 : 32) / (8 * kC);              // threads of a scale block
    __shared__ uint32_t red[kThreads / 32];
    __shared__ __align__(16) uint8_t sc[NV ? 1024 : 512];
    wait_for_stream();
    const uint32_t block = a.backwards ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    const uint32_t row_tile = block / uint32_t(a.col_tiles), col_tile = block - row_tile * uint32_t(a.col_tiles);
    const int64_t row0 = int64_t(row_tile) * kTileRows;
    const int part = threadIdx.x % kParts, sub = threadIdx.x / kParts;
    const int64_t col = int64_t(col_tile) * kTileCols + 8 * kC * part;
    const int rows = int(min(int64_t(kTileRows), a.rows - row0));
    const int n = int(max(int64_t(0), min(int64_t(8 * kC), a.cols - col)));
    const T* x = static_cast<const T*>(a.x) + (row0 + sub) * a.stride + col;
    uint8_t* data = a.data + (row0 + sub) * a.row_bytes + col / 2;
    const bool codes_in = col < 2 * a.row_bytes;
    const int k = part / kOwners;  // the scale block's column in this tile

    float g = 1.0f, g_inv = 1.0f;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(a.x), hi = lo + size_t((a.rows - 1) * a.stride + a.cols) * sizeof(T);
    Raw8<DT> v[kBatch][kC];
#pragma unroll
    for (int p0 = 0; p0 < kSteps; p0 += kBatch) {
        Piece<DT> piece[ROWS == kAnywhere ? kBatch : 1];
#pragma unroll
        for (int p = 0; p < kBatch; ++p) {
            const T* src = x + int64_t(p0 + p) * kRows * a.stride;
            const int have = sub + (p0 + p) * kRows < rows ? n : 0;
            if constexpr (ROWS != kAnywhere) {
#pragma unroll
                for (int c = 0; c < kC; ++c)
                    v[p][c] = ROWS == kWhole ? load_raw8<DT>(src + 8 * c, have ? 8 : 0, 16) : load_raw8<DT>(src + 8 * c, min(have - 8 * c, 8), 8);
            } else {
                piece[p].load(src, have, lo, hi);
            }
        }
        if (NV && p0 == 0) {
            if (a.fixed > 0.0f) {
                g = a.fixed;
            } else if (a.partials > 0) {
                uint32_t m = 0;
                for (int i = threadIdx.x; i < a.partials; i += kThreads) m = max(m, __float_as_uint(a.tensor_scale[1 + i]));
                g = tensor_scale_of(__uint_as_float(block_max(m, red)));
            } else {
                g = tensor_scale_of(abs_value<DT>(block_max(max_of_chunks<DT>(a, threadIdx.x, kThreads), red)));
            }
            g_inv = pow2f(-log2_floor(g));
        }
#pragma unroll
        for (int p = 0; p < kBatch; ++p) {
            const bool in = sub + (p0 + p) * kRows < rows;
            if constexpr (ROWS == kAnywhere) piece[p].take(x + int64_t(p0 + p) * kRows * a.stride, in ? n : 0, v[p]);
            uint32_t m = abs_max8<DT>(v[p][0]);
            if constexpr (kC == 2) m = max(m, abs_max8<DT>(v[p][1]));
            const Block b = block_scale<DT, NV>(lanes_max<kOwners>(m), g, g_inv);
            if (in && codes_in) {
                uint8_t* to = data + int64_t(p0 + p) * kRows * a.row_bytes;
                if constexpr (kC == 2)
                    *reinterpret_cast<uint2*>(to) = make_uint2(quantize8<DT, NV>(v[p][0], b), quantize8<DT, NV>(v[p][1], b));
                else
                    *reinterpret_cast<uint32_t*>(to) = quantize8<DT, NV>(v[p][0], b);
            }
            const int r = sub + (p0 + p) * kRows;
            if (part % kOwners == 0) sc[(k / 4) * 512 + k % 4 + 16 * (r % 32) + 4 * (r / 32)] = in && n ? b.byte : 0;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.tensor_scale[0] = g;
    __syncthreads();
    const int st = int(col_tile) * (NV ? 2 : 1);
    const int tiles = min(NV ? 2 : 1, a.scale_tiles - st);
    if (int(threadIdx.x) < 32 * tiles)
        reinterpret_cast<uint4*>(a.scales + (int64_t(row_tile) * a.scale_tiles + st) * 512)[threadIdx.x] =
            reinterpret_cast<const uint4*>(sc)[threadIdx.x];
}

__global__ void set_scale_kernel(float* tensor_scale, float g) {
    wait_for_stream();
    *tensor_scale = g;
}

struct DequantArgs {
    const uint8_t* data;
    const uint8_t* scales;
    const float* tensor_scale;
    void* out;
    int64_t stride, rows, cols, row_bytes;
    int col_tiles, scale_tiles;
    int rows_lie;     // Rows
};

// The same blocks backwards: scale tiles to shared memory, 4 bytes of codes a thread, 8 elements out.
// Rows anywhere go through shared memory, so that the lanes of a warp store neighbouring elements, or pairs
// of them (5230 x 10463 bf16: 35 us; 8 neighbours a lane, one by one, took several times that).
template <int DT, bool NV, int ROWS>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const __grid_constant__ DequantArgs a) {
    using T = typename Elem<DT>::T;
    __shared__ __align__(16) uint8_t sc[NV ? 1024 : 512];
    __shared__ __align__(16) T staged[ROWS == kAnywhere ? kPassRows * kTileCols : 8];
    wait_for_stream();
    const int64_t row0 = int64_t(blockIdx.x / a.col_tiles) * kTileRows;
    const int64_t col = int64_t(blockIdx.x % a.col_tiles) * kTileCols + 8 * (threadIdx.x % 16);
    const int sub = threadIdx.x / 16;
    const int64_t st = int64_t(blockIdx.x % a.col_tiles) * (NV ? 2 : 1);
    const int tiles = int(min(int64_t(NV ? 2 : 1), a.scale_tiles - st));
    if (int(threadIdx.x) < 32 * tiles)
        reinterpret_cast<uint4*>(sc)[threadIdx.x] =
            reinterpret_cast<const uint4*>(a.scales + ((row0 / kTileRows) * a.scale_tiles + st) * 512)[threadIdx.x];
    const float g = *a.tensor_scale;
    uint32_t codes[kPasses];
    const bool col_in = col < a.cols;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int64_t r = row0 + sub + p * kPassRows;
        codes[p] = col_in && r < a.rows ? *reinterpret_cast<const uint32_t*>(a.data + r * a.row_bytes + col / 2) : 0;
    }
    __syncthreads();
    const int64_t tile0 = col - 8 * (threadIdx.x % 16);
    const int n = int(min(int64_t(kTileCols), a.cols - tile0));  // columns of this tile
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
        const int r = sub + p * kPassRows;
        const int k = (threadIdx.x % 16) / (NV ? 2 : 4);
        const float s = scale_value<NV>(sc[(k / 4) * 512 + 16 * (r % 32) + 4 * (r / 32) + k % 4]);
        float v[8];
        e2m1_values8(codes[p], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * s * g;
        T* row = static_cast<T*>(a.out) + (row0 + r) * a.stride + tile0;
        if constexpr (ROWS != kAnywhere) {
            if (row0 + r < a.rows && col_in)
                store8<DT>(row + 8 * (threadIdx.x % 16), ROWS == kWhole ? 8 : min(8, n - 8 * int(threadIdx.x % 16)), ROWS == kWhole ? 16 : 8, v);
        } else {
            // the warp's two rows, one after the other
            store8<DT>(staged + sub * kTileCols + 8 * (threadIdx.x % 16), 8, 16, v);
            __syncwarp();
            const int lane = threadIdx.x % 32, first = r - sub % 2;
            row -= (sub % 2) * a.stride;
#pragma unroll
            for (int q = 0; q < 2; ++q, row += a.stride) {
                if (row0 + first + q >= a.rows) break;
                const T* from = staged + (sub - sub % 2 + q) * kTileCols;
                if (sizeof(T) == 2 && reinterpret_cast<uintptr_t>(row) % 4 == 0) {
#pragma unroll
                    for (int e = 2 * lane; e < kTileCols; e += 64) {
                        if (e + 1 < n) *reinterpret_cast<uint32_t*>(row + e) = *reinterpret_cast<const uint32_t*>(from + e);
                        else if (e < n) row[e] = from[e];
                    }
                } else {
#pragma unroll
                    for (int e = lane; e < kTileCols; e += 32)
                        if (e < n) row[e] = from[e];
                }
            }
            __syncwarp();
        }
    }
}

template <int DT>
cudaError_t launch_quantize(const QuantArgs& q, bool nv, int64_t grid, int amax_grid, cudaStream_t st) {
    if (amax_grid > 0) {
        cudaError_t e = op::launch(amax_kernel<DT>, dim3(unsigned(amax_grid)), dim3(kThreads), 0, st, q);
        if (e != cudaSuccess) return e;
    }
    const int rows = q.width == 16 && q.cols % 16 == 0 ? kWhole : q.width >= 8 ? kEven : kAnywhere;
    const auto kernel = rows == kWhole  ? (nv ? quantize_kernel<DT, true, kWhole> : quantize_kernel<DT, false, kWhole>)
                        : rows == kEven ? (nv ? quantize_kernel<DT, true, kEven> : quantize_kernel<DT, false, kEven>)
                                        : (nv ? quantize_kernel<DT, true, kAnywhere> : quantize_kernel<DT, false, kAnywhere>);
    return op::launch(kernel, dim3(unsigned(grid)), dim3(kThreads), 0, st, q);
}
template <int DT>
cudaError_t launch_dequantize(const DequantArgs& q, bool nv, int64_t grid, cudaStream_t st) {
    const auto kernel = q.rows_lie == kWhole  ? (nv ? dequantize_kernel<DT, true, kWhole> : dequantize_kernel<DT, false, kWhole>)
                        : q.rows_lie == kEven ? (nv ? dequantize_kernel<DT, true, kEven> : dequantize_kernel<DT, false, kEven>)
                                              : (nv ? dequantize_kernel<DT, true, kAnywhere> : dequantize_kernel<DT, false, kAnywhere>);
    return op::launch(kernel, dim3(unsigned(grid)), dim3(kThreads), 0, st, q);
}

// Tensors of at most this many bytes are searched for their largest value by every block itself
// (from L2, one launch); larger ones in a pass of their own.  (bf16: 16 KB 2.9 us with the search, 4.1
// with a pass; 64 KB 5.4 and 4.0; fp32: 32 KB 4.4 and 5.5, 128 KB 8.5 and 5.3.)
constexpr int64_t kSearchBytes = 32 << 10;

int check_dense(const ep_tensor* t, const char* what, const char* who) {
    const std::string w = std::string(who) + ": " + what;
    const int es = op::elem_bytes(t->dtype);
    if (es == 0) return set_error(EP_ERR_DTYPE, w + " must be EP_BF16, EP_FP16 or EP_F32");
    if (t->rows < 0 || t->cols < 0) return set_error(EP_ERR_SHAPE, w + " has a negative size");
    if (t->rows > 0 && t->cols > 0) {
        if (!t->data) return set_error(EP_ERR_ARG, w + " has no data");
        if (!op::aligned(t->data, size_t(es))) return set_error(EP_ERR_ARG, w + " is not aligned to its elements");
        if (t->row_stride < t->cols) return set_error(EP_ERR_ARG, w + ": row_stride < cols");
    }
    return EP_OK;
}

int check_quantize(const ep_tensor* x, const ep_fp4_tensor* out, double tensor_scale, const char* who) {
    int rc = check_dense(x, "the matrix", who);
    if (rc == EP_OK) rc = op::check_fp4(out, who);
    if (rc != EP_OK) return rc;
    if (x->rows != out->rows || x->cols != out->cols)
        return set_error(EP_ERR_SHAPE, std::string(who) + ": the 4-bit tensor's shape differs from the matrix's");
    int e = 0;
    const bool ok = tensor_scale == 0.0 ||
                    (out->format == EP_NVFP4 && tensor_scale > 0.0 && std::isfinite(tensor_scale) &&
                     std::frexp(tensor_scale, &e) == 0.5 && e - 1 >= -100 && e - 1 <= 117);
    if (!ok)
        return set_error(EP_ERR_ARG, std::string(who) + (out->format == EP_NVFP4
                                                             ? ": tensor_scale must be 0 or a power of two in [2^-100, 2^117]"
                                                             : ": EP_MXFP4 has no tensor scale"));
    return EP_OK;
}

// The current device, which must be the tensors' own.
int device_of(int a, int b, const char* who, int& sms) {
    int dev = 0;
    const int rc = op::current_device(dev, sms);
    if (rc == EP_OK && (a != dev || b != dev))
        return set_error(EP_ERR_ARG, std::string(who) + ": a tensor is not on the current device");
    return rc;
}

int quantize(const ep_tensor* x, const ep_fp4_tensor* out, double tensor_scale, cudaStream_t st, int sms, const char* who) {
    const bool nv = out->format == EP_NVFP4;
    cudaError_t e;
    if (x->rows == 0 || x->cols == 0) {
        const float g = !nv ? 1.0f : tensor_scale > 0.0 ? float(tensor_scale) : std::ldexp(1.0f, -100);
        e = op::launch(set_scale_kernel, dim3(1), dim3(1), 0, st, out->tensor_scale, g);
    } else {
        QuantArgs q = {};
        const int es = op::elem_bytes(x->dtype);
        q.x = x->data;
        q.stride = x->row_stride;
        q.rows = x->rows;
        q.cols = x->cols;
        q.data = static_cast<uint8_t*>(out->data);
        q.scales = static_cast<uint8_t*>(out->scales);
        q.tensor_scale = out->tensor_scale;
        q.row_bytes = op::fp4_row_bytes(x->cols);
        q.col_tiles = int(op::div_up(x->cols, kTileCols));
        q.scale_tiles = int(op::div_up(op::fp4_blocks(out->format, x->cols), 4));
        q.fixed = float(tensor_scale);
        q.width = op::access_width(x->data, x->row_stride * es);
        q.start_width = op::access_width(x->data, 0);
        const int64_t grid = op::div_up(x->rows, kTileRows) * q.col_tiles;
        if (grid > 0x7fffffff) return set_error(EP_ERR_SHAPE, std::string(who) + ": the matrix is too large");
        int amax_grid = 0;
        if (nv && tensor_scale == 0.0 && x->rows * x->cols * es > kSearchBytes) {
            // one round of blocks: 6 an SM for 16-bit elements, 4 for fp32 (8192 x 11008 bf16 in all: 83 us
            // with 4, 74 with 6; 4096 x 11008 fp32: 70 and 77)
            const int64_t per_sm = x->dtype == EP_F32 ? 4 : 6;
            amax_grid = int(std::min<int64_t>({kMaxPartials, per_sm * sms, op::div_up(x->rows * x->cols, 8 * 4 * kThreads)}));
            q.partials = amax_grid;
            q.backwards = true;  // what the first pass read last is still in L2
        }
        e = x->dtype == EP_BF16   ? launch_quantize<EP_BF16>(q, nv, grid, amax_grid, st)
            : x->dtype == EP_FP16 ? launch_quantize<EP_FP16>(q, nv, grid, amax_grid, st)
                                  : launch_quantize<EP_F32>(q, nv, grid, amax_grid, st);
    }
    if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string(who) + ": " + cudaGetErrorString(e));
    return EP_OK;
}

}  // namespace
}  // namespace ep

using namespace ep;

extern "C" int ep_fp4_sizes(int format, int64_t rows, int64_t cols, size_t* data_bytes, size_t* scale_bytes) {
    clear_error();
    if (!data_bytes || !scale_bytes) return set_error(EP_ERR_ARG, "ep_fp4_sizes: NULL argument");
    if (!op::is_fp4(format)) return set_error(EP_ERR_DTYPE, "ep_fp4_sizes: not a 4-bit format");
    if (rows < 0 || cols < 0 || cols > op::kMaxFp4Cols || rows > op::kMaxFp4Rows)
        return set_error(EP_ERR_SHAPE, "ep_fp4_sizes: size out of range");
    *data_bytes = size_t(rows) * size_t(op::fp4_row_bytes(cols));
    *scale_bytes = 512 * size_t(op::div_up(rows, 128)) * size_t(op::div_up(op::fp4_blocks(format, cols), 4));
    return EP_OK;
}

extern "C" int ep_fp4_quantize(const ep_tensor* x, const ep_fp4_tensor* out, double tensor_scale, void* stream) {
    clear_error();
    if (!x || !out) return set_error(EP_ERR_ARG, "ep_fp4_quantize: NULL argument");
    int sms = 0;
    int rc = check_quantize(x, out, tensor_scale, "ep_fp4_quantize");
    if (rc == EP_OK) rc = device_of(x->device, out->device, "ep_fp4_quantize", sms);
    if (rc != EP_OK) return rc;
    return quantize(x, out, tensor_scale, static_cast<cudaStream_t>(stream), sms, "ep_fp4_quantize");
}

extern "C" int ep_fp4_dequantize(const ep_fp4_tensor* x, const ep_tensor* out, void* stream) {
    clear_error();
    if (!x || !out) return set_error(EP_ERR_ARG, "ep_fp4_dequantize: NULL argument");
    int sms = 0;
    int rc = op::check_fp4(x, "ep_fp4_dequantize");
    if (rc == EP_OK) rc = check_dense(out, "the output", "ep_fp4_dequantize");
    if (rc != EP_OK) return rc;
    if (x->rows != out->rows || x->cols != out->cols)
        return set_error(EP_ERR_SHAPE, "ep_fp4_dequantize: the output's shape differs from the 4-bit tensor's");
    rc = device_of(x->device, out->device, "ep_fp4_dequantize", sms);
    if (rc != EP_OK) return rc;
    if (x->rows == 0 || x->cols == 0) return EP_OK;
    DequantArgs q = {};
    q.data = static_cast<const uint8_t*>(x->data);
    q.scales = static_cast<const uint8_t*>(x->scales);
    q.tensor_scale = x->tensor_scale;
    q.out = out->data;
    q.stride = out->row_stride;
    q.rows = x->rows;
    q.cols = x->cols;
    q.row_bytes = op::fp4_row_bytes(x->cols);
    q.col_tiles = int(op::div_up(x->cols, kTileCols));
    q.scale_tiles = int(op::div_up(op::fp4_blocks(x->format, x->cols), 4));
    const int width = op::access_width(out->data, out->row_stride * op::elem_bytes(out->dtype));
    q.rows_lie = width == 16 && x->cols % 8 == 0 ? kWhole : width >= 8 ? kEven : kAnywhere;
    const int64_t grid = op::div_up(x->rows, kTileRows) * q.col_tiles;
    if (grid > 0x7fffffff) return set_error(EP_ERR_SHAPE, "ep_fp4_dequantize: the tensor is too large");
    const bool nv = x->format == EP_NVFP4;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = out->dtype == EP_BF16   ? launch_dequantize<EP_BF16>(q, nv, grid, st)
                          : out->dtype == EP_FP16 ? launch_dequantize<EP_FP16>(q, nv, grid, st)
                                                  : launch_dequantize<EP_F32>(q, nv, grid, st);
    if (e != cudaSuccess) return set_error(EP_ERR_CUDA, std::string("ep_fp4_dequantize: ") + cudaGetErrorString(e));
    return EP_OK;
}

extern "C" int ep_decompress_fp4(const ep_blob* b, const ep_fp4_tensor* out, double tensor_scale, const ep_tensor* work,
                                 void* stream) {
    clear_error();
    if (!b || !out || !work) return set_error(EP_ERR_ARG, "ep_decompress_fp4: NULL argument");
    int sms = 0;
    int rc = check_quantize(work, out, tensor_scale, "ep_decompress_fp4");
    if (rc != EP_OK) return rc;
    if (work->rows != b->layout.rows || work->cols != b->layout.cols)
        return set_error(EP_ERR_SHAPE, "ep_decompress_fp4: the work tensor's shape differs from the blob's");
    rc = device_of(work->device, out->device, "ep_decompress_fp4", sms);
    if (rc != EP_OK) return rc;
    rc = ep_decompress(b, work, stream);
    if (rc != EP_OK) return rc;
    return quantize(work, out, tensor_scale, static_cast<cudaStream_t>(stream), sms, "ep_decompress_fp4");
}
