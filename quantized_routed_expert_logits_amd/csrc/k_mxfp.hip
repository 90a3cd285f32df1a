// Microscaled 4-bit floating point: rounding rows to it, reading them back,
// packing weight matrices, and the (grouped) product of packed weights with
// rounded rows.
//
// Format.  32 consecutive values of a row share a scale 2^(byte - 127); a value
// is a sign and one of 0, .5, 1, 1.5, 2, 3, 4, 6 (code bit 3 the sign, 2..1 the
// exponent, 0 the mantissa), two to a byte, the first in the low half.
#include "block.h"
#include "mxfp.h"

namespace strata_moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;

// ------------------------------------------------------ rounding and reading
// A thread takes 8 consecutive values, 4 threads a block of 32.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* __restrict__ x, int64_t x_stride, uint32_t runs,
                                                            uint32_t row_runs, int vec, uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
    const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
    // runs is a multiple of 4, so the threads of a block stay together
    if (id >= runs) return;
    const uint32_t row = id / row_runs;
    const T* p = x + row * x_stride + (id - row * row_runs) * 8;
    float v[8];
    if (vec) {
        load4_vec(p, v);
        load4_vec(p + 4, v + 4);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = widen(p[i]);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const uint32_t byte = mx_scale_byte(top);
    uint32_t q = mx_code_pair<0>(0, v[0], v[1], byte);
    q = mx_code_pair<1>(q, v[2], v[3], byte);
    q = mx_code_pair<2>(q, v[4], v[5], byte);
    q = mx_code_pair<3>(q, v[6], v[7], byte);
    ((uint32_t*)codes)[id] = byte == 255 ? 0 : q;
    if (id % 4 == 0) scales[id / 4] = (uint8_t)byte;
}

template <typename T, typename V>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, uint32_t runs,
                                                              uint32_t row_runs, T* __restrict__ out,
                                                              int64_t out_stride, int vec) {
    const uint32_t id = blockIdx.x * kThreads + threadIdx.x;
    if (id >= runs) return;
    const uint32_t row = id / row_runs;
    const uint32_t q = ((const uint32_t*)codes)[id];
    const float s = mx_scale(scales[id / 4]);
    float v[8];
    auto put = [&](v2f f, int i) { v[i] = f.x * s, v[i + 1] = f.y * s; };
    put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0), 0);
    put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1), 2);
    put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2), 4);
    put(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3), 6);
    T* p = out + row * out_stride + (id - row * row_runs) * 8;
    store4<T, V>(p, 0, 4, vec, v);
    store4<T, V>(p, 4, 8, vec, v + 4);
}

// ------------------------------------------------------------------- packing
// Tile j of a matrix holds its rows 16 j .. 16 j + 15; with `paired` tile 2 i
// holds rows 16 i .. of the first half and tile 2 i + 1 those of the second.
// Rows and columns past the matrix are zero.
__device__ __forceinline__ int tile_row(int tile, int r, int rows, int paired) {
    if (!paired) return tile * kMxTileRows + r < rows ? tile * kMxTileRows + r : -1;
    const int i = tile / 2 * kMxTileRows + r;
    return i < rows / 2 ? i + (tile & 1) * (rows / 2) : -1;
}

// One wave per (expert, tile, group of 4 steps).  Within a step lane l holds
// row l % 16 and the 32 values 32 (l / 16) on: what the matrix unit reads.  The
// group's scale dword of lane l: its row's scales of block l / 16 of each step.
__global__ __launch_bounds__(64) void pack_kernel(const uint8_t* __restrict__ codes,
                                                  const uint8_t* __restrict__ scales, int rows, int cols, int paired,
                                                  uint8_t* __restrict__ packed, int64_t stride, int64_t tile_bytes) {
    const int lane = threadIdx.x, g = lane / 16, blocks = cols / 32;
    const int steps = (cols + kMxStep - 1) / kMxStep;
    const int s0 = blockIdx.x * 4, n = min(4, steps - s0);
    const int row = tile_row(blockIdx.y, lane % 16, rows, paired);
    const int64_t e = blockIdx.z;
    uint8_t* dst = packed + e * stride + blockIdx.y * tile_bytes + (int64_t)blockIdx.x * (4 * kMxStepBytes + kMxScaleBytes);
    uint32_t sc = 0;
    for (int s = 0; s < n; ++s) {
        const int b = (s0 + s) * 4 + g;
        uint4 q = {0, 0, 0, 0};
        if (row >= 0 && b < blocks) {
            const int64_t at = (e * rows + row) * blocks + b;
            q = ((const uint4*)codes)[at];
            sc |= (uint32_t)scales[at] << (8 * s);
        }
        *(uint4*)(dst + s * kMxStepBytes + lane * 16) = q;
    }
    *(uint32_t*)(dst + n * kMxStepBytes + lane * 4) = sc;
}

// ------------------------------------------------------------------- product
struct ProductArgs {
    MxProduct p;
    int64_t tile_bytes;
    int32_t tiles, n_out;   // packed tiles of an expert; outputs of a row
    int32_t steps, blocks;  // of 128 and of 32 reduction values
    int32_t nb;             // work items along the outputs
    int32_t vec_out;
};

// The work list.  An item is one tile of MT rows of one expert times one run of
// its outputs; items are numbered expert by expert, within an expert run by run,
// and within a run tile by tile, so that the workgroups that read the same
// weights run at about the same time.  pre[e] = row tiles of the experts below
// e; the caller's offsets are clamped to [0, rows], whatever they hold.
constexpr int kMaxE = 1024;
struct List {
    int32_t pre[kMaxE + 1];
};
__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t rows) { return v < 0 ? 0 : v > rows ? rows : v; }

template <int MT>
__device__ void make_list(const MxProduct& p, List& L, int32_t* wave_sum) {
    if (!p.offsets) {
        if (threadIdx.x == 0) L.pre[0] = 0, L.pre[1] = (int32_t)((p.rows + MT - 1) / MT);
        __syncthreads();
        return;
    }
    constexpr int kPer = kMaxE / kThreads;
    int32_t n[kPer], s = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        n[i] = 0;
        if (e < p.E) {
            const int64_t a = clamp_row(p.offsets[e], p.rows), b = clamp_row(p.offsets[e + 1], p.rows);
            n[i] = b > a ? (int32_t)((b - a + MT - 1) / MT) : 0;
        }
        s += n[i];
    }
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    int32_t inc = s;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 63) wave_sum[wave] = inc;
    __syncthreads();
    int32_t at = inc - s;
    for (int w = 0; w < wave; ++w) at += wave_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = threadIdx.x * kPer + i;
        if (e <= p.E) L.pre[e] = at;
        at += n[i];
    }
    // E = 1024: the last entry has no thread of its own
    if (threadIdx.x == kThreads - 1 && p.E == kMaxE) L.pre[kMaxE] = at;
    __syncthreads();
}

struct Item {
    int32_t e, run;
    int64_t row0;
    int32_t rows;  // 1 .. MT
};
template <int MT>
__device__ Item find_item(const MxProduct& p, const List& L, int nb, int64_t u) {
    const int lane = threadIdx.x % 64;
    Item it;
    int e = 0;
    if (p.offsets) {
        // the last expert whose first item is not behind u, 16 at a time, then one by one
        const bool a = lane * 16 <= p.E && (int64_t)L.pre[lane * 16 <= p.E ? lane * 16 : 0] * nb <= u;
        e = (__popcll(__ballot(a)) - 1) * 16;
        const bool b = lane < 16 && e + lane < p.E && (int64_t)L.pre[e + lane < p.E ? e + lane : 0] * nb <= u;
        e += __popcll(__ballot(b)) - 1;
    }
    e = __builtin_amdgcn_readfirstlane(e);
    const int32_t tiles = L.pre[e + 1] - L.pre[e];
    const int64_t left = u - (int64_t)L.pre[e] * nb;
    const int32_t run = (int32_t)(left / tiles), t = (int32_t)(left - (int64_t)run * tiles);
    const int64_t r0 = p.offsets ? clamp_row(p.offsets[e], p.rows) : 0;
    const int64_t r1 = p.offsets ? clamp_row(p.offsets[e + 1], p.rows) : p.rows;
    // rows dealt evenly to the tiles, in whole 16s
    const int32_t frags = (int32_t)((r1 - r0 + 15) / 16);
    const int32_t f0 = (int32_t)((int64_t)frags * t / tiles), f1 = (int32_t)((int64_t)frags * (t + 1) / tiles);
    it.e = e;
    it.run = run;
    it.row0 = r0 + (int64_t)f0 * 16;
    it.rows = (int32_t)(min(r1, r0 + (int64_t)f1 * 16) - it.row0);
    return it;
}

__device__ __forceinline__ v8i operand(v4i q) { return v8i{q[0], q[1], q[2], q[3], 0, 0, 0, 0}; }

// silu(g) u, silu(g) = g / (1 + exp(-g)).  exp by 2^(-g log2 e), the product in
// two parts: its rounding alone would cost |g| 2^-24 of the result.
__device__ __forceinline__ float swiglu(float g, float u) {
    const float hi = -g * 1.44269502f;
    const float lo = fmaf(-g, 1.44269502f, -hi) + -g * 1.92596303e-8f;
    float e = __builtin_amdgcn_exp2f(hi);
    if (e < __builtin_inff()) e = fmaf(e, lo * 0.693147182f, e);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

__device__ __forceinline__ void store_out(const ProductArgs& a, int64_t row, int n, v4f v) {
    float f[4] = {v[0], v[1], v[2], v[3]};
    store4_any(a.p.out, a.p.dtype, row * a.p.out_stride, n, a.n_out, a.vec_out, f);
}

// Few rows: the weights' bytes bound it.  A workgroup's 4 waves share NF tiles
// of weights (16 NF rows) and MF tiles of rows, each a quarter of the steps; the
// quarters are added in wave order through LDS.
constexpr int kWaves = 4;
template <int MF, int NF>
__global__ __launch_bounds__(kThreads) void stream_kernel(ProductArgs a) {
    constexpr int MT = MF * 16;
    __shared__ List L;
    __shared__ int32_t wave_sum[kWaves];
    __shared__ v4f part[kWaves][MF * NF][64];
    const MxProduct& p = a.p;
    make_list<MT>(p, L, wave_sum);
    const int64_t items = (int64_t)L.pre[p.E] * a.nb;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, r16 = lane % 16, g = lane / 16;
    const int s0 = a.steps * wave / kWaves, s1 = a.steps * (wave + 1) / kWaves;
    for (int64_t u = blockIdx.x; u < items; u += gridDim.x) {
        const Item it = find_item<MT>(p, L, a.nb, u);
        const uint8_t* wt[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f)
            wt[f] = p.packed + it.e * p.stride + min(it.run * NF + f, a.tiles - 1) * a.tile_bytes;
        int64_t src[MF];
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            src[m] = -1;
            const int r = m * 16 + r16;
            if (r < it.rows) {
                src[m] = p.src ? p.src[it.row0 + r] : it.row0 + r;
                if (src[m] >= p.x_rows) src[m] = -1;
            }
        }
        v4f acc[MF][NF];
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[m][f] = v4f{0, 0, 0, 0};
        for (int s = s0; s < s1; ++s) {
            const int group = s / 4, in_group = s % 4, of_group = min(4, a.steps - group * 4);
            const int64_t at = (int64_t)group * (4 * kMxStepBytes + kMxScaleBytes);
            v4i w[NF], x[MF];
            int ws[NF], xs[MF];
#pragma unroll
            for (int f = 0; f < NF; ++f) {
                w[f] = *(const v4i*)(wt[f] + at + in_group * kMxStepBytes + lane * 16);
                ws[f] = *(const int*)(wt[f] + at + of_group * kMxStepBytes + lane * 4) >> (8 * in_group);
            }
            const int b = s * 4 + g;
#pragma unroll
            for (int m = 0; m < MF; ++m) {
                x[m] = v4i{0, 0, 0, 0};
                xs[m] = 0;
                if (src[m] >= 0 && b < a.blocks) {
                    x[m] = ((const v4i*)p.codes)[src[m] * a.blocks + b];
                    xs[m] = p.scales[src[m] * a.blocks + b];
                }
            }
#pragma unroll
            for (int m = 0; m < MF; ++m)
#pragma unroll
                for (int f = 0; f < NF; ++f)
                    acc[m][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w[f]), operand(x[m]), acc[m][f],
                                                                                 4, 4, 0, ws[f], 0, xs[m]);
        }
#pragma unroll
        for (int m = 0; m < MF; ++m)
#pragma unroll
            for (int f = 0; f < NF; ++f) part[wave][m * NF + f][lane] = acc[m][f];
        __syncthreads();
        // outputs: lane holds row lane % 16 and 4 consecutive outputs of a tile
        const int per = p.paired ? 2 : 1;
        for (int o = wave; o < MF * NF / per; o += kWaves) {
            const int m = o / (NF / per), f = o % (NF / per) * per;
            v4f v = part[0][m * NF + f][lane];
            for (int w = 1; w < kWaves; ++w) v += part[w][m * NF + f][lane];
            if (p.paired) {
                v4f up = part[0][m * NF + f + 1][lane];
                for (int w = 1; w < kWaves; ++w) up += part[w][m * NF + f + 1][lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], up[i]);
            }
            const int r = m * 16 + r16;
            const int n = (it.run * NF + f) / per * kMxTileRows + 4 * g;
            if (r < it.rows && n < a.n_out) store_out(a, it.row0 + r, n, v);
        }
        __syncthreads();
    }
}

}  // namespace

template <typename T>
static hipError_t quantize_rows(const void* x, int64_t x_stride, int64_t rows, int32_t cols, uint8_t* codes,
                                uint8_t* scales, hipStream_t st) {
    const uint32_t runs = (uint32_t)(rows * (cols / 8));
    const int vec = ((uintptr_t)x | (uintptr_t)(x_stride * (int64_t)sizeof(T))) % (4 * sizeof(T)) == 0;
    hipLaunchKernelGGL(quantize_kernel<T>, dim3((runs + kThreads - 1) / kThreads), dim3(kThreads), 0, st, (const T*)x,
                       x_stride, runs, (uint32_t)cols / 8, vec, codes, scales);
    return hipGetLastError();
}
hipError_t launch_mx_quantize(const void* x, int32_t dtype, int64_t x_stride, int64_t rows, int32_t cols,
                              uint8_t* codes, uint8_t* scales, hipStream_t st) {
    if (dtype == kF32) return quantize_rows<float>(x, x_stride, rows, cols, codes, scales, st);
    if (dtype == kF16) return quantize_rows<_Float16>(x, x_stride, rows, cols, codes, scales, st);
    return quantize_rows<__bf16>(x, x_stride, rows, cols, codes, scales, st);
}

template <typename T, typename V>
static hipError_t dequantize_rows(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, void* out,
                                  int64_t out_stride, hipStream_t st) {
    const uint32_t runs = (uint32_t)(rows * (cols / 8));
    const int vec = ((uintptr_t)out | (uintptr_t)(out_stride * (int64_t)sizeof(T))) % (4 * sizeof(T)) == 0;
    hipLaunchKernelGGL((dequantize_kernel<T, V>), dim3((runs + kThreads - 1) / kThreads), dim3(kThreads), 0, st, codes,
                       scales, runs, (uint32_t)cols / 8, (T*)out, out_stride, vec);
    return hipGetLastError();
}
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t cols, void* out,
                                int32_t dtype, int64_t out_stride, hipStream_t st) {
    if (dtype == kF32) return dequantize_rows<float, v4f>(codes, scales, rows, cols, out, out_stride, st);
    if (dtype == kF16) return dequantize_rows<_Float16, v4h>(codes, scales, rows, cols, out, out_stride, st);
    return dequantize_rows<__bf16, v4b>(codes, scales, rows, cols, out, out_stride, st);
}

hipError_t launch_mx_pack(const uint8_t* codes, const uint8_t* scales, int32_t ne, int32_t rows, int32_t cols,
                          bool paired, uint8_t* packed, int64_t stride, hipStream_t st) {
    const int groups = (cols + 4 * kMxStep - 1) / (4 * kMxStep);
    const dim3 grid(groups, (uint32_t)mx_tiles(rows, paired), ne);
    hipLaunchKernelGGL(pack_kernel, grid, dim3(64), 0, st, codes, scales, rows, cols, paired ? 1 : 0, packed, stride,
                       mx_tile_bytes(cols));
    return hipGetLastError();
}

hipError_t launch_mx_product(const MxProduct& p, hipStream_t st) {
    ProductArgs a{};
    a.p = p;
    a.tile_bytes = mx_tile_bytes(p.cols);
    a.tiles = (int32_t)mx_tiles(p.n, p.paired != 0);
    a.n_out = p.paired ? p.n / 2 : p.n;
    a.steps = (p.cols + kMxStep - 1) / kMxStep;
    a.blocks = p.cols / 32;
    const size_t el = dtype_bytes(p.dtype);
    a.vec_out = ((uintptr_t)p.out | (uintptr_t)(p.out_stride * (int64_t)el)) % (4 * el) == 0;
    constexpr int NF = 4;
    a.nb = (a.tiles + NF - 1) / NF;
    const int64_t hit = p.rows < p.E ? p.rows : p.E;
    auto items = [&](int mt) { return (p.rows / mt + hit) * a.nb; };
    const int64_t most = 256 * 4;
    if (p.rows <= 16 * (int64_t)p.E) {
        const int64_t n = items(16);
        hipLaunchKernelGGL((stream_kernel<1, NF>), dim3((uint32_t)(n < most ? n : most)), dim3(kThreads), 0, st, a);
    } else {
        const int64_t n = items(64);
        hipLaunchKernelGGL((stream_kernel<4, NF>), dim3((uint32_t)(n < most ? n : most)), dim3(kThreads), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace strata_moe
