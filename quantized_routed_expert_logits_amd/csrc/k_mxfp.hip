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

// One wave per (expert, tile, group of n = 4 steps, fewer in the last).  In step s
// of a group lane l holds row l % 16 and the 32 values of block n (l / 16) + s of
// the group: what the matrix unit reads.  A lane's blocks of the group are then
// neighbours, and its scale dword is theirs, byte s for step s.
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
        const int b = s0 * 4 + n * g + s;
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
__device__ __forceinline__ int32_t clamp_row(int32_t v, int32_t rows) { return v < 0 ? 0 : v > rows ? rows : v; }

template <int MT>
__device__ __forceinline__ void make_list(const MxProduct& p, List& L, int32_t* wave_sum) {
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
            const int32_t a = clamp_row(p.offsets[e], (int32_t)p.rows), b = clamp_row(p.offsets[e + 1], (int32_t)p.rows);
            n[i] = b > a ? (b - a + MT - 1) / MT : 0;
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

// Wave-uniform, in scalar registers.
struct Item {
    int32_t e, run, row0;
    int32_t rows;  // 1 .. MT
};
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

template <int MT, int kUnit>
__device__ __forceinline__ Item find_item(const MxProduct& p, const List& L, int nb, int64_t u) {
    const int lane = threadIdx.x % 64;
    Item it;
    int e = 0;
    if (p.offsets) {
        // the last expert whose first item is not behind u: among every 16th, then among the 16
        const bool a = lane * 16 <= p.E && (int64_t)L.pre[lane * 16 <= p.E ? lane * 16 : 0] * nb <= u;
        e = (__popcll(__ballot(a)) - 1) * 16;
        const bool b = lane < 16 && e + lane < p.E && (int64_t)L.pre[e + lane < p.E ? e + lane : 0] * nb <= u;
        e += __popcll(__ballot(b)) - 1;
    }
    e = uniform(e);
    const int32_t first = uniform(L.pre[e]), tiles = uniform(L.pre[e + 1]) - first;
    const uint32_t left = (uint32_t)(u - (int64_t)first * nb);  // below tiles * nb < 2^31
    const uint32_t run = left / (uint32_t)tiles, t = left - run * (uint32_t)tiles;
    const int32_t rows = (int32_t)p.rows;
    const int32_t r0 = p.offsets ? clamp_row(uniform(p.offsets[e]), rows) : 0;
    const int32_t r1 = p.offsets ? clamp_row(uniform(p.offsets[e + 1]), rows) : rows;
    // rows dealt evenly to the tiles, in whole units of 16 kUnit
    const int32_t units = (r1 - r0 + 16 * kUnit - 1) / (16 * kUnit);
    const int32_t f0 = (int32_t)((int64_t)units * t / tiles), f1 = (int32_t)((int64_t)units * (t + 1) / tiles);
    it.e = e;
    it.run = (int32_t)run;
    it.row0 = r0 + f0 * 16 * kUnit;
    it.rows = min(r1, r0 + f1 * 16 * kUnit) - it.row0;
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

__device__ __forceinline__ void store_out(const ProductArgs& a, int32_t row, int n, v4f v) {
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
    const int64_t items = (int64_t)uniform(L.pre[p.E]) * a.nb;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), r16 = lane % 16, g = lane / 16;
    const int s0 = a.steps * wave / kWaves, s1 = a.steps * (wave + 1) / kWaves;
    for (int64_t u = blockIdx.x; u < items; u += gridDim.x) {
        const Item it = find_item<MT, 1>(p, L, a.nb, u);
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
            const int b = group * 16 + of_group * g + in_group;
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

// Many rows: the matrix unit bounds it, or the weights' bytes if an expert has a
// few hundred rows.  A workgroup takes up to 8 tiles of rows (128) and 16 of
// weights, 4 to a wave.  The rows' codes of 512 reduction values (a group) go to
// LDS while the group before is multiplied (two buffers); each wave reads its own
// weights from memory straight into registers, a group ahead.  Row tiles come in
// pairs: an item of fewer rows leaves out the pairs it lacks.
constexpr int kRowTiles = 8;
constexpr int kWaveTiles = 4;
constexpr int kGroupBytes = 4 * kMxStepBytes + kMxScaleBytes;
// [row][16 pieces]: 16 bytes a block; piece c of row r lies at c ^ r % 16, so that
// the 16 rows that a product reads at one c lie in different banks.
struct Rows {
    v4i codes[kRowTiles * 16 * 16];
    int scales[kRowTiles * 64];  // [tile][lane]: the lane's scales of a group, byte s for step s
};

using Resource = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Resource resource(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
using LdsPtr = void __attribute__((address_space(3)))*;

struct TileLoads {
    Resource codes, scales, weights;  // x, its scales, the item's expert
    const uint32_t* first;            // [128] LDS: first block in x of each row of the item
    uint32_t tile[kWaveTiles];        // byte offsets of the wave's weight tiles
    int32_t blocks, steps, lane, wave;
};

// A lane's offset that no array reaches: such a load reads nothing.
constexpr uint32_t kNowhere = 0xf0000000u;

// Start the loads of group q: 4 rows of 256 bytes an instruction.
template <int kPairs>
__device__ __forceinline__ void load_rows(const TileLoads& l, int q, uint32_t off, Rows* __restrict__ to) {
#pragma unroll
    for (int i = 0; i < 2 * kPairs; ++i) {
        const int r4 = (i * kWaves + l.wave) * 4, r = r4 + l.lane / 16;
        const uint32_t at = l.first[r] * 16 + ((l.lane % 16) ^ (r % 16)) * 16;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(l.codes, (LdsPtr)(to->codes + r4 * 16), 16, at | off, q * 256, 0, 0);
    }
}

// The scales of whole group q of tiles wave and wave + 4: a lane's are neighbours.
template <int kPairs>
__device__ __forceinline__ void load_row_scales(const TileLoads& l, int q, uint32_t off, int* sc) {
#pragma unroll
    for (int i = 0; i < (kPairs > 2 ? 2 : 1); ++i) {
        const uint32_t at = l.first[(l.wave + 4 * i) * 16 + l.lane % 16] + 4 * (l.lane / 16);
        sc[i] = __builtin_amdgcn_raw_buffer_load_b32(l.scales, at | off, q * 16, 0);
    }
}
// Those of the last, n steps long and perhaps not whole, byte by byte: a block
// past the row's end gets scale 2^-127 (its codes are any, and meet weights of 0).
template <int kPairs>
__device__ __forceinline__ void load_last_scales(const TileLoads& l, int q, int n, int* sc) {
    const int g = l.lane / 16;
#pragma unroll
    for (int i = 0; i < (kPairs > 2 ? 2 : 1); ++i) {
        const uint32_t at = l.first[(l.wave + 4 * i) * 16 + l.lane % 16] + n * g;
        sc[i] = 0;
        for (int s = 0; s < n; ++s)
            if (q * 16 + n * g + s < l.blocks)
                sc[i] |= (int)__builtin_amdgcn_raw_buffer_load_b8(l.scales, at + s, q * 16, 0) << (8 * s);
    }
}
template <int kPairs>
__device__ __forceinline__ void keep_row_scales(const TileLoads& l, const int* sc, Rows* to) {
#pragma unroll
    for (int i = 0; i < (kPairs > 2 ? 2 : 1); ++i) to->scales[(l.wave + 4 * i) * 64 + l.lane] = sc[i];
}

__device__ __forceinline__ void load_weights(const TileLoads& l, int q, int st, uint32_t off, v4i* w) {
#pragma unroll
    for (int f = 0; f < kWaveTiles; ++f)
        w[f] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(
                                           l.weights, l.lane * 16 | off, l.tile[f] + q * kGroupBytes + st * kMxStepBytes, 0));
}
__device__ __forceinline__ void load_weight_scales(const TileLoads& l, int q, int n, uint32_t off, int* sc) {
#pragma unroll
    for (int f = 0; f < kWaveTiles; ++f)
        sc[f] = __builtin_amdgcn_raw_buffer_load_b32(l.weights, l.lane * 4 | off,
                                                     l.tile[f] + q * kGroupBytes + n * kMxStepBytes, 0);
}

// Step ST of a group of n: the products of every row tile.
template <int kPairs, int ST>
__device__ __forceinline__ void step_products(const Rows* __restrict__ x, const int* xs, const v4i* w, const int* ws,
                                              int n, int lane, v4f (*acc)[kWaveTiles]) {
    const int r16 = lane % 16;
    const v4i* at = x->codes + r16 * 16 + ((n * (lane / 16) + ST) ^ r16);
#pragma unroll
    for (int m = 0; m < 2 * kPairs; ++m) {
        const v8i a = operand(at[m * 256]);
#pragma unroll
        for (int f = 0; f < kWaveTiles; ++f)
            acc[m][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w[f]), a, acc[m][f], 4, 4, ST, ws[f], ST,
                                                                         xs[m]);
    }
}

// Everything this wave wrote to or started into LDS is there, for all waves.
__device__ __forceinline__ void rows_ready() {
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

struct WeightRegs {
    v4i w[2][kWaveTiles];  // steps of the same parity take turns
    int s[kWaveTiles];
};

// Whole group q of `groups` from `now`, the loads of group q + 1 into `next` beside
// it, and those of the weights two steps ahead.
template <int kPairs>
__device__ __forceinline__ void group(const TileLoads& l, int q, int groups, Rows* __restrict__ now,
                                      Rows* __restrict__ next, WeightRegs& r, v4f (*acc)[kWaveTiles]) {
    // behind the last group: loads of nothing (the scalar offset stays in the arrays,
    // since the range check subtracts it from their size)
    const int qn = q + 1 < groups ? q + 1 : q;
    const uint32_t off = q + 1 < groups ? 0 : kNowhere;
    int sc[2], ws[kWaveTiles], xs[2 * kPairs];
    load_rows<kPairs>(l, qn, off, next);
    load_row_scales<kPairs>(l, qn, off, sc);
    load_weight_scales(l, qn, 4, off, ws);
#pragma unroll
    for (int m = 0; m < 2 * kPairs; ++m) xs[m] = now->scales[m * 64 + l.lane];
    __builtin_amdgcn_sched_barrier(0);
    step_products<kPairs, 0>(now, xs, r.w[0], r.s, 4, l.lane, acc);
    __builtin_amdgcn_sched_barrier(0);
    load_weights(l, q, 2, 0, r.w[0]);
    __builtin_amdgcn_sched_barrier(0);
    step_products<kPairs, 1>(now, xs, r.w[1], r.s, 4, l.lane, acc);
    __builtin_amdgcn_sched_barrier(0);
    load_weights(l, q, 3, 0, r.w[1]);
    __builtin_amdgcn_sched_barrier(0);
    step_products<kPairs, 2>(now, xs, r.w[0], r.s, 4, l.lane, acc);
    __builtin_amdgcn_sched_barrier(0);
    load_weights(l, qn, 0, off, r.w[0]);
    __builtin_amdgcn_sched_barrier(0);
    step_products<kPairs, 3>(now, xs, r.w[1], r.s, 4, l.lane, acc);
    __builtin_amdgcn_sched_barrier(0);
    load_weights(l, qn, 1, off, r.w[1]);
    __builtin_amdgcn_sched_barrier(0);
    keep_row_scales<kPairs>(l, sc, next);
#pragma unroll
    for (int f = 0; f < kWaveTiles; ++f) r.s[f] = ws[f];
    rows_ready();
}

// The last group, where it is not whole: n steps of four.
template <int kPairs>
__device__ __forceinline__ void last_group(const TileLoads& l, int q, Rows* __restrict__ b0, v4f (*acc)[kWaveTiles]) {
    const int n = l.steps - 4 * q;
    int sc[2], ws[kWaveTiles], xs[2 * kPairs];
    v4i w[kWaveTiles];
    load_rows<kPairs>(l, q, 0, b0);
    load_weight_scales(l, q, n, 0, ws);
    load_last_scales<kPairs>(l, q, n, sc);
    keep_row_scales<kPairs>(l, sc, b0);
    load_weights(l, q, 0, 0, w);
    rows_ready();
#pragma unroll
    for (int m = 0; m < 2 * kPairs; ++m) xs[m] = b0->scales[m * 64 + l.lane];
    step_products<kPairs, 0>(b0, xs, w, ws, n, l.lane, acc);
    __builtin_amdgcn_sched_barrier(0);
    if (n > 1) {
        load_weights(l, q, 1, 0, w);
        step_products<kPairs, 1>(b0, xs, w, ws, n, l.lane, acc);
    }
    if (n > 2) {
        load_weights(l, q, 2, 0, w);
        step_products<kPairs, 2>(b0, xs, w, ws, n, l.lane, acc);
    }
    if (n > 3) {
        load_weights(l, q, 3, 0, w);
        step_products<kPairs, 3>(b0, xs, w, ws, n, l.lane, acc);
    }
    rows_ready();
}

template <int kPairs>
__device__ __forceinline__ void item_sums(const TileLoads& l, Rows* b0, Rows* b1, v4f (*acc)[kWaveTiles]) {
    const int groups = l.blocks / 16;  // whole ones
    int sc[2];
    if (groups) {
        WeightRegs r;
        load_rows<kPairs>(l, 0, 0, b0);
        load_row_scales<kPairs>(l, 0, 0, sc);
        load_weight_scales(l, 0, 4, 0, r.s);
        load_weights(l, 0, 0, 0, r.w[0]);
        load_weights(l, 0, 1, 0, r.w[1]);
        keep_row_scales<kPairs>(l, sc, b0);
        rows_ready();
        for (int q = 0; q < groups; q += 2) {
            group<kPairs>(l, q, groups, b0, b1, r, acc);
            if (q + 1 < groups) group<kPairs>(l, q + 1, groups, b1, b0, r, acc);
        }
    }
    if (l.blocks % 16) last_group<kPairs>(l, groups, b0, acc);
}

__global__ __launch_bounds__(kThreads, 2) void tile_kernel(ProductArgs a) {
    constexpr int MT = kRowTiles * 16;
    __shared__ Rows b0, b1;
    __shared__ uint32_t first[MT];
    __shared__ List L;
    __shared__ int32_t wave_sum[kWaves];
    const MxProduct& p = a.p;
    make_list<MT>(p, L, wave_sum);
    const int64_t items = (int64_t)uniform(L.pre[p.E]) * a.nb;
    // workgroups of one XCD (every eighth) take one run of the items
    const int xcd = blockIdx.x % 8, per = gridDim.x / 8;
    const int64_t u1 = items * (xcd + 1) / 8;
    TileLoads l;
    l.codes = resource(p.codes, (uint32_t)(p.x_rows * a.blocks * 16));
    l.scales = resource(p.scales, (uint32_t)(p.x_rows * a.blocks));
    l.first = first;
    l.blocks = a.blocks;
    l.steps = a.steps;
    l.lane = threadIdx.x % 64;
    l.wave = uniform(threadIdx.x / 64);
    for (int64_t u = items * xcd / 8 + blockIdx.x / 8; u < u1; u += per) {
        const Item it = find_item<MT, 2>(p, L, a.nb, u);
        if (threadIdx.x < MT) {
            int32_t s = it.row0 + min((int)threadIdx.x, it.rows - 1);
            if (p.src) s = p.src[s];
            first[threadIdx.x] = s < 0 || s >= p.x_rows ? 0u : (uint32_t)s * (uint32_t)a.blocks;
        }
        __syncthreads();
        const int t0 = it.run * (kWaves * kWaveTiles) + l.wave * kWaveTiles, pairs = (it.rows + 31) / 32;
        l.weights = resource(p.packed + it.e * p.stride, (uint32_t)(a.tiles * a.tile_bytes));
#pragma unroll
        for (int f = 0; f < kWaveTiles; ++f) l.tile[f] = (uint32_t)(min(t0 + f, a.tiles - 1) * a.tile_bytes);
        v4f acc[kRowTiles][kWaveTiles];
#pragma unroll
        for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
            for (int f = 0; f < kWaveTiles; ++f) acc[m][f] = v4f{0, 0, 0, 0};
        if (pairs == 1) item_sums<1>(l, &b0, &b1, acc);
        else if (pairs == 2) item_sums<2>(l, &b0, &b1, acc);
        else if (pairs == 3) item_sums<3>(l, &b0, &b1, acc);
        else item_sums<4>(l, &b0, &b1, acc);

        // Four row tiles at a time through 16 KB of LDS of the wave's own (nobody
        // reads rows there now), so that a row's outputs are stored side by side.
        // A row has 16 pieces of 4 outputs, piece c at c ^ row % 16 again.
        v4f* own = (v4f*)((l.wave & 2 ? b1 : b0).codes) + (l.wave & 1) * 1024;
        const int r16 = l.lane % 16, g = l.lane / 16;
        const int width = p.paired ? 8 : 16, n0 = t0 * kMxTileRows / (p.paired ? 2 : 1);  // pieces, first output
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (2 * half >= pairs) break;
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int f = 0; f < kWaveTiles; f += 2) {
                    v4f v = acc[4 * half + m][f], u = acc[4 * half + m][f + 1];
                    v4f* row = own + (m * 16 + r16) * 16;
                    if (p.paired) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], u[i]);
                        row[(f / 2 * 4 + g) ^ r16] = v;
                    } else {
                        row[(f * 4 + g) ^ r16] = v;
                        row[(f * 4 + 4 + g) ^ r16] = u;
                    }
                }
            const int rows = min(64, it.rows - 64 * half), step = 64 / width;
            for (int r = l.lane / width; r < rows; r += step) {
                const int c = l.lane % width, to = it.row0 + 64 * half + r;
                v4f v = own[r * 16 + (c ^ (r % 16))];
                if (p.src && (uint64_t)(int64_t)p.src[to] >= (uint64_t)p.x_rows) v = v4f{0, 0, 0, 0};
                if (n0 + 4 * c < a.n_out) store_out(a, to, n0 + 4 * c, v);
            }
        }
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
    const int64_t hit = p.rows < p.E ? p.rows : p.E;
    if (p.rows <= 16 * (int64_t)p.E) {
        a.nb = (a.tiles + NF - 1) / NF;
        const int64_t n = (p.rows / 16 + hit) * a.nb, most = 256 * 4;
        hipLaunchKernelGGL((stream_kernel<1, NF>), dim3((uint32_t)(n < most ? n : most)), dim3(kThreads), 0, st, a);
    } else {
        a.nb = (a.tiles + kWaves * kWaveTiles - 1) / (kWaves * kWaveTiles);
        const int64_t n = (p.rows / (16 * kRowTiles) + hit) * a.nb, most = 256 * 2;
        hipLaunchKernelGGL(tile_kernel, dim3((uint32_t)(n < most ? (n + 7) / 8 * 8 : most)), dim3(kThreads), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace strata_moe
