// Microscaled 4-bit floating point: rounding rows to it, reading them back,
// packing weight matrices, and the (grouped) product of packed weights with
// rounded rows.
//
// Format.  32 consecutive values of a row share a scale 2^(byte - 127); a value
// is a sign and one of 0, .5, 1, 1.5, 2, 3, 4, 6 (code bit 3 the sign, 2..1 the
// exponent, 0 the mantissa), two to a byte, the first in the low half.
#include <algorithm>

#include "block.h"
#include "mxfp.h"

namespace strata_moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

// ------------------------------------------------------ rounding and reading
// A thread takes 8 consecutive values, 4 threads a block of 32: its largest magnitude
// goes between them by two exchanges, and neighbouring threads read and write
// neighbouring bytes.  The memory bounds both ways: 8192 rows of 2560 in fp32 take
// 23.7 us to round (4.0 TB/s; 14.5 where the rows are still in the last cache) and
// 16.7 to read back (5.7 TB/s, the codes from that cache), 203 rows of 1056 in bf16
// 2.6 and 2.4, a launch.
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

// One wave per (expert, tile, group of 16 blocks).  A group is four steps: in step
// s lane l holds row l % 16 and block 4 (l / 16) + s of the group, what the matrix
// unit reads, so a lane's blocks are neighbours and its scale dword is theirs, byte
// s for step s.  The last group keeps only the blocks there are (mx_step_at).  The
// memory bounds it: 512 matrices of 2048 x 2560 take 690 us, 1.43 GB in and out, 4.1
// TB/s; of 2560 x 1024 322 us, 4.4.
__global__ __launch_bounds__(64) void pack_kernel(const uint8_t* __restrict__ codes,
                                                  const uint8_t* __restrict__ scales, int rows, int cols, int paired,
                                                  uint8_t* __restrict__ packed, int64_t stride, int64_t tile_bytes) {
    const int lane = threadIdx.x, g = lane / 16, blocks = cols / 32;
    const int q = blockIdx.x, have = min(16, blocks - q * 16);
    const int row = tile_row(blockIdx.y, lane % 16, rows, paired);
    const int64_t e = blockIdx.z;
    uint8_t* dst = packed + e * stride + blockIdx.y * tile_bytes + (int64_t)q * kMxGroupBytes;
    uint32_t sc = 0;
    for (int s = 0; s < 4; ++s) {
        const int b = 4 * g + s;
        if (b >= have) continue;
        uint4 v = {0, 0, 0, 0};
        if (row >= 0) {
            const int64_t at = (e * rows + row) * blocks + q * 16 + b;
            v = ((const uint4*)codes)[at];
            sc |= (uint32_t)scales[at] << (8 * s);
        }
        *(uint4*)(dst + mx_step_at(have, s) + lane * 16) = v;
    }
    *(uint32_t*)(dst + have * kMxBlockBytes + lane * 4) = sc;
}

// ------------------------------------------------------------------- product
struct ProductArgs {
    MxProduct p;
    int64_t tile_bytes;
    int32_t tiles, n_out;   // packed tiles of an expert; outputs of a row
    int32_t blocks, groups; // of 32 and of 512 reduction values
    int32_t steps;          // matrix-unit products along the reduction
    int32_t nb;             // work items along the outputs
    int32_t item_rows;      // rows of a work item, at most
    int32_t vec_out;        // rows of out take 16-byte stores
    int32_t vec_out4;       // ... stores of four outputs
};

// The work list.  An item is one tile of at most mt rows of one expert times one run of
// its outputs; items are numbered expert by expert, within an expert kTogether
// tiles by kTogether tiles, there run by run, and within a run tile by tile, so
// that the workgroups that read the same weights or rows run at about the same
// time (in one L2).  pre[e] = row tiles of the experts below
// e; the caller's offsets are clamped to [0, rows], whatever they hold.
constexpr int kMaxE = 1024;
constexpr int kTogether = 8;
struct List {
    int32_t pre[kMaxE + 1];
    int32_t row[kMaxE + 1];  // the clamped offsets
};
__device__ __forceinline__ int32_t clamp_row(int32_t v, int32_t rows) { return v < 0 ? 0 : v > rows ? rows : v; }

__device__ __forceinline__ void make_list(const MxProduct& p, int mt, List& L, int32_t* wave_sum) {
    if (!p.offsets) {
        if (threadIdx.x == 0) {
            L.pre[0] = L.row[0] = 0;
            L.pre[1] = ((int32_t)p.rows + mt - 1) / mt;
            L.row[1] = (int32_t)p.rows;
        }
        __syncthreads();
        return;
    }
    // a thread takes a run of experts, its first sum the scan's
    const int per = (p.E + (int)blockDim.x - 1) / (int)blockDim.x, rows = (int)p.rows;
    const int e0 = threadIdx.x * per, e1 = min(p.E, e0 + per);
    auto tiles = [&](int e, int32_t* first) {
        const int32_t a = clamp_row(p.offsets[e], rows), b = clamp_row(p.offsets[e + 1], rows);
        *first = a;
        if (e == p.E - 1) L.row[p.E] = b;
        return b > a ? (b - a + mt - 1) / mt : 0;
    };
    int32_t s = 0, row;
    for (int e = e0; e < e1; ++e) s += tiles(e, &row);
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
    for (int e = e0; e < e1; ++e) {
        L.pre[e] = at;
        at += tiles(e, &row);
        L.row[e] = row;
    }
    if (e1 == p.E && e0 < e1) L.pre[p.E] = at;
    __syncthreads();
}

// Wave-uniform, in scalar registers.
struct Item {
    int32_t e, run, row0;
    int32_t rows;
};
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }

template <int kUnit>
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
    uint32_t left = (uint32_t)(u - (int64_t)first * nb);  // below tiles * nb < 2^31
    const uint32_t wave = left / (uint32_t)(kTogether * nb);
    left -= wave * (uint32_t)(kTogether * nb);
    const uint32_t wide = min((uint32_t)kTogether, (uint32_t)tiles - wave * kTogether);
    const uint32_t run = left / wide, t = wave * kTogether + left - run * wide;
    const int32_t r0 = uniform(L.row[e]), r1 = uniform(L.row[e + 1]);
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
// two parts: its rounding alone would cost |g| 2^-24 of the result.  Where the power
// is 0 or infinite (also g = +-inf, and g past 2.35e38, where the product is) the
// second part is left out: it is infinite or NaN there itself.  Rounded in fp32 at
// each step, with the unit's power and reciprocal (1 ulp each), for speed: fp32
// outputs of one token's gate/up are 5.0e-8 off in relative terms, 4.6e-8 with
// PyTorch's exp and a division; rounding to 16 bits hides both.
__device__ __forceinline__ float swiglu(float g, float u) {
    const float hi = -g * 1.44269502f;
    const float lo = fmaf(-g, 1.44269502f, -hi) + -g * 1.92596303e-8f;
    float e = __builtin_amdgcn_exp2f(hi);
    if (e > 0.0f && e < __builtin_inff()) e = fmaf(e, lo * 0.693147182f, e);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

__device__ __forceinline__ void store_out(const ProductArgs& a, int32_t row, int n, v4f v) {
    float f[4] = {v[0], v[1], v[2], v[3]};
    store4_any(a.p.out, a.p.dtype, row * a.p.out_stride, n, a.n_out, a.vec_out4, f);
}

// Few rows: latency bounds it (one token's ten experts, 2560 -> 2 x 1024: 8.7 us,
// of which the 28 MB of weights need 5.5, or 7.5 where they are still in the last
// cache; 406 rows of six experts, 544 -> 333: 5.9).  An item is up to 16 rows of an
// expert times kFewTiles tiles of its weights.  A wave takes up to four steps at a
// time, so with a wave for every four of them all loads of an item are in flight
// together; the waves' sums are added in wave order through LDS.
// kList: the items of the work list, shared out.  Otherwise a workgroup per row
// and run, which looks the row's expert up and works if the row begins one of the
// expert's tiles: no list, no scan, the offsets and the rows' sources in one
// round of loads.
constexpr int kFewWaves = 8;
constexpr int kFewTiles = 4;

__device__ __forceinline__ void few_item(const ProductArgs& a, int e, int run, int row, int rows, int src, int wave,
                                         int waves, v4f (*part)[kFewTiles][64]) {
    const MxProduct& p = a.p;
    const int lane = threadIdx.x % 64, r16 = lane % 16, g = lane / 16;
    const uint8_t* wt[kFewTiles];
#pragma unroll
    for (int f = 0; f < kFewTiles; ++f)
        wt[f] = p.packed + e * p.stride + min(run * kFewTiles + f, a.tiles - 1) * a.tile_bytes;
    v4f acc[kFewTiles];
#pragma unroll
    for (int f = 0; f < kFewTiles; ++f) acc[f] = v4f{0, 0, 0, 0};
    const int s1 = a.steps * (wave + 1) / waves;
    constexpr int kAtOnce = 4;
    for (int s0 = a.steps * wave / waves; s0 < s1; s0 += kAtOnce) {
        v4i w[kAtOnce][kFewTiles], x[kAtOnce];
        int ws[kAtOnce][kFewTiles], xs[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            // step st of group q, which has `have` blocks (for a step past the wave's, its last again)
            const int s = min(s0 + i, s1 - 1), q = s / 4, st = s % 4, have = min(16, a.blocks - q * 16);
            const bool mine = 4 * g + st < have;
#pragma unroll
            for (int f = 0; f < kFewTiles; ++f) {
                const uint8_t* at = wt[f] + (int64_t)q * kMxGroupBytes;
                w[i][f] = v4i{0, 0, 0, 0};
                if (mine) w[i][f] = *(const v4i*)(at + mx_step_at(have, st) + lane * 16);
                ws[i][f] = *(const int*)(at + have * kMxBlockBytes + lane * 4) >> (8 * st);
            }
            x[i] = v4i{0, 0, 0, 0};
            xs[i] = 0;
            if (src >= 0 && r16 < rows && mine && s0 + i < s1) {
                const int64_t b = (int64_t)src * a.blocks + q * 16 + 4 * g + st;
                x[i] = ((const v4i*)p.codes)[b];
                xs[i] = p.scales[b];
            }
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
            for (int f = 0; f < kFewTiles; ++f)
                if (s0 + i < s1)
                    acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w[i][f]), operand(x[i]), acc[f],
                                                                              4, 4, 0, ws[i][f], 0, xs[i]);
    }
#pragma unroll
    for (int f = 0; f < kFewTiles; ++f) part[wave][f][lane] = acc[f];
    __syncthreads();
    // outputs: lane holds row lane % 16 and 4 consecutive outputs of a tile
    const int per = p.paired ? 2 : 1;
    for (int f = wave * per; f < kFewTiles; f += waves * per) {
        v4f v = part[0][f][lane];
        for (int w = 1; w < waves; ++w) v += part[w][f][lane];
        if (p.paired) {
            v4f up = part[0][f + 1][lane];
            for (int w = 1; w < waves; ++w) up += part[w][f + 1][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], up[i]);
        }
        if (src < 0) v = v4f{0, 0, 0, 0};  // zeros times a weight of NaN are not 0
        const int n = (run * kFewTiles + f) / per * kMxTileRows + 4 * g;
        if (r16 < rows && n < a.n_out) store_out(a, row + r16, n, v);
    }
}

// The lane's row of x for row `row` + lane % 16 of the output, or -1.
__device__ __forceinline__ int few_source(const MxProduct& p, int row) {
    int src = row + (int)(threadIdx.x % 16);
    if (src >= p.rows) return -1;
    if (p.src) src = p.src[src];
    return src >= p.x_rows ? -1 : src;
}

template <bool kList>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(ProductArgs a) {
    __shared__ v4f part[kFewWaves][kFewTiles][64];
    const MxProduct& p = a.p;
    const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), waves = blockDim.x / 64, rows = (int)p.rows;
    if constexpr (kList) {
        __shared__ List L;
        __shared__ int32_t wave_sum[kFewWaves];
        make_list(p, kMxTileRows, L, wave_sum);
        const int64_t items = (int64_t)uniform(L.pre[p.E]) * a.nb;
        for (int64_t u = blockIdx.x; u < items; u += gridDim.x) {
            const Item it = find_item<1>(p, L, a.nb, u);
            few_item(a, it.e, it.run, it.row0, it.rows, few_source(p, it.row0), wave, waves, part);
            __syncthreads();
        }
        return;
    }
    const int row = p.offsets ? blockIdx.y : blockIdx.y * kMxTileRows;
    const int src = few_source(p, row);
    int e = 0, end = rows;
    if (p.offsets) {
        e = -1;
        for (int e0 = 0; e0 < p.E && e < 0; e0 += 256) {
            int lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = e0 + i * 64 + lane;
                lo[i] = k < p.E ? p.offsets[k] : 0;
                hi[i] = k < p.E ? p.offsets[k + 1] : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = row - clamp_row(lo[i], rows);
                const uint64_t has = __ballot(at >= 0 && at % kMxTileRows == 0 && row < clamp_row(hi[i], rows));
                if (!has || e >= 0) continue;
                const int k = __builtin_ctzll(has);
                e = e0 + i * 64 + k;
                end = clamp_row(__builtin_amdgcn_readlane(hi[i], k), rows);
            }
        }
        if (e < 0) return;
    }
    few_item(a, e, blockIdx.x, row, min(kMxTileRows, end - row), src, wave, waves, part);
}

// Many rows.  A workgroup (two to a CU) takes up to 6 tiles of rows (96) and 16 of
// weights, 4 to a wave.  The rows' codes of 512 reduction values (a group) go to
// LDS while the group before is multiplied (two buffers); each wave reads its own
// weights from memory straight into registers, three steps of 128 ahead.  Row
// tiles come in pairs: an item of fewer rows leaves out the pairs it lacks.
//
// What bounds it: where an expert has a few hundred rows, the memory (8192 tokens,
// ten of 512 experts, 2560 -> 2 x 1024 SwiGLU: 405 us; it moves 1.97 GB, 4.9 TB/s of a
// copy's 5.1, of which 1.6 it cannot do without: the rest is rows read again past an
// L2, 0.26 GB, and weights, 0.09; down 1024 -> 2560: 262 us, 1.2 GB).  With one
// matrix, the matrix unit and what feeds it (8192 rows, 4096 -> 4096: 78 us, 3.5
// PFLOP/s; the unit alone reaches 6.7 to 7.3 on random values; without weight loads
// 63, without rows' 74, without both and the stores 54): in a step of 128 a CU's two
// workgroups load 45 KB, some 700 cycles, for 768 of products.
//
// All 256 registers are in use: 2 to 4 values, which each item needs once, wait in
// scratch memory; nothing in the loop over the groups does.
//
// What was measured against it (us, the three calls above, 405 / 258 / 77): items of
// 128 rows with weights two steps ahead 411 / 278 / 77; weights through the compiler's
// own waits and LDS loads it sees 413 / 255 / 85; weights read past the caches 534 / 317
// / 107; runs of one item after the other without kTogether 408 / 262 / 84; stores
// through the caches 408 / 263 / 78; workgroups that change places to even out odd
// row counts 413 against 414.
constexpr int kWaves = 4;
constexpr int kRowTiles = 6;
constexpr int kTableRows = 128;  // of an item's row table: a multiple of the 64 rows of four scale tiles
constexpr int kWaveTiles = 4;
// [row][16 pieces]: 16 bytes a block; piece c of row r lies at c ^ turned(r % 16).
// A product's read (lane l: row l % 16, piece 4 (l / 16) + step) is served 16 lanes at
// a time, each of lanes 0-3, 12-15, 20-27 and so on in turn: two quarters of the rows
// at c and the other two at c ^ 4, which must all differ.  So the rows' high bits,
// which tell the quarters apart, turn the pieces' low ones (c ^ r % 16 had two lanes
// to a bank: 10.7 million LDS cycles of the projection's, 6.5 with this).
__device__ __forceinline__ int turned(int r) { return r >> 2 | (r & 3) << 2; }
struct Rows {
    v4i codes[kRowTiles * 16 * 16];
    int scales[kTableRows / 16 * 64];  // [tile][lane]: the lane's scales of a group, byte s for step s
};

using Resource = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Resource resource(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, bytes, 0x00027000);
}
using LdsPtr = void __attribute__((address_space(3)))*;

struct TileLoads {
    const uint8_t* codes;    // x
    uint32_t last_codes;     // where its last 16 bytes begin
    Resource scales;
    uint32_t last_scales;    // where their last four bytes begin
    int32_t blocks, groups, tiles, tile_bytes;
    int32_t lane, wave;
};
// One group of one item to load: wave-uniform.
struct Part {
    Resource weights;       // the item's expert
    const uint32_t* first;  // [128] LDS: first block in x of each row of the item (and kZeroRow)
    int32_t t0;             // the wave's first weight tile
    int32_t pairs;          // of the item's row tiles
    int32_t q;              // the group
    uint32_t off;           // 0, or kNowhere: load nothing
};
// In the table: the row's src is outside x, its result zeros (it loads row 0; x has
// less than 2^28 blocks, so the flag leaves the address).
constexpr uint32_t kZeroRow = 0x80000000u;
// A lane's offset that no array reaches.  (The scalar offsets always stay in the
// arrays: the range check subtracts them from the size.)
constexpr uint32_t kNowhere = 0xf0000000u;

// A lane's byte offsets in x of an item's rows: of the 16 bytes that it loads in
// each instruction (4 rows of 256 bytes), and of the scales of its two rows.
struct RowAddresses {
    uint32_t codes[kRowTiles], scales[2];
};
__device__ __forceinline__ void row_addresses(const TileLoads& l, const uint32_t* first, RowAddresses& ad) {
#pragma unroll
    for (int i = 0; i < kRowTiles; ++i) {
        const int r = (i * kWaves + l.wave) * 4 + l.lane / 16;
        ad.codes[i] = (first[r] + ((l.lane % 16) ^ turned(r % 16))) * 16;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) ad.scales[i] = first[(l.wave + 4 * i) * 16 + l.lane % 16] & ~kZeroRow;
}
// Start the loads of a pair of row tiles of group q.  In asm, so that the compiler
// does not have every read of LDS wait for them: its own waits then count too few
// loads in flight and wait for more than they need, never for less.  The wait for
// these is that for the row scales, which are loaded behind them (loads return in
// the order they were issued).  A piece past the row's end is any of x: it meets
// weights of 0.
__device__ __forceinline__ void load_pair(const TileLoads& l, const RowAddresses& ad, int q, int pair, uint32_t to) {
#pragma unroll
    for (int i = 2 * pair; i < 2 * pair + 2; ++i) {
        const uint32_t at = min(ad.codes[i] + q * 256, l.last_codes);
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :
                     : "s"(to + (i * kWaves + l.wave) * 1024), "v"(at), "s"(l.codes)
                     : "memory");
    }
}
__device__ __forceinline__ uint32_t lds(const void* p) { return uniform((uint32_t)(uintptr_t)(LdsPtr)p); }

// The scales of the rows of tiles wave and wave + 4: a lane's are neighbours, one
// unaligned dword, read from at most the array's last four bytes.
__device__ __forceinline__ uint32_t scales_at(const TileLoads& l, const Part& t, uint32_t row) {
    return row + (uint32_t)(t.q * 16 + 4 * (l.lane / 16));
}
__device__ __forceinline__ void load_row_scales(const TileLoads& l, const Part& t, const RowAddresses& ad, int* sc) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t at = min(scales_at(l, t, ad.scales[i]), l.last_scales);
        sc[i] = __builtin_amdgcn_raw_buffer_load_b32(l.scales, at | t.off, 0, 0);
    }
}
// Past the row's end a block gets scale 2^-127 (its codes are any, and meet weights
// of 0).
__device__ __forceinline__ void keep_row_scales(const TileLoads& l, const Part& t, const RowAddresses& ad,
                                                const int* sc, Rows* to) {
    const int have = l.blocks - (t.q * 16 + 4 * (l.lane / 16));  // blocks of the row from the lane's first on
    const uint32_t mask = have >= 4 ? ~0u : have <= 0 ? 0u : (1u << (8 * have)) - 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t at = scales_at(l, t, ad.scales[i]), past = at - min(at, l.last_scales);
        const uint32_t v = past < 4 ? (uint32_t)sc[i] >> (8 * past) : 0u;
        to->scales[(l.wave + 4 * i) * 64 + l.lane] = (int)(v & mask);
    }
}

__device__ __forceinline__ uint32_t weights_at(const TileLoads& l, const Part& t, int f) {
    return (uint32_t)min(t.t0 + f, l.tiles - 1) * (uint32_t)l.tile_bytes + t.q * kMxGroupBytes;
}
// Step st of the wave's tiles; lanes without a block in it get zeros.
__device__ __forceinline__ v4i load_weights(const TileLoads& l, const Part& t, int st, int f) {
    const int have = min(16, l.blocks - t.q * 16);
    const uint32_t off = (uint32_t)l.lane * 16 | (4 * (l.lane / 16) + st < have ? t.off : kNowhere);
    return __builtin_bit_cast(
        v4i, __builtin_amdgcn_raw_buffer_load_b128(t.weights, off, weights_at(l, t, f) + mx_step_at(have, st), 0));
}
__device__ __forceinline__ void load_weight_scales(const TileLoads& l, const Part& t, int* sc) {
    const int have = min(16, l.blocks - t.q * 16);
#pragma unroll
    for (int f = 0; f < kWaveTiles; ++f)
        sc[f] = __builtin_amdgcn_raw_buffer_load_b32(t.weights, l.lane * 4 | t.off,
                                                     weights_at(l, t, f) + have * kMxBlockBytes, 0);
}

// Keeps the products before it before it: they have no side effects, and the
// compiler would gather those of a whole group behind its loads.
__device__ __forceinline__ void stay(v4f& a, v4f& b) { asm volatile("" : "+v"(a), "+v"(b)); }

struct WeightRegs {
    v4i w[4][kWaveTiles];  // [step]
    int s[kWaveTiles];
};
struct Pair {
    v4i x[2];
};
template <int ST>
__device__ __forceinline__ Pair read_pair(const Rows* from, int lane, int pair) {
    const int r16 = lane % 16;
    const v4i* at = from->codes + r16 * 16 + ((4 * (lane / 16) + ST) ^ turned(r16)) + pair * 512;
    return Pair{{at[0], at[256]}};
}

template <int ST>
__device__ __forceinline__ v4f product(v4i w, v4i x, v4f c, int ws, int xs) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(w), operand(x), c, 4, 4, ST, ws, ST, xs);
}

// Step ST of a group: the products of the item's pairs of row tiles, of which
// `first` is read already; returns the first pair of the next step.  Between the
// first pair's products the weights of step `load` of group u are loaded.
template <int ST, int LOAD>
__device__ __forceinline__ Pair step_products(const TileLoads& l, int pairs, const Rows* from, const Pair& first,
                                              const int* xs, WeightRegs& r, const Part& u, v4f (*acc)[kWaveTiles]) {
    static_assert(kRowTiles == 6, "three pairs");
    Pair ahead{}, next = read_pair<ST>(from, l.lane, 1);
    if (ST < 3) ahead = read_pair<ST + 1>(from, l.lane, 0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < kWaveTiles; ++f) {
        acc[0][f] = product<ST>(r.w[ST][f], first.x[0], acc[0][f], r.s[f], xs[0]);
        acc[1][f] = product<ST>(r.w[ST][f], first.x[1], acc[1][f], r.s[f], xs[1]);
        stay(acc[0][f], acc[1][f]);
        __builtin_amdgcn_sched_barrier(0);
        r.w[LOAD][f] = load_weights(l, u, LOAD, f);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (pairs > 1) {
        const Pair last = read_pair<ST>(from, l.lane, 2);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < kWaveTiles; ++f) {
            acc[2][f] = product<ST>(r.w[ST][f], next.x[0], acc[2][f], r.s[f], xs[2]);
            acc[3][f] = product<ST>(r.w[ST][f], next.x[1], acc[3][f], r.s[f], xs[3]);
            stay(acc[2][f], acc[3][f]);
        }
        if (pairs > 2) {
#pragma unroll
            for (int f = 0; f < kWaveTiles; ++f) {
                acc[4][f] = product<ST>(r.w[ST][f], last.x[0], acc[4][f], r.s[f], xs[4]);
                acc[5][f] = product<ST>(r.w[ST][f], last.x[1], acc[5][f], r.s[f], xs[5]);
                stay(acc[4][f], acc[5][f]);
            }
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    return ahead;
}

// What this wave wrote to or read from LDS is done, for all waves.
__device__ __forceinline__ void meet() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Group `t` from `now`, the loads of the group after it, `u`, into `next` beside
// it; each step's weights are loaded three steps ahead.  table: the thread's value
// for the next item's row table at `entry`, there behind any group.
__device__ __forceinline__ void group(const TileLoads& l, const Part& t, const Part& u, const RowAddresses& ad,
                                      Rows* now, Rows* next, WeightRegs& r, uint32_t* entry, uint32_t table,
                                      v4f (*acc)[kWaveTiles]) {
    int sc[2], ws[kWaveTiles], xs[kRowTiles];
    const uint32_t to = lds(next->codes);
    Pair x = read_pair<0>(now, l.lane, 0);
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m) xs[m] = now->scales[m * 64 + l.lane];
    x = step_products<0, 3>(l, t.pairs, now, x, xs, r, t, acc);
    load_pair(l, ad, u.q, 0, to);
    x = step_products<1, 0>(l, t.pairs, now, x, xs, r, u, acc);
    if (u.pairs > 1) load_pair(l, ad, u.q, 1, to);
    load_weight_scales(l, u, ws);
    x = step_products<2, 1>(l, t.pairs, now, x, xs, r, u, acc);
    if (u.pairs > 2) load_pair(l, ad, u.q, 2, to);
    __builtin_amdgcn_sched_barrier(0);
    load_row_scales(l, u, ad, sc);
    __builtin_amdgcn_sched_barrier(0);
    step_products<3, 2>(l, t.pairs, now, x, xs, r, u, acc);
    if (threadIdx.x < kTableRows) entry[threadIdx.x] = table;
    keep_row_scales(l, u, ad, sc, next);
#pragma unroll
    for (int f = 0; f < kWaveTiles; ++f) r.s[f] = ws[f];
    meet();
}

// All groups of an item, the last one beside the loads of the first group of the
// item after it.
__device__ __forceinline__ void item_sums(const TileLoads& l, Part t, const Part& after, RowAddresses& ad, Rows* b,
                                          int& turn, WeightRegs& r, uint32_t* entry, uint32_t table,
                                          v4f (*acc)[kWaveTiles]) {
#pragma unroll 1
    for (int q = 0; q < l.groups; ++q) {
        t.q = q;
        Part u = t;
        u.q = q + 1;
        if (q + 1 == l.groups) {
            u = after;
            if (!after.off) row_addresses(l, after.first, ad);
        }
        group(l, t, u, ad, b + turn, b + (turn ^ 1), r, entry, table, acc);
        turn ^= 1;
    }
}

// An item's results: a row tile at a time through 4 KB of LDS of the wave's own
// (`own`), so that neighbouring lanes store 16 bytes each of one row.  A row has
// kUnits such units; unit c lies at c ^ row, for the banks' sake.
template <typename T, bool kPaired>
__device__ __forceinline__ void store_item(const ProductArgs& a, const Item& it, const Part& t, const TileLoads& l,
                                           v4f* own, v4f (*acc)[kWaveTiles]) {
    typedef T Piece __attribute__((ext_vector_type(4)));
    constexpr int kOutputs = kWaveTiles * kMxTileRows / (kPaired ? 2 : 1), kPer = 16 / (int)sizeof(T);
    constexpr int kUnits = kOutputs / kPer, kRows = 64 / kUnits;  // rows an instruction
    typedef T Unit __attribute__((ext_vector_type(kPer)));
    const int r16 = l.lane % 16, g = l.lane / 16, n0 = t.t0 * kMxTileRows / (kPaired ? 2 : 1);
    const int c = l.lane % kUnits, n = n0 + c * kPer, r0 = l.lane / kUnits;
    const bool whole = a.vec_out && n0 + kOutputs <= a.n_out;  // all of the wave's units are 16-byte stores
    T* out = (T*)a.p.out + (int64_t)(it.row0 + r0) * a.p.out_stride + n;
#pragma unroll
    for (int m = 0; m < kRowTiles; ++m) {
        if (m / 2 >= t.pairs) continue;
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int f = 0; f < kWaveTiles; f += kPaired ? 2 : 1) {
            v4f v = acc[m][f];
            if (kPaired)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], acc[m][f + 1][i]);
            Piece o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = (T)v[i];
            const int piece = (kPaired ? f / 2 : f) * 4 + g, unit = piece * 4 / kPer;
            *(Piece*)((char*)(own + r16 * kUnits + (unit ^ r16 % kUnits)) + piece * 4 % kPer * sizeof(T)) = o;
        }
        const int rows = it.rows - 16 * m;
        if (whole) {
            v4f u[16 / kRows];
#pragma unroll
            for (int i = 0; i < 16 / kRows; ++i)
                u[i] = own[(i * kRows + r0) * kUnits + (c ^ (i * kRows + r0) % kUnits)];
#pragma unroll
            for (int i = 0; i < 16 / kRows; ++i)
                if (i * kRows + r0 < rows)  // past the caches: nobody reads them in this call
                    __builtin_nontemporal_store(u[i], (v4f*)(out + (16 * m + i * kRows) * a.p.out_stride));
        } else {
#pragma unroll 1
            for (int r = r0; r < min(16, rows); r += kRows) {
                const Unit u = __builtin_bit_cast(Unit, own[r * kUnits + (c ^ r % kUnits)]);
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (n + j < a.n_out) out[(16 * m + r - r0) * a.p.out_stride + j] = u[j];
            }
        }
    }
}

__device__ __forceinline__ uint32_t first_block(const ProductArgs& a, const Item& it) {
    if (threadIdx.x >= kTableRows) return 0;
    int32_t s = it.row0 + min((int)threadIdx.x, it.rows - 1);
    if (a.p.src) s = a.p.src[s];
    return s < 0 || s >= a.p.x_rows ? kZeroRow : (uint32_t)s * (uint32_t)a.blocks;
}

template <typename T, bool kPaired>
__global__ __launch_bounds__(kThreads, 2) void tile_kernel(ProductArgs a) {
    __shared__ Rows b[2];
    __shared__ uint32_t first[2][kTableRows];  // of this item and the next, in turn
    __shared__ List L;
    __shared__ int32_t wave_sum[kWaves];
    const MxProduct& p = a.p;
    make_list(p, a.item_rows, L, wave_sum);
    const int64_t items = (int64_t)uniform(L.pre[p.E]) * a.nb;
    // workgroups of one XCD (every eighth) take one run of the items
    const int xcd = blockIdx.x % 8, per = gridDim.x / 8;
    const int64_t u1 = items * (xcd + 1) / 8;
    int64_t u = items * xcd / 8 + blockIdx.x / 8;
    if (u >= u1) return;
    TileLoads l;
    l.codes = p.codes;
    l.last_codes = (uint32_t)(p.x_rows * a.blocks * 16) - 16;
    l.scales = resource(p.scales, (uint32_t)(p.x_rows * a.blocks));
    l.last_scales = (uint32_t)(p.x_rows * a.blocks) - 4;
    l.blocks = a.blocks;
    l.groups = a.groups;
    l.tiles = a.tiles;
    l.tile_bytes = (int32_t)a.tile_bytes;
    l.lane = threadIdx.x % 64;
    l.wave = uniform(threadIdx.x / 64);
    auto part = [&](const Item& it, const uint32_t* table) {
        Part t;
        t.weights = resource(p.packed + it.e * p.stride, (uint32_t)(a.tiles * a.tile_bytes));
        t.first = table;
        t.t0 = it.run * (kWaves * kWaveTiles) + l.wave * kWaveTiles;
        t.pairs = (it.rows + 31) / 32;
        t.q = 0;
        t.off = 0;
        return t;
    };

    // the first item's first group
    Item it = find_item<2>(p, L, a.nb, u);
    if (threadIdx.x < kTableRows) first[0][threadIdx.x] = first_block(a, it);
    meet();
    Part t = part(it, first[0]);
    WeightRegs r;
    RowAddresses ad;
    int turn = 0, table = 0;
    {
        int sc[2];
        row_addresses(l, t.first, ad);
#pragma unroll
        for (int h = 0; h < kRowTiles / 2; ++h)
            if (h < t.pairs) load_pair(l, ad, 0, h, lds(b[0].codes));
        load_weight_scales(l, t, r.s);
        __builtin_amdgcn_sched_barrier(0);
        load_row_scales(l, t, ad, sc);
#pragma unroll
        for (int f = 0; f < kWaveTiles; ++f)
#pragma unroll
            for (int st = 0; st < 3; ++st) r.w[st][f] = load_weights(l, t, st, f);
        keep_row_scales(l, t, ad, sc, b);
    }
    for (;;) {
        const bool more = u + per < u1;
        const Item then = more ? find_item<2>(p, L, a.nb, u + per) : it;
        Part after = part(then, first[table ^ 1]);
        if (!more) after.off = kNowhere;
        uint32_t* entry = first[table ^ 1];
        const uint32_t block = first_block(a, then);
        if (a.groups == 1) {  // the only group already loads by the table
            meet();           // which other waves read to store the item before
            if (threadIdx.x < kTableRows) entry[threadIdx.x] = block;
        }
        meet();
        v4f acc[kRowTiles][kWaveTiles];
#pragma unroll
        for (int m = 0; m < kRowTiles; ++m)
#pragma unroll
            for (int f = 0; f < kWaveTiles; ++f) acc[m][f] = v4f{0, 0, 0, 0};
        item_sums(l, t, after, ad, b, turn, r, entry, block, acc);

        v4f* own = (v4f*)b[turn ^ 1].codes + l.wave * 256;  // the buffer that the last group was read from
        const bool zeros = __any((first[table][l.lane] | first[table][64 + l.lane]) & kZeroRow);
        if (zeros) {
#pragma unroll
            for (int m = 0; m < kRowTiles; ++m)
                if (first[table][m * 16 + l.lane % 16] & kZeroRow)
#pragma unroll
                    for (int f = 0; f < kWaveTiles; ++f) acc[m][f] = v4f{0, 0, 0, 0};
        }
        store_item<T, kPaired>(a, it, t, l, own, acc);
        if (!more) return;
        u += per;
        it = then;
        t = after;
        table ^= 1;
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
    const dim3 grid((cols + 511) / 512, (uint32_t)mx_tiles(rows, paired), ne);
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
    a.blocks = p.cols / 32;
    a.groups = (a.blocks + 15) / 16;
    a.steps = a.blocks / 16 * 4 + std::min(4, a.blocks % 16);
    const size_t el = dtype_bytes(p.dtype);
    const uintptr_t align = (uintptr_t)p.out | (uintptr_t)(p.out_stride * (int64_t)el);
    a.vec_out = align % 16 == 0;
    a.vec_out4 = align % (4 * el) == 0;
    // The kernel by the number of its items, at most (us, MI355X; few: a workgroup
    // per row and run / the list / the tiles of many rows).  The first border lies
    // between 320 lookups and 640, where the first and the last are level; the
    // second between the list's 3930 steps and 11520, with none measured nearer.
    //   one token, ten experts, 2560 -> 2 x 1024 (320 lookups)   7.8 / 12.9 / 11.0
    //   two tokens (640)                                        14.8 / 21.1 / 15.3
    //   128 rows, 2560 -> 2560, one matrix (320)                 6.9 /  9.9 /  8.9
    //   256 rows (640)                                           9.7 / 13.4 /  9.1
    //   406 rows, six experts, 544 -> 333 (2436; 930 steps)      7.4 /  5.9 /  8.5
    //   2000 rows, the same (786 items of 5 steps)              25.2 /  7.5 /  9.1
    //   2048 rows, 16 experts, 512 -> 2 x 640 (2880 of 4)       47.8 / 22.9 /  8.2
    const int64_t hit = p.rows < p.E ? p.rows : p.E, few_runs = (a.tiles + kFewTiles - 1) / kFewTiles;
    auto tiles = [&](int mt) { return p.offsets ? p.rows / mt + hit : (p.rows + mt - 1) / mt; };
    const int64_t lookups = p.offsets ? p.rows : tiles(kMxTileRows), listed = tiles(kMxTileRows) * few_runs;
    const dim3 few(64 * std::min(kFewWaves, (a.steps + 3) / 4));
    if (lookups * few_runs <= 512) {
        a.nb = (int32_t)few_runs;
        hipLaunchKernelGGL(few_kernel<false>, dim3((uint32_t)few_runs, (uint32_t)lookups), few, 0, st, a);
    } else if (listed * a.steps <= 6000 || p.x_rows * a.blocks < 4) {  // (tile_kernel reads scales by four)
        a.nb = (int32_t)few_runs;
        const int64_t most = 256 * 4;
        hipLaunchKernelGGL(few_kernel<true>, dim3((uint32_t)(listed < most ? listed : most)), few, 0, st, a);
    } else {
        // As few rows an item as still leave every CU at most one (512 rows, 2560 ->
        // 2560: 9.5 us with 32, 12.5 with 96), or the most (8192 rows: 54 and 39).
        a.nb = (a.tiles + kWaves * kWaveTiles - 1) / (kWaves * kWaveTiles);
        a.item_rows = 16 * kRowTiles;
        for (int mt = 32; mt < 16 * kRowTiles; mt += 32)
            if (tiles(mt) * a.nb <= 256) {
                a.item_rows = mt;
                break;
            }
        const int64_t n = tiles(a.item_rows) * a.nb, most = 256 * 2;
        const dim3 grid((uint32_t)(n < most ? (n + 7) / 8 * 8 : most));
        auto kernel = p.dtype == kF32   ? (p.paired ? tile_kernel<float, true> : tile_kernel<float, false>)
                      : p.dtype == kF16 ? (p.paired ? tile_kernel<_Float16, true> : tile_kernel<_Float16, false>)
                                        : (p.paired ? tile_kernel<__bf16, true> : tile_kernel<__bf16, false>);
        hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace strata_moe
