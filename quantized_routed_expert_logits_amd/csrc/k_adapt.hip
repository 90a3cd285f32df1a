// Low-rank adapters of many requests beside a projection they share: token t
// of the call carries adapter a = ids[t] and
//   out[t] = y[t] + scale_a B_a (A_a x[t]),   A_a [r_a][in], B_a [out][r_a],
// and out[t] = y[t] where ids[t] is not an adapter.  Two launches: the shrink
// v[t] = A_a x[t] into the workspace, then the expand.
//
// A tile is 16 consecutive tokens, and its tokens fall into groups of one
// adapter.  Prompts give a tile one group or two; the rows of a decode batch
// are groups of their own.  One group's products are matrix products of 16
// columns, of which the group's tokens are used: a column of another group
// costs nothing that counts (the weights are read once per tile and group
// either way) and is never stored, so no value of one request reaches
// another's row.
//
// The products run on the fp32 matrix unit (16x16x4): the activations and
// sums are fp32 and an fp16 or bf16 weight widens exactly, so one kernel
// serves the three types and nothing is rounded but the sums.  A lane's
// operand is one value of k; it loads 4 consecutive values of k and feeds them
// to 4 products, which only permutes k, for both operands alike.
#include "internal.h"

namespace strata_moe {

namespace {

constexpr int kTile = 16;         // tokens of a tile
constexpr int kShrinkWaves = 8;   // waves that split a tile's reduction over in
constexpr int kRowTiles = 4;      // 16-row tiles of A per workgroup: 64 ranks
constexpr int kExpandWaves = 4;
constexpr int kExpandCols = 64;   // outputs per wave
// Calls of up to this many tokens give every group of a tile workgroups of its
// own (the latency of up to 16 groups one after another counts there); longer
// ones have tiles enough to fill the chip.
constexpr int kSpreadTokens = 256;

struct AdaptArgs {
    const float* x;
    const float* y;
    float* out;
    const int32_t* ids;
    const void* a;
    const void* b;
    const float* scale;    // or null: 1
    const int32_t* ranks;  // or null: rank
    float* v;              // [T][vs]
    int64_t T, xs, ys, os;
    int32_t L, rank, in, out_dim;
    int32_t vs;            // rank rounded up to 16
    int32_t spread;        // groups of a tile that run side by side
    int32_t copy;          // out is not y: rows without an adapter are copied
};

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));  // at any float

__device__ __forceinline__ v4f load4(const float* p) { return *reinterpret_cast<const v4f_any*>(p); }

// Four consecutive weights, as loaded and widened.
template <typename W>
struct Four;
template <>
struct Four<float> {
    v4f r;
    __device__ __forceinline__ void load(const float* p) { r = load4(p); }
    __device__ __forceinline__ void set(int j, float w) { r[j] = w; }
    __device__ __forceinline__ float get(int j) const { return r[j]; }
    __device__ __forceinline__ void zero() { r = v4f{0.f, 0.f, 0.f, 0.f}; }
};
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef _Float16 v4h_any __attribute__((ext_vector_type(4), aligned(2)));
template <>
struct Four<_Float16> {
    v4h r;
    __device__ __forceinline__ void load(const _Float16* p) { r = *reinterpret_cast<const v4h_any*>(p); }
    __device__ __forceinline__ void set(int j, _Float16 w) { r[j] = w; }
    __device__ __forceinline__ float get(int j) const { return (float)r[j]; }
    __device__ __forceinline__ void zero() { r = v4h{0, 0, 0, 0}; }
};
struct Bf16 {
    uint16_t bits;
};
typedef uint16_t v4s __attribute__((ext_vector_type(4)));
typedef uint16_t v4s_any __attribute__((ext_vector_type(4), aligned(2)));
template <>
struct Four<Bf16> {
    v4s r;
    __device__ __forceinline__ void load(const Bf16* p) { r = *reinterpret_cast<const v4s_any*>(p); }
    __device__ __forceinline__ void set(int j, Bf16 w) { r[j] = w.bits; }
    __device__ __forceinline__ float get(int j) const { return __builtin_bit_cast(float, (uint32_t)r[j] << 16); }
    __device__ __forceinline__ void zero() { r = v4s{0, 0, 0, 0}; }
};

// p[0..3] where k + j < n, zeros elsewhere (nothing is read past n).
template <typename W>
__device__ __forceinline__ void load_upto(Four<W>& f, const W* p, int k, int n) {
    f.zero();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (k + j < n) f.set(j, p[j]);
}

__device__ __forceinline__ int adapter_rank(const AdaptArgs& g, int a) {
    if (!g.ranks) return g.rank;
    const int r = g.ranks[a];
    return r < 0 ? 0 : (r > g.rank ? g.rank : r);
}

// Calls f(adapter or -1, the group's lanes as a 16-bit mask) for every group
// of the tile that is this workgroup's (the same on every wave).
template <typename F>
__device__ __forceinline__ void for_groups(const AdaptArgs& g, int64_t t0, int share, F f) {
    const int lane = threadIdx.x & 63;
    int id = -1;
    const bool on = lane < kTile && t0 + lane < g.T;
    if (on) {
        id = g.ids[t0 + lane];
        if (id < 0 || id >= g.L) id = -1;
    }
    uint32_t rest = (uint32_t)__ballot(on);
    for (int n = 0; rest; ++n) {
        const int a = __builtin_amdgcn_readlane(id, __builtin_ctz(rest));
        const uint32_t group = (uint32_t)__ballot(on && id == a);
        rest &= ~group;
        if (n % g.spread == share) f(a, group);
    }
}

// Products of steps [s0, s1) of 16 values of k: RT tiles of 16 A rows against
// the tile's tokens.
template <typename W, int RT>
__device__ __forceinline__ void shrink_steps(const AdaptArgs& g, const W* a, const float* x, bool mine, int rows,
                                             int s0, int s1, v4f (&acc)[kRowTiles]) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, k0 = 4 * (lane >> 4);
    constexpr int kUnroll = RT >= 4 ? 2 : 4;
    const int whole = g.in / 16 < s1 ? g.in / 16 : s1;
    const v4f none{0.f, 0.f, 0.f, 0.f};
    int s = s0;
    for (; s + kUnroll <= whole; s += kUnroll) {
        v4f xv[kUnroll];
        Four<W> w[kUnroll][RT];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int k = 16 * (s + u) + k0;
            xv[u] = mine ? load4(x + k) : none;
#pragma unroll
            for (int i = 0; i < RT; ++i)
                if (16 * i + r16 < rows)
                    w[u][i].load(a + (int64_t)(16 * i) * g.in + k);
                else
                    w[u][i].zero();
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[u][i].get(j), xv[u][j], acc[i], 0, 0, 0);
    }
    for (; s < s1; ++s) {  // what is left, and the step that ends inside the row
        const int k = 16 * s + k0;
        Four<float> xv;
        xv.zero();
        if (mine) load_upto<float>(xv, x + k, k, g.in);
        Four<W> w[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            w[i].zero();
            if (16 * i + r16 < rows) load_upto<W>(w[i], a + (int64_t)(16 * i) * g.in + k, k, g.in);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < RT; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i].get(j), xv.get(j), acc[i], 0, 0, 0);
    }
}

// One workgroup: a tile, up to 64 ranks of its groups; the waves split in.
template <typename W>
__global__ void __launch_bounds__(64 * kShrinkWaves) adapt_shrink_kernel(AdaptArgs g) {
    __shared__ float red[kShrinkWaves][kRowTiles][kTile * kTile];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, kg = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * kTile;
    const int r0 = blockIdx.z * 16 * kRowTiles;
    const int steps = (g.in + 15) / 16, per = (steps + kShrinkWaves - 1) / kShrinkWaves;
    const int s0 = wave * per < steps ? wave * per : steps, s1 = s0 + per < steps ? s0 + per : steps;
    for_groups(g, t0, blockIdx.y, [&](int a, uint32_t group) {
        if (a < 0) return;
        const int rows = adapter_rank(g, a) - r0;
        if (rows <= 0) return;
        const int rt = rows >= 16 * kRowTiles ? kRowTiles : (rows + 15) / 16;
        const bool mine = group >> r16 & 1;
        const float* x = g.x + (t0 + r16) * g.xs;
        const W* aw = (const W*)g.a + ((int64_t)a * g.rank + r0 + r16) * g.in;
        v4f acc[kRowTiles];
#pragma unroll
        for (int i = 0; i < kRowTiles; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
        if (rt == 1)
            shrink_steps<W, 1>(g, aw, x, mine, rows, s0, s1, acc);
        else if (rt == 2)
            shrink_steps<W, 2>(g, aw, x, mine, rows, s0, s1, acc);
        else
            shrink_steps<W, 4>(g, aw, x, mine, rows, s0, s1, acc);
        // a lane has ranks 16 i + 4 kg .. + 3 of token r16
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRowTiles; ++i)
            if (i < rt) *reinterpret_cast<v4f*>(&red[wave][i][r16 * 16 + 4 * kg]) = acc[i];
        __syncthreads();
        for (int n = threadIdx.x; n < rt * kTile * kTile; n += blockDim.x) {
            const int i = n >> 8, token = n >> 4 & 15, r = n & 15;
            if (!(group >> token & 1)) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kShrinkWaves; ++w) s += red[w][i][n & 255];
            g.v[(t0 + token) * g.vs + r0 + 16 * i + r] = s;  // past the adapter's rank: 0
        }
    });
}

// One wave: 64 outputs of a tile's groups.
template <typename W>
__global__ void __launch_bounds__(64 * kExpandWaves) adapt_expand_kernel(AdaptArgs g) {
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kTile;
    const int o0 = (blockIdx.x * kExpandWaves + wave) * kExpandCols;
    if (o0 >= g.out_dim) return;
    for_groups(g, t0, blockIdx.z, [&](int a, uint32_t group) {
        const bool mine = group >> r16 & 1;
        const int rank = a < 0 ? 0 : adapter_rank(g, a);
        if (rank == 0 && !g.copy) return;
        constexpr int kTiles = kExpandCols / 16;
        v4f acc[kTiles];
#pragma unroll
        for (int i = 0; i < kTiles; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
        const float* v = g.v + (t0 + r16) * g.vs + 4 * kg;
        const W* bw = (const W*)g.b + ((int64_t)(a < 0 ? 0 : a) * g.out_dim + o0 + r16) * g.rank + 4 * kg;
        for (int r = 0; r < rank; r += 16) {
            v4f vv{0.f, 0.f, 0.f, 0.f};
            if (mine) vv = load4(v + r);
            Four<W> w[kTiles];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const W* p = bw + (int64_t)(16 * i) * g.rank + r;
                w[i].zero();
                if (o0 + 16 * i + r16 < g.out_dim) {
                    if (r + 16 <= rank)
                        w[i].load(p);
                    else
                        load_upto<W>(w[i], p, r + 4 * kg, rank);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < kTiles; ++i)
                    acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i].get(j), vv[j], acc[i], 0, 0, 0);
        }
        // a lane has outputs 16 i + 4 kg .. + 3 of token r16
        if (!mine) return;
        const float scale = a >= 0 && g.scale ? g.scale[a] : 1.0f;
        const float* y = g.y + (t0 + r16) * g.ys + o0 + 4 * kg;
        float* out = g.out + (t0 + r16) * g.os + o0 + 4 * kg;
#pragma unroll
        for (int i = 0; i < kTiles; ++i) {
            const int o = o0 + 16 * i + 4 * kg;
            if (o + 4 <= g.out_dim) {
                v4f s = load4(y + 16 * i);
                if (rank > 0)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[j] = fmaf(scale, acc[i][j], s[j]);
                *reinterpret_cast<v4f_any*>(out + 16 * i) = s;
            } else {
                for (int j = 0; j < 4 && o + j < g.out_dim; ++j) {
                    const float s = y[16 * i + j];
                    out[16 * i + j] = rank > 0 ? fmaf(scale, acc[i][j], s) : s;
                }
            }
        }
    });
}

template <typename W>
hipError_t launch_typed(const AdaptArgs& g, hipStream_t st) {
    const unsigned tiles = (unsigned)((g.T + kTile - 1) / kTile);
    const unsigned ranks = (unsigned)((g.rank + 16 * kRowTiles - 1) / (16 * kRowTiles));
    hipLaunchKernelGGL(adapt_shrink_kernel<W>, dim3(tiles, g.spread, ranks), dim3(64 * kShrinkWaves), 0, st, g);
    const unsigned cols = (unsigned)((g.out_dim + kExpandCols * kExpandWaves - 1) / (kExpandCols * kExpandWaves));
    // grid.y and grid.z hold at most 65535: tiles go over y in pieces
    for (unsigned first = 0; first < tiles; first += 65535) {
        AdaptArgs part = g;
        const int64_t t0 = (int64_t)first * kTile;
        part.x += t0 * g.xs;
        part.y += t0 * g.ys;
        part.out += t0 * g.os;
        part.ids += t0;
        part.v += t0 * g.vs;
        part.T = g.T - t0;
        const unsigned n = tiles - first < 65535 ? tiles - first : 65535;
        hipLaunchKernelGGL(adapt_expand_kernel<W>, dim3(cols, n, g.spread), dim3(64 * kExpandWaves), 0, st, part);
    }
    return hipGetLastError();
}

int32_t padded_rank(int32_t rank) { return (rank + 15) / 16 * 16; }

}  // namespace

size_t adapt_workspace(int64_t T, int32_t rank) { return (size_t)round_up(T * padded_rank(rank) * 4, 256); }

hipError_t launch_adapt(const AdaptLaunch& l, hipStream_t st) {
    AdaptArgs g{};
    g.x = l.x;
    g.y = l.y;
    g.out = l.out;
    g.ids = l.ids;
    g.a = l.a;
    g.b = l.b;
    g.scale = l.scale;
    g.ranks = l.ranks;
    g.v = (float*)l.workspace;
    g.T = l.T;
    g.xs = l.x_stride;
    g.ys = l.y_stride;
    g.os = l.out_stride;
    g.L = l.n_adapter;
    g.rank = l.rank;
    g.in = l.in_dim;
    g.out_dim = l.out_dim;
    g.vs = padded_rank(l.rank);
    g.spread = l.T <= kSpreadTokens ? kTile : 1;
    g.copy = l.out != l.y;
    switch (l.dtype) {
        case kAdapterF32: return launch_typed<float>(g, st);
        case kAdapterF16: return launch_typed<_Float16>(g, st);
        default: return launch_typed<Bf16>(g, st);
    }
}

}  // namespace strata_moe
