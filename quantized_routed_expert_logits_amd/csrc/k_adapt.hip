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
// operand is one value of k; it loads 8 consecutive values of k (16 bytes of a
// 16-bit weight: a wave's load is whole 64-byte pieces of 16 rows) and feeds
// them to 8 products, which only permutes k, for both operands alike.
#include "internal.h"

namespace strata_moe {

namespace {

constexpr int kTile = 16;         // tokens of a tile
constexpr int kShrinkWaves = 8;   // waves that split a workgroup's part of the reduction over in
constexpr int kRowTiles = 4;      // 16-row tiles of A per shrink workgroup: 64 ranks
constexpr int kExpandWaves = 4;
constexpr int kExpandCols = 32;   // outputs of a wave at a time
constexpr int kMaxSplit = 16;     // shrink workgroups that share a reduction
constexpr int kPad = 4;           // floats between the LDS rows of v (spreads the banks)
// Calls of up to this many tokens give every group of a tile workgroups of its
// own (the latency of up to 16 groups one after another counts there); longer
// ones have tiles enough to fill the chip.
constexpr int kSpreadTokens = 256;
constexpr int kFill = 512;        // workgroups that fill the chip

struct AdaptArgs {
    const float* x;
    const float* y;
    float* out;
    const int32_t* ids;
    const void* a;
    const void* b;
    const float* scale;    // or null: 1
    const int32_t* ranks;  // or null: rank
    float* v;              // [split][T][vs]: the parts of A x
    int64_t T, total;      // tokens of the launch, of the call
    int64_t xs, ys, os;
    int32_t L, rank, in, out_dim;
    int32_t vs;            // rank rounded up to 16
    int32_t ls;            // floats of an LDS row of v: rank rounded up to 32, and the pad
    int32_t split;         // parts of the reduction over in
    int32_t spread;        // groups of a tile that run side by side
    int32_t turns;         // expand: turns of kExpandCols outputs per wave
    int32_t copy;          // out is not y: rows without an adapter are copied
};

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));  // at any float

__device__ __forceinline__ v4f load4(const float* p) { return *reinterpret_cast<const v4f_any*>(p); }

// P = 4 or 8 consecutive weights, as loaded and widened.
template <typename W, int P>
struct Run;
template <int P>
struct Run<float, P> {
    v4f r[P / 4];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < P / 4; ++i) r[i] = load4(p + 4 * i);
    }
    __device__ __forceinline__ void set(int j, float w) { r[j / 4][j % 4] = w; }
    __device__ __forceinline__ float get(int j) const { return r[j / 4][j % 4]; }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < P / 4; ++i) r[i] = v4f{0.f, 0.f, 0.f, 0.f};
    }
};
template <int P>
struct Run<_Float16, P> {
    typedef _Float16 V __attribute__((ext_vector_type(P)));
    typedef _Float16 Any __attribute__((ext_vector_type(P), aligned(2)));
    V r;
    __device__ __forceinline__ void load(const _Float16* p) { r = *reinterpret_cast<const Any*>(p); }
    __device__ __forceinline__ void set(int j, _Float16 w) { r[j] = w; }
    __device__ __forceinline__ float get(int j) const { return (float)r[j]; }
    __device__ __forceinline__ void zero() { r = (V)(_Float16)0; }
};
struct Bf16 {
    uint16_t bits;
};
template <int P>
struct Run<Bf16, P> {
    typedef uint16_t V __attribute__((ext_vector_type(P)));
    typedef uint16_t Any __attribute__((ext_vector_type(P), aligned(2)));
    V r;
    __device__ __forceinline__ void load(const Bf16* p) { r = *reinterpret_cast<const Any*>(p); }
    __device__ __forceinline__ void set(int j, Bf16 w) { r[j] = w.bits; }
    __device__ __forceinline__ float get(int j) const { return __builtin_bit_cast(float, (uint32_t)r[j] << 16); }
    __device__ __forceinline__ void zero() { r = (V)(uint16_t)0; }
};

// p[0 .. P) where k + j < n, zeros elsewhere (nothing is read past n).
template <typename W, int P>
__device__ __forceinline__ void load_upto(Run<W, P>& f, const W* p, int k, int n) {
    f.zero();
#pragma unroll
    for (int j = 0; j < P; ++j)
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

// Products of steps [s0, s1) of 32 values of k: RT tiles of 16 A rows against
// the tile's tokens.  a[i], x: the lane's rows (rows and tokens outside the
// group repeat one of it: the loads need no branch, and what comes of them is
// not stored).
template <typename W, int RT>
__device__ __forceinline__ void shrink_steps(const AdaptArgs& g, const W* const (&a)[kRowTiles], const float* x, int s0,
                                             int s1, v4f (&acc)[kRowTiles]) {
    constexpr int kDepth = RT == 1 ? 4 : RT == 2 ? 3 : 2;  // steps in flight
    const int k0 = 8 * ((threadIdx.x & 63) >> 4);
    const int whole = g.in / 32 < s1 ? g.in / 32 : s1;
    Run<float, 8> xr[kDepth];
    Run<W, 8> wr[kDepth][RT];
    auto load = [&](int s, int u) {
        const int k = 32 * (s < whole ? s : whole - 1) + k0;  // past the run: its last step again, never used
        xr[u].load(x + k);
#pragma unroll
        for (int i = 0; i < RT; ++i) wr[u][i].load(a[i] + k);
    };
    auto products = [&](int u) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int i = 0; i < RT; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(wr[u][i].get(j), xr[u].get(j), acc[i], 0, 0, 0);
    };
    int s = s0;
    if (s < whole) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            load(s + u, u);
            __builtin_amdgcn_sched_barrier(0);
        }
        for (; s + kDepth <= whole; s += kDepth)
#pragma unroll
            for (int u = 0; u < kDepth; ++u) {
                products(u);
                __builtin_amdgcn_sched_barrier(0);
                load(s + kDepth + u, u);
                __builtin_amdgcn_sched_barrier(0);
            }
        int left = whole - s;
#pragma unroll
        for (int u = 0; u < kDepth - 1; ++u)
            if (u < left) products(u);
        s = whole;
    }
    if (s < s1) {  // the step that ends inside the row
        const int k = 32 * s + k0;
        load_upto<float, 8>(xr[0], x + k, k, g.in);
#pragma unroll
        for (int i = 0; i < RT; ++i) load_upto<W, 8>(wr[0][i], a[i] + k, k, g.in);
        products(0);
    }
}

// One workgroup: a tile, up to 64 ranks of its groups, one part of the
// reduction over in, which its waves split again.
template <typename W>
__global__ void __launch_bounds__(64 * kShrinkWaves) adapt_shrink_kernel(AdaptArgs g) {
    __shared__ float red[kShrinkWaves][kRowTiles][kTile * kTile];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, kg = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.x * kTile;
    const int part = blockIdx.z % g.split, r0 = blockIdx.z / g.split * 16 * kRowTiles;
    const int steps = (g.in + 31) / 32, runs = g.split * kShrinkWaves, per = (steps + runs - 1) / runs;
    const int first = (part * kShrinkWaves + wave) * per;
    const int s0 = first < steps ? first : steps, s1 = s0 + per < steps ? s0 + per : steps;
    for_groups(g, t0, blockIdx.y, [&](int a, uint32_t group) {
        if (a < 0) return;
        const int rows = adapter_rank(g, a) - r0;
        if (rows <= 0) return;
        const int rt = rows >= 16 * kRowTiles ? kRowTiles : (rows + 15) / 16;
        const float* x = g.x + (t0 + (group >> r16 & 1 ? r16 : __builtin_ctz(group))) * g.xs;
        const W* aw[kRowTiles];
        v4f acc[kRowTiles];
#pragma unroll
        for (int i = 0; i < kRowTiles; ++i) {
            const int row = 16 * i + r16 < rows ? 16 * i + r16 : rows - 1;
            aw[i] = (const W*)g.a + ((int64_t)a * g.rank + r0 + row) * g.in;
            acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        if (rt == 1)
            shrink_steps<W, 1>(g, aw, x, s0, s1, acc);
        else if (rt == 2)
            shrink_steps<W, 2>(g, aw, x, s0, s1, acc);
        else
            shrink_steps<W, 4>(g, aw, x, s0, s1, acc);
        // a lane has ranks 16 i + 4 kg .. + 3 of token r16
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRowTiles; ++i)
            if (i < rt) *reinterpret_cast<v4f*>(&red[wave][i][r16 * 16 + 4 * kg]) = acc[i];
        __syncthreads();
        for (int n = threadIdx.x; n < rt * kTile * kTile; n += blockDim.x) {
            const int i = n >> 8, token = n >> 4 & 15, r = n & 15;
            if (!(group >> token & 1) || 16 * i + r >= rows) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kShrinkWaves; ++w) s += red[w][i][n & 255];
            g.v[((int64_t)part * g.T + t0 + token) * g.vs + r0 + 16 * i + r] = s;
        }
    });
}

// One workgroup: a tile's groups, `turns` runs of 64 outputs per wave.  P
// consecutive ranks per lane: 4 for ranks up to 16, else 8.
template <typename W, int P>
__global__ void __launch_bounds__(64 * kExpandWaves) adapt_expand_kernel(AdaptArgs g) {
    extern __shared__ float v[];  // [16][ls]
    constexpr int kTiles = kExpandCols / 16;
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kTile;
    const int64_t total = g.total;
    for_groups(g, t0, blockIdx.z, [&](int a, uint32_t group) {
        const int rank = a < 0 ? 0 : adapter_rank(g, a);
        if (rank == 0 && !g.copy) return;
        const bool mine = group >> r16 & 1;
        const float scale = a >= 0 && g.scale ? g.scale[a] : 1.0f;
        // the group's v, its parts added in order, zeros past the rank (the
        // other tokens' rows hold anything: their columns are not stored)
        __syncthreads();
        const int ranks = (rank + 4 * P - 1) / (4 * P) * (4 * P);
        for (int n = threadIdx.x; n < kTile * ranks; n += blockDim.x) {
            const int token = n / ranks, r = n % ranks;
            if (!(group >> token & 1)) continue;
            float s = 0.f;
            if (r < rank)
                for (int p = 0; p < g.split; ++p) s += g.v[((int64_t)p * total + t0 + token) * g.vs + r];
            v[token * g.ls + r] = s;
        }
        __syncthreads();
        const float* vr = v + r16 * g.ls + P * kg;
        for (int turn = 0; turn < g.turns; ++turn) {
            const int o0 = ((blockIdx.x * g.turns + turn) * kExpandWaves + wave) * kExpandCols;
            if (o0 >= g.out_dim) break;
            const float* y = g.y + (t0 + r16) * g.ys + o0 + 4 * kg;
            v4f acc[kTiles], s[kTiles];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                acc[i] = s[i] = v4f{0.f, 0.f, 0.f, 0.f};
                if (mine && o0 + 16 * i + 4 * kg + 4 <= g.out_dim) s[i] = load4(y + 16 * i);
            }
            const W* bw[kTiles];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const int o = o0 + 16 * i + r16 < g.out_dim ? o0 + 16 * i + r16 : g.out_dim - 1;
                bw[i] = (const W*)g.b + ((int64_t)(a < 0 ? 0 : a) * g.out_dim + o) * g.rank + P * kg;
            }
            for (int r = 0; r < rank; r += 4 * P) {
                Run<W, P> w[kTiles];
#pragma unroll
                for (int i = 0; i < kTiles; ++i)
                    if (r + 4 * P <= rank)
                        w[i].load(bw[i] + r);
                    else
                        load_upto<W, P>(w[i], bw[i] + r, r + P * kg, rank);
                Run<float, P> vv;
                vv.load(vr + r);
#pragma unroll
                for (int j = 0; j < P; ++j)
#pragma unroll
                    for (int i = 0; i < kTiles; ++i)
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i].get(j), vv.get(j), acc[i], 0, 0, 0);
            }
            // a lane has outputs 16 i + 4 kg .. + 3 of token r16
            if (mine) {
                float* out = g.out + (t0 + r16) * g.os + o0 + 4 * kg;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const int o = o0 + 16 * i + 4 * kg;
                    if (o + 4 <= g.out_dim) {
                        if (rank > 0)
#pragma unroll
                            for (int j = 0; j < 4; ++j) s[i][j] = fmaf(scale, acc[i][j], s[i][j]);
                        *reinterpret_cast<v4f_any*>(out + 16 * i) = s[i];
                    } else {
                        for (int j = 0; j < 4 && o + j < g.out_dim; ++j) {
                            const float yv = y[16 * i + j];
                            out[16 * i + j] = rank > 0 ? fmaf(scale, acc[i][j], yv) : yv;
                        }
                    }
                }
            }
        }
    });
}

template <typename W>
hipError_t launch_typed(AdaptArgs g, hipStream_t st) {
    const unsigned tiles = (unsigned)((g.T + kTile - 1) / kTile);
    const unsigned ranks = (unsigned)((g.rank + 16 * kRowTiles - 1) / (16 * kRowTiles));
    hipLaunchKernelGGL(adapt_shrink_kernel<W>, dim3(tiles, g.spread, ranks * g.split), dim3(64 * kShrinkWaves), 0, st, g);
    // enough workgroups to fill the chip several times, then longer ones
    const unsigned cols = (unsigned)((g.out_dim + kExpandCols * kExpandWaves - 1) / (kExpandCols * kExpandWaves));
    unsigned gx = cols;
    while (gx > 1 && (int64_t)tiles * (gx / 2) >= 4 * kFill) gx /= 2;
    g.turns = (cols + gx - 1) / gx;
    const size_t lds = (size_t)kTile * g.ls * sizeof(float);
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
        if (g.rank <= 16)
            hipLaunchKernelGGL((adapt_expand_kernel<W, 4>), dim3(gx, n, g.spread), dim3(64 * kExpandWaves), lds, st, part);
        else
            hipLaunchKernelGGL((adapt_expand_kernel<W, 8>), dim3(gx, n, g.spread), dim3(64 * kExpandWaves), lds, st, part);
    }
    return hipGetLastError();
}

int32_t padded_rank(int32_t rank) { return (rank + 15) / 16 * 16; }

// The shrink's workgroups share a reduction until they fill the chip, down to
// one step of 32 values per wave.
int32_t shrink_split(int64_t T, int32_t rank, int32_t in) {
    const int64_t groups = T <= kSpreadTokens ? T : (T + kTile - 1) / kTile;
    const int64_t wgs = groups * ((rank + 16 * kRowTiles - 1) / (16 * kRowTiles));
    const int64_t most = (in + 32 * kShrinkWaves - 1) / (32 * kShrinkWaves);
    int64_t s = kFill / (wgs > 0 ? wgs : 1);
    if (s > most) s = most;
    if (s > kMaxSplit) s = kMaxSplit;
    return s < 1 ? 1 : (int32_t)s;
}

}  // namespace

size_t adapt_workspace(int64_t T, int32_t rank, int32_t in) {
    return (size_t)round_up(shrink_split(T, rank, in) * T * padded_rank(rank) * 4, 256);
}

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
    g.T = g.total = l.T;
    g.xs = l.x_stride;
    g.ys = l.y_stride;
    g.os = l.out_stride;
    g.L = l.n_adapter;
    g.rank = l.rank;
    g.in = l.in_dim;
    g.out_dim = l.out_dim;
    g.vs = padded_rank(l.rank);
    g.ls = (l.rank + 31) / 32 * 32 + kPad;
    g.split = shrink_split(l.T, l.rank, l.in_dim);
    g.spread = l.T <= kSpreadTokens ? kTile : 1;
    g.copy = l.out != l.y;
    switch (l.dtype) {
        case kAdapterF32: return launch_typed<float>(g, st);
        case kAdapterF16: return launch_typed<_Float16>(g, st);
        default: return launch_typed<Bf16>(g, st);
    }
}

}  // namespace strata_moe
