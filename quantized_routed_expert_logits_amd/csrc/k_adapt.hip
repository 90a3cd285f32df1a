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
// Products.  The activations and sums are fp32.  fp32 and fp16 weights run on
// the fp32 matrix unit (16x16x4; an fp16 weight widens exactly).  bf16 weights
// run on the bf16 unit (16x16x32): a fp32 activation is the sum of three bf16
// values, exactly (its 24 bits are cut into 8 + 8 + 8 from the top), so three
// products give what one fp32 product gives, in 3/16 of its time.  The parts
// below the first have accumulators of their own: their additions round at
// 2^-8 of the first's.  (Subnormal parts may count as zero: the lowest part of
// values below 2^-110, and beside an infinite factor any value below 2^-126,
// which gives NaN there.)  fp16 weights do not split as cheaply: each is two
// bf16 values, and cutting 64 rows of them costs more vector instructions than
// the fp32 products they replace.
//
// A lane's operand is row lane % 16 and a run of consecutive values of k (8,
// or 4 in the expand of ranks up to 16).  The fp32 unit takes the run one
// value a product, which only permutes k, for both operands alike.
//
// Loads and stores go row by row, 4 or 16 neighbouring lanes to a row, and
// cross to the products' layout (neighbouring lanes in different rows)
// through LDS that belongs to the wave alone: in the products' layout every
// lane's 16 bytes are an access of their own.  (8192 tokens, rank 64, bf16
// weights on the fp32 unit: crossing took the shrink from 50 to 46 us; with
// the bf16 unit and the tiles dealt to the XCDs it was 37.)
//
// What bounds them.  Many tokens: memory, x once for the shrink, y and out
// once for the expand.  8192 tokens of 2560, 16 adapters of rank 64, bf16: the
// shrink 35 us (90 MB, 2.6 TB/s), the expand 51 to 59 us (175 MB, 3.0 to 3.4
// TB/s), against 5.1 TB/s of a large copy.  Few tokens: latency, a chain of
// ids, ranks, weights, the sums' way through the workspace, and the same
// again: 3.8 + 5.0 us for one token at rank 16, 8.6 + 9.7 us for 32 tokens
// with an adapter each (fp16, ranks 1 to 64), of which the products, 15 of
// their 16 columns unused, take 1.6 and 1.2.
#include <algorithm>
#include <type_traits>

#include "few_tokens.h"

namespace strata_moe {

namespace {

constexpr int kTile = 16;         // tokens of a tile
constexpr int kShrinkWaves = 8;   // waves that split a workgroup's part of the reduction over in
constexpr int kRowTiles = 4;      // 16-row tiles of A per shrink workgroup: 64 ranks
constexpr int kExpandWaves = 4;
constexpr int kExpandCols = 64;   // outputs of a wave at a time
constexpr int kMaxSplit = 16;     // shrink workgroups that share a reduction
constexpr int kPad = 4;           // floats between the LDS rows of v (spreads the banks)
// Calls of up to this many tokens give every group of a tile workgroups of its
// own (the latency of up to 16 groups one after another counts there); longer
// ones have tiles enough to fill the chip, if prompts give a tile a group or
// two.  One after another against side by side, in us, 2560 -> 2560, bf16,
// prompts of 64 requests: rank 64 256 tokens 62, 32, 1000 58, 54, 2048 65, 76;
// rank 16 256 tokens 33, 19, 512 31, 26, 1000 27, 32.  Rows of mixed adapters,
// 16 groups a tile, would gain beyond it: rank 64 256 rows 128, 50, 512 139,
// 79, 1000 207, 142, 2048 285, 264, 4096 490, 501.
constexpr int kSpreadTokens = 256;
constexpr int kFill = 512;        // workgroups that fill the chip
// The outputs are stored past the caches, and y is read past them from this
// many bytes on: x then stays in the Infinity Cache (8192 tokens of 2560: 109
// us at rank 64 and 72 at rank 16 without either, 105 and 67 with the stores,
// 90 and 59 with both; 2048 tokens at rank 16: 28.0, 27.4, 29.5).
constexpr int64_t kStreamBytes = (int64_t)48 << 20;
// From this many tiles on every XCD takes a run of neighbouring tiles: prompts
// share adapters with their neighbours, and an L2 then holds two or three of
// them instead of all.  Round robin against runs, in us, 16 adapters, rank 64,
// bf16: 512 tokens 39.1, 38.1, 1024 43.5, 42.2, 4096 65.4, 61.1, 8192 84.8,
// 90.1; fp32 65.4, 64.2 at 2048, 130, 138 at 8192; rank 16 26.4, 26.0 at 2048,
// 58.7, 59.5 at 8192.  (Before the outputs went past the caches round robin
// took longer at 8192 tokens, too.)
constexpr int kDealTiles = 64;

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
    int64_t T, xs, ys, os;
    int32_t L, rank, in, out_dim;
    int32_t vs;            // rank rounded up to 16
    int32_t ls;            // floats of an LDS row of v: rank rounded up to 32, and the pad
    int32_t split;         // parts of the reduction over in
    int32_t spread;        // groups of a tile that run side by side
    int32_t turns;         // expand: turns of kExpandCols outputs per wave
    int32_t tiles;
    int32_t deal;          // tiles are dealt to the XCDs in runs of this many, or 0
    int32_t copy;          // out is not y: rows without an adapter are copied
};

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
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
    __device__ __forceinline__ void keep(int n) {  // the first n, zeros behind them
#pragma unroll
        for (int j = 0; j < P; ++j) r[j] = j < n ? r[j] : (_Float16)0;
    }
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
    __device__ __forceinline__ void keep(int n) {
#pragma unroll
        for (int j = 0; j < P; ++j) r[j] = j < n ? r[j] : (uint16_t)0;
    }
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

// The workgroup's tile, or -1.  Workgroups go to the 8 XCDs in turn.
__device__ __forceinline__ int tile_of(const AdaptArgs& g, int id) {
    const int tile = g.deal > 0 ? (id & 7) * g.deal + (id >> 3) : id;
    return tile < g.tiles && (g.deal == 0 || (id >> 3) < g.deal) ? tile : -1;
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
        if (g.spread == 1 || n == share) f(a, group);
    }
}

// A panel is 16 rows of 4 runs.  Loaded, lane l has run l % 4 of row l / 4;
// crossed, lane l has run l / 16 of row l % 16.  buf: 64 runs of the wave's LDS.
template <typename W, int P>
__device__ __forceinline__ void cross_out(const Run<W, P>& f, char* buf) {
    *reinterpret_cast<Run<W, P>*>(buf + (threadIdx.x & 63) * sizeof(f)) = f;
}
template <typename W, int P>
__device__ __forceinline__ void cross_in(Run<W, P>& f, const char* buf) {
    const int lane = threadIdx.x & 63;
    f = *reinterpret_cast<const Run<W, P>*>(buf + ((lane & 15) * 4 + (lane >> 4)) * sizeof(f));
}

// acc += w x over a run of k, for N tiles of weights (the product's rows) and
// 16 activations (its columns).  lo: the bf16 parts below the first.
template <typename W, int P, int N>
struct Products {
    Run<float, P> x;
    __device__ __forceinline__ void set(const Run<float, P>& v) { x = v; }
    template <int M>
    __device__ __forceinline__ void add(const Run<W, P> (&w)[N], v4f (&acc)[M], v4f (&)[M]) const {
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[i].get(j), x.get(j), acc[i], 0, 0, 0);
    }
};

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4i16 __attribute__((ext_vector_type(4)));

template <int P, int N>
struct Products<Bf16, P, N> {
    uint32_t x[3][P / 2];  // the three parts, two values a dword
    __device__ __forceinline__ void set(const Run<float, P>& v) {
        constexpr uint32_t kTop = 0xffff0000u, kTops = 0x07060302u;  // both upper halves
#pragma unroll
        for (int j = 0; j < P; j += 2) {
            float a = v.get(j), b = v.get(j + 1);
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const uint32_t ab = __builtin_bit_cast(uint32_t, a), bb = __builtin_bit_cast(uint32_t, b);
                x[p][j / 2] = __builtin_amdgcn_perm(bb, ab, kTops);
                if (p < 2) {
                    a -= __builtin_bit_cast(float, ab & kTop);
                    b -= __builtin_bit_cast(float, bb & kTop);
                }
            }
        }
    }
    template <int M>
    __device__ __forceinline__ void add(const Run<Bf16, P> (&w)[N], v4f (&acc)[M], v4f (&lo)[M]) const {
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v4f& s = p == 0 ? acc[i] : lo[i];
                if constexpr (P == 8)
                    s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(v8b, w[i].r),
                        __builtin_bit_cast(v8b, v4u{x[p][0], x[p][1], x[p][2], x[p][3]}), s, 0, 0, 0);
                else
                    s = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
                        __builtin_bit_cast(v4i16, w[i].r), __builtin_bit_cast(v4i16, v2u{x[p][0], x[p][1]}), s, 0, 0, 0);
            }
    }
};

// The sums of a lane: the first parts' and those below them.  An infinite
// value cut into parts leaves NaN below the first, and so does an infinite
// weight times a value with nothing below its first part; the first sum is then
// infinite (or NaN) already, and stays so beside any finite one.
template <typename W>
__device__ __forceinline__ v4f whole_sum(v4f acc, v4f lo) {
    if constexpr (std::is_same<W, Bf16>::value) {
        // in a scalar register: as a constant the compiler keeps it in vector
        // registers, and others spill (8192 tokens, rank 64: 92.3 us, 90.2)
        float most = __FLT_MAX__;
        asm("" : "+s"(most));
#pragma unroll
        for (int j = 0; j < 4; ++j) lo[j] = __builtin_amdgcn_fmed3f(lo[j], -most, most);
    }
    return acc + lo;
}

// Products of steps [s0, s1) of 32 values of k: RT tiles of 16 A rows against
// the tile's tokens.  al[i], xl: the rows that the lane loads, a[i], x: those
// of its operands (rows and tokens outside the group repeat one of it: the
// loads need no branch, and what comes of them is not stored).
template <typename W, int RT>
__device__ __forceinline__ void shrink_steps(const AdaptArgs& g, const W* const (&al)[kRowTiles], const float* xl,
                                             const W* const (&a)[kRowTiles], const float* x, int s0, int s1,
                                             v4f (&acc)[kRowTiles], v4f (&lo)[kRowTiles], char* buf) {
    constexpr int kDepth = RT == 1 ? 4 : RT == 2 ? 3 : 2;  // steps in flight
    constexpr int kPanel = 64 * 8 * (int)sizeof(W);
    const int lane = threadIdx.x & 63;
    const int whole = g.in / 32 < s1 ? g.in / 32 : s1;
    Run<float, 4> xr[kDepth][2];  // values 0..15 and 16..31 of the step
    Run<W, 8> wr[kDepth][RT];
    auto load = [&](int s, int u) {
        const int k = 32 * (s < whole ? s : whole - 1);  // past the run: its last step again, never used
#pragma unroll
        for (int h = 0; h < 2; ++h) xr[u][h].load(xl + k + 16 * h + 4 * (lane & 3));
#pragma unroll
        for (int i = 0; i < RT; ++i) wr[u][i].load(al[i] + k + 8 * (lane & 3));
    };
    auto products = [&](const Run<float, 8>& xv, const Run<W, 8> (&w)[RT]) {
        Products<W, 8, RT> m;
        m.set(xv);
        m.add(w, acc, lo);
    };
    auto step = [&](int u) {
        // x: run kg of 8 is chunks 2 kg, 2 kg + 1 of 4, in panel kg / 2
        cross_out(xr[u][0], buf);
        cross_out(xr[u][1], buf + 1024);
#pragma unroll
        for (int i = 0; i < RT; ++i) cross_out(wr[u][i], buf + 2048 + kPanel * i);
        Run<float, 8> xv = *reinterpret_cast<const Run<float, 8>*>(buf + (lane >> 5) * 1024 + (lane & 15) * 64 +
                                                                   (lane >> 4 & 1) * 32);
        Run<W, 8> w[RT];
#pragma unroll
        for (int i = 0; i < RT; ++i) cross_in(w[i], buf + 2048 + kPanel * i);
        products(xv, w);
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
                step(u);
                __builtin_amdgcn_sched_barrier(0);
                load(s + kDepth + u, u);
                __builtin_amdgcn_sched_barrier(0);
            }
        const int left = whole - s;
#pragma unroll
        for (int u = 0; u < kDepth - 1; ++u)
            if (u < left) step(u);
        s = whole;
    }
    if (s < s1) {  // the step that ends inside the row, straight to the operands
        const int k = 32 * s + 8 * (lane >> 4);
        Run<float, 8> xv;
        Run<W, 8> w[RT];
        load_upto<float, 8>(xv, x + k, k, g.in);
#pragma unroll
        for (int i = 0; i < RT; ++i) load_upto<W, 8>(w[i], a[i] + k, k, g.in);
        products(xv, w);
    }
}

// One workgroup: a tile, up to 64 ranks of its groups, one part of the
// reduction over in, which its waves split again: a wave's run is then a few
// steps of 128 bytes per row, and 8 waves hide each other's loads.  (128
// registers: the bf16 form spills 4, the fp32 form 11.)
template <typename W>
__global__ void __launch_bounds__(64 * kShrinkWaves, 4) adapt_shrink_kernel(AdaptArgs g) {
    // the waves' panels, then their sums
    constexpr int kWaveBytes = 2048 + kRowTiles * 64 * 8 * (int)sizeof(W);
    constexpr int kSumBytes = kRowTiles * kTile * kTile * (int)sizeof(float);
    __shared__ __align__(16) char lds[kShrinkWaves * (kWaveBytes > kSumBytes ? kWaveBytes : kSumBytes)];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, kg = lane >> 4;
    const int tile = tile_of(g, blockIdx.x);
    if (tile < 0) return;
    const int64_t t0 = (int64_t)tile * kTile;
    const int part = blockIdx.z % g.split, r0 = blockIdx.z / g.split * 16 * kRowTiles;
    const int steps = (g.in + 31) / 32, runs = g.split * kShrinkWaves, per = (steps + runs - 1) / runs;
    const int first = (part * kShrinkWaves + wave) * per;
    const int s0 = first < steps ? first : steps, s1 = s0 + per < steps ? s0 + per : steps;
    for_groups(g, t0, blockIdx.y, [&](int a, uint32_t group) {
        if (a < 0) return;
        const int rows = adapter_rank(g, a) - r0;
        if (rows <= 0) return;
        const int rt = rows >= 16 * kRowTiles ? kRowTiles : (rows + 15) / 16;
        const int one = __builtin_ctz(group);
        const float* x = g.x + (t0 + (group >> r16 & 1 ? r16 : one)) * g.xs;
        const float* xl = g.x + (t0 + (group >> (lane >> 2) & 1 ? lane >> 2 : one)) * g.xs;
        const W* aw[kRowTiles];
        const W* al[kRowTiles];
        v4f acc[kRowTiles], lo[kRowTiles];
        const W* a0 = (const W*)g.a + ((int64_t)a * g.rank + r0) * g.in;
#pragma unroll
        for (int i = 0; i < kRowTiles; ++i) {
            const int row = 16 * i + r16, rowl = 16 * i + (lane >> 2);
            aw[i] = a0 + (int64_t)(row < rows ? row : rows - 1) * g.in;
            al[i] = a0 + (int64_t)(rowl < rows ? rowl : rows - 1) * g.in;
            acc[i] = lo[i] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        __syncthreads();  // the last group's sums are read
        char* buf = lds + wave * kWaveBytes;
        if (rt == 1)
            shrink_steps<W, 1>(g, al, xl, aw, x, s0, s1, acc, lo, buf);
        else if (rt == 2)
            shrink_steps<W, 2>(g, al, xl, aw, x, s0, s1, acc, lo, buf);
        else
            shrink_steps<W, 4>(g, al, xl, aw, x, s0, s1, acc, lo, buf);
        // a lane has ranks 16 i + 4 kg .. + 3 of token r16
        float* red = (float*)lds;  // [wave][row tile][token][16]
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRowTiles; ++i)
            if (i < rt)
                *reinterpret_cast<v4f*>(&red[((wave * kRowTiles + i) * 16 + r16) * 16 + 4 * kg]) =
                    whole_sum<W>(acc[i], lo[i]);
        __syncthreads();
        for (int n = threadIdx.x; n < rt * kTile * kTile; n += blockDim.x) {
            const int i = n >> 8, token = n >> 4 & 15, r = n & 15;
            if (!(group >> token & 1) || 16 * i + r >= rows) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kShrinkWaves; ++w) s += red[(w * kRowTiles + i) * 256 + (n & 255)];
            g.v[((int64_t)part * g.T + t0 + token) * g.vs + r0 + 16 * i + r] = s;
        }
    });
}

// One workgroup: a tile's groups, `turns` runs of 64 outputs per wave (256
// bytes of each of 16 rows of y and out at a time).  P
// consecutive ranks per lane: 4 for ranks up to 16, else 8.  kStream: y is
// large, and is read past the caches.  (168 registers: with P = 8 the bf16 and
// fp32 forms spill 6.)
template <typename W, int P, bool kStream>
__global__ void __launch_bounds__(64 * kExpandWaves, 3) adapt_expand_kernel(AdaptArgs g) {
    constexpr int kTiles = kExpandCols / 16;
    constexpr int kRow = kExpandCols + kPad;  // floats of an output row in LDS
    constexpr int kPanel = 64 * P * (int)sizeof(W);
    constexpr int kWaveBytes = kTiles * kPanel > 16 * kRow * 4 ? kTiles * kPanel : 16 * kRow * 4;
    __shared__ __align__(16) char lds[kExpandWaves][kWaveBytes];  // a wave's panels of B, or its outputs
    extern __shared__ float v[];                                  // [16][ls]
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tile = tile_of(g, blockIdx.x);
    if (tile < 0) return;
    const int64_t t0 = (int64_t)tile * kTile;
    const int first = (blockIdx.y * g.turns * kExpandWaves + wave) * kExpandCols;  // the turns are 4 waves apart
    char* buf = lds[wave];
    float* rows = (float*)lds[wave];
    for_groups(g, t0, blockIdx.z, [&](int a, uint32_t group) {
        const int rank = a < 0 ? 0 : adapter_rank(g, a);
        if (rank == 0 && !g.copy) return;
        const int whole = rank / (4 * P) * (4 * P);
        const W* b = (const W*)g.b + (int64_t)(a < 0 ? 0 : a) * g.out_dim * g.rank;
        // the panels of outputs o0 .. and ranks r .. (of a whole step)
        Run<W, P> w[kTiles];
        auto load = [&](int o0, int r) {
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const int o = o0 + 16 * i + (lane >> 2);
                w[i].load(b + (int64_t)(o < g.out_dim ? o : g.out_dim - 1) * g.rank + r + P * (lane & 3));
            }
        };
        if (whole > 0) load(first, 0);
        const float scale = a >= 0 && g.scale ? g.scale[a] : 1.0f;
        // the group's v, its parts added in order, zeros past the rank (the
        // other tokens' rows hold anything: their columns are not stored)
        __syncthreads();
        const int ranks = (rank + 4 * P - 1) / (4 * P) * (4 * P);
        for (int n = threadIdx.x; n < kTile * ranks; n += blockDim.x) {
            const int token = n / ranks, r = n % ranks;
            if (!(group >> token & 1)) continue;
            float s = 0.f;
            if (r < rank) {
                const float* p = g.v + (t0 + token) * g.vs + r;
#pragma unroll 4
                for (int i = 0; i < g.split; ++i) s += p[(int64_t)i * g.T * g.vs];
            }
            v[token * g.ls + r] = s;
        }
        __syncthreads();
        const float* vr = v + r16 * g.ls + P * kg;
        for (int turn = 0; turn < g.turns; ++turn) {
            const int o0 = first + turn * kExpandWaves * kExpandCols, next = o0 + kExpandWaves * kExpandCols;
            if (o0 >= g.out_dim) break;
            const int cols = g.out_dim - o0;
            // a lane loads, adds and stores columns 4 r16 .. + 3 of rows kg + 4 i
            v4f s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((group >> (kg + 4 * i) & 1) && 4 * r16 + 4 <= cols) {
                    const v4f_any* y = reinterpret_cast<const v4f_any*>(g.y + (t0 + kg + 4 * i) * g.ys + o0 + 4 * r16);
                    s[i] = kStream ? __builtin_nontemporal_load(y) : *y;
                }
            v4f acc[kTiles], lo[kTiles];
#pragma unroll
            for (int i = 0; i < kTiles; ++i) acc[i] = lo[i] = v4f{0.f, 0.f, 0.f, 0.f};
            Products<W, P, kTiles> m;
            Run<float, P> vv;
            for (int r = 0; r < whole; r += 4 * P) {
                Run<W, P> u[kTiles];
#pragma unroll
                for (int i = 0; i < kTiles; ++i) cross_out(w[i], buf + kPanel * i);
                // the next step's panels: these ranks', or the next turn's first
                if (r + 4 * P < whole)
                    load(o0, r + 4 * P);
                else
                    load(next, 0);
#pragma unroll
                for (int i = 0; i < kTiles; ++i) cross_in(u[i], buf + kPanel * i);
                vv.load(vr + r);
                m.set(vv);
                m.add(u, acc, lo);
            }
            if (whole < rank) {  // the step that ends inside the rank, straight to the operands
                Run<W, P> u[kTiles];
                const W* at[kTiles];
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    const int o = o0 + 16 * i + r16;
                    at[i] = b + (int64_t)(o < g.out_dim ? o : g.out_dim - 1) * g.rank + whole + P * kg;
                }
                // inside B's rows all the same: whole runs, their end zeroed
                // (32 tokens, ranks 1..64 of 64, fp16: 9.4 us against 11.9;
                // fp32 runs spill more for it, 146 against 137 at 8192 tokens)
                const bool inside = sizeof(W) == 2 && whole + 4 * P <= g.rank;
                if constexpr (sizeof(W) == 2)
                    if (inside) {
#pragma unroll
                        for (int i = 0; i < kTiles; ++i) u[i].load(at[i]);
#pragma unroll
                        for (int i = 0; i < kTiles; ++i) u[i].keep(rank - whole - P * kg);
                    }
                if (!inside) {
#pragma unroll
                    for (int i = 0; i < kTiles; ++i) load_upto<W, P>(u[i], at[i], whole + P * kg, rank);
                }
                vv.load(vr + whole);
                m.set(vv);
                m.add(u, acc, lo);
            }
            // a lane has outputs 16 i + 4 kg .. + 3 of token r16: cross to rows
            if (rank > 0) {
#pragma unroll
                for (int i = 0; i < kTiles; ++i)
                    *reinterpret_cast<v4f*>(&rows[r16 * kRow + 16 * i + 4 * kg]) = whole_sum<W>(acc[i], lo[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int token = kg + 4 * i;
                if (!(group >> token & 1)) continue;
                const v4f d = *reinterpret_cast<const v4f*>(&rows[token * kRow + 4 * r16]);
                const float* y = g.y + (t0 + token) * g.ys + o0 + 4 * r16;
                float* out = g.out + (t0 + token) * g.os + o0 + 4 * r16;
                if (4 * r16 + 4 <= cols) {
                    if (rank > 0)
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[i][j] = fmaf(scale, d[j], s[i][j]);
                    __builtin_nontemporal_store(s[i], reinterpret_cast<v4f_any*>(out));
                } else {
                    for (int j = 0; j < 4 && 4 * r16 + j < cols; ++j) out[j] = rank > 0 ? fmaf(scale, d[j], y[j]) : y[j];
                }
            }
        }
    });
}

template <typename W>
hipError_t launch_typed(AdaptArgs g, hipStream_t st) {
    g.tiles = (int32_t)((g.T + kTile - 1) / kTile);
    g.deal = g.tiles >= kDealTiles ? (g.tiles + 7) / 8 : 0;
    const unsigned gt = g.deal ? 8 * g.deal : g.tiles;
    const unsigned ranks = (unsigned)((g.rank + 16 * kRowTiles - 1) / (16 * kRowTiles));
    hipLaunchKernelGGL(adapt_shrink_kernel<W>, dim3(gt, g.spread, ranks * g.split), dim3(64 * kShrinkWaves), 0, st, g);
    // enough workgroups to fill the chip several times, then longer ones
    const unsigned cols = (unsigned)((g.out_dim + kExpandCols * kExpandWaves - 1) / (kExpandCols * kExpandWaves));
    unsigned gc = cols;
    while (gc > 1 && (int64_t)g.tiles * (gc / 2) >= 4 * kFill) gc /= 2;
    g.turns = (cols + gc - 1) / gc;
    const size_t lds = (size_t)kTile * g.ls * sizeof(float);
    const dim3 grid(gt, gc, g.spread);
    void (*expand)(AdaptArgs);
    if (g.T * g.out_dim * 4 >= kStreamBytes)
        expand = g.rank <= 16 ? adapt_expand_kernel<W, 4, true> : adapt_expand_kernel<W, 8, true>;
    else
        expand = g.rank <= 16 ? adapt_expand_kernel<W, 4, false> : adapt_expand_kernel<W, 8, false>;
    hipLaunchKernelGGL(expand, grid, dim3(64 * kExpandWaves), lds, st, g);
    return hipGetLastError();
}

int32_t padded_rank(int32_t rank) { return (rank + 15) / 16 * 16; }

// The shrink's workgroups share a reduction until they fill the chip, down to
// two steps of 32 values per wave.
int32_t shrink_split(int64_t T, int32_t rank, int32_t in) {
    const int64_t groups = T <= kSpreadTokens ? T : (T + kTile - 1) / kTile;
    const int64_t wgs = groups * ((rank + 16 * kRowTiles - 1) / (16 * kRowTiles));
    const int64_t most = (in + 64 * kShrinkWaves - 1) / (64 * kShrinkWaves);
    int64_t s = kFill / (wgs > 0 ? wgs : 1);
    if (s > most) s = most;
    if (s > kMaxSplit) s = kMaxSplit;
    return s < 1 ? 1 : (int32_t)s;
}

}  // namespace

// The parts of v: split * T rows.  The split falls as T grows, and so may the
// product; the size is the largest of any call of up to T tokens, so that a
// workspace for the largest call serves the smaller ones.
size_t adapt_workspace(int64_t T, int32_t rank, int32_t in) {
    const int64_t parts = (rank + 16 * kRowTiles - 1) / (16 * kRowTiles);
    const int64_t most = (in + 64 * kShrinkWaves - 1) / (64 * kShrinkWaves);
    int64_t rows = T;
    for (int64_t s = 2; s <= most && s <= kMaxSplit; ++s) {
        const int64_t groups = kFill / (s * parts);  // the most that are split into s
        const int64_t spread = std::min({T, (int64_t)kSpreadTokens, groups}), tiled = std::min(T, groups * kTile);
        rows = std::max(rows, s * (tiled > kSpreadTokens ? tiled : spread));
    }
    return (size_t)round_up(rows * padded_rank(rank) * 4, 256);
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
    g.T = l.T;
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
