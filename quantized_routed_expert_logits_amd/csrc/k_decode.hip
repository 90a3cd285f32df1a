// The whole routed-expert layer for a few tokens (T <= 64, the decode batch of
// a server): the layer of strata_moe_prefill (Winery-Strata prefill.cpp page,
// MoE half of Prefill::run; Strata compare v0.1.35...v0.1.37 page,
// moe_fused.hpp) in the form that a handful of rows needs.
//
//   l[t][e] = x[t] . W_r[:, e] (+ bias)          exact products, 64-bit sums
//   ids[t]  = the K largest (ties: lower e), p = softmax over them
//   q, s    = x rounded to int8 per 32 values, s = max|x| / 127
//   G, U    = sum over blocks of d s sum (c - z) q      (2-bit codes c, fp16 d)
//   h       = silu(G) U, rounded to int8 per 32 values again
//   out[t]  = sum_k p_k sum over blocks of d s sum (c - z) q_h, k ascending
//
// The block sums P are exact integers: |P| <= 8128 for Q2_0, and twice the
// symmetric map's reach 12192, 14 bits.  P d s is exact in 64 bits (14 + 11 +
// 24), and the sums over blocks are held in 64, so the H codes are those of the
// definition.  A 32-bit sum can move a code over a rounding border, and the
// output by 1e-4 of its largest value; so can a 32-bit P d of the symmetric map
// where blocks cancel (it rounds from 2^24 on: 12189 times 2047/1024).  Q2_0's
// P d is exact in 32 bits and is taken there (64 tokens on hot experts 93.9 us,
// 94.6 with d s in 64; the symmetric 32 tokens 133.8, 133.3 with the rounded
// product).  One 64-bit FMA per output and block runs at the rate of a 32-bit one.
//
// Two launches.  What bounds them, at H = 2560, I = 1024, E = 512, K = 10: one
// token is a chain of latencies, 4.8 + 24.0 us (router, experts) for 30 MB of
// weights: the top-K takes about 4.5 of it, the gate/up products 3, what
// follows them 3, the hand-off to down 1, down with the combine 6, the launch
// the rest.  32 tokens are bound by memory: 8.0 + 124 to 132 us for 595 MB,
// 4.5 to 4.8 TB/s (a large copy reaches 5.1).  64 tokens on few hot experts
// (131 MB, 10.2 + 87 us) fill neither the memory (1.5 TB/s) nor the vector
// unit, 57% busy (a block's 16 outputs a lane take two conversions, a product
// and a 64-bit FMA each): 144 chunks of unequal rows are 1152 workgroups on 512
// places.
#include <algorithm>

#include "few_tokens.h"

namespace strata_moe {

namespace {

constexpr int kRouterSlices = 8;   // ranges of the router's reduction
constexpr int kThreads = 512;      // 8 waves
constexpr int kWavesD = kThreads / 64;
constexpr int kChunkTokens = 8;    // rows of a chunk at most
// Calls whose pairs read at most this many bytes of weights keep every pair on
// its own, larger ones group the pairs by expert: the grouping and its
// hand-offs cost 7 to 12 us, and the weights of one expert are read once for
// up to 8 rows.  Pairs against groups, in us: 4 tokens of the layer below (98
// MB) 43.9, 43.9, 6 tokens (147 MB) 56, 50, 8 tokens (197 MB) 66, 59; H, I =
// 1280, 512, 60 experts, 4 a token: 16 tokens (39 MB) 27, 33, 32 tokens (79
// MB) 33, 37, 64 tokens (157 MB) 47, 44.
constexpr int64_t kPairBytes = 80000000;
constexpr int kResident = 768;     // workgroups of an expert kernel that run at once, at most
// Polls before a wait gives up (seconds).  A wait ends by itself unless two
// calls at once were given one workspace.  Their results are lost then, but
// every wait still ends, and what a workgroup reads from the workspace as an
// index is held inside its range, so nothing outside the arrays is touched.
constexpr int kMaxPolls = 1 << 21;

// A chunk is up to 8 rows of one expert.  What is polled, counted and drawn has a line of its own (next to
// each other the counters' additions queued behind the polls).
struct Chunk {
    uint64_t head;  // expert << 32 | first row << 16 | rows
    uint64_t mask;  // the tokens, ascending row by row
    int32_t pad0[28];
    int32_t gu_done;  // gate/up workgroups finished
    int32_t pad1[31];
    int32_t ticket;   // workgroups that started: gate/up first, then down
    int32_t pad2[31];
};
static_assert(sizeof(Chunk) == 384, "three lines");

struct DecodeArgs {
    const float* x;
    const float* router_w;
    const float* bias;
    const float* shared_gate;
    const uint8_t* gate_up;
    int64_t gate_up_stride;
    const uint8_t* down;
    int64_t down_stride;
    int32_t T, H, E, K, I, shared;
    int32_t Kg, Eg;        // pairs per token, experts (with the shared one)
    int32_t n;             // T * Kg
    int32_t cap;           // most chunks
    int32_t split_gu, split_dn;  // waves that share a slab's reduction: 2, 4 or 8
    int32_t gw, dw;        // workgroups per chunk: gate/up, down
    float* out;
    double* part;          // [slices][T][Eg] partial logits (column E: the shared gate's dot product)
    int8_t* qx;            // [T][H]
    int2* sx;              // [T][H / 32]: scale (fp32 bits), sum of the codes
    int32_t* ids;          // [T][Kg]
    float* p;              // [T][Kg]
    int32_t* row_pair;     // [n]
    int8_t* qh;            // [n][I]
    int2* sh;              // [n][I / 32]
    float* dm;             // [n][H] weighted rows, by pair
    // cleared by the first kernel
    int32_t* clear;        // the words from here on
    int32_t nclear;
    int32_t* topk_next;    // tokens whose top-K is taken
    int32_t* topk_done;
    int32_t* nchunks;      // the chunk count plus one
    int32_t* dn_done;      // [T][H / 128] weighted rows finished
    Chunk* chunks;         // [cap]
};

// What workgroups of one launch hand to each other goes through agent-scope
// accesses: they pass the L2s, which differ between the XCDs.  The writer
// waits for its stores, then one thread counts them.
template <typename V>
__device__ __forceinline__ V peek(const V* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ void poke(V* p, V v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int bump(int32_t* p) {
    return __hip_atomic_fetch_add(p, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// An index read from the workspace, in [0, n) whatever was read.
__device__ __forceinline__ int in_range(int i, int n) { return (uint32_t)i < (uint32_t)n ? i : n - 1; }
// The wave's stores are done.
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// Every wave's stores are done once the workgroup is past this.
__device__ __forceinline__ void publish() {
    stores_done();
    __syncthreads();
}

__device__ __forceinline__ float round_half_away(float t) {
    const float r = floorf(fabsf(t) + 0.5f);
    return copysignf(fminf(r, 127.0f), t);
}

// ---------------------------------------------------------------- router
// fp64 logits on the fp64 matrix unit (16x16x4): every product of two fp32
// values is exact and the sums are 64-bit.  One workgroup: 16 experts (the
// product's rows), all tokens (its columns, NT tiles of 16), one slice of H,
// which the waves split.  A lane takes 4 consecutive values of h of one token,
// one per product, and the same 4 rows of the weights.  (On the vector unit
// with the tokens' values broadcast from LDS, 64 tokens took 18 us: every
// broadcast read holds the LDS for as long as a full one; this form takes 10.3,
// one token 4.8, of which the weights' 5.2 MB are one at 5.1 TB/s.)
typedef double v4d __attribute__((ext_vector_type(4)));

template <int NT>
__device__ void router_slice(const DecodeArgs& g, int tile, int slice, double* lds) {
    constexpr int kUnroll = NT == 4 ? 1 : 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, kg = lane >> 4;
    const int steps = g.H / 16, runs = kRouterSlices * kWavesD, per = (steps + runs - 1) / runs;
    const int first = (slice * kWavesD + wave) * per;
    const int s0 = first < steps ? first : steps, s1 = s0 + per < steps ? s0 + per : steps;
    const int e = tile * 16 + r16;
    const bool gate = g.shared && e == g.E;  // the shared expert's gate is one more column
    const float* w = gate ? g.shared_gate : g.router_w + (e < g.E ? e : g.E - 1);
    const int stride = gate ? 1 : g.E;
    const float* x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = g.x + (int64_t)(16 * n + r16 < g.T ? 16 * n + r16 : g.T - 1) * g.H + 4 * kg;
    v4d acc[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n] = v4d{0.0, 0.0, 0.0, 0.0};
#pragma unroll kUnroll
    for (int s = s0; s < s1; ++s) {
        float wv[4];
        float4 xv[NT];
#pragma unroll
        for (int j = 0; j < 4; ++j) wv[j] = w[(int64_t)(16 * s + 4 * kg + j) * stride];
#pragma unroll
        for (int n = 0; n < NT; ++n) xv[n] = *reinterpret_cast<const float4*>(x[n] + 16 * s);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float xs[4] = {xv[n].x, xv[n].y, xv[n].z, xv[n].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[n] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)wv[j], (double)xs[j], acc[n], 0, 0, 0);
        }
    }
    // a lane has experts kg + 4 i of token 16 n + r16
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) lds[((wave * NT + n) * 16 + r16) * 16 + kg + 4 * i] = acc[n][i];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 256; i += kThreads) {
        const int t = i >> 4, ee = tile * 16 + (i & 15);
        if (t >= g.T || ee >= g.Eg) continue;
        double s = 0.0;
#pragma unroll
        for (int o = 0; o < kWavesD; ++o) s += lds[o * NT * 256 + i];
        g.part[((int64_t)slice * g.T + t) * g.Eg + ee] = s;
    }
}

// One token's int8 rounding: 8 lanes per block of 32 values.
__device__ void quantize_token(const DecodeArgs& g, int t) {
    const float* x = g.x + (int64_t)t * g.H;
    for (int i = threadIdx.x; i < g.H / 4; i += kThreads) {
        const float4 v = reinterpret_cast<const float4*>(x)[i];
        float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
        for (int o = 1; o < 8; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
        const float s = m / 127.0f;
        const float c[4] = {v.x, v.y, v.z, v.w};
        uint32_t q = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int code = s != 0.0f ? (int)round_half_away(c[j] / s) : 0;
            q |= (uint32_t)(code & 0xff) << (8 * j);
        }
        int sum = __builtin_amdgcn_sdot4((int)q, 0x01010101, 0, false);
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor(sum, o);
        reinterpret_cast<uint32_t*>(g.qx + (int64_t)t * g.H)[i] = q;
        if ((threadIdx.x & 7) == 0)
            g.sx[(int64_t)t * (g.H / kBlock) + i / 8] = make_int2(__builtin_bit_cast(int, s), sum);
    }
}

template <int NT>
__global__ void __launch_bounds__(kThreads) decode_router_kernel(DecodeArgs g) {
    __shared__ double lds[kWavesD * NT * 256];
    const int tiles = (g.Eg + 15) / 16, nr = tiles * kRouterSlices, id = blockIdx.x;
    if (id < nr) {
        router_slice<NT>(g, id % tiles, id / tiles, lds);
    } else {
        for (int i = (id - nr) * kThreads + threadIdx.x; i < g.nclear; i += g.T * kThreads) g.clear[i] = 0;
        quantize_token(g, id - nr);
    }
}

// ------------------------------------------------------------ top-K, softmax
// The largest (or with kMin the smallest) of a wave's values, on every lane.
template <bool kMin>
__device__ __forceinline__ float wave_extreme(float x) {
    auto step = [&](auto ctrl) {
        const float o = __builtin_bit_cast(
            float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, x), __builtin_bit_cast(int, x), ctrl(), 0xf, 0xf, false));
        x = kMin ? fminf(x, o) : fmaxf(x, o);
    };
    step([] { return 0x111; });  // row_shr 1, 2, 4, 8
    step([] { return 0x112; });
    step([] { return 0x114; });
    step([] { return 0x118; });
    step([] { return 0x142; });  // the last lane of each row to the next row, of each half to the next half
    step([] { return 0x143; });
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}

// One workgroup, one token.  A wave takes 64 logits at a time and finds the
// best few of them, on the logits rounded to 32 bits (rounding never turns an
// order around).  The best few of every 64 together are at least K logits, so
// the K-th of those is a floor of the K-th of all: what reaches it, hardly
// more than K logits, is ranked in 64 bits, ties by the lower index.  A NaN
// ranks as -inf, so the ids are always K different ones.
struct TopkLds {
    double v[kMaxExperts];  // the candidates
    int e[kMaxExperts];
    double best[kMaxTopK], w[kMaxTopK];
    float4 top[16];         // the best few of every 64
    int count;
    int id[kMaxTopK];       // the result: experts in rank order,
    float p[kMaxTopK];      // their weights; the shared expert's behind them
};

__device__ void topk_token(const DecodeArgs& g, int t, TopkLds& l) {
    constexpr int kGroups = kMaxExperts / 64 / kWavesD;  // groups of 64 logits per wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float ninf = -__builtin_huge_valf();
    const int groups = (g.E + 63) / 64, few = (g.K + groups - 1) / groups + 1;  // groups * few <= 64
    if (threadIdx.x == 0) l.count = 0;
    float* top = (float*)l.top;
    if (threadIdx.x < 64) top[threadIdx.x] = ninf;
    double v[kGroups];
    float f[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int e = (wave + i * kWavesD) * 64 + lane;
        v[i] = ninf;
        f[i] = ninf;
        if (e < g.E) {
            double q[kRouterSlices];
#pragma unroll
            for (int s = 0; s < kRouterSlices; ++s) q[s] = g.part[((int64_t)s * g.T + t) * g.Eg + e];
            v[i] = 0.0;
#pragma unroll
            for (int s = 0; s < kRouterSlices; ++s) v[i] += q[s];
            if (g.bias) v[i] += (double)g.bias[e];
            if (!(v[i] == v[i])) v[i] = ninf;
            f[i] = (float)v[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int c = wave + i * kWavesD;
        if (c >= groups) break;
        float x = f[i];
        for (int n = 0; n < few; ++n) {  // equal ones count as one: the floor is lower then
            const float m = wave_extreme<false>(x);
            if (lane == 0) top[c * few + n] = m;
            if (x == m) x = ninf;
        }
    }
    __syncthreads();
    float floor;
    {
        const float x = top[lane];
        int above = 0;
        for (int j = 0; 4 * j < groups * few; j += 8) {  // -inf in the places behind
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 o = l.top[j + i];
                above += (int)(o.x > x) + (int)(o.y > x) + (int)(o.z > x) + (int)(o.w > x);
            }
        }
        floor = wave_extreme<true>(above < g.K && lane < groups * few ? x : __builtin_huge_valf());
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int e = (wave + i * kWavesD) * 64 + lane;
        const bool keep = e < g.E && f[i] >= floor;
        const uint64_t kept = __ballot(keep);
        if (kept == 0) continue;
        int base = 0;
        if (lane == 0) base = atomicAdd(&l.count, __popcll(kept));
        base = __builtin_amdgcn_readfirstlane(base);
        if (keep) {
            const int at = base + __popcll(kept & ((1ull << lane) - 1));
            l.v[at] = v[i];
            l.e[at] = e;
        }
    }
    __syncthreads();
    if (wave == 0) {
        const int n = l.count;
        for (int i = lane; i < n; i += 64) {
            const double c = l.v[i];
            const int e = l.e[i];
            int r = 0;
#pragma unroll 8
            for (int j = 0; j < n; ++j) r += (int)(l.v[j] > c) | ((int)(l.v[j] == c) & (int)(l.e[j] < e));
            if (r < g.K) {
                l.best[r] = c;
                l.id[r] = e;
            }
        }
        __builtin_amdgcn_wave_barrier();
        if (lane < g.K) l.w[lane] = exp(l.best[lane] - l.best[0]);
        __builtin_amdgcn_wave_barrier();
        if (lane < g.K) {
            double z = 0.0;
            for (int k = 0; k < g.K; ++k) z += l.w[k];
            l.p[lane] = (float)(l.w[lane] / z);
        }
    } else if (wave == 1 && g.shared) {
        double s = lane < kRouterSlices ? g.part[((int64_t)lane * g.T + t) * g.Eg + g.E] : 0.0;
        for (int o = 1; o < kRouterSlices; o <<= 1) s += __shfl_xor(s, o);
        if (lane == 0) {
            l.id[g.K] = g.E;
            l.p[g.K] = (float)(1.0 / (1.0 + exp(-s)));
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------------- grouping
// The pairs by expert, ascending token inside an expert.  A token picks an
// expert at most once, so an expert's rows are the set bits of a 64-bit mask
// of tokens and a pair's row is a population count.
struct GroupLds {
    uint64_t mask[kMaxExperts];
    int row0[kMaxExperts];
    int wsum[kWavesD];
};

__device__ void group_pairs(const DecodeArgs& g, GroupLds& l) {
    for (int e = threadIdx.x; e < kMaxExperts; e += kThreads) l.mask[e] = 0;
    __syncthreads();
    constexpr int kPer = (kDecodeMaxTokens * (kMaxTopK + 1) + kThreads - 1) / kThreads;
    int id[kPer];  // pairs threadIdx.x + j kThreads
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = threadIdx.x + j * kThreads;
        id[j] = i < g.n ? in_range(peek(&g.ids[i]), g.Eg) : -1;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (id[j] >= 0) atomicOr((unsigned long long*)&l.mask[id[j]], 1ull << ((threadIdx.x + j * kThreads) / g.Kg));
    __syncthreads();
    // exclusive scan of (rows, chunks) over the experts, packed in one int:
    // two experts a thread
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e0 = 2 * threadIdx.x;
    const int c0 = __popcll(l.mask[e0]), c1 = __popcll(l.mask[e0 + 1]);
    auto packed = [](int c) { return c | (c + kChunkTokens - 1) / kChunkTokens << 16; };
    const int mine = packed(c0) + packed(c1);
    int s = mine;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(s, o);
        if (lane >= o) s += v;
    }
    if (lane == 63) l.wsum[wave] = s;
    __syncthreads();
    int at = s - mine;
    for (int w = 0; w < wave; ++w) at += l.wsum[w];
    // the shared expert, the last one, has every token: its chunks go first
    const int first = g.shared ? (g.T + kChunkTokens - 1) / kChunkTokens : 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = e0 + j, c = j ? c1 : c0;
        l.row0[e] = at & 0xffff;
        uint64_t left = l.mask[e];
        for (int r = 0; r < c; r += kChunkTokens) {
            uint64_t rest = left;
            for (int k = 0; k < kChunkTokens; ++k) rest &= rest - 1;  // without the lowest 8 tokens
            const int ci = in_range((g.shared && e == g.E ? 0 : first + (at >> 16)) + r / kChunkTokens, g.cap);
            const int rows = c - r < kChunkTokens ? c - r : kChunkTokens;
            poke(&g.chunks[ci].head, ((uint64_t)e << 32) | ((uint64_t)((at & 0xffff) + r) << 16) | (uint64_t)rows);
            poke(&g.chunks[ci].mask, left ^ rest);
            left = rest;
        }
        at += packed(c);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        if (id[j] >= 0) {
            const int i = threadIdx.x + j * kThreads;
            poke(&g.row_pair[l.row0[id[j]] + __popcll(l.mask[id[j]] & ((1ull << (i / g.Kg)) - 1))], i);
        }
    publish();
    if (threadIdx.x == kThreads - 1) poke(g.nchunks, (at >> 16) + 1);
}

// ----------------------------------------------------------------- experts
// The products of one slab (128 weight rows) with up to 8 activation rows on
// the int8 matrix unit.  A record's dword p holds, per lane (row r = lane %
// 16, codes k = 8 (lane / 16) ..), the 16 codes of its rows in fragments A =
// 2p and B = 2p + 1, two bits each; shifted and masked it is 4 dwords of
// bytes A_k B_k A_k+1 B_k+1: 16 bytes, one operand of the 16x16x64 product.
// Against activations spread to a_k 0 a_k+1 0 that is fragment A's block sum,
// against 0 a_k 0 a_k+1 fragment B's, so the codes need no sorting (the
// 16x16x64 product takes the time of the 16x16x32 one).  Each is a sum over
// one 32-wide block, exact in int32, with the map's offset -z sum a as the
// product's initial value.
// The activations are the product's rows and the weights its columns: a lane
// gets, for its own weight row, the four product rows 4 kg + i, kg = lane /
// 16.  Activation row j has two product rows, 4 (j % 4) + 2 (j / 4) for its A
// spread and the next one for B, so one product serves both fragments, lane
// (r, kg) has rows kg and kg + 4 (NI = 2), and up to 4 rows need only the
// first two results (NI = 1).  Of a single row (kOne) every kg has the same
// sums: each takes the two fragments 2 kg and 2 kg + 1, a quarter of the
// scaling.
typedef int v4i __attribute__((ext_vector_type(4)));

template <bool kSym>
__device__ __forceinline__ v4i code_bytes(uint32_t w) {
    if constexpr (kSym)  // 2q
        return v4i{(int)((w << 1) & 0x06060606u), (int)((w >> 1) & 0x06060606u), (int)((w >> 3) & 0x06060606u),
                   (int)((w >> 5) & 0x06060606u)};
    return v4i{(int)(w & 0x03030303u), (int)((w >> 2) & 0x03030303u), (int)((w >> 4) & 0x03030303u),
               (int)((w >> 6) & 0x03030303u)};
}

// What a wave works on: blocks [b0, b0 + nb) of one slab against its chunk's
// rows, with the other waves of its split on the rest of the blocks.
struct Work {
    int e, row0, rows, c;
    const int* tok;  // [rows] tokens (LDS)
    int slab, part, b0, nb;
    int slab0, nslab;  // the workgroup's slabs
};

typedef unsigned int v2u __attribute__((ext_vector_type(2)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));

struct Weights {
    v4u c, d;    // a lane's 16 code bytes, its weight row's 8 fp16 scales (kOne: the two of its fragments)
};
template <int NI>
struct Acts {
    v2u q;       // a lane's 8 activation codes
    v2u s[NI];   // scale (fp32), code sum of its activation rows
};

constexpr int kBufferWord3 = 0x00020000;  // buffer descriptor word 3 for raw dword loads on gfx9 (gfx950)
constexpr int kAgentLoad = 16;            // a buffer load's sc1 bit: past the L2, as peek()

// p and bytes are the same on every lane (and so in scalar registers).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int bytes) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uintptr_t)p >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void*)(((uintptr_t)hi << 32) | lo), (short)0,
                                             __builtin_amdgcn_readfirstlane(bytes), kBufferWord3);
}

// Sums of a lane: fragments (of 8, or the lane's two) times rows.
template <int NI, bool kOne>
using Sums = double[kOne ? 2 : 8][NI];

// One block's products and scaling.  spread: the byte selectors of the lane's
// product row.
template <bool kSym, int NI, bool kOne>
__device__ __forceinline__ void block_sums(const Weights& r, const Acts<NI>& x, v2u spread, Sums<NI, kOne>& acc) {
    constexpr int zp = kSym ? -3 : -1;
    double sc[NI];
    v4i z{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        sc[i] = (double)__builtin_bit_cast(float, x.s[i][0]);
        z[2 * i] = z[2 * i + 1] = __mul24((int)x.s[i][1], zp);  // |sum| <= 32 * 127: a full-rate 24-bit multiply
    }
    const v4i a{(int)__builtin_amdgcn_perm(0u, x.q[0], spread[0]), (int)__builtin_amdgcn_perm(0u, x.q[0], spread[1]),
                (int)__builtin_amdgcn_perm(0u, x.q[1], spread[0]), (int)__builtin_amdgcn_perm(0u, x.q[1], spread[1])};
    auto product = [&](int p) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, code_bytes<kSym>(r.c[p]), z, 0, 0, 0); };
    // P d s, exactly: the symmetric map's P has 14 bits, so d s is formed first,
    // in 64; Q2_0's has 13, and P d is exact in 32
    auto term = [&](int p, float d, double s, double to) {
        if constexpr (kSym) return fma((double)p, (double)d * s, to);
        return fma((double)((float)p * d), s, to);
    };
    auto scale = [&](int pa, int pb, uint32_t d, int f, int i) {
        const float da = (float)__builtin_bit_cast(_Float16, (uint16_t)(d & 0xffffu));
        const float db = (float)__builtin_bit_cast(_Float16, (uint16_t)(d >> 16));
        acc[f][i] = term(pa, da, sc[i], acc[f][i]);
        acc[f + 1][i] = term(pb, db, sc[i], acc[f + 1][i]);
    };
    // the results that no row uses stay allocated until the product is done: a
    // register that a running product still writes cannot be taken without a stall
    auto hold = [](const v4i& v) { asm volatile("" ::"v"(v)); };
    if constexpr (kOne) {
        const v4i c0 = product(0), c1 = product(1), c2 = product(2), c3 = product(3);
        const int kg = threadIdx.x >> 4 & 3;
        const bool odd = kg & 1, high = kg & 2;
        hold(c0), hold(c1), hold(c2), hold(c3);
        const int a0 = odd ? c1[0] : c0[0], b0 = odd ? c1[1] : c0[1];
        const int a1 = odd ? c3[0] : c2[0], b1 = odd ? c3[1] : c2[1];
        scale(high ? a1 : a0, high ? b1 : b0, r.d[0], 0, 0);
        __builtin_amdgcn_sched_barrier(0);
    } else {
        // product p + 1 runs beside the scaling of product p
        v4i cur = product(0);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            v4i next;
            if (p < 3) next = product(p + 1);
#pragma unroll
            for (int i = 0; i < NI; ++i) scale(cur[2 * i], cur[2 * i + 1], r.d[p], 2 * p, i);
            hold(cur);
            if (p < 3) cur = next;
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// Where a chunk's activation rows are: row j's codes at q + row(j) * Kd, its
// blocks' (scale, code sum) at s + row(j) * Kd / 32 * 8.
struct ActRows {
    const int8_t* q;
    const int2* s;
    int rows_bound;  // rows of the arrays
};

// A chunk's rows in LDS: codes, act_stride() bytes apart (8 banks from row to
// row: the 4 lanes of 8 rows read without conflict), then (scale, code sum) of
// row j and block b at [b * kChunkTokens + j].
__device__ __forceinline__ int act_stride(int Kd) { return Kd + 32; }

template <bool kAgent, typename Row>
__device__ __forceinline__ void stage_acts(const ActRows& a, int Kd, int rows, Row row, char* lds) {
    constexpr int aux = kAgent ? kAgentLoad : 0;
    const int nblk = Kd / kBlock, per = Kd / 16;
    const __amdgpu_buffer_rsrc_t rq = buffer_of(a.q, a.rows_bound * Kd), rs = buffer_of(a.s, a.rows_bound * nblk * 8);
    uint64_t* sa = (uint64_t*)(lds + kChunkTokens * act_stride(Kd));
    for (int i = threadIdx.x; i < rows * per; i += kThreads) {
        const int j = i / per, k = i % per;
        *reinterpret_cast<v4u*>(lds + j * act_stride(Kd) + 16 * k) =
            __builtin_amdgcn_raw_buffer_load_b128(rq, row(j) * Kd + 16 * k, 0, aux);
    }
    for (int i = threadIdx.x; i < rows * nblk; i += kThreads) {
        const int j = i / nblk, k = i % nblk;
        const v2u v = __builtin_amdgcn_raw_buffer_load_b64(rs, (row(j) * nblk + k) * 8, 0, aux);
        sa[k * kChunkTokens + j] = __builtin_bit_cast(uint64_t, v);
    }
}

// acc[f][i]: the sums of weight row f * 16 + r and activation row kg + 4 i
// over the wave's blocks.  ready() is called once the first blocks' weights
// are on their way and before the activations are read; kAgent: they come
// from other workgroups.
// kDirect: the activations come with the weights, block by block, into
// registers (one row, where the latency of the first block counts).
// Otherwise the workgroup stages them in LDS: their loads, 16 bytes a lane or
// less of every 1280-byte block, took as long in the address path as those of
// the weights (32 tokens 151 us, 136 with the activations left out).
template <bool kSym, int NI, bool kOne, bool kAgent, bool kDirect, typename Row, typename Ready>
__device__ __forceinline__ void slab_sums(const Work& w, const uint8_t* rec, const ActRows& a, int Kd, Row row, char* lds,
                                          Sums<NI, kOne>& acc, Ready ready) {
    constexpr int kDepth = kDirect ? 2 : 4;  // blocks in flight
    constexpr int aux = kAgent ? kAgentLoad : 0;
    const int lane = threadIdx.x & 63, r16 = lane & 15, kg = lane >> 4;
    const int nblk = Kd / kBlock;
    const int mine = (r16 >> 2) + 4 * (r16 >> 1 & 1);  // the row in product row r16
    const v2u spread = r16 & 1 ? v2u{0x010c000cu, 0x030c020cu} : v2u{0x0c010c00u, 0x0c030c02u};
    const int last = w.nb > 0 ? w.nb - 1 : 0;     // past the run: its last block again, never used
    const __amdgpu_buffer_rsrc_t rr = buffer_of(rec, (last + 1) * kRecordBytes);
    const __amdgpu_buffer_rsrc_t rq = buffer_of(a.q, a.rows_bound * Kd), rs = buffer_of(a.s, a.rows_bound * nblk * 8);
    const int qrow = mine < w.rows ? mine : 0;
    int srow[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) srow[i] = kg + 4 * i < w.rows ? kg + 4 * i : 0;
    int qo = 0, so[NI] = {};
    const char* ql = lds + qrow * act_stride(Kd) + w.b0 * kBlock + 8 * kg;
    const uint64_t* sl = (const uint64_t*)(lds + kChunkTokens * act_stride(Kd)) + w.b0 * kChunkTokens;
    if constexpr (kDirect) {
        qo = row(qrow) * Kd + w.b0 * kBlock + 8 * kg;
#pragma unroll
        for (int i = 0; i < NI; ++i) so[i] = (row(srow[i]) * nblk + w.b0) * 8;
    }
    auto load_w = [&](int b, Weights& r) {
        const int at = (b < last ? b : last) * kRecordBytes;
        r.c = __builtin_amdgcn_raw_buffer_load_b128(rr, lane * 16, at, 0);
        if constexpr (kOne)
            r.d[0] = __builtin_amdgcn_raw_buffer_load_b32(rr, kRecordCodeBytes + r16 * 16 + 4 * kg, at, 0);
        else
            r.d = __builtin_amdgcn_raw_buffer_load_b128(rr, kRecordCodeBytes + r16 * 16, at, 0);
    };
    auto load_a = [&](int b, Acts<NI>& x) {
        b = b < last ? b : last;
        x.q = __builtin_amdgcn_raw_buffer_load_b64(rq, qo, b * kBlock, aux);
#pragma unroll
        for (int i = 0; i < NI; ++i) x.s[i] = __builtin_amdgcn_raw_buffer_load_b64(rs, so[i], b * 8, aux);
    };
    auto lds_a = [&](int b, Acts<NI>& x) {
        x.q = *reinterpret_cast<const v2u*>(ql + b * kBlock);
#pragma unroll
        for (int i = 0; i < NI; ++i) x.s[i] = __builtin_bit_cast(v2u, sl[b * kChunkTokens + srow[i]]);
    };
    Weights ring[kDepth];
    Acts<NI> act[kDirect ? kDepth : 1];
#pragma unroll
    for (int j = 0; j < kDepth; ++j) load_w(j, ring[j]);
    __builtin_amdgcn_sched_barrier(0);
    ready();
    asm volatile("" ::: "memory");
    if constexpr (kDirect) {
#pragma unroll
        for (int j = 0; j < kDepth; ++j) {
            load_a(j, act[j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    } else {
        stage_acts<kAgent>(a, Kd, w.rows, row, lds);
        __syncthreads();
    }
#pragma unroll
    for (int f = 0; f < (kOne ? 2 : 8); ++f)
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[f][i] = 0.0;
    // whole turns of the ring have no branches inside (each block's wait
    // counts the loads behind it), the rest of the run loads nothing more
    int b = 0;
    for (; b + kDepth <= w.nb; b += kDepth) {
#pragma unroll
        for (int j = 0; j < kDepth; ++j) {
            Acts<NI>& x = act[kDirect ? j : 0];
            if constexpr (!kDirect) lds_a(b + j, x);
            block_sums<kSym, NI, kOne>(ring[j], x, spread, acc);
            load_w(b + j + kDepth, ring[j]);
            if constexpr (kDirect) load_a(b + j + kDepth, x);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int j = 0; j < kDepth - 1; ++j)
        if (b + j < w.nb) {
            Acts<NI>& x = act[kDirect ? j : 0];
            if constexpr (!kDirect) lds_a(b + j, x);
            block_sums<kSym, NI, kOne>(ring[j], x, spread, acc);
        }
    if constexpr (!kDirect) __syncthreads();  // the activations are read: their LDS takes the sums
}

// Every wave's sums to LDS: [wave][4 NI][128], row j of the chunk, fragment
// order f * 16 + r.  The waves of a slab are next to each other.
template <int NI, bool kOne>
__device__ __forceinline__ void share_sums(const Work& w, const Sums<NI, kOne>& acc, double* lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r16 = lane & 15, kg = lane >> 4;
    if constexpr (kOne) {
        lds[wave * 4 * NI * 128 + 2 * kg * 16 + r16] = acc[0][0];
        lds[wave * 4 * NI * 128 + (2 * kg + 1) * 16 + r16] = acc[1][0];
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (kg + 4 * i < w.rows)
#pragma unroll
                for (int f = 0; f < 8; ++f) lds[(wave * 4 * NI + kg + 4 * i) * 128 + f * 16 + r16] = acc[f][i];
    }
    __syncthreads();
}

// Sum `at` (row j, fragment order) of the workgroup's slab s, its waves in order.
template <bool kSym, int NI>
__device__ __forceinline__ double slab_sum(int split, const double* lds, int s, int j, int at) {
    constexpr double unit = kSym ? 0.5 : 1.0;  // the symmetric map's codes are 2 (q - 1.5)
    double v = 0.0;
    for (int o = 0; o < split; ++o) v += lds[((s * split + o) * 4 * NI + j) * 128 + at];
    return unit * v;
}

// Gate/up of the workgroup's slabs: h = silu(G) U, rounded to int8.  Slab
// columns 0..63 are gate rows, 64..127 the up rows of the same H values; half
// a wave takes a block of 32.
template <bool kSym, int NI, bool kOne, bool kDirect>
__device__ void gate_up_slabs(const DecodeArgs& g, const Work& w, double* lds) {
    const uint8_t* rec = g.gate_up + (int64_t)w.e * g.gate_up_stride +
                         ((int64_t)w.slab * (g.H / kBlock) + w.b0) * kRecordBytes;
    Sums<NI, kOne> acc;
    slab_sums<kSym, NI, kOne, false, kDirect>(
        w, rec, ActRows{g.qx, g.sx, g.T}, g.H, [&](int j) { return w.tok[j]; }, (char*)lds, acc, [] {});
    share_sums<NI, kOne>(w, acc, lds);
    const int l = threadIdx.x & 31;
    for (int i = threadIdx.x >> 5; i < 2 * w.nslab * w.rows; i += kThreads / 32) {
        const int hb = i & 1, s = (i >> 1) % w.nslab, j = (i >> 1) / w.nslab;
        const double gt = slab_sum<kSym, NI>(g.split_gu, lds, s, j, 32 * hb + l);
        const double up = slab_sum<kSym, NI>(g.split_gu, lds, s, j, 64 + 32 * hb + l);
        const float h = (float)(gt / (1.0 + exp(-gt)) * up);
        float m = fabsf(h);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
        const float sc = m / 127.0f;
        const int code = sc != 0.0f ? (int)round_half_away(h / sc) : 0;
        int sum = code;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor(sum, o);
        uint32_t word = (uint32_t)(code & 0xff) << (8 * (l & 3));
        word |= __shfl_xor(word, 1);
        word |= __shfl_xor(word, 2);
        const int64_t row = w.row0 + j;
        const int blk = 2 * (w.slab0 + s) + hb;
        if ((l & 3) == 0) poke(reinterpret_cast<uint32_t*>(g.qh + row * g.I + 32 * blk + l), word);
        if (l == 1)
            poke(reinterpret_cast<uint64_t*>(g.sh + row * (g.I / kBlock) + blk),
                 (uint64_t)__builtin_bit_cast(uint32_t, sc) | (uint64_t)(uint32_t)sum << 32);
    }
    publish();
    if (threadIdx.x == 0) bump(&g.chunks[w.c].gu_done);
}

// Down of the workgroup's slabs: the weighted rows, and for every token and
// slab whose last row this is the sum of the rows, k ascending.
struct Rows {
    int pair[kChunkTokens];
    float weight[kChunkTokens];
    int last[kChunkTokens * kWavesD];  // [slab][row]
};

template <bool kSym, int NI, bool kOne, bool kDirect>
__device__ void down_slabs(const DecodeArgs& g, const Work& w, double* lds, Rows& rows, bool known) {
    const int nslab = g.H / kSlabRows;
    const uint8_t* rec = g.down + (int64_t)w.e * g.down_stride +
                         ((int64_t)w.slab * (g.I / kBlock) + w.b0) * kRecordBytes;
    Sums<NI, kOne> acc;
    auto ready = [&] {
        // the rows' pairs and weights, then the chunk's H rows
        if (!known && (int)threadIdx.x < w.rows) {
            const int pair = in_range(peek(&g.row_pair[w.row0 + threadIdx.x]), g.n);
            rows.pair[threadIdx.x] = pair;
            rows.weight[threadIdx.x] = peek(&g.p[pair]);
        }
        if (threadIdx.x == 0)
            for (int n = 0; n < kMaxPolls && peek(&g.chunks[w.c].gu_done) < g.gw; ++n) __builtin_amdgcn_s_sleep(2);
        __syncthreads();
    };
    slab_sums<kSym, NI, kOne, true, kDirect>(
        w, rec, ActRows{g.qh, g.sh, g.n}, g.I, [&](int j) { return w.row0 + j; }, (char*)lds, acc, ready);
    share_sums<NI, kOne>(w, acc, lds);
    for (int i = threadIdx.x; i < w.nslab * w.rows * 128; i += kThreads) {
        const int at = i & 127, s = (i >> 7) % w.nslab, j = (i >> 7) / w.nslab;
        poke(&g.dm[(int64_t)rows.pair[j] * g.H + 128 * (w.slab0 + s) + at],
             (float)((double)rows.weight[j] * slab_sum<kSym, NI>(g.split_dn, lds, s, j, at)));
    }
    publish();
    if ((int)threadIdx.x < w.nslab * w.rows) {
        const int s = threadIdx.x % w.nslab, j = threadIdx.x / w.nslab;
        rows.last[threadIdx.x] = bump(&g.dn_done[w.tok[j] * nslab + w.slab0 + s]) == g.Kg - 1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < w.nslab * w.rows * 64; i += kThreads) {
        if (!rows.last[i >> 6]) continue;
        const int s = (i >> 6) % w.nslab;
        const int64_t t = w.tok[(i >> 6) / w.nslab];
        const uint64_t* row = reinterpret_cast<const uint64_t*>(g.dm + t * g.Kg * g.H + 128 * (w.slab0 + s)) + (i & 63);
        double s0 = 0.0, s1 = 0.0;
#pragma unroll 4
        for (int k = 0; k < g.Kg; ++k) {
            const uint64_t v = peek(row + (int64_t)k * g.H / 2);
            s0 += (double)__builtin_bit_cast(float, (uint32_t)v);
            s1 += (double)__builtin_bit_cast(float, (uint32_t)(v >> 32));
        }
        reinterpret_cast<float2*>(g.out + t * g.H + 128 * (w.slab0 + s))[i & 63] = make_float2((float)s0, (float)s1);
    }
}

// Everything after the router in one launch.  A workgroup's number gives its
// chunk (chunk_of); what it does for the chunk is its next group of slabs,
// gate/up before down, by the chunk's ticket.  A workgroup that waits for the
// H rows of its chunk thus knows that their slabs are all in the hands of
// workgroups that run, and those wait for nothing but the top-K, which any
// waiting workgroup takes on itself while there are tokens left: every wait
// ends whatever order the workgroups start in and whatever else runs on the
// GPU.  (One ticket for all workgroups in a loop over the work, with the next
// ticket drawn ahead, took 162 us for 32 tokens against 138.)
__device__ int chunk_of(const DecodeArgs& g, int id, int nch) {
    // gate/up runs `lag` chunks ahead of down, more than run at once
    int lag = kResident / g.gw + 1;
    if (lag > nch) lag = nch;
    if (id < lag * g.gw) return id / g.gw;
    id -= lag * g.gw;
    const int both = g.gw + g.dw, whole = (nch - lag) * both;
    if (id < whole) return id % both < g.gw ? lag + id / both : id / both;
    return nch - lag + (id - whole) / g.dw;
}

// The wave's part of the workgroup's slabs.
__device__ __forceinline__ bool split_slabs(const DecodeArgs& g, int ticket, Work& w) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    ticket = in_range(ticket, g.gw + g.dw);
    const bool gate_up = ticket < g.gw;
    const int slabs = gate_up ? g.I / 64 : g.H / kSlabRows, split = gate_up ? g.split_gu : g.split_dn;
    const int per = kWavesD / split;
    w.slab0 = (gate_up ? ticket : ticket - g.gw) * per;
    w.nslab = slabs - w.slab0 < per ? slabs - w.slab0 : per;
    w.slab = w.slab0 + wave / split;
    w.part = wave % split;
    const int nblk = (gate_up ? g.H : g.I) / kBlock, run = (nblk + split - 1) / split;
    w.b0 = w.part * run;
    w.nb = w.b0 + run <= nblk ? run : nblk - w.b0;
    // a wave without blocks or a slab still meets the others' barriers
    if (w.nb <= 0) w.nb = 0, w.b0 = 0;
    if (w.slab >= slabs) w.nb = 0, w.slab = w.slab0;
    return gate_up;
}

// A chunk is one pair, and every workgroup finds its expert by the token's
// top-K itself.  Two blocks in flight leave room for 3 workgroups per CU (4
// tokens: 42.7 us, with four blocks and 2 workgroups 48.5; one token 27.4,
// 28.1).
template <bool kSym>
__global__ void __launch_bounds__(kThreads, 6) decode_pairs_kernel(DecodeArgs g) {
    extern __shared__ double lds[];
    __shared__ int taken;
    __shared__ int tok[kChunkTokens];
    __shared__ Rows rows;
    const int c = chunk_of(g, blockIdx.x, g.n);
    int ticket = 0;
    if (threadIdx.x == 0) ticket = bump(&g.chunks[c].ticket);
    TopkLds& l = *(TopkLds*)lds;
    const int t = c / g.Kg, k = c % g.Kg;
    topk_token(g, t, l);
    Work w;
    w.c = w.row0 = c;
    w.tok = tok;
    w.e = __builtin_amdgcn_readfirstlane(l.id[k]);
    w.rows = 1;
    if (threadIdx.x == 0) {
        taken = ticket;
        tok[0] = t;
        rows.pair[0] = c;
        rows.weight[0] = l.p[k];
    }
    __syncthreads();
    if (split_slabs(g, __builtin_amdgcn_readfirstlane(taken), w))
        gate_up_slabs<kSym, 1, true, true>(g, w, lds);
    else
        down_slabs<kSym, 1, true, true>(g, w, lds, rows, true);
}

// More tokens: the top-K of the tokens and the grouping by whichever
// workgroups come first, then a chunk's slabs each.
template <bool kSym>
__global__ void __launch_bounds__(kThreads, 4) decode_chunks_kernel(DecodeArgs g) {
    extern __shared__ double lds[];
    __shared__ int todo[4];  // what thread 0 found
    __shared__ Chunk chunk;
    __shared__ int tok[kChunkTokens];
    __shared__ Rows rows;
    for (;;) {
        if (threadIdx.x == 0) {
            int what = 2;  // nothing
            for (int n = 0; n < kMaxPolls; ++n) {
                int nch = peek(g.nchunks) - 1;
                if (nch >= 0) {
                    if (nch > g.cap) nch = g.cap;
                    // (more workgroups are launched than the chunks may need)
                    if ((int)blockIdx.x < nch * (g.gw + g.dw)) {
                        const int c = chunk_of(g, blockIdx.x, nch);
                        const uint64_t head = peek(&g.chunks[c].head), mask = peek(&g.chunks[c].mask);
                        chunk.ticket = bump(&g.chunks[c].ticket);
                        chunk.head = head, chunk.mask = mask;
                        todo[1] = c;
                        what = 0;
                    }
                    break;
                }
                if (peek(g.topk_next) < g.T) {
                    const int t = bump(g.topk_next);
                    if ((uint32_t)t < (uint32_t)g.T) {
                        todo[1] = t;
                        what = 1;
                        break;
                    }
                }
                __builtin_amdgcn_s_sleep(1);
            }
            todo[0] = what;
        }
        __syncthreads();
        const int what = __builtin_amdgcn_readfirstlane(todo[0]);
        if (what == 2) return;
        if (what == 0) break;
        TopkLds& l = *(TopkLds*)lds;
        const int t = todo[1];
        topk_token(g, t, l);
        if ((int)threadIdx.x < g.Kg) {
            poke(&g.ids[t * g.Kg + threadIdx.x], l.id[threadIdx.x]);
            poke(&g.p[t * g.Kg + threadIdx.x], l.p[threadIdx.x]);
        }
        publish();
        if (threadIdx.x == 0) todo[2] = bump(g.topk_done) == g.T - 1;
        __syncthreads();
        if (todo[2]) group_pairs(g, *(GroupLds*)lds);
        __syncthreads();
    }
    const uint64_t mask = chunk.mask;
    const int most = g.n < kChunkTokens ? g.n : kChunkTokens, rows_of = (int)(chunk.head & 0xffff);
    Work w;
    w.c = __builtin_amdgcn_readfirstlane(todo[1]);
    w.e = in_range(__builtin_amdgcn_readfirstlane((int)(chunk.head >> 32)), g.Eg);
    w.rows = __builtin_amdgcn_readfirstlane(rows_of < most ? rows_of : most);
    w.row0 = in_range(__builtin_amdgcn_readfirstlane((int)(chunk.head >> 16 & 0xffff)), g.n - w.rows + 1);
    w.tok = tok;
    if (threadIdx.x < 64) {
        const int row = __popcll(mask & ((1ull << threadIdx.x) - 1));
        if ((mask >> threadIdx.x & 1) && row < kChunkTokens) tok[row] = in_range(threadIdx.x, g.T);
        if ((int)threadIdx.x >= __popcll(mask) && threadIdx.x < kChunkTokens) tok[threadIdx.x] = 0;
    }
    __syncthreads();
    if (split_slabs(g, __builtin_amdgcn_readfirstlane(chunk.ticket), w)) {
        if (w.rows > 4)
            gate_up_slabs<kSym, 2, false, false>(g, w, lds);
        else if (w.rows > 1)
            gate_up_slabs<kSym, 1, false, false>(g, w, lds);
        else
            gate_up_slabs<kSym, 1, true, false>(g, w, lds);
    } else {
        if (w.rows > 4)
            down_slabs<kSym, 2, false, false>(g, w, lds, rows, false);
        else if (w.rows > 1)
            down_slabs<kSym, 1, false, false>(g, w, lds, rows, false);
        else
            down_slabs<kSym, 1, true, false>(g, w, lds, rows, false);
    }
}

// Most chunks of n pairs: one for every expert hit, and one more for every 8
// rows of an expert.
int64_t chunk_cap(int64_t n, int64_t Eg, bool pairs) {
    return pairs || n < Eg + n / kChunkTokens ? n : Eg + n / kChunkTokens;
}

// The form of a call: up to this many pairs each stays on its own, more are grouped.
int64_t most_pairs(int32_t H, int32_t I) { return kPairBytes / ((int64_t)3 * H * I / 16 * 5); }

// The workspace of one call.
struct Plan {
    size_t part, qx, sx, ids, p, row_pair, qh, sh, dm, words, dn_done, chunks, total;
};

Plan plan(int32_t T, int32_t H, int32_t E, int32_t K, int32_t I, bool shared) {
    const int64_t Eg = E + shared, n = (int64_t)T * (K + shared), cap = chunk_cap(n, Eg, n <= most_pairs(H, I));
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        const size_t at = off;
        off += (size_t)round_up(bytes > 0 ? bytes : 1, 256);
        return at;
    };
    Plan o;
    o.part = take((int64_t)kRouterSlices * T * Eg * 8);
    o.qx = take((int64_t)T * H);
    o.sx = take((int64_t)T * (H / kBlock) * 8);
    o.ids = take(n * 4);
    o.p = take(n * 4);
    o.row_pair = take(n * 4);
    o.qh = take(n * I);
    o.sh = take(n * (I / kBlock) * 8);
    o.dm = take(n * H * 4);
    o.words = take(3 * 256);
    o.dn_done = take((int64_t)T * (H / kSlabRows) * 4);
    o.chunks = take(cap * (int64_t)sizeof(Chunk));
    o.total = off;
    return o;
}

}  // namespace

size_t decode_workspace(int32_t T, int32_t H, int32_t E, int32_t K, int32_t I, bool shared) {
    // Grouped calls need room for fewer chunks than the last call of pairs; the
    // size is the largest of any call of up to T tokens, so that a workspace for
    // the largest call serves the smaller ones.
    const int64_t last = most_pairs(H, I) / (K + shared);
    const size_t own = plan(T, H, E, K, I, shared).total;
    return last < T ? std::max(own, plan((int32_t)last, H, E, K, I, shared).total) : own;
}

hipError_t launch_decode(const DecodeLaunch& l, hipStream_t st) {
    DecodeArgs g{};
    g.x = l.x;
    g.router_w = l.router_w;
    g.bias = l.bias;
    g.shared_gate = l.shared_gate;
    g.gate_up = l.gate_up;
    g.gate_up_stride = l.gate_up_stride;
    g.down = l.down;
    g.down_stride = l.down_stride;
    g.T = l.T;
    g.H = l.H;
    g.E = l.E;
    g.K = l.K;
    g.I = l.I;
    g.shared = l.shared_gate != nullptr;
    g.Kg = l.K + g.shared;
    g.Eg = l.E + g.shared;
    g.n = l.T * g.Kg;
    g.out = l.out;
    const Plan o = plan(l.T, l.H, l.E, l.K, l.I, g.shared);
    char* ws = l.workspace;
    const bool pairs = g.n <= most_pairs(g.H, g.I);
    g.cap = (int32_t)chunk_cap(g.n, g.Eg, pairs);
    g.part = (double*)(ws + o.part);
    g.qx = (int8_t*)(ws + o.qx);
    g.sx = (int2*)(ws + o.sx);
    g.ids = (int32_t*)(ws + o.ids);
    g.p = (float*)(ws + o.p);
    g.row_pair = (int32_t*)(ws + o.row_pair);
    g.qh = (int8_t*)(ws + o.qh);
    g.sh = (int2*)(ws + o.sh);
    g.dm = (float*)(ws + o.dm);
    g.clear = (int32_t*)(ws + o.words);
    g.nclear = (int32_t)((o.total - o.words) / 4);
    g.topk_next = (int32_t*)(ws + o.words);
    g.topk_done = (int32_t*)(ws + o.words + 256);
    g.nchunks = (int32_t*)(ws + o.words + 512);
    g.dn_done = (int32_t*)(ws + o.dn_done);
    g.chunks = (Chunk*)(ws + o.chunks);
    void (*router)(DecodeArgs) =
        g.T <= 16 ? decode_router_kernel<1> : g.T <= 32 ? decode_router_kernel<2> : decode_router_kernel<4>;
    hipLaunchKernelGGL(router, dim3((g.Eg + 15) / 16 * kRouterSlices + g.T), dim3(kThreads), 0, st, g);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    // The waves of a slab: all 8 while the slabs are few (the latency of one
    // counts), fewer as the workgroups fill the chip anyway; down, whose
    // reduction is the shorter one, halves first.  In us at H = 2560, I = 1024,
    // E = 512, K = 10, (gate/up, down) waves (8, 8), (8, 4), (4, 4), (4, 2),
    // (2, 2): one token 29.2, 27.9, 27.8, 30.6, 36.9; 4 tokens 46.7, 43.0, 48.8,
    // 51.6, 51.8; 8 tokens 70.1, 61.8, 57.5, 57.1, 62.1; 16 tokens 120, 104,
    // 93.4, 88.0, 84.7; 32 tokens 202, 170, 150, 137, 133.  The slabs are those
    // of the most chunks possible.  Where few of these exist the rule can miss:
    // 64 tokens on hot experts of I = 640 (144 chunks of 601 possible) 163, 128,
    // 111, 93.1, 94.0; 8 tokens there 59.8, 50.3, 50.7, 56.9, 62.2.
    // But a wave has 4 blocks at least where the reduction gives them: H = 512,
    // I = 640, 6 experts, 33 tokens 26.5 us, without this 36; H = I = 256, 64
    // experts, 64 tokens 29, 37.
    const int gu = g.I / 64, dn = g.H / kSlabRows;
    const int64_t slabs = (int64_t)g.cap * (gu + dn);
    g.split_gu = slabs <= 2000 ? 8 : slabs <= 4000 ? 4 : 2;
    g.split_dn = slabs <= 288 ? 8 : slabs <= 2000 ? 4 : 2;
    while (g.split_gu > 2 && g.H / kBlock < 4 * g.split_gu) g.split_gu /= 2;
    while (g.split_dn > 2 && g.I / kBlock < 4 * g.split_dn) g.split_dn /= 2;
    g.gw = (gu * g.split_gu + kWavesD - 1) / kWavesD;
    g.dw = (dn * g.split_dn + kWavesD - 1) / kWavesD;
    size_t lds = sizeof(TopkLds) > sizeof(GroupLds) ? sizeof(TopkLds) : sizeof(GroupLds);
    const size_t sums = (size_t)kWavesD * (pairs ? 4 : 8) * 128 * 8;
    if (sums > lds) lds = sums;
    if (!pairs)
        for (const int Kd : {g.H, g.I}) {
            const size_t acts = (size_t)kChunkTokens * (Kd + 32) + (size_t)kChunkTokens * (Kd / kBlock) * 8;
            if (acts > lds) lds = acts;
        }
    const dim3 grid(g.cap * (g.gw + g.dw));
    void (*kernel)(DecodeArgs);
    if (pairs)
        kernel = l.sym ? decode_pairs_kernel<true> : decode_pairs_kernel<false>;
    else
        kernel = l.sym ? decode_chunks_kernel<true> : decode_chunks_kernel<false>;
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), lds, st, g);
    return hipGetLastError();
}

}  // namespace strata_moe
