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
// The block sums are exact integers; a block sum times the fp16 d is exact in
// 32 bits (13 + 11 bits), and the sums over blocks are held in 64 bits: one
// 64-bit FMA per output and block runs at the rate of a 32-bit one here, and
// it makes the H codes those of the definition (a 32-bit G moves about one
// code in 10^5 over a rounding border).
#include "internal.h"

namespace strata_moe {

namespace {

constexpr int kRouterSlices = 16;  // ranges of the router's reduction
constexpr int kThreads = 512;      // 8 waves
constexpr int kWavesD = kThreads / 64;
constexpr int kPassRows = 8;       // rows per pass over a chunk's weights
constexpr int kResident = 512;     // workgroups of the expert kernel that run at once, about
// Polls before a wait gives up (seconds).  A wait ends by itself unless the
// caller let two calls share a workspace; then the results are lost, not the GPU.
constexpr int kMaxPolls = 1 << 21;

// A chunk is the rows of one expert.  Both words are nonzero once written.
struct Chunk {
    uint64_t head;  // expert << 32 | first row << 16 | rows
    uint64_t mask;  // the tokens, ascending row by row
};

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
    int32_t cap;           // most chunks: min(n, Eg)
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
    int32_t* ticket;       // [cap] slabs taken of a chunk: gate/up first, then down
    int32_t* gu_done;      // [cap] gate/up slabs finished
    int32_t* dn_done;      // [T][H / 128] weighted rows finished
    Chunk* chunks;         // [cap]
};

// What workgroups of one launch hand to each other goes through agent-scope
// accesses: they pass the L2s, which differ between the XCDs.  The writer
// waits for its stores (publish), then one thread counts them.
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
// Every wave's stores are done once the workgroup is past this.
__device__ __forceinline__ void publish() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
}

__device__ __forceinline__ float round_half_away(float t) {
    const float r = floorf(fabsf(t) + 0.5f);
    return copysignf(fminf(r, 127.0f), t);
}

// ---------------------------------------------------------------- router
// One workgroup: 64 experts (a lane each), one slice of H, TT tokens.
template <int TT>
__device__ void router_slice(const DecodeArgs& g, int group, int slice, int t0, double* lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int hs = g.H / kRouterSlices, h0 = slice * hs;
    double* xs = lds;                       // [hs][TT]
    double* red = lds + (size_t)hs * TT;    // [waves][TT][64]
    for (int i = threadIdx.x; i < hs * TT; i += kThreads) {
        const int t = t0 + i / hs, h = i % hs;
        xs[h * TT + i / hs] = t < g.T ? (double)g.x[(int64_t)t * g.H + h0 + h] : 0.0;
    }
    __syncthreads();
    const int e = group * 64 + lane;
    double acc[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[j] = 0.0;
    const bool gate = e == g.E && g.shared;
    if (e < g.E || gate) {
        const float* w = gate ? g.shared_gate + h0 : g.router_w + (int64_t)h0 * g.E + e;
        const int64_t step = gate ? 1 : g.E;
#pragma unroll 4
        for (int h = wave; h < hs; h += kWavesD) {
            const double wv = (double)w[h * step];
#pragma unroll
            for (int j = 0; j < TT; ++j) acc[j] = fma(wv, xs[h * TT + j], acc[j]);
        }
    }
#pragma unroll
    for (int j = 0; j < TT; ++j) red[(wave * TT + j) * 64 + lane] = acc[j];
    __syncthreads();
    for (int i = threadIdx.x; i < TT * 64; i += kThreads) {
        const int j = i >> 6, l = i & 63, ee = group * 64 + l;
        if (t0 + j >= g.T || ee >= g.Eg) continue;
        double s = 0.0;
        for (int w = 0; w < kWavesD; ++w) s += red[(w * TT + j) * 64 + l];
        g.part[((int64_t)slice * g.T + t0 + j) * g.Eg + ee] = s;
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

template <int TT>
__global__ void __launch_bounds__(kThreads) decode_router_kernel(DecodeArgs g) {
    extern __shared__ double lds[];
    const int groups = (g.Eg + 63) / 64, tg = (g.T + TT - 1) / TT;
    const int nr = groups * kRouterSlices * tg;
    const int id = blockIdx.x;
    if (id < nr)
        router_slice<TT>(g, id % groups, id / groups % kRouterSlices, id / groups / kRouterSlices * TT, lds);
    else {
        for (int i = (id - nr) * kThreads + threadIdx.x; i < g.nclear; i += g.T * kThreads) g.clear[i] = 0;
        quantize_token(g, id - nr);
    }
}

// ------------------------------------------------------------ top-K, softmax
// One workgroup, one token.  A wave takes 64 logits and keeps those with
// fewer than K larger ones among them, counted on the logits rounded to 32
// bits (rounding never turns an order around, so a superset of the wave's
// best K stays); the kept ones are ranked in 64 bits, ties by the lower
// index.  A NaN ranks as -inf, so the ids are always K different ones.
struct TopkLds {
    double v[kMaxExperts];
    int e[kMaxExperts];
    int rank[kMaxExperts];
    double best[kMaxTopK], w[kMaxTopK];
    int id[kMaxTopK];
    int count;
};

__device__ void topk_token(const DecodeArgs& g, int t, TopkLds& l) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double ninf = -__builtin_huge_val();
    if (threadIdx.x == 0) l.count = 0;
    for (int i = threadIdx.x; i < kMaxExperts; i += kThreads) l.rank[i] = 0;
    __syncthreads();
    for (int c = wave; c * 64 < g.E; c += kWavesD) {
        const int e = c * 64 + lane;
        double v = ninf;
        if (e < g.E) {
            double q[kRouterSlices];
#pragma unroll
            for (int s = 0; s < kRouterSlices; ++s) q[s] = g.part[((int64_t)s * g.T + t) * g.Eg + e];
            v = 0.0;
#pragma unroll
            for (int s = 0; s < kRouterSlices; ++s) v += q[s];
            if (g.bias) v += (double)g.bias[e];
            if (!(v == v)) v = ninf;
        }
        const float f = (float)v;
        int larger = 0;
#pragma unroll 16
        for (int j = 0; j < 64; ++j) {
            const float o = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), j));
            larger += o > f ? 1 : 0;
        }
        const bool keep = e < g.E && larger < g.K;
        const uint64_t kept = __ballot(keep);
        int base = 0;
        if (lane == 0) base = atomicAdd(&l.count, __popcll(kept));
        base = __builtin_amdgcn_readfirstlane(base);
        if (keep) {
            const int at = base + __popcll(kept & ((1ull << lane) - 1));
            l.v[at] = v;
            l.e[at] = e;
        }
    }
    __syncthreads();
    const int n = l.count;
    // rank candidate i among 4 quarters of the candidates
    for (int i = threadIdx.x & 127; i < n; i += 128) {
        const double v = l.v[i];
        const int e = l.e[i], part = threadIdx.x >> 7;
        int r = 0;
#pragma unroll 8
        for (int j = part; j < n; j += 4) r += (l.v[j] > v || (l.v[j] == v && l.e[j] < e)) ? 1 : 0;
        if (r) atomicAdd(&l.rank[i], r);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (l.rank[i] < g.K) {
            l.best[l.rank[i]] = l.v[i];
            l.id[l.rank[i]] = l.e[i];
        }
    __syncthreads();
    if ((int)threadIdx.x < g.K) l.w[threadIdx.x] = exp(l.best[threadIdx.x] - l.best[0]);
    __syncthreads();
    if ((int)threadIdx.x < g.K) {
        double z = 0.0;
        for (int k = 0; k < g.K; ++k) z += l.w[k];
        poke(&g.ids[t * g.Kg + threadIdx.x], l.id[threadIdx.x]);
        poke(&g.p[t * g.Kg + threadIdx.x], (float)(l.w[threadIdx.x] / z));
    }
    if (g.shared && threadIdx.x == 64) {
        double v = 0.0;
        for (int s = 0; s < kRouterSlices; ++s) v += g.part[((int64_t)s * g.T + t) * g.Eg + g.E];
        poke(&g.ids[t * g.Kg + g.K], g.E);
        poke(&g.p[t * g.Kg + g.K], (float)(1.0 / (1.0 + exp(-v))));
    }
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
    for (int i = threadIdx.x; i < g.n; i += kThreads)
        atomicOr((unsigned long long*)&l.mask[peek(&g.ids[i]) & (kMaxExperts - 1)], 1ull << (i / g.Kg));
    __syncthreads();
    // exclusive scan of (rows, hit experts) over the experts, packed in one
    // int: two experts a thread
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e0 = 2 * threadIdx.x;
    const int c0 = __popcll(l.mask[e0]), c1 = __popcll(l.mask[e0 + 1]);
    const int mine = (c0 | (c0 > 0 ? 1 << 16 : 0)) + (c1 | (c1 > 0 ? 1 << 16 : 0));
    int s = mine;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(s, o);
        if (lane >= o) s += v;
    }
    if (lane == 63) l.wsum[wave] = s;
    __syncthreads();
    int at = s - mine;
    for (int w = 0; w < wave; ++w) at += l.wsum[w];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = e0 + j, c = j ? c1 : c0;
        l.row0[e] = at & 0xffff;
        if (c > 0) {
            // the shared expert's chunk has every token: it goes first
            const int ci = g.shared ? (e == g.E ? 0 : (at >> 16) + 1) : at >> 16;
            poke(&g.chunks[ci].head, ((uint64_t)e << 32) | ((uint64_t)(at & 0xffff) << 16) | (uint64_t)c);
            poke(&g.chunks[ci].mask, l.mask[e]);
            at += c | (1 << 16);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.n; i += kThreads) {
        const int e = peek(&g.ids[i]) & (kMaxExperts - 1), t = i / g.Kg;
        poke(&g.row_pair[l.row0[e] + __popcll(l.mask[e] & ((1ull << t) - 1))], i);
    }
    publish();
    if (threadIdx.x == kThreads - 1) poke(g.nchunks, (at >> 16) + 1);
}

// ----------------------------------------------------------------- experts
// The products of one slab (128 weight rows) with up to 8 activation rows
// on the int8 matrix unit.  A record's dword p holds, per lane (row r = lane
// % 16, codes k = 8 (lane / 16) ..), the 16 codes of its rows in fragments A =
// 2p and B = 2p + 1, two bits each; shifted and masked it is 4 dwords of
// bytes A_k B_k A_k+1 B_k+1: 16 bytes, one operand of the 16x16x64 product.
// Against activations spread to a_k 0 a_k+1 0 that is fragment A's block sum,
// against 0 a_k 0 a_k+1 fragment B's, so the codes need no sorting (the
// 16x16x64 product takes the time of the 16x16x32 one).  Each is a sum over
// one 32-wide block, exact in int32, with the map's offset -z sum a as the
// product's initial value.
// The activations are the product's rows and the weights its columns: a lane
// gets, for its own weight row, the four activation rows 4 (lane / 16) + i.
// Row j of the pass sits in product row 4 (j % 4) + j / 4, so up to 4 NI rows
// need only the results i < NI.
// The thread's index, opaque to the compiler: what is computed from it stays
// inside the pass that needs it (hoisted out of the loop over passes it took
// some 40 registers through every pass).
__device__ __forceinline__ int pass_thread() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

typedef int v4i __attribute__((ext_vector_type(4)));

struct Block {
    uint4 c, d;  // a lane's 16 code bytes, its row's 8 fp16 scales
};

template <bool kSym>
__device__ __forceinline__ v4i code_bytes(uint32_t w) {
    if constexpr (kSym)  // 2q
        return v4i{(int)((w << 1) & 0x06060606u), (int)((w >> 1) & 0x06060606u), (int)((w >> 3) & 0x06060606u),
                   (int)((w >> 5) & 0x06060606u)};
    return v4i{(int)(w & 0x03030303u), (int)((w >> 2) & 0x03030303u), (int)((w >> 4) & 0x03030303u),
               (int)((w >> 6) & 0x03030303u)};
}

// The activations of a pass in LDS: code rows `stride` bytes apart, then
// (scale, code sum) of row j and block b at [b * rows + j].
__device__ __forceinline__ int act_stride(int Kd) { return Kd + 8; }

// One pass: `rows` activation rows of a Kd-long reduction against the slab at
// rec0.  stage(codes, scales) fills the LDS once the first blocks' loads are
// out.  Returns in lds tot[4 NI][128] doubles: row j, fragment order f * 16 + r.
template <bool kSym, int NI, typename Stage>
__device__ void slab_pass(const uint8_t* rec0, int Kd, char* lds, Stage stage) {
    constexpr int R = 4 * NI;
    constexpr int kDepth = NI == 1 ? 5 : 4;  // blocks in flight per wave, as the registers allow
    const int nblk = Kd / kBlock;
    const int tid = pass_thread();
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r16 = lane & 15, kg = lane >> 4;
    const int per = (nblk + kWavesD - 1) / kWavesD;
    const int b0 = wave * per, nb = b0 + per <= nblk ? per : (b0 < nblk ? nblk - b0 : 0);
    auto load = [&](int b, Block& r) {
        const int bb = b < nb ? b0 + b : (nb > 0 ? b0 + nb - 1 : 0);  // past the run: a block that is never used
        const uint8_t* rec = rec0 + (int64_t)bb * kRecordBytes;
        r.c = *reinterpret_cast<const uint4*>(rec + lane * 16);
        r.d = *reinterpret_cast<const uint4*>(rec + kRecordCodeBytes + r16 * 16);
    };
    Block ring[kDepth];
#pragma unroll
    for (int j = 0; j < kDepth; ++j) load(j, ring[j]);
    __builtin_amdgcn_sched_barrier(0);
    uint8_t* qa = (uint8_t*)lds;
    int2* sa = (int2*)(lds + R * act_stride(Kd));
    stage(qa, sa, tid);
    __syncthreads();
    const int slot = r16 >> 2 | (r16 & 3) << 2;  // product row m holds row m / 4 + 4 (m % 4)
    const uint8_t* qrow = qa + (slot < R ? slot : 0) * act_stride(Kd) + 8 * kg;
    constexpr int zp = kSym ? -3 : -1;
    double acc[8][NI];
#pragma unroll
    for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[f][i] = 0.0;
    for (int b = 0; b < nb; b += kDepth) {
#pragma unroll
        for (int j = 0; j < kDepth; ++j) {
            if (b + j < nb) {
                const Block r = ring[j];
                const int blk = b0 + b + j;
                const uint2 q = *reinterpret_cast<const uint2*>(qrow + blk * kBlock);
                double s[NI];
                v4i z{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int2 v = sa[blk * R + kg + 4 * i];
                    s[i] = (double)__builtin_bit_cast(float, v.x);
                    z[i] = zp * v.y;
                }
                v4i aA, aB;
                aA[0] = (int)__builtin_amdgcn_perm(0u, q.x, 0x0c010c00u);
                aA[1] = (int)__builtin_amdgcn_perm(0u, q.x, 0x0c030c02u);
                aA[2] = (int)__builtin_amdgcn_perm(0u, q.y, 0x0c010c00u);
                aA[3] = (int)__builtin_amdgcn_perm(0u, q.y, 0x0c030c02u);
#pragma unroll
                for (int i = 0; i < 4; ++i) aB[i] = (int)((uint32_t)aA[i] << 8);
                const uint32_t c[4] = {r.c.x, r.c.y, r.c.z, r.c.w};
                const uint32_t d[4] = {r.d.x, r.d.y, r.d.z, r.d.w};
                // the products of dword p + 1 run beside the scaling of dword p
                v4i w = code_bytes<kSym>(c[0]);
                v4i pa = __builtin_amdgcn_mfma_i32_16x16x64_i8(aA, w, z, 0, 0, 0);
                v4i pb = __builtin_amdgcn_mfma_i32_16x16x64_i8(aB, w, z, 0, 0, 0);
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    v4i na, nb;
                    if (p < 3) {
                        w = code_bytes<kSym>(c[p + 1]);
                        na = __builtin_amdgcn_mfma_i32_16x16x64_i8(aA, w, z, 0, 0, 0);
                        nb = __builtin_amdgcn_mfma_i32_16x16x64_i8(aB, w, z, 0, 0, 0);
                    }
                    const float da = (float)__builtin_bit_cast(_Float16, (uint16_t)(d[p] & 0xffffu));
                    const float db = (float)__builtin_bit_cast(_Float16, (uint16_t)(d[p] >> 16));
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        acc[2 * p][i] = fma((double)((float)pa[i] * da), s[i], acc[2 * p][i]);
                        acc[2 * p + 1][i] = fma((double)((float)pb[i] * db), s[i], acc[2 * p + 1][i]);
                    }
                    if (p < 3) pa = na, pb = nb;
                    __builtin_amdgcn_sched_barrier(0);
                }
                // no block's work moves into another's: the ring is what is in
                // flight, and the registers hold one block's products
                load(b + j + kDepth, ring[j]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }
    // the waves' sums, halved three times: the upper half of the waves hands
    // its sums to the lower (a fixed order)
    double* red = (double*)lds;
#pragma unroll
    for (int half = kWavesD / 2; half >= 1; half /= 2) {
        __syncthreads();  // the activations, or the last round's sums, are read
        if (wave >= half && wave < 2 * half)
#pragma unroll
            for (int f = 0; f < 8; ++f)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    red[((wave - half) * R + kg + 4 * i) * 128 + f * 16 + r16] = acc[f][i];
        __syncthreads();
        if (wave < half)
#pragma unroll
            for (int f = 0; f < 8; ++f)
#pragma unroll
                for (int i = 0; i < NI; ++i) acc[f][i] += red[(wave * R + kg + 4 * i) * 128 + f * 16 + r16];
    }
    __syncthreads();
    constexpr double unit = kSym ? 0.5 : 1.0;  // the symmetric map's codes are 2 (q - 1.5)
    if (wave == 0)
#pragma unroll
        for (int f = 0; f < 8; ++f)
#pragma unroll
            for (int i = 0; i < NI; ++i) red[(kg + 4 * i) * 128 + f * 16 + r16] = unit * acc[f][i];
    __syncthreads();
}

// What the whole workgroup knows about its piece of work.
struct Piece {
    int e, row0, rows, slab, c;
    const int* tok;  // [rows] tokens (LDS)
};

// Gate/up of rows [r, r + rows) of a chunk: h = silu(G) U rounded to int8,
// half a wave per row and block of 32.
template <bool kSym, int NI>
__device__ void gate_up_pass(const DecodeArgs& g, const Piece& w, int r, int rows, char* lds) {
    const int nblk = g.H / kBlock;
    const uint8_t* rec = g.gate_up + (int64_t)w.e * g.gate_up_stride + (int64_t)w.slab * nblk * kRecordBytes;
    slab_pass<kSym, NI>(rec, g.H, lds, [&](uint8_t* qa, int2* sa, int tid) {
        for (int i = tid; i < rows * (g.H / 8); i += kThreads) {
            const int j = i / (g.H / 8), k = i % (g.H / 8);
            *reinterpret_cast<uint2*>(qa + j * act_stride(g.H) + 8 * k) =
                reinterpret_cast<const uint2*>(g.qx + (int64_t)w.tok[r + j] * g.H)[k];
        }
        for (int i = tid; i < rows * nblk; i += kThreads) {
            const int j = i / nblk, k = i % nblk;
            sa[k * 4 * NI + j] = g.sx[(int64_t)w.tok[r + j] * nblk + k];
        }
    });
    const double* tot = (const double*)lds;
    const int tid = pass_thread();
    const int half = tid >> 5, l = tid & 31;
    for (int i = half; i < 2 * rows; i += kThreads / 32) {
        const int j = i >> 1, col = (i & 1) * 32 + l;
        const double gt = tot[j * 128 + col], up = tot[j * 128 + 64 + col];
        const float h = (float)(gt / (1.0 + exp(-gt)) * up);
        float m = fabsf(h);
        for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 32));
        const float s = m / 127.0f;
        const int q = s != 0.0f ? (int)round_half_away(h / s) : 0;
        int sum = q;
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor(sum, o, 32);
        uint32_t word = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) word |= (uint32_t)(__shfl(q, (l & 7) * 4 + k, 32) & 0xff) << (8 * k);
        const int64_t row = w.row0 + r + j;
        if (l < 8) poke(reinterpret_cast<uint32_t*>(g.qh + row * g.I + 64 * w.slab + 32 * (i & 1)) + l, word);
        if (l == 8)
            poke(reinterpret_cast<uint64_t*>(g.sh + row * (g.I / kBlock) + 2 * w.slab + (i & 1)),
                 (uint64_t)__builtin_bit_cast(uint32_t, s) | (uint64_t)(uint32_t)sum << 32);
    }
}

// Down of rows [r, r + rows): the weighted rows, and for every token whose
// last row this is the sum of its rows, k ascending.
template <bool kSym, int NI>
__device__ void down_pass(const DecodeArgs& g, const Piece& w, int r, int rows, char* lds, int* flags) {
    const int nblk = g.I / kBlock, nslab = g.H / kSlabRows;
    const uint8_t* rec = g.down + (int64_t)w.e * g.down_stride + (int64_t)w.slab * nblk * kRecordBytes;
    slab_pass<kSym, NI>(rec, g.I, lds, [&](uint8_t* qa, int2* sa, int tid) {
        if (r == 0) {  // the chunk's H rows are finished
            if (tid == 0)
                for (int n = 0; n < kMaxPolls && peek(&g.gu_done[w.c]) < g.I / 64; ++n) __builtin_amdgcn_s_sleep(1);
            __syncthreads();
        }
        for (int i = tid; i < rows * (g.I / 8); i += kThreads) {
            const int j = i / (g.I / 8), k = i % (g.I / 8);
            *reinterpret_cast<uint64_t*>(qa + j * act_stride(g.I) + 8 * k) =
                peek(reinterpret_cast<const uint64_t*>(g.qh + (int64_t)(w.row0 + r + j) * g.I) + k);
        }
        for (int i = tid; i < rows * nblk; i += kThreads) {
            const int j = i / nblk, k = i % nblk;
            reinterpret_cast<uint64_t*>(sa)[k * 4 * NI + j] =
                peek(reinterpret_cast<const uint64_t*>(g.sh + (int64_t)(w.row0 + r + j) * nblk) + k);
        }
    });
    const double* tot = (const double*)lds;
    const int tid = pass_thread();
    for (int i = tid; i < rows * 128; i += kThreads) {
        const int pair = peek(&g.row_pair[w.row0 + r + i / 128]);
        poke(&g.dm[(int64_t)pair * g.H + 128 * w.slab + i % 128], (float)((double)peek(&g.p[pair]) * tot[i]));
    }
    publish();
    if (tid < rows)
        flags[tid] = bump(&g.dn_done[w.tok[r + tid] * nslab + w.slab]) == g.Kg - 1;
    __syncthreads();
    for (int i = tid; i < rows * 128; i += kThreads) {
        if (!flags[i / 128]) continue;
        const int64_t t = w.tok[r + i / 128];
        const int col = 128 * w.slab + i % 128;
        double s = 0.0;
        for (int k = 0; k < g.Kg; ++k) s += (double)peek(&g.dm[(t * g.Kg + k) * g.H + col]);
        g.out[t * g.H + col] = (float)s;
    }
    __syncthreads();
}

template <bool kSym, bool kWide>
__device__ void expert_piece(const DecodeArgs& g, const Piece& w, bool gate_up, char* lds, int* flags) {
    for (int r = 0; r < w.rows; r += kPassRows) {
        const int rows = w.rows - r < kPassRows ? w.rows - r : kPassRows;
        if (gate_up) {
            if (kWide && rows > 4)
                gate_up_pass<kSym, 2>(g, w, r, rows, lds);
            else
                gate_up_pass<kSym, 1>(g, w, r, rows, lds);
            __syncthreads();
        } else {
            if (kWide && rows > 4)
                down_pass<kSym, 2>(g, w, r, rows, lds, flags);
            else
                down_pass<kSym, 1>(g, w, r, rows, lds, flags);
        }
    }
}

// Everything after the router in one launch.  Workgroup id -> chunk is fixed
// (chunk_of); what the workgroup does for its chunk is the next slab in the
// order gate/up 0 .. I/64 - 1, down 0 .. H/128 - 1, by the chunk's ticket.  A
// workgroup that waits for the H rows of its chunk thus knows that their
// slabs are all in the hands of workgroups that run, and those wait for
// nothing but the top-K, which any waiting workgroup takes on itself while
// there are tokens left: every wait ends whatever order the workgroups start
// in and whatever else runs on the GPU.
__device__ int chunk_of(const DecodeArgs& g, int id) {
    const int gu = g.I / 64, dn = g.H / kSlabRows;
    // gate/up runs `lag` chunks ahead of down, more than run at once
    int lag = kResident / gu + 1;
    if (lag > g.cap) lag = g.cap;
    if (id < lag * gu) return id / gu;
    id -= lag * gu;
    const int whole = (g.cap - lag) * (gu + dn);
    if (id < whole) return id % (gu + dn) < gu ? lag + id / (gu + dn) : id / (gu + dn);
    return g.cap - lag + (id - whole) / dn;
}

template <bool kSym, bool kWide>
__global__ void __launch_bounds__(kThreads, 4) decode_experts_kernel(DecodeArgs g) {
    extern __shared__ double lds[];
    __shared__ int todo[4];      // what thread 0 found
    __shared__ uint64_t chunk[2];
    __shared__ int tok[kDecodeMaxTokens];
    __shared__ int flags[kPassRows];
    const int c = chunk_of(g, blockIdx.x);
    int ticket = 0;
    if (threadIdx.x == 0) ticket = bump(&g.ticket[c]);
    for (;;) {
        if (threadIdx.x == 0) {
            int what = 3;  // give up
            for (int n = 0; n < kMaxPolls; ++n) {
                const uint64_t head = peek(&g.chunks[c].head), mask = peek(&g.chunks[c].mask);
                const int nch = peek(g.nchunks);
                if (nch > 0 && c >= nch - 1) break;
                if (nch > 0 && head != 0 && mask != 0) {
                    chunk[0] = head, chunk[1] = mask;
                    what = 0;
                    break;
                }
                if (nch == 0 && peek(g.topk_next) < g.T) {
                    const int t = bump(g.topk_next);
                    if (t < g.T) {
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
        const int what = todo[0];
        if (what == 3) return;
        if (what == 0) break;
        topk_token(g, todo[1], *(TopkLds*)lds);
        publish();
        if (threadIdx.x == 0) todo[2] = bump(g.topk_done) == g.T - 1;
        __syncthreads();
        if (todo[2]) group_pairs(g, *(GroupLds*)lds);
        __syncthreads();
    }
    if (threadIdx.x == 0) todo[3] = ticket;
    if (threadIdx.x < 64) {
        const uint64_t mask = chunk[1];
        if (mask >> threadIdx.x & 1) tok[__popcll(mask & ((1ull << threadIdx.x) - 1))] = threadIdx.x;
    }
    __syncthreads();
    const int gu = g.I / 64;
    const int tk = __builtin_amdgcn_readfirstlane(todo[3]);
    Piece w;
    w.e = __builtin_amdgcn_readfirstlane((int)(chunk[0] >> 32));
    w.row0 = __builtin_amdgcn_readfirstlane((int)(chunk[0] >> 16 & 0xffff));
    w.rows = __builtin_amdgcn_readfirstlane((int)(chunk[0] & 0xffff));
    w.c = c;
    w.tok = tok;
    w.slab = tk < gu ? tk : tk - gu;
    expert_piece<kSym, kWide>(g, w, tk < gu, (char*)lds, flags);
    if (tk < gu) {
        publish();
        if (threadIdx.x == 0) bump(&g.gu_done[c]);
    }
}

// The workspace of one call.
struct Plan {
    size_t part, qx, sx, ids, p, row_pair, qh, sh, dm, words, ticket, gu_done, dn_done, chunks, total;
};

Plan plan(int32_t T, int32_t H, int32_t E, int32_t K, int32_t I, bool shared) {
    const int64_t Eg = E + shared, n = (int64_t)T * (K + shared), cap = n < Eg ? n : Eg;
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
    o.ticket = take(cap * 4);
    o.gu_done = take(cap * 4);
    o.dn_done = take((int64_t)T * (H / kSlabRows) * 4);
    o.chunks = take(cap * 16);
    o.total = off;
    return o;
}

// LDS of a pass of up to `rows` rows: the activations (codes, and 8 bytes a
// block), then half the waves' sums of 4 NI rows in the same place.
size_t pass_lds(int Kd, int rows) {
    const size_t R = rows <= 4 ? 4 : kPassRows;
    const size_t act = R * (Kd + 8) + R * (Kd / kBlock) * 8, sums = (size_t)(kWavesD / 2) * R * 128 * 8;
    return act > sums ? act : sums;
}

template <int TT>
hipError_t launch_router_tt(const DecodeArgs& g, hipStream_t st) {
    const int groups = (g.Eg + 63) / 64, tg = (g.T + TT - 1) / TT;
    const size_t lds = ((size_t)(g.H / kRouterSlices) * TT + (size_t)kWavesD * TT * 64) * 8;
    hipLaunchKernelGGL(decode_router_kernel<TT>, dim3(groups * kRouterSlices * tg + g.T), dim3(kThreads), lds, st, g);
    return hipGetLastError();
}

}  // namespace

size_t decode_workspace(int32_t T, int32_t H, int32_t E, int32_t K, int32_t I, bool shared) {
    return plan(T, H, E, K, I, shared).total;
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
    g.cap = g.n < g.Eg ? g.n : g.Eg;
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
    g.ticket = (int32_t*)(ws + o.ticket);
    g.gu_done = (int32_t*)(ws + o.gu_done);
    g.dn_done = (int32_t*)(ws + o.dn_done);
    g.chunks = (Chunk*)(ws + o.chunks);
    hipError_t e = g.T == 1 ? launch_router_tt<1>(g, st) : g.T <= 4 ? launch_router_tt<4>(g, st) : launch_router_tt<8>(g, st);
    if (e != hipSuccess) return e;
    // a chunk has at most T rows
    size_t lds = sizeof(TopkLds) > sizeof(GroupLds) ? sizeof(TopkLds) : sizeof(GroupLds);
    for (const size_t need : {pass_lds(g.H, g.T), pass_lds(g.I, g.T)})
        if (need > lds) lds = need;
    const dim3 grid(g.cap * (g.I / 64 + g.H / kSlabRows));
    void (*kernel)(DecodeArgs);
    if (g.T <= 4)  // every pass is a narrow one
        kernel = l.sym ? decode_experts_kernel<true, false> : decode_experts_kernel<false, false>;
    else
        kernel = l.sym ? decode_experts_kernel<true, true> : decode_experts_kernel<false, true>;
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), lds, st, g);
    return hipGetLastError();
}

}  // namespace strata_moe
