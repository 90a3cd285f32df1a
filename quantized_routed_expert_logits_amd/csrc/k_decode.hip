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
constexpr int kDepth = 4;          // blocks in flight per wave

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
    int32_t Kg, Eg;      // pairs per token, experts (with the shared one)
    int32_t n;           // T * Kg
    float* out;
    double* part;        // [slices][T][Eg] partial logits (column E: the shared gate's dot product)
    int8_t* qx;          // [T][H]
    float* sx;           // [T][H / 32]
    int32_t* ids;        // [T][Kg]
    float* p;            // [T][Kg]
    int4* chunks;        // [min(n, Eg)]: expert, first row, rows
    int32_t* nchunks;
    int32_t* row_token;  // [n]
    int32_t* row_pair;   // [n]
    int8_t* qh;          // [n][I]
    float* sh;           // [n][I / 32]
    float* dm;           // [n][H] weighted rows, by pair
};

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
        reinterpret_cast<uint32_t*>(g.qx + (int64_t)t * g.H)[i] = q;
        if ((threadIdx.x & 7) == 0) g.sx[(int64_t)t * (g.H / kBlock) + i / 8] = s;
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
    else
        quantize_token(g, id - nr);
}

// ------------------------------------------------------------ top-K, softmax
// One workgroup per token.  Each wave ranks 64 logits at a time by counting
// the larger ones (ties: the lower index first), the best K of every 64 are
// ranked again.  A NaN ranks as -inf, so the ids are always K different ones.
__device__ void topk_token(const DecodeArgs& g, int t, double* lds) {
    double* cv = lds;                    // [16 * 16] candidates
    int* ce = (int*)(lds + 256);
    double* sv = lds + 512;              // [16] selected
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int nch = (g.E + 63) / 64;
    const double ninf = -__builtin_huge_val();
    for (int c = wave; c < nch; c += kWavesD) {
        const int e = c * 64 + lane;
        double v = ninf;
        if (e < g.E) {
            v = 0.0;
            for (int s = 0; s < kRouterSlices; ++s) v += g.part[((int64_t)s * g.T + t) * g.Eg + e];
            if (g.bias) v += (double)g.bias[e];
            if (!(v == v)) v = ninf;
        }
        int rank = 0;
        const uint64_t bits = __builtin_bit_cast(uint64_t, v);
        for (int j = 0; j < 64; ++j) {
            const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)bits, j);
            const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(bits >> 32), j);
            const double o = __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
            rank += (o > v || (o == v && j < lane)) ? 1 : 0;
        }
        if (rank < g.K) cv[c * g.K + rank] = v, ce[c * g.K + rank] = e;
    }
    __syncthreads();
    const int nc = nch * g.K;
    if ((int)threadIdx.x < nc) {
        const double v = cv[threadIdx.x];
        const int e = ce[threadIdx.x];
        int rank = 0;
        for (int j = 0; j < nc; ++j) rank += (cv[j] > v || (cv[j] == v && ce[j] < e)) ? 1 : 0;
        if (rank < g.K) {
            sv[rank] = v;
            g.ids[t * g.Kg + rank] = e;
        }
    }
    __syncthreads();
    if ((int)threadIdx.x < g.K) {
        double z = 0.0;
        for (int k = 0; k < g.K; ++k) z += exp(sv[k] - sv[0]);
        g.p[t * g.Kg + threadIdx.x] = (float)(exp(sv[threadIdx.x] - sv[0]) / z);
    }
    if (g.shared && threadIdx.x == 64) {
        double v = 0.0;
        for (int s = 0; s < kRouterSlices; ++s) v += g.part[((int64_t)s * g.T + t) * g.Eg + g.E];
        g.ids[t * g.Kg + g.K] = g.E;
        g.p[t * g.Kg + g.K] = (float)(1.0 / (1.0 + exp(-v)));
    }
}

__global__ void __launch_bounds__(kThreads) decode_topk_kernel(DecodeArgs g) {
    __shared__ double lds[544];
    topk_token(g, blockIdx.x, lds);
}

// ---------------------------------------------------------------- grouping
// The pairs by expert, ascending token inside an expert.  A token picks an
// expert at most once, so an expert's rows are the set bits of a 64-bit mask
// of tokens and a pair's row is a population count.
__device__ void group_pairs(const DecodeArgs& g, uint64_t* mask, int* row0, int* wsum) {
    for (int e = threadIdx.x; e < kMaxExperts; e += kThreads) mask[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < g.n; i += kThreads)
        atomicOr((unsigned long long*)&mask[g.ids[i]], 1ull << (i / g.Kg));
    __syncthreads();
    // exclusive scan of (rows, hit experts) over the experts, packed in one
    // int: two experts a thread
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int e0 = 2 * threadIdx.x;
    const int c0 = __popcll(mask[e0]), c1 = __popcll(mask[e0 + 1]);
    const int mine = (c0 | (c0 > 0 ? 1 << 16 : 0)) + (c1 | (c1 > 0 ? 1 << 16 : 0));
    int s = mine;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(s, o);
        if (lane >= o) s += v;
    }
    if (lane == 63) wsum[wave] = s;
    __syncthreads();
    int at = s - mine;
    for (int w = 0; w < wave; ++w) at += wsum[w];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = e0 + j, c = j ? c1 : c0;
        row0[e] = at & 0xffff;
        if (c > 0) {
            g.chunks[at >> 16] = make_int4(e, at & 0xffff, c, 0);
            at += c | (1 << 16);
        }
    }
    if (threadIdx.x == kThreads - 1) *g.nchunks = at >> 16;
    __syncthreads();
    for (int i = threadIdx.x; i < g.n; i += kThreads) {
        const int e = g.ids[i], t = i / g.Kg;
        const int row = row0[e] + __popcll(mask[e] & ((1ull << t) - 1));
        g.row_token[row] = t;
        g.row_pair[row] = i;
    }
}

__global__ void __launch_bounds__(kThreads) decode_group_kernel(DecodeArgs g) {
    __shared__ uint64_t mask[kMaxExperts];
    __shared__ int row0[kMaxExperts];
    __shared__ int wsum[kWavesD];
    group_pairs(g, mask, row0, wsum);
}

// ----------------------------------------------------------------- experts
// One record dword -> its two rows' codes as int8 (the packing of k_pack.hip;
// q, or 2q for the symmetric map): lo / hi[0] = row A k 0..3 / 4..7, [1] = B.
template <bool kSym>
__device__ __forceinline__ void row_codes(uint32_t w, uint32_t (&lo)[2], uint32_t (&hi)[2]) {
    uint32_t x[4];
    if constexpr (kSym) {
        x[0] = (w << 1) & 0x06060606u;
#pragma unroll
        for (int j = 1; j < 4; ++j) x[j] = (w >> (2 * j - 1)) & 0x06060606u;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = (w >> (2 * j)) & 0x03030303u;
    }
    lo[0] = __builtin_amdgcn_perm(x[1], x[0], 0x06040200u);
    hi[0] = __builtin_amdgcn_perm(x[3], x[2], 0x06040200u);
    lo[1] = __builtin_amdgcn_perm(x[1], x[0], 0x07050301u);
    hi[1] = __builtin_amdgcn_perm(x[3], x[2], 0x07050301u);
}

struct Block {
    uint4 c, d;  // a lane's 16 code bytes, its row's 8 fp16 scales
};

// R rows of one slab (128 outputs): lds gets tot[R][128], the outputs of the
// slab in fragment order f * 16 + r, valid after the call for every thread.
// act(i) / scl(i): the int8 codes and block scales of row i.
template <bool kSym, int R, typename Act, typename Scl>
__device__ void slab_rows(const uint8_t* rec0, int nblk, Act act, Scl scl, char* lds, double*& tot) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
    double* red = (double*)lds;                                   // [waves][R][128]
    uint32_t* qa = (uint32_t*)(lds + kWavesD * R * 128 * 8);      // [R][nblk * 8] code dwords
    float* sa = (float*)(qa + R * nblk * 8);                      // [R][nblk]
    __syncthreads();  // lds may hold the last pass's results
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(act(i));
        const float* s = scl(i);
        for (int j = threadIdx.x; j < nblk * 8; j += kThreads) qa[i * nblk * 8 + j] = q[j];
        for (int j = threadIdx.x; j < nblk; j += kThreads) sa[i * nblk + j] = s[j];
    }
    __syncthreads();
    constexpr int zp = kSym ? 3 : 1;
    double acc[8][R];
#pragma unroll
    for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int i = 0; i < R; ++i) acc[f][i] = 0.0;
    for (int b = 0; b < nb; b += kDepth) {
#pragma unroll
        for (int j = 0; j < kDepth; ++j) {
            if (b + j < nb) {
                const Block r = ring[j];
                const int blk = b0 + b + j;
                int a0[R], a1[R], z[R];
                double s[R];
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const uint2 av = *reinterpret_cast<const uint2*>(&qa[(i * nblk + blk) * 8 + 2 * kg]);
                    a0[i] = (int)av.x, a1[i] = (int)av.y;
                    s[i] = (double)sa[i * nblk + blk];
                    z[i] = -zp * __builtin_amdgcn_sdot4(a1[i], 0x01010101,
                                                        __builtin_amdgcn_sdot4(a0[i], 0x01010101, 0, false), false);
                }
                const uint32_t c[4] = {r.c.x, r.c.y, r.c.z, r.c.w};
                const uint32_t d[4] = {r.d.x, r.d.y, r.d.z, r.d.w};
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    uint32_t lo[2], hi[2];
                    row_codes<kSym>(c[p], lo, hi);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float dv = (float)__builtin_bit_cast(_Float16, (uint16_t)(d[p] >> (16 * h)));
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            int v = __builtin_amdgcn_sdot4((int)lo[h], a0[i], z[i], false);
                            v = __builtin_amdgcn_sdot4((int)hi[h], a1[i], v, false);
                            acc[2 * p + h][i] = fma((double)((float)v * dv), s[i], acc[2 * p + h][i]);
                        }
                    }
                }
                load(b + j + kDepth, ring[j]);
            }
        }
    }
    constexpr double half = kSym ? 0.5 : 1.0;  // the symmetric map's codes are 2 (q - 1.5)
#pragma unroll
    for (int f = 0; f < 8; ++f)
#pragma unroll
        for (int i = 0; i < R; ++i) {
            double v = acc[f][i];
            v += __shfl_xor(v, 16);
            v += __shfl_xor(v, 32);
            if (kg == 0) red[(wave * R + i) * 128 + f * 16 + r16] = v * half;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < R * 128; i += kThreads) {
        double v = 0.0;
        for (int w = 0; w < kWavesD; ++w) v += red[w * R * 128 + i];
        red[i] = v;  // its own element of the first wave's part
    }
    __syncthreads();
    tot = red;
}

// h = silu(G) U and its int8 rounding: a thread per H value, 32 lanes a block.
template <int R>
__device__ __forceinline__ void store_h(const DecodeArgs& g, const double* tot, int row0, int slab) {
    const int i = threadIdx.x >> 6, j = threadIdx.x & 63;  // row, H column in the slab
    if (i >= R) return;
    const double gt = tot[i * 128 + j], up = tot[i * 128 + 64 + j];
    const float h = (float)(gt / (1.0 + exp(-gt)) * up);
    float m = fabsf(h);
    for (int o = 1; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
    const float s = m / 127.0f;
    const int64_t row = row0 + i;
    g.qh[row * g.I + 64 * slab + j] = (int8_t)(s != 0.0f ? (int)round_half_away(h / s) : 0);
    if ((j & 31) == 0) g.sh[row * (g.I / kBlock) + 2 * slab + j / 32] = s;
}

template <bool kSym, int R>
__device__ void gate_up_rows(const DecodeArgs& g, const int4& ch, int slab, int r, char* lds) {
    const int nblk = g.H / kBlock;
    const uint8_t* rec = g.gate_up + (int64_t)ch.x * g.gate_up_stride + (int64_t)slab * nblk * kRecordBytes;
    double* tot;
    slab_rows<kSym, R>(
        rec, nblk, [&](int i) { return g.qx + (int64_t)g.row_token[ch.y + r + i] * g.H; },
        [&](int i) { return g.sx + (int64_t)g.row_token[ch.y + r + i] * nblk; }, lds, tot);
    store_h<R>(g, tot, ch.y + r, slab);
}

template <bool kSym, int R>
__device__ void down_rows(const DecodeArgs& g, const int4& ch, int slab, int r, char* lds) {
    const int nblk = g.I / kBlock;
    const uint8_t* rec = g.down + (int64_t)ch.x * g.down_stride + (int64_t)slab * nblk * kRecordBytes;
    double* tot;
    slab_rows<kSym, R>(
        rec, nblk, [&](int i) { return g.qh + (int64_t)(ch.y + r + i) * g.I; },
        [&](int i) { return g.sh + (int64_t)(ch.y + r + i) * nblk; }, lds, tot);
    for (int i = threadIdx.x; i < R * 128; i += kThreads) {
        const int pair = g.row_pair[ch.y + r + i / 128];
        g.dm[(int64_t)pair * g.H + 128 * slab + i % 128] = (float)((double)g.p[pair] * tot[i]);
    }
}

template <bool kSym>
__global__ void __launch_bounds__(kThreads) decode_gate_up_kernel(DecodeArgs g) {
    extern __shared__ double lds[];
    const int nslab = g.I / 64;
    const int c = blockIdx.x / nslab, slab = blockIdx.x % nslab;
    if (c >= *g.nchunks) return;
    const int4 ch = g.chunks[c];
    int r = 0;
    for (; r + 2 <= ch.z; r += 2) gate_up_rows<kSym, 2>(g, ch, slab, r, (char*)lds);
    if (r < ch.z) gate_up_rows<kSym, 1>(g, ch, slab, r, (char*)lds);
}

template <bool kSym>
__global__ void __launch_bounds__(kThreads) decode_down_kernel(DecodeArgs g) {
    extern __shared__ double lds[];
    const int nslab = g.H / kSlabRows;
    const int c = blockIdx.x / nslab, slab = blockIdx.x % nslab;
    if (c >= *g.nchunks) return;
    const int4 ch = g.chunks[c];
    int r = 0;
    for (; r + 2 <= ch.z; r += 2) down_rows<kSym, 2>(g, ch, slab, r, (char*)lds);
    if (r < ch.z) down_rows<kSym, 1>(g, ch, slab, r, (char*)lds);
}

// out[t] = the sum of its Kg weighted rows, k ascending.
__global__ void __launch_bounds__(256) decode_combine_kernel(DecodeArgs g) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= (int64_t)g.T * g.H) return;
    const int64_t t = i / g.H, o = i % g.H;
    float s = 0.f;
    for (int k = 0; k < g.Kg; ++k) s += g.dm[(t * g.Kg + k) * g.H + o];
    g.out[i] = s;
}

// The workspace of one call.
struct Plan {
    size_t part, qx, sx, ids, p, chunks, nchunks, row_token, row_pair, qh, sh, dm, total;
};

Plan plan(int32_t T, int32_t H, int32_t E, int32_t K, int32_t I, bool shared) {
    const int64_t Eg = E + shared, n = (int64_t)T * (K + shared);
    size_t off = 0;
    auto take = [&](int64_t bytes) {
        const size_t at = off;
        off += (size_t)round_up(bytes > 0 ? bytes : 1, 256);
        return at;
    };
    Plan o;
    o.part = take((int64_t)kRouterSlices * T * Eg * 8);
    o.qx = take((int64_t)T * H);
    o.sx = take((int64_t)T * (H / kBlock) * 4);
    o.ids = take(n * 4);
    o.p = take(n * 4);
    o.chunks = take((n < Eg ? n : Eg) * 16);
    o.nchunks = take(4);
    o.row_token = take(n * 4);
    o.row_pair = take(n * 4);
    o.qh = take(n * I);
    o.sh = take(n * (I / kBlock) * 4);
    o.dm = take(n * H * 4);
    o.total = off;
    return o;
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
    g.part = (double*)(ws + o.part);
    g.qx = (int8_t*)(ws + o.qx);
    g.sx = (float*)(ws + o.sx);
    g.ids = (int32_t*)(ws + o.ids);
    g.p = (float*)(ws + o.p);
    g.chunks = (int4*)(ws + o.chunks);
    g.nchunks = (int32_t*)(ws + o.nchunks);
    g.row_token = (int32_t*)(ws + o.row_token);
    g.row_pair = (int32_t*)(ws + o.row_pair);
    g.qh = (int8_t*)(ws + o.qh);
    g.sh = (float*)(ws + o.sh);
    g.dm = (float*)(ws + o.dm);
    hipError_t e = g.T == 1 ? launch_router_tt<1>(g, st) : g.T <= 4 ? launch_router_tt<4>(g, st) : launch_router_tt<8>(g, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(decode_topk_kernel, dim3(g.T), dim3(kThreads), 0, st, g);
    hipLaunchKernelGGL(decode_group_kernel, dim3(1), dim3(kThreads), 0, st, g);
    const int cap = g.n < g.Eg ? g.n : g.Eg;
    auto lds = [&](int nblk) { return (size_t)kWavesD * 2 * 128 * 8 + 2 * (size_t)nblk * 36; };
    const dim3 gu(cap * (g.I / 64)), dn(cap * (g.H / kSlabRows));
    if (l.sym) {
        hipLaunchKernelGGL(decode_gate_up_kernel<true>, gu, dim3(kThreads), lds(g.H / kBlock), st, g);
        hipLaunchKernelGGL(decode_down_kernel<true>, dn, dim3(kThreads), lds(g.I / kBlock), st, g);
    } else {
        hipLaunchKernelGGL(decode_gate_up_kernel<false>, gu, dim3(kThreads), lds(g.H / kBlock), st, g);
        hipLaunchKernelGGL(decode_down_kernel<false>, dn, dim3(kThreads), lds(g.I / kBlock), st, g);
    }
    hipLaunchKernelGGL(decode_combine_kernel, dim3((unsigned)(((int64_t)g.T * g.H + 255) / 256)), dim3(256), 0, st, g);
    return hipGetLastError();
}

}  // namespace strata_moe
