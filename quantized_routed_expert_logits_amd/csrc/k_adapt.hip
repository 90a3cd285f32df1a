// Low-rank adapters of many requests beside a projection they share: token t
// of the call carries adapter a = ids[t] and
//   out[t] = y[t] + scale_a B_a (A_a x[t]),   A_a [r_a][in], B_a [out][r_a],
// and out[t] = y[t] where ids[t] is not an adapter.  Two launches: the shrink
// v[t] = A_a x[t] into the workspace, then the expand.
#include <hip/hip_bf16.h>

#include "internal.h"

namespace strata_moe {

namespace {

struct AdaptArgs {
    const float* x;
    const float* y;
    float* out;
    const int32_t* ids;
    const void* a;
    const void* b;
    const float* scale;    // or null: 1
    const int32_t* ranks;  // or null: rank
    float* v;              // [T][rank]
    int64_t T, xs, ys, os;
    int32_t L, rank, in, out_dim;
};

__device__ __forceinline__ float widen(float w) { return w; }
__device__ __forceinline__ float widen(_Float16 w) { return (float)w; }
__device__ __forceinline__ float widen(__bf16 w) { return (float)w; }

__device__ __forceinline__ int adapter_rank(const AdaptArgs& g, int a) {
    if (!g.ranks) return g.rank;
    const int r = g.ranks[a];
    return r < 0 ? 0 : (r > g.rank ? g.rank : r);
}

// One wave per (token, row of A).
template <typename W>
__global__ void __launch_bounds__(256) adapt_shrink_kernel(AdaptArgs g) {
    const int64_t t = blockIdx.x;
    const int a = g.ids[t];
    if (a < 0 || a >= g.L) return;
    const int lane = threadIdx.x & 63;
    const int R = adapter_rank(g, a);
    const float* x = g.x + t * g.xs;
    for (int r = threadIdx.x >> 6; r < R; r += blockDim.x >> 6) {
        const W* w = (const W*)g.a + ((int64_t)a * g.rank + r) * g.in;
        float s = 0.f;
        for (int h = lane; h < g.in; h += 64) s = fmaf(widen(w[h]), x[h], s);
        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
        if (lane == 0) g.v[t * g.rank + r] = s;
    }
}

// One thread per output.
template <typename W>
__global__ void __launch_bounds__(256) adapt_expand_kernel(AdaptArgs g) {
    const int64_t t = blockIdx.x;
    const int o = blockIdx.y * 256 + threadIdx.x;
    if (o >= g.out_dim) return;
    const int a = g.ids[t];
    float acc = g.y[t * g.ys + o];
    if (a >= 0 && a < g.L) {
        const int R = adapter_rank(g, a);
        const W* w = (const W*)g.b + ((int64_t)a * g.out_dim + o) * g.rank;
        float s = 0.f;
        for (int r = 0; r < R; ++r) s = fmaf(widen(w[r]), g.v[t * g.rank + r], s);
        acc = fmaf(g.scale ? g.scale[a] : 1.0f, s, acc);
    }
    g.out[t * g.os + o] = acc;
}

template <typename W>
hipError_t launch_typed(const AdaptArgs& g, hipStream_t st) {
    hipLaunchKernelGGL(adapt_shrink_kernel<W>, dim3((unsigned)g.T), dim3(256), 0, st, g);
    const dim3 grid((unsigned)g.T, (unsigned)((g.out_dim + 255) / 256));
    hipLaunchKernelGGL(adapt_expand_kernel<W>, grid, dim3(256), 0, st, g);
    return hipGetLastError();
}

}  // namespace

size_t adapt_workspace(int64_t T, int32_t rank) { return (size_t)round_up(T * rank * 4, 256); }

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
    switch (l.dtype) {
        case kAdapterF32: return launch_typed<float>(g, st);
        case kAdapterF16: return launch_typed<_Float16>(g, st);
        default: return launch_typed<__bf16>(g, st);
    }
}

}  // namespace strata_moe
