// Norms before and after a block, with the residual stream between them.  Per
// token t, with h the stream, y the block's output rows and u_j = (offset + w_j):
//   v = sum_k p[t][k] y[slot[t][k]]          (or v = y[t])
//   b = u v / sqrt(mean(v^2) + eps)          (or b = v)
//   h' = residual_scale h + block_scale gate b, rounded to the stream's type
//   x = u' h' / sqrt(mean(h'^2) + eps'), and x rounded to 4 bits per 32 values
// A call has the part up to h', the part from h' (h' = h then), or both.
//
// One workgroup per token; its row stays in registers between the sums, so
// every array is read or written once.  A thread holds runs of 4 neighbouring
// columns, so 8 neighbouring threads hold the 32 columns of one 4-bit block.
// All arithmetic is in 64 bits and an output is rounded to fp32, and from there
// to 16 bits: the stored stream and the 4-bit codes are those of the exact row
// except where it lies within about 2^-50 of a border.  The memory bounds these
// kernels, so the wider arithmetic is free.
#include "block.h"
#include "mxfp.h"

namespace strata_moe {
namespace {

constexpr int kMaxThreads = 1024;

struct NormArgs {
    NormLaunch l;
    int32_t vec_h, vec_y, vec_out, vec_x, vec_gate, vec_w, vec_u;  // rows of this array take 4-wide accesses
};

// 4 columns from j on (columns at and past H: 0).
template <typename T>
__device__ __forceinline__ void load4(const T* row, int j, int H, bool vec, double* v) {
    if (vec && j + 4 <= H) {
        float f[4];
        load4_vec(row + j, f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = f[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = j + i < H ? (double)widen(row[j + i]) : 0.0;
}

__device__ __forceinline__ void load4_any(const void* base, int dtype, int64_t at, int j, int H, bool vec, double* v) {
    if (dtype == kF32) load4((const float*)base + at, j, H, vec, v);
    else if (dtype == kF16) load4((const _Float16*)base + at, j, H, vec, v);
    else load4((const __bf16*)base + at, j, H, vec, v);
}

// The sum over the workgroup, in a fixed order, in every thread.  red: one
// double per wave, not used by an earlier sum of the same kernel.
__device__ __forceinline__ double block_sum(double s, double* red) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
    const int waves = blockDim.x / 64;
    if (waves == 1) return s;
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = s;
    __syncthreads();
    s = 0.0;
    for (int w = 0; w < waves; ++w) s += red[w];
    return s;
}

template <int NC>
__device__ __forceinline__ void apply_norm(double (*v)[4], const NormScale& n, bool vec, int H, double* red) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fma(v[c][i], v[c][i], s);
    s = block_sum(s, red);
    const double r = 1.0 / sqrt(s / H + n.eps);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        double w[4] = {1.0, 1.0, 1.0, 1.0};
        const int j = (c * blockDim.x + threadIdx.x) * 4;
        if (n.weight) {
            load4(n.weight, j, H, vec, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] += n.offset;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[c][i] = v[c][i] * r * w[i];
    }
}

template <int NC>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(NormArgs a) {
    __shared__ double red[2][kMaxThreads / 64];
    const NormLaunch& l = a.l;
    const int H = l.H;
    const int64_t t = blockIdx.x;
    double v[NC][4], h[NC][4];
    if (l.y) {
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[c][i] = 0.0;
        if (l.slot) {
            for (int k = 0; k < l.K; ++k) {
                const int row = l.slot[t * l.K + k];
                if (row < 0 || row >= l.y_rows) continue;
                const double p = l.p[t * l.K + k];
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    double y[4];
                    load4_any(l.y, l.y_dtype, row * l.y_stride, (c * blockDim.x + threadIdx.x) * 4, H, a.vec_y, y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[c][i] = fma(p, y[i], v[c][i]);
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < NC; ++c)
                load4_any(l.y, l.y_dtype, t * l.y_stride, (c * blockDim.x + threadIdx.x) * 4, H, a.vec_y, v[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
        load4_any(l.h, l.dtype, t * l.h_stride, (c * blockDim.x + threadIdx.x) * 4, H, a.vec_h, h[c]);
    if (l.y) {
        if (l.after.on) apply_norm<NC>(v, l.after, a.vec_w, H, red[0]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const int j = (c * blockDim.x + threadIdx.x) * 4;
            double g[4] = {1.0, 1.0, 1.0, 1.0};
            if (l.gate) {
                const float* gr = l.gate + t * l.gate_row_stride;
                if (l.gate_col_stride) load4(gr, j, H, a.vec_gate, g);
                else g[0] = g[1] = g[2] = g[3] = *gr;
            }
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                h[c][i] = round_to(fma(l.residual_scale, h[c][i], l.block_scale * (g[i] * v[c][i])), l.dtype, &o[i]);
            store4_any(l.out, l.dtype, t * l.out_stride, j, H, a.vec_out, o);
        }
    }
    if (!l.before.on) return;
    apply_norm<NC>(h, l.before, a.vec_u, H, red[1]);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int j = (c * blockDim.x + threadIdx.x) * 4;
        float o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = (float)h[c][i];
        if (l.x) store4_any(l.x, kF32, t * H, j, H, a.vec_x, o);
        if (l.codes) {  // H is a multiple of 32, so a block's 8 threads are all inside or all outside
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = max(top, __float_as_uint(o[i]) & 0x7fffffffu);
            top = max(top, (uint32_t)__shfl_xor((int)top, 1));
            top = max(top, (uint32_t)__shfl_xor((int)top, 2));
            top = max(top, (uint32_t)__shfl_xor((int)top, 4));
            const uint32_t byte = mx_scale_byte(top);
            if (j < H) {
                uint32_t q = mx_code_pair<0>(0, o[0], o[1], byte);
                q = mx_code_pair<1>(q, o[2], o[3], byte);
                *(uint16_t*)(l.codes + (t * H + j) / 2) = byte == 255 ? 0 : (uint16_t)q;
                if (threadIdx.x % 8 == 0) l.scales[(t * H + j) / 32] = (uint8_t)byte;
            }
        }
    }
}

}  // namespace

hipError_t launch_norm(const NormLaunch& l, hipStream_t st) {
    NormArgs a{};
    a.l = l;
    auto vec = [](const void* p, int64_t stride, size_t el) {
        return ((uintptr_t)p | (uintptr_t)(stride * (int64_t)el)) % (4 * el) == 0 ? 1 : 0;
    };
    a.vec_h = vec(l.h, l.h_stride, dtype_bytes(l.dtype));
    a.vec_out = vec(l.out, l.out_stride, dtype_bytes(l.dtype));
    a.vec_y = vec(l.y, l.y_stride, dtype_bytes(l.y_dtype));
    a.vec_x = vec(l.x, l.H, 4);
    a.vec_gate = vec(l.gate, l.gate_row_stride, 4);
    a.vec_w = vec(l.after.weight, 0, 4);
    a.vec_u = vec(l.before.weight, 0, 4);
    const int chunks = (l.H + 3) / 4;
    const int threads = chunks >= kMaxThreads ? kMaxThreads : (chunks + 63) / 64 * 64;
    const dim3 grid((uint32_t)l.T), block(threads);
    if (chunks <= threads) hipLaunchKernelGGL(norm_kernel<1>, grid, block, 0, st, a);
    else if (chunks <= 2 * threads) hipLaunchKernelGGL(norm_kernel<2>, grid, block, 0, st, a);
    else hipLaunchKernelGGL(norm_kernel<4>, grid, block, 0, st, a);
    return hipGetLastError();
}

}  // namespace strata_moe
