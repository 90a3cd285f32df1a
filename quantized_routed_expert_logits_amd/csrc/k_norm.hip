// Norms before and after a block, with the residual stream between them.  Per
// token t, with h the stream, y the block's output rows and u_j = (offset + w_j):
//   v = sum_k p[t][k] y[slot[t][k]]          (or v = y[t])
//   b = u v / sqrt(mean(v^2) + eps)          (or b = v)
//   h' = residual_scale h + block_scale gate b, rounded to the stream's type
//   x = u' h' / sqrt(mean(h'^2) + eps'), and x rounded to 4 bits per 32 values
// A call has the part up to h', the part from h' (h' = h then), or both.
//
// One workgroup per token; its row stays in registers between the sums, so
// every array is read or written once.  A thread holds runs of 8 neighbouring
// columns, so 4 neighbouring threads hold the 32 columns of one 4-bit block; it
// takes them in 16-byte accesses wherever the row begins, the last run of a row that
// is no multiple of 8 one by one.
//
// What bounds it: with few tokens the latency of a chain of loads (slots, rows,
// the norms' sums), with many the memory, as far as enough tokens are in flight
// per CU to cover that chain.  So a token has few waves with few registers: 8192
// tokens of 2560, K = 10 bf16 rows, with the next norm and codes, take 152 us (599
// MB, 3.9 TB/s); runs of 4 columns (twice the waves) took 213, and 5 or 10 rows
// loaded before the first is used, which costs registers, 183 and 280.
//
// All arithmetic is in 64 bits and an output is rounded to fp32, and from there
// to 16 bits: the stored stream and the 4-bit codes are those of the exact row
// except where it lies within about 2^-50 of a border.  The memory bounds these
// kernels, so the wider arithmetic is free.
#include <algorithm>

#include "block.h"
#include "mxfp.h"

namespace strata_moe {
namespace {

constexpr int kMaxThreads = 1024;
constexpr int kRun = 8;  // columns of a thread's run

// The first column of a thread's run c.
__device__ __forceinline__ int column(int c) { return (c * (int)blockDim.x + (int)threadIdx.x) * kRun; }

// A thread's run c of a row (columns at and past H: 0).
template <typename T>
__device__ __forceinline__ void load_run(const T* row, int c, int H, float* v) {
    const int j = column(c);
    if (j + kRun <= H) {
        load8(row + j, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) v[i] = j + i < H ? widen(row[j + i]) : 0.0f;
}
__device__ __forceinline__ void load_run(const void* base, int dtype, int64_t at, int c, int H, float* v) {
    if (dtype == kF32) load_run((const float*)base + at, c, H, v);
    else if (dtype == kF16) load_run((const _Float16*)base + at, c, H, v);
    else load_run((const __bf16*)base + at, c, H, v);
}
__device__ __forceinline__ void store_run(void* base, int dtype, int64_t at, int c, int H, const float* v) {
    const int j = column(c);
    if (dtype == kF32) store8<float, v4f_any>((float*)base + at, j, H, v);
    else if (dtype == kF16) store8<_Float16, v8h_any>((_Float16*)base + at, j, H, v);
    else store8<__bf16, v8b_any>((__bf16*)base + at, j, H, v);
}

// v = sum_k p[t][k] y[slot[t][k]], k ascending.  Lane k holds slot and p of k, so
// that their loads are one, begun with the kernel (in the loop they cost 32 tokens
// 8.1 us against 7.5, and 8192 159 against 156).
template <int NC, typename T>
__device__ __forceinline__ void gather(const NormLaunch& l, int slot, int p_bits, double (*v)[kRun]) {
    constexpr int kBatch = 2;
    for (int k0 = 0; k0 < l.K; k0 += kBatch) {
        int row[kBatch];
        float p[kBatch], y[kBatch][NC][kRun];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            row[b] = __builtin_amdgcn_readlane(slot, k0 + b);  // -1 from K on
            p[b] = __int_as_float(__builtin_amdgcn_readlane(p_bits, k0 + b));
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            // a row to read; used if it is the slot's
            const int64_t at = row[b] < 0 || row[b] >= l.y_rows ? 0 : row[b];
#pragma unroll
            for (int c = 0; c < NC; ++c) load_run((const T*)l.y + at * l.y_stride, c, l.H, y[b][c]);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (row[b] < 0 || row[b] >= l.y_rows) continue;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < kRun; ++i) v[c][i] = fma((double)p[b], (double)y[b][c][i], v[c][i]);
        }
    }
}

// The sum over the wave's 64 lanes, the same in each.  Lanes change places within
// the registers; through the LDS path (__shfl_xor) 32 tokens took 7.6 us against
// 7.0, one token's norm 2.7 against 2.5 and 8192 156 against 153.
template <int kCtrl>
__device__ __forceinline__ double moved(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_mov_dpp((int)(uint32_t)u, kCtrl, 0xf, 0xf, true);
    const uint32_t hi = __builtin_amdgcn_mov_dpp((int)(uint32_t)(u >> 32), kCtrl, 0xf, 0xf, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double s) {
    s += moved<0xb1>(s);   // quad_perm [1, 0, 3, 2]: lane ^ 1
    s += moved<0x4e>(s);   // quad_perm [2, 3, 0, 1]: lane ^ 2
    s += moved<0x141>(s);  // mirrored within 8 lanes: the other four's sum
    s += moved<0x140>(s);  // mirrored within 16: the other eight's
    // of two registers with the same rows of 16 lanes (halves of 32) a swap of one's odd
    // rows with the other's even ones leaves a row and its neighbour side by side
    auto both = [](double v, auto swap) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const auto lo = swap((uint32_t)u), hi = swap((uint32_t)(u >> 32));
        return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) +
               __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
    };
    s = both(s, [](uint32_t w) { return __builtin_amdgcn_permlane16_swap(w, w, false, false); });
    return both(s, [](uint32_t w) { return __builtin_amdgcn_permlane32_swap(w, w, false, false); });
}

// The sum over the workgroup, in a fixed order, in every thread.  red: one
// double per possible wave, not used by an earlier sum of the same kernel.
constexpr int kMaxWaves = kMaxThreads / 64;
__device__ __forceinline__ double block_sum(double s, double* red) {
    s = wave_sum(s);
    const int waves = blockDim.x / 64;
    if (waves == 1) return s;
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = s;
    if ((int)threadIdx.x >= waves && threadIdx.x < kMaxWaves) red[threadIdx.x] = 0.0;
    __syncthreads();
    s = red[0];
#pragma unroll
    for (int w = 1; w < kMaxWaves; ++w) s += red[w];
    return s;
}

// 1 / sqrt(v): the unit's estimate and two Newton steps, which square its error
// (2^-25 or less) twice; at 0 and infinity the estimate is the result.
__device__ __forceinline__ double inverse_root(double v) {
    const double e = __builtin_amdgcn_rsq(v);
    double r = e;
#pragma unroll
    for (int i = 0; i < 2; ++i) r = r * fma(-0.5 * v * r, r, 1.5);
    return __builtin_isfinite(r) ? r : e;
}

template <int NC>
__device__ __forceinline__ void apply_norm(double (*v)[kRun], const NormScale& n, int H, double* red) {
    float w[NC][kRun];
    if (n.weight)
#pragma unroll
        for (int c = 0; c < NC; ++c) load_run(n.weight, c, H, w[c]);
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < kRun; ++i) s = fma(v[c][i], v[c][i], s);
    s = block_sum(s, red);
    const double r = inverse_root(s / H + n.eps);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
            v[c][i] *= r;
            if (n.weight) v[c][i] *= n.offset + (double)w[c][i];
        }
}

template <int NC>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(NormLaunch l) {
    __shared__ double red[2][kMaxWaves];
    const int H = l.H;
    const int64_t t = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (t >= l.T) return;
    int slot = -1, p_bits = 0;
    const int lane = threadIdx.x % 64;
    if (l.slot && lane < l.K) slot = l.slot[t * l.K + lane], p_bits = __float_as_int(l.p[t * l.K + lane]);
    double v[NC][kRun], h[NC][kRun];
    float in[NC][kRun];
#pragma unroll
    for (int c = 0; c < NC; ++c) load_run(l.h, l.dtype, t * l.h_stride, c, H, in[c]);
    if (l.y) {
        if (l.slot) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < kRun; ++i) v[c][i] = 0.0;
            if (l.y_dtype == kF32) gather<NC, float>(l, slot, p_bits, v);
            else if (l.y_dtype == kF16) gather<NC, _Float16>(l, slot, p_bits, v);
            else gather<NC, __bf16>(l, slot, p_bits, v);
        } else {
            float y[NC][kRun];
#pragma unroll
            for (int c = 0; c < NC; ++c) load_run(l.y, l.y_dtype, t * l.y_stride, c, H, y[c]);
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < kRun; ++i) v[c][i] = y[c][i];
        }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < kRun; ++i) h[c][i] = in[c][i];
    if (l.y) {
        if (l.after.on) apply_norm<NC>(v, l.after, H, red[0]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float g[kRun], o[kRun];
#pragma unroll
            for (int i = 0; i < kRun; ++i) g[i] = 1.0f;
            if (l.gate) {
                const float* gr = l.gate + t * l.gate_row_stride;
                if (l.gate_col_stride) load_run(gr, c, H, g);
                else
#pragma unroll
                    for (int i = 0; i < kRun; ++i) g[i] = *gr;
            }
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                h[c][i] = round_to(fma(l.residual_scale, h[c][i], l.block_scale * (g[i] * v[c][i])), l.dtype, &o[i]);
            store_run(l.out, l.dtype, t * l.out_stride, c, H, o);
        }
    }
    if (!l.before.on) return;
    apply_norm<NC>(h, l.before, H, red[1]);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        float o[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) o[i] = (float)h[c][i];
        if (l.x) store_run(l.x, kF32, t * H, c, H, o);
        if (l.codes) {  // H is a multiple of 32, so a block's 4 threads are all inside or all outside
            const int j = column(c);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < kRun; ++i) top = max(top, __float_as_uint(o[i]) & 0x7fffffffu);
            top = max(top, (uint32_t)__shfl_xor((int)top, 1));
            top = max(top, (uint32_t)__shfl_xor((int)top, 2));
            const uint32_t byte = mx_scale_byte(top);
            if (j < H) {
                uint32_t q = mx_code_pair<0>(0, o[0], o[1], byte);
                q = mx_code_pair<1>(q, o[2], o[3], byte);
                q = mx_code_pair<2>(q, o[4], o[5], byte);
                q = mx_code_pair<3>(q, o[6], o[7], byte);
                *(uint32_t*)(l.codes + (t * H + j) / 2) = byte == 255 ? 0 : q;
                if (threadIdx.x % 4 == 0) l.scales[(t * H + j) / 32] = (uint8_t)byte;
            }
        }
    }
}

}  // namespace

hipError_t launch_norm(const NormLaunch& l, hipStream_t st) {
    static_assert(kNormMaxH <= 2 * kMaxThreads * kRun, "two runs a thread");
    const int runs = (l.H + kRun - 1) / kRun;
    const int threads = runs >= kMaxThreads ? kMaxThreads : (runs + 63) / 64 * 64;
    // less than 2^32 threads along x
    const int64_t most = (int64_t)1 << 21;
    const dim3 grid((uint32_t)std::min(l.T, most), (uint32_t)((l.T + most - 1) / most)), block(threads);
    if (runs <= threads) hipLaunchKernelGGL(norm_kernel<1>, grid, block, 0, st, l);
    else hipLaunchKernelGGL(norm_kernel<2>, grid, block, 0, st, l);
    return hipGetLastError();
}

}  // namespace strata_moe
