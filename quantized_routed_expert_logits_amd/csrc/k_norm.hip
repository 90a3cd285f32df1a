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
// columns, so 4 neighbouring threads hold the 32 columns of one 4-bit block; where
// an array's rows do not take wide accesses (and no codes are written) it holds
// single columns, neighbouring threads neighbouring ones.
//
// What bounds it: with few tokens the latency of a chain of loads (slots, rows,
// the norms' sums), with many the memory, as far as enough tokens are in flight
// per CU to cover that chain.  So a token has few waves with few registers: 8192
// tokens of 2560, K = 10 bf16 rows, with the next norm and codes, take 153 us (671
// MB, 4.4 TB/s); runs of 4 columns (twice the waves) took 213, and 5 or 10 rows
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

struct NormArgs {
    NormLaunch l;
    int32_t vec_h, vec_y, vec_out, vec_x, vec_gate, vec_w, vec_u;  // rows of this array take 16-byte accesses
};

// Column i of a thread's run c.
template <bool kSingle>
__device__ __forceinline__ int column(int c, int i) {
    const int n = blockDim.x, t = threadIdx.x;
    return kSingle ? (c * kRun + i) * n + t : (c * n + t) * kRun + i;
}

// A thread's run c of a row (columns at and past H: 0).
template <bool kSingle, typename T>
__device__ __forceinline__ void load_run(const T* row, int c, int H, bool vec, float* v) {
    const int j = column<kSingle>(c, 0);
    if (!kSingle && vec && j + kRun <= H) {
        load8_vec(row + j, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) v[i] = column<kSingle>(c, i) < H ? widen(row[column<kSingle>(c, i)]) : 0.0f;
}
template <bool kSingle>
__device__ __forceinline__ void load_run(const void* base, int dtype, int64_t at, int c, int H, bool vec, float* v) {
    if (dtype == kF32) load_run<kSingle>((const float*)base + at, c, H, vec, v);
    else if (dtype == kF16) load_run<kSingle>((const _Float16*)base + at, c, H, vec, v);
    else load_run<kSingle>((const __bf16*)base + at, c, H, vec, v);
}
template <bool kSingle>
__device__ __forceinline__ void store_run(void* base, int dtype, int64_t at, int c, int H, bool vec, const float* v) {
    if (!kSingle) {
        const int j = column<kSingle>(c, 0);
        if (dtype == kF32) store8<float, v4f>((float*)base + at, j, H, vec, v);
        else if (dtype == kF16) store8<_Float16, v8h>((_Float16*)base + at, j, H, vec, v);
        else store8<__bf16, v8b>((__bf16*)base + at, j, H, vec, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
        const int j = column<kSingle>(c, i);
        if (j >= H) continue;
        if (dtype == kF32) ((float*)base)[at + j] = v[i];
        else if (dtype == kF16) ((_Float16*)base)[at + j] = (_Float16)v[i];
        else ((__bf16*)base)[at + j] = (__bf16)v[i];
    }
}

// v = sum_k p[t][k] y[slot[t][k]], k ascending.  Lane k holds slot and p of k, so
// that their loads are one, begun with the kernel (in the loop they cost 32 tokens
// 8.1 us against 7.5, and 8192 159 against 156).
template <int NC, bool kSingle, typename T>
__device__ __forceinline__ void gather(const NormArgs& a, int slot, int p_bits, double (*v)[kRun]) {
    const NormLaunch& l = a.l;
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
            for (int c = 0; c < NC; ++c) load_run<kSingle>((const T*)l.y + at * l.y_stride, c, l.H, a.vec_y, y[b][c]);
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

template <int NC, bool kSingle>
__device__ __forceinline__ void apply_norm(double (*v)[kRun], const NormScale& n, bool vec, int H, double* red) {
    float w[NC][kRun];
    if (n.weight)
#pragma unroll
        for (int c = 0; c < NC; ++c) load_run<kSingle>(n.weight, c, H, vec, w[c]);
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

template <int NC, bool kSingle>
__global__ __launch_bounds__(kMaxThreads) void norm_kernel(NormArgs a) {
    __shared__ double red[2][kMaxWaves];
    const NormLaunch& l = a.l;
    const int H = l.H;
    const int64_t t = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (t >= l.T) return;
    int slot = -1, p_bits = 0;
    const int lane = threadIdx.x % 64;
    if (l.slot && lane < l.K) slot = l.slot[t * l.K + lane], p_bits = __float_as_int(l.p[t * l.K + lane]);
    double v[NC][kRun], h[NC][kRun];
    float in[NC][kRun];
#pragma unroll
    for (int c = 0; c < NC; ++c) load_run<kSingle>(l.h, l.dtype, t * l.h_stride, c, H, a.vec_h, in[c]);
    if (l.y) {
        if (l.slot) {
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int i = 0; i < kRun; ++i) v[c][i] = 0.0;
            if (l.y_dtype == kF32) gather<NC, kSingle, float>(a, slot, p_bits, v);
            else if (l.y_dtype == kF16) gather<NC, kSingle, _Float16>(a, slot, p_bits, v);
            else gather<NC, kSingle, __bf16>(a, slot, p_bits, v);
        } else {
            float y[NC][kRun];
#pragma unroll
            for (int c = 0; c < NC; ++c) load_run<kSingle>(l.y, l.y_dtype, t * l.y_stride, c, H, a.vec_y, y[c]);
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
        if (l.after.on) apply_norm<NC, kSingle>(v, l.after, a.vec_w, H, red[0]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            float g[kRun], o[kRun];
#pragma unroll
            for (int i = 0; i < kRun; ++i) g[i] = 1.0f;
            if (l.gate) {
                const float* gr = l.gate + t * l.gate_row_stride;
                if (l.gate_col_stride) load_run<kSingle>(gr, c, H, a.vec_gate, g);
                else
#pragma unroll
                    for (int i = 0; i < kRun; ++i) g[i] = *gr;
            }
#pragma unroll
            for (int i = 0; i < kRun; ++i)
                h[c][i] = round_to(fma(l.residual_scale, h[c][i], l.block_scale * (g[i] * v[c][i])), l.dtype, &o[i]);
            store_run<kSingle>(l.out, l.dtype, t * l.out_stride, c, H, a.vec_out, o);
        }
    }
    if (!l.before.on) return;
    apply_norm<NC, kSingle>(h, l.before, a.vec_u, H, red[1]);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        float o[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) o[i] = (float)h[c][i];
        if (l.x) store_run<kSingle>(l.x, kF32, t * H, c, H, a.vec_x, o);
        if (!kSingle && l.codes) {  // H is a multiple of 32, so a block's 4 threads are all inside or all outside
            const int j = column<kSingle>(c, 0);
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

template <bool kSingle>
hipError_t launch_rows(const NormArgs& a, hipStream_t st) {
    const int runs = (a.l.H + kRun - 1) / kRun;
    const int threads = runs >= kMaxThreads ? kMaxThreads : (runs + 63) / 64 * 64;
    // less than 2^32 threads along x
    const int64_t most = (int64_t)1 << 21;
    const dim3 grid((uint32_t)std::min(a.l.T, most), (uint32_t)((a.l.T + most - 1) / most)), block(threads);
    if (runs <= threads) hipLaunchKernelGGL((norm_kernel<1, kSingle>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((norm_kernel<2, kSingle>), grid, block, 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormLaunch& l, hipStream_t st) {
    NormArgs a{};
    a.l = l;
    auto vec = [](const void* p, int64_t stride, size_t el) {
        return ((uintptr_t)p | (uintptr_t)(stride * (int64_t)el)) % 16 == 0 ? 1 : 0;
    };
    static_assert(kNormMaxH <= 2 * kMaxThreads * kRun, "two runs a thread");
    a.vec_h = vec(l.h, l.h_stride, dtype_bytes(l.dtype));
    a.vec_out = vec(l.out, l.out_stride, dtype_bytes(l.dtype));
    a.vec_y = vec(l.y, l.y_stride, dtype_bytes(l.y_dtype));
    a.vec_x = vec(l.x, l.H, 4);
    a.vec_gate = vec(l.gate, l.gate_row_stride, 4);
    a.vec_w = vec(l.after.weight, 0, 4);
    a.vec_u = vec(l.before.weight, 0, 4);
    const bool wide = l.H % kRun == 0 && a.vec_h && a.vec_out && a.vec_y && a.vec_x && a.vec_gate && a.vec_w && a.vec_u;
    return wide || l.codes ? launch_rows<false>(a, st) : launch_rows<true>(a, st);
}

}  // namespace strata_moe
