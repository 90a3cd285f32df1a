// Launches of the few-token layer and of the adapters: what the entry points
// in strata_moe.hip hand to k_decode.hip and k_adapt.hip.
#pragma once

#include "internal.h"

namespace strata_moe {

// ---- the few-token layer (k_decode.hip)
constexpr int kDecodeMaxTokens = 64;  // a token is one bit of an expert's 64-bit row mask
// Everything one call needs.
struct DecodeLaunch {
    const float* x;
    const float* router_w;
    const float* bias;         // or null
    const float* shared_gate;  // or null: no shared expert
    const uint8_t* gate_up;
    int64_t gate_up_stride;
    const uint8_t* down;
    int64_t down_stride;
    int32_t T, H, E, K, I;
    int32_t sym;  // the symmetric weight map
    float* out;
    char* workspace;
};
size_t decode_workspace(int32_t T, int32_t H, int32_t E, int32_t K, int32_t I, bool shared);
hipError_t launch_decode(const DecodeLaunch& l, hipStream_t st);

// ---- per-request low-rank adapters (k_adapt.hip)
constexpr int kAdapterF32 = 1, kAdapterF16 = 2, kAdapterBF16 = 3;  // STRATA_MOE_ADAPTER_*
constexpr int kAdapterMaxRank = 256;
struct AdaptLaunch {
    const float* x;
    int64_t x_stride;
    const int32_t* ids;
    const void* a;
    const void* b;
    const float* scale;
    const int32_t* ranks;
    int32_t n_adapter, rank, in_dim, out_dim, dtype;
    int64_t T;
    const float* y;
    int64_t y_stride;
    float* out;
    int64_t out_stride;
    char* workspace;
};
size_t adapt_workspace(int64_t T, int32_t rank, int32_t in_dim);
hipError_t launch_adapt(const AdaptLaunch& l, hipStream_t st);

}  // namespace strata_moe
