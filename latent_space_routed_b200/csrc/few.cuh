// The whole layer for a few tokens in one kernel: host interface.
#pragma once

#include <cuda.h>

#include "lmoe_internal.cuh"

namespace lmoe {

constexpr int FEW_MAX_T = 8;            // one column of an m16n8k16 product per token
constexpr int FEW_MAX_SLOTS = 64 * FEW_MAX_T;

// Tensor maps of the weights as the kernel streams them (built once per handle).
struct FewMaps {
    CUtensorMap router, down, shared_gu, routed_gu, shared_down, routed_down, up, routed_gu_scales, routed_down_scales;
};

// Weights of a handle, in its own layouts.
struct FewWeights {
    const float *Wr;
    const uint32_t *Wr_top;              // largest magnitude in Wr, as bits
    const void *Wdown, *Wgu_s, *Wcat;
    const void *Wgu, *D;                 // token type; codes when mx4
    const void *Wgu_scales, *D_scales;   // mx4: [rows, pitch] with pitches mx4_scale_pitch(l), (f)
    bool mx4;
};

// Bytes between the scale rows of a handle's 4-bit experts, for rows of K values.
inline int64_t mx4_scale_pitch(int64_t K) { return (K / 32 + 15) / 16 * 16; }

// The largest magnitude of n fp32 values, as bits, to *top (device).
cudaError_t few_largest(const float *v, int64_t n, uint32_t *top, cudaStream_t s);

bool few_make_maps(const lmoe_config &c, const FewWeights &w, FewMaps *m);

// Bytes of one call's workspace, which begins with the status word.
size_t few_workspace_bytes(const lmoe_config &c, int64_t T);

cudaError_t few_launch(const lmoe_config &c, const FewMaps &m, const FewWeights &w, const float *bias, const void *x, int T,
                       void *y, int32_t *sel, void *p_out, void *u_out, void *workspace, bool stall_test,
                       cudaStream_t s);

}  // namespace lmoe
