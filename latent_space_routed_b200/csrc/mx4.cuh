// Microscaled 4-bit tensors: launchers (kernels in mx4.cu, products in mx4_gemm.cu).
#pragma once

#include "lmoe_internal.cuh"

namespace lmoe {

// x [rows, cols] (row stride ld elements) to codes [rows, cols / 2] and scales [rows, cols / 32].
cudaError_t launch_mx4_quantize(const void *x, int bf16_in, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                                uint8_t *scales, cudaStream_t s);
cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *y,
                                  int bf16_out, int64_t ld, cudaStream_t s);
// Scale rows of `blocks` bytes to rows `pitch` bytes apart, zero behind them.  With U != nullptr the rows
// of G and U [nE, F] are interleaved in blocks of ib, as launch_pack_glu does with the codes.  `codes`: the
// codes in the new order, where blocks of scale 255 (NaN) become zeros (the few-token kernel multiplies
// them by infinity).
cudaError_t launch_mx4_pack_scales(const uint8_t *G, const uint8_t *U, uint8_t *out, void *codes, int64_t nE, int F,
                                   int blocks, int64_t pitch, int ib, cudaStream_t s);

// C [M, N] = A W^T of 4-bit matrices (mx4_gemm.cu); grouped when offsets != nullptr
// (device [E + 1], W of expert e at rows e N).  K a multiple of 64, codes 16-byte
// aligned; scale rows a_pitch / w_pitch bytes apart.
enum Mx4Mode {
    MX4_STORE = 0,       // out [M, N], bf16 or fp32
    MX4_WEIGHTED = 1,    // bf16 out, row m times row_w[m]
    MX4_GLU = 2,         // columns alternate 32 gates, 32 ups: SwiGLU requantised to out (codes) and out_scales
    MX4_GLU_SITU = 3     // the same with the SiTU gate
};
constexpr int MX4_GLU_BLOCK = 32;
struct Mx4GemmArgs {
    int mode;
    uint8_t *out_scales;
    const float *row_w;
    float gate_cap, up_cap;
    const uint8_t *a_codes, *a_scales, *w_codes, *w_scales;
    int64_t a_pitch, w_pitch;
    int M, N, K, E;
    const int32_t *offsets;
    void *out;
    int out_bf16;
    int64_t ldo;
};
cudaError_t launch_mx4_gemm(const Mx4GemmArgs &g, int32_t *status, cudaStream_t s);
// Failure-detection test hook: a wait of the next launch_mx4_gemm runs out.
void mx4_debug_stall_next();

}  // namespace lmoe
