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
// of G and U [nE, F] are interleaved in blocks of ib, as launch_pack_glu does with the codes.
cudaError_t launch_mx4_pack_scales(const uint8_t *G, const uint8_t *U, uint8_t *out, int64_t nE, int F, int blocks,
                                   int64_t pitch, int ib, cudaStream_t s);

}  // namespace lmoe
