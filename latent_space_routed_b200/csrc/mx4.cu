// Microscaled 4-bit values (OCP MXFP4): quantisation and its inverse.
//
// A block of 32 values along a row has one scale 2^E, E = floor(log2 m) - 2 with
// m its largest magnitude (clamped to E >= -127), so that m / 2^E is in [4, 8);
// a value becomes the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 with its sign, ties
// to the even code, values past 6 to 6.  floor(log2 m) is m's exponent field,
// and dividing by 2^E is exact, so the codes do not depend on how it is computed.
//
// Both directions move bytes and little else (6 to 9 bytes per pair of bf16
// values, 10 to 17 per pair of fp32).  Four lanes share a block: each loads 8
// values with 16-byte loads and stores one word of codes, so that a warp's loads and
// stores are whole lines; the block's maximum is two shuffles.  360448 x 512 fp32 values
// to 4 bits and back (1.67 GB): 275 us, 94 % of the copy rate.  More groups in flight per
// thread (2, 4) or other grids were no faster.
#include "mx4.cuh"
#include "ptx.cuh"

#include <cuda_fp16.h>

namespace lmoe {
namespace {
using namespace ptx;

constexpr int THREADS = 256;

__device__ __forceinline__ void load8(float (&v)[8], const bf16 *p)
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(float (&v)[8], const float *p)
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(bf16 *p, const float (&v)[8], bool)
{
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
// `whole`: 32-byte aligned, one store.  Two 16-byte stores of a lane leave every store of the warp with half
// sectors (360448 x 512 values to 4 bits and back: 323 us against 275).
__device__ __forceinline__ void store8(float *p, const float (&v)[8], bool whole)
{
    if (whole) {
        asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(v[0]), "f"(v[1]), "f"(v[2]),
                     "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "l"(p)
                     : "memory");
        return;
    }
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Element offset of the 8 values with index i (in units of 8) of rows of c8 such units, ld elements apart.
template <typename Idx>
__device__ __forceinline__ int64_t place(Idx i, Idx c8, int64_t ld, bool dense)
{
    if (dense) return (int64_t)i * 8;
    const Idx row = i / c8;
    return (int64_t)row * ld + (int64_t)(i - row * c8) * 8;
}

template <typename T, typename Idx>
__global__ void __launch_bounds__(THREADS) quantize_kernel(const T *__restrict__ x, Idx n, Idx c8, int64_t ld,
                                                           uint32_t *__restrict__ codes, uint8_t *__restrict__ scales)
{
    const bool dense = ld == (int64_t)c8 * 8;
    const Idx step = (Idx)gridDim.x * THREADS;
    // n is a multiple of 4 (blocks of 32), so the four lanes of a block are in or out together
    for (Idx i = (Idx)blockIdx.x * THREADS + threadIdx.x; i < n; i += step) {
        float v[8];
        load8(v, x + place<Idx>(i, c8, ld, dense));
        uint32_t m = 0u;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
        const unsigned mates = 0xfu << (threadIdx.x & 28);
        m = max(m, __shfl_xor_sync(mates, m, 1));
        m = max(m, __shfl_xor_sync(mates, m, 2));
        const uint32_t e = m >> 23;
        const bool finite = e < 255u;
        const uint32_t sc = e > 2u ? e - 2u : 0u;
        const float inv = __uint_as_float((254u - sc) << 23);        // 2^-(sc - 127)
        uint32_t w = 0u;
        if (finite) {
#pragma unroll
            for (int j = 0; j < 4; ++j) w |= f32_to_e2m1x2(v[2 * j] * inv, v[2 * j + 1] * inv) << (8 * j);
        }
        codes[i] = w;
        if ((threadIdx.x & 3) == 0) scales[i / 4] = (uint8_t)(finite ? sc : 255u);
    }
}

template <typename T, typename Idx>
__global__ void __launch_bounds__(THREADS) dequantize_kernel(const uint32_t *__restrict__ codes,
                                                             const uint8_t *__restrict__ scales, Idx n, Idx c8,
                                                             int64_t ld, T *__restrict__ y, bool whole)
{
    const bool dense = ld == (int64_t)c8 * 8;
    const Idx step = (Idx)gridDim.x * THREADS;
    for (Idx i = (Idx)blockIdx.x * THREADS + threadIdx.x; i < n; i += step) {
        const uint32_t e = scales[i / 4];
        const float s = __uint_as_float(e == 255u ? 0x7fffffffu : e == 0u ? 0x00400000u : e << 23);
        uint32_t h[4];
        e2m1x8_to_f16(h, codes[i]);
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const __half2 p = *reinterpret_cast<const __half2 *>(&h[j]);
            v[2 * j] = __low2float(p) * s;
            v[2 * j + 1] = __high2float(p) * s;
        }
        store8(y + place<Idx>(i, c8, ld, dense), v, whole);
    }
}

__global__ void pack_scales_kernel(const uint8_t *__restrict__ G, const uint8_t *__restrict__ U,
                                   uint8_t *__restrict__ out, uint4 *__restrict__ codes, int64_t rows, int F, int blocks,
                                   int64_t pitch, int ib)
{
    const int64_t total = rows * pitch;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t r = i / pitch;
        const int c = (int)(i - r * pitch);
        uint8_t v = 0;
        if (c < blocks) {
            if (U) {
                const int64_t e = r / (2 * F);
                const int row = (int)(r - e * 2 * F), q = row / (2 * ib), w = row % (2 * ib);
                v = (w < ib ? G : U)[(e * F + q * ib + w % ib) * blocks + c];
            } else {
                v = G[r * blocks + c];
            }
        }
        out[i] = v;
        if (v == 255u) codes[r * blocks + c] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Blocks for n units: enough to fill the GPU, looping beyond.
unsigned grid_for(int64_t n)
{
    const int64_t g = (n + THREADS - 1) / THREADS;
    return (unsigned)(g < 1 ? 1 : g > 148 * 64 ? 148 * 64 : g);
}
constexpr int64_t IDX32 = (int64_t)1 << 31;      // 32-bit indices while index + grid stride stays below 2^32
}  // namespace

cudaError_t launch_mx4_quantize(const void *x, int bf16_in, int64_t rows, int64_t cols, int64_t ld, uint8_t *codes,
                                uint8_t *scales, cudaStream_t s)
{
    const int64_t n = rows * (cols / 8), c8 = cols / 8;
    const unsigned g = grid_for(n);
    uint32_t *w = (uint32_t *)codes;
    if (n < IDX32) {
        if (bf16_in) quantize_kernel<bf16, uint32_t><<<g, THREADS, 0, s>>>((const bf16 *)x, (uint32_t)n, (uint32_t)c8, ld, w, scales);
        else quantize_kernel<float, uint32_t><<<g, THREADS, 0, s>>>((const float *)x, (uint32_t)n, (uint32_t)c8, ld, w, scales);
    } else {
        if (bf16_in) quantize_kernel<bf16, uint64_t><<<g, THREADS, 0, s>>>((const bf16 *)x, (uint64_t)n, (uint64_t)c8, ld, w, scales);
        else quantize_kernel<float, uint64_t><<<g, THREADS, 0, s>>>((const float *)x, (uint64_t)n, (uint64_t)c8, ld, w, scales);
    }
    return cudaGetLastError();
}

cudaError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *y,
                                  int bf16_out, int64_t ld, cudaStream_t s)
{
    const int64_t n = rows * (cols / 8), c8 = cols / 8;
    const unsigned g = grid_for(n);
    const uint32_t *w = (const uint32_t *)codes;
    const bool whole = (uintptr_t)y % 32 == 0 && (rows == 1 || ld % 8 == 0);
    if (n < IDX32) {
        if (bf16_out) dequantize_kernel<bf16, uint32_t><<<g, THREADS, 0, s>>>(w, scales, (uint32_t)n, (uint32_t)c8, ld, (bf16 *)y, whole);
        else dequantize_kernel<float, uint32_t><<<g, THREADS, 0, s>>>(w, scales, (uint32_t)n, (uint32_t)c8, ld, (float *)y, whole);
    } else {
        if (bf16_out) dequantize_kernel<bf16, uint64_t><<<g, THREADS, 0, s>>>(w, scales, (uint64_t)n, (uint64_t)c8, ld, (bf16 *)y, whole);
        else dequantize_kernel<float, uint64_t><<<g, THREADS, 0, s>>>(w, scales, (uint64_t)n, (uint64_t)c8, ld, (float *)y, whole);
    }
    return cudaGetLastError();
}

cudaError_t launch_mx4_pack_scales(const uint8_t *G, const uint8_t *U, uint8_t *out, void *codes, int64_t nE, int F,
                                   int blocks, int64_t pitch, int ib, cudaStream_t s)
{
    pack_scales_kernel<<<2048, 256, 0, s>>>(G, U, out, (uint4 *)codes, nE * F * (U ? 2 : 1), F, blocks, pitch, ib);
    return cudaGetLastError();
}

}  // namespace lmoe
