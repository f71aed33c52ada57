// Product of microscaled 4-bit matrices on the tensor cores (sm_100a).
//
// C[m, n] = sum_k A[m, k] W[n, k], both operands 4-bit codes with one scale per 32
// values of K, fp32 sums in tensor memory, bf16 or fp32 out; dense, or grouped: the
// rows [offsets[e], offsets[e + 1]) of A against the N rows of W of expert e.
//
// tcgen05.mma kind::mxf4 (block_scale, scale_vec::2X) takes the codes from shared memory
// (128-byte-swizzled tiles, 256 values per row) and the scales from tensor memory.
// One tile is 128 x 192: two fp32 accumulators take 384 of the 512 TMEM columns, so
// that the epilogue of a tile overlaps the next one's main loop, and the scales of four
// ring stages take 96 more (24 each: 4 per 128 rows and 128 values).  With 256
// columns per tile there would be room for one accumulator only.
//
// What bounds it is memory wherever the layer uses it: codes and scales are 17/32 of
// a byte per value, the outputs 2 or 4 bytes each (prompt slot rows: outputs are 55 %
// of the bytes), and with few rows per expert the weights are nearly all of them.
// Measured in turn with other work, and (in brackets) alone in a loop: 32 decode tokens (1024 x 4096 x 1792 over 384
// experts, fp32 out) 313 us, 70 % of the copy rate (262, 84 %); prompt rows (196608 x 5376 x 1024, 512 experts)
// 1244 us, 1740 TFLOP/s, 46 % of the copy rate (1120-1165), where operands from L2 (40 KB per stage and tile) and the
// stores share the time: when it took 1086 us, 845 with one product of four, 920 without stores.
//
// Epilogues: plain (bf16 or fp32 rows); rows times a weight each (the routed down-projection);
// and the gate of the routed experts with requantisation: columns alternate between 32
// gates and their 32 ups, so that a lane holds one row's gates and ups of a whole block of 32
// outputs, applies the gate to the fp32 sums and stores 16 bytes of codes and the scale.
//
// Warps: 0 TMA producer; 1 TMEM owner and MMA issuer; 2-5 scales: rows of K / 32 bytes
// are read with plain loads one stage ahead (any row start, so that a group may begin
// anywhere) and written as the 32 x 16-byte matrices that tcgen05.cp spreads over the
// lanes; 6-13 epilogue, two per TMEM lane quarter.
//
// Every wait is bounded; one that gives up sets the status word and ends its role.
#include <atomic>

#include "gemm_tc.cuh"
#include "mx4.cuh"
#include "ptx.cuh"

namespace lmoe {
namespace {
using namespace ptx;

constexpr int BM = 128, BN = 192, KB = 256;              // tile; K values per stage (128 bytes of codes)
constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
constexpr int SFA_BYTES = 2 * 512, SFB_BYTES = 2 * 1024;  // two 128-value chunks; 128 and 256 rows each
constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
constexpr int STAGES = 4;                                 // five: prompt rows 2 % slower, the rest the same
constexpr int SF_WARPS = 4, EPI_WARPS = 8;
constexpr int THREADS = 32 * (2 + SF_WARPS + EPI_WARPS);
constexpr int MAX_E = 1024;
constexpr int SF_COL = 2 * BN, SF_COLS = 24;
constexpr size_t SMEM = 1024 + (size_t)STAGES * STAGE_BYTES + 256 + 2 * sizeof(int) * (MAX_E + 1);
static_assert(SMEM <= 232448, "shared memory");
static_assert(SF_COL + STAGES * SF_COLS <= 512, "tensor memory");
static_assert(STAGE_BYTES % 1024 == 0, "stage alignment");

// kind::mxf4: both operands e2m1, scales ue8m0, M = 128, N = BN; the scale ids (which
// two of a column's four bytes) are added per instruction.
constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((uint32_t)(BM >> 7) << 27);

struct Params {
    const uint8_t *a_scales, *w_scales;
    int64_t a_pitch, w_pitch;     // bytes between scale rows
    int M, N, K, E, grouped;
    const int32_t *offsets;
    void *out;                    // GLU: codes [M, N / 4]
    int64_t ldo;
    uint8_t *out_scales;          // GLU: [M, N / 64]
    const float *row_w;           // WEIGHTED: weight of each row
    float gate_cap, up_cap;
    int32_t *status;
    int stall_test;
};

// Shared-memory descriptor: K-major, 128-byte swizzle, 8-row atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t a)
{
    return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
// No swizzle, 16-byte rows, 8-row groups 128 bytes apart (the scale matrices).
__device__ __forceinline__ uint64_t desc_plain(uint32_t a)
{
    return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc));
}

__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}

__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[32])
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

struct Tile {
    int row0, row_end;    // rows of A and C that are real
    int wrow;             // first row of W
    int n0;
};

__device__ __forceinline__ Tile decode(const Params &p, const int *tile_off, const int *row_off, int item, int ntn)
{
    Tile t;
    const int mt = item / ntn;
    t.n0 = (item - mt * ntn) * BN;
    if (p.grouped) {
        int lo = 0, hi = p.E - 1;    // last e with tile_off[e] <= mt
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (tile_off[mid] <= mt) lo = mid; else hi = mid - 1;
        }
        t.row0 = row_off[lo] + (mt - tile_off[lo]) * BM;
        t.row_end = row_off[lo + 1];
        t.wrow = lo * p.N + t.n0;
    } else {
        t.row0 = mt * BM;
        t.row_end = p.M;
        t.wrow = t.n0;
    }
    return t;
}

// Eight scale bytes of a row from byte `at` on; those past `n` read as 1 (the codes
// there are zero), rows that do not exist as well.
__device__ __forceinline__ uint2 load_scales(const uint8_t *row, int at, int n, bool real, int align)
{
    uint2 v = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
    if (!real) return v;
    if (at + 8 <= n && align >= 8) return __ldg(reinterpret_cast<const uint2 *>(row + at));
    if (align >= 4) {
        if (at + 4 <= n) v.x = __ldg(reinterpret_cast<const uint32_t *>(row + at));
        if (at + 8 <= n) v.y = __ldg(reinterpret_cast<const uint32_t *>(row + at + 4));
        // K is a multiple of 64: at most two bytes are left
        if (at + 2 == n) v.x = 0x7f7f0000u | __ldg(reinterpret_cast<const uint16_t *>(row + at));
        if (at + 6 == n) v.y = 0x7f7f0000u | __ldg(reinterpret_cast<const uint16_t *>(row + at + 4));
        return v;
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = 0x7f7fu;
        if (at + 2 * i + 2 <= n) {
            if (align >= 2) h[i] = __ldg(reinterpret_cast<const uint16_t *>(row + at + 2 * i));
            else h[i] = (uint32_t)__ldg(row + at + 2 * i) | (uint32_t)__ldg(row + at + 2 * i + 1) << 8;
        }
    }
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

// 16-byte pieces: piece j of the lane's row -> piece lane % 4 of the row of lane (lane & ~3) + j.
__device__ __forceinline__ void transpose4(uint4 (&c)[4], int lane)
{
    auto exchange = [&](uint32_t &lo, uint32_t &hi, int bit) {
        const bool upper = (lane & bit) != 0;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? lo : hi, bit);
        if (upper) lo = got; else hi = got;
    };
    auto pieces = [&](uint4 &lo, uint4 &hi, int bit) {
        exchange(lo.x, hi.x, bit);
        exchange(lo.y, hi.y, bit);
        exchange(lo.z, hi.z, bit);
        exchange(lo.w, hi.w, bit);
    };
    pieces(c[0], c[1], 1);
    pieces(c[2], c[3], 1);
    pieces(c[0], c[2], 2);
    pieces(c[1], c[3], 2);
}

// 32 columns of 32 rows (a row per lane, `rows` of them real) to dst = the first row's, ldo apart.  Four lanes
// first exchange pieces, so that a store writes 64-byte parts of eight rows: a lane that stores its own row
// 16 bytes at a time makes every store touch 32 lines (prompt rows: 1488 us against 1086).
template <typename TO>
__device__ __forceinline__ void store_block(TO *dst, int64_t ldo, const float (&v)[32], int rows, int n, bool vec, int lane)
{
    constexpr int PER = 16 / (int)sizeof(TO);        // values per piece
    if (vec && n >= 32) {
#pragma unroll
        for (int part = 0; part < 32 / (4 * PER); ++part) {
            uint4 c[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float *x = v + 4 * PER * part + PER * j;
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if constexpr (sizeof(TO) == 2) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                        w[i] = *reinterpret_cast<const uint32_t *>(&b);
                    } else {
                        w[i] = __float_as_uint(x[i]);
                    }
                c[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            transpose4(c, lane);
            TO *at = dst + 4 * PER * part + PER * (lane & 3);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = (lane & ~3) + j;
                if (row < rows) *reinterpret_cast<uint4 *>(at + row * ldo) = c[j];
            }
        }
    } else if (lane < rows) {
        dst += lane * ldo;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < n) {
                if constexpr (sizeof(TO) == 2) dst[i] = __float2bfloat16_rn(v[i]);
                else dst[i] = v[i];
            }
    }
}

// The gate of 32 outputs.  SwiGLU with the hardware's exponential and reciprocal: the exponential is off by up to
// 2 + 1.173 |g| units in the last place, so the value by up to (8 + 1.2 |g|) 2^-23 (2^-20 at |g| = 0, 2^-18 at 20),
// where what follows rounds to 4 bits; gates below -87, whose silu is below 2^-118, give 0.  SiTU is its own instantiation: both in one unrolled body (with
// full-precision functions) made the kernel wait for instructions (98304 slot rows x 2816 x 512: 783 us, now 195).
template <bool SITU>
__device__ __forceinline__ void gate(float (&g)[32], const float (&u)[32], float cg, float cu)
{
    if (SITU) {
#pragma unroll
        for (int i = 0; i < 32; ++i) g[i] = glu_act(LMOE_ACT_SITU, g[i], u[i], cg, cu);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) g[i] = g[i] * __fdividef(1.f, 1.f + __expf(-g[i])) * u[i];
    }
}

// A block of 32 values as 16 bytes of codes and its scale byte (see mx4.cu).
__device__ __forceinline__ uint4 quantize_block(const float (&v)[32], uint32_t *scale)
{
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    const uint32_t e = m >> 23, sc = e > 2u ? e - 2u : 0u;
    *scale = e < 255u ? sc : 255u;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    if (e < 255u) {
        const float inv = __uint_as_float((254u - sc) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i >> 2] |= f32_to_e2m1x2(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * (i & 3));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename TO, int MODE>
__global__ void __launch_bounds__(THREADS, 1)
mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, const __grid_constant__ Params p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *g = smem_raw + (base - raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(g + (size_t)STAGES * STAGE_BYTES);
    const uint32_t full = smem_u32(bars), empty = full + 8 * STAGES, accf = empty + 8 * STAGES, acce = accf + 16;
    const uint32_t idle = acce + 16;                                  // after a failure: no product in flight
    int *words = reinterpret_cast<int *>(bars + 2 * STAGES + 5);     // [0] TMEM base, [1] abort, [2] issued, [3] scan
    volatile int *abort = words + 1;
    int *tile_off = reinterpret_cast<int *>(g + (size_t)STAGES * STAGE_BYTES + 256);
    int *row_off = tile_off + MAX_E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full + 8 * s, 2);                        // the copies, the scales
            mbar_init(empty + 8 * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(accf + 8 * a, 1);
            mbar_init(acce + 8 * a, EPI_WARPS);
        }
        mbar_init(idle, 1);
        words[1] = words[2] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(words)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (p.grouped && warp == 0) {
        // row offsets, clamped to [0, M] and to ascending order, and the m-tiles before each expert
        int tiles = 0, last = 0;
        for (int e0 = 0; e0 <= p.E; e0 += 32) {
            const int e = e0 + lane;
            int o = e <= p.E ? __ldg(p.offsets + e) : 0;
            o = max(0, min(o, p.M));
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, o, d);
                if (lane >= d) o = max(o, v);
            }
            o = max(o, last);
            int prev = __shfl_up_sync(0xffffffffu, o, 1);
            if (lane == 0) prev = last;
            int t = e > 0 && e <= p.E ? (o - prev + BM - 1) / BM : 0;    // tiles of expert e - 1
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, t, d);
                if (lane >= d) t += v;
            }
            if (e <= p.E) {
                row_off[e] = o;
                tile_off[e] = tiles + t;
            }
            tiles += __shfl_sync(0xffffffffu, t, 31);
            last = __shfl_sync(0xffffffffu, o, 31);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = (uint32_t)*reinterpret_cast<volatile int *>(words);

    const int ntn = (p.N + BN - 1) / BN, nkb = (p.K + KB - 1) / KB;
    const int total = (p.grouped ? tile_off[p.E] : (p.M + BM - 1) / BM) * ntn;
    auto give_up = [&](int code) {
        atomicOr(p.status, code);
        *abort = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------ TMA producer
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int item = blockIdx.x; item < total && ok; item += gridDim.x) {
                const Tile t = decode(p, tile_off, row_off, item, ntn);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!(ok = mbar_wait(empty + 8 * s, ph ^ 1u, abort))) break;
                    const uint32_t st = base + (uint32_t)(s * STAGE_BYTES);
                    mbar_expect_tx(full + 8 * s, A_BYTES + B_BYTES);
                    tma_load_2d(st, &tmA, full + 8 * s, kb * (KB / 2), t.row0);
                    tma_load_2d(st + A_BYTES, &tmW, full + 8 * s, kb * (KB / 2), t.wrow);
                    words[2] = ++issued;
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) give_up(0x1);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ------------------------------------------------------ MMA issuer
            int s = 0, local = 0;
            uint32_t ph = 0;
            bool ok = !p.stall_test || mbar_wait(accf, 0u, abort);      // (the failure-detection test: nothing arrives there)
            for (int item = blockIdx.x; item < total && ok; item += gridDim.x, ++local) {
                const int acc = local & 1;
                if (!(ok = mbar_wait(acce + 8 * acc, ((uint32_t)(local >> 1) & 1u) ^ 1u, abort))) break;
                fence_after();
                const uint32_t d = tmem + (uint32_t)(acc * BN);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!(ok = mbar_wait(full + 8 * s, ph, abort))) break;
                    const uint32_t st = base + (uint32_t)(s * STAGE_BYTES);
                    const uint32_t sf = st + A_BYTES + B_BYTES;
                    const uint32_t tsf = tmem + (uint32_t)(SF_COL + s * SF_COLS);
                    // scales of this stage: A chunks at columns 0, 4; W chunks at 8, 16 (256 rows each)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        copy_scales(tsf + 4 * c, desc_plain(sf + 512 * c));
                        copy_scales(tsf + 8 + 8 * c, desc_plain(sf + SFA_BYTES + 1024 * c));
                        copy_scales(tsf + 12 + 8 * c, desc_plain(sf + SFA_BYTES + 1024 * c + 512));
                    }
                    const uint64_t da = desc_sw128(st), db = desc_sw128(st + A_BYTES);
                    const int left = p.K - kb * KB;            // steps of 64 values; zeros past K need no product
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (64 * k >= left) break;
                        const uint32_t id = 2u * (k & 1);
                        mma_mxf4(d, da + 2 * k, db + 2 * k, IDESC | id << 4 | id << 29, tsf + 4 * (k >> 1),
                                 tsf + 8 + 8 * (k >> 1), (kb | k) != 0);
                    }
                    commit(empty + 8 * s);
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) commit(accf + 8 * acc);
            }
            if (!ok) give_up(0x2);
        }
    } else if (warp < 2 + SF_WARPS) {
        // ---------------------------------------------------------- scales
        // Warp w brings every fourth stage, all 320 rows of it (lane: rows lane + 32 i), and asks for
        // its next one before it waits for the slot: four stages of small loads are in flight
        const int n = p.K / 32;
        auto align_of = [](const uint8_t *b, int64_t pitch) {
            const uint64_t v = (uint64_t)b | (uint64_t)pitch;
            return (v & 7) == 0 ? 8 : (v & 3) == 0 ? 4 : (v & 1) == 0 ? 2 : 1;
        };
        const int al_a = align_of(p.a_scales, p.a_pitch), al_w = align_of(p.w_scales, p.w_pitch);
        const int64_t wrows = (int64_t)(p.grouped ? p.E : 1) * p.N;
        const int first = warp - 2;
        int item = blockIdx.x, kb = 0, at = -1;
        Tile t;
        uint2 r[10];                                           // rows of A, then of W
        auto advance = [&](int by) {                           // `by` stages on; the tile where it changes
            for (kb += by; kb >= nkb; kb -= nkb) item += gridDim.x;
            if (item < total && item != at) t = decode(p, tile_off, row_off, item, ntn);
            at = item;
        };
        auto fetch = [&]() {
            const uint8_t *pa = p.a_scales + (int64_t)(t.row0 + lane) * p.a_pitch;
            const uint8_t *pw = p.w_scales + (int64_t)(t.wrow + lane) * p.w_pitch;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[i] = load_scales(pa + 32 * i * p.a_pitch, kb * 8, n, t.row0 + 32 * i + lane < t.row_end, al_a);
#pragma unroll
            for (int i = 0; i < 6; ++i)
                r[4 + i] = load_scales(pw + 32 * i * p.w_pitch, kb * 8, n, t.wrow + 32 * i + lane < wrows, al_w);
        };
        bool ok = true;
        int s = first % STAGES;
        uint32_t ph = 0;
        advance(first);
        if (item < total) fetch();
        while (item < total) {
            uint2 v[10];
#pragma unroll
            for (int i = 0; i < 10; ++i) v[i] = r[i];
            advance(SF_WARPS);
            if (item < total) fetch();                         // while this stage's slot is awaited
            ok = __all_sync(0xffffffffu, mbar_wait(empty + 8 * s, ph ^ 1u, abort));
            if (!ok) break;
            // row r of a 128-row chunk: 4 bytes at (r % 32) * 16 + (r / 32) * 4
            const uint32_t sf = base + (uint32_t)(s * STAGE_BYTES + A_BYTES + B_BYTES) + (uint32_t)(lane * 16);
            const uint32_t sw = sf + SFA_BYTES;
            sts128(sf, v[0].x, v[1].x, v[2].x, v[3].x);
            sts128(sf + 512, v[0].y, v[1].y, v[2].y, v[3].y);
            sts128(sw, v[4].x, v[5].x, v[6].x, v[7].x);
            sts64(sw + 512, v[8].x, v[9].x);
            sts128(sw + 1024, v[4].y, v[5].y, v[6].y, v[7].y);
            sts64(sw + 1536, v[8].y, v[9].y);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(full + 8 * s);
            s += SF_WARPS;
            if (s >= STAGES) {
                s -= STAGES;
                ph ^= 1u;
            }
        }
        if (!ok && lane == 0) give_up(0x4);
    } else {
        // ---------------------------------------------------------- epilogue
        constexpr bool GLU = MODE == MX4_GLU || MODE == MX4_GLU_SITU;
        const int q = warp & 3, hset = (warp - 2 - SF_WARPS) >> 2;     // lane quarter; half of the columns
        const bool vec = ((uintptr_t)p.out & 15u) == 0 && (p.ldo * (int)sizeof(TO)) % 16 == 0;
        int local = 0;
        bool ok = true;
        for (int item = blockIdx.x; item < total; item += gridDim.x, ++local) {
            const int acc = local & 1;
            const Tile t = decode(p, tile_off, row_off, item, ntn);
            ok = __all_sync(0xffffffffu, mbar_wait(accf + 8 * acc, (uint32_t)(local >> 1) & 1u, abort));
            if (!ok) break;
            fence_after();
            const int row = t.row0 + 32 * q + lane;
            TO *dst = (TO *)p.out + (int64_t)(t.row0 + 32 * q) * p.ldo + t.n0;
            const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(acc * BN);
            if (t.row0 + 32 * q < t.row_end) {                  // uniform: some row of this quarter is real
                if (GLU) {
#pragma unroll 1
                    for (int c = 64 * (hset ^ (local & 1)); c < BN && t.n0 + c < p.N; c += 128) {  // N: a multiple of 64
                        float v[32], u[32];
                        tmem_ld32(src + c, v);
                        tmem_ld32(src + c + 32, u);
                        gate<MODE == MX4_GLU_SITU>(v, u, p.gate_cap, p.up_cap);
                        uint32_t scale;
                        const uint4 w = quantize_block(v, &scale);
                        if (row < t.row_end) {
                            const int64_t block = (int64_t)row * (p.N / 64) + (t.n0 + c) / 64;
                            reinterpret_cast<uint4 *>(p.out)[block] = w;
                            p.out_scales[block] = (uint8_t)scale;
                        }
                    }
                } else {
                    const float weight = MODE == MX4_WEIGHTED && row < t.row_end ? p.row_w[row] : 1.f;
#pragma unroll 1
                    for (int c = 96 * hset; c < 96 * hset + 96; c += 32) {
                        const int left = p.N - t.n0 - c;
                        if (left <= 0) break;
                        float v[32];
                        tmem_ld32(src + c, v);
                        if (MODE == MX4_WEIGHTED) {
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] *= weight;
                        }
                        store_block<TO>(dst + c, p.ldo, v, t.row_end - t.row0 - 32 * q, left, vec, lane);
                    }
                }
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acce + 8 * acc);
        }
        if (!ok && lane == 0) give_up(0x8);
    }

    fence_before();
    __syncthreads();
    fence_after();
    if (*abort && threadIdx.x == 0) {
        // copies in flight must land before the block's memory goes away (the scale warps' arrivals may be
        // missing, so the wait may run out; it is bounded)
        int none = 0;
        const int issued = words[2];
        for (int i = max(0, issued - STAGES); i < issued; ++i)
            if (!mbar_wait(full + 8 * (i % STAGES), (uint32_t)(i / STAGES) & 1u, &none)) break;
    }
    if (*abort && threadIdx.x == 32) {       // (the issuer) and products in flight before their memory goes away
        int none = 0;
        commit(idle);
        mbar_wait(idle, 0u, &none);
    }
    __syncthreads();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

std::atomic<int> g_stall_next{0};

template <typename TO, int MODE>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &w, const Params &p, int grid, cudaStream_t s)
{
    static std::atomic<uint64_t> ready{0};       // devices (the first 64) whose shared-memory limit is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load() >> dev & 1u)) {
        e = cudaFuncSetAttribute(mx4_gemm_kernel<TO, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or((uint64_t)1 << dev);
    }
    mx4_gemm_kernel<TO, MODE><<<grid, THREADS, SMEM, s>>>(a, w, p);
    return cudaGetLastError();
}
}  // namespace

void mx4_debug_stall_next() { g_stall_next.store(1); }

cudaError_t launch_mx4_gemm(const Mx4GemmArgs &g, int32_t *status, cudaStream_t s)
{
    CUtensorMap a, w;
    const uint64_t kb = (uint64_t)g.K / 2, wrows = (uint64_t)(g.offsets ? g.E : 1) * g.N;
    if (!tc_encode_map(&a, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.a_codes, 2, {kb, (uint64_t)g.M}, {kb}, {128, BM}, true) ||
        !tc_encode_map(&w, CU_TENSOR_MAP_DATA_TYPE_UINT8, g.w_codes, 2, {kb, wrows}, {kb}, {128, BN}, true))
        return cudaErrorInvalidValue;
    Params p = {};
    p.a_scales = g.a_scales; p.w_scales = g.w_scales; p.a_pitch = g.a_pitch; p.w_pitch = g.w_pitch;
    p.M = g.M; p.N = g.N; p.K = g.K; p.E = g.E; p.grouped = g.offsets != nullptr; p.offsets = g.offsets;
    p.out = g.out; p.ldo = g.ldo; p.status = status; p.stall_test = g_stall_next.exchange(0);
    const int64_t ntn = (g.N + BN - 1) / BN;
    const int64_t tiles = ((g.M + BM - 1) / BM + (g.offsets ? g.E : 0)) * ntn;     // at most
    const int sms = tc_num_sms() > 0 ? tc_num_sms() : 148;
    const int grid = (int)(tiles < sms ? tiles : sms);
    p.out_scales = g.out_scales; p.row_w = g.row_w; p.gate_cap = g.gate_cap; p.up_cap = g.up_cap;
    if (g.mode == MX4_GLU) return launch<bf16, MX4_GLU>(a, w, p, grid, s);
    if (g.mode == MX4_GLU_SITU) return launch<bf16, MX4_GLU_SITU>(a, w, p, grid, s);
    if (g.mode == MX4_WEIGHTED) return launch<bf16, MX4_WEIGHTED>(a, w, p, grid, s);
    return g.out_bf16 ? launch<bf16, MX4_STORE>(a, w, p, grid, s) : launch<float, MX4_STORE>(a, w, p, grid, s);
}

}  // namespace lmoe
