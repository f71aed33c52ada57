// The whole layer forward for 1 to 8 tokens in one kernel.
//
// With a few tokens the layer does nothing but read weights: each of the seven
// products below streams its matrix once and does 2 T operations per weight.
// What costs time beside the stream is the gaps between dependent stages, so
// the stages are not separate launches: the layer is a list of work items, in
// the order
//
//   router       4 rows of W_r                     -> r = sigmoid(W_r x), in 64 bits
//   down         16 rows of W_down                 -> z
//   route        (no weights) top-k, p, the touched experts and their slots
//   shared gu    16 gate and 16 up rows            -> shared hidden
//   routed gu    16 gate and 16 up rows of expert  -> hidden H of each of its slots
//   shared down  32 rows of one shared expert      -> fp32 partial of y
//   routed down  32 rows of D of one expert        -> p (D h) of each of its slots
//   combine      (no weights) 32 latent columns    -> u = sum over a token's slots, in slot order
//   up           16 rows of W_up                   -> y
//
// and every block takes the next item from a counter (a ticket) until none is
// left.  An item waits (on counters in global memory) only for items of lower
// tickets, and a block works its tickets off in order, so the lowest unfinished
// ticket can always proceed, whatever number of blocks is resident: there is no
// grid barrier and no co-residency requirement.  The weights of an item depend
// on nothing but its ticket (for routed ones: and the selection), so a block's
// producer warps keep the next items' tiles in flight while its other warps
// still wait for the activations: HBM does not idle between the stages.
//
// Roles (14 warps, one block per SM):
//   warps 0-7   consumers: products from shared memory, sums over the warps, epilogues
//   warp 8, 9   producers: TMA copies of 16-row (router: 4-row) tiles into a ring of 16 KB stages;
//               a stage is two boxes of 8 KB, one per producer (one thread's copies go out one
//               after another, and one thread alone would not reach HBM's rate).  Items with two
//               row groups (gate and up, or 32 rows) put one in each box; the others put two
//               successive K ranges of one row group
//   warps 10-13 loaders: bring an item's activations from global memory into one of two
//               shared-memory slots, in the form that the product wants, one set ahead
//
// Arithmetic: bf16 weights are the A operand of m16n8k16 (16 weight rows), the tokens its
// eight columns, fp32 sums.  tcgen05 would need 128 rows per tile and gains nothing here: the
// products are at a few percent of the warp-level rate, the bytes are what count.  x is bf16;
// z, H, the shared hidden and RMSNorm(u) are fp32 and enter as two bf16 terms (hi + lo, about
// 16 bits), one product each, so that no intermediate is rounded to 8 bits.  4-bit experts:
// codes become halves exactly (cvt e2m1x2), activations enter as two halves of the row scaled by a
// power of two (largest value in [2^14, 2^15)), and a block's scale multiplies its 32-wide partial
// sum in fp32.  fp32 layers: fp32 FMA.  Router: products and sums in 64 bits, because the selection
// has to be that of the scores and not of their rounding.
#include <algorithm>

#include <cuda_fp16.h>

#include "few.cuh"
#include "gemm_tc.cuh"
#include "ptx.cuh"

namespace lmoe {

namespace {
using namespace ptx;

constexpr int CONSUMERS = 8, LOADERS = 4;
constexpr int THREADS = 32 * (CONSUMERS + 2 + LOADERS);
constexpr int CT = 32 * CONSUMERS, LT = 32 * LOADERS;
constexpr int STAGE_BYTES = 16384, BOX_BYTES = 8192;
constexpr int SCALE_BOX = 512;                   // 16 rows of 32 scales (1024 values), per box
constexpr int MAX_STAGES = 12, QUEUE = 32;
constexpr int MAX_E = 1024;
constexpr int SMEM_MAX = 232448;

enum Kind { ROUTER, DOWN, ROUTE, SHARED_GU, ROUTED_GU, SHARED_DOWN, ROUTED_DOWN, COMBINE, UP, END };

// Words of the control area (zero at launch).
enum Ctl { C_STATUS = 0, C_TICKET = 32, C_ROUTER = 64, C_Z = 96, C_ROUTED = 128, C_HS = 160, C_H = 192, C_PART = 224,
           C_YS = 256, C_U = 288, C_AMAX_Z = 320, C_AMAX_X = 328, C_AMAX_H = 352, C_WORDS = C_AMAX_H + FEW_MAX_SLOTS };

struct Item {
    int kind;
    int row0, row1;      // rows of the two boxes (one row group: equal)
    int kb0, nkb;        // first k-block (128 bytes of a row) in the matrix, and their number
    int ncol;            // columns of the product in use
    int ti;              // touched-expert index, or half of the shared experts
    int out0;            // first output row
};

// A touched expert: its id, the number of its slots and the slots in token order.
struct Touched {
    int16_t expert, n, slot[FEW_MAX_T];
};

struct FewParams {
    int T, d, l, f, E, k, fs, act, standard;
    float gate_cap, up_cap, eps;
    const void *x;
    const float *bias;
    void *y, *p_out, *u_out;
    int32_t *sel;
    unsigned *ctl;
    double *r64;             // [T, E] biased scores' raw scores
    float *p32;              // [T, k]
    Touched *tab;
    float *z, *hs, *H, *part, *ysl, *u;
    int stages, slot_bytes, scales;
    int stall_test;
};

// ------------------------------------------------------------------ activations
// How an item's activations lie in a slot: `planes` arrays (hi, lo) of ncol
// rows of Kseg values, row stride `stride` bytes; a row longer than a slot holds
// comes in nseg segments.
struct ActPlan {
    int K, eb, planes, kseg, nseg, stride, key;
};

enum Wt { W_BF16, W_MX4, W_F32 };    // weights of the routed experts; the others are W_F32 or bf16

// Row stride: products read 8 rows at 16-byte pieces (ldmatrix), or for 4-bit
// weights two rows at 64 bytes per eight lanes; either way the rows of one
// access fall in distinct banks.
__host__ __device__ __forceinline__ int act_stride(int K, int eb, bool mx4)
{
    return (K * eb + 127) / 128 * 128 + (mx4 ? 64 : 16);
}

template <int WT>
__device__ __forceinline__ ActPlan act_plan(const FewParams &p, const Item &it)
{
    ActPlan a;
    const bool from_x = it.kind <= SHARED_GU || (it.kind == ROUTED_GU && p.standard);
    const bool mx4 = WT == W_MX4 && (it.kind == ROUTED_GU || it.kind == ROUTED_DOWN);
    a.eb = WT == W_F32 ? 4 : 2;
    a.planes = WT == W_F32 || (from_x && !mx4) ? 1 : 2;
    switch (it.kind) {
    case ROUTED_GU: a.K = p.l; a.key = from_x && !mx4 ? 0 : 1; break;
    case SHARED_DOWN: a.K = p.fs; a.key = 2 + it.ti; break;
    case UP: a.K = p.l; a.key = 4; break;
    case ROUTED_DOWN: a.K = p.f; a.key = 5 + it.ti; break;
    default: a.K = p.d; a.key = 0;
    }
    a.kseg = a.K;
    a.nseg = 1;
    if (it.ncol * a.planes * act_stride(a.K, a.eb, mx4) > p.slot_bytes) {
        // whole steps of 1024 values (a stage holds 128 to 1024), as many as fit
        const int per = p.slot_bytes / (it.ncol * a.planes) - 64;
        a.kseg = per / (1024 * a.eb) * 1024;
        a.nseg = (a.K + a.kseg - 1) / a.kseg;
    }
    a.stride = act_stride(a.kseg, a.eb, mx4);
    return a;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Store four values at column c of a row as fp32, or as the hi and lo terms.
enum Form { F_F32, F_BF16X2, F_F16X2 };
template <int FORM>
__device__ __forceinline__ void put4(uint32_t row, uint32_t plane, int c, float4 v)
{
    if (FORM == F_F32) {
        sts128(row + 4u * c, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
    } else if (FORM == F_BF16X2) {
        const uint32_t h0 = pack_bf16(v.x, v.y), h1 = pack_bf16(v.z, v.w);
        sts64(row + 2u * c, h0, h1);
        sts64(row + plane + 2u * c,
              pack_bf16(v.x - __uint_as_float(h0 << 16), v.y - __uint_as_float(h0 & 0xffff0000u)),
              pack_bf16(v.z - __uint_as_float(h1 << 16), v.w - __uint_as_float(h1 & 0xffff0000u)));
    } else {
        const uint32_t h0 = pack_f16(v.x, v.y), h1 = pack_f16(v.z, v.w);
        const __half2 g0 = *reinterpret_cast<const __half2 *>(&h0), g1 = *reinterpret_cast<const __half2 *>(&h1);
        sts64(row + 2u * c, h0, h1);
        sts64(row + plane + 2u * c, pack_f16(v.x - __low2float(g0), v.y - __high2float(g0)),
              pack_f16(v.z - __low2float(g1), v.w - __high2float(g1)));
    }
}

// Power of two that brings a row of largest magnitude `amax` into [2^14, 2^15),
// and its inverse; both exact normal numbers for any amax.
__device__ __forceinline__ float f16_scale(float amax, float *inverse)
{
    int e = (int)(__float_as_uint(amax) >> 23);
    e = e < 15 ? 15 : e;
    *inverse = __uint_as_float((uint32_t)(e - 14) << 23);
    return __uint_as_float((uint32_t)(268 - e) << 23);
}

__device__ __forceinline__ float4 scaled(float4 v, float s) { return make_float4(v.x * s, v.y * s, v.z * s, v.w * s); }

// One row of `n` fp32 values (a multiple of 32) into the slot, by the loader threads.
template <int FORM>
__device__ __forceinline__ void load_row(uint32_t row, uint32_t plane, const float *src, int n, float s, int tid)
{
    const float4 *v = reinterpret_cast<const float4 *>(src);
    const int n4 = n / 4;
    int c = tid;
    for (; c + 3 * LT < n4; c += 4 * LT) {
        float4 t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = __ldcg(v + c + i * LT);
#pragma unroll
        for (int i = 0; i < 4; ++i) put4<FORM>(row, plane, 4 * (c + i * LT), scaled(t[i], s));
    }
    for (; c < n4; c += LT) put4<FORM>(row, plane, 4 * c, scaled(__ldcg(v + c), s));
}

// One row of tokens x (bf16) as fp32 scaled terms, for 4-bit experts at the model width.
__device__ __forceinline__ void load_row_bf16_scaled(uint32_t row, uint32_t plane, const bf16 *src, int n, float s,
                                                     int tid)
{
    for (int c = tid; c < n / 4; c += LT) {
        const uint2 w = *reinterpret_cast<const uint2 *>(src + 4 * c);
        put4<F_F16X2>(row, plane, 4 * c,
                      make_float4(__uint_as_float(w.x << 16) * s, __uint_as_float(w.x & 0xffff0000u) * s,
                                  __uint_as_float(w.y << 16) * s, __uint_as_float(w.y & 0xffff0000u) * s));
    }
}

// Wait until a counter reaches `want`; gives up on the limit, on another
// role's abort, or when any block has recorded a failure.
__device__ __forceinline__ bool wait_count(const unsigned *ctl, int word, unsigned want, volatile int *abort)
{
    if (ld_acquire(ctl + word) >= want) return true;
    const long long t0 = clock64();
    for (;;) {
        __nanosleep(32);
        if (ld_acquire(ctl + word) >= want) return true;
        if (*abort || ld_acquire(ctl + C_STATUS) != 0u || clock64() - t0 > WAIT_LIMIT_CYCLES) return false;
    }
}

// Order-preserving 64-bit key of a double (-0 counts as 0).
__device__ __forceinline__ unsigned long long key64(double v)
{
    const unsigned long long u = (unsigned long long)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// Barrier of the warps of one role (an mbarrier with one arrival per warp):
// bounded, unlike bar.sync, so that a role whose peer gave up still ends.
struct RoleBarrier {
    uint32_t bar, parity;
    const volatile int *abort;
    __device__ __forceinline__ bool sync()
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
        const bool ok = mbar_wait(bar, parity, abort);
        parity ^= 1u;
        return ok;
    }
};

struct Shared {
    uint32_t ring, scales, act, full, empty, act_full, act_empty, cons, load;   // shared-memory addresses
    float *red;              // [2][8 warps][16 rows][8 columns]
    Touched *tab;
    Item *queue;
    int2 *meta;              // per stage: queue index, chunk
    float *inv;              // [2 slots][8]: inverse of the activations' scale
    float *lred;             // loaders' sums [4]
    // [0] abort, [1] items published, [2] stages issued by A, [4] stages consumed,
    // [8, 16) scan, [16, 20) items passed by each loader, [20] by B
    int *flags;
};

// ------------------------------------------------------------------ items
struct Counts {
    int router, down, shared_gu, routed_gu, shared_down, routed_down, combine, up, touched;
};

template <int WT> constexpr int k_elems() { return WT == W_F32 ? 32 : 64; }   // values per 128-byte k-block

template <int WT>
__device__ __forceinline__ bool decode(const FewParams &p, const Counts &n, const Touched *tab, unsigned tk, Item *it)
{
    constexpr int KE = k_elems<WT>();
    int i = (int)tk;
    it->ti = 0;
    it->kb0 = 0;
    it->ncol = p.T;
    it->row1 = it->row0 = it->out0 = 0;
    it->nkb = 0;
    if (i < n.router) {
        it->kind = ROUTER; it->row0 = it->row1 = it->out0 = 4 * i; it->nkb = p.d / 32;
        return true;
    }
    i -= n.router;
    if (i < n.down) {
        it->kind = DOWN; it->row0 = it->row1 = it->out0 = 16 * i; it->nkb = p.d / KE;
        return true;
    }
    i -= n.down;
    if (i < 1) {
        it->kind = ROUTE;
        return true;
    }
    i -= 1;
    if (i < n.shared_gu) {      // gate and up rows interleaved in blocks of 64
        it->kind = SHARED_GU; it->out0 = 16 * i; it->nkb = p.d / KE;
        it->row0 = 128 * (i / 4) + 16 * (i % 4); it->row1 = it->row0 + 64;
        return true;
    }
    i -= n.shared_gu;
    if (i < n.routed_gu) {
        const int per = p.f / 16, j = i % per;
        it->kind = ROUTED_GU; it->ti = i / per; it->out0 = 16 * j;
        it->nkb = WT == W_MX4 ? (p.l + 255) / 256 : p.l / KE;
        it->row0 = tab[it->ti].expert * 2 * p.f + 128 * (j / 4) + 16 * (j % 4); it->row1 = it->row0 + 64;
        return true;
    }
    i -= n.routed_gu;
    if (i < n.shared_down) {
        const int per = p.d / 32;
        it->kind = SHARED_DOWN; it->ti = i / per; it->row0 = it->out0 = 32 * (i % per); it->row1 = it->row0 + 16;
        it->nkb = p.fs / KE; it->kb0 = it->ti * it->nkb;
        return true;
    }
    i -= n.shared_down;
    if (i < n.routed_down) {
        const int per = p.l / 32;
        it->kind = ROUTED_DOWN; it->ti = i / per; it->out0 = 32 * (i % per);
        it->row0 = tab[it->ti].expert * p.l + it->out0; it->row1 = it->row0 + 16;
        it->nkb = WT == W_MX4 ? (p.f + 255) / 256 : p.f / KE;
        it->ncol = tab[it->ti].n;
        return true;
    }
    i -= n.routed_down;
    if (i < n.combine) {
        it->kind = COMBINE; it->out0 = 32 * i;
        return true;
    }
    i -= n.combine;
    if (i < n.up) {
        it->kind = UP; it->row0 = it->row1 = it->out0 = 16 * i; it->nkb = p.l / KE; it->kb0 = 2 * p.fs / KE;
        return true;
    }
    it->kind = END;
    return false;
}

__device__ __forceinline__ bool weightless(int kind) { return kind == ROUTE || kind == COMBINE || kind == END; }
__device__ __forceinline__ bool two_groups(int kind)
{
    return kind == SHARED_GU || kind == ROUTED_GU || kind == SHARED_DOWN || kind == ROUTED_DOWN;
}
// k-blocks per box
__device__ __forceinline__ int box_kb(int kind) { return kind == ROUTER ? 16 : 4; }
__device__ __forceinline__ int chunks(const Item &it)
{
    const int per = box_kb(it.kind) * (two_groups(it.kind) ? 1 : 2);
    return weightless(it.kind) ? 1 : (it.nkb + per - 1) / per;
}

// ------------------------------------------------------------------ consumers
struct Consumer {
    int warp, lane, s;
    uint32_t ph;
    int set;                 // activation sets taken so far - 1
    int cur_key, cur_seg;
    int parity;              // reduction buffer
};

// Sum of the warps' partial products: thread (row, column) of 16 x 8, warps [w0, w0 + n).
__device__ __forceinline__ float red_sum(const float *red, int w0, int n, int cell)
{
    float v = 0.f;
    for (int w = w0; w < w0 + n; ++w) v += red[w * 128 + cell];
    return v;
}

template <int WT>
__device__ __forceinline__ float token_value(const void *x, int64_t i)
{
    return WT == W_F32 ? ((const float *)x)[i] : __bfloat162float(((const bf16 *)x)[i]);
}
template <int WT>
__device__ __forceinline__ void store_token(void *x, int64_t i, float v)
{
    if (WT == W_F32) ((float *)x)[i] = v;
    else ((bf16 *)x)[i] = __float2bfloat16_rn(v);
}

// Selection of every token, its weights, and the touched experts in ascending
// order with their slots.  One warp per token: k rounds of a warp maximum over
// 64-bit score keys, lowest index first among equals.
template <int WT>
__device__ __noinline__ bool route_item(const FewParams &p, const Shared &sh, RoleBarrier &bar, int warp, int lane)
{
    constexpr unsigned FULL = 0xffffffffu;
    uint8_t *slot_of = reinterpret_cast<uint8_t *>(sh.red);       // [8 tokens][MAX_E]: slot + 1
    const int tid = warp * 32 + lane;
    for (int i = tid; i < FEW_MAX_T * MAX_E / 4; i += CT) reinterpret_cast<uint32_t *>(slot_of)[i] = 0u;
    if (!bar.sync()) return false;
    if (warp < p.T) {
        const int t = warp;
        const double *r = p.r64 + (int64_t)t * p.E;
        unsigned long long key[MAX_E / 32];
#pragma unroll
        for (int j = 0; j < MAX_E / 32; ++j) {
            const int e = lane + 32 * j;
            key[j] = e < p.E ? key64(__ldcg(r + e) + (double)p.bias[e]) : 0ull;   // real keys > 0 unless -NaN
        }
        unsigned long long best = 0ull;
        int at = lane;
        auto rescan = [&]() {
            best = 0ull;
            at = MAX_E;
#pragma unroll
            for (int j = 0; j < MAX_E / 32; ++j)
                if (key[j] > best) {
                    best = key[j];
                    at = lane + 32 * j;
                }
        };
        rescan();
        int mine0 = 0, mine1 = 0;
        for (int i = 0; i < p.k; ++i) {
            const uint32_t hi = (uint32_t)(best >> 32);
            const uint32_t mh = __reduce_max_sync(FULL, hi);
            const uint32_t lo = hi == mh ? (uint32_t)best : 0u;
            const uint32_t ml = __reduce_max_sync(FULL, lo);
            const unsigned cand = hi == mh && lo == ml ? (unsigned)at : (unsigned)MAX_E;
            const int e = (int)__reduce_min_sync(FULL, cand) & (MAX_E - 1);
            if ((i & 31) == lane) {
                if (i < 32) mine0 = e;
                else mine1 = e;
            }
            if ((e & 31) == lane) {
#pragma unroll
                for (int j = 0; j < MAX_E / 32; ++j)
                    if (e == lane + 32 * j) key[j] = 0ull;
                rescan();
            }
            if (lane == 0) slot_of[t * MAX_E + e] = (uint8_t)(i + 1);
        }
        const double r0 = lane < p.k ? __ldcg(r + mine0) : 0.0, r1 = lane + 32 < p.k ? __ldcg(r + mine1) : 0.0;
        double sum = r0 + r1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = lane + 32 * h;
            if (j < p.k) {
                const float pv = (float)((h ? r1 : r0) / sum);
                p.sel[t * p.k + j] = h ? mine1 : mine0;
                p.p32[t * p.k + j] = pv;
                store_token<WT>(p.p_out, t * p.k + j, pv);
            }
        }
        if (WT == W_MX4 && p.standard) {      // the routed experts read x itself: its largest magnitude
            float m = 0.f;
            for (int c = lane; c < p.d; c += 32) m = fmaxf(m, fabsf(token_value<WT>(p.x, (int64_t)t * p.d + c)));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
            if (lane == 0) p.ctl[C_AMAX_X + t] = __float_as_uint(m);
        }
    }
    if (!bar.sync()) return false;
    // touched experts: thread i takes experts [4 i, 4 i + 4)
    int mask[4], mine = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        mask[q] = 0;
        for (int t = 0; t < p.T; ++t) mask[q] |= (slot_of[t * MAX_E + 4 * tid + q] != 0) << t;
        mine += mask[q] != 0;
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl += v;
    }
    int *scan = sh.flags + 8;
    if (lane == 31) scan[warp] = incl;
    if (!bar.sync()) return false;
    int at = incl - mine;
    for (int w = 0; w < warp; ++w) at += scan[w];
    for (int q = 0; q < 4; ++q)
        if (mask[q]) {
            Touched e;
            e.expert = (int16_t)(4 * tid + q);
            e.n = (int16_t)__popc(mask[q]);
            int c = 0;
            for (int t = 0; t < FEW_MAX_T; ++t) e.slot[t] = -1;
            for (int t = 0; t < p.T; ++t)
                if (mask[q] >> t & 1) e.slot[c++] = (int16_t)(t * p.k + slot_of[t * MAX_E + 4 * tid + q] - 1);
            p.tab[at++] = e;
        }
    int total = 0;
    for (int w = 0; w < CONSUMERS; ++w) total += scan[w];
    if (!bar.sync()) return false;
    if (tid == 0) red_release(p.ctl + C_ROUTED, (unsigned)total);   // never 0: T, k >= 1
    return true;
}

template <int WT>
__device__ __forceinline__ void combine_item(const FewParams &p, const Item &it, int warp, int lane)
{
    const int t = warp, c = it.out0 + lane;
    if (t < p.T) {
        const float *src = p.ysl + (int64_t)t * p.k * p.l + c;
        float u = 0.f;
        int j = 0;
        for (; j + 8 <= p.k; j += 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __ldcg(src + (int64_t)(j + i) * p.l);
#pragma unroll
            for (int i = 0; i < 8; ++i) u += v[i];
        }
        for (; j < p.k; ++j) u += __ldcg(src + (int64_t)j * p.l);
        store_token<WT>(p.u_out, (int64_t)t * p.l + c, u);
        if (p.standard) {
            const float *q = p.part + (int64_t)t * p.d + c;
            store_token<WT>(p.y, (int64_t)t * p.d + c, __ldcg(q) + __ldcg(q + (int64_t)p.T * p.d) + u);
        } else {
            p.u[(int64_t)t * p.l + c] = u;
        }
    }
    __syncwarp();
    if (lane == 0) red_release(p.ctl + C_U, 1u);
}

// ------------------------------------------------------------------ the kernel
template <int WT>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewParams p)
{
    constexpr int KE = k_elems<WT>();
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *g = smem_raw + (base - raw);
    Shared sh;
    uint32_t o = 0;
    sh.ring = base; o += (uint32_t)p.stages * STAGE_BYTES;
    sh.scales = base + o; o += p.scales ? (uint32_t)p.stages * 2 * SCALE_BOX : 0u;
    sh.act = base + o; o += 2u * (uint32_t)p.slot_bytes;
    sh.red = reinterpret_cast<float *>(g + o); o += 2 * 8 * 128 * 4;
    sh.tab = reinterpret_cast<Touched *>(g + o); o += sizeof(Touched) * FEW_MAX_SLOTS;
    sh.queue = reinterpret_cast<Item *>(g + o); o += sizeof(Item) * QUEUE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(g + o); o += 8 * (2 * MAX_STAGES + 6);
    sh.meta = reinterpret_cast<int2 *>(g + o); o += sizeof(int2) * MAX_STAGES;
    sh.inv = reinterpret_cast<float *>(g + o); o += 64;
    sh.lred = reinterpret_cast<float *>(g + o); o += 64;
    sh.flags = reinterpret_cast<int *>(g + o);
    sh.full = smem_u32(bars);
    sh.empty = sh.full + 8u * MAX_STAGES;
    sh.act_full = sh.empty + 8u * MAX_STAGES;
    sh.act_empty = sh.act_full + 16u;
    sh.cons = sh.act_empty + 16u;
    sh.load = sh.cons + 8u;
    volatile int *abort = sh.flags;
    volatile int *published = sh.flags + 1, *issued_a = sh.flags + 2, *passed = sh.flags + 16;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.stages;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(sh.full + 8u * s, 1);
            mbar_init(sh.empty + 8u * s, CONSUMERS);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(sh.act_full + 8u * s, LOADERS);
            mbar_init(sh.act_empty + 8u * s, CONSUMERS);
        }
        mbar_init(sh.cons, CONSUMERS);
        mbar_init(sh.load, LOADERS);
        for (int i = 0; i < 24; ++i) sh.flags[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();

    Counts n;
    n.router = (p.E + 3) / 4;
    n.down = p.standard ? 0 : p.l / 16;
    n.shared_gu = 2 * p.fs / 16;
    n.shared_down = 2 * (p.d / 32);
    n.combine = p.l / 32;
    n.up = p.standard ? 0 : p.d / 16;
    n.touched = n.routed_gu = n.routed_down = 0;
    auto give_up = [&](int code) {
        atomicOr(p.ctl + C_STATUS, (unsigned)code);
        *abort = 1;
    };
    auto with_touched = [&](int touched) {
        n.touched = touched;
        n.routed_gu = touched * (p.f / 16);
        n.routed_down = touched * (p.l / 32);
    };

    if (warp == CONSUMERS) {
        // ------------------------------------------------------------ producer A: tickets, box 0
        unsigned next = 0;
        if (lane == 0) next = atomicAdd(p.ctl + C_TICKET, 1u);
        const unsigned fixed = (unsigned)(n.router + n.down + 1 + n.shared_gu);   // tickets that need no selection
        int q = 0, s = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        while (ok) {
            const unsigned tk = __shfl_sync(0xffffffffu, next, 0);
            if (tk >= fixed && n.touched == 0) {
                int touched = 0;
                if (lane == 0) touched = wait_count(p.ctl, C_ROUTED, 1u, abort) ? (int)ld_acquire(p.ctl + C_ROUTED) : 0;
                touched = __shfl_sync(0xffffffffu, touched, 0);
                if (touched == 0) {
                    if (lane == 0) give_up(0x10);
                    break;
                }
                with_touched(touched);
                const uint32_t *src = reinterpret_cast<const uint32_t *>(p.tab);
                uint32_t *dst = reinterpret_cast<uint32_t *>(sh.tab);
                const int words = touched * (int)(sizeof(Touched) / 4);
                for (int i = lane; i < words; i += 32) dst[i] = __ldcg(src + i);
                __threadfence_block();
                __syncwarp();
            }
            Item it;
            const bool more = decode<WT>(p, n, sh.tab, tk, &it);
            if (lane == 0) {
                if (more) next = atomicAdd(p.ctl + C_TICKET, 1u);   // used in the next round
                // the entry's previous item must be behind every reader (rarely a wait)
                const long long t0 = clock64();
                for (int r = 0; r < LOADERS + 1 && ok; ++r)
                    while (q - passed[r] >= QUEUE && ok)
                        if (*abort || clock64() - t0 > WAIT_LIMIT_CYCLES) ok = false;
                if (!ok) give_up(0x1);
                sh.queue[q % QUEUE] = it;
                __threadfence_block();
                *published = q + 1;
                const int nc = chunks(it), kb = box_kb(it.kind);
                const bool two = two_groups(it.kind), light = weightless(it.kind);
                const bool mx4 = WT == W_MX4 && (it.kind == ROUTED_GU || it.kind == ROUTED_DOWN);
                const CUtensorMap *map = it.kind == ROUTER      ? &maps.router
                                         : it.kind == DOWN      ? &maps.down
                                         : it.kind == SHARED_GU ? &maps.shared_gu
                                         : it.kind == ROUTED_GU ? &maps.routed_gu
                                         : it.kind == ROUTED_DOWN ? &maps.routed_down
                                                                  : &maps.cat;
                for (int c = 0; c < nc && ok; ++c) {
                    if (!mbar_wait(sh.empty + 8u * s, ph ^ 1u, abort)) {
                        give_up(0x1);
                        ok = false;
                        break;
                    }
                    sh.meta[s] = make_int2(q, c);
                    const uint32_t fb = sh.full + 8u * s;
                    if (light) {
                        mbar_arrive(fb);
                    } else {
                        const int kb0 = two ? c * kb : 2 * c * kb;
                        const bool second = two || kb0 + kb < it.nkb;
                        mbar_expect_tx(fb, (uint32_t)((BOX_BYTES + (mx4 ? SCALE_BOX : 0)) * (second ? 2 : 1)));
                        tma_load_3d(sh.ring + (uint32_t)s * STAGE_BYTES, map, fb, it.row0, it.kb0 + kb0);
                        if (mx4)
                            tma_load_2d(sh.scales + (uint32_t)s * 2 * SCALE_BOX,
                                        it.kind == ROUTED_GU ? &maps.routed_gu_scales : &maps.routed_down_scales, fb,
                                        32 * c, it.row0);
                    }
                    *issued_a = ++issued;
                    if (++s == S) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
            ++q;
            if (!more) break;
        }
    } else if (warp == CONSUMERS + 1) {
        // ------------------------------------------------------------ producer B: box 1
        if (lane == 0) {
            // Box 1 of a stage follows producer A's box 0: A has waited for the slot, and
            // A's expected bytes keep the consumers from releasing it without this box.
            int s = 0, stage = 0;
            bool ok = true;
            for (int q = 0; ok; ++q) {
                passed[LOADERS] = q;
                const long long t0 = clock64();
                while (*published <= q && ok) {
                    __nanosleep(20);
                    if (*abort || clock64() - t0 > 2 * WAIT_LIMIT_CYCLES) ok = false;
                }
                if (!ok) {
                    give_up(0x2);
                    break;
                }
                __threadfence_block();
                const Item it = sh.queue[q % QUEUE];
                if (it.kind == END) break;
                const int nc = chunks(it), kb = box_kb(it.kind);
                const bool two = two_groups(it.kind), light = weightless(it.kind);
                const bool mx4 = WT == W_MX4 && (it.kind == ROUTED_GU || it.kind == ROUTED_DOWN);
                const CUtensorMap *map = it.kind == ROUTER      ? &maps.router
                                         : it.kind == DOWN      ? &maps.down
                                         : it.kind == SHARED_GU ? &maps.shared_gu
                                         : it.kind == ROUTED_GU ? &maps.routed_gu
                                         : it.kind == ROUTED_DOWN ? &maps.routed_down
                                                                  : &maps.cat;
                for (int c = 0; c < nc && ok; ++c, ++stage) {
                    const long long t1 = clock64();
                    while (*issued_a <= stage && ok) {
                        __nanosleep(20);
                        if (*abort || clock64() - t1 > WAIT_LIMIT_CYCLES) ok = false;
                    }
                    if (!ok) {
                        give_up(0x2);
                        break;
                    }
                    const int kb0 = two ? c * kb : (2 * c + 1) * kb;
                    if (!light && kb0 < it.nkb) {
                        const uint32_t fb = sh.full + 8u * s;
                        tma_load_3d(sh.ring + (uint32_t)s * STAGE_BYTES + BOX_BYTES, map, fb, it.row1, it.kb0 + kb0);
                        if (mx4)
                            tma_load_2d(sh.scales + (uint32_t)s * 2 * SCALE_BOX + SCALE_BOX,
                                        it.kind == ROUTED_GU ? &maps.routed_gu_scales : &maps.routed_down_scales, fb,
                                        32 * c, it.row1);
                    }
                    if (++s == S) s = 0;
                }
            }
        }
    } else if (warp > CONSUMERS + 1) {
        // ------------------------------------------------------------ loaders
        const int tid = threadIdx.x - 32 * (CONSUMERS + 2), lw = warp - CONSUMERS - 2;
        RoleBarrier bar = {sh.load, 0u, abort};
        int set = 0, cur_key = -1, cur_seg = -1;
        bool ok = true;
        for (int q = 0; ok; ++q) {
            int good = 1;
            if (lane == 0) passed[lw] = q;
            if (lane == 0) {
                const long long t0 = clock64();
                while (*published <= q && good) {
                    __nanosleep(20);
                    if (*abort || clock64() - t0 > 2 * WAIT_LIMIT_CYCLES) good = 0;
                }
                __threadfence_block();
            }
            ok = __shfl_sync(0xffffffffu, good, 0) != 0;
            if (!ok) {
                if (lane == 0) give_up(0x4);
                break;
            }
            const Item it = sh.queue[q % QUEUE];
            if (it.kind == END) break;
            if (weightless(it.kind)) continue;
            const ActPlan a = act_plan<WT>(p, it);
            const bool mx4 = WT == W_MX4 && (it.kind == ROUTED_GU || it.kind == ROUTED_DOWN);
            for (int seg = 0; seg < a.nseg && ok; ++seg) {
                if (a.key == cur_key && seg == cur_seg) continue;
                const bool same_rows = a.key == cur_key;
                cur_key = a.key;
                cur_seg = seg;
                const int slot = set & 1;
                if (lane == 0) {
                    good = mbar_wait(sh.act_empty + 8u * slot, (uint32_t)((set >> 1) & 1) ^ 1u, abort);
                    // the producers of these values, once per set of rows
                    if (good && !same_rows) {
                        if (it.kind == ROUTED_GU && !p.standard) good = wait_count(p.ctl, C_Z, 4u * n.down, abort);
                        // (the failure-detection test waits for one count too many)
                        if (it.kind == SHARED_DOWN)
                            good = wait_count(p.ctl, C_HS, 4u * n.shared_gu + (p.stall_test ? 1u : 0u), abort);
                        if (it.kind == ROUTED_DOWN)
                            good = wait_count(p.ctl, C_H, 4u * ld_acquire(p.ctl + C_ROUTED) * (p.f / 16), abort);
                        if (it.kind == UP)
                            good = wait_count(p.ctl, C_U, 8u * n.combine, abort) &&
                                   wait_count(p.ctl, C_PART, 8u * n.shared_down, abort);
                    }
                }
                ok = __shfl_sync(0xffffffffu, good, 0) != 0;
                if (!ok) {
                    if (lane == 0) give_up(0x4);
                    break;
                }
                const uint32_t dst = sh.act + (uint32_t)(slot * p.slot_bytes);
                const uint32_t plane = (uint32_t)(it.ncol * a.stride);
                const int k0 = seg * a.kseg, kn = a.K - k0 < a.kseg ? a.K - k0 : a.kseg;
                float *inv = sh.inv + 8 * slot;
                if (it.kind == UP) {
                    // RMSNorm: the sum of squares over the whole row, in a fixed order
                    for (int t = 0; t < it.ncol; ++t) {
                        const float4 *v = reinterpret_cast<const float4 *>(p.u + (int64_t)t * p.l);
                        float ss = 0.f;
#pragma unroll 4
                        for (int c = tid; c < p.l / 4; c += LT) {
                            const float4 w = __ldcg(v + c);
                            ss += w.x * w.x + w.y * w.y + w.z * w.z + w.w * w.w;
                        }
#pragma unroll
                        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                        if (lane == 0) sh.lred[lw] = ss;
                        if (!(ok = bar.sync())) break;
                        const float rms = 1.0f / sqrtf((sh.lred[0] + sh.lred[1] + sh.lred[2] + sh.lred[3]) / (float)p.l +
                                                       p.eps);
                        if (!(ok = bar.sync())) break;
                        const uint32_t row = dst + (uint32_t)(t * a.stride);
                        const float *src = p.u + (int64_t)t * p.l + k0;
                        if (WT == W_F32) load_row<F_F32>(row, plane, src, kn, rms, tid);
                        else load_row<F_BF16X2>(row, plane, src, kn, rms, tid);
                    }
                } else {
                    for (int t = 0; t < it.ncol; ++t) {
                        const uint32_t row = dst + (uint32_t)(t * a.stride);
                        const float *src = nullptr;
                        const unsigned *amax = nullptr;
                        if (it.kind == ROUTED_GU && !p.standard) {
                            src = p.z + (int64_t)t * p.l;
                            amax = p.ctl + C_AMAX_Z + t;
                        } else if (it.kind == SHARED_DOWN) {
                            src = p.hs + (int64_t)t * 2 * p.fs + it.ti * p.fs;
                        } else if (it.kind == ROUTED_DOWN) {
                            const int sl = sh.tab[it.ti].slot[t];
                            src = p.H + (int64_t)sl * p.f;
                            amax = p.ctl + C_AMAX_H + sl;
                        } else if (mx4) {
                            amax = p.ctl + C_AMAX_X + t;
                        }
                        if (!src && !mx4) {          // x as it is
                            if (WT == W_F32) {
                                const uint4 *v = reinterpret_cast<const uint4 *>((const float *)p.x + (int64_t)t * p.d + k0);
                                for (int c = tid; c < kn / 4; c += LT) {
                                    const uint4 w = v[c];
                                    sts128(row + 16u * c, w.x, w.y, w.z, w.w);
                                }
                            } else {
                                const uint4 *v = reinterpret_cast<const uint4 *>((const bf16 *)p.x + (int64_t)t * p.d + k0);
                                for (int c = tid; c < kn / 8; c += LT) {
                                    const uint4 w = v[c];
                                    sts128(row + 16u * c, w.x, w.y, w.z, w.w);
                                }
                            }
                        } else if (mx4) {
                            float back;
                            const float sc = f16_scale(__uint_as_float(__ldcg(amax)), &back);
                            if (tid == 0) inv[t] = back;
                            if (src) load_row<F_F16X2>(row, plane, src + k0, kn, sc, tid);
                            else load_row_bf16_scaled(row, plane, (const bf16 *)p.x + (int64_t)t * p.d + k0, kn, sc, tid);
                        } else if (WT == W_F32) {
                            load_row<F_F32>(row, plane, src + k0, kn, 1.f, tid);
                        } else {
                            load_row<F_BF16X2>(row, plane, src + k0, kn, 1.f, tid);
                        }
                    }
                }
                if (!ok) {
                    if (lane == 0) give_up(0x4);
                    break;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sh.act_full + 8u * slot);
                ++set;
            }
        }
    } else {
        // ------------------------------------------------------------ consumers
        RoleBarrier bar = {sh.cons, 0u, abort};
        int s = 0, set = -1, cur_key = -1, cur_seg = -1, par = 0, consumed = 0;
        uint32_t ph = 0;
        const int box = warp >> 2, sub = warp & 3;
        const int gid = lane >> 2, c4 = lane & 3;
        bool ok = true;
        for (;;) {
            if (!mbar_wait(sh.full + 8u * s, ph, abort)) {
                if (lane == 0) give_up(0x8);
                break;
            }
            const int2 m0 = sh.meta[s];
            const Item it = sh.queue[m0.x % QUEUE];
            auto release = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(sh.empty + 8u * s);
                if (threadIdx.x == 0) sh.flags[4] = ++consumed;
                if (++s == S) {
                    s = 0;
                    ph ^= 1u;
                }
            };
            if (it.kind == END) {
                release();
                break;
            }
            if (weightless(it.kind)) {
                int good = 1;
                if (lane == 0) {
                    if (it.kind == ROUTE) {
                        good = wait_count(p.ctl, C_ROUTER, (unsigned)n.router, abort);
                    } else {
                        good = wait_count(p.ctl, C_YS, 8u * ld_acquire(p.ctl + C_ROUTED) * (p.l / 32), abort);
                        if (good && p.standard) good = wait_count(p.ctl, C_PART, 8u * n.shared_down, abort);
                    }
                }
                ok = __shfl_sync(0xffffffffu, good, 0) != 0;
                if (ok && it.kind == ROUTE) ok = bar.sync() && route_item<WT>(p, sh, bar, warp, lane);
                else if (ok) combine_item<WT>(p, it, warp, lane);
                if (!ok) break;
                release();
                continue;
            }

            const ActPlan a = act_plan<WT>(p, it);
            const bool two = two_groups(it.kind);
            const int kb = box_kb(it.kind), nc = chunks(it);
            const int col = gid < it.ncol ? gid : it.ncol - 1;   // columns past the tokens repeat the last one
            // activations of the segment that holds value k; false when a wait gave up
            uint32_t act = 0;
            auto segment = [&](int k) -> bool {
                const int seg = a.nseg == 1 ? 0 : k / a.kseg;
                if (a.key != cur_key || seg != cur_seg) {
                    if (set >= 0) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sh.act_empty + 8u * (set & 1));
                    }
                    ++set;
                    cur_key = a.key;
                    cur_seg = seg;
                    if (!mbar_wait(sh.act_full + 8u * (set & 1), (uint32_t)(set >> 1) & 1u, abort)) return false;
                }
                act = sh.act + (uint32_t)((set & 1) * p.slot_bytes);
                return true;
            };
            auto next_stage = [&](int c) -> bool {
                if (c > 0 && !mbar_wait(sh.full + 8u * s, ph, abort)) return false;
                return true;
            };
            float *red = sh.red + par * 1024;

            if (it.kind == ROUTER) {
                // ---- 4 rows, 64-bit products: lane (row, 4-value piece)
                double acc[FEW_MAX_T] = {};
                const int row = lane >> 3, piece = lane & 7;
                for (int c = 0; c < nc; ++c) {
                    if (!(ok = next_stage(c) && segment(c * 1024))) break;
                    const uint32_t tile = sh.ring + (uint32_t)s * STAGE_BYTES + (uint32_t)box * BOX_BYTES;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int ko = sub * 4 + i, kblk = (2 * c + box) * 16 + ko;
                        if (kblk >= it.nkb) break;
                        const int R = ko * 4 + row;
                        const uint4 w = lds128(tile + (uint32_t)(R * 128 + ((piece ^ (R & 7)) << 4)));
                        const double w0 = __uint_as_float(w.x), w1 = __uint_as_float(w.y), w2 = __uint_as_float(w.z),
                                     w3 = __uint_as_float(w.w);
                        const int k = kblk * 32 + 4 * piece - cur_seg * a.kseg;
#pragma unroll
                        for (int t = 0; t < FEW_MAX_T; ++t)
                            if (t < p.T) {
                                float x0, x1, x2, x3;
                                if (WT == W_F32) {
                                    const uint4 v = lds128(act + (uint32_t)(t * a.stride + 4 * k));
                                    x0 = __uint_as_float(v.x); x1 = __uint_as_float(v.y);
                                    x2 = __uint_as_float(v.z); x3 = __uint_as_float(v.w);
                                } else {
                                    const uint2 v = lds64(act + (uint32_t)(t * a.stride + 2 * k));
                                    x0 = __uint_as_float(v.x << 16); x1 = __uint_as_float(v.x & 0xffff0000u);
                                    x2 = __uint_as_float(v.y << 16); x3 = __uint_as_float(v.y & 0xffff0000u);
                                }
                                acc[t] = fma(w0, (double)x0, acc[t]);
                                acc[t] = fma(w1, (double)x1, acc[t]);
                                acc[t] = fma(w2, (double)x2, acc[t]);
                                acc[t] = fma(w3, (double)x3, acc[t]);
                            }
                    }
                    release();
                }
                if (!ok) break;
                double *rd = reinterpret_cast<double *>(red);      // [8 warps][4 rows][8 tokens]
#pragma unroll
                for (int t = 0; t < FEW_MAX_T; ++t)
                    if (t < p.T) {
#pragma unroll
                        for (int off = 1; off < 8; off <<= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], off);
                        if (piece == 0) rd[warp * 32 + row * 8 + t] = acc[t];
                    }
                if (!(ok = bar.sync())) break;
                if (warp == 0) {
                    const int e = it.out0 + (lane >> 3), t = lane & 7;
                    if (e < p.E && t < p.T) {
                        double v = 0.0;
                        for (int w = 0; w < CONSUMERS; ++w) v += rd[w * 32 + lane];
                        p.r64[(int64_t)t * p.E + e] = 1.0 / (1.0 + exp(-v));
                    }
                    __syncwarp();
                    if (lane == 0) red_release(p.ctl + C_ROUTER, 1u);
                }
                par ^= 1;
                continue;
            }

            const bool mx4 = WT == W_MX4 && (it.kind == ROUTED_GU || it.kind == ROUTED_DOWN);
            if (WT == W_F32) {
                // ---- fp32: lane (4-value piece, rows rq + 4 i)
                float acc[4][FEW_MAX_T] = {};
                const int piece = lane & 7, rq = lane >> 3;
                for (int c = 0; c < nc; ++c) {
                    if (!(ok = next_stage(c) && segment(c * (two ? 128 : 256)))) break;
                    const uint32_t tile = sh.ring + (uint32_t)s * STAGE_BYTES + (uint32_t)(box * BOX_BYTES + sub * 2048);
                    const int kblk = two ? c * 4 + sub : (2 * c + box) * 4 + sub;
                    if (kblk < it.nkb) {
                        const int k = kblk * 32 + 4 * piece - cur_seg * a.kseg;
                        float4 w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int R = rq + 4 * i;
                            const uint4 v = lds128(tile + (uint32_t)(R * 128 + ((piece ^ (R & 7)) << 4)));
                            w[i] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                                               __uint_as_float(v.w));
                        }
#pragma unroll
                        for (int t = 0; t < FEW_MAX_T; ++t)
                            if (t < it.ncol) {
                                const uint4 v = lds128(act + (uint32_t)(t * a.stride + 4 * k));
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    acc[i][t] = fmaf(w[i].x, __uint_as_float(v.x), acc[i][t]);
                                    acc[i][t] = fmaf(w[i].y, __uint_as_float(v.y), acc[i][t]);
                                    acc[i][t] = fmaf(w[i].z, __uint_as_float(v.z), acc[i][t]);
                                    acc[i][t] = fmaf(w[i].w, __uint_as_float(v.w), acc[i][t]);
                                }
                            }
                    }
                    release();
                }
                if (!ok) break;
#pragma unroll
                for (int t = 0; t < FEW_MAX_T; ++t)
                    if (t < it.ncol) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
#pragma unroll
                            for (int off = 1; off < 8; off <<= 1)
                                acc[i][t] += __shfl_xor_sync(0xffffffffu, acc[i][t], off);
                            if (piece == 0) red[warp * 128 + (rq + 4 * i) * 8 + t] = acc[i][t];
                        }
                    }
            } else {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                if (mx4) {
                    // ---- 4-bit rows: a 16-byte piece of a row is one block of 32 values, eight of
                    // them (a word) per lane; the block's partial sum times its row's scale
                    const int nblk = (it.kind == ROUTED_GU ? p.l : p.f) / 32;
                    const uint32_t plane = (uint32_t)(it.ncol * a.stride);
                    for (int c = 0; c < nc; ++c) {
                        if (!(ok = next_stage(c) && segment(c * 1024))) break;
                        const uint32_t tile =
                            sh.ring + (uint32_t)s * STAGE_BYTES + (uint32_t)(box * BOX_BYTES + sub * 2048) + 128u * gid;
                        const int kblk = c * 4 + sub;
                        int nb = nblk - kblk * 8;
                        if (nb > 0) {
                            if (nb > 8) nb = 8;
                            const uint32_t sc = sh.scales + (uint32_t)(s * 2 * SCALE_BOX + box * SCALE_BOX + 32 * gid + 8 * sub);
                            const uint2 sa = lds64(sc), sb = lds64(sc + 8 * 32);
                            const uint32_t arow = act + (uint32_t)(col * a.stride + 2 * (kblk * 256 - cur_seg * a.kseg + 8 * c4));
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (j < nb) {
                                    const uint32_t off = (uint32_t)(((j ^ gid) << 4) + 4 * c4);
                                    uint32_t wa[4], wb[4];
                                    e2m1x8_to_f16(wa, lds32(tile + off));
                                    e2m1x8_to_f16(wb, lds32(tile + 1024 + off));
                                    const uint4 h = lds128(arow + 64u * j), lo = lds128(arow + plane + 64u * j);
                                    float t[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma_f16(t, wa[0], wb[0], wa[1], wb[1], h.x, h.y);
                                    mma_f16(t, wa[0], wb[0], wa[1], wb[1], lo.x, lo.y);
                                    mma_f16(t, wa[2], wb[2], wa[3], wb[3], h.z, h.w);
                                    mma_f16(t, wa[2], wb[2], wa[3], wb[3], lo.z, lo.w);
                                    // 2^(e - 127); e = 0 counts as zero (below fp32's normal range), 255 is NaN
                                    const uint32_t ea = __byte_perm(j < 4 ? sa.x : sa.y, 0, 0x4440 + (j & 3));
                                    const uint32_t eb = __byte_perm(j < 4 ? sb.x : sb.y, 0, 0x4440 + (j & 3));
                                    const float fa = __uint_as_float(ea == 255u ? 0x7fffffffu : ea << 23);
                                    const float fb = __uint_as_float(eb == 255u ? 0x7fffffffu : eb << 23);
                                    acc[0] = fmaf(t[0], fa, acc[0]);
                                    acc[1] = fmaf(t[1], fa, acc[1]);
                                    acc[2] = fmaf(t[2], fb, acc[2]);
                                    acc[3] = fmaf(t[3], fb, acc[3]);
                                }
                            }
                        }
                        release();
                    }
                } else {
                    // ---- bf16 rows: 64 values of 16 rows per k-block
                    const uint32_t plane = (uint32_t)(it.ncol * a.stride);
                    const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8, lpiece = lane >> 4;
                    const int arow = (lane & 7) < it.ncol ? (lane & 7) : it.ncol - 1;
                    for (int c = 0; c < nc; ++c) {
                        if (!(ok = next_stage(c) && segment(c * (two ? 256 : 512)))) break;
                        const uint32_t tile =
                            sh.ring + (uint32_t)s * STAGE_BYTES + (uint32_t)(box * BOX_BYTES + sub * 2048 + lrow * 128);
                        const int kblk = two ? c * 4 + sub : (2 * c + box) * 4 + sub;
                        if (kblk < it.nkb) {
                            const uint32_t arow_at =
                                act + (uint32_t)(arow * a.stride + 2 * (kblk * 64 - cur_seg * a.kseg) + 16 * (lane >> 3));
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t w0[4], w1[4], b[4];
                                ldmatrix_x4(w0, tile + (uint32_t)(((4 * h + lpiece) ^ (lrow & 7)) << 4));
                                ldmatrix_x4(w1, tile + (uint32_t)(((4 * h + 2 + lpiece) ^ (lrow & 7)) << 4));
                                ldmatrix_x4(b, arow_at + 64u * h);
                                mma_bf16(acc, w0, b[0], b[1]);
                                mma_bf16(acc, w1, b[2], b[3]);
                                if (a.planes == 2) {
                                    ldmatrix_x4(b, arow_at + plane + 64u * h);
                                    mma_bf16(acc, w0, b[0], b[1]);
                                    mma_bf16(acc, w1, b[2], b[3]);
                                }
                            }
                        }
                        release();
                    }
                }
                if (!ok) break;
                float2 *r = reinterpret_cast<float2 *>(red + warp * 128 + gid * 8 + 2 * c4);
                r[0] = make_float2(acc[0], acc[1]);
                r[32] = make_float2(acc[2], acc[3]);
            }
            if (!(ok = bar.sync())) break;

            // ---- sums over the warps, and what becomes of them
            const int cell = threadIdx.x & 127, row = cell >> 3, t = cell & 7, grp = threadIdx.x >> 7;
            const bool real = t < it.ncol;
            const float back = mx4 && real ? sh.inv[8 * (set & 1) + t] : 1.f;
            if (it.kind == SHARED_GU || it.kind == ROUTED_GU) {
                if (grp == 0) {
                    const float gv = red_sum(red, 0, 4, cell) * back, uv = red_sum(red, 4, 4, cell) * back;
                    const float h = glu_act(p.act, gv, uv, p.gate_cap, p.up_cap);
                    if (it.kind == SHARED_GU) {
                        if (real) p.hs[(int64_t)t * 2 * p.fs + it.out0 + row] = h;
                    } else {
                        int slot = -1;
#pragma unroll
                        for (int i = 0; i < FEW_MAX_T; ++i) {
                            const int v = sh.tab[it.ti].slot[i];
                            if (v >= 0 && v / p.k == t) slot = v;
                        }
                        if (slot >= 0) p.H[(int64_t)slot * p.f + it.out0 + row] = h;
                        if (WT == W_MX4) {
                            float m = slot >= 0 ? fabsf(h) : 0.f;
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            if (lane < 8 && slot >= 0) atomicMax(p.ctl + C_AMAX_H + slot, __float_as_uint(m));
                        }
                    }
                    __syncwarp();
                    if (lane == 0) red_release(p.ctl + (it.kind == SHARED_GU ? C_HS : C_H), 1u);
                }
            } else if (it.kind == DOWN || it.kind == UP) {
                if (grp == 0) {
                    const float v = red_sum(red, 0, 8, cell);
                    const int r = it.out0 + row;
                    if (it.kind == DOWN) {
                        if (real) p.z[(int64_t)t * p.l + r] = v;
                        if (WT == W_MX4) {
                            float m = real ? fabsf(v) : 0.f;
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                            if (lane < 8 && real) atomicMax(p.ctl + C_AMAX_Z + t, __float_as_uint(m));
                        }
                        __syncwarp();
                        if (lane == 0) red_release(p.ctl + C_Z, 1u);
                    } else if (real) {
                        const float *q = p.part + (int64_t)t * p.d + r;
                        store_token<WT>(p.y, (int64_t)t * p.d + r, v + (__ldcg(q) + __ldcg(q + (int64_t)p.T * p.d)));
                    }
                }
            } else {
                const float v = red_sum(red, 4 * grp, 4, cell) * back;
                const int r = it.out0 + 16 * grp + row;
                if (it.kind == SHARED_DOWN) {
                    if (real) p.part[((int64_t)it.ti * p.T + t) * p.d + r] = v;
                } else if (real) {
                    const int slot = sh.tab[it.ti].slot[t];
                    p.ysl[(int64_t)slot * p.l + r] = __ldcg(p.p32 + slot) * v;
                }
                __syncwarp();
                if (lane == 0) red_release(p.ctl + (it.kind == SHARED_DOWN ? C_PART : C_YS), 1u);
            }
            par ^= 1;
        }
        if (!ok && lane == 0) give_up(0x8);
    }

    __syncthreads();
    if (*abort && threadIdx.x == 0) {
        // copies issued but not consumed must land before the block's memory goes away
        const int issued = sh.flags[2];
        int none = 0;
        for (int i = sh.flags[4]; i < issued; ++i)
            if (!mbar_wait(sh.full + 8u * (i % S), (uint32_t)(i / S) & 1u, &none)) break;
    }
}

// ------------------------------------------------------------------ host side
size_t fixed_smem()
{
    return 1024 + 2 * 8 * 128 * 4 + sizeof(Touched) * FEW_MAX_SLOTS + sizeof(Item) * QUEUE + 8 * (2 * MAX_STAGES + 6) +
           sizeof(int2) * MAX_STAGES + 64 + 64 + 128;
}

struct FewLayout {
    size_t ctl, r64, p32, tab, z, hs, H, part, ysl, u, total;
};

FewLayout few_layout(const lmoe_config &c, int64_t T)
{
    FewLayout L;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = (o + bytes + 255) / 256 * 256;
        return at;
    };
    const size_t S = (size_t)T * c.k;
    L.ctl = take(4 * C_WORDS);
    L.r64 = take(8 * (size_t)T * c.E);
    L.p32 = take(4 * S);
    L.tab = take(sizeof(Touched) * FEW_MAX_SLOTS);
    L.z = take(c.standard ? 0 : 4 * (size_t)T * c.l);
    L.hs = take(4 * (size_t)T * 2 * c.f_shared);
    L.H = take(4 * S * c.f);
    L.part = take(8 * (size_t)T * c.d);
    L.ysl = take(4 * S * c.l);
    L.u = take(c.standard ? 0 : 4 * (size_t)T * c.l);
    L.total = o;
    return L;
}

template <int WT>
cudaError_t launch(const FewMaps &m, const FewParams &p, size_t smem, cudaStream_t s)
{
    cudaError_t e = cudaFuncSetAttribute(few_kernel<WT>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
    if (e != cudaSuccess) return e;
    few_kernel<WT><<<tc_num_sms(), THREADS, smem, s>>>(m, p);
    return cudaGetLastError();
}
}  // namespace

size_t few_workspace_bytes(const lmoe_config &c, int64_t T) { return T > 0 ? few_layout(c, T).total : 0; }

bool few_make_maps(const lmoe_config &c, const FewWeights &w, FewMaps *m)
{
    const bool f32 = c.dtype == LMOE_F32;
    const CUtensorMapDataType ty = f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint32_t ke = f32 ? 32 : 64;
    const uint64_t eb = f32 ? 4 : 2;
    // rows of K values in 128-byte k-blocks: a box is 16 rows of four of them
    auto rows = [&](CUtensorMap *t, const void *base, uint64_t K, uint64_t nrows) {
        return tc_encode_map(t, ty, base, ke, nrows, K / ke, K * eb, 128, ke, 16, 4, true);
    };
    auto codes = [&](CUtensorMap *t, const void *base, uint64_t K, uint64_t nrows) {
        return tc_encode_map(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 128, nrows, (K / 2 + 127) / 128, K / 2, 128, 128, 16, 4,
                             true);
    };
    auto scales = [&](CUtensorMap *t, const void *base, uint64_t K, uint64_t nrows) {
        const uint64_t pitch = (uint64_t)mx4_scale_pitch((int64_t)K);
        return tc_encode_map(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, pitch, nrows, 0, pitch, 0, 32, 16, 0, false);
    };
    const uint64_t E = (uint64_t)c.E, fs = (uint64_t)c.f_shared, cat = 2 * fs + (c.standard ? 0 : (uint64_t)c.l);
    *m = FewMaps{};
    bool ok = tc_encode_map(&m->router, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, w.Wr, 32, E, (uint64_t)c.d / 32, (uint64_t)c.d * 4,
                            128, 32, 4, 16, true) &&
              (c.standard || rows(&m->down, w.Wdown, (uint64_t)c.d, (uint64_t)c.l)) &&
              rows(&m->shared_gu, w.Wgu_s, (uint64_t)c.d, 4 * fs) && rows(&m->cat, w.Wcat, cat, (uint64_t)c.d);
    if (w.mx4)
        return ok && codes(&m->routed_gu, w.Wgu, (uint64_t)c.l, E * 2 * c.f) &&
               codes(&m->routed_down, w.D, (uint64_t)c.f, E * c.l) &&
               scales(&m->routed_gu_scales, w.Wgu_scales, (uint64_t)c.l, E * 2 * c.f) &&
               scales(&m->routed_down_scales, w.D_scales, (uint64_t)c.f, E * c.l);
    return ok && rows(&m->routed_gu, w.Wgu, (uint64_t)c.l, E * 2 * c.f) &&
           rows(&m->routed_down, w.D, (uint64_t)c.f, E * c.l);
}

cudaError_t few_launch(const lmoe_config &c, const FewMaps &m, bool mx4, const float *bias, const void *x, int T,
                       void *y, int32_t *sel, void *p_out, void *u_out, void *workspace, bool stall_test,
                       cudaStream_t s)
{
    const FewLayout L = few_layout(c, T);
    char *ws = (char *)workspace;
    FewParams p = {};
    p.T = T; p.d = c.d; p.l = c.l; p.f = c.f; p.E = c.E; p.k = c.k; p.fs = c.f_shared; p.act = c.act;
    p.standard = c.standard; p.gate_cap = c.gate_cap; p.up_cap = c.up_cap; p.eps = c.eps;
    p.x = x; p.bias = bias; p.y = y; p.p_out = p_out; p.u_out = u_out; p.sel = sel;
    p.ctl = (unsigned *)(ws + L.ctl); p.r64 = (double *)(ws + L.r64); p.p32 = (float *)(ws + L.p32);
    p.tab = (Touched *)(ws + L.tab); p.z = (float *)(ws + L.z); p.hs = (float *)(ws + L.hs); p.H = (float *)(ws + L.H);
    p.part = (float *)(ws + L.part); p.ysl = (float *)(ws + L.ysl); p.u = (float *)(ws + L.u);
    p.scales = mx4; p.stall_test = stall_test;
    // Activation slots: the longest row set of any item, up to 58 KB (longer ones
    // come in segments); the rest of shared memory is the weight ring.
    const bool f32 = c.dtype == LMOE_F32;
    auto need = [&](int K, int eb, int planes, bool q) { return T * planes * act_stride(K, eb, q); };
    int slot = need(c.d, f32 ? 4 : 2, 1, false);
    const int two = f32 ? 1 : 2, eb = f32 ? 4 : 2;
    slot = std::max(slot, need(c.l, eb, two, true));
    slot = std::max(slot, need(c.f, eb, two, true));
    slot = std::max(slot, need(c.f_shared, eb, two, true));
    slot = std::min(slot, 58 * 1024);
    slot = (slot + 1023) / 1024 * 1024;
    p.slot_bytes = slot;
    const int stage = STAGE_BYTES + (mx4 ? 2 * SCALE_BOX : 0);
    p.stages = std::min(MAX_STAGES, (int)((SMEM_MAX - (int)fixed_smem() - 2 * slot) / stage));
    const size_t smem = fixed_smem() + 2 * (size_t)slot + (size_t)p.stages * stage;
    cudaError_t e = cudaMemsetAsync(p.ctl, 0, 4 * C_WORDS, s);
    if (e != cudaSuccess) return e;
    if (f32) return launch<W_F32>(m, p, smem, s);
    if (mx4) return launch<W_MX4>(m, p, smem, s);
    return launch<W_BF16>(m, p, smem, s);
}

}  // namespace lmoe
