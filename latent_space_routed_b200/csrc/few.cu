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
//   shared gu    16 gate and 16 up rows            -> shared hidden
//   routed gu    16 gate and 16 up rows of expert  -> hidden H of each of its slots
//   shared down  32 rows of the first shared expert  -> fp32 partial of y
//   routed down  32 rows of D of one expert        -> p (D h) of each of its slots
//   shared down  of the second shared expert (each half streams while the stage before it ends)
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
// Roles (16 warps, one block per SM):
//   warps 0-7   consumers: products from shared memory.  Two teams of four warps, each with half
//               of the ring.  An item is a run of sub-items (32 rows, or 16); the teams take them in
//               turn and leave their warps' partial sums in one of two buffers a team.  (Router
//               items are one sub-item, whose K the teams halve.)
//   warp 8      producer: one thread keeps a ring of 16 KB stages full, one TMA copy each (measured:
//               one thread issuing 16 KB boxes streams 7.3 TB/s, as 8 KB boxes 6.4 TB/s).  A box is
//               four 128-byte k-blocks of two groups of 16 rows (gate and up, or 32 rows), eight
//               k-blocks of 16 rows, or 32 of 4 rows (router)
//   warp 9      scheduler: takes tickets and describes their items in a queue, at most three items
//               ahead of the producer (its integer work per item would stall the copies)
//   warps 10-12 loaders: bring an item's activations from global memory into one of two
//               shared-memory slots, in the form that the product wants, one set ahead.  Before the
//               first routed item they select the experts, a warp per token, in every block: the same
//               work takes no longer than another block's result would take to arrive
//   warp 13     signaller: publishes finished items to the other blocks (the fence before the
//               counter costs 1000 to 2000 cycles, which others would otherwise spend per item)
//   warps 14-15 finishers, one a team: sums over the team's warps, gates, weights and stores.  By the
//               consumers themselves these cost 67 us of 439 with 6 tokens and 4-bit experts
//
// What it takes (d 7168, l 1792, f 2048, 384 experts, 32 a token; bytes at the copy rate of 6.46 TB/s), in turn with
// other work, and (in brackets) alone in a loop:
//   1 token            161 us (157), 91 % of the rate
//   8 tokens           772 us (714), 90 %
//   1 token, 4 bits    130 us (129), 51 %; 6 tokens 352 us (348), 51 %: the consumers' instructions bound the 4-bit
//                      stages (with the products skipped, 277 us were left of 500 at the time).  Eight warps
//                      a team or deeper unrolling were slower: warps compete for the instruction buffers
// and at d 2048, l 512, f 1408, 256 experts, 24 a token, 1 token: 56 us, 40 %: the seven dependent
// stages have latencies (selection 5 us, the last three stages 13 us) that a stream of 22 us cannot hide.
// 512 threads leave 128 registers each, which the 4-bit and fp32 instantiations use up.  fp32 spills (32 bytes of
// stores, 108 of loads); the 4-bit one does not, and how the compiler gets by shows in the time of 6 tokens: variants
// of the selection's code that left 4 to 52 bytes of spills there ran at 348 to 358 us.
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
#include <cfloat>

#include <cuda_fp16.h>

#include "few.cuh"
#include "gemm_tc.cuh"
#include "ptx.cuh"

namespace lmoe {

namespace {
using namespace ptx;

constexpr int CONSUMERS = 8, LOADERS = 3, FINISHERS = 2;
constexpr int THREADS = 32 * (CONSUMERS + 2 + LOADERS + 1 + FINISHERS);
constexpr int LT = 32 * LOADERS;
constexpr int STAGE_BYTES = 16384, KBLK_BYTES = 2048;   // a k-block of 16 rows
constexpr int SCALE_BYTES = 1024;                // 2 x 16 rows of 32 scales (1024 values)
constexpr int MAX_STAGES = 12, QUEUE = 32, AHEAD = 3;
constexpr int ITEM_BYTES = 512 * 1024, MAX_REPS = 8;
constexpr int SMEM_MAX = 232448;

enum Kind { ROUTER, DOWN, SHARED_GU, ROUTED_GU, SHARED_DOWN, ROUTED_DOWN, COMBINE, UP, END, SELECT };

// Words of the control area (zero at launch).
enum Ctl { C_STATUS = 0, C_TICKET = 32, C_ROUTER = 64, C_Z = 96, C_HS = 160, C_H = 192, C_PART = 224,
           C_YS = 256, C_U = 288, C_AMAX_Z = 320, C_AMAX_H = 352, C_WORDS = C_AMAX_H + FEW_MAX_SLOTS };

struct Item {
    int kind;
    int j0, reps;        // first sub-item of the matrix (of the expert, the half), and how many
    int block0;          // first block of rows of the matrix (two groups)
    int kb0, nkb;        // first k-block (128 bytes of a row) in the matrix, and their number
    int ncol;            // rows of activations in the slot
    int ti;              // touched-expert index, or half of the shared experts
};

// A touched expert: its id, the tokens that selected it (a bit each) and its slots in token order.
struct Touched {
    int16_t expert, mask, slot[FEW_MAX_T];
};

// How the phases are cut into items (host side): sub-items per item (_r), items of the
// phase, of a half or of an expert (_n).
struct Plan {
    int router_n, down_r, down_n, sgu_r, sgu_n, rgu_r, rgu_n, sd_r, sd_n, rd_r, rd_n, up_r, up_n, combine_n;
    float rgu_inv, rd_inv;       // 1 / rgu_n, 1 / rd_n
};

struct FewParams {
    Plan n;
    int T, d, l, f, E, k, fs, act, standard;
    float gate_cap, up_cap, eps;
    const void *x;
    const float *bias;
    const float *Wr;
    const uint32_t *wr_top;  // largest |W_r| (bits)
    void *y, *p_out, *u_out;
    int32_t *sel;
    unsigned *ctl;
    double *r64;             // [T, E] biased scores' raw scores
    float *z, *hs, *H, *part, *ysl, *u, *ssq;   // ssq: [T, l / 32] sums of squares of u
    int stages, slot_bytes, scales;
    const char *wgu, *wd;    // routed weights, and bytes of their rows
    int64_t gu_row, d_row;
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
    if (it.ncol * a.planes * min(act_stride(a.K, a.eb, mx4), 1 << 24) > p.slot_bytes) {     // (within 32 bits)
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

// The loaders' rows: `rows` rows of n4 groups of four values, dealt to the loader
// threads one after another so that every thread keeps four loads in flight
// across rows.  src(row) is the row's first value, mul(row) its factor.
template <int FORM, typename Src, typename Mul>
__device__ __forceinline__ void load_rows(uint32_t dst, int stride, uint32_t plane, int rows, int n4, int tid, Src src,
                                          Mul mul)
{
    int row = 0, c = tid;
    auto settle = [&]() {
        while (c >= n4 && row < rows) {
            c -= n4;
            ++row;
        }
    };
    settle();
    while (row < rows) {
        float4 v[4];
        float m[4];
        int r[4], cc[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] = row;
            cc[i] = c;
            if (row < rows) {
                v[i] = __ldcg(reinterpret_cast<const float4 *>(src(row)) + c);
                m[i] = mul(row);
                c += LT;
                settle();
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] < rows)
                put4<FORM>(dst + (uint32_t)(r[i] * stride), plane, 4 * cc[i],
                           make_float4(v[i].x * m[i], v[i].y * m[i], v[i].z * m[i], v[i].w * m[i]));
    }
}

// One row of tokens x (bf16) as scaled terms, for 4-bit experts at the model width.
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

// fp32 bits (those of a bf16 in the upper half) as a double by integer operations: the conversion
// instruction takes 8 cycles of a quarter SM, these 3 to 5.  They know no exponents 0 and 255: zeros and
// subnormals come out as 2^-127 (1 + m), infinities and NaN as finite numbers.  So they serve only where
// every value of x and W_r is below 2^32 (ROUTER_WIDE): a zero's term is then below 2^-95, a whole sum of
// them below 2^-71, and 1/2, the score where a sum begins to tell, has neighbours 2^-54 apart.  Otherwise
// exact_scores takes the item's products anew.
constexpr uint32_t ROUTER_WIDE = (127u + 32u) << 23;
__device__ __forceinline__ double widen(uint32_t f)
{
    return __hiloint2double((int)((f & 0x80000000u) | (((f & 0x7fffffffu) >> 3) + 0x38000000u)), (int)(f << 29));
}
__device__ __forceinline__ double widen_bf16(uint32_t f)
{
    return __hiloint2double((int)((f & 0x80000000u) | (((f & 0x7fff0000u) >> 3) + 0x38000000u)), 0);
}

// The largest magnitude of fp32 values, as bits (NaN above infinity), into *top.
__global__ void largest_kernel(const uint32_t *__restrict__ v, int64_t n, uint32_t *top)
{
    uint32_t m = 0u;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
        m = max(m, v[i] & 0x7fffffffu);
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) atomicMax(top, m);
}

// Order-preserving 64-bit key of a biased score (-0 counts as 0).  NaN and what is below -FLT_MAX
// count as -FLT_MAX, as in the selection of lmoe_forward: they come last, lower index first.
__device__ __forceinline__ unsigned long long key64(double v)
{
    v = v > -(double)FLT_MAX ? v + 0.0 : -(double)FLT_MAX;       // (fmax takes more instructions)
    const unsigned long long u = (unsigned long long)__double_as_longlong(v);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

// mbar_wait by a whole warp: one answer for all lanes, and the lanes together again,
// as the warp-wide loads and products that follow need them.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const volatile int *abort)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}

// Barrier of the warps of one role (an mbarrier with one arrival per warp):
// bounded, unlike bar.sync, so that a role whose peer gave up still ends.
struct RoleBarrier {
    uint32_t bar, parity;
    const volatile int *abort;
    bool ok;                 // false once a wait gave up
    __device__ __forceinline__ bool sync()
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
        ok = warp_wait(bar, parity, abort);
        parity ^= 1u;
        return ok;
    }
};

// The selection in shared memory.
struct Select {
    uint32_t *mask;              // [E rounded up to 128]: tokens that selected an expert, then its index as well
    uint16_t *sel;               // [T, k] experts in order
    float *weight;               // [T, k]
    Touched *tab;
};
// Scratch of one warp's token: score keys' high and low words and scores of E rounded up to 128
// experts; keys and experts of the selected.
__host__ __device__ constexpr int select_bytes(int E128) { return 12 * E128 + 64 * 8 + 64 * 2; }

struct Shared {
    uint32_t ring, scales, act, full, empty, act_full, act_empty, cons, load, cells, free;   // shared-memory addresses
    float *red;              // [2 buffers][2 teams][4 warps][RED_WARP]
    float *sums;             // [SUM_BYTES / 4]
    Touched *tab;
    Select select;
    Item *queue;
    float *inv;              // [2 slots][8]: inverse of the activations' scale
    float *lred;             // loaders' sums [4]
    // [0] abort, [1] items published, [3] sets of x issued, [25] touched experts, [26, 28) stages issued to each
    // team; items passed: [16, 19) by each loader, [19] by the producer, [20] by the signaller; [32, 42) items
    // finished by each consumer and finisher warp; [44] the router's scores are to be taken anew (exact_scores)
    int *flags;
};

// ------------------------------------------------------------------ items

template <int WT> constexpr int k_elems() { return WT == W_F32 ? 32 : 64; }   // values per 128-byte k-block

// n / d for 0 <= n < 2^24 by a reciprocal (whose quotient is off by one at most).
__device__ __forceinline__ int divide(int n, int d, float inv)
{
    int q = (int)((float)n * inv);
    q -= q * d > n;
    q += (q + 1) * d <= n;
    return q;
}

// The item of ticket `tk`; kind END past the last.
template <int WT>
__device__ __forceinline__ Item item_of(const FewParams &p, int touched, const Touched *tab, unsigned tk)
{
    constexpr int KE = k_elems<WT>();
    const Plan &n = p.n;
    Item it = {END, 0, 1, 0, 0, 0, p.T, 0};
    const int rgu_total = touched * n.rgu_n, rd_total = touched * n.rd_n;
    int i = (int)tk, per = 0;
    if (i < n.router_n) {
        it.kind = ROUTER; it.j0 = i; it.nkb = p.d / 32;
        return it;
    }
    if ((i -= n.router_n) < n.down_n) {
        it.kind = DOWN; it.reps = n.down_r; it.nkb = p.d / KE; per = p.l / 16;
    } else if ((i -= n.down_n) < n.sgu_n) {
        it.kind = SHARED_GU; it.reps = n.sgu_r; it.nkb = p.d / KE; per = p.fs / 8;
    } else if ((i -= n.sgu_n) < rgu_total) {
        it.kind = ROUTED_GU; it.ti = divide(i, n.rgu_n, n.rgu_inv); i -= it.ti * n.rgu_n;
        it.reps = n.rgu_r; it.nkb = WT == W_MX4 ? (p.l + 255) / 256 : p.l / KE; per = p.f / 16;
        it.block0 = tab[it.ti].expert * (p.f / (WT == W_MX4 ? 16 : 32));
    } else if ((i -= rgu_total) < n.sd_n || (i >= n.sd_n + rd_total && i < 2 * n.sd_n + rd_total)) {
        it.kind = SHARED_DOWN; it.ti = i >= n.sd_n; i -= it.ti ? n.sd_n + rd_total : 0;
        it.reps = n.sd_r; it.nkb = p.fs / KE; it.kb0 = it.ti * it.nkb; per = p.d / 32;
    } else if ((i -= n.sd_n) < rd_total) {
        it.kind = ROUTED_DOWN; it.ti = divide(i, n.rd_n, n.rd_inv); i -= it.ti * n.rd_n;
        it.reps = n.rd_r; it.nkb = WT == W_MX4 ? (p.f + 255) / 256 : p.f / KE; per = p.l / 32;
        it.block0 = tab[it.ti].expert * (p.l / 16);
        it.ncol = __popc((unsigned)tab[it.ti].mask);
    } else if ((i -= rd_total + n.sd_n) < n.combine_n) {
        it.kind = COMBINE; it.j0 = i;
        return it;
    } else if ((i -= n.combine_n) < n.up_n) {
        it.kind = UP; it.reps = n.up_r; it.nkb = p.l / KE; it.kb0 = 2 * p.fs / KE; per = p.d / 16;
    } else {
        return it;
    }
    it.j0 = i * it.reps;
    it.reps = min(it.reps, per - it.j0);
    return it;
}

__device__ __forceinline__ bool weightless(int kind) { return kind == COMBINE || kind == END || kind == SELECT; }
__device__ __forceinline__ bool two_groups(int kind)
{
    return kind == SHARED_GU || kind == ROUTED_GU || kind == SHARED_DOWN || kind == ROUTED_DOWN;
}
// k-blocks per stage: 4, 8 or 32
__device__ __forceinline__ int stage_kb_log2(int kind) { return kind == ROUTER ? 5 : two_groups(kind) ? 2 : 3; }
// First output row of a sub-item.
__device__ __forceinline__ int out_row(int kind, int j)
{
    return j * (kind == ROUTER ? 4 : kind == SHARED_DOWN || kind == ROUTED_DOWN ? 32 : 16);
}
// Coordinates of a sub-item's boxes: row (of its block), block of rows.
template <int WT>
__device__ __forceinline__ void box_at(const Item &it, int j, int *c1, int *c2)
{
    if (it.kind == SHARED_GU || it.kind == ROUTED_GU) {     // gate and up rows in blocks of 64 (4 bits: 32)
        const int sh = WT == W_MX4 && it.kind == ROUTED_GU ? 1 : 2;
        *c1 = 16 * (j & ((1 << sh) - 1));
        *c2 = it.block0 + 2 * (j >> sh);
    } else if (it.kind == SHARED_DOWN || it.kind == ROUTED_DOWN) {
        *c1 = 0;
        *c2 = it.block0 + 2 * j;
    } else {
        *c1 = out_row(it.kind, j);
        *c2 = 0;
    }
}
__device__ __forceinline__ int chunks(const Item &it)
{
    const int sh = stage_kb_log2(it.kind);
    return (it.nkb + (1 << sh) - 1) >> sh;
}

// ------------------------------------------------------------------ consumers
// Partial products of an item: per warp two groups of 16 rows x 8 columns, the groups
// RED_GROUP floats apart (16 more than a group, so that both are read without conflicts).
constexpr int RED_GROUP = 144, RED_WARP = 2 * RED_GROUP, RED_FLOATS = 2 * CONSUMERS * RED_WARP;
constexpr int SUM_BYTES = 2048;          // sums of the router's and the combine items' warps
// Sum over a team's warps of one cell; `packed`: the lo terms' sums are four columns further.
__device__ __forceinline__ float red_sum(const float *cell, bool packed)
{
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < CONSUMERS / 2; ++w) v += cell[w * RED_WARP];
    if (packed)
#pragma unroll
        for (int w = 0; w < CONSUMERS / 2; ++w) v += cell[w * RED_WARP + 4];
    return v;
}

// A 128-byte k-block (eight blocks of 32 values, nb of them real) of two groups of 16
// rows of 4-bit weights against eight columns: acc += scale of the row's block *
// partial sum.  Two blocks per round, rolled: the body stays in the instruction buffers.
// A scale byte becomes fp32's exponent field: 2^(e - 127), but 0 for e = 0 (2^-127, below
// fp32's normal range) and infinity for 255, whose blocks the handle's codes hold as zeros:
// 0 x infinity is the NaN that they stand for.
template <bool PACKED>
__device__ __forceinline__ void mx4_kblock(float (&acc)[2][4], uint32_t tile, uint32_t arow, uint32_t plane,
                                           uint32_t scales, int gid, int c4, int nb)
{
#pragma unroll 1
    for (int j0 = 0; j0 < nb; j0 += 2) {             // nb is even: K is a multiple of 64
        uint32_t w[2][2][2], e[2][2];                // block, group, row gid + 8 h; scales of both blocks
        uint4 x[2], y[2];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                e[g][h] = lds16(scales + (uint32_t)(512 * g + 256 * h + j0));
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    w[j][g][h] = lds32(tile + (uint32_t)(KBLK_BYTES * g + 1024 * h + (((j0 + j) ^ gid) << 4) + 4 * c4));
            }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[j] = lds128(arow + 64u * (j0 + j));
            if (!PACKED) y[j] = lds128(arow + plane + 64u * (j0 + j));
        }
        float t[2][2][4] = {};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                uint32_t wa[4], wb[4];
                e2m1x8_to_f16(wa, w[j][g][0]);
                e2m1x8_to_f16(wb, w[j][g][1]);
                mma_f16(t[j][g], wa[0], wb[0], wa[1], wb[1], x[j].x, x[j].y);
                mma_f16(t[j][g], wa[2], wb[2], wa[3], wb[3], x[j].z, x[j].w);
                if (!PACKED) {
                    mma_f16(t[j][g], wa[0], wb[0], wa[1], wb[1], y[j].x, y[j].y);
                    mma_f16(t[j][g], wa[2], wb[2], wa[3], wb[3], y[j].z, y[j].w);
                }
            }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                const float fa = __uint_as_float(e[g][0] << (23 - 8 * j) & 0x7f800000u);
                const float fb = __uint_as_float(e[g][1] << (23 - 8 * j) & 0x7f800000u);
                acc[g][0] = fmaf(t[j][g][0], fa, acc[g][0]);
                acc[g][1] = fmaf(t[j][g][1], fa, acc[g][1]);
                acc[g][2] = fmaf(t[j][g][2], fb, acc[g][2]);
                acc[g][3] = fmaf(t[j][g][3], fb, acc[g][3]);
            }
    }
}

// The largest magnitude of a warp's 16 rows of one column (two columns side by side), into *word.
__device__ __forceinline__ void largest_of_rows(unsigned *word, float v, bool real, int lane)
{
    float m = real ? fabsf(v) : 0.f;
#pragma unroll
    for (int off = 2; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane < 2 && real) atomicMax(word, __float_as_uint(m));
}

// Wait until item q is in the queue.
__device__ __forceinline__ bool wait_published(volatile int *published, int q, volatile int *abort)
{
    if (*published <= q) {
        const long long t0 = clock64();
        while (*published <= q) {
            __nanosleep(20);
            if (*abort || clock64() - t0 > 2 * WAIT_LIMIT_CYCLES) return false;
        }
    }
    __threadfence_block();
    return true;
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

// Scores of a lane's selected experts (the first of `left` > 0, the second of `left` > 32) over the token's largest.
__device__ __noinline__ float2 score_ratios(const double *r, int e0, int e1, int left)
{
    const double a = left > 0 ? __ldcg(r + e0) : 0.0, b = left > 32 ? __ldcg(r + e1) : 0.0;
    double m = fmax(a, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    return make_float2((float)(a / m), (float)(b / m));
}

// Selection and weights of token t by one warp: the k-th largest 64-bit score key by
// bisection on the bits of its high word that the keys do not share; low words and
// indices decide only where the high words tie (rare); then the k in order of key, equal
// keys by lower index.  Loops stay rolled: this runs once per call, and unrolled code costs
// more to fetch than to run (an unrolled top-k took 50 us).
template <int WT>
__device__ __forceinline__ void select_token(const FewParams &p, const Select &q, uint8_t *scratch, int t, int lane)
{
    constexpr unsigned FULL = 0xffffffffu;
    const int E = p.E, E4 = (E + 127) / 128 * 32;      // keys in groups of four
    const unsigned lt = (1u << lane) - 1u;
    uint32_t *hi = reinterpret_cast<uint32_t *>(scratch), *lo = hi + 4 * E4;
    float *score = reinterpret_cast<float *>(lo + 4 * E4);
    unsigned long long *cand = reinterpret_cast<unsigned long long *>(score + 4 * E4);
    uint16_t *cand_e = reinterpret_cast<uint16_t *>(cand + 64);
    {
        const double *r = p.r64 + (int64_t)t * E;
        uint32_t all_and = FULL, all_or = 0u;
        __syncwarp();
#pragma unroll 1
        for (int e0 = lane; e0 < 4 * E4; e0 += 256) {      // eight loads in flight
            double v[8];
            float b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] = e0 + 32 * i < E ? __ldcg(r + e0 + 32 * i) : 0.0;
                b[i] = e0 + 32 * i < E ? __ldg(p.bias + e0 + 32 * i) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = e0 + 32 * i;
                if (e >= 4 * E4) break;
                unsigned long long key = 0ull;             // real keys > 0
                if (e < E) {
                    key = key64(v[i] + (double)b[i]);
                    all_and &= (uint32_t)(key >> 32);
                    all_or |= (uint32_t)(key >> 32);
                }
                hi[e] = (uint32_t)(key >> 32);
                lo[e] = (uint32_t)key;
                score[e] = (float)v[i];
            }
        }
        all_and = __reduce_and_sync(FULL, all_and);
        const uint32_t diff = all_and ^ __reduce_or_sync(FULL, all_or);
        __syncwarp();
        // largest th with at least k keys >= th, two bits at a time
        const int top = 31 - __clz(diff);              // -1: all equal
        uint32_t th = top == 31 ? 0u : all_and >> (top + 1) << (top + 1);
        int count = E;
        const uint4 *h4 = reinterpret_cast<const uint4 *>(hi);
#pragma unroll 1
        for (int b = top | 1; b >= 0 && count != p.k; b -= 2) {     // (b = -1 | 1 = -1: none)
            const uint32_t step = 1u << (b - 1), c1 = th | step, c2 = th | 2u * step, c3 = c2 | step;
            unsigned n12 = 0, n3 = 0;                  // counts of c1 and (16 bits further) c2; of c3
#pragma unroll 2
            for (int e = lane; e < E4; e += 32) {
                const uint4 h = h4[e];
                n12 += (h.x >= c1) + (h.y >= c1) + (h.z >= c1) + (h.w >= c1);
                n12 += ((h.x >= c2) + (h.y >= c2) + (h.z >= c2) + (h.w >= c2)) << 16;
                n3 += (h.x >= c3) + (h.y >= c3) + (h.z >= c3) + (h.w >= c3);
            }
            n12 = __reduce_add_sync(FULL, n12);
            n3 = __reduce_add_sync(FULL, n3);
            const int n1 = (int)(n12 & 0xffffu), n2 = (int)(n12 >> 16);
            if ((int)n3 >= p.k) {
                th = c3;
                count = (int)n3;
            } else if (n2 >= p.k) {
                th = c2;
                count = n2;
            } else if (n1 >= p.k) {
                th = c1;
                count = n1;
            }
        }
        // compact the selected in index order; where more keys tie on the high word than are
        // wanted, a tied one is in if fewer than the wanted tied ones are ahead of it
        int above = 0;
        if (count != p.k) {
#pragma unroll 1
            for (int e = lane; e < E; e += 32) above += hi[e] > th;
            above = (int)__reduce_add_sync(FULL, (unsigned)above);
        }
        int pos = 0;
#pragma unroll 1
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const uint32_t h = e < E ? hi[e] : 0u;
            bool in = e < E && h >= th;
            if (count != p.k && e < E && h == th) {
                const uint32_t mine = lo[e];
                int ahead = above;
#pragma unroll 1
                for (int i = 0; i < E; ++i) ahead += hi[i] == th && (lo[i] > mine || (lo[i] == mine && i < e));
                in = ahead < p.k;
            }
            const unsigned b = __ballot_sync(FULL, in);
            const int at = pos + __popc(b & lt);
            if (in && at < 64) cand_e[at] = (uint16_t)e;
            pos += __popc(b);
        }
        __syncwarp();
        float rv[2] = {0.f, 0.f};
        int ex[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (lane + 32 * h < p.k) {
                ex[h] = min((int)cand_e[lane + 32 * h], E - 1);
                rv[h] = score[ex[h]];
                cand[lane + 32 * h] = (unsigned long long)hi[ex[h]] << 32 | lo[ex[h]];
            }
        float sum;
#pragma unroll 1
        for (bool again = false;; again = true) {
            sum = rv[0] + rv[1];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);      // (the same in all lanes)
            if (sum >= 1e-30f || again) break;
            // scores that fp32 holds roughly or not at all
            const float2 r = score_ratios(p.r64 + (int64_t)t * E, ex[0], ex[1], p.k - lane);
            rv[0] = r.x;
            rv[1] = r.y;
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = lane + 32 * h;
            if (i >= p.k) break;
            const unsigned long long mine = cand[i];
            int place = 0;
#pragma unroll 4
            for (int c = 0; c < p.k; ++c) {
                const unsigned long long other = cand[c];
                place += other > mine || (other == mine && c < i);
            }
            const float w = rv[h] / sum;
            q.sel[t * p.k + place] = (uint16_t)ex[h];
            q.weight[t * p.k + place] = w;
            atomicOr(q.mask + ex[h], 1u << t);
            if (blockIdx.x == 0) {
                p.sel[t * p.k + place] = ex[h];
                store_token<WT>(p.p_out, t * p.k + place, w);
            }
        }
    }
}

// The touched experts in ascending order with their slots, by one warp; returns their number.
__device__ __forceinline__ int touched_experts(const FewParams &p, const Select &q, int lane)
{
    constexpr unsigned FULL = 0xffffffffu;
    const unsigned lt = (1u << lane) - 1u;
    int n = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        const uint32_t m = q.mask[e0 + lane];
        const unsigned b = __ballot_sync(FULL, m != 0u);
        const int at = n + __popc(b & lt);
        if (m) {
            q.tab[at].expert = (int16_t)(e0 + lane);
            q.tab[at].mask = (int16_t)m;
            q.mask[e0 + lane] = m | (uint32_t)at << 8;
        }
        n += __popc(b);
    }
    __syncwarp();
#pragma unroll 1
    for (int t = 0; t < p.T; ++t)
#pragma unroll 1
        for (int j = lane; j < p.k; j += 32) {
            const uint32_t m = q.mask[q.sel[t * p.k + j]];
            q.tab[m >> 8].slot[__popc(m & 0xffu & ((1u << t) - 1u))] = (int16_t)(t * p.k + j);
        }
    __syncwarp();
    return n;
}

// Scores of four experts from e0 on with converted values, a warp per pair of token and expert: for x or W_r
// with values that `widen` does not know (see there).  Out of line: it is rarely called.
template <int WT>
__device__ __noinline__ void exact_scores(const FewParams &p, int e0, int warp, int lane)
{
    for (int i = warp; i < 4 * p.T; i += CONSUMERS) {
        const int e = e0 + (i & 3), t = i >> 2;
        if (e >= p.E) continue;
        const float *w = p.Wr + (int64_t)e * p.d;
        double v = 0.0;
        for (int c = lane; c < p.d; c += 32)
            v = fma((double)__ldg(w + c), (double)token_value<WT>(p.x, (int64_t)t * p.d + c), v);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) p.r64[(int64_t)t * p.E + e] = 1.0 / (1.0 + exp(-v));
    }
}

// u for 32 latent columns (one per lane) of every token: the token's slots dealt to 8 / T
// warps (a power of two), their parts summed in order.
template <int WT>
__device__ __forceinline__ bool combine_item(const FewParams &p, const Item &it, float *red, RoleBarrier &bar, int warp,
                                             int lane)
{
    const int parts = p.T == 1 ? 8 : p.T == 2 ? 4 : p.T <= 4 ? 2 : 1;
    const int t = warp / parts, part = warp - t * parts, c = 32 * it.j0 + lane;
    float u = 0.f;
    if (t < p.T) {
        const float *src = p.ysl + (int64_t)t * p.k * p.l + c;
        int j = part;
#pragma unroll 1
        for (; j + 3 * parts < p.k; j += 4 * parts) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __ldcg(src + (int64_t)(j + i * parts) * p.l);
            u += (v[0] + v[1]) + (v[2] + v[3]);
        }
#pragma unroll 1
        for (; j < p.k; j += parts) u += __ldcg(src + (int64_t)j * p.l);
    }
    if (parts > 1) {
        red[warp * 32 + lane] = u;
        if (!bar.sync()) return false;
        if (part == 0)
#pragma unroll 1
            for (int i = 1; i < parts; ++i) u += red[(warp + i) * 32 + lane];
    }
    if (t < p.T && part == 0) {
        store_token<WT>(p.u_out, (int64_t)t * p.l + c, u);
        if (p.standard) {
            const float *q = p.part + (int64_t)t * p.d + c;
            store_token<WT>(p.y, (int64_t)t * p.d + c, __ldcg(q) + __ldcg(q + (int64_t)p.T * p.d) + u);
        } else {
            p.u[(int64_t)t * p.l + c] = u;
            float ss = u * u;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (lane == 0) p.ssq[t * (p.l / 32) + it.j0] = ss;
        }
    }
    return parts == 1 || bar.sync();      // the sums' memory is free again
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
    sh.scales = base + o; o += p.scales ? (uint32_t)p.stages * SCALE_BYTES : 0u;
    sh.act = base + o; o += 2u * (uint32_t)p.slot_bytes;
    sh.red = reinterpret_cast<float *>(g + o); o += 4 * RED_FLOATS;
    sh.sums = reinterpret_cast<float *>(g + o); o += SUM_BYTES;
    const int E128 = (p.E + 127) & ~127, TK = p.T * p.k, TK8 = (TK + 7) & ~7;
    sh.select.mask = reinterpret_cast<uint32_t *>(g + o); o += 4 * E128;
    sh.select.weight = reinterpret_cast<float *>(g + o); o += 4 * TK8;
    sh.select.sel = reinterpret_cast<uint16_t *>(g + o); o += 2 * TK8;
    sh.tab = sh.select.tab = reinterpret_cast<Touched *>(g + o); o += (uint32_t)sizeof(Touched) * (TK8 < E128 ? TK8 : E128);
    o = (o + 15u) & ~15u;
    sh.queue = reinterpret_cast<Item *>(g + o); o += sizeof(Item) * QUEUE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(g + o); o += 8 * (2 * MAX_STAGES + 14);
    sh.inv = reinterpret_cast<float *>(g + o); o += 64;
    sh.lred = reinterpret_cast<float *>(g + o); o += 64;
    sh.flags = reinterpret_cast<int *>(g + o);
    sh.full = smem_u32(bars);
    sh.empty = sh.full + 8u * MAX_STAGES;
    sh.act_full = sh.empty + 8u * MAX_STAGES;
    sh.act_empty = sh.act_full + 16u;
    sh.cons = sh.act_empty + 16u;
    sh.load = sh.cons + 8u;
    sh.cells = sh.load + 8u;         // [team][buffer]: partial sums written
    sh.free = sh.cells + 32u;        // [team][buffer]: and read
    volatile int *abort = sh.flags;
    volatile int *published = sh.flags + 1, *passed = sh.flags + 16;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int S = p.stages, half = (S + 1) / 2;      // team 0's slots are [0, half), team 1's [half, S)
    unsigned first_ticket = 0;
    if (threadIdx.x == 32 * (CONSUMERS + 1)) first_ticket = atomicAdd(p.ctl + C_TICKET, 1u);
    for (int e = threadIdx.x; e < E128; e += THREADS) sh.select.mask[e] = 0u;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(sh.full + 8u * s, 1);
            mbar_init(sh.empty + 8u * s, CONSUMERS / 2);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(sh.act_full + 8u * s, LOADERS);
            mbar_init(sh.act_empty + 8u * s, CONSUMERS);
        }
        mbar_init(sh.cons, CONSUMERS);
        mbar_init(sh.load, LOADERS);
        for (int t = 0; t < 4; ++t) {
            mbar_init(sh.cells + 8u * t, CONSUMERS / 2);
            mbar_init(sh.free + 8u * t, 1);
        }
        for (int i = 0; i < 48; ++i) sh.flags[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();

    auto give_up = [&](int code) {
        atomicOr(p.ctl + C_STATUS, (unsigned)code);
        *abort = 1;
    };

    if (warp == CONSUMERS) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            int slot0 = 0, slot1 = half, issued0 = 0, issued1 = 0;     // next slot of each team
            uint32_t ph0 = 0, ph1 = 0;
            bool ok = true;
            for (int q = 0; ok; ++q) {
                passed[LOADERS] = q;
                if (!(ok = wait_published(published, q, abort))) break;
                const Item it = sh.queue[q % QUEUE];
                if (it.kind == END) break;
                if (weightless(it.kind)) continue;
                const int nc = chunks(it), kb = 1 << stage_kb_log2(it.kind);
                const bool two = two_groups(it.kind), split = it.kind == ROUTER;
                const bool mx4 = WT == W_MX4 && (it.kind == ROUTED_GU || it.kind == ROUTED_DOWN);
                const uint32_t bytes = STAGE_BYTES + (mx4 ? SCALE_BYTES : 0);
                const CUtensorMap *map = it.kind == ROUTER        ? &maps.router
                                         : it.kind == DOWN        ? &maps.down
                                         : it.kind == SHARED_GU   ? &maps.shared_gu
                                         : it.kind == ROUTED_GU   ? &maps.routed_gu
                                         : it.kind == SHARED_DOWN ? &maps.shared_down
                                         : it.kind == ROUTED_DOWN ? &maps.routed_down
                                                                  : &maps.up;
                const CUtensorMap *smap = it.kind == ROUTED_GU ? &maps.routed_gu_scales : &maps.routed_down_scales;
                // stages in the order in which the teams take them: chunk by chunk of a pair of sub-items
                for (int r = 0; r < it.reps && ok; r += 2) {
                    int c1[2], c2[2];
                    box_at<WT>(it, it.j0 + r, &c1[0], &c2[0]);
                    box_at<WT>(it, it.j0 + r + 1, &c1[1], &c2[1]);
                    const bool pair = !split && r + 1 < it.reps;
                    for (int i = 0; i < (pair ? 2 * nc : nc) && ok; ++i) {
                        const int team = split || pair ? i & 1 : 0, c = pair ? i >> 1 : i;
                        const int s = team ? slot1 : slot0, x1 = pair && team ? c1[1] : c1[0], x2 = pair && team ? c2[1] : c2[0];
                        const uint32_t fb = sh.full + 8u * s;
                        if (!(ok = mbar_wait(sh.empty + 8u * s, (team ? ph1 : ph0) ^ 1u, abort))) break;
                        mbar_expect_tx(fb, bytes);
                        const uint32_t dst = sh.ring + (uint32_t)s * STAGE_BYTES;
                        if (two) tma_load_4d(dst, map, fb, x1, x2, it.kb0 + c * kb);
                        else tma_load_3d(dst, map, fb, x1, it.kb0 + c * kb);
                        if (mx4) tma_load_3d_at(sh.scales + (uint32_t)s * SCALE_BYTES, smap, fb, 32 * c, x1, x2);
                        if (team) {
                            sh.flags[27] = ++issued1;
                            if (++slot1 == S) {
                                slot1 = half;
                                ph1 ^= 1u;
                            }
                        } else {
                            sh.flags[26] = ++issued0;
                            if (++slot0 == half) {
                                slot0 = 0;
                                ph0 ^= 1u;
                            }
                        }
                    }
                }
            }
            if (!ok) give_up(0x1);
        }
    } else if (warp == CONSUMERS + 1) {
        // ------------------------------------------------------------ scheduler
        const unsigned fixed = (unsigned)(p.n.router_n + p.n.down_n + p.n.sgu_n);     // tickets that need no selection
        unsigned next = first_ticket;
        int touched = 0;
        bool selecting = false;
        for (int q = 0;; ++q) {
            const unsigned tk = __shfl_sync(0xffffffffu, next, 0);
            int good = 1;
            if (tk >= fixed && selecting && touched == 0) {
                // the loaders have the selection as their next item
                if (lane == 0) {
                    const volatile int *found = sh.flags + 25;
                    const long long t0 = clock64();
                    while (*found == 0 && good) {
                        __nanosleep(20);
                        if (*abort || clock64() - t0 > 2 * WAIT_LIMIT_CYCLES) good = 0;
                    }
                    __threadfence_block();
                }
                good = __shfl_sync(0xffffffffu, good, 0);
                if (!good) {
                    if (lane == 0) give_up(0x10);
                    break;
                }
                touched = sh.flags[25];
            }
            Item it = {SELECT, 0, 0, 0, 0, 0, 0, 0};      // (no ticket)
            if (tk < fixed || touched) it = item_of<WT>(p, touched, sh.tab, tk);
            else selecting = true;
            if (it.kind == ROUTED_GU || it.kind == ROUTED_DOWN) {
                int c1, c2;
                box_at<WT>(it, it.j0 + lane, &c1, &c2);
                if (lane < it.reps)
                    prefetch_l2((it.kind == ROUTED_GU ? p.wgu + ((WT == W_MX4 ? 32 : 64) * (int64_t)c2 + c1) * p.gu_row
                                                      : p.wd + 16 * (int64_t)c2 * p.d_row));
            }
            if (lane == 0) {
                // not far ahead of the producer, and (looked at every eight items) far from every reader's tail
                const long long t0 = clock64();
                const volatile int *finished = sh.flags + 32;
                auto behind = [&](const volatile int *reader, int by) {
                    while (q - *reader >= by && good) {
                        __nanosleep(20);
                        if (*abort || clock64() - t0 > 2 * WAIT_LIMIT_CYCLES) good = 0;
                    }
                };
                behind(passed + LOADERS, AHEAD);
                if ((q & 7) == 0) {
                    for (int r = 0; r < LOADERS + 2; ++r) behind(passed + r, QUEUE - 8);
                    for (int r = 0; r < CONSUMERS + FINISHERS; ++r) behind(finished + r, QUEUE - 8);
                }
                if (good) {
                    sh.queue[q % QUEUE] = it;
                    __threadfence_block();
                    *published = q + 1;
                    if (it.kind != END && it.kind != SELECT) next = atomicAdd(p.ctl + C_TICKET, 1u);   // used in the next round
                } else {
                    give_up(0x10);
                }
            }
            good = __shfl_sync(0xffffffffu, good, 0);
            if (!good || it.kind == END) break;
        }
    } else if (warp > CONSUMERS + 1 && warp < CONSUMERS + 2 + LOADERS) {
        // ------------------------------------------------------------ loaders
        const int tid = threadIdx.x - 32 * (CONSUMERS + 2), lw = warp - CONSUMERS - 2;
        RoleBarrier bar = {sh.load, 0u, abort, true};
        int set = 0, cur_key = -1, cur_seg = -1, ready = -1;   // ready: last kind whose inputs are complete
        bool ok = true;
        for (int q = 0; ok; ++q) {
            int good = 1;
            if (lane == 0) passed[lw] = q;
            if (lane == 0) good = wait_published(published, q, abort);
            ok = __shfl_sync(0xffffffffu, good, 0) != 0;
            if (!ok) {
                if (lane == 0) give_up(0x4);
                break;
            }
            const Item it = sh.queue[q % QUEUE];
            if (it.kind == END) break;
            if (it.kind == SELECT) {
                // the next set's slot is the scratch
                if (lane == 0) {
                    good = mbar_wait(sh.act_empty + 8u * (set & 1), (uint32_t)((set >> 1) & 1) ^ 1u, abort);
                    if (good && lw == 0) good = wait_count(p.ctl, C_ROUTER, (unsigned)p.n.router_n, abort);
                }
                ok = __shfl_sync(0xffffffffu, good, 0) != 0 && bar.sync();
                if (ok) {
                    uint8_t *scratch = g + (sh.act - base) + (set & 1) * p.slot_bytes + lw * select_bytes(E128);
#pragma unroll 1
                    for (int t = lw; t < p.T; t += LOADERS) select_token<WT>(p, sh.select, scratch, t, lane);
                    ok = bar.sync();
                }
                if (ok && lw == 0) {
                    const int touched = touched_experts(p, sh.select, lane);
                    __threadfence_block();
                    if (lane == 0) *(volatile int *)(sh.flags + 25) = touched;
                }
                if (!ok) {
                    if (lane == 0) give_up(0x4);
                    break;
                }
                continue;
            }
            if (weightless(it.kind)) continue;
            const ActPlan a = act_plan<WT>(p, it);
            const bool mx4 = WT == W_MX4 && (it.kind == ROUTED_GU || it.kind == ROUTED_DOWN);
            const int sets = a.nseg == 1 ? 1 : a.nseg * ((it.reps + 1) / 2);     // segments again for every pair
            for (int i = 0, seg = 0; i < sets && ok; ++i, seg = seg + 1 == a.nseg ? 0 : seg + 1) {
                if (a.key == cur_key && seg == cur_seg) continue;
                cur_key = a.key;
                cur_seg = seg;
                const int slot = set & 1;
                if (lane == 0) {
                    good = mbar_wait(sh.act_empty + 8u * slot, (uint32_t)((set >> 1) & 1) ^ 1u, abort);
                    if (good && lw == 0 && it.kind != ready) {          // the items that write these values
                        if (it.kind == ROUTED_GU && !p.standard) good = wait_count(p.ctl, C_Z, (unsigned)p.n.down_n, abort);
                        // (the failure-detection test waits for one count too many)
                        if (it.kind == SHARED_DOWN)
                            good = wait_count(p.ctl, C_HS, (unsigned)p.n.sgu_n + (p.stall_test ? 1u : 0u), abort);
                        if (it.kind == ROUTED_DOWN)
                            good = wait_count(p.ctl, C_H, (unsigned)(sh.flags[25] * p.n.rgu_n), abort);
                        if (it.kind == UP)
                            good = wait_count(p.ctl, C_U, (unsigned)p.n.combine_n, abort) &&
                                   wait_count(p.ctl, C_PART, 2u * p.n.sd_n, abort);
                    }
                }
                // one warp of a block polls (all of them on one word kept each other waiting for 3 us)
                ok = __shfl_sync(0xffffffffu, good, 0) != 0 && (it.kind == ready || bar.sync());
                ready = it.kind;
                if (!ok) {
                    if (lane == 0) give_up(0x4);
                    break;
                }
                const uint32_t dst = sh.act + (uint32_t)(slot * p.slot_bytes);
                const uint32_t plane = (uint32_t)(it.ncol * a.stride);
                const int k0 = seg * a.kseg, kn = a.K - k0 < a.kseg ? a.K - k0 : a.kseg;
                float *inv = sh.inv + 8 * slot;
                const bool x_rows = it.kind <= SHARED_GU || (it.kind == ROUTED_GU && p.standard);
                if (x_rows && !mx4) {
                    // x as it is: one bulk copy per row
                    if (tid == 0) {
                        sh.flags[3] = set + 1;
                        const uint32_t bytes = (uint32_t)(kn * a.eb);
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        mbar_expect_tx(sh.act_full + 8u * slot, bytes * (uint32_t)it.ncol);
                        for (int t = 0; t < it.ncol; ++t)
                            bulk_load(dst + (uint32_t)(t * a.stride),
                                      (const char *)p.x + ((int64_t)t * p.d + k0) * a.eb, bytes, sh.act_full + 8u * slot);
                    } else if (lane == 0) {
                        mbar_arrive(sh.act_full + 8u * slot);
                    }
                    ++set;
                    continue;
                }
                if (it.kind == UP) {
                    // RMSNorm: each token's sum of squares from the combine items' parts, in a fixed order
                    const int nb = p.l / 32;
                    for (int t = lw; t < it.ncol; t += LOADERS) {
                        float ss = 0.f;
                        for (int c = lane; c < nb; c += 32) ss += __ldcg(p.ssq + t * nb + c);
#pragma unroll
                        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
                        if (lane == 0) sh.lred[t] = 1.0f / sqrtf(ss / (float)p.l + p.eps);
                    }
                    if (!(ok = bar.sync())) {
                        if (lane == 0) give_up(0x4);
                        break;
                    }
                    load_rows<WT == W_F32 ? F_F32 : F_BF16X2>(
                        dst, a.stride, plane, it.ncol, kn / 4, tid,
                        [&](int t) { return p.u + (int64_t)t * p.l + k0; }, [&](int t) { return sh.lred[t]; });
                } else if (mx4) {
                    const unsigned *amax = p.ctl + (it.kind == ROUTED_DOWN ? C_AMAX_H : C_AMAX_Z);
                    const Touched &e = sh.tab[it.ti];
                    if (x_rows) {       // the experts read x itself: its rows' largest magnitudes first
                        for (int t = lw; t < it.ncol; t += LOADERS) {
                            const uint32_t *v = reinterpret_cast<const uint32_t *>((const bf16 *)p.x + (int64_t)t * p.d);
                            uint32_t m = 0u;
#pragma unroll 4
                            for (int c = lane; c < p.d / 2; c += 32) {
                                const uint32_t w = __ldg(v + c) & 0x7fff7fffu;
                                m = max(m, max(w << 16, w & 0xffff0000u));
                            }
                            m = __reduce_max_sync(0xffffffffu, m);
                            if (lane == 0) sh.lred[t] = __uint_as_float(m);
                        }
                        if (!(ok = bar.sync())) {
                            if (lane == 0) give_up(0x4);
                            break;
                        }
                    }
                    auto at = [&](int t) { return it.kind == ROUTED_DOWN ? (int)e.slot[t] : t; };
                    auto largest = [&](int t) { return x_rows ? sh.lred[t] : __uint_as_float(__ldcg(amax + at(t))); };
                    auto mul = [&](int t) {
                        float back;
                        return f16_scale(largest(t), &back);
                    };
                    if (tid < it.ncol) f16_scale(largest(tid), &inv[tid]);
                    if (x_rows) {
                        for (int t = 0; t < it.ncol; ++t)
                            load_row_bf16_scaled(dst + (uint32_t)(t * a.stride), plane,
                                                 (const bf16 *)p.x + (int64_t)t * p.d + k0, kn, mul(t), tid);
                    } else {
                        const float *src = (it.kind == ROUTED_DOWN ? p.H : p.z) + k0;
                        load_rows<F_F16X2>(dst, a.stride, plane, it.ncol, kn / 4, tid,
                                           [&](int t) { return src + (int64_t)at(t) * a.K; }, mul);
                    }
                } else {
                    const Touched &e = sh.tab[it.ti];
                    const int kind = it.kind;
                    const float *src = (kind == ROUTED_DOWN ? p.H : kind == SHARED_DOWN ? p.hs + it.ti * p.fs : p.z) + k0;
                    const int64_t ld = kind == ROUTED_DOWN ? p.f : kind == SHARED_DOWN ? 2 * p.fs : p.l;
                    load_rows<WT == W_F32 ? F_F32 : F_BF16X2>(
                        dst, a.stride, plane, it.ncol, kn / 4, tid,
                        [&](int t) { return src + (int64_t)(kind == ROUTED_DOWN ? (int)e.slot[t] : t) * ld; },
                        [](int) { return 1.f; });
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(sh.act_full + 8u * slot);
                ++set;
            }
        }
    } else if (warp < CONSUMERS) {
        // ------------------------------------------------------------ consumers
        const int team = warp >> 2, sub = warp & 3;
        const int gid = lane >> 2, c4 = lane & 3;
        RoleBarrier bar = {sh.cons, 0u, abort, true};                     // all eight warps
        int s = team ? half : 0;                         // slot and phase of this team's next stage
        uint32_t ph = 0, cell_n = 0;                     // sub-items of this team so far
        int set = -1, cur_key = -1, cur_seg = -1;
        bool ok = true;
        auto full = [&]() -> bool { return warp_wait(sh.full + 8u * s, ph, abort); };
        auto release = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(sh.empty + 8u * s);
            if (++s == (team ? S : half)) {
                s = team ? half : 0;
                ph ^= 1u;
            }
        };
        for (int q = 0;; ++q) {
            if (!(ok = __all_sync(0xffffffffu, wait_published(published, q, abort)))) break;
            auto done = [&]() {              // this warp's part of the item is stored
                __syncwarp();
                if (lane == 0) sts_release(smem_u32(sh.flags + 32 + warp), (unsigned)(q + 1));
            };
            const Item it = sh.queue[q % QUEUE];
            const int kind = it.kind;
            if (kind == END) break;
            if (kind == SELECT) {
                done();
                continue;
            }
            if (weightless(kind)) {
                int good = 1;
                if (threadIdx.x == 0) {
                    good = wait_count(p.ctl, C_YS, (unsigned)(sh.flags[25] * p.n.rd_n), abort);
                    if (good && p.standard) good = wait_count(p.ctl, C_PART, 2u * p.n.sd_n, abort);
                }
                ok = __shfl_sync(0xffffffffu, good, 0) != 0 && bar.sync() && combine_item<WT>(p, it, sh.sums, bar, warp, lane);
                if (!ok) break;
                done();
                continue;
            }

            const ActPlan a = act_plan<WT>(p, it);
            const bool two = two_groups(kind), split = kind == ROUTER;
            const int nc = chunks(it), nkb = it.nkb;
            const uint32_t plane = (uint32_t)(it.ncol * a.stride);
            // Columns of the product: the slot's rows, but of the routed gate/up (whose slot holds
            // every token) only the expert's tokens.  `tok`: the row of column lane % 8 (past the
            // last column: the last one's)
            const unsigned mask = kind == ROUTED_GU ? (unsigned)sh.tab[it.ti].mask : 0u;
            const int ncol = kind == ROUTED_GU ? __popc(mask) : it.ncol;
            int tok = min(lane & 7, ncol - 1);
            if (kind == ROUTED_GU) {
                unsigned m = mask;
                for (; tok > 0; --tok) m &= m - 1u;
                tok = __ffs(m) - 1;
            }
            // Four columns or fewer of two terms: hi in columns 0-3, lo in 4-7 of one product
            const bool packed = a.planes == 2 && ncol <= 4;
            const bool mx4 = WT == W_MX4 && (kind == ROUTED_GU || kind == ROUTED_DOWN);
            // values of K per stage
            const int kshift = kind == ROUTER ? 10 : mx4 ? 10 : (WT == W_F32 ? 5 : 6) + (two ? 2 : 3);
            const uint32_t mytile = (uint32_t)(2 * sub * KBLK_BYTES);   // this warp's two tiles of 16 rows
            uint32_t act = 0;
            // The activations of segment `seg`; false when a wait gave up.
            auto take = [&](int seg) -> bool {
                if (a.key != cur_key || seg != cur_seg) {
                    if (set >= 0) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(sh.act_empty + 8u * (set & 1));
                    }
                    ++set;
                    cur_key = a.key;
                    cur_seg = seg;
                    if (!warp_wait(sh.act_full + 8u * (set & 1), (uint32_t)(set >> 1) & 1u, abort)) return false;
                }
                act = sh.act + (uint32_t)((set & 1) * p.slot_bytes);
                return true;
            };
            // The stages of this team's sub-item (`mine`: it has one in this pair): body(c, k0), k0 the
            // segment's first value.  body calls release() as soon as its tiles are in registers, before
            // the products.
            auto stages = [&](bool mine, auto body) -> bool {
                int c = split ? team : 0;
                for (int seg = 0; seg < a.nseg; ++seg) {
                    if (!take(seg)) return false;
                    const int end = !mine ? 0 : seg + 1 < a.nseg ? ((seg + 1) * a.kseg) >> kshift : nc;
                    for (; c < end; c += split ? 2 : 1) {
                        if (!full()) return false;
                        body(c, seg * a.kseg);
                    }
                }
                return true;
            };
            // The cells for this sub-item's partial sums, once their last use has been read, and their hand-over
            // to the finishers: two buffers a team, so that the next products do not wait for the epilogue.
            float *myred = nullptr;
            auto cells_free = [&]() -> bool {
                myred = sh.red + (8 * (cell_n & 1u) + warp) * RED_WARP;
                return warp_wait(sh.free + 16u * team + 8u * (cell_n & 1u), (cell_n >> 1 & 1u) ^ 1u, abort);
            };
            auto cells_written = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(sh.cells + 16u * team + 8u * (cell_n & 1u));
                ++cell_n;
            };

            if (kind == ROUTER) {
                // ---- 4 rows, 64-bit products: lane (row, 4-value piece)
                double acc[FEW_MAX_T] = {};
                const int row = lane >> 3, piece = lane & 7;
                uint32_t top = __ldg(p.wr_top);        // the largest of |W_r| and this warp's share of x
                ok = stages(true, [&](int c, int k0) {
                    const uint32_t tile = sh.ring + (uint32_t)s * STAGE_BYTES + mytile;
                    {
                        // (read again, a 16-byte piece per lane; a pass over all of x at the start cost 2 us)
                        constexpr int EB = WT == W_F32 ? 4 : 2;
                        const int kblk = c * 32 + sub * 8, bytes = 32 * EB * min(8, nkb - kblk);
                        const uint32_t at = act + (uint32_t)(EB * (kblk * 32 - k0));
#pragma unroll
                        for (int i = 16 * lane; i < 256 * EB; i += 512)
                            if (i < bytes)
#pragma unroll 2
                                for (int t = 0; t < p.T; ++t) {
                                    const uint4 v = lds128(at + (uint32_t)(t * a.stride + i));
                                    if (WT == W_F32) {
                                        top = max(max(top, v.x & 0x7fffffffu), max(v.y & 0x7fffffffu, v.z & 0x7fffffffu));
                                        top = max(top, v.w & 0x7fffffffu);
                                    } else {
                                        const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                                    __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                                        top = max(top, max(m, m << 16));
                                    }
                                }
                    }
                    // two k-blocks (512 bytes each: 4 rows) per round: the body stays in the
                    // instruction buffers (unrolled over a stage it took 3 K cycles, most of them fetches)
#pragma unroll 1
                    for (int i0 = 0; i0 < 8; i0 += 2) {
                        const int kblk = c * 32 + sub * 8 + i0, left = nkb - kblk;
                        if (left <= 0) break;
                        double w[2][4];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {             // zero-filled past K
                            const int R = (i0 + i) * 4 + row;
                            const uint4 v = lds128(tile + (uint32_t)(R * 128 + ((piece ^ (R & 7)) << 4)));
                            w[i][0] = widen(v.x);
                            w[i][1] = widen(v.y);
                            w[i][2] = widen(v.z);
                            w[i][3] = widen(v.w);
                        }
                        const uint32_t at = act + (uint32_t)((WT == W_F32 ? 4 : 2) * (kblk * 32 + 4 * piece - k0));
#pragma unroll
                        for (int t = 0; t < FEW_MAX_T; ++t) {
                            if (t >= p.T) break;
                            double sum[2];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                sum[i] = 0.0;
                                if (i < left) {
                                    double x[4];
                                    if (WT == W_F32) {
                                        const uint4 v = lds128(at + (uint32_t)(t * a.stride + 128 * i));
                                        x[0] = widen(v.x); x[1] = widen(v.y); x[2] = widen(v.z); x[3] = widen(v.w);
                                    } else {
                                        const uint2 v = lds64(at + (uint32_t)(t * a.stride + 64 * i));
                                        x[0] = widen_bf16(v.x << 16); x[1] = widen_bf16(v.x);
                                        x[2] = widen_bf16(v.y << 16); x[3] = widen_bf16(v.y);
                                    }
                                    sum[i] = fma(w[i][0], x[0], w[i][1] * x[1]) + fma(w[i][2], x[2], w[i][3] * x[3]);
                                }
                            }
                            acc[t] += sum[0] + sum[1];
                        }
                    }
                    release();
                });
                if (!ok) break;
                volatile int *anew = sh.flags + 44;
                if (top >= ROUTER_WIDE) *anew = 1;
                double *rd = reinterpret_cast<double *>(sh.sums);     // [8 warps][4 rows][8 tokens]
#pragma unroll
                for (int t = 0; t < FEW_MAX_T; ++t)
                    if (t < p.T) {
#pragma unroll
                        for (int off = 1; off < 8; off <<= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], off);
                        if (piece == 0) rd[warp * 32 + row * 8 + t] = acc[t];
                    }
                if (!(ok = bar.sync())) break;
                if (*anew) {
                    exact_scores<WT>(p, 4 * it.j0, warp, lane);
                } else if (warp == 0) {
                    const int e = 4 * it.j0 + (lane >> 3), t = lane & 7;
                    if (e < p.E && t < p.T) {
                        double v = 0.0;
                        for (int w = 0; w < CONSUMERS; ++w) v += rd[w * 32 + lane];
                        p.r64[(int64_t)t * p.E + e] = 1.0 / (1.0 + exp(-v));
                    }
                }
                if (!(ok = bar.sync())) break;                // the sums' memory is free again
                done();
                continue;
            }

            for (int r0 = 0; ok && r0 < it.reps; r0 += 2) {
            const int rr = r0 + team;                      // this team's sub-item
            const bool mine = rr < it.reps;
            if (WT == W_F32) {
                // ---- fp32: lane (4-value piece, rows rq + 4 i); two tiles, of one k-block or of two
                float acc[2][4][FEW_MAX_T] = {};
                const int piece = lane & 7, rq = lane >> 3;
                uint32_t off[FEW_MAX_T];                   // of the columns' rows
#pragma unroll
                for (int t = 0; t < FEW_MAX_T; ++t) off[t] = (uint32_t)(__shfl_sync(0xffffffffu, tok, t) * a.stride);
                ok = stages(mine, [&](int c, int k0) {
                    const uint32_t tile = sh.ring + (uint32_t)s * STAGE_BYTES + mytile;
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int kblk = two ? c * 4 + sub : c * 8 + 2 * sub + g;
                        if (kblk < nkb) {
                            const int k = kblk * 32 + 4 * piece - k0;
                            float4 w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int R = rq + 4 * i;
                                const uint4 v = lds128(tile + (uint32_t)(g * KBLK_BYTES + R * 128 + ((piece ^ (R & 7)) << 4)));
                                w[i] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                                                   __uint_as_float(v.w));
                            }
#pragma unroll
                            for (int t = 0; t < FEW_MAX_T; ++t)
                                if (t < ncol) {
                                    const uint4 v = lds128(act + off[t] + (uint32_t)(4 * k));
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        acc[g][i][t] = fmaf(w[i].x, __uint_as_float(v.x), acc[g][i][t]);
                                        acc[g][i][t] = fmaf(w[i].y, __uint_as_float(v.y), acc[g][i][t]);
                                        acc[g][i][t] = fmaf(w[i].z, __uint_as_float(v.z), acc[g][i][t]);
                                        acc[g][i][t] = fmaf(w[i].w, __uint_as_float(v.w), acc[g][i][t]);
                                    }
                                }
                        }
                    }
                    release();
                });
                if (!ok) break;
                if (!mine) continue;
                if (!(ok = cells_free())) break;
#pragma unroll
                for (int t = 0; t < FEW_MAX_T; ++t)
                    if (t < ncol) {
#pragma unroll
                        for (int g = 0; g < 2; ++g)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
#pragma unroll
                                for (int off = 1; off < 8; off <<= 1)
                                    acc[g][i][t] += __shfl_xor_sync(0xffffffffu, acc[g][i][t], off);
                                if (piece == 0) myred[g * RED_GROUP + (rq + 4 * i) * 8 + t] = acc[g][i][t];
                            }
                    }
            } else {
                float acc[2][4] = {};
                // where column r's activations are
                auto column = [&](int r) -> uint32_t {
                    return (uint32_t)(__shfl_sync(0xffffffffu, tok, packed ? (r & 3) : r) * a.stride) +
                           (packed && r >= 4 ? plane : 0u);
                };
                if (mx4) {
                    // ---- 4-bit rows: a 16-byte piece of a row is one block of 32 values, eight of
                    // them (a word) per lane
                    const int nblk = (kind == ROUTED_GU ? p.l : p.f) / 32;
                    const uint32_t mycol = column(gid) + 16u * c4;
                    ok = stages(mine, [&](int c, int k0) {
                        const int kblk = c * 4 + sub;
                        const int nb = min(nblk - kblk * 8, 8);
                        if (nb > 0) {
                            const uint32_t tile = sh.ring + (uint32_t)s * STAGE_BYTES + mytile + 128u * gid;
                            const uint32_t sc = sh.scales + (uint32_t)(s * SCALE_BYTES + 32 * gid + 8 * sub);
                            const uint32_t arow = act + mycol + (uint32_t)(2 * (kblk * 256 - k0));
                            if (packed) mx4_kblock<true>(acc, tile, arow, 0u, sc, gid, c4, nb);
                            else mx4_kblock<false>(acc, tile, arow, plane, sc, gid, c4, nb);
                        }
                        release();
                    });
                } else {
                    // ---- bf16 rows: 64 values of 16 rows per tile
                    const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8;
                    const uint32_t mycol = column(lane & 7) + 16u * (lane >> 3);
                    uint32_t piece[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        piece[i] = mytile + (uint32_t)(lrow * 128 + (((2 * i + (lane >> 4)) ^ (lrow & 7)) << 4));
                    const bool lo_too = a.planes == 2 && !packed;
                    float acl[2][4] = {};
                    ok = stages(mine, [&](int c, int k0) {
                        const uint32_t tile = sh.ring + (uint32_t)s * STAGE_BYTES;
                        const int kblk = two ? c * 4 + sub : c * 8 + 2 * sub;
                        if (kblk < nkb) {
                            const uint32_t arow = act + mycol + (uint32_t)(2 * (kblk * 64 - k0));
                            uint32_t w[2][4][4];
#pragma unroll
                            for (int g = 0; g < 2; ++g)
#pragma unroll
                                for (int i = 0; i < 4; ++i) ldmatrix_x4(w[g][i], tile + piece[i] + (uint32_t)(g * KBLK_BYTES));
                            release();
                            // neighbouring products go to different sums: a chain on one costs its latency
                            auto columns = [&](uint32_t (&x)[8], uint32_t at) {
                                uint32_t y[4];
                                ldmatrix_x4(y, at);
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[i] = y[i];
                                ldmatrix_x4(y, at + 64u);
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[4 + i] = y[i];
                            };
                            uint32_t b0[8], b1[8];
                            columns(b0, arow);
                            if (two) {
                                if (lo_too) columns(b1, arow + plane);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    mma_bf16(acc[0], w[0][i], b0[2 * i], b0[2 * i + 1]);
                                    mma_bf16(acc[1], w[1][i], b0[2 * i], b0[2 * i + 1]);
                                    if (lo_too) {
                                        mma_bf16(acl[0], w[0][i], b1[2 * i], b1[2 * i + 1]);
                                        mma_bf16(acl[1], w[1][i], b1[2 * i], b1[2 * i + 1]);
                                    }
                                }
                            } else {                       // the second tile is the next k-block
                                if (kblk + 1 < nkb) columns(b1, arow + 128u);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    mma_bf16(acc[0], w[0][i], b0[2 * i], b0[2 * i + 1]);
                                    if (kblk + 1 < nkb) mma_bf16(acc[1], w[1][i], b1[2 * i], b1[2 * i + 1]);
                                }
                                if (lo_too) {
                                    columns(b0, arow + plane);
                                    if (kblk + 1 < nkb) columns(b1, arow + plane + 128u);
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        mma_bf16(acl[0], w[0][i], b0[2 * i], b0[2 * i + 1]);
                                        if (kblk + 1 < nkb) mma_bf16(acl[1], w[1][i], b1[2 * i], b1[2 * i + 1]);
                                    }
                                }
                            }
                        } else {
                            release();
                        }
                    });
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[0][i] += acl[0][i];
                        acc[1][i] += acl[1][i];
                    }
                }
                if (!ok) break;
                if (!mine) continue;
                if (!(ok = cells_free())) break;
                // 4-bit experts: the activations' scale comes out here, while their slot is held
                float back[2] = {1.f, 1.f};
                if (mx4) {
                    const float *inv = sh.inv + 8 * (set & 1);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int col = 2 * c4 + i;
                        back[i] = inv[__shfl_sync(0xffffffffu, tok, packed ? (col & 3) : col)];
                    }
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    float2 *r = reinterpret_cast<float2 *>(myred + g * RED_GROUP + gid * 8 + 2 * c4);
                    r[0] = make_float2(acc[g][0] * back[0], acc[g][1] * back[1]);
                    r[32] = make_float2(acc[g][2] * back[0], acc[g][3] * back[1]);
                }
            }
            cells_written();
            }
            if (!ok) break;
            done();
        }
        if (!ok && lane == 0) give_up(0x8);
    } else if (warp >= THREADS / 32 - FINISHERS) {
        // ------------------------------------------------------------ finishers
        // A warp for each team: sums over the team's warps and what becomes of them; lane (row, column)
        // of 16 x 2, both groups of rows, then the next two columns
        const int fw = warp - (THREADS / 32 - FINISHERS), row = lane >> 1;
        uint32_t n = 0;                                   // sub-items of the team so far
        bool ok = true;
        for (int q = 0; ok; ++q) {
            if (!(ok = __all_sync(0xffffffffu, wait_published(published, q, abort)))) break;
            const Item it = sh.queue[q % QUEUE];
            const int kind = it.kind;
            if (kind == END) break;
            const bool cells = kind != ROUTER && !weightless(kind);
            const bool routed = kind == ROUTED_GU || kind == ROUTED_DOWN;
            const int ncol = kind == ROUTED_GU ? __popc((unsigned)sh.tab[it.ti].mask) : it.ncol;
            const bool packed = cells && ncol <= 4 && act_plan<WT>(p, it).planes == 2;
            for (int rr = fw; cells && rr < it.reps; rr += 2, ++n) {
                const int r = out_row(kind, it.j0 + rr) + row;
                const float *cell = sh.red + (8 * (n & 1u) + 4 * fw) * RED_WARP + row * 8 + (lane & 1);
#pragma unroll 1
                for (int t0 = 0; t0 < ncol; t0 += 2) {
                    const int t = t0 + (lane & 1);
                    const bool real = t < ncol;
                    if (t0 == 0) {
                        ok = warp_wait(sh.cells + 16u * fw + 8u * (n & 1u), n >> 1 & 1u, abort);
                        if (!ok) break;
                    }
                    float add = 0.f;
                    int slot = -1;
                    if (kind == UP) {        // (complete only now: the products' activations waited for the shared experts)
                        if (real) {
                            const float *q2 = p.part + (int64_t)t * p.d + r;
                            add = __ldcg(q2) + __ldcg(q2 + (int64_t)p.T * p.d);
                        }
                    } else if (routed && real) {
                        slot = sh.tab[it.ti].slot[t];
                        if (kind == ROUTED_DOWN) add = sh.select.weight[slot];
                    }
                    const float v0 = red_sum(cell + t0, packed), v1 = red_sum(cell + t0 + RED_GROUP, packed);
                    if (kind == SHARED_GU || kind == ROUTED_GU) {
                        const float h = glu_act(p.act, v0, v1, p.gate_cap, p.up_cap);
                        if (kind == SHARED_GU) {
                            if (real) p.hs[(int64_t)t * 2 * p.fs + r] = h;
                        } else {
                            if (real) p.H[(int64_t)slot * p.f + r] = h;
                            if (WT == W_MX4) largest_of_rows(p.ctl + C_AMAX_H + slot, h, real, lane);
                        }
                    } else if (kind == DOWN) {
                        const float z = v0 + v1;
                        if (real) p.z[(int64_t)t * p.l + r] = z;
                        if (WT == W_MX4) largest_of_rows(p.ctl + C_AMAX_Z + t, z, real, lane);
                    } else if (kind == UP) {
                        if (real) store_token<WT>(p.y, (int64_t)t * p.d + r, v0 + v1 + add);
                    } else if (kind == SHARED_DOWN) {
                        if (real) {
                            float *q2 = p.part + ((int64_t)it.ti * p.T + t) * p.d + r;
                            q2[0] = v0;
                            q2[16] = v1;
                        }
                    } else if (real) {
                        float *q2 = p.ysl + (int64_t)slot * p.l + r;
                        q2[0] = add * v0;
                        q2[16] = add * v1;
                    }
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(sh.free + 16u * fw + 8u * (n & 1u));
            }
            __syncwarp();
            if (ok && lane == 0) sts_release(smem_u32(sh.flags + 32 + CONSUMERS + fw), (unsigned)(q + 1));
        }
        if (!ok && lane == 0) give_up(0x40);
    } else {
        // ------------------------------------------------------------ signaller
        if (lane == 0) {
            bool ok = true;
            for (int q = 0; ok; ++q) {
                passed[LOADERS + 1] = q;
                if (!(ok = wait_published(published, q, abort))) break;
                const int kind = sh.queue[q % QUEUE].kind;
                if (kind == END) break;
                const uint32_t word = smem_u32(sh.flags + 32);
                const long long t1 = clock64();
                for (int w = 0; w < CONSUMERS + FINISHERS; ++w)
                    while ((int)lds_acquire(word + 4 * w) <= q && ok) {
                        __nanosleep(20);
                        if (*abort || clock64() - t1 > 2 * WAIT_LIMIT_CYCLES) ok = false;
                    }
                if (!ok) break;
                const int at = kind == ROUTER        ? C_ROUTER
                               : kind == DOWN        ? C_Z
                               : kind == SHARED_GU   ? C_HS
                               : kind == ROUTED_GU   ? C_H
                               : kind == SHARED_DOWN ? C_PART
                               : kind == ROUTED_DOWN ? C_YS
                               : kind == COMBINE     ? C_U
                                                     : C_WORDS;
                if (at < C_WORDS) red_release(p.ctl + at, 1u);      // (nothing waits for UP)
            }
            if (!ok) give_up(0x20);
        }
    }

    __syncthreads();
    if (*abort && threadIdx.x == 0) {
        // copies in flight must land before the block's memory goes away: the last
        // use of every stage, and the last two sets of x (each wait bounded)
        int none = 0;
        const int sets = sh.flags[3];
        for (int team = 0; team < 2; ++team) {
            const int issued = sh.flags[26 + team], n2 = team ? S - half : half, at = team ? half : 0;
            for (int i = max(0, issued - n2); i < issued; ++i)
                mbar_wait(sh.full + 8u * (at + i % n2), (uint32_t)(i / n2) & 1u, &none);
        }
        for (int i = max(0, sets - 2); i < sets; ++i)
            if (!mbar_wait(sh.act_full + 8u * (i & 1), (uint32_t)(i >> 1) & 1u, &none)) break;
    }
}

// ------------------------------------------------------------------ host side
size_t fixed_smem(const lmoe_config &c, int T)
{
    const int E128 = (c.E + 127) / 128 * 128, TK8 = (T * c.k + 7) / 8 * 8;
    return 1024 + 4 * RED_FLOATS + SUM_BYTES + 4 * (size_t)E128 + 6 * (size_t)TK8 +
           sizeof(Touched) * (size_t)std::min(TK8, E128) + 16 + sizeof(Item) * QUEUE + 8 * (2 * MAX_STAGES + 14) +
 64 + 64 + 192;
}

struct FewLayout {
    size_t ctl, r64, z, hs, H, part, ysl, u, ssq, total;
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
    L.z = take(c.standard ? 0 : 4 * (size_t)T * c.l);
    L.hs = take(4 * (size_t)T * 2 * c.f_shared);
    L.H = take(4 * S * c.f);
    L.part = take(8 * (size_t)T * c.d);
    L.ysl = take(4 * S * c.l);
    L.u = take(c.standard ? 0 : 4 * (size_t)T * c.l);
    L.ssq = take(c.standard ? 0 : 4 * (size_t)T * (c.l / 32));
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

namespace {
// Sub-items per item: pairs (one for each team) until an item has ITEM_BYTES, but leaving every block about
// eight items of the phase, or two where sub-items are below 64 KB: there the costs per item (its activations,
// its signal) weigh more than the blocks' uneven ends.  Eight against two: 1 token at d 2048 60 against 56 us, 6
// tokens with 4-bit experts at d 7168 365 against 351; above 64 KB four against eight: 159 against 156 us.
int reps_for(int64_t sub_bytes, int64_t subs, int blocks)
{
    const int64_t most = std::min<int64_t>(MAX_REPS, ITEM_BYTES / sub_bytes) / 2 * 2;
    const int64_t items = sub_bytes < 64 * 1024 ? 2 : 8;
    return (int)std::max<int64_t>(2, std::min<int64_t>(most, subs / (items * blocks) / 2 * 2));
}

Plan make_plan(const lmoe_config &c, bool mx4, int T, int blocks)
{
    const int64_t eb = c.dtype == LMOE_F32 ? 4 : 2;
    auto row = [&](int64_t K, bool routed) { return mx4 && routed ? K / 2 + K / 32 : K * eb; };
    auto items = [](int64_t subs, int reps) { return (int)((subs + reps - 1) / reps); };
    // touched experts, were the selections independent and even
    double miss = 1.0;
    for (int t = 0; t < T; ++t) miss *= 1.0 - (double)c.k / c.E;
    const int64_t touched = std::max<int64_t>(1, (int64_t)(c.E * (1.0 - miss)));
    Plan n = {};
    const int64_t down = 16 * row(c.d, false), sgu = 32 * row(c.d, false), rgu = 32 * row(c.l, true),
                  sd = 32 * row(c.f_shared, false), rd = 32 * row(c.f, true), up = 16 * row(c.l, false);
    n.router_n = (c.E + 3) / 4;
    n.combine_n = c.l / 32;
    n.down_r = reps_for(down, c.l / 16, blocks);
    n.down_n = c.standard ? 0 : items(c.l / 16, n.down_r);
    n.sgu_r = reps_for(sgu, c.f_shared / 8, blocks);
    n.sgu_n = items(c.f_shared / 8, n.sgu_r);
    n.rgu_r = reps_for(rgu, touched * (c.f / 16), blocks);
    n.rgu_n = items(c.f / 16, n.rgu_r);
    n.sd_r = reps_for(sd, c.d / 16, blocks);
    n.sd_n = items(c.d / 32, n.sd_r);
    n.rd_r = reps_for(rd, touched * (c.l / 32), blocks);
    n.rd_n = items(c.l / 32, n.rd_r);
    n.up_r = reps_for(up, c.d / 16, blocks);
    n.up_n = c.standard ? 0 : items(c.d / 16, n.up_r);
    n.rgu_inv = 1.0f / (float)n.rgu_n;
    n.rd_inv = 1.0f / (float)n.rd_n;
    return n;
}
}  // namespace

size_t few_workspace_bytes(const lmoe_config &c, int64_t T) { return T > 0 ? few_layout(c, T).total : 0; }

bool few_make_maps(const lmoe_config &c, const FewWeights &w, FewMaps *m)
{
    const bool f32 = c.dtype == LMOE_F32;
    const CUtensorMapDataType ty = f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint32_t ke = f32 ? 32 : 64;
    const uint64_t eb = f32 ? 4 : 2;
    // Rows of K values as 128-byte k-blocks.  One group: a box is eight k-blocks of
    // 16 rows.  Two groups: rows in blocks of `block` (64, for 4 bits 32: gate
    // and up alternate; 16: consecutive rows), a box is four k-blocks of 16 rows of two blocks.
    auto one = [&](CUtensorMap *t, const void *base, uint64_t K, uint64_t nrows) {
        return tc_encode_map(t, ty, base, 3, {ke, nrows, K / ke}, {K * eb, 128}, {ke, 16, 8}, true);
    };
    auto two = [&](CUtensorMap *t, const void *base, uint64_t K, uint64_t nrows, uint64_t block) {
        return tc_encode_map(t, ty, base, 4, {ke, block, nrows / block, K / ke}, {K * eb, K * eb * block, 128},
                             {ke, 16, 2, 4}, true);
    };
    auto codes = [&](CUtensorMap *t, const void *base, uint64_t K, uint64_t nrows, uint64_t block) {
        return tc_encode_map(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 4, {128, block, nrows / block, (K / 2 + 127) / 128},
                             {K / 2, K / 2 * block, 128}, {128, 16, 2, 4}, true);
    };
    auto scales = [&](CUtensorMap *t, const void *base, uint64_t K, uint64_t nrows, uint64_t block) {
        const uint64_t pitch = (uint64_t)mx4_scale_pitch((int64_t)K);
        return tc_encode_map(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, 3, {pitch, block, nrows / block},
                             {pitch, pitch * block}, {32, 16, 2}, false);
    };
    const uint64_t E = (uint64_t)c.E, d = (uint64_t)c.d, l = (uint64_t)c.l, f = (uint64_t)c.f, fs = (uint64_t)c.f_shared;
    const uint64_t cat = 2 * fs + (c.standard ? 0 : l);
    *m = FewMaps{};
    const bool ok = tc_encode_map(&m->router, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, w.Wr, 3, {32, E, d / 32}, {d * 4, 128},
                                  {32, 4, 32}, true) &&
                    (c.standard || (one(&m->down, w.Wdown, d, l) && one(&m->up, w.Wcat, cat, d))) &&
                    two(&m->shared_gu, w.Wgu_s, d, 4 * fs, 64) && two(&m->shared_down, w.Wcat, cat, d, 16);
    if (w.mx4)
        return ok && codes(&m->routed_gu, w.Wgu, l, E * 2 * f, 32) && codes(&m->routed_down, w.D, f, E * l, 16) &&
               scales(&m->routed_gu_scales, w.Wgu_scales, l, E * 2 * f, 32) &&
               scales(&m->routed_down_scales, w.D_scales, f, E * l, 16);
    return ok && two(&m->routed_gu, w.Wgu, l, E * 2 * f, 64) && two(&m->routed_down, w.D, f, E * l, 16);
}

cudaError_t few_largest(const float *v, int64_t n, uint32_t *top, cudaStream_t s)
{
    cudaError_t e = cudaMemsetAsync(top, 0, sizeof(uint32_t), s);
    if (e != cudaSuccess) return e;
    largest_kernel<<<1024, 256, 0, s>>>((const uint32_t *)v, n, top);
    return cudaGetLastError();
}

cudaError_t few_launch(const lmoe_config &c, const FewMaps &m, const FewWeights &w, const float *bias, const void *x, int T,
                       void *y, int32_t *sel, void *p_out, void *u_out, void *workspace, bool stall_test,
                       cudaStream_t s)
{
    const bool mx4 = w.mx4;
    const FewLayout L = few_layout(c, T);
    char *ws = (char *)workspace;
    FewParams p = {};
    p.n = make_plan(c, mx4, T, tc_num_sms());
    p.T = T; p.d = c.d; p.l = c.l; p.f = c.f; p.E = c.E; p.k = c.k; p.fs = c.f_shared; p.act = c.act;
    p.standard = c.standard; p.gate_cap = c.gate_cap; p.up_cap = c.up_cap; p.eps = c.eps;
    p.x = x; p.bias = bias; p.Wr = w.Wr; p.wr_top = w.Wr_top; p.y = y; p.p_out = p_out; p.u_out = u_out; p.sel = sel;
    p.ctl = (unsigned *)(ws + L.ctl); p.r64 = (double *)(ws + L.r64);
    p.z = (float *)(ws + L.z); p.hs = (float *)(ws + L.hs); p.H = (float *)(ws + L.H);
    p.part = (float *)(ws + L.part); p.ysl = (float *)(ws + L.ysl); p.u = (float *)(ws + L.u);
    p.ssq = (float *)(ws + L.ssq);
    p.scales = mx4; p.stall_test = stall_test;
    p.wgu = (const char *)w.Wgu; p.wd = (const char *)w.D;
    p.gu_row = mx4 ? c.l / 2 : (int64_t)c.l * (c.dtype == LMOE_F32 ? 4 : 2);
    p.d_row = mx4 ? c.f / 2 : (int64_t)c.f * (c.dtype == LMOE_F32 ? 4 : 2);
    // Activation slots: the longest row set of any item, up to 58 KB (longer ones
    // come in segments); the rest of shared memory is the weight ring.
    const bool f32 = c.dtype == LMOE_F32;
    constexpr int SLOT_MAX = 58 * 1024;
    auto need = [&](int K, int eb, int planes, bool q) { return T * planes * std::min(act_stride(K, eb, q), SLOT_MAX); };
    int slot = need(c.d, f32 ? 4 : 2, 1, false);
    const int two = f32 ? 1 : 2, eb = f32 ? 4 : 2;
    slot = std::max(slot, need(c.l, eb, two, true));
    slot = std::max(slot, need(c.f, eb, two, true));
    slot = std::max(slot, need(c.f_shared, eb, two, true));
    slot = std::min(slot, SLOT_MAX);
    slot = std::max(slot, std::min(T, LOADERS) * select_bytes((c.E + 127) / 128 * 128));     // the selection's scratch
    slot = (slot + 1023) / 1024 * 1024;
    p.slot_bytes = slot;
    const int stage = STAGE_BYTES + (mx4 ? SCALE_BYTES : 0);
    p.stages = std::min(MAX_STAGES, (int)((SMEM_MAX - (int)fixed_smem(c, T) - 2 * slot) / stage));
    const size_t smem = fixed_smem(c, T) + 2 * (size_t)slot + (size_t)p.stages * stage;
    cudaError_t e = cudaMemsetAsync(p.ctl, 0, 4 * C_WORDS, s);
    if (e != cudaSuccess) return e;
    if (f32) return launch<W_F32>(m, p, smem, s);
    if (mx4) return launch<W_MX4>(m, p, smem, s);
    return launch<W_BF16>(m, p, smem, s);
}

}  // namespace lmoe
