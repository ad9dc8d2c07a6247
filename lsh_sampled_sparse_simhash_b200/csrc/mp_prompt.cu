// Causal attention over packed prompts (mp_prompt_attend) on the tcgen05
// tensor cores.
//
// For the token i of a sequence and a query head h of kv head u:
//   s_j = q_ih . k_ju / sqrt(d),  out_ih = sum_{j <= i} e^{s_j} v_ju / sum_{j <= i} e^{s_j}
// in one pass over the keys, with a running maximum and sum per row.  Bound by
// the tensor rate (4 d multiply-adds a visible pair, 128^3 per tile product)
// and, as closely, by the exponentials (one per pair).
//
// An item is 2 kTok tokens of one sequence and one kv head: two 128-row query
// tiles whose rows are (token, head of the group), so the G heads share every
// K and V tile (kTok = 128 / G tokens a tile).  Key tiles are 128 tokens,
// walked from the last visible one down to the first.
//   warps 0-3, 4-7  softmax of query tile 0, 1: thread = row.  S from TMEM,
//                   maximum, P = 2^(s - m) in bf16 back into the columns of S,
//                   sum; rescaling of O (TMEM) only when the maximum grows by
//                   more than 2^8; at the end O / sum to memory.
//   warp 8          MMA issuer (one thread): S = Q K^T, O += P V with P as the
//                   A operand in TMEM; the two tiles alternate, so one tile's
//                   products run under the other's softmax.
//   warp 9          TMA producer: Q (both tiles), then the ring of K and V tiles.
//   warp 10         zeroes the rows of the last V tile behind the sequence's end.
//   warp 11         holds the TMEM allocation.
// TMEM: S0, S1, O0, O1, 128 columns each.
//
// Every wait is bounded (1 s); on expiry MP_ERR_CUDA is recorded and the block
// winds down, waiting for its copies and products in flight.
#include <cuda.h>
#include <math.h>

#include "mp_pages.cuh"

namespace mp {
namespace prompt {

constexpr int kRows = 128;                    // rows of a query tile = TMEM lanes
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kHalfBytes = 128 * 128;         // 128 rows x 64 elements
constexpr int kTileBytes = 2 * kHalfBytes;    // 32 KB
constexpr int kSlots = 5;                     // ring of K and V tiles
constexpr int kSmemBytes = 1024 + (2 + kSlots) * kTileBytes;
constexpr int kWarpMma = 8, kWarpLoad = 9, kWarpFix = 10, kWarpTmem = 11;
constexpr int kThreads = 32 * 12;
constexpr uint32_t kColS = 0, kColO = 256;    // + 128 t
constexpr int kPoly = 2;                      // of 8 pairs of weights, those computed by polynomial
constexpr float kMargin = 8.f;                // log2 units between rescales
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Args {
    PromptShape s;
    const int32_t *cu;
    uint16_t *out;
    float *lse;
    int32_t *status;
    int n_items;  // upper bound
};

enum {
    B_Q = 0,                 // [2] query tile landed
    B_KV = B_Q + 2,          // [kSlots] K or V tile landed
    B_FREE = B_KV + kSlots,  // [kSlots] products on the slot complete
    B_S = B_FREE + kSlots,   // [2] S in TMEM (and all products before it complete)
    B_P = B_S + 2,           // [2] P in TMEM, O rescaled (4 warps)
    B_O = B_P + 2,           // [2] the item's last product into O complete
    B_FIX = B_O + 2,         // last V tile's rows behind the sequence's end zeroed
    B_END = B_FIX + 1,       // teardown
    kBars = B_END + 1
};

__device__ __noinline__ bool wait_slow(uint32_t a, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(a, parity)) {
        if (*abort_flag) return false;
        if (globaltimer() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            set_status(status, MP_ERR_CUDA);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool wait(uint32_t a, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    return mbar_try_wait(a, parity) || wait_slow(a, parity, abort_flag, status);
}
__device__ __forceinline__ bool warp_wait(uint32_t a, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    const bool ok = wait(a, parity, abort_flag, status);
    return __all_sync(0xffffffffu, ok);
}
// Teardown wait: bounded by time alone.
__device__ __noinline__ void wait_teardown(uint32_t a, uint32_t parity)
{
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(a, parity))
        if (globaltimer() - t0 > kWaitLimitNs) return;
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// K-major operand, 128B swizzle: rows of 128 B, 8-row groups 1024 B apart.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// MN-major operand, 128B swizzle (V: rows are keys, the product's K): 64 dims
// to a 128-byte row, 8 keys to a 1024-byte group, the other 64 dims kHalfBytes
// further.
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t saddr)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((kHalfBytes >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: bf16 x bf16 -> f32, M = 128, N = 128; B MN-major if b_mn.
__device__ __forceinline__ constexpr uint32_t idesc(bool b_mn)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accum)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t accum)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
            d),
        "r"(a_tmem), "l"(b), "r"(id), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
// After wait_ld(): the registers of a load may be used from here on (keeps the
// compiler from moving their use over the wait).
__device__ __forceinline__ void tie32(uint32_t *r)
{
#pragma unroll
    for (int i = 0; i < 32; i++) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Two fp32 in a register pair, for the packed add and multiply-add.
__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &x, float &y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// 2^x of a pair on the multiply-add pipe, x <= 126 (below -126: 2^-126).
// x = n + f with n whole and |f| <= 1/2 (adding and taking away 1.5 2^23
// rounds to whole numbers), 2^f by a degree-4 polynomial, n added to the
// exponent.  The coefficients minimise the largest relative error on
// [-1/2, 1/2] (fitted by Lawson's iteration): 2.7e-6 = 2^-18.5.
__device__ __forceinline__ void ex2_poly(uint64_t x2, float &y0, float &y1)
{
    float x0, x1;
    unpair(x2, x0, x1);
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(x0));  // -126
    asm("max.NaN.f32 %0, %0, 0fC2FC0000;" : "+f"(x1));
    const uint64_t x = pair(x0, x1);
    const uint64_t t = add2(x, pair(12582912.f, 12582912.f));
    const uint64_t f = add2(x, fma2(t, pair(-1.f, -1.f), pair(12582912.f, 12582912.f)));
    uint64_t p = fma2(f, pair(0.009570102207362652f, 0.009570102207362652f), pair(0.05591785907745361f, 0.05591785907745361f));
    p = fma2(p, f, pair(0.240247443318367f, 0.240247443318367f));
    p = fma2(p, f, pair(0.6931217908859253f, 0.6931217908859253f));
    p = fma2(p, f, pair(0.9999992847442627f, 0.9999992847442627f));
    float t0, t1, p0, p1;
    unpair(t, t0, t1);
    unpair(p, p0, p1);
    y0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(t0) << 23));
    y1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(t1) << 23));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Keys past the row's last visible one (lim: its column within these 32) get
// a score of -inf.
__device__ __forceinline__ void hide(uint32_t *u, int lim)
{
#pragma unroll
    for (int c = 0; c < 32; c++)
        if (c > lim) u[c] = 0xff800000u;
}

__device__ __forceinline__ void row_max(const uint32_t *u, float *mx)
{
#pragma unroll
    for (int c = 0; c < 32; c += 8)
#pragma unroll
        for (int i = 0; i < 4; i++)
            mx[i] = max3(mx[i], __uint_as_float(u[c + 2 * i]), __uint_as_float(u[c + 2 * i + 1]));
}

// The weights of 32 keys of a row, 2^(s scale + ms), as bf16 into 16 columns
// at p_col, and their sums (of the unrounded values) into l.  NPOLY of every 8
// pairs go by ex2_poly, the others by the special function unit.
template <int NPOLY>
__device__ __forceinline__ void weights(const uint32_t *u, uint64_t scale2, uint64_t ms, uint64_t *l, uint32_t p_col)
{
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const uint64_t x = fma2(pair(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), scale2, ms);
        float e0, e1;
        if ((i * NPOLY) % 8 < NPOLY) {
            ex2_poly(x, e0, e1);
        } else {
            unpair(x, e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
        }
        l[i & 1] = add2(l[i & 1], pair(e0, e1));
        p[i] = pack_bf16(e0, e1);
    }
    tmem_st16(p_col, p);
}

// All 128 weights of a row: keys 0..63 are in a and b, the others come from
// TMEM once more (three buffers of 32 scores; all 128 at once spill).
template <int NPOLY>
__device__ __forceinline__ void weights_row(uint32_t *a, uint32_t *b, int lim, uint64_t scale2, uint64_t ms, uint64_t *l,
                                            uint32_t s_col)
{
    uint32_t c[32];
    tmem_ld32(s_col + 64, c);
    weights<NPOLY>(a, scale2, ms, l, s_col);
    weights<NPOLY>(b, scale2, ms, l, s_col + 16);
    wait_ld();
    tie32(c);
    if (NPOLY == 0) hide(c, lim - 64);
    tmem_ld32(s_col + 96, a);
    weights<NPOLY>(c, scale2, ms, l, s_col + 32);
    wait_ld();
    tie32(a);
    if (NPOLY == 0) hide(a, lim - 96);
    weights<NPOLY>(a, scale2, ms, l, s_col + 48);
}

// One item: tokens [m0, m0 + 2 kTok) of the sequence of n tokens whose rows
// start at row0.
struct Item {
    int kvh, row0, n, m0;
};

// Rows of sequence b; a pair of entries that breaks the rules holds none.
__device__ __forceinline__ int seq_rows(const Args &a, int b, int &row0)
{
    const int lo = a.cu[b], hi = a.cu[b + 1];
    row0 = lo;
    return lo < 0 || hi < lo || hi > a.s.T ? 0 : hi - lo;
}

// The item of rank r, longest rows first.  With c_b = ceil(n_b / M) items in
// sequence b (M tokens each), F(x) = sum_b max(0, c_b - x) items have index >=
// x in their sequence; rank r has the largest index x with F(x) > r, in the
// (r - F(x + 1))-th sequence that has one.  Run by one warp; false: no such item.
__device__ __forceinline__ bool item_of(const Args &a, int r, int M, int lane, Item &it)
{
    const int Hkv = a.s.Hkv, B = a.s.B;
    it.kvh = r % Hkv;
    r /= Hkv;
    auto F = [&](int x) {
        int f = 0, row0;
        for (int b = lane; b < B; b += 32) f += max((seq_rows(a, b, row0) + M - 1) / M - x, 0);
        return __reduce_add_sync(0xffffffffu, f);
    };
    if (F(0) <= r) return false;
    int lo = 0, hi = (a.s.T + M - 1) / M;  // F(lo) > r >= F(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (F(mid) > r) lo = mid;
        else hi = mid;
    }
    int k = r - F(lo + 1);
    for (int b0 = 0; b0 < B; b0 += 32) {
        int row0 = 0, n = 0;
        if (b0 + lane < B) n = seq_rows(a, b0 + lane, row0);
        const unsigned has = __ballot_sync(0xffffffffu, (n + M - 1) / M > lo);
        const int here = __popc(has);
        if (k < here) {
            const int l = (int)__fns(has, 0, k + 1);
            it.n = __shfl_sync(0xffffffffu, n, l);
            it.row0 = __shfl_sync(0xffffffffu, row0, l);
            it.m0 = lo * M;
            return true;
        }
        k -= here;
    }
    return false;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attend_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv, const Args a)
{
    constexpr int kTok = kRows / G;  // tokens of a query tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kBars];
    __shared__ uint32_t tmem_sh;
    __shared__ Item item_sh;
    __shared__ int live_sh;
    __shared__ volatile int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_smem = smem, ring = smem + 2 * kTileBytes;
    const uint32_t bar0 = smem_u32(&bars[0]);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    grid_dependency_wait();

    if (blockIdx.x == 0)
        for (int b = tid; b < a.s.B; b += kThreads) {
            const int lo = a.cu[b], hi = a.cu[b + 1];
            if (lo < 0 || hi < lo || hi > a.s.T) set_status(a.status, MP_ERR_CAPACITY);
        }
    if (warp == 0) {
        Item it;
        const bool live = item_of(a, blockIdx.x, 2 * kTok, lane, it);
        if (lane == 0) {
            live_sh = live;
            item_sh = it;
            abort_flag = 0;
            for (int i = 0; i < kBars; i++) mbar_init(bar(i), i == B_P || i == B_P + 1 ? 4 : 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
    }
    __syncthreads();
    if (!live_sh) return;
    if (warp == kWarpTmem) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_sh)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_sh;
    const Item it = item_sh;
    const int last_tok = min(it.m0 + 2 * kTok, it.n) - 1;  // the item's last token
    const int nt = last_tok / kKeys + 1;                   // key tiles, walked from nt - 1 to 0
    const bool fix = nt * kKeys > it.n;                    // the first of them has rows behind the sequence's end

    if (warp == kWarpLoad && lane == 0) {
        // ------------------------------------------------------- producer ----
        for (int t = 0; t < 2; t++) {
            mbar_expect_tx(bar(B_Q + t), 2 * kTok * G * 128);
            for (int h = 0; h < 2; h++)
                tma_3d(q_smem + t * kTileBytes + h * kHalfBytes, &mq, bar(B_Q + t), 64 * h, it.kvh * G,
                       it.row0 + it.m0 + t * kTok);
            if (t == 0) {  // the first K tile before the second query tile
                mbar_expect_tx(bar(B_KV), kTileBytes);
                for (int h = 0; h < 2; h++)
                    tma_3d(ring + h * kHalfBytes, &mk, bar(B_KV), 64 * h, it.kvh, it.row0 + (nt - 1) * kKeys);
            }
        }
        int last = 0;
        for (int i = 1; i < 2 * nt; i++) {  // tile i: K (even) or V (odd) of key tile nt - 1 - i / 2
            const int slot = i % kSlots;
            if (i >= kSlots && !wait(bar(B_FREE + slot), (i / kSlots - 1) & 1, &abort_flag, a.status)) break;
            mbar_expect_tx(bar(B_KV + slot), kTileBytes);
            for (int h = 0; h < 2; h++)
                tma_3d(ring + slot * kTileBytes + h * kHalfBytes, (i & 1) ? &mv : &mk, bar(B_KV + slot), 64 * h, it.kvh,
                       it.row0 + (nt - 1 - i / 2) * kKeys);
            last = i;
        }
        // own copies land before the block leaves
        wait_teardown(bar(B_Q), 0);
        wait_teardown(bar(B_Q + 1), 0);
        for (int i = max(0, last - kSlots + 1); i <= last; i++) wait_teardown(bar(B_KV + i % kSlots), (i / kSlots) & 1);
    } else if (warp == kWarpMma && lane == 0) {
        // ------------------------------------------------------------ MMA ----
        auto qk = [&](int t, int slot) {
#pragma unroll
            for (int ks = 0; ks < 8; ks++) {
                const uint32_t off = (uint32_t)((ks >> 2) * kHalfBytes + (ks & 3) * 32);
                mma_ss(tmem + kColS + 128 * t, desc_kmajor(q_smem + t * kTileBytes + off),
                       desc_kmajor(ring + slot * kTileBytes + off), idesc(false), ks > 0);
            }
        };
        auto pv = [&](int t, int slot, bool accum) {
#pragma unroll
            for (int ks = 0; ks < 8; ks++)
                mma_ts(tmem + kColO + 128 * t, tmem + kColS + 128 * t + 8 * ks,
                       desc_mnmajor(ring + slot * kTileBytes + ks * 2048), idesc(true), accum || ks > 0);
        };
        auto arrived = [&](int i) { return wait(bar(B_KV + i % kSlots), (i / kSlots) & 1, &abort_flag, a.status); };
        bool ok = true;
        for (int t = 0; t < 2 && ok; t++) {
            ok = wait(bar(B_Q + t), 0, &abort_flag, a.status) && arrived(0);
            if (!ok) break;
            fence_after();
            qk(t, 0);
            commit(bar(B_S + t));
        }
        if (ok) commit(bar(B_FREE));
        for (int j = 0; j < nt && ok; j++) {
            const int vi = 2 * j + 1, ki = 2 * j + 2;
            ok = arrived(vi) && (j > 0 || !fix || wait(bar(B_FIX), 0, &abort_flag, a.status));
            for (int t = 0; t < 2 && ok; t++) {
                ok = wait(bar(B_P + t), j & 1, &abort_flag, a.status);
                if (!ok) break;
                fence_after();
                pv(t, vi % kSlots, j > 0);
                if (j + 1 == nt) {
                    commit(bar(B_O + t));
                } else {
                    ok = arrived(ki);
                    if (!ok) break;
                    qk(t, ki % kSlots);
                    commit(bar(B_S + t));
                }
            }
            if (!ok) break;
            commit(bar(B_FREE + vi % kSlots));
            if (j + 1 < nt) commit(bar(B_FREE + ki % kSlots));
        }
        commit(bar(B_END));
        wait_teardown(bar(B_END), 0);
    } else if (warp == kWarpFix && fix) {
        // --------------------------- zero V behind the end of the sequence ----
        if (warp_wait(bar(B_KV + 1), 0, &abort_flag, a.status)) {
            const int r0 = it.n - (nt - 1) * kKeys;  // first row of the tile behind the end
            for (int i = lane; i < (kKeys - r0) * 16; i += 32) {
                const uint32_t at = ring + kTileBytes + (uint32_t)((i & 1) * kHalfBytes + r0 * 128 + (i >> 1) * 16);
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_FIX));
        }
    } else if (warp < 8) {
        // --------------------------------------------------------- softmax ----
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_col = tmem + lanes + kColS + 128 * t, o_col = tmem + lanes + kColO + 128 * t;
        const int tok = it.m0 + t * kTok + r / G, head = r % G;
        const bool stored = r < kTok * G && tok < it.n;
        const int limit = r < kTok * G ? min(tok, it.n - 1) : -1;  // last visible key
        const float scale2 = kLog2e * 0.08838834764831845f;        // log2(e) / sqrt(128)
        float m = -INFINITY;
        uint64_t l[2] = {0ull, 0ull};  // four partial sums
        bool ok = true;
        for (int j = 0; j < nt; j++) {
            if (!warp_wait(bar(B_S + t), j & 1, &abort_flag, a.status)) {
                ok = false;
                break;
            }
            fence_after();
            const int lim = limit - (nt - 1 - j) * kKeys;
            const bool masked = __any_sync(0xffffffffu, lim < kKeys - 1);
            uint32_t ua[32], ub[32];
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 2; c >= 0; c -= 2) {
                tmem_ld32(s_col + 32 * c, ua);
                tmem_ld32(s_col + 32 * c + 32, ub);
                wait_ld();
                tie32(ua);
                tie32(ub);
                if (masked) {
                    hide(ua, lim - 32 * c);
                    hide(ub, lim - 32 * c - 32);
                }
                row_max(ua, mx);
                row_max(ub, mx);
            }
            const float top = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * scale2;
            const bool grow = top > m + kMargin;
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? (m == -INFINITY ? 0.f : ex2(m - top)) : 1.f;
                if (grow) m = top;
                l[0] = fma2(l[0], pair(f, f), 0ull);
                l[1] = fma2(l[1], pair(f, f), 0ull);
                if (j > 0) {  // every product into O so far is complete (it was issued before this S)
#pragma unroll 1
                    for (int c = 0; c < 4; c++) {
                        uint32_t o[32];
                        tmem_ld32(o_col + 32 * c, o);
                        wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(o_col + 32 * c, o);
                    }
                }
            }
            const float ms = m == -INFINITY ? 0.f : -m;
            const uint64_t scale_2 = pair(scale2, scale2), ms_2 = pair(ms, ms);
            // hidden keys have to come out as 0 and not as 2^-126: a masked tile takes the exact path
            if (masked) {
                weights_row<0>(ua, ub, lim, scale_2, ms_2, l, s_col);
            } else {
                weights_row<kPoly>(ua, ub, lim, scale_2, ms_2, l, s_col);
            }
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + t));
        }
        if (ok && warp_wait(bar(B_O + t), 0, &abort_flag, a.status)) {
            fence_after();
            const size_t row = (size_t)(it.row0 + tok) * a.s.Hq + (size_t)it.kvh * G + head;
            float l0, l1;
            unpair(add2(l[0], l[1]), l0, l1);
            const float sum = l0 + l1, inv = 1.f / sum;
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + row * kHeadDim);
            uint32_t o[128];
#pragma unroll
            for (int c = 0; c < 4; c++) tmem_ld32(o_col + 32 * c, o + 32 * c);
            wait_ld();
            if (stored) {
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    uint32_t v[4];
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        v[k] = pack_bf16(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                    dst[i] = make_uint4(v[0], v[1], v[2], v[3]);
                }
            }
            if (stored && a.lse) a.lse[row] = (m + log2f(sum)) * kLn2;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kWarpTmem) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
}

// [rows][heads][128] view with rows `stride` elements apart; a box is 64
// elements of `heads_box` heads of `rows_box` rows.
static bool make_map(CUtensorMap *m, const void *ptr, int rows, int heads, int64_t stride, int heads_box, int rows_box)
{
    const uint64_t dims[3] = {kHeadDim, (uint64_t)heads, (uint64_t)rows};
    const uint64_t strides[2] = {2 * kHeadDim, 2 * (uint64_t)stride};
    const uint32_t box[3] = {64, (uint32_t)heads_box, (uint32_t)rows_box};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, ptr, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int G>
static cudaError_t launch_g(const PromptShape &s, const uint16_t *q, const uint16_t *k, const uint16_t *v, Args a,
                            cudaStream_t st)
{
    constexpr int kTok = kRows / G;
    CUtensorMap mq, mk, mv;
    if (!make_map(&mq, q, s.T, s.Hq, s.qs, G, kTok) || !make_map(&mk, k, s.T, s.Hkv, s.ks, 1, kKeys) ||
        !make_map(&mv, v, s.T, s.Hkv, s.vs, 1, kKeys))
        return cudaErrorInvalidValue;
    const long long items = ((long long)s.T / (2 * kTok) + s.B) * s.Hkv;  // sum ceil(n_b / M) <= T / M + B
    if (items > 0x7fffffffll) return cudaErrorInvalidValue;
    const void *fn = reinterpret_cast<const void *>(prompt_attend_kernel<G>);
    cudaError_t e = ensure_smem(fn, kSmemBytes);
    if (e != cudaSuccess) return e;
    a.n_items = (int)items;
    return launch_pdl(prompt_attend_kernel<G>, dim3((unsigned)items), dim3(kThreads), kSmemBytes, st, mq, mk, mv, a);
}

}  // namespace prompt

cudaError_t launch_prompt(const PromptShape &s, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                          const int32_t *cu_lens, uint16_t *out, float *lse, int32_t *status, cudaStream_t st)
{
    if (s.T == 0) return cudaSuccess;
    prompt::Args a;
    a.s = s;
    a.cu = cu_lens;
    a.out = out;
    a.lse = lse;
    a.status = status;
    a.n_items = 0;
    switch (s.G) {
    case 1: return prompt::launch_g<1>(s, q, k, v, a, st);
    case 2: return prompt::launch_g<2>(s, q, k, v, a, st);
    case 3: return prompt::launch_g<3>(s, q, k, v, a, st);
    case 4: return prompt::launch_g<4>(s, q, k, v, a, st);
    case 5: return prompt::launch_g<5>(s, q, k, v, a, st);
    case 6: return prompt::launch_g<6>(s, q, k, v, a, st);
    case 7: return prompt::launch_g<7>(s, q, k, v, a, st);
    case 8: return prompt::launch_g<8>(s, q, k, v, a, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace mp
