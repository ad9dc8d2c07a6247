// Causal attention over packed prompts (mp_prompt_attend) on the tcgen05
// tensor cores.
//
// For the token i of a sequence and a query head h of kv head u:
//   s_j = q_ih . k_ju / sqrt(d),  out_ih = sum_{j <= i} e^{s_j} v_ju / sum_{j <= i} e^{s_j}
// in one pass over the keys, with a running maximum and sum per row.  Bound by
// the tensor rate (2 x 128^3 multiply-adds a tile of 128 rows and 128 keys) and,
// as closely, by the exponentials (128^2 a tile, 16 a cycle and SM): 1024
// cycles each at the nominal rates.  Measured at 16384 tokens, 32 / 8 heads:
// 1.85 ms, 1190 TFLOP/s of causal work (72% of the measured burst rate of a
// library product, 90% of its rate under the power cap, which holds here too),
// tensor pipe and special functions 64% busy each.
//
// An item is 2 kTok tokens of one sequence and one kv head: two 128-row query
// tiles whose rows are (token, head of the group), so the G heads share every
// K and V tile (kTok = 128 / G tokens a tile).  Key tiles are 128 tokens,
// walked from the last visible one down to the first; a query tile joins at
// its own last one.  One block per SM lives on by taking over the blocks of the
// grid that have not started yet, an item each, longest first:
//   warps 0-3, 4-7  softmax of query tile 0, 1: thread = row.  S from TMEM,
//                   P = 2^(s - m) in bf16 back into the columns of S, sum; at
//                   the end of an item O / sum to memory.
//   warp 8          MMA issuer: S = Q K^T, O += P V with P as the A operand in
//                   TMEM; the two tiles alternate, so one tile's products run
//                   under the other's softmax, and the first S of the next
//                   item under the last softmax of this one.
//   warp 9          TMA producer: Q (both tiles), the ring of K and V tiles.
//   warp 10         zeroes the rows of the last V tile behind the sequence's end.
//   warp 11         finds the next items; holds the TMEM allocation.
// TMEM: S0, S1, O0, O1, 128 columns each.
//
// Where a round (both query tiles over one key tile, about 3100 cycles) goes:
// a tile's softmax takes 1950 and its products 1100 before the next S is there,
// one after the other, and TMEM has no room for a third S.  The 32 products of
// a round alone take 2580 (80 cycles each where 64 are nominal, alike with Q
// from TMEM and without copies: an N = 128 product's own overhead), so no order
// of the rest gets below that.  Measured and not kept: 16 softmax warps with 64
// keys each (16k tokens 2.06 ms: they have to agree on the reference through
// shared memory, whose bandwidth the products use up), key tiles of 64 with two
// S each (products 3310 a round), an eighth to a half of the exponentials by a
// polynomial (within 2%: the power cap), all 128 scores of a row in registers
// (within 1%).
//
// Every wait is bounded (4 s, as a role may wait for a whole item of the others:
// 262144 rounds for the last of 2^25 tokens, 0.41 s at 1965 MHz and 0.69 s at the
// 1185 MHz of a long run under the power cap); on expiry MP_ERR_CUDA is recorded
// and the block winds down, waiting (1 s each) for its copies and products in
// flight.
#include <cuda.h>
#include <math.h>

#include "mp_pages.cuh"

namespace mp {
namespace prompt {

constexpr int kRows = 128;                    // rows of a query tile = TMEM lanes
constexpr int kKeys = 128;                    // keys of a tile
constexpr int kHalfBytes = 128 * 128;         // 128 rows x 64 elements
constexpr int kTileBytes = 2 * kHalfBytes;    // 32 KB
constexpr int kSlots = 4;                     // ring of K and V tiles
constexpr int kStageBytes = 4096;             // a softmax warp's stage for results: 32 rows x 64 dims
constexpr int kItems = 2;                     // items known: the running one and the next
constexpr int kFixes = 4;                     // more than the V tiles that the ring can hold
constexpr int kSmemBytes = 1024 + (2 + kSlots) * kTileBytes + 8 * kStageBytes;
constexpr int kWarpMma = 8, kWarpLoad = 9, kWarpFix = 10, kWarpItems = 11;
constexpr int kThreads = 32 * 12;
constexpr uint32_t kColS = 0, kColO = 256;    // + 128 t
constexpr long long kGroupBytes = 32ll << 20;  // K and V of the items in hand: a quarter of L2 (16 prompts of 8192
                                               // tokens: 6.7 ms, without groups 8.4)
constexpr float kMargin = 24.f;               // log2 units that a score may exceed its row's reference by
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kScale = kLog2e * 0.08838834764831845f;  // log2(e) / sqrt(128)
constexpr float kFar = 67108864.f;            // 2^26: a reference of at least this size is kept as the score itself

struct Args {
    PromptShape s;
    const int32_t *cu;
    uint16_t *out;
    float *lse;
    int32_t *status;
};

enum {
    B_Q = 0,                   // [2] query tile landed
    B_QFREE = B_Q + 2,         // [2] the item's last product on it complete
    B_KV = B_QFREE + 2,        // [kSlots] K or V tile landed (and its rows behind the sequence's end zeroed)
    B_FREE = B_KV + kSlots,    // [kSlots] products on the slot complete
    B_S = B_FREE + kSlots,     // [2] S in TMEM (and all products before it complete)
    B_P = B_S + 2,             // [2][2] P of keys 0-63, 64-127 in TMEM, O rescaled (4 warps each)
    B_O = B_P + 4,             // [2] the item's last product into O complete
    B_FIX = B_O + 2,           // [kFixes] V tile landed that has rows behind the sequence's end, in turn
    B_ITEM = B_FIX + kFixes,   // [kItems] item known
    B_TAKEN = B_ITEM + kItems, // [kItems] item done with by all roles
    B_NEXT = B_TAKEN + kItems, // the next block's number is here
    B_END = B_NEXT + 1,        // teardown
    kBars = B_END + 1
};
constexpr int kRoles = 8 + 3;  // warps that read an item
constexpr unsigned long long kItemWaitNs = 4 * kWaitLimitNs;

__device__ __noinline__ bool wait_slow(uint32_t a, uint32_t parity, volatile int *abort_flag, int32_t *status)
{
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(a, parity)) {
        if (*abort_flag) return false;
        if (globaltimer() - t0 > kItemWaitNs) {
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

// One lane of a converged warp, always the same.
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// Takes the next block of the grid that has not started: it will not start
// any more, and its number arrives at dst (16 bytes) and completes on bar.
__device__ __forceinline__ void next_block(uint32_t dst, uint32_t bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst),
                 "r"(bar)
                 : "memory");
}
// False: there was none left (and none may be asked for again).
__device__ __forceinline__ bool block_taken(uint32_t src, int &block)
{
    uint32_t ok, x;
    asm volatile(
        "{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%2];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
        " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}\n"
        : "=r"(ok), "=r"(x)
        : "r"(src)
        : "memory");
    if (ok) block = (int)x;
    return ok != 0;
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
// at p_col, their sums (of the unrounded values) into l.
__device__ __forceinline__ void weights(const uint32_t *u, uint64_t scale2, uint64_t ms, uint64_t *l, uint32_t p_col)
{
    uint32_t p[16];
#pragma unroll
    for (int i = 0; i < 16; i++) {
        float e0, e1;
        unpair(fma2(pair(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), scale2, ms), e0, e1);
        e0 = ex2(e0);
        e1 = ex2(e1);
        l[i & 1] = add2(l[i & 1], pair(e0, e1));
        p[i] = pack_bf16(e0, e1);
    }
    tmem_st16(p_col, p);
}

// The warp's writes to TMEM so far are complete: tells the MMA issuer.
__device__ __forceinline__ void publish(uint32_t bar, int lane)
{
    wait_st();
    fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
}

// The reference of a row whose sums may be relative to a score beyond kFar.
struct Reference {
    float m;   // log2 units; far: the score
    float f;   // what the sums so far are multiplied by
    bool far;
};
__device__ __forceinline__ bool is_far(float score) { return fabsf(score) >= kFar && fabsf(score) < INFINITY; }

// The reference after a tile whose largest visible score is `top`, in a warp
// that has a far one, before or after; far rows' scores become relative to it,
// in place, and are hidden past lim.  Out of line: it is rare, and a short
// item's code is mostly run from cold instruction caches (4096 one-token prompts
// 0.79 ms, with this in line 0.84, without far references 0.75).
__device__ __noinline__ Reference far_reference(Reference r, float top, int lim, uint32_t s_col)
{
    const float lead = r.far ? (top - r.m) * kScale : top * kScale - r.m;
    r.f = 1.f;
    if (lead > kMargin) {
        const bool far = is_far(top);
        r.f = r.m == -INFINITY ? 0.f
                               : ex2(fmaf((r.far ? r.m : 0.f) - (far ? top : 0.f), kScale,
                                          (r.far ? 0.f : r.m) - (far ? 0.f : top * kScale)));
        r.m = far ? top : top * kScale;
        r.far = far;
    }
    const float base = r.far ? r.m : 0.f;
#pragma unroll 1
    for (int k = 0; k < 4; k++) {
        uint32_t a[32];
        tmem_ld32(s_col + 32 * k, a);
        wait_ld();
        tie32(a);
        hide(a, lim - 32 * k);
#pragma unroll
        for (int i = 0; i < 32; i++) a[i] = __float_as_uint(__uint_as_float(a[i]) - base);
        tmem_st32(s_col + 32 * k, a);
    }
    wait_st();
    return r;
}

// A key tile of every row of a warp: P into the columns of S, 64 keys at a
// time, each half published on its own barrier, the sums into l.  lim: the
// row's last visible key (masked: some row of the warp does not see all).
// m: the reference (log2 units) of the row's sums, kept while no score passes
// it by kMargin (bf16 and fp32 hold their relative precision there, and no sum
// comes near fp32's range); past that, or with no reference yet, the tile's
// maximum takes its place and l and O are rescaled (`o_used`: O holds
// something; all products into it are complete, as they were issued before
// this S).  A weight is 2^(s kScale - m), one multiply-add a score; m is a
// rounded product, so all weights and sums of a row share a factor of up to
// 2^(half a unit in the last place of m), which would leave fp32's range for
// scores past 2^33.  So a reference beyond kFar is kept as the score itself
// (`far`), and every score of the row is taken relative to it first.  Scores
// are read twice from TMEM, through three buffers of 32: all 128 at once spill
// (three buffers do not for G = 1, 2 and 4; 4 bytes for 8, 32 for the others).
__device__ __forceinline__ void row_tile(float &m, bool &far, uint64_t *l, int lim, bool masked, bool o_used, uint32_t s_col,
                                         uint32_t o_col, uint32_t p_bar, int lane)
{
    const float scale = kScale;
    uint32_t a[32], b[32], c[32];
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int k = 2; k >= 0; k -= 2) {
        tmem_ld32(s_col + 32 * k, a);
        tmem_ld32(s_col + 32 * k + 32, b);
        wait_ld();
        tie32(a);
        tie32(b);
        if (masked) {
            hide(a, lim - 32 * k);
            hide(b, lim - 32 * k - 32);
        }
        row_max(a, mx);
        row_max(b, mx);
    }
    const float raw = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]), top = raw * scale;
    const bool grow = top > m + kMargin;
    if (__any_sync(0xffffffffu, grow || far)) {
        float f = 1.f;
        if (__any_sync(0xffffffffu, far || is_far(raw))) {
            const Reference r = far_reference(Reference{m, 1.f, far}, raw, lim, s_col);
            m = r.m;
            f = r.f;
            far = r.far;
            tmem_ld32(s_col, a);
            tmem_ld32(s_col + 32, b);
            wait_ld();
            tie32(a);
            tie32(b);
        } else if (grow) {
            f = m == -INFINITY ? 0.f : ex2(m - top);
            m = top;
        }
        l[0] = fma2(l[0], pair(f, f), 0ull);
        l[1] = fma2(l[1], pair(f, f), 0ull);
        if (o_used) {
#pragma unroll 1
            for (int k = 0; k < 4; k++) {
                tmem_ld32(o_col + 32 * k, c);
                wait_ld();
                tie32(c);
#pragma unroll
                for (int i = 0; i < 32; i++) c[i] = __float_as_uint(__uint_as_float(c[i]) * f);
                tmem_st32(o_col + 32 * k, c);
            }
        }
    }
    const float neg = far || m == -INFINITY ? 0.f : -m;
    const uint64_t scale2 = pair(scale, scale), ms = pair(neg, neg);
    tmem_ld32(s_col + 64, c);
    weights(a, scale2, ms, l, s_col);
    weights(b, scale2, ms, l, s_col + 16);
    publish(p_bar, lane);
    wait_ld();
    tie32(c);
    if (masked) hide(c, lim - 64);
    tmem_ld32(s_col + 96, a);
    weights(c, scale2, ms, l, s_col + 32);
    wait_ld();
    tie32(a);
    if (masked) hide(a, lim - 96);
    weights(a, scale2, ms, l, s_col + 48);
    publish(p_bar + 8, lane);
}

// One item: tokens [m0, m0 + 2 kTok) of the sequence of n tokens whose rows
// start at row0 (n = 0: no more items).
struct Item {
    int kvh, row0, n, m0;
};

// Key tiles that query tile t (kTok tokens) sees; 0: it has no token.
__device__ __forceinline__ int key_tiles(const Item &it, int t, int kTok)
{
    const int first = it.m0 + t * kTok;
    return first < it.n ? (min(first + kTok, it.n) - 1) / kKeys + 1 : 0;
}

// Rows of sequence b; -1 for a pair of entries that breaks the order or lies
// outside the rows.
__device__ __forceinline__ int seq_rows(const Args &a, int b, int &row0)
{
    const int lo = a.cu[b], hi = a.cu[b + 1];
    row0 = lo;
    return lo < 0 || hi < lo || hi > a.s.T ? -1 : hi - lo;
}

// The place of the k-th set bit of a word (k from 0; there are more than k).
__device__ __forceinline__ int nth_bit(unsigned bits, int k, int lane)
{
    return __ffs((int)__ballot_sync(0xffffffffu, ((bits >> lane) & 1u) && __popc(bits & ((1u << lane) - 1u)) == k)) - 1;
}

// Items by rank.  Sequences whose K and V together fit kGroupBytes form a
// group (a longer one goes alone, as many kv heads at a time as fit), and the
// groups follow one another, so that what the blocks read at a time stays in
// L2.  Within a group the longest rows come first: with c_b = ceil(n_b / M)
// items in sequence b (M tokens each), F(x) = sum_b max(0, c_b - x) items have
// index >= x in their sequence; rank r has the largest index x with F(x) > r,
// in the (r - F(x + 1))-th sequence that has one.  Ranks are asked for in
// rising order, so groups only follow, x only falls and the search for the
// sequence goes on where it was (4096 one-token prompts 2.15 ms -> 0.78 ms).
// The list ends before the first sequence whose entries break the order: those
// before it share no row, so all of their items fit the grid and no sum wraps.
// Run by one warp, rarely and from cold instruction caches, so short code
// counts: a group of up to 32 sequences is kept in the lanes (packed prompts
// 168.5 -> 166 us, one short prompt 8.4 -> 7.9; with 64 or 128 kept, more
// code, 4096 one-token prompts take 11% longer).
template <int M>
struct ItemList {
    const Args &a;
    int lane;
    int base;            // rank of the group's first item
    int b0, b1, h0, h1;  // sequences and kv heads of the group
    int end;             // the list goes up to here: B, or the first sequence whose entries break the order
    int heads;           // kv heads a group of this sequence takes
    int x, fx, above;    // F(x) = fx, F(x + 1) = above
    int last;            // rank asked for last
    int seen_b, seen;    // `seen` sequences before seen_b have an item of index x (a search goes on from there)
    bool kept;           // the group has up to 32 sequences, and lane l the (b0 + l)-th
    int n_kept, row_kept;
    __device__ __forceinline__ ItemList(const Args &args, int ln) : a(args), lane(ln) { start(); }
    __device__ __forceinline__ void start()
    {
        last = base = b0 = b1 = x = fx = above = seen_b = seen = 0;
        kept = false;
        h0 = h1 = heads = a.s.Hkv;
        end = a.s.B;
    }
    __device__ __forceinline__ int items(int b) const
    {
        int row0;
        return (seq_rows(a, b, row0) + M - 1) / M;
    }
    // The list ends before sequence b, the first of the group that breaks the order.
    __device__ __forceinline__ void cut(int b) { end = b1 = b; }
    __device__ __forceinline__ int F(int y) const
    {
        int f = 0;
        if (kept)
            f = max((n_kept + M - 1) / M - y, 0);
        else
            for (int b = b0 + lane; b < b1; b += 32) f += max(items(b) - y, 0);
        return __reduce_add_sync(0xffffffffu, f);
    }
    __device__ __forceinline__ bool next_group()
    {
        base += fx * (h1 - h0);  // x = 0 here: fx is all of the last group
        if (h1 < a.s.Hkv) {
            h0 = h1;
            h1 = min(h0 + heads, a.s.Hkv);
        } else {
            if (b1 >= end) return false;
            b0 = b1;
            const long long most = kGroupBytes / (2 * 2 * kHeadDim * (long long)a.s.Hkv);  // tokens
            long long sum = 0;
            if (a.s.T <= most) b1 = end;  // all of them
            for (bool open = true; open && b1 < end;) {
                int row0;
                const int n = b1 + lane < end ? max(seq_rows(a, b1 + lane, row0), 0) : 0;
                long long pre = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, pre, o);
                    if (lane >= o) pre += y;
                }
                const unsigned over = __ballot_sync(0xffffffffu, sum + pre > most);
                const int fit = over ? __ffs((int)over) - 1 : 32;
                if (fit > 0) sum += __shfl_sync(0xffffffffu, pre, fit - 1);
                b1 = min(b1 + fit, end);
                open = fit == 32;
            }
            heads = a.s.Hkv;
            if (b1 == b0) {  // one that does not fit
                int row0;
                const int n = seq_rows(a, b1++, row0);
                heads = max((int)(kGroupBytes / (2 * 2 * kHeadDim) / n), 1);
            }
            h0 = 0;
            h1 = min(heads, a.s.Hkv);
        }
        int most = 0;
        kept = b1 - b0 <= 32;
        if (kept) {
            n_kept = row_kept = 0;
            if (b0 + lane < b1) n_kept = seq_rows(a, b0 + lane, row_kept);
            const unsigned bad = __ballot_sync(0xffffffffu, n_kept < 0);
            if (bad) {
                cut(b0 + __ffs((int)bad) - 1);
                if (b0 + lane >= b1) n_kept = 0;
            }
            most = (n_kept + M - 1) / M;
        } else {
            for (int stop = -1; stop != b1;) {  // a second time without those that do not count
                if (stop >= 0) cut(stop);
                stop = b1;
                most = 0;
                for (int b = b0 + lane; b < b1; b += 32) {
                    int row0;
                    const int n = seq_rows(a, b, row0);
                    if (n < 0) stop = min(stop, b);
                    most = max(most, (n + M - 1) / M);
                }
                stop = __reduce_min_sync(0xffffffffu, stop);
            }
        }
        x = __reduce_max_sync(0xffffffffu, most);
        fx = above = 0;
        return true;
    }
    __device__ __forceinline__ bool get(int r, Item &it)
    {
        if (r < last) start();  // (blocks are handed out in rising order)
        last = r;
        int k;
        for (;;) {
            const int nh = max(h1 - h0, 1);
            k = (r - base) / nh;
            it.kvh = h0 + (r - base) % nh;
            while (fx <= k && x > 0) {
                x--;
                above = fx;
                fx = F(x);
                seen_b = b0;
                seen = 0;
            }
            if (fx > k) break;
            if (!next_group()) return false;
        }
        k -= above;
        if (kept) {
            const int l = nth_bit(__ballot_sync(0xffffffffu, (n_kept + M - 1) / M > x), k, lane);
            it.n = __shfl_sync(0xffffffffu, n_kept, l);
            it.row0 = __shfl_sync(0xffffffffu, row_kept, l);
            it.m0 = x * M;
            return true;
        }
        for (; seen_b < b1; seen_b += 32) {
            int row0 = 0, n = 0;
            if (seen_b + lane < b1) n = seq_rows(a, seen_b + lane, row0);
            const unsigned has = __ballot_sync(0xffffffffu, (n + M - 1) / M > x);
            const int here = __popc(has);
            if (k < seen + here) {
                const int l = nth_bit(has, k - seen, lane);
                it.n = __shfl_sync(0xffffffffu, n, l);
                it.row0 = __shfl_sync(0xffffffffu, row0, l);
                it.m0 = x * M;
                return true;
            }
            seen += here;
        }
        return false;
    }
};

// A role's walk over the block's items.
struct ItemWalk {
    Item *items;
    uint32_t bar0;
    int k;
    volatile int *abort_flag;
    int32_t *status;
    // Waits for the next item; false at the end.
    __device__ __forceinline__ bool next(Item &it)
    {
        if (!warp_wait(bar0 + 8u * (B_ITEM + k % kItems), (k / kItems) & 1, abort_flag, status)) return false;
        it = items[k % kItems];
        return it.n > 0;
    }
    // The warp has read all that it needs of the item.
    __device__ __forceinline__ void done(int lane)
    {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar0 + 8u * (B_TAKEN + k % kItems));
        k++;
    }
};

// A running tile number of the ring: slot and parity.
struct Slot {
    int slot = 0;
    uint32_t par = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == kSlots) {
            slot = 0;
            par ^= 1u;
        }
    }
};

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attend_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv, const Args a)
{
    constexpr int kTok = kRows / G;  // tokens of a query tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t bars[kBars];
    __shared__ uint32_t tmem_sh;
    __shared__ __align__(16) uint4 next_sh;
    __shared__ Item items[kItems];
    __shared__ volatile int abort_flag;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t q_smem = smem, ring = smem + 2 * kTileBytes;
    const uint32_t bar0 = smem_u32(&bars[0]);
    auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    auto wwait = [&](int i, uint32_t parity) { return warp_wait(bar(i), parity, &abort_flag, a.status); };

    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < kBars; i++)
            mbar_init(bar(i), i >= B_P && i < B_P + 4 ? 4 : i >= B_TAKEN && i < B_TAKEN + kItems ? kRoles : 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kWarpLoad && lane < 3)  // the descriptors are ready when the first item is
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(lane == 0 ? &mq : lane == 1 ? &mk : &mv)) : "memory");
    // rows of a query tile that no (token, head) fills: the copies never write them
    if (kTok * G < kRows && warp < 8) {
        for (int i = tid; i < 2 * 2 * (kRows - kTok * G) * 8; i += 256) {
            const int piece = i & 7, h = (i >> 3) & 3, r = kTok * G + (i >> 5);
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(q_smem + (uint32_t)(h * kHalfBytes + r * 128 + piece * 16)),
                         "r"(0)
                         : "memory");
        }
        fence_proxy_async_smem();
    }
    grid_dependency_wait();
    if (warp == kWarpItems) {  // after the wait: a kernel before this one may hold TMEM until it ends
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_sh)), "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    fence_before();
    __syncthreads();
    fence_after();
    constexpr uint32_t tmem = 0;  // the base of an allocation of all columns
    ItemWalk walk{items, bar0, 0, &abort_flag, a.status};
    Item it;

    if (warp == kWarpItems) {
        // ----------------------------------------------------------- items ----
        if (blockIdx.x == 0)
            for (int b = lane; b < a.s.B; b += 32) {
                const int lo = a.cu[b], hi = a.cu[b + 1];
                if (lo < 0 || hi < lo || hi > a.s.T) set_status(a.status, MP_ERR_CAPACITY);
            }
        ItemList<2 * kTok> list(a, lane);
        int r = blockIdx.x;  // its own item, then those of blocks that have not started yet
        bool more = true, live = true;
        for (int k = 0; more; k++) {
            if (live && k >= kItems && !wwait(B_TAKEN + k % kItems, (k / kItems - 1) & 1)) break;
            if (k > 0) {
                if (lane == 0) {
                    fence_proxy_async_smem();
                    mbar_expect_tx(bar(B_NEXT), 16);
                    next_block(smem_u32(&next_sh), bar(B_NEXT));
                }
                __syncwarp();
                if (!wwait(B_NEXT, (k - 1) & 1)) {
                    wait_teardown(bar(B_NEXT), (k - 1) & 1);  // the answer lands before the block leaves
                    break;
                }
                more = block_taken(smem_u32(&next_sh), r);
                __syncwarp();
            }
            if (!live) continue;  // past the last item: the blocks that are left have none either
            live = more && list.get(r, it);
            if (!live) it.n = 0;
            if (lane == 0) {
                items[k % kItems] = it;
                mbar_arrive(bar(B_ITEM + k % kItems));
            }
        }
    } else if (warp == kWarpLoad) {
        // -------------------------------------------------------- producer ----
        Slot sl;
        int used = 0;             // tiles issued so far (kSlots and more: wait for the slot)
        int nq[2] = {0, 0};       // items that query tile t took part in
        int n_fix = 0;            // V tiles handed to the warp that zeroes
        bool ok = true;
        auto load_kv = [&](const CUtensorMap *m, int kt, bool fix) {
            const uint32_t landed = bar(fix ? B_FIX + n_fix % kFixes : B_KV + sl.slot);
            n_fix += fix;
            if (used >= kSlots && !wwait(B_FREE + sl.slot, sl.par ^ 1u)) return false;
            if (elect_one()) {
                mbar_expect_tx(landed, kTileBytes);
#pragma unroll
                for (int h = 0; h < 2; h++)
                    tma_3d(ring + sl.slot * kTileBytes + h * kHalfBytes, m, landed, 64 * h, it.kvh, it.row0 + kt * kKeys);
            }
            __syncwarp();
            sl.next();
            used = min(used + 1, kSlots);
            return true;
        };
        while (ok && walk.next(it)) {
            const int nt = max(key_tiles(it, 0, kTok), key_tiles(it, 1, kTok));
            const int first = key_tiles(it, 0, kTok) == nt ? 0 : 1;  // the query tile that needs the first K tile
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const int t = i ^ first;
                if (ok && key_tiles(it, t, kTok) > 0) {
                    ok = nq[t] == 0 || wwait(B_QFREE + t, (nq[t] - 1) & 1);
                    if (ok && elect_one()) {
                        mbar_expect_tx(bar(B_Q + t), 2 * kTok * G * 128);
                        for (int h = 0; h < 2; h++)
                            tma_3d(q_smem + t * kTileBytes + h * kHalfBytes, &mq, bar(B_Q + t), 64 * h, it.kvh * G,
                                   it.row0 + it.m0 + t * kTok);
                    }
                    __syncwarp();
                    if (ok) nq[t]++;
                }
                if (i == 0) ok = ok && load_kv(&mk, nt - 1, false);
            }
            for (int kt = nt - 1; kt >= 0 && ok; kt--)
                ok = load_kv(&mv, kt, (kt + 1) * kKeys > it.n) && (kt == 0 || load_kv(&mk, kt - 1, false));
            walk.done(lane);
        }
        // own copies land before the block leaves
        for (int t = 0; t < 2; t++)
            if (nq[t] > 0) wait_teardown(bar(B_Q + t), (nq[t] - 1) & 1);
        if (n_fix > 0) wait_teardown(bar(B_FIX + (n_fix - 1) % kFixes), ((n_fix - 1) / kFixes) & 1);
        for (int i = 0; i < used; i++) {  // the last `used` tiles, from the latest back
            sl.slot = sl.slot == 0 ? kSlots - 1 : sl.slot - 1;
            if (sl.slot == kSlots - 1) sl.par ^= 1u;
            wait_teardown(bar(B_KV + sl.slot), sl.par);
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------- MMA ----
        // The whole warp walks the loop and one elected lane issues, so that
        // descriptors and addresses stay in uniform registers (a lone lane's
        // have to be moved there before every product: 90 cycles a product
        // against the 64 that it takes).
        const uint64_t q_desc = desc_kmajor(q_smem), k_desc = desc_kmajor(ring), v_desc = desc_mnmajor(ring);
        auto qk = [&](int t, int slot) {
            const uint64_t qd = q_desc + (uint64_t)(t * (kTileBytes >> 4));
            const uint64_t kd = k_desc + (uint64_t)(slot * (kTileBytes >> 4));
#pragma unroll
            for (int ks = 0; ks < 8; ks++) {
                const uint64_t off = (uint64_t)(((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4);
                mma_ss(tmem + kColS + 128 * t, qd + off, kd + off, idesc(false), ks > 0);
            }
        };
        auto pv = [&](int t, int slot, int half, bool accum) {
            const uint64_t vd = v_desc + (uint64_t)(slot * (kTileBytes >> 4));
#pragma unroll
            for (int ks = 4 * half; ks < 4 * half + 4; ks++)
                mma_ts(tmem + kColO + 128 * t, tmem + kColS + 128 * t + 8 * ks, vd + (uint64_t)(ks * (2048 >> 4)),
                       idesc(true), accum || ks > 0);
        };
        const bool leader = elect_one();
        // A wait that only the tensor pipe's pace should hold up: no vote over
        // the warp; after an abort every wait returns at once and the walk over
        // the items ends.
        auto lwait = [&](int i, uint32_t parity) {
            if (!mbar_try_wait(bar(i), parity)) wait_slow(bar(i), parity, &abort_flag, a.status);
        };
        // A step is one key tile of one item.  Each round does the P V products
        // of a step and the Q K^T products of the one after it (of the next
        // item at an item's end), query tile by query tile.
        Slot vsl, ksl;  // V tile of the step, K tile of the next; K and V tiles alternate in the ring
        uint32_t q_par[2] = {0, 0}, p_par[2] = {0, 0};
        int kt = 0, nt[2] = {0, 0};  // the step: key tile, key tiles of the item per query tile (0: not there)
        bool more = walk.next(it);
        int nkt = 0, nnt[2] = {0, 0};  // the next step
        if (more) {
            nnt[0] = key_tiles(it, 0, kTok);
            nnt[1] = key_tiles(it, 1, kTok);
            nkt = max(nnt[0], nnt[1]) - 1;
        }
        bool have = false;
        while (have || more) {
            if (have) lwait(B_KV + vsl.slot, vsl.par);
            if (more) lwait(B_KV + ksl.slot, ksl.par);
#pragma unroll
            for (int t = 0; t < 2; t++) {
                const bool do_pv = kt < nt[t], do_qk = nkt < nnt[t];
                if (do_qk && nkt == nnt[t] - 1) {  // its first key tile
                    lwait(B_Q + t, q_par[t]);
                    q_par[t] ^= 1u;
                }
                if (do_pv) {
                    lwait(B_P + 2 * t, p_par[t]);
                    fence_after();
                    if (leader) pv(t, vsl.slot, 0, kt < nt[t] - 1);
                    __syncwarp();
                    lwait(B_P + 2 * t + 1, p_par[t]);
                    p_par[t] ^= 1u;
                }
                fence_after();
                if (leader) {
                    if (do_pv) {
                        pv(t, vsl.slot, 1, true);
                        if (kt == 0) commit(bar(B_O + t));
                    }
                    if (do_qk) {
                        qk(t, ksl.slot);
                        commit(bar(B_S + t));
                        if (nkt == 0) commit(bar(B_QFREE + t));
                    }
                    if (t == 1) {
                        if (have) commit(bar(B_FREE + vsl.slot));
                        if (more) commit(bar(B_FREE + ksl.slot));
                    }
                }
                __syncwarp();
            }
            // the next step becomes this one
            have = more;
            kt = nkt;
            nt[0] = nnt[0];
            nt[1] = nnt[1];
            vsl = ksl;
            vsl.next();
            ksl = vsl;
            ksl.next();
            if (more && --nkt < 0) {
                walk.done(lane);
                more = walk.next(it);
                nnt[0] = more ? key_tiles(it, 0, kTok) : 0;
                nnt[1] = more ? key_tiles(it, 1, kTok) : 0;
                nkt = max(nnt[0], nnt[1]) - 1;
                if (!more) nkt = 0;
            }
        }
        if (leader) commit(bar(B_END));
        __syncwarp();
        wait_teardown(bar(B_END), 0);
    } else if (warp == kWarpFix) {
        // ----------------------------- zero V behind the end of the sequence ----
        int tile = 0, n_fix = 0;  // running number of the item's first tile in the ring; such items so far
        while (walk.next(it)) {
            const int nt = max(key_tiles(it, 0, kTok), key_tiles(it, 1, kTok));
            if (nt * kKeys > it.n) {
                const int slot = (tile + 1) % kSlots, r0 = it.n - (nt - 1) * kKeys;  // first row behind the end
                if (!wwait(B_FIX + n_fix % kFixes, (n_fix / kFixes) & 1)) break;
                for (int i = lane; i < (kKeys - r0) * 16; i += 32)
                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                                     ring + (uint32_t)(slot * kTileBytes + (i & 1) * kHalfBytes + r0 * 128 + (i >> 1) * 16)),
                                 "r"(0)
                                 : "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_KV + slot));
                n_fix++;
            }
            tile = (tile + 2 * nt) % kSlots;
            walk.done(lane);
        }
    } else {
        // --------------------------------------------------------- softmax ----
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        const uint32_t s_col = tmem + lanes + kColS + 128 * t, o_col = tmem + lanes + kColO + 128 * t;
        uint32_t par = 0, o_par = 0;  // parities of the tile's steps and items
        bool live = walk.next(it);
        while (live) {
            const int nt = key_tiles(it, t, kTok);
            const int limit = min(it.m0 + t * kTok + r / G, it.n - 1);  // last visible key
            const size_t out0 = (size_t)(it.row0 + it.m0 + t * kTok) * a.s.Hq + (size_t)it.kvh * G;  // the tile's first row
            const int rows = min(kTok, it.n - it.m0 - t * kTok) * G;  // rows of the tile that exist
            walk.done(lane);
            if (nt == 0) {
                live = walk.next(it);
                continue;
            }
            float m = -INFINITY;
            bool far = false;
            uint64_t l[2] = {0ull, 0ull};  // four partial sums
            bool ok = true;
            for (int kt = nt - 1; kt >= 0 && ok; kt--, par ^= 1u) {
                ok = wwait(B_S + t, par);
                if (!ok) break;
                fence_after();
                const int lim = limit - kt * kKeys;
                const bool masked = __any_sync(0xffffffffu, lim < kKeys - 1);
                row_tile(m, far, l, lim, masked, kt < nt - 1, s_col, o_col, bar(B_P + 2 * t), lane);
            }
            if (!ok) break;
            live = walk.next(it);  // while the last product runs
            if (!wwait(B_O + t, o_par)) break;
            o_par ^= 1u;
            fence_after();
            float l0, l1;
            unpair(add2(l[0], l[1]), l0, l1);
            const float sum = l0 + l1, inv = sum == 0.f ? 0.f : 1.f / sum;  // 0: every score is -inf
            // 64 dims at a time through the warp's stage, so that a warp's store covers
            // four whole 128-byte lines and not 16 bytes of 32 (packed prompts 200 -> 184 us)
            const uint32_t stage = ring + kSlots * kTileBytes + warp * kStageBytes;
            const int r0 = (warp & 3) * 32 + (lane >> 3);  // the first row that this lane stores
            uint4 *dst = reinterpret_cast<uint4 *>(a.out + (out0 + (4 % G == 0 ? (size_t)(r0 / G) * a.s.Hq + r0 % G : 0)) * kHeadDim) +
                         (lane & 7);
#pragma unroll
            for (int c = 0; c < 2; c++) {
                uint32_t o[64];
                tmem_ld32(o_col + 64 * c, o);
                tmem_ld32(o_col + 64 * c + 32, o + 32);
                wait_ld();
                tie32(o);
                tie32(o + 32);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    uint32_t v[4];
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        v[k] = pack_bf16(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((i ^ (lane & 7)) << 4)),
                                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                                 : "memory");
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int lr = 4 * i + (lane >> 3), rr = (warp & 3) * 32 + lr;  // row of the warp, of the tile
                    uint32_t v[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                                 : "r"(stage + lr * 128 + (((lane & 7) ^ (lr & 7)) << 4))
                                 : "memory");
                    if (rr < rows) {
                        const int at = 4 % G == 0 ? i * (4 / G) * a.s.Hq : (rr / G) * a.s.Hq + rr % G;  // rows of out from dst
                        dst[(long long)at * (kHeadDim / 8) + 8 * c] = make_uint4(v[0], v[1], v[2], v[3]);
                    }
                }
                __syncwarp();
            }
            if (a.lse && r < rows) a.lse[out0 + (size_t)(r / G) * a.s.Hq + r % G] = ((far ? m * kScale : m) + log2f(sum)) * kLn2;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kWarpItems)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_sh), "r"(512));
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
    const long long items = ((long long)s.T / (2 * kTok) + (s.B < s.T ? s.B : s.T)) * s.Hkv;  // sum ceil(n_b / M), at most
    if (items > 0x7fffffffll) return cudaErrorInvalidValue;
    const void *fn = reinterpret_cast<const void *>(prompt_attend_kernel<G>);
    cudaError_t e = ensure_smem(fn, kSmemBytes);
    if (e != cudaSuccess) return e;
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
