// Exact decode attention over a paged key-value cache (mp_paged_attend).
//
// For each unit (sequence b, kv head) and the G query heads of its group:
//   s_ih = q_h . k_i / sqrt(d),  out_h = sum_i e^{s_ih} v_i / sum_i e^{s_ih},
// one pass over the unit's tokens with a running maximum and sum per head.
// The floor is HBM: 512 bytes per (token, kv head), each read once; the
// products are 2 d G multiply-adds on them, far below the tensor rate.  Measured
// with 32 / 8 heads, 16 sequences of 32k to 131k tokens in pages of 16: 775 us
// for 5.46 GB, 7.0 TB/s (a copy runs at 6.55); one sequence of 16k 19 us (floor
// 10: launches, the first loads' latency and the join, whose grid of C - 1 blocks
// a head of the group is 1180 for 32 results and finds no room beside the
// attention's blocks, are the rest); 256 of up to 300 37 us (floor 25), 47 with
// units' ends counted as nothing.
//
// Split: the 64-token blocks of all units, unit after unit, form one line of
// W places (a unit's end takes kEndCost, as it costs about as much), and the C
// thread blocks of the grid (two per SM) take equal runs of it, c W / C to
// (c + 1) W / C.  So every thread block has the same work whatever the lengths
// are, one long sequence is split over all SMs and a batch of short ones hardly
// at all.  A run that covers a whole
// unit writes its result; a unit cut by the ends of runs leaves one partial
// (m, l, acc) per run, at most two per thread block, and merge_partials_kernel
// joins them.
//
// Within a thread block, warp w takes the 16-token tiles 4 j + w of a run,
// each warp on its own: its rows come through its own ring of cp.async copies
// (kStages tiles of 16 K and 16 V rows), S^T = K Q^T and O^T += V^T P^T run on
// mma.sync m16n8k16 (tokens or dims x 8 heads x 16), the softmax state stays
// in registers, and the warps meet only at the end of a unit.  mma.sync and
// not tcgen05: 8 heads fill a 16-row tile of either poorly, and the tensor
// pipe idles here anyway.  P enters its product as three bf16 parts (24 bits):
// the result is fp32, and one bf16 part would be off by up to 2^-8 of a weight.
#include <math.h>

#include "mp_pages.cuh"

namespace mp {
namespace paged {

constexpr int kWarps = 4;
constexpr int kTile = 16;                    // tokens of a warp's tile
constexpr int kBlockTok = kWarps * kTile;    // tokens of a block of the split
constexpr int kStages = 3;
constexpr int kRowBytes = 256;
constexpr int kTileBytes = 2 * kTile * kRowBytes;        // K rows, then V rows
constexpr int kRingBytes = kWarps * kStages * kTileBytes; // 96 KB
constexpr int kAccBytes = 2 * kWarps * 4 * kHeadDim * 4;  // the warps' sums of four heads, where they are joined: two in turn
constexpr int kSmemBytes = kRingBytes + kAccBytes;        // 112 KB: two thread blocks per SM
constexpr int kEndCost = 1;                  // what a unit's end (its queries, the join) costs, in blocks
constexpr int kBlocksPerSm = 2;
constexpr int kMergeWarps = 4, kMergeBatch = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMargin = 8.f;               // log2 units that a maximum may grow before the sums are rescaled

struct Args {
    PagesShape s;
    const uint16_t *q, *kp, *vp;
    const int32_t *table, *lens;
    int max_len, C;
    uint32_t magic;  // floor(2^32 / page_size) + 1, for tokens / page_size
    float *out, *lse;
    float *pml;   // [C][2][8][2]: m, l (log2 units) of the partials
    float *pacc;  // [C][2][8][128]
    int32_t *status;
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// {lo, hi} as two bf16
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ void ldmatrix_x4_s(uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans_s(uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr)
                 : "memory");
}
// Byte offset of 16-byte piece c (0..15) of a 256-byte row in a tile: pieces
// XOR-swizzled by the row within each 128-byte line, so the 8 rows that one
// ldmatrix phase reads hit distinct banks.
__device__ __forceinline__ uint32_t row_off(int r, int c) { return (uint32_t)(r * kRowBytes + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ int clamped_len(const Args &a, int b)
{
    return min(max(a.lens[b], 0), a.max_len);
}
__device__ __forceinline__ int blocks_of(int len) { return (len + kBlockTok - 1) / kBlockTok; }
// Places of a unit on the line: its blocks, then its end.
__device__ __forceinline__ int places_of(int nb) { return nb > 0 ? nb + kEndCost : 0; }

// tok / page_size and the remainder: the product's high word is the quotient
// or one more (tokens are below 2^30).
__device__ __forceinline__ int page_of(const Args &a, int tok, int &off)
{
    int q = a.s.S == 1 ? tok : (int)__umulhi((uint32_t)tok, a.magic);
    off = tok - q * a.s.S;
    if (off < 0) {
        q--;
        off += a.s.S;
    }
    return q;
}

// Inclusive prefix sums over a warp.
__device__ __forceinline__ long long warp_prefix(long long v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

// The line as a warp sees it: lane l has the blocks of sequences l chunk to
// (l + 1) chunk, and of all before.
struct Line {
    int chunk;
    long long own, upto, W;
    __device__ __forceinline__ Line(const Args &a, int lane)
    {
        constexpr int kLens = 2;
        chunk = (a.s.B + 31) / 32;
        long long n = 0;
        for (int i0 = 0; i0 < chunk; i0 += kLens) {
            int v[kLens];  // loads in flight
#pragma unroll
            for (int i = 0; i < kLens; i++) {
                const int b = lane * chunk + i0 + i;
                v[i] = i0 + i < chunk && b < a.s.B ? clamped_len(a, b) : 0;
            }
#pragma unroll
            for (int i = 0; i < kLens; i++) n += places_of(blocks_of(v[i]));
        }
        own = n * a.s.Hkv;
        upto = warp_prefix(own, lane);
        W = __shfl_sync(0xffffffffu, upto, 31);
    }
};

// Runs that the line is cut into: C, or W where that is less (so no run is
// empty).  The run that holds place x is the largest c with c W / C <= x.
__device__ __forceinline__ int live_runs(long long W, int C) { return (int)min(W, (long long)C); }
__device__ __forceinline__ int run_of(long long x, long long W, int C) { return (int)(((x + 1) * C - 1) / W); }

// Adds a partial (m, l, v) of weights relative to 2^m2 to another.
__device__ __forceinline__ void fold(float &m, float &l, float4 &v, float m2, float l2, const float4 &v2)
{
    const float mn = fmaxf(m, m2), f = m == -INFINITY ? 0.f : ex2(m - mn), g = ex2(m2 - mn);
    l = l * f + l2 * g;
    v.x = v.x * f + v2.x * g;
    v.y = v.y * f + v2.y * g;
    v.z = v.z * f + v2.z * g;
    v.w = v.w * f + v2.w * g;
    m = mn;
}

// A walk over a run of the line, block by block: unit after unit, the kv heads
// of a sequence side by side, sequences without tokens passed over.
struct Walk {
    long long left;  // places of the run from here on
    int b, kvh, blk, len, nb;
    __device__ __forceinline__ void next(const Args &a)
    {
        left--;
        if (++blk >= nb) next_unit(a, kEndCost);
    }
    // Past the places that are left of the unit's end.
    __device__ __forceinline__ void next_unit(const Args &a, int end)
    {
        left -= end;
        if (left <= 0) return;
        blk = 0;
        if (++kvh < a.s.Hkv) return;
        kvh = 0;
        do {
            len = clamped_len(a, ++b);
            nb = blocks_of(len);
        } while (nb == 0);
    }
};

// Where place x of the line lies.
__device__ __forceinline__ void locate(const Args &a, const Line &line, long long x, int lane, Walk &w)
{
    const int l = __ffs((int)__ballot_sync(0xffffffffu, line.upto > x)) - 1;  // the lane whose sequences hold it
    long long first = __shfl_sync(0xffffffffu, line.upto - line.own, l);     // the line's position of the step's first sequence
    for (int b0 = l * line.chunk;; b0 += 32) {
        const int bb = b0 + lane;
        const long long n = bb < a.s.B ? (long long)places_of(blocks_of(clamped_len(a, bb))) * a.s.Hkv : 0;
        const long long pre = warp_prefix(n, lane);
        const unsigned over = __ballot_sync(0xffffffffu, first + pre > x);
        if (over) {
            const int k = __ffs((int)over) - 1;
            w.b = b0 + k;
            first += __shfl_sync(0xffffffffu, pre - n, k);
            break;
        }
        first += __shfl_sync(0xffffffffu, pre, 31);
    }
    w.len = clamped_len(a, w.b);
    w.nb = blocks_of(w.len);
    w.kvh = (int)((x - first) / places_of(w.nb));
    w.blk = (int)((x - first) - (long long)w.kvh * places_of(w.nb));  // nb and more: in the unit's end
}

// The K and V pieces of rows I, I + 1, .. (of 8) of a lane: 512 bytes apart in
// the pools, swizzled in the ring (offsets as immediates).
template <int I>
__device__ __forceinline__ void copy_rows(const uint32_t (&d)[4], const uint16_t *k, const uint16_t *v)
{
    if constexpr (I < 8) {
        asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;\n" ::"r"(d[I & 3]), "l"(k), "n"(512 * I) : "memory");
        asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;\n" ::"r"(d[I & 3]), "l"(v),
                     "n"(512 * I + kTile * kRowBytes), "n"(512 * I)
                     : "memory");
        copy_rows<I + 1>(d, k, v);
    }
}

// ALIGNED: pages are whole tiles (page_size % 16 == 0), so a tile lies in one
// page and its table entry is read once, not per row.
template <bool ALIGNED>
__global__ void __launch_bounds__(32 * kWarps, kBlocksPerSm) paged_attend_kernel(const Args a)
{
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ uint32_t seen_sh[kWarps][kStages];  // bit i: token i of the stage's tile counts
    __shared__ float red_sh[2][kWarps][2][8];
    const PagesShape &s = a.s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g4 = lane >> 2, t4 = lane & 3;  // mma fragment row and column group
    const int h0 = 2 * t4, h1 = h0 + 1;       // this lane's heads of the group
    const float scale2 = kLog2e * 0.08838834764831845f;  // log2(e) / sqrt(128)
    grid_dependency_wait();

    // this thread block's run of the line
    const Line line(a, lane);
    const long long W = line.W;
    const int c = blockIdx.x, C = live_runs(W, a.C);
    if (c == 0)
        for (int j = tid; j < s.B; j += blockDim.x)
            if (a.lens[j] > a.max_len || a.lens[j] < 0) set_status(a.status, MP_ERR_CAPACITY);
    for (int j = c; j < s.B; j += gridDim.x)  // sequences without tokens
        if (clamped_len(a, j) == 0) {
            for (int i = tid; i < s.Hq * kHeadDim; i += blockDim.x) a.out[(size_t)j * s.Hq * kHeadDim + i] = 0.f;
            for (int i = tid; i < s.Hq; i += blockDim.x) a.lse[(size_t)j * s.Hq + i] = -INFINITY;
        }
    if (c >= C) return;
    const long long x = c * W / C;
    Walk rd;  // what is read next
    rd.left = (c + 1) * W / C - x;
    locate(a, line, x, lane, rd);
    if (rd.blk >= rd.nb) rd.next_unit(a, rd.nb + kEndCost - rd.blk);
    Walk at = rd;  // what is computed next, kStages - 1 blocks behind

    const uint32_t my_ring = smem_u32(ring) + (uint32_t)(warp * kStages * kTileBytes);
    float *acc_sh = reinterpret_cast<float *>(ring + kRingBytes);  // [2][warp][4 heads][128], columns swizzled by head
    int turn = 0, red = 0;  // which of the two joins are in
    auto acc_at = [&](int w, int h, int d) -> float & {
        return acc_sh[((turn * kWarps + w) * 4 + (h & 3)) * kHeadDim + (d ^ ((h & 2) << 2))];
    };

    // The table entry of the next tile is fetched a tile ahead of its copies:
    // lane i < 16 holds that of token i (ALIGNED: all lanes the tile's one).
    int tok0 = 0, page = -1, off_pg = 0;  // off_pg: the token's row in its page
    bool inside = false;                  // the token is one of the sequence's
    auto fetch = [&]() {
        if (rd.left <= 0) return;
        tok0 = (rd.blk * kWarps + warp) * kTile;
        const int tok = ALIGNED ? tok0 : tok0 + (lane & 15);
        const int col = page_of(a, tok, off_pg);
        inside = tok < rd.len;
        page = inside ? a.table[(size_t)rd.b * s.M + col] : -1;
        if (rd.blk == 0 && lane < 2 * s.G)  // a unit begins: its queries (2 lines a head) into L1
            asm volatile("prefetch.global.L1 [%0];" ::"l"(
                a.q + ((size_t)rd.b * s.Hq + rd.kvh * s.G) * kHeadDim + lane * 64));
    };
    // row 2 i + lane / 16 of a tile goes to its swizzled place: lane_dst[i % 4] + 512 i
    uint32_t lane_dst[4];
#pragma unroll
    for (int i = 0; i < 4; i++) lane_dst[i] = my_ring + row_off(2 * i + (lane >> 4), lane & 15) - 512 * i;
    int slot_rd = 0;
    auto issue = [&]() {
        if (rd.left > 0) {
            const uint32_t dst = my_ring + (uint32_t)(slot_rd * kTileBytes);
            const bool good = page >= 0 && page < s.P;
            if (!good && inside) set_status(a.status, MP_ERR_CAPACITY);
            const int p = lane & 15, r0 = lane >> 4;
            unsigned seen;
            if (ALIGNED) {
                const int n = good ? min(rd.len - tok0, kTile) : 0;  // rows that count
                seen = (1u << max(n, 0)) - 1u;
                const size_t off = good ? (((size_t)page * s.Hkv + rd.kvh) * s.S + off_pg + r0) * kHeadDim + p * 8 : 0;
                const uint16_t *k0 = a.kp + off, *v0 = a.vp + off;
                uint32_t d[4];
#pragma unroll
                for (int i = 0; i < 4; i++) d[i] = lane_dst[i] + slot_rd * kTileBytes;
                if (n == kTile) {
                    copy_rows<0>(d, k0, v0);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const int r = 2 * i + r0, bytes = r < n ? 16 : 0;  // a row that does not count is zeros: 0 times anything else may be NaN
                        const size_t o = r < n ? (size_t)(2 * i) * kHeadDim : 0;
                        cp_async_16_s(d[i & 3] + 512 * i, k0 + o, bytes);
                        cp_async_16_s(d[i & 3] + 512 * i + kTile * kRowBytes, v0 + o, bytes);
                    }
                }
            } else {
                // lanes 0..15: the row of token tok0 + lane in the pools (-1: none)
                const long long row = good ? ((long long)page * s.Hkv + rd.kvh) * s.S + off_pg : -1;
                seen = __ballot_sync(0xffffffffu, row >= 0) & 0xffffu;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const int r = 2 * i + r0;
                    const long long ar = __shfl_sync(0xffffffffu, row, r);
                    const size_t off = (size_t)max(ar, 0ll) * kHeadDim + p * 8;
                    const int bytes = ar >= 0 ? 16 : 0;
                    cp_async_16_s(dst + row_off(r, p), a.kp + off, bytes);
                    cp_async_16_s(dst + kTile * kRowBytes + row_off(r, p), a.vp + off, bytes);
                }
            }
            if (lane == 0) seen_sh[warp][slot_rd] = seen;
            rd.next(a);
            fetch();
        }
        cp_async_commit();
        slot_rd = slot_rd == kStages - 1 ? 0 : slot_rd + 1;
    };
    fetch();
    for (int t = 0; t < kStages - 1; t++) issue();

    // query fragments of a unit: B of m16n8k16 (k = dims, n = heads), zero for heads past G
    // (plain loads: this grid may have started before the queries were written, so they are not constant in it)
    uint32_t qf[8][2];
    auto load_q = [&]() {
        const uint16_t *qr = a.q + ((size_t)at.b * s.Hq + at.kvh * s.G + g4) * kHeadDim + t4 * 2;
#pragma unroll
        for (int ks = 0; ks < 8; ks++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                qf[ks][j] = g4 < s.G ? *reinterpret_cast<const uint32_t *>(qr + ks * 16 + j * 8) : 0u;
    };
    load_q();

    int slot = 0;
    while (at.left > 0) {
        const int hq0 = at.kvh * s.G, b = at.b, nb = at.nb, blk0 = at.blk;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        float o[8][4];
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) o[i][j] = 0.f;
        // the unit's blocks of this run
        const int nt = (int)min((long long)(nb - blk0), at.left);
        for (int t = 0; t < nt; t++) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            const uint32_t kt = my_ring + (uint32_t)(slot * kTileBytes), vt = kt + kTile * kRowBytes;
            const unsigned seen = seen_sh[warp][slot];
            slot = slot == kStages - 1 ? 0 : slot + 1;
            // S^T: 16 tokens x 8 heads
            float sc[2][4] = {};  // two chains of products
#pragma unroll
            for (int ks = 0; ks < 8; ks++) {
                uint32_t r0, r1, r2, r3;
                ldmatrix_x4_s(r0, r1, r2, r3, kt + row_off(lane & 15, 2 * ks + (lane >> 4)));
                float(&d)[4] = sc[ks & 1];
                mma_bf16_16816(d[0], d[1], d[2], d[3], r0, r1, r2, r3, qf[ks][0], qf[ks][1]);
            }
            float c0 = sc[0][0] + sc[1][0], c1 = sc[0][1] + sc[1][1], c2 = sc[0][2] + sc[1][2], c3 = sc[0][3] + sc[1][3];
            const bool s0 = (seen >> g4) & 1u, s1 = (seen >> (g4 + 8)) & 1u;
            c0 = s0 ? c0 * scale2 : -INFINITY;
            c1 = s0 ? c1 * scale2 : -INFINITY;
            c2 = s1 ? c2 * scale2 : -INFINITY;
            c3 = s1 ? c3 * scale2 : -INFINITY;
            const float x0 = fmaxf(c0, c2), x1 = fmaxf(c1, c3);
            if (__any_sync(0xffffffffu, x0 > m0 + kMargin || x1 > m1 + kMargin)) {
                float y0 = x0, y1 = x1;
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) {
                    y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, w));
                    y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, w));
                }
                y0 = fmaxf(y0, m0);
                y1 = fmaxf(y1, m1);
                const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - y0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - y1);
                m0 = y0;
                m1 = y1;
                l0 *= f0;
                l1 *= f1;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    o[i][0] *= f0;
                    o[i][1] *= f1;
                    o[i][2] *= f0;
                    o[i][3] *= f1;
                }
            }
            const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
            float p0 = ex2(c0 - u0), p1 = ex2(c1 - u1), p2 = ex2(c2 - u0), p3 = ex2(c3 - u1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            uint32_t pb[3][2];  // P^T as B fragments (k = tokens, n = heads), three bf16 parts
#pragma unroll
            for (int j = 0; j < 3; j++) {
                const uint32_t a0 = pack_bf16(p0, p1), a1 = pack_bf16(p2, p3);
                p0 -= bf16_lo(a0);
                p1 -= bf16_hi(a0);
                p2 -= bf16_lo(a1);
                p3 -= bf16_hi(a1);
                pb[j][0] = transpose8(a0);
                pb[j][1] = transpose8(a1);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {  // 16 dims each
                uint32_t r0, r1, r2, r3;
                ldmatrix_x4_trans_s(r0, r1, r2, r3, vt + row_off((lane & 7) + ((lane >> 4) << 3), 2 * i + ((lane >> 3) & 1)));
                // the tile's own sum, then one rounded add: the tensor core cuts low bits off, not
                // rounds, and over the thousands of tiles of a long run that adds up (2.5e-5
                // relative where all tiles went into one accumulator)
                float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
#pragma unroll
                for (int j = 2; j >= 0; j--) mma_bf16_16816(d0, d1, d2, d3, r0, r1, r2, r3, pb[j][0], pb[j][1]);
                o[i][0] += d0;
                o[i][1] += d1;
                o[i][2] += d2;
                o[i][3] += d3;
            }
            __syncwarp();  // every lane has read the tile before its slot is refilled
            issue();
            at.next(a);
        }
        if (at.left > 0) load_q();  // of the next unit, under the join
        // ---- the warps' states, joined in shared memory (copies of what follows are in flight) ----
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, w);
            l1 += __shfl_xor_sync(0xffffffffu, l1, w);
        }
        // (two buffers in turn: whoever writes one again has met, in the join between, all that read it)
        float(&red_ml)[kWarps][2][8] = red_sh[red];
        red ^= 1;
        if (g4 == 0) {
            red_ml[warp][0][h0] = m0;
            red_ml[warp][0][h1] = m1;
            red_ml[warp][1][h0] = l0;
            red_ml[warp][1][h1] = l1;
        }
        const bool whole = blk0 == 0 && nt == nb;
        const int part = c * 2 + (blk0 == 0 ? 1 : 0);
        for (int q = 0; q < s.G; q += 4) {  // four heads at a time
            if (h0 >> 2 == q >> 2) {
                float *lo = &acc_at(warp, h0, g4), *hi = &acc_at(warp, h0, g4 + 8);  // h1: the next row, alike
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    lo[i * 16] = o[i][0];
                    lo[i * 16 + kHeadDim] = o[i][1];
                    hi[i * 16] = o[i][2];
                    hi[i * 16 + kHeadDim] = o[i][3];
                }
            }
            __syncthreads();
            const int h = q + warp;  // a warp a head, a lane four dims
            if (h < s.G) {
                float mw[kWarps], l = 0.f;
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; w++) mw[w] = red_ml[w][0][h];
                const float m = fmaxf(fmaxf(mw[0], mw[1]), fmaxf(mw[2], mw[3]));
#pragma unroll
                for (int w = 0; w < kWarps; w++) {
                    if (red_ml[w][1][h] == 0.f) continue;  // no token (a sum that is NaN goes on)
                    const float f = ex2(mw[w] - m);
                    const float4 x = *reinterpret_cast<const float4 *>(&acc_at(w, h, 4 * lane));
                    l = fmaf(f, red_ml[w][1][h], l);
                    v.x = fmaf(f, x.x, v.x);
                    v.y = fmaf(f, x.y, v.y);
                    v.z = fmaf(f, x.z, v.z);
                    v.w = fmaf(f, x.w, v.w);
                }
                if (whole) {
                    const size_t bh = (size_t)b * s.Hq + hq0 + h;
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    reinterpret_cast<float4 *>(a.out + bh * kHeadDim)[lane] = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
                    if (lane == 0) a.lse[bh] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
                } else {
                    const size_t e = (size_t)part * 8 + h;
                    reinterpret_cast<float4 *>(a.pacc + e * kHeadDim)[lane] = v;
                    if (lane == 0) reinterpret_cast<float2 *>(a.pml)[e] = make_float2(m, l);
                }
            }
            turn ^= 1;
        }
    }
    cp_async_wait<0>();
}

// Joins the partials of the units that several runs share.  Block (c, head of
// the group): the unit that run c ends, if it began in a run before.  Its warps
// take the runs in turn (lane = 4 dims), kMergeBatch loads in flight each, then
// meet in shared memory.
__global__ void __launch_bounds__(32 * kMergeWarps) merge_partials_kernel(const Args a)
{
    __shared__ float red_m[kMergeWarps], red_l[kMergeWarps];
    __shared__ float4 red_v[kMergeWarps][32];
    const PagesShape &s = a.s;
    const int c1 = blockIdx.x + 1, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the lengths are older than this kernel's predecessor: read before the wait
    const Line line(a, lane);
    const long long W = line.W;
    const int C = live_runs(W, a.C);
    int c0 = 0;
    Walk u;
    bool mine = false;
    if (c1 < C) {
        const long long x = c1 * W / C;
        locate(a, line, x, lane, u);
        mine = u.blk > 0 && u.blk < u.nb && x - u.blk + u.nb <= (c1 + 1) * W / C;
        c0 = run_of(x - u.blk, W, C);
    }
    grid_dependency_wait();
    if (!mine) return;
    float m = -INFINITY, l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int cb = c0 + warp; cb <= c1; cb += kMergeWarps * kMergeBatch) {
        float2 ml[kMergeBatch];
        float4 acc[kMergeBatch];
#pragma unroll
        for (int i = 0; i < kMergeBatch; i++) {
            const int c = cb + kMergeWarps * i;
            ml[i] = make_float2(-INFINITY, 0.f);
            if (c <= c1) {
                const size_t e = (size_t)(c * 2 + (c == c0 ? 1 : 0)) * 8 + h;
                ml[i] = reinterpret_cast<const float2 *>(a.pml)[e];
                acc[i] = reinterpret_cast<const float4 *>(a.pacc + e * kHeadDim)[lane];
            }
        }
#pragma unroll
        for (int i = 0; i < kMergeBatch; i++)
            if (ml[i].y != 0.f) fold(m, l, v, ml[i].x, ml[i].y, acc[i]);
    }
    red_v[warp][lane] = v;
    if (lane == 0) {
        red_m[warp] = m;
        red_l[warp] = l;
    }
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < kMergeWarps; w++)
        if (red_l[w] != 0.f) fold(m, l, v, red_m[w], red_l[w], red_v[w][lane]);
    const size_t bh = (size_t)u.b * s.Hq + u.kvh * s.G + h;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    reinterpret_cast<float4 *>(a.out + bh * kHeadDim)[lane] = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    if (lane == 0) a.lse[bh] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Runs of the split for sequences up to max_len: two per SM, fewer where the
// longest possible line has fewer blocks.
static int num_runs(const PagesShape &s, int max_len)
{
    static const int kMaxRuns = 148 * kBlocksPerSm;
    const long long line = (long long)s.B * s.Hkv * ((max_len + kBlockTok - 1) / kBlockTok);
    return (int)(line < kMaxRuns ? line : kMaxRuns);
}

}  // namespace paged

size_t paged_workspace_bytes(const PagesShape &s, int max_len)
{
    return (size_t)paged::num_runs(s, max_len) * 2 * 8 * (kHeadDim + 2) * sizeof(float);
}

cudaError_t launch_paged_attend(const PagesShape &s, const uint16_t *q, const uint16_t *kp, const uint16_t *vp,
                                const int32_t *table, const int32_t *lens, int max_len, float *out, float *lse,
                                void *workspace, int32_t *status, cudaStream_t st)
{
    paged::Args a;
    a.s = s;
    a.q = q;
    a.kp = kp;
    a.vp = vp;
    a.table = table;
    a.lens = lens;
    a.max_len = max_len;
    a.magic = (uint32_t)((1ull << 32) / (uint64_t)s.S) + 1u;
    a.C = paged::num_runs(s, max_len);
    a.out = out;
    a.lse = lse;
    a.pacc = static_cast<float *>(workspace);
    a.pml = a.pacc + (size_t)a.C * 2 * 8 * kHeadDim;
    a.status = status;
    auto kernel = s.S % paged::kTile == 0 ? paged::paged_attend_kernel<true> : paged::paged_attend_kernel<false>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(kernel), paged::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(a.C > 0 ? a.C : 1), dim3(32 * paged::kWarps), paged::kSmemBytes, st, a);
    if (e != cudaSuccess || a.C < 2) return e;  // one run: no unit is cut
    return launch_pdl(paged::merge_partials_kernel, dim3(a.C - 1, s.G), dim3(32 * paged::kMergeWarps), 0, st, a);
}

}  // namespace mp
