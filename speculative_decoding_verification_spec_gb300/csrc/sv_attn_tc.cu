// sv_attn_tc.cu -- verify_attention for many rows, on the tensor cores (tcgen05).
//
// The arithmetic is that of sv_attn.cu: u_j = log2(e) s_j + e_j, weights 2^(u_j - m) against a lazily moved reference m,
// o = sum p' c / sum p' 2^(-e).  Tokens lie on the 128 lanes of an accumulator and the rows of q, up to 128 of one
// key/value head, are its columns, so a tile costs what its rows cost, without padding to 128:
//   S^T [128 tokens, rows] = K [128, D] Q^T:   the codes of K go from memory to the product as they are (e4m3 x e4m3);
//       a row of q, scaled by a power of two to a largest element in [128, 256), is split into e4m3 terms that sum to it,
//       two for bf16 (4 bits each, the residual's sign the ninth: exact for elements above 2^-10 of the largest, off by at
//       most 2^-17 of it below) and three for halfs (exact above 2^-6, and the same below), whose products accumulate.
//   O^T [D, rows] += V^T [D, 128] P^T:   halfs; six warps widen the codes of V into shared memory, and the weights are
//       rounded to halfs (half a step, 2^-11: under a bf16 output's own rounding, as much as an fp16 output's; a weight below
//       2^-14 is off by 2^-25 absolute, 2^-32 of the row's largest, as HEAD says).  The product needs 16-bit operands, and a
//       bf16 weight would be off by 2^-9.
// The round's own rows come last, as tiles of their own: keys and values as halfs scaled by a power of two per token, and a
// copy of q as halfs.
//
// One CTA per SM works through an equal run of all groups' tiles (as in sv_attn.cu), with a role per warp:
//   0      copies: the keys' codes by TMA into a ring of stages, the pages' numbers and scales beside them; the values' codes
//          it only calls into L2 by then
//   1      products: one lane issues them; S is double-buffered, so S of the next tile runs under this tile's softmax
//   2 - 7  values: the next tile's codes from L2 into registers while this tile's are widened into shared memory
//   8 - 15 softmax, two groups of four warps; a thread is a token, a group takes half of the columns.  The sums l stay in
//          tensor memory beside S^T and O^T, one per token lane and column, so a thread holds 16 columns at a time.  The
//          weights are taken against the reference as it stands; only when one passes 2^15.9 (the first tile of a group, and
//          rarely after) does the group find the columns' maxima, move the reference, rescale its part of O^T and l and
//          repeat the tile.
// What bounds it: neither memory nor the tensor cores, but the chain that each tile goes through (S^T, softmax, P, O^T): some
// 2000 to 2800 cycles up to 48 rows and 3600 at 87, of which a product takes about 100 whatever its columns, and some 12000
// to 20000 more where a CTA changes the group (q, the first reference, the round's own rows, the outputs).  The issue slots are
// 44% used, DRAM 25%.  B = 32, contexts to 8192, T = 6, four query heads a head: 132 us for 347 MB (2.6 TB/s); to 4096, T = 65
// (three row tiles of 87): 382 us for 89 GFLOP (233 TFLOP/s).  A third softmax group (spills), S^T fetched a chunk ahead, and
// both terms of q stacked into one product of twice the columns were slower: 202, 142 and 147 us where this took 139.
// Every wait on an mbarrier is bounded; when one runs out the CTA's remaining groups report SPEC_ROW_TIMEOUT.  Between named
// barriers the threads of a softmax group never part: what a wait returned is agreed on before anyone acts on it.
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "sv_attn.cuh"

namespace sv {

namespace {

constexpr int TT = 128;          // tokens of a tile
constexpr int VW0 = 2, VWN = 6;  // warps that widen the values
constexpr int SMW0 = 8, NG = 2;  // first softmax warp (a multiple of 4), groups of four softmax warps
constexpr int TNT = (SMW0 + 4 * NG) * 32;
constexpr int MAXR = 128;        // rows of a group: S^T twice, O^T and the sums l take four times as many columns
constexpr int MAXC = (MAXR / 16 + NG - 1) / NG * 16;  // columns of a softmax group
constexpr int MAXSTAGES = 6;
constexpr float WINDOW = 15.9f;  // a weight may reach 2^WINDOW (the largest half is just under 2^16)
constexpr float HEAD = 7.0f;     // a moved reference leaves the maximum at 2^HEAD, so a weight 2^-32 of the largest is the least that a
                                 // half still holds, as on the few-rows path.  More room above means fewer repeated tiles: with 3
                                 // (and 2^-28) B = 32, T = 6, T = 65 and eight query heads a head took 134, 362 and 169 us, with 7
                                 // 137, 384 and 186; but with 3 a row whose weight lies nearly all on one token has the others'
                                 // weights off by up to 2%, with 7 by 0.13% at 32768 of them
constexpr float LATE = 7.0f;     // where a move is due, columns past 2^LATE move with it: later repeats are fewer (B = 32, T = 65:
                                 // 384 us, 417 with 11; T = 6, eight query heads a head: 186 and 209).  Under WINDOW by more than the
                                 // two passes' roundings differ, so that a weight past it does move
constexpr float HOLD = 14.0f;    // where a weight is put that no reference brings under the window
constexpr size_t TC_SMEM = 214 * 1024;  // dynamic shared memory; the static arrays take the rest of the SM's 227 KB

struct TcParams {
    AttnParams A;
    int MR, RN;          // rows of a row tile; padded to a multiple of 16
    int stages, np, nv;  // ring stages; buffers of P and of the widened values (1 or 2)
    uint32_t o_p, o_v, o_kh, o_stage, v_buf, p_buf;  // offsets in dynamic shared memory, sizes
    bool qvec, kvec, vvec;  // rows that allow wide loads: 16 bytes of q, D / 32 elements of the others
    int wait_limit;
    uint64_t inv_g;      // r / G = r * inv_g >> 32 for the rows of a head: a division costs a role hundreds of cycles
};

// ---------------------------------------------------------------- tcgen05

// A shared-memory operand's descriptor in two words.  Low: the address and the stride between 64-channel blocks (operands
// with M or N contiguous); high: the stride between groups of eight rows, the descriptor version of this architecture
// (bit 46) and the swizzle (bits 61-63).
constexpr uint32_t SW128 = 2, SW64 = 4;
__host__ __device__ constexpr uint32_t desc_hi(uint32_t swizzle, uint32_t sbo) { return sbo >> 4 | 1u << 14 | swizzle << 29; }
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4 & 0x3fffu) | lbo >> 4 << 16; }

// instruction descriptor: fp32 accumulator, M = 128, N, both operands of format 0 (e4m3 / half); `mn`: both with their M / N
// dimension contiguous
__device__ __forceinline__ uint32_t idesc(int N, bool mn)
{
    return 1u << 4 | (mn ? 1u << 15 | 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | (128u >> 4) << 24;
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a, uint32_t ah, uint32_t b, uint32_t bh, uint32_t id, bool acc)
{
    asm volatile("{ .reg .pred p; .reg .b64 x, y; mov.b64 x, {%1, %2}; mov.b64 y, {%3, %4}; setp.ne.u32 p, %6, 0;"
                 " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %5, p; }"
                 :: "r"(d), "r"(a), "r"(ah), "r"(b), "r"(bh), "r"(id), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void mma_h(uint32_t d, uint32_t a, uint32_t ah, uint32_t b, uint32_t bh, uint32_t id, bool acc)
{
    asm volatile("{ .reg .pred p; .reg .b64 x, y; mov.b64 x, {%1, %2}; mov.b64 y, {%3, %4}; setp.ne.u32 p, %6, 0;"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %5, p; }"
                 :: "r"(d), "r"(a), "r"(ah), "r"(b), "r"(bh), "r"(id), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ bool elected()
{
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// 16 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
}
// one column
__device__ __forceinline__ void tmem_ld1(uint32_t addr, uint32_t& r)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1]; tcgen05.wait::ld.sync.aligned;" : "=r"(r) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st16_nowait(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                    "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ unsigned long long f2_mul(unsigned long long a, unsigned long long b)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// a box of one page's codes of one head
__device__ __forceinline__ void tma_page(uint32_t dst, const CUtensorMap* map, int block, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(map), "r"(0), "r"(0), "r"(block), "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" :: "r"(smem_addr(bar)), "r"(bytes) : "memory");
}

// ---------------------------------------------------------------- shared state

struct Shared {
    uint64_t full[MAXSTAGES], empty[MAXSTAGES];
    uint64_t info[MAXSTAGES];     // the stage's pages and scales are there
    uint64_t sfull[2], ready[2], pv[2], own[2], qfull, done;
    float2 scale[MAXSTAGES][8];   // of the stage's pages: keys, values
    int status[MAXSTAGES], page[MAXSTAGES][8];
    float4 fr[2][MAXR / 2];       // per pair of columns: factors, references negated; two copies, one being rewritten
    float wred[NG][4][MAXC];      // column maxima and sums of the softmax warps
    float4 col[NG][MAXC];         // a moved reference's factors; the outputs' columns
    float unseen[NG][MAXC];       // 1: no token of the group so far was seen by the column
    uint32_t mask[MAXR][4];       // round's rows: which tokens of the tile a column sees
    float fks[2][TT], fve[2][TT]; // round's rows: scale of the keys and exponent of the values, per token
    int vbad[4][VWN];               // round's rows: a tile's values hold a NaN or an infinity, per warp
    int fail;
    int lost[NG][2];              // requests that a softmax group left without outputs: first and one past the last
    uint32_t tmem;
    Place place;
};

// Bounded wait; ends early once another role has given up.  Out of line, as the path that is seldom taken; the rest is inline,
// since what a call takes by reference lives in local memory, and beside this much shared memory hardly any L1 is left for it.
__device__ __noinline__ bool wait_on(Shared& sh, uint64_t* bar, uint32_t parity, int limit)
{
    const uint32_t a = smem_addr(bar);
#pragma unroll 1
    for (int n = 0; n < limit; ++n) {
        uint32_t done;
        // suspended for up to 2 us a poll: a spinning warp would take its scheduler's slots from the working ones
        asm volatile("{ .reg .pred q; mbarrier.try_wait.parity.shared::cta.b64 q, [%1], %2, 2000; selp.u32 %0, 1, 0, q; }"
                     : "=r"(done) : "r"(a), "r"(parity) : "memory");
        if (done) return true;
        if ((n & 63) == 63 && *reinterpret_cast<volatile int*>(&sh.fail)) return false;
    }
    *reinterpret_cast<volatile int*>(&sh.fail) = 1;
    return false;
}
__device__ __forceinline__ bool wait_warp(Shared& sh, uint64_t* bar, uint32_t parity, int limit)
{
    return __all_sync(0xffffffffu, (limit > 0 && mbar_wait(bar, parity, 1)) || wait_on(sh, bar, parity, limit));
}

__device__ __forceinline__ void group_sync(int id) { asm volatile("barrier.cta.sync %0, 128;" :: "r"(id) : "memory"); }
// barrier of a softmax group that also tells whether any thread's x is set
__device__ __forceinline__ bool group_any(int id, bool x)
{
    uint32_t r;
    asm volatile("{ .reg .pred p, q; setp.ne.u32 p, %2, 0; barrier.cta.red.or.pred q, %1, 128, p; selp.u32 %0, 1, 0, q; }"
                 : "=r"(r) : "r"(id), "r"((uint32_t)x) : "memory");
    return r != 0;
}

// ---------------------------------------------------------------- the groups of a CTA

struct Walk {
    long long u, u1, pre;
    int b, RT;
    ReqInfo rq;
    // the current group
    int h, rt, tile0, tile1;
    bool whole;

    __device__ __forceinline__ Walk(const AttnParams& P, const Place& at)
    {
        u = at.total * blockIdx.x / at.ctas;
        u1 = at.total * (blockIdx.x + 1) / at.ctas;
        pre = at.pre;
        b = at.b;
        RT = P.RT;
        rq = req_info<TT>(P, b);
    }
    // the group at u, or the next one where u lies past a group's tiles; false where the run has ended
    __device__ __forceinline__ bool open(const AttnParams& P)
    {
        while (u < u1) {
            while (u >= pre + (long long)rq.span * P.Hkv * RT) {
                pre += (long long)rq.span * P.Hkv * RT;
                rq = req_info<TT>(P, ++b);
            }
            const long long rem = u - pre;
            const int grp = (int)(rem / rq.span);
            tile0 = (int)(rem % rq.span);
            if (tile0 < rq.n) {
                h = grp / RT;
                rt = grp % RT;
                tile1 = (int)min((long long)rq.n, tile0 + (u1 - u));
                whole = tile0 == 0 && tile1 == rq.n;
                return true;
            }
            u += rq.span - tile0;
        }
        return false;
    }
    __device__ __forceinline__ void next() { u += tile1 - tile0; }
};

// ---------------------------------------------------------------- roles

template <int D>
__device__ void role_copy(const TcParams& T, Shared& sh, const Place& at, uint32_t ring, const CUtensorMap* mk, const CUtensorMap* mv)
{
    const AttnParams& P = T.A;
    const int lane = threadIdx.x & 31;
    const int ppt = TT >> P.page_shift;    // pages of a tile
    const int per = 32 >> (7 - P.page_shift);  // tiles whose pages the warp's lanes hold at once
    const int my_tile = lane >> (7 - P.page_shift), my_page = lane & (ppt - 1);
    constexpr uint32_t KB = TT * D;
    int it = 0, s = 0, par = 1;  // tiles so far, the next stage and the parity of its last use's end
    bool ok = true;
    for (Walk w(P, at); ok && w.open(P); w.next()) {
        const int32_t* table = P.page_table + (size_t)w.b * P.table_width;
        const int c0 = min(w.tile0, w.rq.ncache), c1 = min(w.tile1, w.rq.ncache), len = w.rq.len;
        // Lane k holds page k of a batch of `per` tiles with its scales.  Two batches ahead the page numbers are loaded, one
        // ahead the scales, so that neither is waited for in the loop.
        const auto live_at = [&](int tile) { return tile + my_tile < c1 && (long long)tile * TT + (long long)lane * P.page < len; };
        const auto page_of = [&](int tile) { return live_at(tile) ? __ldg(table + (((long long)tile * TT + (long long)lane * P.page) >> P.page_shift)) : -1; };
        const auto block_of = [&](int page) { return (unsigned)page < (unsigned)P.pages ? (size_t)page * P.Hkv + w.h : 0; };
        int page = -1, page1 = page_of(c0), page2 = page_of(c0 + per);
        float ks = 1.0f, vs = 1.0f, ks1 = __ldg(P.ks + block_of(page1)), vs1 = __ldg(P.vs + block_of(page1));
        for (int tile = w.tile0; tile < w.tile1; ++tile, ++it) {
            // (a stage's first use asks for the phase before the first, which counts as over)
            if (!wait_warp(sh, &sh.empty[s], par, T.wait_limit)) {
                ok = false;
                break;
            }
            if (tile < c1) {
                const int k = (tile - c0) & (per - 1);
                if (k == 0) {
                    page = page1;
                    ks = ks1;
                    vs = vs1;
                    page1 = page2;
                    ks1 = __ldg(P.ks + block_of(page1));
                    vs1 = __ldg(P.vs + block_of(page1));
                    page2 = page_of(tile + 2 * per);
                }
                const bool mine = my_tile == k && live_at(tile - k);
                const bool good = mine && (unsigned)page < (unsigned)P.pages;
                const unsigned use = __ballot_sync(0xffffffffu, good), want = __ballot_sync(0xffffffffu, mine);
                if (lane == 0) {
                    mbar_expect(&sh.full[s], (uint32_t)__popc(use) * (uint32_t)(P.page * D));
                    sh.status[s] = use != want ? ROW_BAD_PAGE : ROW_OK;
                }
                __syncwarp();
                if (mine) {
                    sh.scale[s][my_page] = make_float2(ks, vs);
                    sh.page[s][my_page] = good ? page : -1;
                }
                if (good) {
                    tma_page(ring + s * KB + my_page * P.page * D, mk, page * P.Hkv + w.h, &sh.full[s]);
                    // the values go from L2 to the registers of the warps that widen them, some tiles later
                    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
                                 :: "l"(mv), "r"(0), "r"(0), "r"(page * P.Hkv + w.h) : "memory");
                }
            } else if (lane == 0) {
                sh.status[s] = ROW_OK;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.info[s]);
                mbar_arrive(&sh.full[s]);
            }
            if (++s == T.stages) s = 0, par ^= 1;
        }
    }
    // no copy may be in flight when the CTA ends: the last fill of every stage
    if (lane == 0)
        for (int j = max(0, it - T.stages); j < it; ++j) (void)mbar_wait(&sh.full[j % T.stages], (j / T.stages) & 1, MBAR_SPIN_LIMIT);
    __syncwarp();
}

// Products of tile `it`: S^T as soon as its keys are there; O^T of the tile before after that, except where the next S^T
// needs what the softmax does only after that O^T (a group's first tile, the round's rows).  S^T may be rewritten once the
// weights of the tile before last are ready, which its O^T has waited for.  The whole warp walks through, so that the
// operands are uniform registers; one elected lane issues.
template <int DT, int D>
__device__ void role_mma(const TcParams& T, Shared& sh, const Place& at, uint32_t base, uint32_t tmem)
{
    const AttnParams& P = T.A;
    constexpr int TERMS = DT == DT_BF16 ? 2 : 3;
    constexpr uint32_t KB = TT * D;
    const uint32_t sp = base + T.o_p, sv_ = base + T.o_v, ring = base + T.o_stage;
    const uint32_t qterm = (uint32_t)T.RN * D;
    constexpr uint32_t H_K = D == 128 ? desc_hi(SW128, 1024) : desc_hi(SW64, 512), H_128 = desc_hi(SW128, 1024);
    const uint32_t id_s = idesc(T.RN, false), id_o = idesc(T.RN, true);
    const uint32_t t_o = tmem + 2 * T.RN;
    const auto uni = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    int it = 0, stage = 0, stage_par = 0, seg = 0;
    uint32_t own = 0;                                        // phases of the two barriers of the rounds' rows
    int pending = 0, pending_first = 0, ok = 1;              // pending: O^T of the tile before is still to be issued
    int have = 0;                                            // the next tile's codes have been waited for

    const auto pv = [&]() {  // O^T of the tile before
        const int i = it - 1;
        pending = 0;
        if (!uni(wait_warp(sh, &sh.ready[i & 1], (i >> 1) & 1, T.wait_limit))) return 0;
        tc_fence_after();
        const int vi = T.nv == 2 ? i & 1 : 0, pi = T.np == 2 ? i & 1 : 0;
        // the second block of 64 channels: the next 16 KB, or (D = 64) the block of zeros after the buffers
        const uint32_t lbo = D == 128 ? 16384 : (T.nv - vi) * T.v_buf;
        const uint32_t a = desc_lo(sv_ + vi * T.v_buf, lbo), b = desc_lo(sp + pi * T.p_buf, 16384);
        if (elected()) {
#pragma unroll 2
            for (int k = 0; k < TT / 16; ++k)
                mma_h(t_o, a + k * (2048 >> 4), H_128, b + k * (2048 >> 4), H_128, id_o, !pending_first || k > 0);
            mma_commit(&sh.pv[i & 1]);
        }
        __syncwarp();
        return 1;
    };

    for (Walk w(P, at); ok && w.open(P); w.next(), ++seg) {
        const int tile0 = uni(w.tile0), tile1 = uni(w.tile1), ncache = uni(w.rq.ncache);
        for (int tile = tile0; tile < tile1; ++tile) {
            const bool fresh = tile >= ncache, first = tile == tile0;
            // O^T of the tile before goes in front of S^T or after it: step 0 or 2, so that its code is here once
#pragma unroll 1
            for (int step = pending && (first || fresh) ? 0 : 1; ok && step < 3; ++step) {
            if (step != 1) {
                if (pending) ok = pv();
                continue;
            }
            if (!have) ok = ok && uni(wait_warp(sh, &sh.full[stage], stage_par, T.wait_limit));
            if (first) ok = ok && uni(wait_warp(sh, &sh.qfull, seg & 1, T.wait_limit));
            if (fresh) {
                ok = ok && uni(wait_warp(sh, &sh.own[it & 1], own >> (it & 1) & 1, T.wait_limit));
                own ^= 1u << (it & 1);
            }
            if (!ok) continue;
            tc_fence_after();
            const uint32_t ts = tmem + (it & 1) * T.RN, kb = ring + stage * KB;
            if (!fresh) {
                const uint32_t a = desc_lo(kb, 16), b = desc_lo(base, 16);
                if (elected()) {
#pragma unroll 1
                    for (int q = 0; q < TERMS; ++q)
#pragma unroll 2
                        for (int k = 0; k < D / 32; ++k)
                            mma_f8(ts, a + k * 2, H_K, b + q * (qterm >> 4) + k * 2, H_K, id_s, q + k > 0);
                    mma_commit(&sh.sfull[it & 1]);
                    mma_commit(&sh.empty[stage]);
                }
            } else {
                const uint32_t a = desc_lo(base + T.o_kh, 16), b = desc_lo(sp + (T.np == 2 ? it & 1 : 0) * T.p_buf, 16);
                if (elected()) {
#pragma unroll 2
                    for (int k = 0; k < D / 16; ++k)
                        mma_h(ts, a + (k >> 2) * (16384 >> 4) + (k & 3) * 2, H_128, b + (k >> 2) * (T.RN * 128 >> 4) + (k & 3) * 2, H_128,
                              id_s, k > 0);
                    mma_commit(&sh.sfull[it & 1]);
                    mma_commit(&sh.empty[stage]);
                }
            }
            __syncwarp();
            // the next tile's codes, while the weights are still being computed
            if (++stage == T.stages) stage = 0, stage_par ^= 1;
            have = tile + 1 < tile1;
            if (have) ok = uni(wait_warp(sh, &sh.full[stage], stage_par, T.wait_limit));
            }
            if (!ok) break;
            pending = 1;
            pending_first = first;
            ++it;
        }
    }
    if (ok && pending) (void)pv();
    // everything issued has ended before the accumulators are given back
    if (elected()) mma_commit(&sh.done);
    __syncwarp();
    (void)mbar_wait(&sh.done, 0, MBAR_SPIN_LIMIT);
}

// byte offset of channel d of a row of q in a term's tile (swizzled over 128 or 64 bytes, a row)
template <int D>
__device__ __forceinline__ uint32_t q_off(int col, int d)
{
    return D == 128 ? col * 128 + (((d >> 4) ^ (col & 7)) << 4) + (d & 15) : col * 64 + (((d >> 4) ^ ((col >> 1) & 3)) << 4) + (d & 15);
}

// byte offset of channels d .. (within 8) of a token in a [token][64 channels] block of halfs, 128-byte swizzle
__device__ __forceinline__ uint32_t half_off(int token, int d)
{
    return (uint32_t)(d >> 6) * 16384u + token * 128u + ((((d & 63) >> 3) ^ (token & 7)) << 4) + (d & 7) * 2;
}

// EPL consecutive elements, in one load where `vec` says that every row allows it
template <int DT, int EPL>
__device__ __forceinline__ void load_run(const void* p, int64_t i, bool vec, float (&x)[EPL])
{
    uint32_t u[EPL / 2];
    if (vec) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + i;
        if constexpr (EPL == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(q));
            u[0] = v.x;
            u[1] = v.y;
        } else {
            u[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
        }
#pragma unroll
        for (int k = 0; k < EPL / 2; ++k) {
            if constexpr (DT == DT_BF16) {
                x[2 * k] = bf16lo(u[k]);
                x[2 * k + 1] = bf16hi(u[k]);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
                x[2 * k] = f.x;
                x[2 * k + 1] = f.y;
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < EPL; ++k) x[k] = load_elem<DT>(p, i + k);
    }
}

// A thread's share of a tile's values: 16 codes each of up to VPT (token, channel) places.
constexpr int VTHREADS = VWN * 32;
template <int D>
struct Codes {
    static constexpr int CH = D / 16, N = (TT * CH + VTHREADS - 1) / VTHREADS;
    uint4 x[N];
};

// Loads them; tokens from `valid` on, and those of a page that is none, are zeros.
template <int D>
__device__ __forceinline__ void load_codes(Codes<D>& c, const AttnParams& P, const int* pages, int h, int ct, int valid)
{
    constexpr int CH = D / 16;
#pragma unroll
    for (int q = 0; q < Codes<D>::N; ++q) {
        const int i = ct + q * VTHREADS, tok = i / CH;
        c.x[q] = make_uint4(0, 0, 0, 0);
        if (i < TT * CH && tok < valid) {
            const int page = pages[tok >> P.page_shift];
            if (page >= 0)
                c.x[q] = ld_stream_v4(P.vc + ((((size_t)page * P.Hkv + h) << P.page_shift) + (tok & (P.page - 1))) * D + (i % CH) * 16);
        }
    }
}

template <int D>
__device__ __forceinline__ void store_halfs(const Codes<D>& c, uint8_t* vb, int ct)
{
    constexpr int CH = D / 16;
#pragma unroll
    for (int q = 0; q < Codes<D>::N; ++q) {
        const int i = ct + q * VTHREADS, tok = i / CH, ch = i % CH;
        if (i >= TT * CH) break;
        const uint32_t u[4] = {c.x[q].x, c.x[q].y, c.x[q].z, c.x[q].w};
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            y[2 * k] = e4m3x2_to_half2((uint16_t)u[k]);
            y[2 * k + 1] = e4m3x2_to_half2((uint16_t)(u[k] >> 16));
        }
        const uint4 lo = make_uint4(y[0], y[1], y[2], y[3]), hi = make_uint4(y[4], y[5], y[6], y[7]);
        // the two blocks of 64 channels start with opposite halves, so a quarter-warp's stores meet no bank twice
        const int f = ch >> 2;
        *reinterpret_cast<uint4*>(vb + half_off(tok, ch * 16 + 8 * f)) = f ? hi : lo;
        *reinterpret_cast<uint4*>(vb + half_off(tok, ch * 16 + 8 * (f ^ 1))) = f ? lo : hi;
    }
}

// The round's rows of one tile: keys into the stage, values into the buffer, as halfs scaled by a power of two per token.  True
// when a value is not finite.
template <int DT, int D>
__device__ __forceinline__ bool own_rows(const TcParams& T, Shared& sh, uint8_t* kb, uint8_t* vb, int it, int b, int h, int j0, int rows)
{
    const AttnParams& P = T.A;
    constexpr int EPL = D / 32;
    const int ct = threadIdx.x - VW0 * 32, wv = ct >> 5, lane = ct & 31;
    const int live = P.kn ? min(max(rows - j0, 0), TT) : 0;
#pragma unroll 1
    for (int i = ct; i < TT * (D / 8); i += VWN * 32)  // tokens that are none: zero values
        if (i / (D / 8) >= live) *reinterpret_cast<uint4*>(vb + half_off(i / (D / 8), i % (D / 8) * 8)) = make_uint4(0, 0, 0, 0);
    if (ct < TT && ct >= live) sh.fks[it & 1][ct] = 1.0f, sh.fve[it & 1][ct] = 0.0f;
    bool vbad = false;
#pragma unroll 1
    for (int i = wv; i < live; i += VWN) {
        const int64_t j = j0 + i;
        float x[2][EPL];
        load_run<DT, EPL>(P.kn, b * P.kb + j * P.kt + h * P.kh + lane * EPL, T.kvec, x[0]);
        load_run<DT, EPL>(P.vn, b * P.vb + j * P.vt + h * P.vh + lane * EPL, T.vvec, x[1]);
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float amax = 0.0f;
            bool fin = true;
#pragma unroll
            for (int k = 0; k < EPL; ++k) {
                if (fabsf(x[which][k]) < __int_as_float(0x7f800000)) amax = fmaxf(amax, fabsf(x[which][k]));
                else fin = false, x[which][k] = 0.0f;
            }
            fin = __all_sync(0xffffffffu, fin);
            amax = redux_max(amax);
            const int e = min(max(exponent_of(amax), CACHE_E_MIN), 126) - 14;
            const float mul = exp2_int(-e);
            uint8_t* to = (which ? vb : kb) + half_off(i, lane * EPL);
            if constexpr (EPL == 4)
                *reinterpret_cast<uint2*>(to) = make_uint2(pack_half2(x[which][0] * mul, x[which][1] * mul),
                                                           pack_half2(x[which][2] * mul, x[which][3] * mul));
            else
                *reinterpret_cast<uint32_t*>(to) = pack_half2(x[which][0] * mul, x[which][1] * mul);
            if (which) vbad = vbad || !fin;
            if (lane == 0) {
                if (which) sh.fve[it & 1][i] = (float)e;
                else sh.fks[it & 1][i] = fin ? exp2_int(e) : __int_as_float(0x7fc00000);  // a key that is not finite: NaN
            }
        }
    }
    return vbad;
}

// The next tile's codes are loaded into registers before this tile's are widened.
template <int DT, int D>
__device__ void role_values(const TcParams& T, Shared& sh, const Place& at, uint8_t* smem)
{
    const AttnParams& P = T.A;
    const int ct = threadIdx.x - VW0 * 32, wv = ct >> 5, lane = ct & 31;
    int it = 0, s = 0, par = 0;  // s, par: stage and phase of the tile after the loaded one
    bool ok = true;
    for (Walk w(P, at); ok && w.open(P); w.next()) {
        Codes<D> c;
        const auto fetch = [&](int tile) {
            ok = ok && wait_warp(sh, &sh.info[s], par, T.wait_limit);
            if (ok && tile < w.rq.ncache) load_codes<D>(c, P, sh.page[s], w.h, ct, w.rq.len - tile * TT);
        };
        fetch(w.tile0);
#pragma unroll 1
        for (int tile = w.tile0; ok && tile < w.tile1; ++tile, ++it) {
            uint8_t* vb = smem + T.o_v + (T.nv == 2 ? it & 1 : 0) * T.v_buf;
            const bool own = tile >= w.rq.ncache;
            Codes<D> now = c;
            // the stage may be filled again once its pages are read: this is the codes' own end of it
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(&sh.empty[s]);
            if (++s == T.stages) s = 0, par ^= 1;
            if (tile + 1 < w.tile1) fetch(tile + 1);
            // the buffer's last use (the first ones ask for a phase before the first, which counts as over)
            ok = ok && wait_warp(sh, &sh.pv[(it + T.nv) & 1], ((it - T.nv) >> 1) & 1, T.wait_limit);
            // the keys of a round's rows have one buffer: S^T of the tile before has to be done with it.  (S^T two tiles on, whose
            // commit ends the next phase, follows the O^T that waits for this tile's values.)
            if (own) ok = ok && wait_warp(sh, &sh.sfull[(it + 1) & 1], ((it - 1) >> 1) & 1, T.wait_limit);
            if (!ok) break;
            if (own) {
                const bool vbad = own_rows<DT, D>(T, sh, smem + T.o_kh, vb, it, w.b, w.h, (tile - w.rq.ncache) * TT, w.rq.rows);
                if (lane == 0) sh.vbad[it & 3][wv] = vbad;
            } else {
                store_halfs<D>(now, vb, ct);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (own) mbar_arrive(&sh.own[it & 1]);
                mbar_arrive(&sh.ready[it & 1]);
            }
        }
    }
}

// The sum of the values of channel d that are not finite over the rows that row t sees: products with a weight of zero would
// carry them to every row, so they are kept out of the product and added to the rows that see them.
template <int DT>
__device__ __noinline__ float unfinite_values(const AttnParams& P, int b, int h, int t, int d)
{
    float add = 0.0f;
#pragma unroll 1
    for (int cur = t;;) {
        const float y = load_elem<DT>(P.vn, b * P.vb + cur * P.vt + h * P.vh + d);
        if (!(fabsf(y) < __int_as_float(0x7f800000))) add += y;
        if (cur == 0) break;
        const int p = P.parents ? __ldg(P.parents + (size_t)b * (P.T - 1) + cur - 1) : cur - 2;
        if (p < -1 || p >= cur - 1) break;
        cur = p + 1;
    }
    return add;
}

__device__ __forceinline__ int row_token(const TcParams& T, int r) { return (int)((uint64_t)(uint32_t)r * T.inv_g >> 32); }

// What a thread of a softmax group keeps for the kernel's life.
struct Lane {
    uint8_t* smem;
    uint32_t tl;            // this warp's lanes of tensor memory
    int g, quad, lane, tok; // group, warp of the group, lane; this thread's token of a tile and channel of O^T
    int bar_id, col0, nch;  // the group's barrier, first column and 16-column chunks
};

// What softmax_run stopped at.
struct RunEnd {
    int n;              // tiles done
    int status;
    uint32_t left_out;  // of the tile it stopped at: the 16-column chunks whose sums this warp has not taken: those past the window
    bool stopped, fail;
};

// Scale of the keys and scale exponent of the values of this thread's token, and the columns that see it (bit c: column c
// of the group).
__device__ __forceinline__ void token_terms(const Shared& sh, const Lane& L, int it, int s_at, int page_shift, int left, bool own, uint64_t see_own,
                                            float& ks, float& ve, uint64_t& see)
{
    ks = 1.0f;
    ve = 0.0f;
    if (own) {
        ks = sh.fks[it & 1][L.tok];
        ve = sh.fve[it & 1][L.tok];
        see = see_own;
    } else {
        see = 0;
        if (L.tok < left) {
            const float2 sc = sh.scale[s_at][L.tok >> page_shift];
            ks = sc.x;
            ve = (float)exponent_of(sc.y);
            see = ~0ull;
        }
    }
}

// The softmax over tiles that have a reference: tiles of the cache in a row, or (own) one of the round's rows.  One pass per
// tile; the run ends where a weight passes the window (for any thread of the group) or a wait runs out.  `take`: chunks whose
// sums the first tile adds to l.  The difference to the reference comes before the exponent of the values: near the maximum it is
// exact, however large the scores.  Nearly all of the kernel's time goes through this loop.
__device__ __forceinline__ RunEnd softmax_run(const TcParams& T, Shared& sh, const Lane L, const float4* fr, int it, int s_at, int tile, int end, int len,
                                           bool own, uint64_t see_own, uint32_t take)
{
    const int RN = T.RN, np = T.np, limit = T.wait_limit, stages = T.stages, page_shift = T.A.page_shift;
    const uint32_t p_buf = T.p_buf, t_l = L.tl + 3 * RN + L.col0;
    uint8_t* const prow = L.smem + T.o_p + L.tok * 128;
    RunEnd r = {0, ROW_OK, 0u, false, false};
#pragma unroll 1
    for (; tile < end; ++tile, ++it, ++r.n) {
        bool fail = !wait_warp(sh, &sh.sfull[it & 1], (it >> 1) & 1, limit);
        // Where P has one buffer, its last use; of two, S^T's commit stands for the use before last, which it followed.  (The
        // kernel's first tile finds it free, and asks for a phase before the first, which counts as over.)
        if (np == 1) fail = fail || !wait_warp(sh, &sh.pv[(it + 1) & 1], ((it - 1) >> 1) & 1, limit);
        float vmax = NEG_INF;
        r.left_out = 0;
        if (!fail) {
            tc_fence_after();
            float ks, ve;
            uint64_t see;
            token_terms(sh, L, it, s_at, page_shift, len - tile * TT, own, see_own, ks, ve, see);
            r.status = max(r.status, own ? 0 : sh.status[s_at]);
            if (++s_at == stages) s_at = 0;
            const bool some = __any_sync(0xffffffffu, see != ~0ull);
            const float inv = exp2_int(min(max(-(int)ve, -126), 127));
            const unsigned long long ks2 = f2_pack(ks, ks), ve2 = f2_pack(ve, ve), inv2 = f2_pack(inv, inv);
            const uint32_t ts = L.tl + (it & 1) * RN + L.col0;
            uint8_t* row = prow + (np == 2 ? it & 1 : 0) * p_buf;
#pragma unroll 1
            for (int ch = 0; ch < L.nch; ++ch) {
                uint32_t s[16], l[16], h[8];
                uint4 f[8];
                tmem_ld16_nowait(ts + ch * 16, s);
                // all eight in flight at once, beside the scores
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = lds128(reinterpret_cast<const uint4*>(&fr[ch * 8 + j]));
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const unsigned long long x = f2_mul(f2_pack(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])),
                                                        f2_pack(__uint_as_float(f[j].x), __uint_as_float(f[j].y)));
                    float a, b;
                    f2_unpack(f2_add(f2_fma(x, ks2, f2_pack(__uint_as_float(f[j].z), __uint_as_float(f[j].w))), ve2), a, b);
                    s[2 * j] = __float_as_uint(a);
                    s[2 * j + 1] = __float_as_uint(b);
                }
                tmem_ld16_nowait(t_l + ch * 16, l);
                if (some) {
                    const uint32_t m = (uint32_t)(see >> (16 * ch));
#pragma unroll
                    for (int j = 0; j < 16; ++j) s[j] = m >> j & 1u ? s[j] : __float_as_uint(NEG_INF);
                }
                float t8[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) t8[j] = fmaxf(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
                const float top = fmaxf(fmaxf(fmaxf(t8[0], t8[1]), fmaxf(t8[2], t8[3])), fmaxf(fmaxf(t8[4], t8[5]), fmaxf(t8[6], t8[7])));
                vmax = fmaxf(vmax, top);
                const bool far = __any_sync(0xffffffffu, top > WINDOW);
                if (far) r.left_out |= take & 1u << ch;
#pragma unroll
                for (int j = 0; j < 16; ++j) s[j] = __float_as_uint(ex2(__uint_as_float(s[j])));
#pragma unroll
                for (int j = 0; j < 8; ++j) h[j] = pack_half2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
                const int col = L.col0 + ch * 16, unit = (col & 63) >> 3;
                uint8_t* to = row + (size_t)(col >> 6) * 16384;
                *reinterpret_cast<uint4*>(to + ((unit ^ (L.tok & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(to + (((unit + 1) ^ (L.tok & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
                tmem_wait_ld();
                if (!far && (take >> ch & 1u)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float c, d;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), inv2,
                                         f2_pack(__uint_as_float(l[2 * j]), __uint_as_float(l[2 * j + 1]))), c, d);
                        l[2 * j] = __float_as_uint(c);
                        l[2 * j + 1] = __float_as_uint(d);
                    }
                    tmem_st16_nowait(t_l + ch * 16, l);
                }
            }
            take = ~0u;
            fence_proxy_async_smem();
            tmem_wait_st();
        }
        if (group_any(L.bar_id, fail || vmax > WINDOW)) {
            r.stopped = true;
            r.fail = fail;
            return r;
        }
        tc_fence_before();
        __syncwarp();
        if (L.lane == 0) {
            mbar_arrive(&sh.ready[it & 1]);
            mbar_arrive(&sh.empty[s_at == 0 ? stages - 1 : s_at - 1]);
        }
    }
    return r;
}

// A tile whose weights pass the window even against the reference that was set for it: its scores are replaced by their differences
// to the reference over the scale of the keys (softmax_run then takes factors of one and no reference, and computes what it did),
// and those past the window put under it.
__device__ __noinline__ void hold_scores(const float4* fr, uint32_t t_s, int cw, float ks, float ve)
{
#pragma unroll 1
    for (int c = 0; c < cw; c += 16) {
        uint32_t s[16];
        tmem_ld16_nowait(t_s + c, s);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float* f = reinterpret_cast<const float*>(&fr[(c + j) >> 1]);
            float d = __fmaf_rn(__fmul_rn(__uint_as_float(s[j]), f[j & 1]), ks, f[2 + (j & 1)]);
            if (__fadd_rn(d, ve) > WINDOW) d = HOLD - ve;
            s[j] = __float_as_uint(d / ks);
        }
        tmem_st16_nowait(t_s + c, s);
    }
    tmem_wait_st();
}

// The reference of the columns that tile `it` takes past the window (or that have none): at 2^HEAD under the maximum, rounded down,
// so that no rounding takes the maximum's own weight under 2^HEAD.  (From |u| = 2^27 on neighbouring floats are 16 and more apart,
// so the weight may still come out above the window; scores that near are equal to within their own rounding.)  The sums so far
// follow.  `hold`: that has happened, and the tile's weights are held at the window, by scores and factors (in the other copy) of
// their own.  False when a wait ran out.  All of the group calls it.
__device__ __forceinline__ bool move_reference(const TcParams& T, Shared& sh, const Lane L, int rb, int it, int s_at, int left, bool own, uint64_t see_own, bool first, bool hold)
{
    const float4* fr = &sh.fr[rb][L.col0 / 2];
    float4* to = &sh.fr[rb ^ 1][L.col0 / 2];
    const uint32_t t_s = L.tl + (it & 1) * T.RN + L.col0, t_o = L.tl + 2 * T.RN + L.col0, t_l = t_o + T.RN;
    const int cw = L.nch * 16;
    const bool ok = wait_warp(sh, &sh.sfull[it & 1], (it >> 1) & 1, T.wait_limit) &&
                    // O^T of the tile before has to be whole before it is rescaled
                    (first || wait_warp(sh, &sh.pv[(it + 1) & 1], ((it - 1) >> 1) & 1, T.wait_limit));
    if (ok) {
        tc_fence_after();
        float ks, ve;
        uint64_t see;
        token_terms(sh, L, it, s_at, T.A.page_shift, left, own, see_own, ks, ve, see);
        if (hold) hold_scores(fr, t_s, cw, ks, ve);
#pragma unroll 1
        for (int c = hold ? cw : 0; c < cw; c += 16) {
            uint32_t s[16];
            tmem_ld16_nowait(t_s + c, s);
            tmem_wait_ld();
            float mine = NEG_INF;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float* f = reinterpret_cast<const float*>(&fr[(c + j) >> 1]);
                const float d = __fadd_rd(__fmaf_rd(__uint_as_float(s[j]) * f[j & 1], ks, first ? 0.0f : f[2 + (j & 1)]), ve);
                const float x = see >> (c + j) & 1ull ? d : NEG_INF;
                const float m = redux_max(x);
                if (L.lane == j) mine = m;
            }
            if (L.lane < 16) sh.wred[L.g][L.quad][c + L.lane] = mine;
        }
    }
    if (group_any(L.bar_id, !ok)) return false;
    if (hold) {
        if (L.tok < cw / 2) to[L.tok] = make_float4(1.0f, 1.0f, 0.0f, 0.0f);
        group_sync(L.bar_id);
        return true;
    }
    if (L.tok < cw) {
        const float(*w)[MAXC] = sh.wred[L.g];
        const float top = fmaxf(fmaxf(w[0][L.tok], w[1][L.tok]), fmaxf(w[2][L.tok], w[3][L.tok]));
        // a column that has seen nothing yet keeps the reference 0, which its zero sums do not feel
        const float* f = reinterpret_cast<const float*>(&fr[L.tok >> 1]);
        float* n = reinterpret_cast<float*>(&to[L.tok >> 1]);
        const float was = first ? 0.0f : -f[2 + (L.tok & 1)];
        const bool none = first || sh.unseen[L.g][L.tok] != 0.0f;
        const bool move = none ? top > NEG_INF : top > LATE;
        const float now = move ? __fadd_rd(was, __fadd_rd(top, -HEAD)) : was;
        n[L.tok & 1] = f[L.tok & 1];
        n[2 + (L.tok & 1)] = -now;
        sh.col[L.g][L.tok].x = first ? 0.0f : move && !none ? ex2(was - now) : 1.0f;  // of the sums so far
        sh.unseen[L.g][L.tok] = none && !move ? 1.0f : 0.0f;
    }
    group_sync(L.bar_id);
    // a group's first tile: l starts from zero, and O^T's first product overwrites it
#pragma unroll 1
    for (int c = first ? cw : 0; c < 2 * cw; c += 16) {
        const uint32_t a = c < cw ? t_o + c : t_l + c - cw;
        const float4* f = &sh.col[L.g][c < cw ? c : c - cw];
        uint32_t o[16];
        if (!first) {
            tmem_ld16_nowait(a, o);
            tmem_wait_ld();
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] = first ? 0u : __float_as_uint(__uint_as_float(o[j]) * f[j].x);
        tmem_st16_nowait(a, o);
    }
    tmem_wait_st();
    return true;
}

// The rows of q as e4m3 terms, and the columns' factors.  A thread takes 16 channels, so a warp four rows (eight of 64 channels).
template <int DT, int D>
__device__ __forceinline__ void load_q(const TcParams& T, Shared& sh, const Lane L, int b, int h, int rt, int rows)
{
    const AttnParams& P = T.A;
    constexpr int TERMS = DT == DT_BF16 ? 2 : 3, LPR = D / 16, RPW = 32 / LPR;  // lanes of a row, rows of a warp
    const int cw = L.nch * 16, d = (L.lane % LPR) * 16;
    const auto load = [&](int c, uint32_t (&u)[8]) {
        const int col = L.col0 + c, r = rt * T.MR + col, t = row_token(T, r);
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = 0u;
        if (c < cw && col < T.MR && r < P.R && t < rows) {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(P.q) + (int64_t)b * P.qb + (int64_t)t * P.qt + (int64_t)(h * P.G + r - t * P.G) * P.qh + d;
            if (T.qvec) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(q)), z = __ldg(reinterpret_cast<const uint4*>(q) + 1);
                u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
                u[4] = z.x; u[5] = z.y; u[6] = z.z; u[7] = z.w;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) u[k] = (uint32_t)__ldg(q + 2 * k) | (uint32_t)__ldg(q + 2 * k + 1) << 16;
            }
        }
    };
    // the next rows are on their way while these are split
    const int c0 = L.quad * RPW + L.lane / LPR;
    uint32_t u[8], next[8];
    load(c0, next);
#pragma unroll 1
    for (int c = c0; c < cw; c += 4 * RPW) {
        const int col = L.col0 + c;
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = next[k];
        load(c + 4 * RPW, next);
        float x[16], amax = 0.0f;
        bool fin = true;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if constexpr (DT == DT_BF16) {
                x[2 * k] = bf16lo(u[k]);
                x[2 * k + 1] = bf16hi(u[k]);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
                x[2 * k] = f.x;
                x[2 * k + 1] = f.y;
            }
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            fin = fin && fabsf(x[k]) < __int_as_float(0x7f800000);
            amax = fmaxf(amax, fabsf(x[k]));
        }
        // (cw is a multiple of 16 and the rows of a warp divide it, so all lanes of a row are here)
        const unsigned row_lanes = (LPR == 8 ? 0xffu : 0xfu) << (L.lane / LPR * LPR);
#pragma unroll
        for (int o = LPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(row_lanes, amax, o));
        fin = __all_sync(row_lanes, fin);
        const int e = fin ? min(max(7 - exponent_of(amax), -120), 126) : 0;
        const float mul = exp2_int(e);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = fin ? x[k] * mul : 0.0f;
        uint8_t* to = L.smem + q_off<D>(col, d);
#pragma unroll
        for (int q = 0; q < TERMS; ++q, to += (size_t)T.RN * D) {
            uint32_t code[4];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint16_t c2;  // magnitudes stay under 448
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c2) : "f"(x[2 * k + 1]), "f"(x[2 * k]));
                const uint32_t h2 = e4m3x2_to_half2(c2);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                x[2 * k] -= f.x;
                x[2 * k + 1] -= f.y;
                code[k >> 1] = k & 1 ? code[k >> 1] | (uint32_t)c2 << 16 : c2;
            }
            *reinterpret_cast<uint4*>(to) = make_uint4(code[0], code[1], code[2], code[3]);
        }
        // a row of q with a NaN or an infinity has no scores
        if (L.lane % LPR < 2)
            reinterpret_cast<float*>(&sh.fr[L.lane % LPR][col >> 1])[c & 1] = fin ? P.scale * LOG2E * exp2_int(-e) : __int_as_float(0x7fc00000);
    }
    fence_proxy_async_smem();
    group_sync(L.bar_id);
    if (L.lane == 0) mbar_arrive(&sh.qfull);
}

// Before a tile of the round's rows: q as halfs (the terms' sums) where P will be, and which columns see this thread's token.
// Returns whether a wait ran out; *bad: whether a parent is out of range.
template <int DT, int D>
__device__ __forceinline__ bool own_tile(const TcParams& T, Shared& sh, const Lane L, int it, int b, int rt, int rows, int j0, uint64_t* see, bool* bad)
{
    const AttnParams& P = T.A;
    constexpr int TERMS = DT == DT_BF16 ? 2 : 3;
    const int cw = L.nch * 16;
    uint8_t* pb = L.smem + T.o_p + (T.np == 2 ? it & 1 : 0) * T.p_buf;
    bool badp = false;
    if (j0 > 0) group_sync(L.bar_id);  // the masks of the tile before have been read (another group's before its outputs)
    if (L.tok < cw) {
        // a thread per column: the rows on its row's path, as bits of the tile's 128 tokens
        const int t = row_token(T, rt * T.MR + L.col0 + L.tok);
        uint32_t* m = sh.mask[L.col0 + L.tok];
        m[0] = m[1] = m[2] = m[3] = 0u;
        if (P.kn && t < rows) {
#pragma unroll 1
            for (int cur = t;;) {
                if ((unsigned)(cur - j0) < (unsigned)TT) m[(cur - j0) >> 5] |= 1u << ((cur - j0) & 31);
                if (cur == 0) break;
                const int p = P.parents ? __ldg(P.parents + (size_t)b * (P.T - 1) + cur - 1) : cur - 2;
                if (p < -1 || p >= cur - 1) break;  // reported below; the walk always ends
                cur = p + 1;
            }
        }
    }
    if (P.parents)
#pragma unroll 1
        for (int i = L.tok; i < rows - 1; i += 128) {
            const int p = __ldg(P.parents + (size_t)b * (P.T - 1) + i);
            badp = badp || p < -1 || p >= i;
        }
    // (the kernel's first tile asks for a phase before the first, which counts as over)
    const bool ok = wait_warp(sh, &sh.pv[(it + 1) & 1], ((it - 1) >> 1) & 1, T.wait_limit);
    if (ok) {
#pragma unroll 1
        for (int i = L.tok; i < cw * (D / 8); i += 128) {
            const int col = L.col0 + i / (D / 8), d = i % (D / 8) * 8;
            alignas(16) __half2 x[4];
#pragma unroll
            for (int q = 0; q < TERMS; ++q) {
                const uint2 code = *reinterpret_cast<const uint2*>(L.smem + (size_t)q * T.RN * D + q_off<D>(col, d));
                const uint32_t u[4] = {e4m3x2_to_half2((uint16_t)code.x), e4m3x2_to_half2((uint16_t)(code.x >> 16)),
                                       e4m3x2_to_half2((uint16_t)code.y), e4m3x2_to_half2((uint16_t)(code.y >> 16))};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __half2 y = *reinterpret_cast<const __half2*>(&u[k]);
                    x[k] = q ? __hadd2(x[k], y) : y;
                }
            }
            *reinterpret_cast<uint4*>(pb + (size_t)(d >> 6) * T.RN * 128 + col * 128 + ((((d & 63) >> 3) ^ (col & 7)) << 4)) =
                *reinterpret_cast<const uint4*>(x);
        }
        fence_proxy_async_smem();
    }
    *bad = group_any(L.bar_id, badp);
    uint64_t v = 0;
#pragma unroll 4
    for (int c = 0; c < cw; ++c) v |= (uint64_t)(sh.mask[L.col0 + c][L.quad] >> L.lane & 1u) << c;
    *see = v;
    if (ok && L.lane == 0) mbar_arrive(&sh.own[it & 1]);
    return !ok;
}

// A group's outputs: o = O^T / l and lse, or the part for attn_merge_kernel.
template <int DT, int D>
__device__ __forceinline__ void put_outputs(const TcParams& T, Shared& sh, const Lane L, int rb, int b, int h, int rt, int rows, bool whole, float* part,
                                         int status, bool dead, bool vbad)
{
    const AttnParams& P = T.A;
    const int cw = L.nch * 16;
    const uint32_t t_o = L.tl + 2 * T.RN + L.col0, t_l = t_o + T.RN;
    if (!dead) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < cw; c += 16) {
            uint32_t l[16];
            float v[16];
            tmem_ld16_nowait(t_l + c, l);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(l[j]);
            // the sums of 16 columns over the warp's lanes: half of the columns travel at each step
#pragma unroll
            for (int n = 8, bit = 16; n; n >>= 1, bit >>= 1) {
                const bool up = L.lane & bit;
#pragma unroll
                for (int k = 0; k < n; ++k) {
                    const float send = up ? v[k] : v[k + n], keep = up ? v[k + n] : v[k];
                    v[k] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
                }
            }
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
            if (!(L.lane & 1)) sh.wred[L.g][L.quad][c + (L.lane >> 1)] = v[0];
        }
    }
    group_sync(L.bar_id);
    if (L.tok < cw) {
        // a column's row of the output (-1: none), and the factor of its sums
        const int col = L.col0 + L.tok, r = rt * T.MR + col, t = row_token(T, r), row = t * P.Hq + h * P.G + r - t * P.G;
        const float(*w)[MAXC] = sh.wred[L.g];
        const float l = dead ? 0.0f : (w[0][L.tok] + w[1][L.tok]) + (w[2][L.tok] + w[3][L.tok]);
        const float m = dead || sh.unseen[L.g][L.tok] != 0.0f ? NEG_INF : -reinterpret_cast<const float*>(&sh.fr[rb][col >> 1])[2 + (col & 1)];
        float4 c = make_float4(1.0f, __int_as_float(-1), __int_as_float(t), 0.0f);
        if (col < T.MR && r < P.R) {
            c.y = __int_as_float(row);
            const bool live = t < rows && l != 0.0f;
            if (whole) {
                float lse = live ? (m + log2f(l)) * LN2 : NEG_INF;
                c.x = live ? 1.0f / l : 0.0f;
                if (status != ROW_OK) lse = c.x = __int_as_float(0x7fc00000);
                if (P.lse) P.lse[(size_t)b * P.T * P.Hq + row] = lse;
            } else {
                part[(size_t)T.MR * D + col] = m;
                part[(size_t)T.MR * D + T.MR + col] = l;
            }
        }
        sh.col[L.g][L.tok] = c;
    }
    group_sync(L.bar_id);
    uint16_t* out = reinterpret_cast<uint16_t*>(P.out) + (size_t)b * P.T * P.Hq * D + L.tok;
    const auto put = [&](int c, float x) {
        const float2 q = *reinterpret_cast<const float2*>(&sh.col[L.g][c]);
        // a dead row's sums are zeros that no token touched; with a status they become NaN
        const float y = q.x == 0.0f ? 0.0f : x * q.x;
        if (__float_as_int(q.y) >= 0)
            out[(size_t)__float_as_int(q.y) * D] = DT == DT_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
    };
    const auto put_part = [&](int c, float x) {
        if (__float_as_int(sh.col[L.g][c].y) >= 0) part[(size_t)(L.col0 + c) * D + L.tok] = x;
    };
    if (vbad && !dead) {
#pragma unroll 1
        for (int c = 0; c < cw; ++c) {
            uint32_t o;
            tmem_ld1(t_o + c, o);
            if (L.tok >= D) continue;
            const float4 q = sh.col[L.g][c];
            float x = __uint_as_float(o);
            if (__float_as_int(q.y) >= 0 && __float_as_int(q.z) < rows) x += unfinite_values<DT>(P, b, h, __float_as_int(q.z), L.tok);
            if (whole) put(c, x);
            else put_part(c, x);
        }
    } else
#pragma unroll 1
    for (int c = 0; c < cw; c += 16) {
        uint32_t o[16];
        if (!dead) tmem_ld16_nowait(t_o + c, o);
        tmem_wait_ld();
        if (L.tok >= D) continue;
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (dead) o[j] = 0u;
        if (whole) {
#pragma unroll
            for (int j = 0; j < 16; ++j) put(c + j, __uint_as_float(o[j]));
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) put_part(c + j, __uint_as_float(o[j]));
        }
    }
    tc_fence_before();
    group_sync(L.bar_id);
}

template <int DT, int D>
__device__ void role_softmax(const TcParams& T, Shared& sh, const Place& at, uint8_t* smem, uint32_t tmem)
{
    const AttnParams& P = T.A;
    const int wid = (threadIdx.x >> 5) - SMW0, chunks = T.RN / 16;
    Lane L;
    L.smem = smem;
    L.g = wid >> 2;
    L.quad = wid & 3;
    L.lane = threadIdx.x & 31;
    L.tok = L.quad * 32 + L.lane;
    L.tl = tmem + ((uint32_t)(L.quad * 32) << 16);
    L.bar_id = 1 + L.g;
    L.col0 = L.g * chunks / NG * 16;
    L.nch = (L.g + 1) * chunks / NG - L.g * chunks / NG;
    int it = 0, s_at = 0, rb = 0;
    bool dead = false;
    for (Walk w(P, at); w.open(P); w.next()) {
        int status = w.rq.status;
        bool vbad = false;
        if (!dead) load_q<DT, D>(T, sh, L, w.b, w.h, w.rt, w.rq.rows);
        for (int tile = w.tile0; tile < w.tile1 && !dead;) {
            const bool own = tile >= w.rq.ncache;
            uint64_t see = 0;
            bool fail = false;
            if (own) {
                bool bad;
                fail = own_tile<DT, D>(T, sh, L, it, w.b, w.rt, w.rq.rows, (tile - w.rq.ncache) * TT, &see, &bad);
                if (bad) status = ROW_BAD_PARENT;
            }
            // A group's first tile has no reference yet; another's may turn out too low, and the tile is repeated.  `stops`: how
            // often the present tile has passed the window: it gets a reference, then weights held at the window; a third time
            // would end the CTA's work as a wait that ran out does, so no tile can keep the loop running, whatever its scores are.
            bool first = tile == w.tile0;
            int stops = first ? 1 : 0;
            uint32_t take = ~0u;
            const int end = own ? tile + 1 : min(w.tile1, w.rq.ncache);
            while (tile < end) {
                if (stops > 0) {
                    if (stops > 2 || !move_reference(T, sh, L, rb, it, s_at, w.rq.len - tile * TT, own, see, first, stops == 2)) {
                        *reinterpret_cast<volatile int*>(&sh.fail) = 1;
                        dead = true;
                        break;
                    }
                    if (stops == 1) rb ^= 1;
                }
                const bool hold = stops == 2;
                const RunEnd r = softmax_run(T, sh, L, &sh.fr[hold ? rb ^ 1 : rb][L.col0 / 2], it, s_at, tile, hold ? tile + 1 : end, w.rq.len, own, see, take);
                status = max(status, r.status);
                tile += r.n;
                it += r.n;
                for (s_at += r.n; s_at >= T.stages;) s_at -= T.stages;
                if (r.stopped && group_any(L.bar_id, fail || r.fail)) {
                    dead = true;
                    break;
                }
                stops = !r.stopped ? 0 : r.n > 0 ? 1 : stops + 1;
                first = false;
                take = r.stopped ? r.left_out : ~0u;
            }
            if (own && !dead)
                for (int k = 0; k < VWN; ++k) vbad = vbad || sh.vbad[(it - 1) & 3][k];
        }
        if (!dead) dead = group_any(L.bar_id, !wait_warp(sh, &sh.pv[(it - 1) & 1], ((it - 1) >> 1) & 1, T.wait_limit));
        if (dead) {
            status = ROW_TIMEOUT;
            if (L.tok == 0) {
                if (sh.lost[L.g][1] == 0) sh.lost[L.g][0] = w.b;
                sh.lost[L.g][1] = w.b + 1;
            }
        }
        float* part = P.parts + ((size_t)blockIdx.x * 2 + (w.tile0 != 0 ? 0 : 1)) * part_floats(T.MR, D);
        put_outputs<DT, D>(T, sh, L, rb, w.b, w.h, w.rt, w.rq.rows, w.whole, part, status, dead, vbad);
        // (but for waits that ran out, which `lost` tells of, the softmax groups' statuses are the same)
        if (threadIdx.x == SMW0 * 32) {
            begin_status(P, w.b, w.h, w.rt, w.tile0, status);
            if (!w.whole) {
                part[(size_t)T.MR * D + 2 * T.MR] = __int_as_float(status);
                if (w.tile0 == 0) P.joins[blockIdx.x] = {parts_of(at.total, blockIdx.x, at.ctas, w.u + w.rq.n), w.b, w.h, w.rt, w.rq.rows};
            }
        }
    }
}

template <int DT, int D>
__global__ void __launch_bounds__(TNT, 1)
attn_tc_kernel(const __grid_constant__ TcParams T, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv)
{
    extern __shared__ uint8_t raw[];
    uint8_t* const smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);  // the swizzled tiles' alignment
    __shared__ Shared sh;
    const AttnParams& P = T.A;
    const int tid = threadIdx.x, w = tid >> 5;
    if (tid == 0) {
        P.joins[blockIdx.x] = {};
        for (int i = 0; i < T.stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.info[i], 1);
            mbar_init(&sh.empty[i], 1 + VWN + 4 * NG);  // the products' commit, and the warps that read the pages and the scales
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.sfull[i], 1);
            mbar_init(&sh.ready[i], 4 * NG + VWN);  // weights and values
            mbar_init(&sh.own[i], 4 * NG + VWN);    // the round's rows: q, keys and values as halfs
            mbar_init(&sh.pv[i], 1);
        }
        mbar_init(&sh.qfull, 4 * NG);
        mbar_init(&sh.done, 1);
        sh.fail = 0;
        for (int g = 0; g < NG; ++g) sh.lost[g][1] = 0;
        fence_mbar_init();
    }
    launch_dependents();
    if constexpr (D == 64) {  // the block of zeros that stands for channels 64 .. 127
        uint8_t* z = smem + T.o_v + T.nv * T.v_buf;
        for (int i = tid; i < 16384 / 16; i += TNT) reinterpret_cast<uint4*>(z)[i] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    const Place at = find_place<TT>(P, blockIdx.x, gridDim.x, &sh.place);  // a barrier for all
    if ((int)blockIdx.x >= at.ctas) return;
    if (w == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" :: "r"(smem_addr(&sh.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (w == 0) role_copy<D>(T, sh, at, smem_addr(smem) + T.o_stage, &mk, &mv);
    else if (w == 1) {
        role_mma<DT, D>(T, sh, at, smem_addr(smem), tmem);
    } else if (w < VW0 + VWN) role_values<DT, D>(T, sh, at, smem);
    else if (w >= SMW0) role_softmax<DT, D>(T, sh, at, smem, tmem);
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        int lo = P.B, hi = 0;
        for (int g = 0; g < NG; ++g)
            if (sh.lost[g][1] > 0) lo = min(lo, sh.lost[g][0]), hi = max(hi, sh.lost[g][1]);
        if (hi > 0) {
            P.joins[blockIdx.x].lost0 = lo;
            P.joins[blockIdx.x].lost1 = hi;
        }
    }
    if (w == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" :: "r"(tmem));
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// codes [pages * Hkv, page, D]; a box is one page of one head
bool cache_map(CUtensorMap* m, const AttnParams& P, const uint8_t* codes, CUtensorMapSwizzle swizzle)
{
    const cuuint64_t dims[3] = {(cuuint64_t)P.D, (cuuint64_t)P.page, (cuuint64_t)P.pages * P.Hkv};
    const cuuint64_t strides[2] = {(cuuint64_t)P.D, (cuuint64_t)P.D * P.page};
    const cuuint32_t box[3] = {(cuuint32_t)P.D, (cuuint32_t)P.page, 1}, step[3] = {1, 1, 1};
    const EncodeTiled f = encode_tiled();
    return f && f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(codes), dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT, int D>
cudaError_t launch_tc(AttnParams& P, int sms, cudaStream_t st)
{
    TcParams T;
    P.RT = (P.R + MAXR - 1) / MAXR;
    T.MR = (P.R + P.RT - 1) / P.RT;
    T.RN = (T.MR + 15) / 16 * 16;
    T.A = P;
    T.wait_limit = P.wait_limit;
    T.inv_g = (1ull << 32) / (uint64_t)P.G + 1;
    const uint32_t terms = DT == DT_BF16 ? 2 : 3, blocks = (uint32_t)(T.RN + 63) / 64;
    T.p_buf = blocks * 16384;
    T.v_buf = D / 64 * 16384;
    const uint32_t stage = TT * D, keys = 2 * TT * D;
    // second buffers of the values and of P where three stages of keys still fit beside them
    for (int extra = 2;; --extra) {
        T.nv = extra >= 1 ? 2 : 1;
        T.np = extra >= 2 ? 2 : 1;
        T.o_p = terms * T.RN * D;
        T.o_v = T.o_p + T.np * T.p_buf;
        T.o_kh = T.o_v + T.nv * T.v_buf + (D == 64 ? 16384 : 0);
        T.o_stage = T.o_kh + keys;
        T.stages = (int)(((int)TC_SMEM - 1024 - (int)T.o_stage) / (int)stage);
        if (T.stages >= 3 || extra == 0) break;
    }
    if (T.stages > MAXSTAGES) T.stages = MAXSTAGES;
    const auto vec = [](const void* p, int64_t a, int64_t b, int64_t c, int64_t n) {
        return reinterpret_cast<uintptr_t>(p) % (2 * n) == 0 && a % n == 0 && b % n == 0 && c % n == 0;
    };
    T.qvec = vec(P.q, P.qb, P.qt, P.qh, 8);
    T.kvec = vec(P.kn, P.kb, P.kt, P.kh, D / 32);
    T.vvec = vec(P.vn, P.vb, P.vt, P.vh, D / 32);
    const size_t bytes = 1024 + T.o_stage + (size_t)T.stages * stage;
    auto* k = attn_tc_kernel<DT, D>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)TC_SMEM);
    if (e != cudaSuccess) return e;
    CUtensorMap mk, mv;
    if (!cache_map(&mk, P, P.kc, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B) ||
        !cache_map(&mv, P, P.vc, CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    const int ctas = sms < ATTN_MAX_TC_CTAS ? sms : ATTN_MAX_TC_CTAS;
    k<<<ctas, TNT, bytes, st>>>(T, mk, mv);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_attn_merge(P, DT, ctas, T.MR, st);
}

}  // namespace

cudaError_t launch_attention_tc(AttnParams& P, int dtype, int sms, cudaStream_t st)
{
    if (dtype == DT_BF16) return P.D == 128 ? launch_tc<DT_BF16, 128>(P, sms, st) : launch_tc<DT_BF16, 64>(P, sms, st);
    return P.D == 128 ? launch_tc<DT_F16, 128>(P, sms, st) : launch_tc<DT_F16, 64>(P, sms, st);
}

}  // namespace sv
