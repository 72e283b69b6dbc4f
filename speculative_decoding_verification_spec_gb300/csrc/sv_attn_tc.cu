// sv_attn_tc.cu -- verify_attention for many rows, on the tensor cores (tcgen05).
//
// The arithmetic is that of sv_attn.cu: u_j = log2(e) s_j + e_j, weights 2^(u_j - m) against a lazily moved reference m,
// o = sum p' c / sum p' 2^(-e).  Tokens lie on the 128 lanes of an accumulator and the rows of q, up to 160 of one
// key/value head, are its columns, so a tile costs what its rows cost, without padding to 128:
//   S^T [128 tokens, rows] = K [128, D] Q^T:   the codes of K go from memory to the product as they are (e4m3 x e4m3);
//       a row of q, scaled by a power of two to a largest element in [128, 256), is split into e4m3 terms that sum to it,
//       two for bf16 (4 bits each, the residual's sign the ninth: exact for elements above 2^-10 of the largest, off by at
//       most 2^-17 of it below) and three for halfs, whose products accumulate.
//   O^T [D, rows] += V^T [D, 128] P^T:   halfs; two warps widen the codes of V into shared memory, and the weights are
//       rounded to halfs (half a step, 2^-11, under the output's own rounding).
// The round's own rows come last, as tiles of their own: keys and values as halfs scaled by a power of two per token, and a
// copy of q as halfs.
//
// One CTA per SM works through an equal run of all groups' tiles (as in sv_attn.cu), with a role per warp:
//   0      copies: the pages' codes by TMA into a ring of stages, the pages' scales beside them
//   1      products: one lane issues them; S is double-buffered, so S of the next tile runs under this tile's softmax
//   2, 3   values to halfs
//   4 - 11 softmax, two groups of four warps; a thread is a token, a group takes half of the columns.  The weights are taken
//          against the reference as it stands; only when one passes 2^15 (the first tile of a group, and rarely after) does the
//          group find the columns' maxima, move the reference, rescale its part of O^T and repeat the tile.
// Every wait on an mbarrier is bounded; when one runs out the CTA's remaining groups report SPEC_ROW_TIMEOUT.  Between named
// barriers the threads of a softmax group never part: what a wait returned is agreed on before anyone acts on it.
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "sv_attn.cuh"

namespace sv {

namespace {

constexpr int TT = 128;          // tokens of a tile
constexpr int TNT = 384;         // threads
constexpr int SMW0 = 4;          // first softmax warp
constexpr int MAXR = 160;        // rows of a group, columns of S^T: S twice and O within 512 columns
constexpr int HALFR = MAXR / 2;  // columns of a softmax group
constexpr int MAXSTAGES = 6;
constexpr float WINDOW = 15.0f;  // a weight may reach 2^WINDOW (the largest half is near 2^16)
constexpr float HEAD = 7.0f;     // a moved reference leaves the maximum at 2^HEAD
constexpr float FAR = 40.0f;     // log2 of a weight that the first pass keeps out of l: with the 2^74 of a scale it could soon
                                 // leave fp32's range
constexpr size_t TC_SMEM = 216 * 1024;  // dynamic shared memory; the static arrays take the rest of the SM's 227 KB

struct TcParams {
    AttnParams A;
    int MR, RN;          // rows of a row tile; padded to a multiple of 16
    int stages, np, nv;  // ring stages; buffers of P and of the widened values (1 or 2)
    uint32_t o_p, o_v, o_stage, v_buf, p_buf;  // offsets in dynamic shared memory, sizes
    int wait_limit;
};

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ uint64_t desc_base(uint32_t layout, uint32_t lbo, uint32_t sbo)
{
    // strides in bytes; bit 46: the descriptor version of this architecture; bits 61-63: the swizzle
    return (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 | (uint64_t)layout << 61;
}
__device__ __forceinline__ uint64_t desc_at(uint64_t base, uint32_t addr) { return base | (uint64_t)((addr >> 4) & 0x3fffu); }
constexpr uint32_t SW128 = 2, SW64 = 4;

// instruction descriptor: fp32 accumulator, M = 128, N, both operands of format 0 (e4m3 / half); `mn`: both with their M / N
// dimension contiguous
__device__ __forceinline__ uint32_t idesc(int N, bool mn)
{
    return 1u << 4 | (mn ? 1u << 15 | 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 | (128u >> 4) << 24;
}

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }"
                 :: "r"(d), "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void mma_h(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc)
{
    asm volatile("{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }"
                 :: "r"(d), "l"(a), "l"(b), "r"(id), "r"((uint32_t)acc) : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// 16 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                    "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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
    uint64_t sfull[2], sfree[2], pfull[2], vfull[2], pv[2], qfull, q16, done;
    float2 scale[MAXSTAGES][8];   // of the stage's pages: keys, values
    int status[MAXSTAGES];
    float4 fr[2][MAXR / 2];       // per pair of columns: factors, references; two copies, one being rewritten
    float wmax[2][4][HALFR];      // column maxima (and sums of l) of the softmax warps
    float fac[2][HALFR];
    uint32_t mask[MAXR][4];       // round's rows: which tokens of the tile a column sees
    float fks[2][TT], fve[2][TT]; // round's rows: scale of the keys and exponent of the values, per token
    int vbad[4][2];               // round's rows: a tile's values hold a NaN or an infinity, per warp
    int fail;
    uint32_t tmem;
    Place place;
};

// Bounded wait; ends early once another role has given up.  The result is the warp's.
__device__ __forceinline__ bool wait_on(Shared& sh, uint64_t* bar, uint32_t parity, int limit)
{
    for (int n = 0; n < limit; n += 64) {
        if (mbar_wait(bar, parity, min(64, limit - n))) return true;
        if (*reinterpret_cast<volatile int*>(&sh.fail)) return false;
    }
    *reinterpret_cast<volatile int*>(&sh.fail) = 1;
    return false;
}
__device__ __forceinline__ bool wait_warp(Shared& sh, uint64_t* bar, uint32_t parity, int limit)
{
    return __all_sync(0xffffffffu, wait_on(sh, bar, parity, limit));
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
    bool whole, first;

    __device__ Walk(const AttnParams& P, const Place& at)
    {
        u = at.total * blockIdx.x / at.ctas;
        u1 = at.total * (blockIdx.x + 1) / at.ctas;
        pre = at.pre;
        b = at.b;
        RT = P.RT;
        rq = req_info<TT>(P, b);
        first = true;
    }
    __device__ bool more() const { return u < u1; }
    __device__ void open()
    {
        const long long rem = u - pre;
        const int grp = (int)(rem / rq.n);
        tile0 = (int)(rem % rq.n);
        h = grp / RT;
        rt = grp % RT;
        tile1 = (int)min((long long)rq.n, tile0 + (u1 - u));
        whole = tile0 == 0 && tile1 == rq.n;
    }
    __device__ void next(const AttnParams& P)
    {
        first = false;
        u += tile1 - tile0;
        while (u < u1 && u >= pre + (long long)rq.n * P.Hkv * RT) {
            pre += (long long)rq.n * P.Hkv * RT;
            rq = req_info<TT>(P, ++b);
        }
    }
};

// ---------------------------------------------------------------- roles

template <int D>
__device__ void role_copy(const TcParams& T, Shared& sh, const Place& at, uint32_t ring, const CUtensorMap* mk, const CUtensorMap* mv)
{
    const AttnParams& P = T.A;
    const int lane = threadIdx.x & 31;
    const int ppt = TT / P.page;           // pages of a tile
    const int per = 32 / ppt;              // tiles whose pages the warp's lanes hold at once
    constexpr uint32_t KB = TT * D;
    int it = 0;
    bool ok = true;
    for (Walk w(P, at); ok && w.more(); w.next(P)) {
        w.open();
        const int32_t* table = P.page_table + (size_t)w.b * P.table_width;
        const int c0 = min(w.tile0, w.rq.ncache), c1 = min(w.tile1, w.rq.ncache);
        // lane k holds page k of a batch of `per` tiles: its number, and a batch ahead the next one's
        const auto page_of = [&](int tile) {
            const long long tok = (long long)tile * TT + (long long)lane * P.page;
            return tile < c1 && tok < w.rq.len ? __ldg(table + (tok >> P.page_shift)) : 0;
        };
        int page = 0, ahead = c0 < c1 ? page_of(c0) : 0;
        float ks = 1.0f, vs = 1.0f;
        for (int tile = w.tile0; tile < w.tile1; ++tile, ++it) {
            const int s = it % T.stages;
            if (it >= T.stages && !wait_warp(sh, &sh.empty[s], ((it / T.stages) & 1) ^ 1, T.wait_limit)) {
                ok = false;
                break;
            }
            if (tile < c1) {
                const int at_lane = (tile - c0) % per * ppt;
                if (at_lane == 0) {
                    page = ahead;
                    const bool good = (unsigned)page < (unsigned)P.pages;
                    const size_t blk = good ? (size_t)page * P.Hkv + w.h : 0;
                    const bool live = (long long)tile * TT + (long long)lane * P.page < w.rq.len && tile + lane / ppt < c1;
                    ks = live ? __ldg(P.ks + blk) : 1.0f;
                    vs = live ? __ldg(P.vs + blk) : 1.0f;
                    ahead = page_of(tile + per);
                }
                const int live_pages = min(ppt, (w.rq.len - tile * TT + P.page - 1) >> P.page_shift);
                const bool mine = lane >= at_lane && lane < at_lane + live_pages;
                const bool good = (unsigned)page < (unsigned)P.pages;
                const unsigned use = __ballot_sync(0xffffffffu, mine && good);
                if (lane == 0) mbar_expect(&sh.full[s], (uint32_t)__popc(use) * 2u * (uint32_t)(P.page * D));
                __syncwarp();
                if (mine && good) {
                    const uint32_t dst = ring + s * 2 * KB + (lane - at_lane) * P.page * D;
                    tma_page(dst, mk, page * P.Hkv + w.h, &sh.full[s]);
                    tma_page(dst + KB, mv, page * P.Hkv + w.h, &sh.full[s]);
                }
                if (mine) sh.scale[s][lane - at_lane] = make_float2(ks, vs);
                const bool bad = __any_sync(0xffffffffu, mine && !good);
                if (lane == 0) sh.status[s] = bad ? ROW_BAD_PAGE : ROW_OK;
            } else if (lane == 0) {
                sh.status[s] = ROW_OK;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.full[s]);
        }
    }
    // no copy may be in flight when the CTA ends: the last fill of every stage
    if (lane == 0)
        for (int j = max(0, it - T.stages); j < it; ++j) (void)mbar_wait(&sh.full[j % T.stages], (j / T.stages) & 1, MBAR_SPIN_LIMIT);
    __syncwarp();
}

// One lane.  Products of tile `it`: S^T as soon as its keys are there; O^T of the tile before after that, except
// where the next S^T needs what the softmax does only after that O^T (a group's first tile, the round's rows).
template <int DT, int D>
__device__ void role_mma(const TcParams& T, Shared& sh, const Place& at, uint32_t base, uint32_t tmem)
{
    const AttnParams& P = T.A;
    constexpr int TERMS = DT == DT_BF16 ? 2 : 3;
    constexpr uint32_t KB = TT * D;
    const uint32_t sp = base + T.o_p, sv_ = base + T.o_v, ring = base + T.o_stage;
    const uint32_t qterm = (uint32_t)T.RN * D;
    const uint64_t dk = D == 128 ? desc_base(SW128, 16, 1024) : desc_base(SW64, 16, 512);
    const uint64_t dkh = desc_base(SW128, 16, 1024);
    const uint64_t dp = desc_base(SW128, 16384, 1024);
    const uint32_t id_s = idesc(T.RN, false), id_o = idesc(T.RN, true);
    const uint32_t t_o = tmem + 2 * T.RN;
    int it = 0, seg = 0, own = 0;  // own: tiles of the rounds' rows so far
    bool ok = true;
    int pending = -1;
    bool pending_first = false;

    const auto pv = [&]() {  // O^T of tile `pending`
        const int i = pending;
        pending = -1;
        if (!wait_on(sh, &sh.pfull[i & 1], (i >> 1) & 1, T.wait_limit) || !wait_on(sh, &sh.vfull[i & 1], (i >> 1) & 1, T.wait_limit)) return false;
        tc_fence_after();
        const uint32_t vb = sv_ + (i % T.nv) * T.v_buf, pb = sp + (i % T.np) * T.p_buf;
        // the second block of 64 channels: the next 16 KB, or (D = 64) the block of zeros after the buffers
        const uint64_t dv = desc_base(SW128, D == 128 ? 16384 : T.nv * T.v_buf - (i % T.nv) * T.v_buf, 1024);
#pragma unroll
        for (int k = 0; k < TT / 16; ++k)
            mma_h(t_o, desc_at(dv, vb + k * 2048), desc_at(dp, pb + k * 2048), id_o, !(pending_first && k == 0));
        mma_commit(&sh.pv[i & 1]);
        return true;
    };

    for (Walk w(P, at); ok && w.more(); w.next(P), ++seg) {
        w.open();
        for (int tile = w.tile0; ok && tile < w.tile1; ++tile, ++it) {
            const int s = it % T.stages;
            const bool fresh = tile >= w.rq.ncache;
            const bool first = tile == w.tile0;
            if (pending >= 0 && (first || fresh)) ok = pv();
            ok = ok && wait_on(sh, &sh.full[s], (it / T.stages) & 1, T.wait_limit);
            if (it >= 2) ok = ok && wait_on(sh, &sh.sfree[it & 1], ((it >> 1) & 1) ^ 1, T.wait_limit);
            if (first) ok = ok && wait_on(sh, &sh.qfull, seg & 1, T.wait_limit);
            if (fresh) {
                ok = ok && wait_on(sh, &sh.vfull[it & 1], (it >> 1) & 1, T.wait_limit) && wait_on(sh, &sh.q16, own & 1, T.wait_limit);
                ++own;
            }
            if (!ok) break;
            tc_fence_after();
            const uint32_t ts = tmem + (it & 1) * T.RN, kb = ring + s * 2 * KB;
            if (!fresh) {
#pragma unroll
                for (int q = 0; q < TERMS; ++q)
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        mma_f8(ts, desc_at(dk, kb + k * 32), desc_at(dk, base + q * qterm + k * 32), id_s, q + k > 0);
            } else {
                const uint32_t qb = sp + (it % T.np) * T.p_buf;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    mma_h(ts, desc_at(dkh, kb + (k >> 2) * 16384 + (k & 3) * 32),
                          desc_at(dkh, qb + (k >> 2) * T.RN * 128 + (k & 3) * 32), id_s, k > 0);
            }
            mma_commit(&sh.sfull[it & 1]);
            mma_commit(&sh.empty[s]);
            if (pending >= 0) ok = pv();
            pending = it;
            pending_first = first;
        }
    }
    if (ok && pending >= 0) (void)pv();
    // everything issued has ended before the accumulators are given back
    mma_commit(&sh.done);
    (void)mbar_wait(&sh.done, 0, MBAR_SPIN_LIMIT);
}

// byte offset of channels d .. (within 8) of a token in a [token][64 channels] block of halfs, 128-byte swizzle
__device__ __forceinline__ uint32_t half_off(int token, int d)
{
    return (uint32_t)(d >> 6) * 16384u + token * 128u + ((((d & 63) >> 3) ^ (token & 7)) << 4) + (d & 7) * 2;
}

template <int DT, int D>
__device__ void role_values(const TcParams& T, Shared& sh, const Place& at, uint8_t* smem)
{
    const AttnParams& P = T.A;
    constexpr int KB = TT * D, CH = D / 16, EPL = D / 32;
    const int ct = threadIdx.x - 64, w2 = ct >> 5, lane = ct & 31;
    int it = 0;
    bool ok = true;
    for (Walk w(P, at); ok && w.more(); w.next(P)) {
        w.open();
        for (int tile = w.tile0; tile < w.tile1; ++tile, ++it) {
            const int s = it % T.stages;
            uint8_t* vb = smem + T.o_v + (it % T.nv) * T.v_buf;
            uint8_t* kb = smem + T.o_stage + s * 2 * KB;
            ok = wait_warp(sh, &sh.full[s], (it / T.stages) & 1, T.wait_limit);
            if (it >= T.nv) ok = ok && wait_warp(sh, &sh.pv[(it - T.nv) & 1], ((it - T.nv) >> 1) & 1, T.wait_limit);
            if (!ok) break;
            if (tile < w.rq.ncache) {
                const int valid = w.rq.len - tile * TT;
#pragma unroll 4
                for (int i = ct; i < TT * CH; i += 64) {
                    const int tok = i / CH, ch = i % CH;
                    uint4 x = *reinterpret_cast<const uint4*>(kb + KB + i * 16);
                    if (tok >= valid) x = make_uint4(0, 0, 0, 0);  // whatever the slot holds
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
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
            } else {
                // the round's rows: keys into the stage, values into the buffer, scaled by a power of two per token
                const int j0 = (tile - w.rq.ncache) * TT;
                bool vbad = false;
                for (int i = w2; i < TT; i += 2) {
                    const int j = j0 + i;
                    const bool live = P.kn && j < w.rq.rows;
#pragma unroll
                    for (int which = 0; which < 2; ++which) {
                        const void* src = which ? P.vn : P.kn;
                        const int64_t off = which ? w.b * P.vb + j * P.vt + w.h * P.vh : w.b * P.kb + j * P.kt + w.h * P.kh;
                        float x[EPL], amax = 0.0f;
                        bool fin = true;
#pragma unroll
                        for (int k = 0; k < EPL; ++k) {
                            x[k] = live ? load_elem<DT>(src, off + lane * EPL + k) : 0.0f;
                            if (fabsf(x[k]) < __int_as_float(0x7f800000)) amax = fmaxf(amax, fabsf(x[k]));
                            else fin = false, x[k] = 0.0f;
                        }
                        fin = __all_sync(0xffffffffu, fin);
#pragma unroll
                        for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                        const int e = min(max(exponent_of(amax), CACHE_E_MIN), 126) - 14;
                        const float mul = exp2_int(-e);
                        uint8_t* to = (which ? vb : kb) + half_off(i, lane * EPL);
                        if constexpr (EPL == 4)
                            *reinterpret_cast<uint2*>(to) = make_uint2(pack_half2(x[0] * mul, x[1] * mul), pack_half2(x[2] * mul, x[3] * mul));
                        else
                            *reinterpret_cast<uint32_t*>(to) = pack_half2(x[0] * mul, x[1] * mul);
                        if (which) vbad = vbad || !fin;
                        if (lane == 0) {
                            if (which) sh.fve[it & 1][i] = (float)e;
                            else sh.fks[it & 1][i] = fin ? exp2_int(e) : __int_as_float(0x7fc00000);  // a key that is not finite: NaN
                        }
                    }
                }
                if (lane == 0) sh.vbad[it & 3][w2] = vbad;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.vfull[it & 1]);
                mbar_arrive(&sh.empty[s]);
            }
        }
    }
}

template <int DT, int D>
__device__ void role_softmax(const TcParams& T, Shared& sh, const Place& at, uint8_t* smem, uint32_t tmem)
{
    const AttnParams& P = T.A;
    constexpr int TERMS = DT == DT_BF16 ? 2 : 3;
    const int wid = (threadIdx.x >> 5) - SMW0, g = wid >> 2, quad = wid & 3, lane = threadIdx.x & 31;
    const int tok = quad * 32 + lane;       // this thread's token of a tile, and its channel of O^T
    const int bar_id = 1 + g;
    const int ca = ((T.RN / 16 + 1) / 2) * 16;           // columns of group 0
    const int col0 = g ? ca : 0, cw = g ? T.RN - ca : ca;
    const int nch = cw / 16;
    const uint32_t tl = tmem + ((uint32_t)(quad * 32) << 16);  // this warp's lanes
    const uint32_t t_o = tl + 2 * T.RN + col0;
    float4* const fr0 = &sh.fr[0][col0 / 2];
    float4* const fr1 = &sh.fr[1][col0 / 2];
    int it = 0, rb = 0;
    bool dead = false;

    for (Walk w(P, at); w.more(); w.next(P)) {
        w.open();
        int status = w.rq.status;
        bool vbad = false;
        unsigned long long l2[HALFR / 2];
#pragma unroll
        for (int i = 0; i < HALFR / 2; ++i) l2[i] = 0ull;

        if (!dead) {
            // ---- the rows of q as e4m3 terms; a warp takes every fourth column of its group
            for (int c = quad; c < cw; c += 4) {
                const int col = col0 + c, r = w.rt * T.MR + col, t = r / P.G;
                const bool live = col < T.MR && r < P.R && t < w.rq.rows;
                constexpr int EPL = D / 32;
                float x[EPL], amax = 0.0f;
                bool fin = true;
                const int64_t off = live ? (int64_t)w.b * P.qb + (int64_t)t * P.qt + (int64_t)(w.h * P.G + r % P.G) * P.qh : 0;
#pragma unroll
                for (int k = 0; k < EPL; ++k) {
                    x[k] = live ? load_elem<DT>(P.q, off + lane * EPL + k) : 0.0f;
                    fin = fin && fabsf(x[k]) < __int_as_float(0x7f800000);
                    amax = fmaxf(amax, fabsf(x[k]));
                }
                fin = __all_sync(0xffffffffu, fin);
#pragma unroll
                for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                const int e = fin ? min(max(7 - exponent_of(amax), -120), 126) : 0;
                const float mul = exp2_int(e);
                if (!fin) {
#pragma unroll
                    for (int k = 0; k < EPL; ++k) x[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < EPL; ++k) x[k] *= mul;
                const int d = lane * EPL;
                const uint32_t at_q = D == 128 ? col * 128 + (((d >> 4) ^ (col & 7)) << 4) + (d & 15)
                                               : col * 64 + (((d >> 4) ^ ((col >> 1) & 3)) << 4) + (d & 15);
#pragma unroll
                for (int q = 0; q < TERMS; ++q) {
                    uint32_t code = 0;
#pragma unroll
                    for (int k = 0; k < EPL; k += 2) {
                        const uint16_t c2 = e4m3x2_from(x[k], x[k + 1]);
                        const uint32_t h2 = e4m3x2_to_half2(c2);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
                        x[k] -= f.x;
                        x[k + 1] -= f.y;
                        code |= (uint32_t)c2 << (8 * k);
                    }
                    uint8_t* to = smem + (size_t)q * T.RN * D + at_q;
                    if constexpr (EPL == 4) *reinterpret_cast<uint32_t*>(to) = code;
                    else *reinterpret_cast<uint16_t*>(to) = (uint16_t)code;
                }
                if (lane == 0) {
                    // a row of q with a NaN or an infinity has no scores
                    const float F = fin ? P.scale * LOG2E * exp2_int(-e) : __int_as_float(0x7fc00000);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float* f = reinterpret_cast<float*>(k ? &fr1[c >> 1] : &fr0[c >> 1]);
                        f[c & 1] = F;
                        f[2 + (c & 1)] = 0.0f;
                    }
                }
            }
            fence_proxy_async_smem();
        }
        group_sync(bar_id);
        if (!dead && lane == 0) mbar_arrive(&sh.qfull);

        for (int tile = w.tile0; tile < w.tile1; ++tile, ++it) {
            if (dead) break;
            const bool first = tile == w.tile0, fresh = tile >= w.rq.ncache;
            uint8_t* pb = smem + T.o_p + (it % T.np) * T.p_buf;
            bool fail = false;
            if (fresh) {
                // a copy of q as halfs where P will be, and which rows each column sees
                if (it >= 1) fail = !wait_warp(sh, &sh.pv[(it - 1) & 1], ((it - 1) >> 1) & 1, T.wait_limit);
                const int j0 = (tile - w.rq.ncache) * TT;
                bool badp = false;
                if (!fail) {
                    for (int c = quad; c < cw; c += 4) {
                        const int col = col0 + c, r = w.rt * T.MR + col, t = r / P.G;
                        const bool live = col < T.MR && r < P.R && t < w.rq.rows;
                        constexpr int EPL = D / 32;
                        const int64_t off = live ? (int64_t)w.b * P.qb + (int64_t)t * P.qt + (int64_t)(w.h * P.G + r % P.G) * P.qh : 0;
                        float x[EPL], amax = 0.0f;
#pragma unroll
                        for (int k = 0; k < EPL; ++k) {
                            x[k] = live ? load_elem<DT>(P.q, off + lane * EPL + k) : 0.0f;
                            if (!(fabsf(x[k]) < __int_as_float(0x7f800000))) x[k] = 0.0f;  // its factor is NaN
                            amax = fmaxf(amax, fabsf(x[k]));
                        }
#pragma unroll
                        for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                        const float mul = exp2_int(min(max(7 - exponent_of(amax), -120), 126));
                        const int d = lane * EPL;
                        uint8_t* to = pb + (size_t)(d >> 6) * T.RN * 128 + col * 128 + ((((d & 63) >> 3) ^ (col & 7)) << 4) + (d & 7) * 2;
                        if constexpr (EPL == 4)
                            *reinterpret_cast<uint2*>(to) = make_uint2(pack_half2(x[0] * mul, x[1] * mul), pack_half2(x[2] * mul, x[3] * mul));
                        else
                            *reinterpret_cast<uint32_t*>(to) = pack_half2(x[0] * mul, x[1] * mul);
                    }
                    if (tok < cw) {
                        const int r = w.rt * T.MR + col0 + tok, t = r / P.G;
                        uint32_t m[4] = {0, 0, 0, 0};
                        if (P.kn && t < w.rq.rows) {
                            if (!P.parents) {
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const int n = t + 1 - j0 - 32 * k;
                                    m[k] = n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
                                }
                            } else {
                                for (int cur = t;;) {
                                    const int o = cur - j0;
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        if ((o >> 5) == k && o >= 0) m[k] |= 1u << (o & 31);
                                    if (cur == 0) break;
                                    const int p = __ldg(P.parents + (size_t)w.b * (P.T - 1) + cur - 1);
                                    if (p < -1 || p >= cur - 1) break;  // reported below; the walk always ends
                                    cur = p + 1;
                                }
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) sh.mask[col0 + tok][k] = m[k];
                    }
                    if (P.parents)
                        for (int i = tok; i < w.rq.rows - 1; i += 128) {
                            const int p = __ldg(P.parents + (size_t)w.b * (P.T - 1) + i);
                            badp = badp || p < -1 || p >= i;
                        }
                    fence_proxy_async_smem();
                }
                if (group_any(bar_id, badp)) status = ROW_BAD_PARENT;
                if (!fail && lane == 0) mbar_arrive(&sh.q16);
            }

            fail = fail || !wait_warp(sh, &sh.sfull[it & 1], (it >> 1) & 1, T.wait_limit);
            if (!fresh && it >= T.np) fail = fail || !wait_warp(sh, &sh.pv[(it - T.np) & 1], ((it - T.np) >> 1) & 1, T.wait_limit);
            float ks = 0.0f, ve = 0.0f;
            bool okt = false, partial = false;
            float vmax = NEG_INF;
            const uint32_t ts = tl + (it & 1) * T.RN + col0;
            if (!fail) {
                tc_fence_after();
                if (!fresh) {
                    const int s = it % T.stages;
                    const float2 sc = sh.scale[s][tok >> P.page_shift];
                    ks = sc.x;
                    ve = (float)exponent_of(sc.y);
                    const int left = w.rq.len - tile * TT;
                    partial = left < TT;
                    okt = tok < left;
                    if (!okt) ks = 1.0f, ve = 0.0f;
                    status = max(status, sh.status[s]);
                } else {
                    ks = sh.fks[it & 1][tok];
                    ve = sh.fve[it & 1][tok];
                    partial = true;
                    vbad = vbad || sh.vbad[it & 3][0] || sh.vbad[it & 3][1];
                }
            }
            const float inv = exp2_int(min(max(-(int)ve, -126), 127));
            const unsigned long long ks2 = f2_pack(ks, ks), ve2 = f2_pack(ve, ve), inv2 = f2_pack(inv, inv);
            // which columns see this thread's token
            const auto sees = [&](int c) {
                return fresh ? (sh.mask[col0 + c][quad] >> lane & 1u) != 0 : okt;
            };
            // A pass over the tile: weights to shared memory, their sums to l.  The first pass goes by the reference as it
            // stands.  Where that turns out too low the sums are rescaled, this pass's share with them, and a second
            // one repeats the weights; it adds to l only what the first left out because it would have passed fp32's range.
            const auto weights = [&](auto again) {
                const float4* fr = rb ? fr1 : fr0;
                const float4* old = rb ? fr0 : fr1;
#pragma unroll
                for (int ch = 0; ch < HALFR / 16; ++ch) {
                    if (ch >= nch) break;
                    uint32_t s[16], h[8];
                    unsigned long long p2[8];
                    tmem_ld16(ts + ch * 16, s);
                    float top = NEG_INF;
                    unsigned far = 0;  // second pass: elements that the first left out
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float4 f = fr[ch * 8 + j];
                        const unsigned long long x = f2_mul(f2_pack(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])), f2_pack(f.x, f.y));
                        float a, b;
                        f2_unpack(f2_fma(x, ks2, f2_add(ve2, f2_pack(-f.z, -f.w))), a, b);
                        if (again.value && !first) {
                            const float4 o = old[ch * 8 + j];
                            float c, d;
                            f2_unpack(f2_fma(x, ks2, f2_add(ve2, f2_pack(-o.z, -o.w))), c, d);
                            far |= (unsigned)(c > FAR) << (2 * j) | (unsigned)(d > FAR) << (2 * j + 1);
                        }
                        if (partial) {
                            a = sees(ch * 16 + 2 * j) ? a : NEG_INF;
                            b = sees(ch * 16 + 2 * j + 1) ? b : NEG_INF;
                        }
                        top = fmaxf(top, fmaxf(a, b));
                        s[2 * j] = __float_as_uint(a);
                        s[2 * j + 1] = __float_as_uint(b);
                        a = ex2(a);
                        b = ex2(b);
                        p2[j] = f2_pack(a, b);
                        h[j] = pack_half2(a, b);
                    }
                    vmax = fmaxf(vmax, top);
                    const bool all = again.value ? first : !__any_sync(0xffffffffu, top > FAR);
                    if (all) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) l2[ch * 8 + j] = f2_fma(p2[j], inv2, l2[ch * 8 + j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            float a, b;
                            f2_unpack(p2[j], a, b);
                            if (again.value ? !(far >> (2 * j) & 1u) : __uint_as_float(s[2 * j]) > FAR) a = 0.0f;
                            if (again.value ? !(far >> (2 * j + 1) & 1u) : __uint_as_float(s[2 * j + 1]) > FAR) b = 0.0f;
                            l2[ch * 8 + j] = f2_fma(f2_pack(a, b), inv2, l2[ch * 8 + j]);
                        }
                    }
                    const int col = col0 + ch * 16;
                    uint8_t* row = pb + (size_t)(col >> 6) * 16384 + tok * 128;
                    const int unit = (col & 63) >> 3;
                    *reinterpret_cast<uint4*>(row + ((unit ^ (tok & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
                    *reinterpret_cast<uint4*>(row + (((unit + 1) ^ (tok & 7)) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
                }
            };
            // the first tile of a group has no reference yet
            if (!fail && !first) {
                weights(std::false_type{});
                fence_proxy_async_smem();
            }
            if (group_any(bar_id, fail || first || vmax > WINDOW)) {
                if (group_any(bar_id, fail)) {
                    dead = true;
                    break;
                }
                // the columns' maxima over the tile
                const float4* fr = rb ? fr1 : fr0;
                float4* to = rb ? fr0 : fr1;
                for (int ch = 0; ch < nch; ++ch) {
                    uint32_t s[16];
                    tmem_ld16(ts + ch * 16, s);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float F = reinterpret_cast<const float*>(&fr[ch * 8 + (j >> 1)])[j & 1];
                        float x = fmaf(__uint_as_float(s[j]) * F, ks, ve);
                        x = sees(ch * 16 + j) ? x : NEG_INF;
#pragma unroll
                        for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                        if (lane == 0) sh.wmax[g][quad][ch * 16 + j] = x;
                    }
                }
                // O^T of the tile before has to be whole before it is rescaled
                const bool okp = first || wait_warp(sh, &sh.pv[(it - 1) & 1], ((it - 1) >> 1) & 1, T.wait_limit);
                if (group_any(bar_id, !okp)) {
                    dead = true;
                    break;
                }
                if (tok < cw) {
                    float top = sh.wmax[g][0][tok];
#pragma unroll
                    for (int k = 1; k < 4; ++k) top = fmaxf(top, sh.wmax[g][k][tok]);
                    // the reference of a column without a token yet is 0, which its zero sums do not feel
                    const float* f = reinterpret_cast<const float*>(&fr[tok >> 1]);
                    float* n = reinterpret_cast<float*>(&to[tok >> 1]);
                    const float was = f[2 + (tok & 1)];
                    const bool none = first || sh.fac[g][tok] == -1.0f;
                    const bool move = none ? top > NEG_INF : top > was + WINDOW;
                    const float now = move ? top - HEAD : (first ? 0.0f : was);
                    n[tok & 1] = f[tok & 1];
                    n[2 + (tok & 1)] = now;
                    // factor of the sums so far; -1: still no token
                    sh.wmax[g][0][tok] = none ? 0.0f : move ? ex2(was - now) : 1.0f;
                    sh.fac[g][tok] = none && !move ? -1.0f : 0.0f;
                }
                group_sync(bar_id);
                rb ^= 1;
                if (!first) {
                    tc_fence_after();
#pragma unroll
                    for (int ch = 0; ch < HALFR / 16; ++ch) {
                        if (ch >= nch) break;
                        uint32_t o[16];
                        tmem_ld16(t_o + ch * 16, o);
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * sh.wmax[g][0][ch * 16 + j]);
                        tmem_st16(t_o + ch * 16, o);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 f = *reinterpret_cast<const float2*>(&sh.wmax[g][0][ch * 16 + 2 * j]);
                            l2[ch * 8 + j] = f2_mul(l2[ch * 8 + j], f2_pack(f.x, f.y));
                        }
                    }
                }
                weights(std::true_type{});
                fence_proxy_async_smem();
                tc_fence_before();
                group_sync(bar_id);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.sfree[it & 1]);
                mbar_arrive(&sh.pfull[it & 1]);
            }
        }

        // ---- outputs
        if (!dead) {
            const bool okp = wait_warp(sh, &sh.pv[(it - 1) & 1], ((it - 1) >> 1) & 1, T.wait_limit);
            dead = group_any(bar_id, !okp);
        }
        if (dead) status = ROW_TIMEOUT;
        else tc_fence_after();
        float4* const fr = rb ? fr1 : fr0;
        const AttnParams& A = P;
        float* part = A.parts + ((size_t)blockIdx.x * 2 + (w.first && w.tile0 != 0 ? 0 : 1)) * part_floats(T.MR, D);
#pragma unroll
        for (int ch = 0; ch < HALFR / 16; ++ch) {
            if (ch >= nch) break;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float a, b;
                f2_unpack(l2[ch * 8 + (j >> 1)], a, b);
                float x = j & 1 ? b : a;
#pragma unroll
                for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (lane == 0) sh.wmax[g][quad][ch * 16 + j] = x;
            }
        }
        group_sync(bar_id);
        for (int ch = 0; ch < nch; ++ch) {
            uint32_t o[16];
            if (!dead) tmem_ld16(t_o + ch * 16, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int c = ch * 16 + j, col = col0 + c, r = w.rt * T.MR + col;
                if (col >= T.MR || r >= A.R) continue;
                const float l = (sh.wmax[g][0][c] + sh.wmax[g][1][c]) + (sh.wmax[g][2][c] + sh.wmax[g][3][c]);
                const float m = sh.fac[g][c] == -1.0f ? NEG_INF : reinterpret_cast<const float*>(&fr[c >> 1])[2 + (c & 1)];
                const int t = r / A.G, hq = w.h * A.G + r % A.G;
                float x = dead ? 0.0f : __uint_as_float(o[j]);
                if (vbad && tok < D && t < w.rq.rows) {
                    // values that are not finite reach the rows that see them
                    for (int cur = t;;) {
                        const float y = load_elem<DT>(A.vn, w.b * A.vb + cur * A.vt + w.h * A.vh + tok);
                        if (!(fabsf(y) < __int_as_float(0x7f800000))) x += y;
                        if (cur == 0) break;
                        const int p = A.parents ? __ldg(A.parents + (size_t)w.b * (A.T - 1) + cur - 1) : cur - 2;
                        if (p < -1 || p >= cur - 1) break;
                        cur = p + 1;
                    }
                }
                if (w.whole) {
                    const bool live = t < w.rq.rows && l != 0.0f;
                    float y = live ? x / l : 0.0f, lse = live ? (m + log2f(l)) * LN2 : NEG_INF;
                    if (status != ROW_OK) y = lse = __int_as_float(0x7fc00000);
                    const size_t row = ((size_t)w.b * A.T + t) * A.Hq + hq;
                    if (tok < D) {
                        const uint16_t v = DT == DT_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y)) : __half_as_ushort(__float2half_rn(y));
                        reinterpret_cast<uint16_t*>(A.out)[row * D + tok] = v;
                    }
                    if (tok == 0 && A.lse) A.lse[row] = lse;
                } else {
                    if (tok < D) part[(size_t)col * D + tok] = x;
                    if (tok == 0) {
                        part[(size_t)T.MR * D + col] = m;
                        part[(size_t)T.MR * D + T.MR + col] = l;
                    }
                }
            }
        }
        if (threadIdx.x == SMW0 * 32) {
            if (w.whole) {
                if (A.row_status && w.h == 0 && w.rt == 0) A.row_status[w.b] = status;
            } else {
                part[(size_t)T.MR * D + 2 * T.MR] = __int_as_float(status);
                if (w.tile0 == 0) A.joins[blockIdx.x] = {parts_of(at.total, blockIdx.x, at.ctas, w.u + w.rq.n), w.b, w.h, w.rt, w.rq.rows};
            }
        }
        tc_fence_before();
        group_sync(bar_id);
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
        P.joins[blockIdx.x].parts = 0;
        for (int i = 0; i < T.stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 3);  // the products' commit and the two warps that widen the values
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.sfull[i], 1);
            mbar_init(&sh.sfree[i], 8);
            mbar_init(&sh.pfull[i], 8);
            mbar_init(&sh.vfull[i], 2);
            mbar_init(&sh.pv[i], 1);
        }
        mbar_init(&sh.qfull, 8);
        mbar_init(&sh.q16, 8);
        mbar_init(&sh.done, 1);
        sh.fail = 0;
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
        if ((tid & 31) == 0) role_mma<DT, D>(T, sh, at, smem_addr(smem), tmem);
        __syncwarp();
    } else if (w < SMW0) role_values<DT, D>(T, sh, at, smem);
    else role_softmax<DT, D>(T, sh, at, smem, tmem);
    tc_fence_before();
    __syncthreads();
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
    const uint32_t terms = DT == DT_BF16 ? 2 : 3, blocks = (uint32_t)(T.RN + 63) / 64;
    T.p_buf = blocks * 16384;
    T.np = T.nv = blocks == 1 ? 2 : 1;
    T.v_buf = D / 64 * 16384;
    T.o_p = terms * T.RN * D;
    T.o_v = T.o_p + T.np * T.p_buf;
    T.o_stage = T.o_v + T.nv * T.v_buf + (D == 64 ? 16384 : 0);
    const uint32_t stage = 2 * TT * D;
    T.stages = (int)((TC_SMEM - 1024 - T.o_stage) / stage);
    if (T.stages > MAXSTAGES) T.stages = MAXSTAGES;
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
