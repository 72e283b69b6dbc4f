// sv_attn.cu -- verify_attention for few rows: attention of a round's rows over the 8-bit paged cache
// and over the round's own rows.
//
// For row t and query head h, with g the key/value head that h shares and s_j = scale * (q . k_j),
//   o = sum_j p_j v_j,  p_j = exp(s_j - lse),  lse = log sum_j exp(s_j)
// over the committed tokens and the rows of the round that t sees (a chain: 0 .. t; a tree: row 0, the
// ancestors' rows and itself).  The rows of the round are not quantised.
//
// Arithmetic.  An e4m3 code is exact as a half, so products are half x half, summed in fp32.  A row of q is scaled by a
// power of two so that its largest element lies in [2^14, 2^15): a bf16 or half element is then exact as a
// half unless it is 2^-28 of the largest or less, and off by at most 2^-39 of it.  With u_j = log2(e) s_j + e_j, 2^(e_j) the scale of
// v_j's page (a power of two), the kernel keeps a reference m per row, within 2^8 of the running maximum of
// u, and sums p'_j = 2^(u_j - m):
//   o = (sum_j p'_j c_j) / (sum_j p'_j 2^(-e_j)),   c_j the codes of v_j,
// so pages with different scales need no second scaling of the sums.  p' <= 2^15 is rounded to a half for the
// product (half a step, 2^-11: under a bf16 output's own rounding, as much as an fp16 output's; what lies under 2^-14 is off by
// 2^-25 absolute, 2^-32 of the row's largest term); the denominator takes it in fp32.
//
// Schedule.  The work is cut into tiles of 64 tokens; every CTA takes an equal run of the tiles of all (request,
// head, row tile) groups in a row, so ragged lengths balance and one long request spreads over the GPU.  A
// group that one CTA covers is written out directly; otherwise its parts (m, l, o) go to the workspace and
// attn_merge_kernel joins them in a fixed order.  Each of a CTA's four warps streams its own 16 tokens of a
// tile through a private ring of cp.async stages, so the loop has no barrier; the warps join at the end.
//
// What bounds it: a slice is some 500 instructions of one dependent chain (fragments, products, reference, weights, products),
// and the registers leave eight warps an SM to hide it; DRAM is 41% used.  At B = 32, contexts to 8192, four rows a head: 88 us
// for 343 MB at T = 1 (3.9 TB/s, over half of a copy's rate), 95 us at T = 4.  A group's start and its own rows cost latency
// alone: calling the first slices before q is read, and loading the rows of q and of the round together, took 102 to 91 us and
// 122 to 101; the schedule's units for a group's change the rest.
#include "sv_attn.cuh"

namespace sv {

namespace {

constexpr int AW = 4;           // warps per CTA
constexpr int ANT = AW * 32;
constexpr int SLICE = 16;       // tokens of a warp per tile
constexpr int TILE = AW * SLICE;
constexpr int ASTAGES = 4;
constexpr int MT = 1, MR = MT * 16;  // rows: one 16-row tile of the product

__device__ __forceinline__ uint32_t swz_off(int D, int row, int chunk)
{
    // byte offset of 16-byte chunk `chunk` of token `row`: spread so that the 8 (row, chunk) pairs that one
    // phase of a fragment load touches fall into different banks
    if (D == 128) return row * 128 + ((chunk ^ (row & 7)) << 4);
    const int line = row >> 1;
    return line * 128 + (((((row & 1) << 2) | chunk) ^ (((line & 1) << 2) | (line & 2))) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- the streaming kernel

template <int D>
struct RowState {
    float o[MT][D / 8][4];
    float m[MT][2], l[MT][2];
};

// One slice of 16 tokens (two n-tiles of 8 columns) against the CTA's rows.  kfrag(nt, cc, kb) and vfrag(q, vb) give the operand
// pairs of four product steps; u_scale, u_add, l_scale (nt, j): key scale, value exponent and 2^-exponent of column 2 t4 + j of
// n-tile nt; see(mt, hi, nt, j): whether row g (+ 8 hi) of m-tile mt sees that column.
template <int D, class KFrag, class VFrag, class Scale, class Add, class LScale, class See>
__device__ __forceinline__ void slice_step(RowState<D>& S, const uint32_t (&qf)[MT][D / 16][4], const float (&F)[MT][2],
                                           KFrag kfrag, VFrag vfrag, Scale u_scale, Add u_add, LScale l_scale, See see)
{
    float s[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][nt][i] = 0.0f;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int cc = 0; cc < D / 64; ++cc) {
            uint32_t kb[4][2];
            kfrag(nt, cc, kb);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) mma_f16(s[mt][nt], qf[mt][cc * 4 + k], kb[k][0], kb[k][1]);
        }
    }
    uint32_t pf[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
            float u[2][2], top = NEG_INF;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float x = fmaf(s[mt][nt][2 * hi + j], F[mt][hi] * u_scale(nt, j), u_add(nt, j));
                    u[nt][j] = see(mt, hi, nt, j) ? x : NEG_INF;
                    top = fmaxf(top, u[nt][j]);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            float m = S.m[mt][hi];
            // the reference moves only when the maximum has left its 2^8 window, so the sums are rarely rescaled (the difference,
            // not the sum: from |u| = 2^27 on m + 15 rounds to the next float, 16 away, and a weight of 2^16 is no half)
            const bool move = top - m > 15.0f;
            if (__any_sync(0xffffffffu, move)) {
                const float now = move ? top - 7.0f : m;
                const float f = move ? (m == NEG_INF ? 0.0f : ex2(m - now)) : 1.0f;
                S.m[mt][hi] = m = now;
                S.l[mt][hi] *= f;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    S.o[mt][i][2 * hi] *= f;
                    S.o[mt][i][2 * hi + 1] *= f;
                }
            }
            const float ref = m == NEG_INF ? 0.0f : m;
            float p[2][2], l[2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                for (int j = 0; j < 2; ++j) p[nt][j] = ex2(u[nt][j] - ref);
                l[nt] = fmaf(p[nt][0], l_scale(nt, 0), p[nt][1] * l_scale(nt, 1));
            }
            S.l[mt][hi] += l[0] + l[1];  // one rounding a slice beside a large sum, where small weights may be many
            pf[mt][hi] = pack_half2(p[0][0], p[0][1]);
            pf[mt][2 + hi] = pack_half2(p[1][0], p[1][1]);
        }
    }
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {  // four n-tiles (four channels of the thread's run) at a time
        uint32_t vb[4][2];
        vfrag(q, vb);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma_f16(S.o[mt][4 * q + i], pf[mt], vb[i][0], vb[i][1]);
    }
}

// token (row of the slice's n-tile) that column n of an n-tile stands for; with it, the rows that one
// phase of a fragment load reads lie in different banks for keys and values alike
__device__ __forceinline__ int col_token(int n) { return n & 1 ? (n - 1) ^ 5 : n; }

// Resident CTAs: with 128 channels two of 242 registers a thread run 5% faster than three of 168, which spill (104 to 110 us at
// B = 32, T = 1, contexts to 8192, four rows a head).
template <int DT, int D>
__global__ void __launch_bounds__(ANT, D == 64 ? 3 : 2) attn_rows_kernel(AttnParams P)
{
    constexpr int KB = SLICE * D;        // bytes of a slice's keys (or values)
    constexpr int STAGE = 2 * KB;
    extern __shared__ __align__(128) uint8_t ring[];  // [AW][ASTAGES][STAGE]; at a group's end [AW][MR][D] floats
    __shared__ float2 scales[AW][ASTAGES];            // of the stage's page: keys, values
    __shared__ __half sq[MR][D + 8];
    __shared__ float sf[MR], wm[AW][MR], wl[AW][MR];
    __shared__ uint64_t smask[MR];
    __shared__ float fks[AW][SLICE], fve[AW][SLICE];
    __shared__ int sstatus;
    __shared__ Place place;

    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const Place at = find_place<TILE>(P, blockIdx.x, gridDim.x, &place);
    if (tid == 0) P.joins[blockIdx.x] = {};
    launch_dependents();
    if ((int)blockIdx.x >= at.ctas) return;
    long long u = at.total * blockIdx.x / at.ctas;
    const long long u1 = at.total * (blockIdx.x + 1) / at.ctas;
    int b = at.b;
    long long pre = at.pre;
    ReqInfo rq = req_info<TILE>(P, b);
    uint8_t* my = ring + w * ASTAGES * STAGE;
    const uint32_t my_a = smem_addr(my), sc_a = smem_addr(&scales[w][0]);
    int ltok[2];  // this lane's key token of each n-tile
    ltok[0] = col_token(g);
    ltok[1] = 8 + col_token(g);
    uint32_t piece[D / 32];  // where this lane's pieces of a slice go
#pragma unroll
    for (int k = 0; k < D / 32; ++k) piece[k] = swz_off(D, (lane + 32 * k) / (D / 16), (lane + 32 * k) % (D / 16));

    while (u < u1) {
        while (u >= pre + (long long)rq.span * P.Hkv * P.RT) {
            pre += (long long)rq.span * P.Hkv * P.RT;
            rq = req_info<TILE>(P, ++b);
        }
        const long long rem = u - pre;
        const int grp = (int)(rem / rq.span), tile0 = (int)(rem % rq.span);
        if (tile0 >= rq.n) {
            u += rq.span - tile0;
            continue;
        }
        const int h = grp / P.RT, rt = grp % P.RT;
        const int tile1 = (int)min((long long)rq.n, tile0 + (u1 - u));
        const bool whole = tile0 == 0 && tile1 == rq.n;

        // ---- the first slices of the cache, which arrive while q is looked at
        __syncthreads();  // the previous group's use of the shared arrays is over
        const int c0 = min(tile0, rq.ncache), c1 = min(tile1, rq.ncache), nc = c1 - c0;
        const int32_t* table = P.page_table + (size_t)b * P.table_width;
        bool bad_page = false;
        int page_reg = 0;  // lane k holds the page of the slice c0 + 32 i + k
        auto fetch = [&](int i) {
            if (i < nc) {
                const int base = (c0 + i) * TILE + w * SLICE;
                if ((i & 31) == 0) {
                    const long long tk = (long long)(c0 + i + lane) * TILE + w * SLICE;
                    page_reg = tk < rq.len ? __ldg(table + (tk >> P.page_shift)) : 0;
                    if (tk < rq.len && c0 + i + lane < c1 && (unsigned)page_reg >= (unsigned)P.pages) bad_page = true;
                }
                const int page = __shfl_sync(0xffffffffu, page_reg, i & 31);
                if (base < rq.len) {
                    const bool good = (unsigned)page < (unsigned)P.pages;
                    const size_t blk = good ? (size_t)page * P.Hkv + h : 0;
                    const int valid = good ? rq.len - base : 0;
                    // the slice's tokens are contiguous, 16-byte piece by piece
                    const size_t off = (blk * P.page + (good ? (base & (P.page - 1)) : 0)) * D + lane * 16;
                    const uint32_t st = my_a + (i % ASTAGES) * STAGE;
                    if (valid >= SLICE) {
                        const uint8_t *fk = P.kc + off, *fv = P.vc + off;
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            cp_async16(st + piece[k], fk + k * 512, 16);
                            cp_async16(st + KB + piece[k], fv + k * 512, 16);
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            const int bytes = (lane + 32 * k) / (D / 16) < valid ? 16 : 0;  // tokens past the length are filled with zeros
                            const size_t from = bytes ? off + k * 512 : 0;
                            cp_async16(st + piece[k], P.kc + from, bytes);
                            cp_async16(st + KB + piece[k], P.vc + from, bytes);
                        }
                    }
                    if (lane < 2) cp_async4(sc_a + (i % ASTAGES) * 8 + lane * 4, (lane ? P.vs : P.ks) + blk, good ? 4 : 0);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < ASTAGES - 1; ++i) fetch(i);

        // ---- the rows of q: those of a warp are all on their way before the first is needed
        if (tid == 0) sstatus = rq.status;
        float x[MR / AW][D / 32];
#pragma unroll
        for (int j = 0; j < MR / AW; ++j) {
            const int r = rt * MR + w + j * AW, t = r / P.G;
            const bool live = r < P.R && t < rq.rows;
            const int64_t base = live ? (int64_t)b * P.qb + (int64_t)t * P.qt + (int64_t)(h * P.G + r % P.G) * P.qh : 0;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) x[j][k] = live ? load_elem<DT>(P.q, base + lane + 32 * k) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < MR / AW; ++j) {
            const int i = w + j * AW;
            float amax = 0.0f;
            bool fin = true;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                fin = fin && fabsf(x[j][k]) < __int_as_float(0x7f800000);
                amax = fmaxf(amax, fabsf(x[j][k]));
            }
            fin = __all_sync(0xffffffffu, fin);
            amax = redux_max(amax);
            const int e = fin ? min(max(14 - exponent_of(amax), -113), 126) : 0;
            const float mul = exp2_int(e);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) sq[i][lane + 32 * k] = __float2half_rn(x[j][k] * mul);
            // a row of q with a NaN or an infinity has no scores
            if (lane == 0) sf[i] = fin ? P.scale * LOG2E * exp2_int(-e) : __int_as_float(0x7fc00000);
        }
        __syncthreads();
        uint32_t qf[MT][D / 16][4];
        float F[MT][2];
        RowState<D> S;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                F[mt][hi] = sf[mt * 16 + 8 * hi + g];
                S.m[mt][hi] = NEG_INF;
                S.l[mt][hi] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) S.o[mt][i][k] = 0.0f;
            // product step cc * 4 + k takes channels 16 (t4 + 4 cc) + 4 k .. + 3 of this lane's rows
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                    const uint2 v = *reinterpret_cast<const uint2*>(&sq[mt * 16 + 8 * hi + g][16 * (t4 + 4 * (c >> 2)) + 4 * (c & 3)]);
                    qf[mt][c][hi] = v.x;
                    qf[mt][c][2 + hi] = v.y;
                }
        }

        // ---- the cache
        for (int i = 0; i < nc; ++i) {
            asm volatile("cp.async.wait_group %0;" :: "n"(ASTAGES - 2) : "memory");
            __syncwarp();  // every lane's copies of stage i have landed, and stage i - 1 is read to the end
            fetch(i + ASTAGES - 1);
            const int base = (c0 + i) * TILE + w * SLICE;
            if (base >= rq.len) continue;
            const uint8_t* st = my + (i % ASTAGES) * STAGE;
            const float2 sc = scales[w][i % ASTAGES];
            const float ve = (float)exponent_of(sc.y);
            const float inv = exp2_int(min(max(-exponent_of(sc.y), -126), 127));
            const int left = rq.len - base;
            auto kfrag = [&](int nt, int cc, uint32_t (&kb)[4][2]) {
                const uint4 x = *reinterpret_cast<const uint4*>(st + swz_off(D, ltok[nt], t4 + 4 * cc));
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    kb[k][0] = e4m3x2_to_half2((uint16_t)xs[k]);
                    kb[k][1] = e4m3x2_to_half2((uint16_t)(xs[k] >> 16));
                }
            };
            // channels (D / 8) g .. of the four tokens that this lane's columns 2 t4, 2 t4 + 1 of both n-tiles name
            constexpr int VW = D / 32;  // 32-bit words per token
            uint32_t vw[4][VW];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = (k >> 1) * 8 + (k & 1 ? (2 * t4) ^ 5 : 2 * t4);
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(st + KB + swz_off(D, row, g));
                    vw[k][0] = x.x; vw[k][1] = x.y; vw[k][2] = x.z; vw[k][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(st + KB + swz_off(D, row, g >> 1) + (g & 1) * 8);
                    vw[k][0] = x.x; vw[k][1] = x.y;
                }
            }
            auto vfrag = [&](int q, uint32_t (&vb)[4][2]) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t a = vw[2 * half][q], c = vw[2 * half + 1][q];
                    const uint32_t lo = __byte_perm(a, c, 0x5140), hi = __byte_perm(a, c, 0x7362);
                    vb[0][half] = e4m3x2_to_half2((uint16_t)lo);
                    vb[1][half] = e4m3x2_to_half2((uint16_t)(lo >> 16));
                    vb[2][half] = e4m3x2_to_half2((uint16_t)hi);
                    vb[3][half] = e4m3x2_to_half2((uint16_t)(hi >> 16));
                }
            };
            auto uscale = [&](int, int) { return sc.x; };
            auto uadd = [&](int, int) { return ve; };
            auto lscale = [&](int, int) { return inv; };
            if (left >= SLICE)
                slice_step<D>(S, qf, F, kfrag, vfrag, uscale, uadd, lscale, [](int, int, int, int) { return true; });
            else
                slice_step<D>(S, qf, F, kfrag, vfrag, uscale, uadd, lscale, [&](int, int, int nt, int j) {
                    return nt * 8 + (j ? (2 * t4) ^ 5 : 2 * t4) < left;
                });
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (bad_page) sstatus = ROW_BAD_PAGE;

        // ---- the round's own rows
        for (int tile = max(tile0, rq.ncache); P.kn && tile < tile1; ++tile) {
            const int j0 = (tile - rq.ncache) * TILE;
            __syncthreads();
            for (int i = tid; i < MR; i += ANT) {
                // bit j - j0: row t sees row j
                const int t = (rt * MR + i) / P.G;
                uint64_t bits = 0;
                if (t < rq.rows) {
                    if (!P.parents) {
                        const int n = t + 1 - j0;
                        bits = n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
                    } else {
                        int cur = t;
                        for (;;) {
                            if ((unsigned)(cur - j0) < 64u) bits |= 1ull << (cur - j0);
                            if (cur == 0) break;
                            const int p = __ldg(P.parents + (size_t)b * (P.T - 1) + cur - 1);
                            if (p < -1 || p >= cur - 1) break;  // reported below; the walk always ends
                            cur = p + 1;
                        }
                    }
                }
                smask[i] = bits;
            }
            if (P.parents)
                for (int i = tid; i < rq.rows - 1; i += ANT) {
                    const int p = __ldg(P.parents + (size_t)b * (P.T - 1) + i);
                    if (p < -1 || p >= i) sstatus = ROW_BAD_PARENT;
                }
            __syncthreads();
            const int jw = j0 + w * SLICE;
            if (jw >= rq.rows) continue;
            // 16 rows as halves, each scaled by a power of two as q is: keys [16][D], then values
            __half* fk = reinterpret_cast<__half*>(my);
            __half* fv = fk + SLICE * D;
            unsigned bad = 0;  // rows of the slice whose values hold a NaN or an infinity
            constexpr int FU = 4;  // rows in flight
            const int live = min(rq.rows - jw, SLICE);
            for (int i = lane; i < 2 * (SLICE - live) * D / 8; i += 32) {
                const int n = (SLICE - live) * D / 8;
                reinterpret_cast<uint4*>((i < n ? fk : fv) + live * D)[i < n ? i : i - n] = make_uint4(0, 0, 0, 0);
            }
            if (lane >= live && lane < SLICE) fks[w][lane] = 1.0f, fve[w][lane] = 0.0f;
#pragma unroll 1
            for (int i0 = 0; i0 < live; i0 += FU) {
                float x[FU][2][D / 32];
#pragma unroll
                for (int f = 0; f < FU; ++f) {
                    const int64_t j = jw + i0 + f;
#pragma unroll
                    for (int k = 0; k < D / 32; ++k) {
                        x[f][0][k] = i0 + f < live ? load_elem<DT>(P.kn, b * P.kb + j * P.kt + h * P.kh + lane + 32 * k) : 0.0f;
                        x[f][1][k] = i0 + f < live ? load_elem<DT>(P.vn, b * P.vb + j * P.vt + h * P.vh + lane + 32 * k) : 0.0f;
                    }
                }
#pragma unroll
                for (int f = 0; f < FU; ++f) {
                    const int i = i0 + f;
                    if (i >= live) break;
#pragma unroll
                    for (int which = 0; which < 2; ++which) {
                        float amax = 0.0f;
                        bool fin = true;
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            if (fabsf(x[f][which][k]) < __int_as_float(0x7f800000)) amax = fmaxf(amax, fabsf(x[f][which][k]));
                            else fin = false;
                        }
                        fin = __all_sync(0xffffffffu, fin);
                        amax = redux_max(amax);
                        const int e = min(max(exponent_of(amax), CACHE_E_MIN), 126) - 14;
                        const float mul = exp2_int(-e);
                        if (which && !fin) bad |= 1u << i;
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            // a value that only some rows see must not meet the others' zero weights as NaN
                            const bool drop = which && !(fabsf(x[f][which][k]) < __int_as_float(0x7f800000));
                            (which ? fv : fk)[i * D + lane + 32 * k] = __float2half_rn(drop ? 0.0f : x[f][which][k] * mul);
                        }
                        if (lane == 0) {
                            if (which) fve[w][i] = (float)e;
                            else fks[w][i] = fin ? exp2_int(e) : __int_as_float(0x7fc00000);  // a key that is not finite: NaN
                        }
                    }
                }
            }
            __syncwarp();
            auto ctok = [&](int nt, int j) { return nt * 8 + (j ? (2 * t4) ^ 5 : 2 * t4); };
            auto kfrag = [&](int nt, int cc, uint32_t (&kb)[4][2]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint2 v = *reinterpret_cast<const uint2*>(&fk[ltok[nt] * D + 16 * (t4 + 4 * cc) + 4 * k]);
                    kb[k][0] = v.x;
                    kb[k][1] = v.y;
                }
            };
            auto vfrag = [&](int q, uint32_t (&vb)[4][2]) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const int ch = (D / 8) * g + 4 * q + i;
                        vb[i][nt] = (uint32_t)__half_as_ushort(fv[ctok(nt, 0) * D + ch]) |
                                    (uint32_t)__half_as_ushort(fv[ctok(nt, 1) * D + ch]) << 16;
                    }
            };
            auto vis = [&](int mt, int hi, int nt, int j) {
                return (smask[mt * 16 + 8 * hi + g] >> (w * SLICE + ctok(nt, j)) & 1ull) != 0;
            };
            slice_step<D>(S, qf, F, kfrag, vfrag, [&](int nt, int j) { return fks[w][ctok(nt, j)]; },
                              [&](int nt, int j) { return fve[w][ctok(nt, j)]; },
                              [&](int nt, int j) { return exp2_int(-(int)fve[w][ctok(nt, j)]); }, vis);
            // values that are not finite reach the rows that see them
            for (unsigned left = bad; left; left &= left - 1) {
                const int i = __ffs(left) - 1, j = jw + i;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi) {
                        if (!(smask[mt * 16 + 8 * hi + g] >> (w * SLICE + i) & 1ull)) continue;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int ch = (D / 8) * (2 * t4 + k) + n;
                                const float x = load_elem<DT>(P.vn, b * P.vb + j * P.vt + h * P.vh + ch);
                                if (!(fabsf(x) < __int_as_float(0x7f800000))) S.o[mt][n][2 * hi + k] += x;
                            }
                    }
            }
            __syncwarp();
        }

        // ---- join the warps: o to shared memory, m and l beside it
        __syncwarp();
        float* so = reinterpret_cast<float*>(my);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hi = 0; hi < 2; ++hi) {
                float l = S.l[mt][hi];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                const int row = mt * 16 + 8 * hi + g;
                if (t4 == 0) {
                    wm[w][row] = S.m[mt][hi];
                    wl[w][row] = l;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int n = 0; n < D / 8; n += 4)
                        *reinterpret_cast<float4*>(&so[row * D + (D / 8) * (2 * t4 + k) + n]) =
                            make_float4(S.o[mt][n][2 * hi + k], S.o[mt][n + 1][2 * hi + k], S.o[mt][n + 2][2 * hi + k], S.o[mt][n + 3][2 * hi + k]);
            }
        __syncthreads();
        const int status = sstatus;
        float* part = P.parts + ((size_t)blockIdx.x * 2 + (tile0 != 0 ? 0 : 1)) * part_floats(MR, D);
        for (int i = tid; i < MR * (D / 4); i += ANT) {
            const int row = i / (D / 4), d = i % (D / 4) * 4;
            const int r = rt * MR + row;
            if (r >= P.R) break;
            float m = NEG_INF;
#pragma unroll
            for (int k = 0; k < AW; ++k) m = fmaxf(m, wm[k][row]);
            float l = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < AW; ++k) {
                // a warp that saw no token has m = -inf and sums of zero (or NaN, which stays)
                const float f = wm[k][row] == NEG_INF ? 1.0f : ex2(wm[k][row] - m);
                const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring + k * ASTAGES * STAGE) + row * D + d);
                l = fmaf(wl[k][row], f, l);
                o.x = fmaf(x.x, f, o.x);
                o.y = fmaf(x.y, f, o.y);
                o.z = fmaf(x.z, f, o.z);
                o.w = fmaf(x.w, f, o.w);
            }
            if (whole) {
                finish_row4<DT>(P, b, h, r, rq.rows, status, d, o, m, l);
            } else {
                *reinterpret_cast<float4*>(&part[row * D + d]) = o;
                if (d == 0) {
                    part[MR * D + row] = m;
                    part[MR * D + MR + row] = l;
                }
            }
        }
        if (tid == 0) {
            begin_status(P, b, h, rt, tile0, status);
            if (!whole) {
                part[MR * D + 2 * MR] = __int_as_float(status);
                // the group's first part: tell the joining kernel how far the group reaches
                if (tile0 == 0) P.joins[blockIdx.x] = {parts_of(at.total, blockIdx.x, at.ctas, u + rq.n), b, h, rt, rq.rows};
            }
        }
        u += tile1 - tile0;
    }
}

// Joins the parts of the group that starts in streaming CTA blockIdx.x and ends in a later one: part 0 is that
// CTA's second slot, part k the first slot of CTA blockIdx.x + k.  Four warps share a row: each takes
// every fourth part.
template <int DT, int D>
__global__ void __launch_bounds__(256) attn_merge_kernel(AttnParams P, int MR)
{
    __shared__ float4 so[8][32];
    __shared__ float sm[8], sl[8];
    __shared__ int ss[8];
    depend_wait();
    const AttnJoin J = P.joins[blockIdx.x];
    if (blockIdx.y == 0)
        for (int b = max(J.lost0, 0) + threadIdx.x; b < min(J.lost1, P.B); b += blockDim.x) raise_status(P, b, ROW_TIMEOUT);
    if (J.parts == 0) return;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, q = w & 3;
    const size_t pf = part_floats(MR, D);
    for (int row0 = blockIdx.y * 2; row0 < MR; row0 += gridDim.y * 2) {
        const int row = row0 + (w >> 2), r = J.rt * MR + row;
        const bool have = row < MR && r < P.R;
        float m = NEG_INF, l = 0.0f;
        int status = ROW_OK;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (have) {
            const auto part_of = [&](int k) { return P.parts + ((size_t)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * pf; };
            // the largest reference of this warp's parts first, so that the sums need no rescaling
            for (int k = q + 4 * lane; k < J.parts; k += 128) {
                const float* part = part_of(k);
                m = fmaxf(m, part[(size_t)MR * D + row]);
                status = max(status, __float_as_int(part[(size_t)MR * D + 2 * MR]));
                const AttnJoin& c = P.joins[blockIdx.x + k];
                if (c.lost0 <= J.b && J.b < c.lost1) status = max(status, (int)ROW_TIMEOUT);
            }
#pragma unroll
            for (int s = 16; s; s >>= 1) {
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
                status = max(status, __shfl_xor_sync(0xffffffffu, status, s));
            }
            constexpr int JU = 8;
            for (int k0 = q; k0 < J.parts; k0 += 4 * JU) {
                float4 x[JU];
                float mk[JU], lk[JU];
#pragma unroll
                for (int j = 0; j < JU; ++j) {
                    const int k = k0 + 4 * j;
                    mk[j] = NEG_INF;
                    lk[j] = 0.0f;
                    x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (k < J.parts) {
                        const float* part = part_of(k);
                        mk[j] = part[(size_t)MR * D + row];
                        lk[j] = part[(size_t)MR * D + MR + row];
                        if (lane < D / 4) x[j] = *reinterpret_cast<const float4*>(&part[(size_t)row * D + lane * 4]);
                    }
                }
#pragma unroll
                for (int j = 0; j < JU; ++j) {
                    const float f = mk[j] == NEG_INF ? 1.0f : ex2(mk[j] - m);  // without a token: zeros, or NaN, which stays
                    l = fmaf(lk[j], f, l);
                    o.x = fmaf(x[j].x, f, o.x);
                    o.y = fmaf(x[j].y, f, o.y);
                    o.z = fmaf(x[j].z, f, o.z);
                    o.w = fmaf(x[j].w, f, o.w);
                }
            }
        }
        so[w][lane] = o;
        if (lane == 0) {
            sm[w] = m;
            sl[w] = l;
            ss[w] = status;
        }
        __syncthreads();
        if (q == 0 && have) {
            float M = NEG_INF, L = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                M = fmaxf(M, sm[w + k]);
                status = max(status, ss[w + k]);
            }
            float4 O = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float f = sm[w + k] == NEG_INF ? 1.0f : ex2(sm[w + k] - M);
                const float4 x = so[w + k][lane];
                L = fmaf(sl[w + k], f, L);
                O.x = fmaf(x.x, f, O.x);
                O.y = fmaf(x.y, f, O.y);
                O.z = fmaf(x.z, f, O.z);
                O.w = fmaf(x.w, f, O.w);
            }
            if (lane < D / 4) finish_row4<DT>(P, J.b, J.h, r, J.rows, status, lane * 4, O, M, L);
            if (row == 0 && lane == 0) raise_status(P, J.b, status);
        }
        __syncthreads();
    }
}

// the joining kernel, launched so that its CTAs are in place when the streaming kernel ends
template <int DT, int D>
cudaError_t launch_merge(const AttnParams& P, int ctas, int MR, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)((MR + 1) / 2));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_merge_kernel<DT, D>, P, MR);
}

template <int DT, int D>
cudaError_t launch_rows(AttnParams& P, int sms, cudaStream_t st)
{
    P.RT = 1;
    const size_t smem = (size_t)AW * ASTAGES * 2 * SLICE * D;
    static_assert((size_t)AW * ASTAGES * 2 * SLICE * D >= (size_t)AW * MR * D * 4, "the ring holds the warps' sums");
    auto* k = attn_rows_kernel<DT, D>;
    static PerDevice kept;
    int& per_sm = kept.here();
    if (per_sm == 0) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k, ANT, smem);
        if (e != cudaSuccess) return e;
        per_sm = n < 1 ? 1 : n;
    }
    int ctas = per_sm * sms;
    if (ctas > ATTN_MAX_CTAS) ctas = ATTN_MAX_CTAS;
    k<<<ctas, ANT, smem, st>>>(P);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_attn_merge(P, DT, ctas, MR, st);
}

template <int DT, int D>
cudaError_t launch_dim(AttnParams& P, int sms, cudaStream_t st)
{
    // Rows that fill one 16-row tile of mma.sync stay below the memory's pace there.  More rows take the tensor cores' own path:
    // with 24 rows (B = 32, T = 6, contexts to 8192) two such tiles took 181 us where it took 139 (now 132); with 20 or 24 rows of one short
    // context both are launch and latency.  With 8 to 16 rows it cannot pay, its tiles cost the same from one row to 48.
    return P.R <= MR ? launch_rows<DT, D>(P, sms, st) : launch_attention_tc(P, DT, sms, st);
}

}  // namespace

cudaError_t launch_attn_merge(const AttnParams& P, int dtype, int ctas, int MR, cudaStream_t st)
{
    if (dtype == DT_BF16)
        return P.D == 128 ? launch_merge<DT_BF16, 128>(P, ctas, MR, st) : launch_merge<DT_BF16, 64>(P, ctas, MR, st);
    return P.D == 128 ? launch_merge<DT_F16, 128>(P, ctas, MR, st) : launch_merge<DT_F16, 64>(P, ctas, MR, st);
}

// Never less for more rows, so that a workspace for the longest round serves the shorter ones.
size_t attn_workspace_bytes(int rows, int D)
{
    const size_t few = ATTN_MAX_CTAS * part_floats(MR, D), many = rows > MR ? ATTN_MAX_TC_CTAS * part_floats(rows, D) : 0;
    return ATTN_MAX_CTAS * sizeof(AttnJoin) + 2 * (few > many ? few : many) * sizeof(float);
}

cudaError_t launch_attention(AttnParams& P, int dtype, int sms, cudaStream_t st)
{
    if (dtype == DT_BF16) return P.D == 128 ? launch_dim<DT_BF16, 128>(P, sms, st) : launch_dim<DT_BF16, 64>(P, sms, st);
    return P.D == 128 ? launch_dim<DT_F16, 128>(P, sms, st) : launch_dim<DT_F16, 64>(P, sms, st);
}

}  // namespace sv
