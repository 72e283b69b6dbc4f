// sv_attn.cuh -- what the two attention kernels share: the schedule, the parts of split groups and the outputs.
#pragma once

#include "sv_round.cuh"

namespace sv {

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

// a part of a group of MR rows in the workspace: o [MR][D], then m, l [MR], then the status; a multiple of 16 bytes, as o
// is read in vectors
__host__ __device__ constexpr size_t part_floats(int MR, int D) { return ((size_t)MR * D + 2 * MR + 1 + 3) / 4 * 4; }

// The status of a request: the CTA that begins its first group (head 0, row tile 0) writes what it knows, and attn_merge_kernel,
// which runs after all of them, raises it where a joined group or a wait that ran out (AttnJoin::lost0) says more.
__device__ __forceinline__ void begin_status(const AttnParams& P, int b, int h, int rt, int tile0, int status)
{
    if (P.row_status && h == 0 && rt == 0 && tile0 == 0) P.row_status[b] = status;
}
__device__ __forceinline__ void raise_status(const AttnParams& P, int b, int status)
{
    if (P.row_status && status != ROW_OK) atomicMax(P.row_status + b, status);
}

// parts of the group that starts in CTA c and ends at unit `end`: CTA k holds units [total k / ctas, total (k + 1) / ctas)
__device__ __forceinline__ int parts_of(long long total, int c, int ctas, long long end)
{
    int last = c;
    while (total * (last + 1) / ctas < end) ++last;
    return last - c + 1;
}

__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void depend_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i)
{
    if constexpr (DT == DT_BF16)
        return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p) + i) << 16);
    else
        return __half2float(__ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(p) + i)));
}

__device__ __forceinline__ float redux_max(float x)
{
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// the exponent x of a finite a >= 0, a = f * 2^x with f in [1, 2), -127 below the normal range
__device__ __forceinline__ int exponent_of(float a) { return (int)(__float_as_uint(a) >> 23) - 127; }

// ---------------------------------------------------------------- schedule

// The units that a group takes beside its tiles, at its end: what its own rows, its q, its first reference and its outputs cost
// beside a tile, so that a CTA that ends one group and begins the next gets fewer tiles.  A run that starts in them begins
// with the next group.  In tiles of 128 tokens on the many-rows path (B = 32: 65 rows a round 402, 376 and 376 us with 3, 6 and
// 10 units; 48 rows a head 176, 171 and 175 us; none: 447 and 183), of 64 on the few-rows path (T = 4: 101, 97, 95 and 95 us with
// none, 6, 8 and 10).
template <int TILE>
constexpr int REST = TILE == 128 ? 6 : 8;

struct ReqInfo {
    int len;     // committed tokens (0 when the length is bad)
    int rows;    // live rows
    int ncache;  // tiles of the cache
    int n;       // tiles of a group, at least one: a group without tokens still writes its outputs
    int span;    // its units
    int status;
};

template <int TILE>
__device__ __forceinline__ ReqInfo req_info(const AttnParams& P, int b)
{
    ReqInfo q;
    q.len = __ldg(P.lens + b);
    q.rows = P.n_rows ? min(max(__ldg(P.n_rows + b), 0), P.T) : P.T;
    q.status = ROW_OK;
    if (q.len < 0 || (long long)q.len > (long long)P.table_width * P.page) {
        q.len = 0;
        q.status = ROW_BAD_LENGTH;
    }
    q.ncache = (q.len + TILE - 1) / TILE;
    const int fresh = P.kn ? (q.rows + TILE - 1) / TILE : 0;
    q.n = max(1, q.ncache + fresh);
    q.span = q.n + REST<TILE>;
    return q;
}

// total units of all groups, and the request that unit `u0(total)` falls into; every thread of the CTA calls
// it, warp 0 works
struct Place {
    long long total, pre;  // pre: units of the requests before b
    int b, ctas;           // CTAs that work: no more than there are units
};

template <int TILE>
__device__ Place find_place(const AttnParams& P, int cta, int ctas, Place* sh)
{
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const long long per = (long long)P.Hkv * P.RT;
        long long total = 0;
        for (int b0 = 0; b0 < P.B; b0 += 32) {
            long long v = b0 + lane < P.B ? req_info<TILE>(P, b0 + lane).span * per : 0;
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            total += v;
        }
        if (total < ctas) ctas = (int)total;
        const long long u0 = cta < ctas ? total * cta / ctas : total;
        long long pre = 0;
        int found = P.B;
        for (int b0 = 0; b0 < P.B; b0 += 32) {
            long long v = b0 + lane < P.B ? req_info<TILE>(P, b0 + lane).span * per : 0, s = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += x;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, u0 < pre + s);
            if (hit) {
                const int l = __ffs(hit) - 1;
                pre += __shfl_sync(0xffffffffu, s - v, l);
                found = b0 + l;
                break;
            }
            pre += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) {
            sh->total = total;
            sh->pre = pre;
            sh->b = found;
            sh->ctas = ctas;
        }
    }
    __syncthreads();
    return *sh;
}

// ---------------------------------------------------------------- outputs of a row

template <int DT>
__device__ __forceinline__ void store_out4(const AttnParams& P, int b, int t, int hq, int d, float4 o)
{
    uint32_t lo, hi;
    if constexpr (DT == DT_BF16) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(o.y), "f"(o.x));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(o.w), "f"(o.z));
    } else {
        lo = pack_half2(o.x, o.y);
        hi = pack_half2(o.z, o.w);
    }
    uint16_t* p = reinterpret_cast<uint16_t*>(P.out) + (((size_t)b * P.T + t) * P.Hq + hq) * P.D + d;
    *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
}

// o = O / l and lse of row r of (b, h); rows past the live ones, and rows that see nothing, give 0 and -inf
template <int DT>
__device__ __forceinline__ void finish_row4(const AttnParams& P, int b, int h, int r, int rows, int status, int d,
                                            float4 O, float m, float l)
{
    const int t = r / P.G, hq = h * P.G + r % P.G;
    const bool live = t < rows && l != 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float lse = NEG_INF;
    if (live) {
        o = make_float4(O.x / l, O.y / l, O.z / l, O.w / l);
        lse = (m + log2f(l)) * LN2;
    }
    if (status != ROW_OK) {
        lse = __int_as_float(0x7fc00000);
        o = make_float4(lse, lse, lse, lse);
    }
    store_out4<DT>(P, b, t, hq, d, o);
    if (d == 0 && P.lse) P.lse[((size_t)b * P.T + t) * P.Hq + hq] = lse;
}

// joins the parts that `ctas` streaming CTAs left (sv_attn.cu)
cudaError_t launch_attn_merge(const AttnParams& P, int dtype, int ctas, int MR, cudaStream_t st);

// verify_attention for many rows, on the tensor cores (sv_attn_tc.cu)
cudaError_t launch_attention_tc(AttnParams& P, int dtype, int sms, cudaStream_t st);

}  // namespace sv
