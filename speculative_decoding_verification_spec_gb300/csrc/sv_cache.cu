// sv_cache.cu -- kv_cache_write and kv_cache_read: quantising key/value rows into the 8-bit paged cache
// and reading them back.
//
// Write.  A block is one page of one key/value head, for the keys and for the values apart.  With A the
// largest magnitude among the rows that the call puts into the block, the scale is the smallest 2^e with
// A <= 448 * 2^e; a block that already holds tokens of the request (its length ends inside the page)
// keeps the larger of that and its old scale, and its earlier codes move to the new one.  A block begun by the
// call ignores whatever scale the page had.  One CTA per block: the rows are read once, into registers,
// reduced to A, scaled (exactly) and rounded.  For a prompt two thirds of the time are the memory's: 200 MB (four of up to 8191
// bf16 tokens, eight heads of 128 channels) in 43 us, 4.6 TB/s, with 78% of the issue slots used, so the magnitudes are folded
// as pairs of 16-bit integers and the codes come two to a conversion.  A round's few rows are bound by the launch and a chain
// of four dependent loads (length, page, rows, scale).
//
// Read.  One 16-byte vector of codes per thread and step, scaled and rounded once to the type asked for.  Bound by the writes:
// 805 MB of bf16 from 255 MB of codes in 213 us, and a fill of the output alone takes 203 (3.96 TB/s, where a copy of as many
// bytes in all moves 6.7).
#include <cuda_bf16.h>

#include <algorithm>

#include "sv_round.cuh"

namespace sv {

namespace {

template <int DT>
struct Elem;
template <>
struct Elem<DT_F32> {
    static constexpr int VEC = 4;
};
template <>
struct Elem<DT_BF16> {
    static constexpr int VEC = 8;
};
template <>
struct Elem<DT_F16> {
    static constexpr int VEC = 8;
};

template <int DT>
__device__ __forceinline__ void widen(const uint4& w, float (&x)[Elem<DT>::VEC])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == DT_F32) {
            x[i] = __uint_as_float(u[i]);
        } else if constexpr (DT == DT_BF16) {
            x[2 * i] = bf16lo(u[i]);
            x[2 * i + 1] = bf16hi(u[i]);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

// Source rows are read 16 bytes at a time where `ALIGNED`, else element by element.
template <int DT, bool ALIGNED>
__device__ __forceinline__ uint4 load16(const void* base, int64_t elem)
{
    constexpr int ES = DT == DT_F32 ? 4 : 2;
    const char* p = reinterpret_cast<const char*>(base) + elem * ES;
    if constexpr (ALIGNED) {
        return ld_stream_v4(p);
    } else {
        uint4 w;
        uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (ES == 4) {
                u[i] = __ldg(reinterpret_cast<const uint32_t*>(p) + i);
            } else {
                const unsigned short* h = reinterpret_cast<const unsigned short*>(p) + 2 * i;
                u[i] = (uint32_t)__ldg(h) | (uint32_t)__ldg(h + 1) << 16;
            }
        }
        return w;
    }
}

// The magnitudes of a vector's elements folded into one word as bit patterns, whose order is the magnitudes' (an infinity and
// NaN above all numbers): 16-bit types keep two maxima side by side.
template <int DT>
__device__ __forceinline__ uint32_t fold_magnitude(uint32_t m, const uint4& w)
{
    if constexpr (DT == DT_F32) {
        constexpr uint32_t A = 0x7fffffffu;
        return max(max(max(m, w.x & A), max(w.y & A, w.z & A)), w.w & A);
    } else {
        constexpr uint32_t A = 0x7fff7fffu;
        return __vmaxu2(__vmaxu2(m, __vmaxu2(w.x & A, w.y & A)), __vmaxu2(w.z & A, w.w & A));
    }
}
// the larger of the folded maxima as a float
template <int DT>
__device__ __forceinline__ float magnitude(uint32_t m)
{
    if constexpr (DT == DT_F32) return __uint_as_float(m);
    const uint32_t h = max(m & 0xffffu, m >> 16);
    return DT == DT_BF16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
}

// two scaled values as codes, `lo` in the low byte, where both are numbers of at most 448
__device__ __forceinline__ uint16_t e4m3x2_plain(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Whether request b's rows can be written, looked at by every CTA of the request alike, so that either
// all of them write or none.  Called by all threads.
__device__ int write_status(const CacheWriteParams& P, int b, int len, int count)
{
    __shared__ int bad;
    const long long room = (long long)P.table_width * P.page;
    int mine = ROW_OK;
    if (len < 0 || count > P.T || (long long)len + count > room ||
        (P.out_nodes && count - 1 > P.nodes_width)) {
        mine = ROW_BAD_LENGTH;
    } else if (count > 0) {
        const int p0 = len / P.page, p1 = (int)(((long long)len + count - 1) / P.page);
        for (int j = p0 + threadIdx.x; j <= p1; j += blockDim.x)
            if ((unsigned)__ldg(P.page_table + (size_t)b * P.table_width + j) >= (unsigned)P.pages) mine = ROW_BAD_PAGE;
        if (P.out_nodes)
            for (int i = threadIdx.x; i < count - 1; i += blockDim.x)
                if ((unsigned)__ldg(P.out_nodes + (size_t)b * P.nodes_width + i) >= (unsigned)(P.T - 1)) mine = max(mine, (int)ROW_BAD_NODE);
    }
    if (!__syncthreads_or(mine != ROW_OK)) return ROW_OK;
    if (threadIdx.x == 0) bad = ROW_OK;
    __syncthreads();
    atomicMax(&bad, mine);
    __syncthreads();
    return bad;
}

// NV: 16-byte source vectors per thread, at most (a page's worth over NT threads, rounded up to a power of two).  LONG: a CTA takes
// several pages; of its own, as the loop costs registers that the kernel for one page has not.
template <int DT, int NV, bool ALIGNED, bool LONG>
__global__ void __launch_bounds__(NT, NV <= 4 ? (LONG ? 4 : 6) : 1) cache_write_kernel(CacheWriteParams P)
{
    constexpr int VEC = Elem<DT>::VEC;
    __shared__ uint32_t red[WARPS];
    const int which = blockIdx.y & 1, h = blockIdx.y >> 1, b = blockIdx.z, t = threadIdx.x;
    const int len = __ldg(P.lens + b);
    const int count = P.accepted_len ? min(max(__ldg(P.accepted_len + b), -1), P.T) + 1 : P.T;
    for (int at_page = blockIdx.x; at_page < P.span; at_page += gridDim.x) {
        if (LONG && at_page != (int)blockIdx.x) __syncthreads();  // `red` has been read
        const int j = len / P.page + at_page;                          // page of the request
        const int first = max((int)(len - (long long)j * P.page), 0);  // slots the request held before
        const long long r0 = (long long)j * P.page + first - len;      // the first row that goes into this page
        const int rows = len < 0 ? 0 : (int)max(0LL, min(min((long long)count, (long long)P.T) - r0, (long long)(P.page - first)));

        // The rows are on their way while the request is looked over: a prompt's CTAs spend their time in that chain of loads.
        // (A node that is out of range is clamped here and refused below.)
        const int vshift = 31 - __clz(P.D / VEC), vpr = 1 << vshift;  // vectors per row
        uint4 x[NV];
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = t + k * NT;
            x[k] = make_uint4(0, 0, 0, 0);
            if (i < rows * vpr) {
                const int at = (int)r0 + (i >> vshift);
                int row = at;
                if (P.out_nodes && at > 0)
                    row = at - 1 < P.nodes_width ? min(max(__ldg(P.out_nodes + (size_t)b * P.nodes_width + at - 1), -1), P.T - 2) + 1 : 0;
                x[k] = load16<DT, ALIGNED>(P.src[which], b * P.sb[which] + row * P.st[which] + h * P.sh[which] + (i & (vpr - 1)) * VEC);
            }
        }
        const int page = rows > 0 && j < P.table_width ? __ldg(P.page_table + (size_t)b * P.table_width + j) : 0;
        if (!LONG || at_page == (int)blockIdx.x) {
            const int status = write_status(P, b, len, count);
            if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) {
                if (P.row_status) P.row_status[b] = status;
                if (P.lens_out) P.lens_out[b] = status == ROW_OK ? len + count : len;
            }
            if (status != ROW_OK) return;
        }
        if (rows <= 0) return;  // and the pages after this one have none
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) top = fold_magnitude<DT>(top, x[k]);
        top = __reduce_max_sync(0xffffffffu, __float_as_uint(magnitude<DT>(top)));
        if ((t & 31) == 0) red[t >> 5] = top;
        float* sp = P.scale[which] + (size_t)page * P.Hkv + h;
        const float old = first > 0 ? *sp : 0.0f;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = max(top, red[w]);
        float amax = __uint_as_float(top);
        const bool plain = amax <= CACHE_MAX_CODE * 0x1p60f;
        if (!plain) {
            // something that no scale holds (or an infinity, or NaN): it becomes NaN and sets no scale
            amax = 0.0f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float f[VEC];
                widen<DT>(x[k], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (fabsf(f[e]) <= CACHE_MAX_CODE * 0x1p60f) amax = fmaxf(amax, fabsf(f[e]));
            }
            amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
            __syncthreads();
            if ((t & 31) == 0) red[t >> 5] = __float_as_uint(amax);
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WARPS; ++w) amax = fmaxf(amax, __uint_as_float(red[w]));
        }
        const int e = cache_scale_exp(amax);
        float s = exp2_int(e);
        float inv = exp2_int(-e);
        uint8_t* dst = P.codes[which] + ((size_t)page * P.Hkv + h) * P.page * P.D;
        if (old >= s) {
            s = old;
            inv = 1.0f / old;
        } else if (first > 0) {
            // the page's earlier codes move to the larger scale: exact but for subnormals
            const float ratio = old * inv;
            for (int i = t; i < first * P.D / 16; i += NT) {
                uint4 w = reinterpret_cast<uint4*>(dst)[i];
                uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t lo = e4m3x2_to_half2((uint16_t)u[k]), hi = e4m3x2_to_half2((uint16_t)(u[k] >> 16));
                    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                    const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                    u[k] = (uint32_t)e4m3x2_from(a.x * ratio, a.y * ratio) |
                           (uint32_t)e4m3x2_from(c.x * ratio, c.y * ratio) << 16;
                }
                reinterpret_cast<uint4*>(dst)[i] = w;
            }
        }
        if (t == 0) *sp = s;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int i = t + k * NT;
            if (i < rows * vpr) {
                float f[VEC];
                widen<DT>(x[k], f);
                uint16_t c[VEC / 2];
#pragma unroll
                for (int q = 0; q < VEC / 2; ++q)
                    c[q] = plain ? e4m3x2_plain(f[2 * q] * inv, f[2 * q + 1] * inv) : e4m3x2_from(f[2 * q] * inv, f[2 * q + 1] * inv);
                uint8_t* o = dst + first * P.D + i * VEC;
                if constexpr (VEC == 8)
                    *reinterpret_cast<uint2*>(o) = make_uint2(c[0] | (uint32_t)c[1] << 16, c[2] | (uint32_t)c[3] << 16);
                else
                    *reinterpret_cast<uint32_t*>(o) = c[0] | (uint32_t)c[1] << 16;
            }
        }
        if (!LONG) break;
    }
}

template <int DT, bool ALIGNED, bool LONG>
cudaError_t write_grid(const CacheWriteParams& P, dim3 grid, cudaStream_t st)
{
    const int vecs = (min(P.page, P.T) * P.D / Elem<DT>::VEC + NT - 1) / NT;
    if (vecs <= 1) cache_write_kernel<DT, 1, ALIGNED, LONG><<<grid, NT, 0, st>>>(P);
    else if (vecs <= 4) cache_write_kernel<DT, 4, ALIGNED, LONG><<<grid, NT, 0, st>>>(P);
    else if (vecs <= 8) cache_write_kernel<DT, 8, ALIGNED, LONG><<<grid, NT, 0, st>>>(P);
    else cache_write_kernel<DT, 16, ALIGNED, LONG><<<grid, NT, 0, st>>>(P);
    return cudaGetLastError();
}

template <int DT, bool ALIGNED>
cudaError_t write_launch(CacheWriteParams& P, cudaStream_t st)
{
    // Every CTA looks at all of its request's page-table entries: with up to SCAN of them (four loads a thread) it takes one page,
    // in a longer request as many more, so that the entries read grow with the tokens and not with their square.  One request of 131072
    // tokens, eight heads of 128 channels: 369 us with pages of 16 and 168 with 64 (740 and 188 with one page a CTA throughout; 461 and
    // 190 with 16 NT, 437 and 244 at 4 NT with three CTAs an SM).
    constexpr int SCAN = 4 * NT;
    P.span = (P.T + P.page - 2) / P.page + 1;  // pages that T rows can touch
    const int per = (P.span + SCAN - 1) / SCAN;
    const dim3 grid((unsigned)((P.span + per - 1) / per), (unsigned)(2 * P.Hkv), (unsigned)P.B);
    return per == 1 ? write_grid<DT, ALIGNED, false>(P, grid, st) : write_grid<DT, ALIGNED, true>(P, grid, st);
}

// ---------------------------------------------------------------- read

template <int DT>
__device__ __forceinline__ void store_codes(void* out, int64_t elem, const uint4& w, float s)
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    float x[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = e4m3x2_to_half2((uint16_t)u[i]), hi = e4m3x2_to_half2((uint16_t)(u[i] >> 16));
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
        const float2 c = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        x[4 * i] = a.x * s;
        x[4 * i + 1] = a.y * s;
        x[4 * i + 2] = c.x * s;
        x[4 * i + 3] = c.y * s;
    }
    if constexpr (DT == DT_F32) {
        float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + elem);
#pragma unroll
        for (int i = 0; i < 4; ++i) __stcs(o + i, make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
    } else {
        uint32_t r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (DT == DT_BF16)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
            else
                asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
        }
        uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + elem);
        __stcs(o, make_uint4(r[0], r[1], r[2], r[3]));
        __stcs(o + 1, make_uint4(r[4], r[5], r[6], r[7]));
    }
}

// A thread keeps one place (16 channels of a head) and steps through tokens, so consecutive threads store consecutive
// vectors and load runs of a head's D bytes, and no index needs a division.
constexpr int RU = 8;  // tokens in flight per thread

template <int DT>
__global__ void __launch_bounds__(NT) cache_read_kernel(CacheReadParams P)
{
    const int which = blockIdx.z, b = blockIdx.y, t = threadIdx.x;
    const int vpt = P.Hkv * P.D / 16;                // places of a token
    const int tpb = max(1, NT / vpt);                // tokens a CTA takes per step
    const int start = P.start ? __ldg(P.start + b) : 0;
    const int len = __ldg(P.lens + b);
    const long long room = (long long)P.table_width * P.page;
    const bool bad_len = start < 0 || len < 0 || len > room;
    const int32_t* table = P.page_table + (size_t)b * P.table_width;
    if (blockIdx.x == 0 && which == 0 && P.row_status) {
        int mine = bad_len ? ROW_BAD_LENGTH : ROW_OK;
        if (!bad_len) {
            const long long stop = min((long long)len, (long long)start + P.max_len);
            for (long long j = start / P.page + (long long)t; j * P.page < stop; j += NT)
                if ((unsigned)__ldg(table + j) >= (unsigned)P.pages) mine = ROW_BAD_PAGE;
        }
        mine = __syncthreads_or(mine == ROW_BAD_PAGE) ? ROW_BAD_PAGE : mine;
        if (t == 0) P.row_status[b] = mine;
    }
    if (t >= tpb * vpt && vpt <= NT) return;
    const float nan = __int_as_float(0x7fc00000);
    const int shift = P.page_shift;
    for (int place = vpt <= NT ? t % vpt : t; place < vpt; place += NT) {
        const int h = place / (P.D / 16), ch = place % (P.D / 16) * 16;
        const uint8_t* codes = P.codes[which] + ((size_t)h << shift) * P.D + ch;
        const float* scale = P.scale[which] + h;
        const long long block = (long long)P.Hkv * P.D << shift;  // codes of a page
        for (long long i0 = (long long)blockIdx.x * tpb * RU + (vpt <= NT ? t / vpt : 0); i0 < P.max_len; i0 += (long long)gridDim.x * tpb * RU) {
            uint4 w[RU];
            float s[RU];
#pragma unroll
            for (int k = 0; k < RU; ++k) {
                const long long i = i0 + k * tpb, tok = start + i;
                w[k] = make_uint4(0, 0, 0, 0);
                s[k] = bad_len ? nan : 0.0f;
                if (i < P.max_len && !bad_len && tok < len) {
                    const int page = __ldg(table + (tok >> shift));
                    if ((unsigned)page < (unsigned)P.pages) {
                        s[k] = __ldg(scale + (size_t)page * P.Hkv);
                        w[k] = ld_stream_v4(codes + page * block + (tok & (P.page - 1)) * P.D);
                    } else {
                        s[k] = nan;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < RU; ++k) {
                const long long i = i0 + k * tpb;
                if (i < P.max_len) store_codes<DT>(P.out[which], (((long long)b * P.max_len + i) * vpt + place) * 16, w[k], s[k]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_cache_write(CacheWriteParams& P, int dtype, cudaStream_t st)
{
    const int vec = dtype == DT_F32 ? 4 : 8;
    bool aligned = true;
    for (int i = 0; i < 2; ++i)
        aligned = aligned && reinterpret_cast<uintptr_t>(P.src[i]) % 16 == 0 && P.sb[i] % vec == 0 &&
                  P.st[i] % vec == 0 && P.sh[i] % vec == 0;
    if (dtype == DT_F32) return aligned ? write_launch<DT_F32, true>(P, st) : write_launch<DT_F32, false>(P, st);
    if (dtype == DT_BF16) return aligned ? write_launch<DT_BF16, true>(P, st) : write_launch<DT_BF16, false>(P, st);
    return aligned ? write_launch<DT_F16, true>(P, st) : write_launch<DT_F16, false>(P, st);
}

cudaError_t launch_cache_read(const CacheReadParams& P, int dtype, int sms, cudaStream_t st)
{
    const int vpt = P.Hkv * P.D / 16, step = std::max(1, NT / vpt) * RU;
    const long long want = (P.max_len + step - 1) / step;
    const long long most = std::max(1LL, 32LL * sms / P.B);  // several waves, so that ragged requests even out
    const dim3 grid((unsigned)std::max(1LL, std::min(want, most)), (unsigned)P.B, 2);
    if (dtype == DT_F32) cache_read_kernel<DT_F32><<<grid, NT, 0, st>>>(P);
    else if (dtype == DT_BF16) cache_read_kernel<DT_BF16><<<grid, NT, 0, st>>>(P);
    else cache_read_kernel<DT_F16><<<grid, NT, 0, st>>>(P);
    return cudaGetLastError();
}

}  // namespace sv
