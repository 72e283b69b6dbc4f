// sv_round.cuh -- parameter blocks and launchers of the calls around the verify step: logit
// processing, the 8-bit paged key/value cache (write, read) and attention over it.
//
// The cache.  A page holds page_size tokens of every key/value head as e4m3 codes,
// [pages, heads, page_size, head_dim], and one fp32 scale per page and head for the keys and one for
// the values.  A scale is a power of two 2^e, e in [-60, 60]: x / scale is then exact, so a code is the
// value rounded once (half a step, 2^-4 of it, and 2^-10 of the scale for the smallest values), and
// raising a page's scale by 2^k moves the earlier codes exactly, but for those that fall among
// e4m3's subnormals.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "sv_common.cuh"

namespace sv {

enum { DT_F16 = 2 };                 // beside DT_F32, DT_BF16
enum { ROW_BAD_PAGE = 9, ROW_BAD_LENGTH = 10, ROW_BAD_NODE = 11 };

constexpr int CACHE_E_MIN = -60, CACHE_E_MAX = 60;  // a scale's exponent
constexpr float CACHE_MAX_CODE = 448.0f;            // the largest e4m3 value

// What a launcher keeps for each device (0: nothing yet): attributes of a kernel belong to the device that was current when they
// were set.  On a device past the last slot it is found anew by every call.
struct PerDevice {
    int slot[65] = {0};
    int& here()
    {
        int dev = 64;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) slot[dev = 64] = 0;
        return slot[dev];
    }
};

// 2^e for a normal result
__host__ __device__ __forceinline__ float exp2_int(int e)
{
#ifdef __CUDA_ARCH__
    return __int_as_float((e + 127) << 23);
#else
    union { uint32_t u; float f; } x;
    x.u = (uint32_t)(e + 127) << 23;
    return x.f;
#endif
}

// the smallest e with amax <= 448 * 2^e, clamped to the cache's range: 448 = 1.75 * 2^8
__device__ __forceinline__ int cache_scale_exp(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    const int x = (int)(u >> 23) - 127;  // amax = f * 2^x (a zero or subnormal gives -127)
    const int e = x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return min(max(e, CACHE_E_MIN), CACHE_E_MAX);
}

// two e4m3 codes (low byte first) as two halfs, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t c)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}
// two floats as e4m3 codes, `lo` in the low byte; nearest, ties to even.  A magnitude above 448 (and an
// infinity) becomes NaN, which the instruction alone would clamp.
__device__ __forceinline__ uint16_t e4m3x2_from(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    if (!(fabsf(lo) <= CACHE_MAX_CODE)) r = (uint16_t)((r & 0xff00u) | 0x7fu);
    if (!(fabsf(hi) <= CACHE_MAX_CODE)) r = (uint16_t)((r & 0x00ffu) | 0x7f00u);
    return r;
}

// ---------------------------------------------------------------- logit processing

constexpr int LOGITS_MAX_NODES = 4096;
constexpr int LOGITS_MAX_BIASES = 16384;

struct LogitsParams {
    const void* logits;
    void* out;
    int64_t in_b, in_r, out_b, out_r;  // strides in elements
    int B, R, V;
    const int32_t* tokens;   // [B, N] or null
    const int32_t* parents;  // [B, N] or null (a chain)
    int N;
    const int32_t* history;  // [B, H] or null
    int H;
    const int32_t* prompt_len;
    const int32_t* history_len;
    const float* repetition;
    const float* presence;
    const float* frequency;
    const int32_t* bias_tokens;  // [B, nb]
    const float* bias_values;
    int nb;
    const uint32_t* allowed;     // [B, R, mwords]
    int mwords;
    int32_t* row_status;
    int chunk, rows;             // vocabulary entries and rows per CTA
};

cudaError_t launch_process_logits(LogitsParams& P, int dtype, int sms, cudaStream_t st);

// ---------------------------------------------------------------- the cache

struct CacheWriteParams {
    const void* src[2];            // keys, values [B, T, Hkv, D]
    int64_t sb[2], st[2], sh[2];   // their strides in elements
    uint8_t* codes[2];
    float* scale[2];
    const int32_t* page_table;     // [B, table_width]
    const int32_t* lens;
    const int32_t* accepted_len;   // nullable: all T rows
    const int32_t* out_nodes;      // [B, nodes_width] or null
    int nodes_width;
    int32_t* lens_out;
    int32_t* row_status;
    int B, T, Hkv, D, page, pages, table_width;
    int span;                      // pages that a request's rows may touch
};

cudaError_t launch_cache_write(CacheWriteParams& P, int dtype, cudaStream_t st);

struct CacheReadParams {
    const uint8_t* codes[2];
    const float* scale[2];
    const int32_t* page_table;
    const int32_t* lens;
    const int32_t* start;          // nullable: 0
    void* out[2];                  // [B, max_len, Hkv, D]
    int32_t* row_status;
    int B, max_len, Hkv, D, page, page_shift, pages, table_width;
};

cudaError_t launch_cache_read(const CacheReadParams& P, int dtype, int sms, cudaStream_t st);

// ---------------------------------------------------------------- attention

constexpr int ATTN_MAX_ROWS = 256;   // rows of a round (T)
constexpr int ATTN_MAX_CTAS = 512;   // CTAs of one launch (few rows; three an SM): the workspace holds two parts for each
constexpr int ATTN_MAX_TC_CTAS = 160;  // and of the kernel for many rows (one an SM)

// a group of rows that starts in one streaming CTA and ends in a later one (parts == 0: none starts there)
struct AttnJoin {
    int parts, b, h, rt, rows;
    int lost0, lost1;  // requests [lost0, lost1) of the CTA are without some of their outputs: a wait ran out
    int pad;
};

struct AttnParams {
    const void* q;                 // [B, T, Hq, D]
    int64_t qb, qt, qh;
    const void* kn;                // [B, T, Hkv, D] or null
    const void* vn;
    int64_t kb, kt, kh, vb, vt, vh;
    const uint8_t* kc;
    const uint8_t* vc;
    const float* ks;
    const float* vs;
    const int32_t* page_table;
    const int32_t* lens;
    const int32_t* parents;        // [B, T-1] or null
    const int32_t* n_rows;         // [B] or null
    void* out;                     // [B, T, Hq, D]
    float* lse;                    // [B, T, Hq] or null
    int32_t* row_status;
    AttnJoin* joins;               // workspace: [CTAs]
    float* parts;                  // workspace: partial results, two slots per CTA
    int B, T, Hq, Hkv, G, D, page, pages, table_width;
    int page_shift;
    int R;                         // T * G rows of a key/value head
    int RT;                        // row tiles
    float scale;
    int wait_limit;                // polls of a wait before it gives up (ROW_TIMEOUT)
};

// polls of a bounded wait (spec_set_wait_limit)
int wait_limit_polls();

size_t attn_workspace_bytes(int rows, int D);  // rows: of a row tile, at most 128
cudaError_t launch_attention(AttnParams& P, int dtype, int sms, cudaStream_t st);

}  // namespace sv
