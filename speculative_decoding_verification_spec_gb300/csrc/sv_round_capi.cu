// sv_round_capi.cu -- the C ABI of the calls around the verify step (include/spec_verify.h): host-side
// validation and launches.  No allocation, no host synchronisation.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/spec_verify.h"
#include "sv_round.cuh"

namespace sv {

static int round_sm_count()
{
    static PerDevice cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    int& n = cache.here();
    if (n == 0 && (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)) n = 152;
    return n;
}

static bool on(const void* p, size_t a) { return p && reinterpret_cast<uintptr_t>(p) % a == 0; }
static bool on_or_null(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
static size_t dtype_size(spec_dtype d) { return d == SPEC_F32 ? 4 : 2; }

static int page_shift_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// what the three cache calls share
static bool cache_ok(const void* kc, const void* vc, const float* ks, const float* vs, const int32_t* table,
                     const int32_t* lens, int pages, int table_width, int Hkv, int page, int D)
{
    if (Hkv < 1 || Hkv > 4096 || pages < 1 || table_width < 1) return false;
    if (page != 16 && page != 32 && page != 64 && page != 128) return false;
    if (D != 64 && D != 128) return false;
    if ((long long)table_width * page > (1LL << 30)) return false;
    return on(kc, 16) && on(vc, 16) && on(ks, 4) && on(vs, 4) && on(table, 4) && on(lens, 4);
}

}  // namespace sv

using namespace sv;

extern "C" {

spec_status process_logits(const void* logits, void* out, spec_dtype dtype, int B, int R, int V,
                           const int64_t* in_strides, const int64_t* out_strides, const int32_t* tokens,
                           const int32_t* parents, int N, const int32_t* history, int H,
                           const int32_t* prompt_len, const int32_t* history_len, const float* repetition,
                           const float* presence, const float* frequency, const int32_t* bias_tokens,
                           const float* bias_values, int nb, const uint32_t* allowed, int32_t* row_status,
                           void* stream)
{
    if (B < 0 || R < 1 || V < 1 || N < 0 || H < 0 || nb < 0) return SPEC_ERR_INVALID_ARG;
    if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
    if (B > 65535 || N > LOGITS_MAX_NODES || R > N + 1 || H > (1 << 28) || nb > LOGITS_MAX_BIASES) return SPEC_ERR_INVALID_ARG;
    if (V > (1 << 30)) return SPEC_ERR_INVALID_ARG;
    if (B == 0) return SPEC_OK;
    const size_t es = dtype_size(dtype);
    if (!on(logits, es) || !on(out, es)) return SPEC_ERR_INVALID_ARG;
    if ((N > 0 && !on(tokens, 4)) || !on_or_null(parents, 4)) return SPEC_ERR_INVALID_ARG;
    if (H > 0 && !on(history, 4)) return SPEC_ERR_INVALID_ARG;
    if (nb > 0 && (!on(bias_tokens, 4) || !on(bias_values, 4))) return SPEC_ERR_INVALID_ARG;
    const void* opt[] = {prompt_len, history_len, repetition, presence, frequency, allowed, row_status};
    for (const void* p : opt)
        if (!on_or_null(p, 4)) return SPEC_ERR_INVALID_ARG;

    LogitsParams P;
    std::memset(&P, 0, sizeof P);
    P.logits = logits;
    P.out = out;
    P.in_b = in_strides ? in_strides[0] : (int64_t)R * V;
    P.in_r = in_strides ? in_strides[1] : V;
    P.out_b = out_strides ? out_strides[0] : (int64_t)R * V;
    P.out_r = out_strides ? out_strides[1] : V;
    if (P.in_b < 0 || P.in_r < 0 || P.out_b < 0 || P.out_r < 0) return SPEC_ERR_INVALID_ARG;
    // rows of the output must not overlap
    if ((R > 1 && P.out_r < V) || (B > 1 && P.out_b < (int64_t)(R - 1) * P.out_r + V)) return SPEC_ERR_INVALID_ARG;
    // in place: the same rows
    if (logits == out && ((R > 1 && P.in_r != P.out_r) || (B > 1 && P.in_b != P.out_b))) return SPEC_ERR_INVALID_ARG;
    P.B = B;
    P.R = R;
    P.V = V;
    P.tokens = tokens;
    P.parents = N > 0 ? parents : nullptr;
    P.N = N;
    P.history = H > 0 ? history : nullptr;
    P.H = H;
    P.prompt_len = prompt_len;
    P.history_len = history_len;
    P.repetition = repetition;
    P.presence = presence;
    P.frequency = frequency;
    P.bias_tokens = bias_tokens;
    P.bias_values = bias_values;
    P.nb = nb;
    P.allowed = allowed;
    P.mwords = (V + 31) / 32;
    P.row_status = row_status;
    const cudaError_t e = launch_process_logits(P, dtype == SPEC_BF16 ? DT_BF16 : DT_F32, round_sm_count(),
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status kv_cache_write(const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides,
                           spec_dtype dtype, int B, int T, int Hkv, int D, void* k_cache, void* v_cache,
                           float* k_scale, float* v_scale, int pages, int page_size, const int32_t* page_table,
                           int table_width, const int32_t* lens, const int32_t* accepted_len,
                           const int32_t* out_nodes, int nodes_width, int32_t* lens_out, int32_t* row_status,
                           void* stream)
{
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (B < 0 || T < 1 || B > 65535 || T > (1 << 24) || nodes_width < 0) return SPEC_ERR_INVALID_ARG;
    if (B == 0) return SPEC_OK;
    if (!cache_ok(k_cache, v_cache, k_scale, v_scale, page_table, lens, pages, table_width, Hkv, page_size, D))
        return SPEC_ERR_INVALID_ARG;
    const size_t es = dtype_size(dtype);
    if (!on(k, es) || !on(v, es)) return SPEC_ERR_INVALID_ARG;
    if (!on_or_null(accepted_len, 4) || !on_or_null(out_nodes, 4) || !on_or_null(lens_out, 4) ||
        !on_or_null(row_status, 4))
        return SPEC_ERR_INVALID_ARG;
    // every CTA of a request reads its length, so the new one needs a place of its own; nodes need a count
    if (lens_out == lens || (out_nodes && !accepted_len)) return SPEC_ERR_INVALID_ARG;

    CacheWriteParams P;
    std::memset(&P, 0, sizeof P);
    const int64_t dense[3] = {(int64_t)T * Hkv * D, (int64_t)Hkv * D, D};
    const int64_t* strides[2] = {k_strides ? k_strides : dense, v_strides ? v_strides : dense};
    for (int i = 0; i < 2; ++i) {
        P.src[i] = i ? v : k;
        P.sb[i] = strides[i][0];
        P.st[i] = strides[i][1];
        P.sh[i] = strides[i][2];
        P.codes[i] = static_cast<uint8_t*>(i ? v_cache : k_cache);
        P.scale[i] = i ? v_scale : k_scale;
    }
    P.page_table = page_table;
    P.lens = lens;
    P.accepted_len = accepted_len;
    P.out_nodes = out_nodes;
    P.nodes_width = nodes_width;
    P.lens_out = lens_out;
    P.row_status = row_status;
    P.B = B;
    P.T = T;
    P.Hkv = Hkv;
    P.D = D;
    P.page = page_size;
    P.pages = pages;
    P.table_width = table_width;
    const cudaError_t e = launch_cache_write(P, (int)dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

spec_status kv_cache_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                          int pages, int page_size, int Hkv, int D, const int32_t* page_table, int table_width,
                          const int32_t* lens, const int32_t* start, int B, int max_len, void* k_out, void* v_out,
                          spec_dtype dtype, int32_t* row_status, void* stream)
{
    if (dtype != SPEC_F32 && dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (B < 0 || max_len < 1 || B > 65535) return SPEC_ERR_INVALID_ARG;
    if (B == 0) return SPEC_OK;
    if (!cache_ok(k_cache, v_cache, k_scale, v_scale, page_table, lens, pages, table_width, Hkv, page_size, D))
        return SPEC_ERR_INVALID_ARG;
    if (!on(k_out, 16) || !on(v_out, 16) || !on_or_null(start, 4) || !on_or_null(row_status, 4))
        return SPEC_ERR_INVALID_ARG;
    CacheReadParams P;
    std::memset(&P, 0, sizeof P);
    P.codes[0] = static_cast<const uint8_t*>(k_cache);
    P.codes[1] = static_cast<const uint8_t*>(v_cache);
    P.scale[0] = k_scale;
    P.scale[1] = v_scale;
    P.page_table = page_table;
    P.lens = lens;
    P.start = start;
    P.out[0] = k_out;
    P.out[1] = v_out;
    P.row_status = row_status;
    P.B = B;
    P.max_len = max_len;
    P.Hkv = Hkv;
    P.D = D;
    P.page = page_size;
    P.page_shift = page_shift_of(page_size);
    P.pages = pages;
    P.table_width = table_width;
    const cudaError_t e = launch_cache_read(P, (int)dtype, round_sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

size_t verify_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D)
{
    if (B < 0 || T < 1 || T > ATTN_MAX_ROWS || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || (D != 64 && D != 128)) return 0;
    const long long rows = (long long)T * (Hq / Hkv);
    return attn_workspace_bytes(rows < 128 ? (int)rows : 128, D);
}

spec_status verify_attention(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                             const void* v, const int64_t* v_strides, spec_dtype dtype, int B, int T, int Hq,
                             int Hkv, int D, const void* k_cache, const void* v_cache, const float* k_scale,
                             const float* v_scale, int pages, int page_size, const int32_t* page_table,
                             int table_width, const int32_t* lens, const int32_t* parents, const int32_t* n_rows,
                             float scale, void* out, float* lse, int32_t* row_status, void* workspace,
                             size_t workspace_bytes, void* stream)
{
    if (dtype != SPEC_BF16 && dtype != SPEC_F16) return SPEC_ERR_INVALID_ARG;
    if (B < 0 || T < 1 || T > ATTN_MAX_ROWS || B > 65535) return SPEC_ERR_INVALID_ARG;
    if (Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq > 4096) return SPEC_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return SPEC_ERR_INVALID_ARG;
    if (B == 0) return SPEC_OK;
    if (!cache_ok(k_cache, v_cache, k_scale, v_scale, page_table, lens, pages, table_width, Hkv, page_size, D))
        return SPEC_ERR_INVALID_ARG;
    if (!on(q, 2) || !on(out, 16) || (!k) != (!v) || !on_or_null(k, 2) || !on_or_null(v, 2)) return SPEC_ERR_INVALID_ARG;
    if (!on_or_null(parents, 4) || !on_or_null(n_rows, 4) || !on_or_null(lse, 4) || !on_or_null(row_status, 4))
        return SPEC_ERR_INVALID_ARG;
    if (!on(workspace, 16) || workspace_bytes < verify_attention_workspace_bytes(B, T, Hq, Hkv, D))
        return SPEC_ERR_WORKSPACE;
    AttnParams P;
    std::memset(&P, 0, sizeof P);
    const int64_t dq[3] = {(int64_t)T * Hq * D, (int64_t)Hq * D, D}, dk[3] = {(int64_t)T * Hkv * D, (int64_t)Hkv * D, D};
    const int64_t *sq = q_strides ? q_strides : dq, *sk = k_strides ? k_strides : dk, *sv = v_strides ? v_strides : dk;
    P.q = q;
    P.qb = sq[0];
    P.qt = sq[1];
    P.qh = sq[2];
    P.kn = k;
    P.vn = v;
    P.kb = sk[0];
    P.kt = sk[1];
    P.kh = sk[2];
    P.vb = sv[0];
    P.vt = sv[1];
    P.vh = sv[2];
    P.kc = static_cast<const uint8_t*>(k_cache);
    P.vc = static_cast<const uint8_t*>(v_cache);
    P.ks = k_scale;
    P.vs = v_scale;
    P.page_table = page_table;
    P.lens = lens;
    P.parents = T > 1 && k ? parents : nullptr;  // of rows that are there
    P.n_rows = n_rows;
    P.out = out;
    P.lse = lse;
    P.row_status = row_status;
    P.joins = static_cast<AttnJoin*>(workspace);
    P.parts = reinterpret_cast<float*>(P.joins + ATTN_MAX_CTAS);
    P.B = B;
    P.T = T;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.G = Hq / Hkv;
    P.D = D;
    P.page = page_size;
    P.page_shift = page_shift_of(page_size);
    P.pages = pages;
    P.table_width = table_width;
    P.R = T * P.G;
    P.scale = scale;
    P.wait_limit = wait_limit_polls();
    const cudaError_t e = launch_attention(P, (int)dtype, round_sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // extern "C"
