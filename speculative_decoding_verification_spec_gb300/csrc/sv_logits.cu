// sv_logits.cu -- process_logits: penalties for repeated tokens, biases and grammar masks on the
// rows of one verification round.
//
// Row r of request b scores the token that follows the request's history and the drafted tokens on
// the path to row r (a chain: tokens 0 .. r-1; a tree: node r-1 and its ancestors).  With
// c(v) = how often v was generated (history past the prompt, and the path), and seen(v) = c(v) > 0 or
// v in the prompt,
//   x <- seen(v) ? (x > 0 ? x / repetition : x * repetition) : x
//   x <- x - (frequency * c(v) + presence * [c(v) > 0])
//   x <- x + bias(v);   x <- -inf where the mask disallows v
// in fp32, rounded once to the logits' type.
//
// Bound by HBM: every logit is read and written once.  One CTA owns a run of `chunk` vocabulary entries of one
// request for all its rows: it counts the history tokens that fall into its run in shared memory (a
// 32-bit word per entry, so no count is kept from call to call), then streams the rows.  An entry's word and
// bias serve every row.  A drafted token changes single entries of single rows: its entry's word
// carries a flag, and the owning thread, alone, asks which of the run's drafted tokens lie on the row's
// path; so rows need no barrier between them.
#include "sv_round.cuh"

namespace sv {

namespace {

constexpr uint32_t LW_SEEN = 0x80000000u;   // the entry is in the prompt
constexpr uint32_t LW_DRAFT = 0x40000000u;  // a drafted token names the entry
constexpr uint32_t LW_COUNT = 0x3fffffffu;
constexpr int LROWS = 4;                    // rows whose loads are in flight together

// the node of row r - 1 (or its ancestors) is `node`: walks towards the frontier, whose parent is -1.
// A parent outside [-1, i) ends the walk, so it always ends.
__device__ bool on_path(const LogitsParams& P, int b, int r, int node)
{
    int i = r - 1;
    if (!P.parents) return node <= i;
    const int32_t* par = P.parents + (size_t)b * P.N;
    while (i > node) {
        const int p = __ldg(par + i);
        if (p < 0 || p >= i) return false;
        i = p;
    }
    return i == node;
}

template <int DT, int VEC>
__device__ __forceinline__ void store_vec(char* row, long long v, const float (&x)[VEC])
{
    if constexpr (DT == DT_BF16) {
        auto pack = [](float lo, float hi) {
            uint32_t r;
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
            return r;
        };
        if constexpr (VEC == 8) {
            uint4 w;
            w.x = pack(x[0], x[1]);
            w.y = pack(x[2], x[3]);
            w.z = pack(x[4], x[5]);
            w.w = pack(x[6], x[7]);
            __stcs(reinterpret_cast<uint4*>(row) + v, w);
        } else {
            reinterpret_cast<unsigned short*>(row)[v] = (unsigned short)pack(x[0], 0.0f);
        }
    } else if constexpr (VEC == 4) {
        __stcs(reinterpret_cast<float4*>(row) + v, make_float4(x[0], x[1], x[2], x[3]));
    } else {
        reinterpret_cast<float*>(row)[v] = x[0];
    }
}

template <int DT, int VEC>
__device__ __forceinline__ void load_row_vec(const char* row, long long v, float (&x)[VEC])
{
    // plain loads: `out` may be the logits themselves, so the read-only path is not used
    if constexpr (DT == DT_BF16 && VEC == 8) {
        const uint4 w = __ldcs(reinterpret_cast<const uint4*>(row) + v);
        x[0] = bf16lo(w.x); x[1] = bf16hi(w.x); x[2] = bf16lo(w.y); x[3] = bf16hi(w.y);
        x[4] = bf16lo(w.z); x[5] = bf16hi(w.z); x[6] = bf16lo(w.w); x[7] = bf16hi(w.w);
    } else if constexpr (DT == DT_BF16) {
        x[0] = __uint_as_float((uint32_t)reinterpret_cast<const unsigned short*>(row)[v] << 16);
    } else if constexpr (VEC == 4) {
        const float4 w = __ldcs(reinterpret_cast<const float4*>(row) + v);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
    } else {
        x[0] = reinterpret_cast<const float*>(row)[v];
    }
}

template <int DT, int VEC>
__global__ void __launch_bounds__(NT) process_logits_kernel(LogitsParams P)
{
    extern __shared__ uint32_t smem[];
    uint32_t* words = smem;                                   // [chunk]
    int32_t* bidx = reinterpret_cast<int32_t*>(smem) + P.chunk;  // [chunk], only with biases
    __shared__ int ndraft, bad;
    __shared__ uint16_t draft[LOGITS_MAX_NODES];              // nodes whose token falls into the run

    const int b = blockIdx.y;
    const int v0 = blockIdx.x * P.chunk;
    const int n = min(P.chunk, P.V - v0);
    const int t = threadIdx.x;
    for (int i = t; i < P.chunk; i += NT) words[i] = 0u;
    if (P.nb)
        for (int i = t; i < P.chunk; i += NT) bidx[i] = 0;
    if (t == 0) ndraft = 0, bad = 0;
    __syncthreads();

    if (P.history) {
        const int hl = min(max(P.history_len ? __ldg(P.history_len + b) : P.H, 0), P.H);
        const int pl = P.prompt_len ? __ldg(P.prompt_len + b) : 0;
        const int32_t* h = P.history + (size_t)b * P.H;
        for (int i = t; i < hl; i += NT) {
            const uint32_t k = (uint32_t)(__ldg(h + i) - v0);
            if (k < (uint32_t)n) {
                if (i < pl) atomicOr(&words[k], LW_SEEN);
                else atomicAdd(&words[k], 1u);
            }
        }
    }
    for (int i = t; i < P.N; i += NT) {
        const uint32_t k = (uint32_t)(__ldg(P.tokens + (size_t)b * P.N + i) - v0);
        if (k < (uint32_t)n) {
            atomicOr(&words[k], LW_DRAFT);
            draft[atomicAdd(&ndraft, 1)] = (uint16_t)i;
        }
        if (P.parents && blockIdx.x == 0) {
            const int p = __ldg(P.parents + (size_t)b * P.N + i);
            if (p < -1 || p >= i) bad = 1;
        }
    }
    for (int i = t; i < P.nb; i += NT) {
        const uint32_t k = (uint32_t)(__ldg(P.bias_tokens + (size_t)b * P.nb + i) - v0);
        if (k < (uint32_t)n) atomicMax(&bidx[k], i + 1);  // of entries that name one token the last holds
    }
    __syncthreads();
    if (P.row_status && blockIdx.x == 0 && t == 0) P.row_status[b] = bad ? ROW_BAD_PARENT : ROW_OK;

    const float rep = P.repetition ? __ldg(P.repetition + b) : 1.0f;
    const float pres = P.presence ? __ldg(P.presence + b) : 0.0f;
    const float freq = P.frequency ? __ldg(P.frequency + b) : 0.0f;
    constexpr size_t ES = DT == DT_BF16 ? 2 : 4;
    const char* in = reinterpret_cast<const char*>(P.logits) + (size_t)b * P.in_b * ES;
    char* out = reinterpret_cast<char*>(P.out) + (size_t)b * P.out_b * ES;
    const uint32_t* allowed = P.allowed ? P.allowed + (size_t)b * P.R * P.mwords : nullptr;

    for (int k = t; k < n / VEC; k += NT) {
        const long long v = v0 / VEC + k;
        uint32_t any = 0, w[VEC];
        float bias[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[e] = words[k * VEC + e];
            any |= w[e];
            bias[e] = 0.0f;
        }
        if (P.nb) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const int i = bidx[k * VEC + e];
                if (i) {
                    bias[e] = __ldg(P.bias_values + (size_t)b * P.nb + i - 1);
                    any |= 1u;
                }
            }
        }
        for (int r0 = 0; r0 < P.R; r0 += LROWS) {
            float x[LROWS][VEC];
            uint32_t ok[LROWS];
#pragma unroll
            for (int j = 0; j < LROWS; ++j) {
                const int r = r0 + j;
                ok[j] = 0xffffffffu;
                if (r < P.R) {
                    load_row_vec<DT, VEC>(in + (size_t)r * P.in_r * ES, v, x[j]);
                    if (allowed) ok[j] = __ldg(allowed + (size_t)r * P.mwords + (v * VEC >> 5)) >> (v * VEC & 31);
                }
            }
#pragma unroll
            for (int j = 0; j < LROWS; ++j) {
                const int r = r0 + j;
                if (r >= P.R) break;
                if (any) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        int c = (int)(w[e] & LW_COUNT);
                        if (w[e] & LW_DRAFT) {
                            for (int i = 0; i < ndraft; ++i) {
                                const int node = draft[i];
                                if (node < r && __ldg(P.tokens + (size_t)b * P.N + node) == (int)(v * VEC) + e &&
                                    on_path(P, b, r, node))
                                    ++c;
                            }
                        }
                        float y = x[j][e];
                        if (c > 0 || (w[e] & LW_SEEN)) y = y > 0.0f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
                        if (c > 0) y = __fsub_rn(y, __fadd_rn(__fmul_rn(freq, (float)c), pres));
                        x[j][e] = __fadd_rn(y, bias[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (!(ok[j] >> e & 1u)) x[j][e] = NEG_INF;
                store_vec<DT, VEC>(out + (size_t)r * P.out_r * ES, v, x[j]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_process_logits(LogitsParams& P, int dtype, int sms, cudaStream_t st)
{
    const size_t es = dtype == DT_BF16 ? 2 : 4;
    const int vmax = 16 / (int)es;
    const bool vec = P.V % vmax == 0 && P.in_b % vmax == 0 && P.in_r % vmax == 0 && P.out_b % vmax == 0 &&
                     P.out_r % vmax == 0 && reinterpret_cast<uintptr_t>(P.logits) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(P.out) % 16 == 0;
    // longer runs read the history less often; shorter ones give a small batch more CTAs
    P.chunk = 4096;
    while (P.chunk > 1024 && (long long)P.B * ((P.V + P.chunk - 1) / P.chunk) < 2LL * sms) P.chunk /= 2;
    const dim3 grid((unsigned)((P.V + P.chunk - 1) / P.chunk), (unsigned)P.B);
    const size_t smem = (size_t)P.chunk * 4 * (P.nb ? 2 : 1);
    if (dtype == DT_BF16) {
        if (vec) process_logits_kernel<DT_BF16, 8><<<grid, NT, smem, st>>>(P);
        else process_logits_kernel<DT_BF16, 1><<<grid, NT, smem, st>>>(P);
    } else {
        if (vec) process_logits_kernel<DT_F32, 4><<<grid, NT, smem, st>>>(P);
        else process_logits_kernel<DT_F32, 1><<<grid, NT, smem, st>>>(P);
    }
    return cudaGetLastError();
}

}  // namespace sv
