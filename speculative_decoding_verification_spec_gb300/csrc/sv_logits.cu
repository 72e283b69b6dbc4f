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
// request for all its rows.  It counts the history tokens that fall into its run in shared memory (a 32-bit word per
// entry, so nothing is kept from call to call) and lists the entries that anything touches.  Then it copies the rows in
// 16-byte vectors, with the mask, and at last rewrites the touched entries, one thread per (entry, row): a
// text's words crowd into few runs (frequent tokens have low numbers), and in the copy loop each of them would hold up
// the 31 other lanes of its warp, row after row.  Rows need not start on a 16-byte boundary (an odd V): each row's
// vectors start at its own first boundary, the few entries before it and after its last whole vector go one by one.
//
// Measured: 59 us for the 197 MB of (B, R, V) = (64, 6, 128256) bf16 (3.4 TB/s), 290 us for the 1.1 GB of (32, 65, 128256) under
// a mask (3.8 TB/s, where a copy moves 6.8).  What keeps it from a copy's rate are a CTA's phases: history, barriers, first loads,
// copy and touched entries follow one another, and the touched entries are read and written a second time after their
// lines have gone out.
#include <type_traits>

#include "sv_round.cuh"

namespace sv {

namespace {

constexpr uint32_t LW_SEEN = 0x80000000u;   // the entry is in the prompt
constexpr uint32_t LW_DRAFT = 0x40000000u;  // a drafted token names the entry
constexpr uint32_t LW_BIAS = 0x20000000u;   // a bias names the entry
constexpr uint32_t LW_COUNT = 0x1fffffffu;
constexpr int LU = 4;                       // vectors in flight per thread
constexpr int HU = 8;                       // history tokens in flight per thread
constexpr int LOGITS_MAX_SMEM = 160 * 1024; // more than the longest run, draft and biases take
constexpr int LMASK = 64;                   // drafted tokens of a run whose paths are kept as bit masks
constexpr int LMASK_ROWS = 512;             // and the rows that this is done for

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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int DT>
__device__ __forceinline__ float load_one(const char* row, int v)
{
    // plain loads: `out` may be the logits themselves, so the read-only path is not used
    if constexpr (DT == DT_BF16) return __uint_as_float((uint32_t)reinterpret_cast<const unsigned short*>(row)[v] << 16);
    else return reinterpret_cast<const float*>(row)[v];
}
template <int DT>
__device__ __forceinline__ void store_one(char* row, int v, float x)
{
    if constexpr (DT == DT_BF16) reinterpret_cast<unsigned short*>(row)[v] = (unsigned short)pack_bf16(x, 0.0f);
    else reinterpret_cast<float*>(row)[v] = x;
}

// four mask bits as the top bits of four bytes, which a byte permutation can then spread
__device__ __forceinline__ uint32_t spread4(uint32_t bits) { return (bits & 15u) * 0x10204080u & 0x80808080u; }

// a vector with -inf where its entry's bit is not set
template <int DT>
__device__ __forceinline__ uint4 masked_vec(uint4 w, uint32_t ok)
{
    const auto pick = [](uint32_t x, uint32_t keep, uint32_t inf) { return (x & keep) | (inf & ~keep); };
    const auto sign = [](uint32_t y, uint32_t sel) {
        uint32_t r;
        asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(y), "r"(sel));  // selector nibbles 8 + j: byte j's top bit, eight times
        return r;
    };
    if constexpr (DT == DT_BF16) {
        const uint32_t a = spread4(ok), b = spread4(ok >> 4);
        w.x = pick(w.x, sign(a, 0x9988), 0xff80ff80u);
        w.y = pick(w.y, sign(a, 0xbbaa), 0xff80ff80u);
        w.z = pick(w.z, sign(b, 0x9988), 0xff80ff80u);
        w.w = pick(w.w, sign(b, 0xbbaa), 0xff80ff80u);
    } else {
        const uint32_t a = spread4(ok);
        w.x = pick(w.x, sign(a, 0x8888), 0xff800000u);
        w.y = pick(w.y, sign(a, 0x9999), 0xff800000u);
        w.z = pick(w.z, sign(a, 0xaaaa), 0xff800000u);
        w.w = pick(w.w, sign(a, 0xbbbb), 0xff800000u);
    }
    return w;
}

// what a CTA knows of its request and run
struct Run {
    int b, v0, ndraft, nbias;
    float rep, pres, freq;
    const uint32_t* words;
    const uint16_t* draft;
    const uint16_t* bias;
    const uint32_t* base;      // word of a drafted entry (its own holds the entry's number)
    const uint64_t* same;      // which of the run's drafted tokens name that entry, or null
    const uint64_t* row_path;  // which of them lie on each row's path
};

// the penalties of an entry that was generated c times
__device__ __forceinline__ float penalised(const Run& q, float x, int c, bool seen)
{
    if (c > 0 || seen) x = x > 0.0f ? x / q.rep : x * q.rep;
    if (c > 0) x -= fmaf(q.freq, (float)c, q.pres);
    return x;
}

// an entry that a drafted token or a bias names
__device__ __noinline__ float touched_rare(const LogitsParams& P, const Run& q, int r, int v, float x, uint32_t w)
{
    int extra = 0;
    float add = 0.0f;
    if (w & LW_DRAFT) {
        const int g = (int)(w & LW_COUNT);
        w = q.base[g];
        if (q.same) {
            extra = __popcll(q.same[g] & q.row_path[r]);
        } else {
            for (int i = 0; i < q.ndraft; ++i) {
                const int node = q.draft[i];
                if (node < r && __ldg(P.tokens + (size_t)q.b * P.N + node) == v && on_path(P, q.b, r, node)) ++extra;
            }
        }
    }
    if (w & LW_BIAS) {
        int last = -1;  // of entries that name one token the last holds
        for (int i = 0; i < q.nbias; ++i) {
            const int k = q.bias[i];
            if (k > last && __ldg(P.bias_tokens + (size_t)q.b * P.nb + k) == v) last = k;
        }
        if (last >= 0) add = __ldg(P.bias_values + (size_t)q.b * P.nb + last);
    }
    return penalised(q, x, (int)(w & LW_COUNT) + extra, (w & LW_SEEN) != 0) + add;
}

// logit x of touched entry v in row r
__device__ __forceinline__ float touched(const LogitsParams& P, const Run& q, int r, int v, float x)
{
    const uint32_t w = q.words[v - q.v0];
    if (w & (LW_DRAFT | LW_BIAS)) return touched_rare(P, q, r, v, x, w);
    return penalised(q, x, (int)(w & LW_COUNT), (w & LW_SEEN) != 0);
}

// The CTA that owns entry v of a row writes it: the one whose run holds the start of v's vector, or v itself where the
// row has no whole vector around it (s entries before the first boundary, those from `tail` on).
template <int VEC>
__device__ __forceinline__ bool owns(int v, int s, int V, int v0, int n)
{
    const int tail = s + ((V - s) & ~(VEC - 1));
    const int start = v < s || v >= tail ? v : s + ((v - s) & ~(VEC - 1));
    return start >= v0 && start < v0 + n;
}

template <int DT, int VEC>
__device__ __forceinline__ int lead_in(const char* row)  // entries before the row's first 16-byte boundary
{
    constexpr int ES = DT == DT_BF16 ? 2 : 4;
    return VEC == 1 ? 0 : (int)((0u - (uint32_t)reinterpret_cast<uintptr_t>(row)) & 15u) / ES;
}

// VEC: elements of a 16-byte vector, or 1 where a row of the output is not aligned as its input is
template <int DT, int VEC, bool MASK>
__global__ void __launch_bounds__(NT, 5) process_logits_kernel(LogitsParams P)
{
    constexpr size_t ES = DT == DT_BF16 ? 2 : 4;
    extern __shared__ uint32_t smem[];
    // a vector that starts in the run may reach VEC - 1 entries past it: words and bits cover those too
    const int room = P.chunk + 32;
    uint32_t* words = smem;                                          // [room]
    uint32_t* bits = smem + room;                                    // [room / 32] touched entries
    uint32_t* base = bits + room / 32;                               // [N] words of the drafted entries
    uint16_t* list = reinterpret_cast<uint16_t*>(base + P.N);        // [room] touched entries
    uint16_t* draft = list + room;                                   // [N] nodes whose token is in the run
    uint16_t* bias = draft + P.N;                                    // [nb]
    __shared__ int ndraft, nentry, nbias, nlist, bad;
    __shared__ uint64_t same[LMASK], row_path[LMASK_ROWS];

    Run q;
    const int b = q.b = blockIdx.y;
    const int v0 = q.v0 = blockIdx.x * P.chunk;
    const int n = min(P.chunk, P.V - v0);              // entries of the run
    const int nw = min(n + VEC - 1, P.V - v0);         // and those that its last vectors may reach
    const int t = threadIdx.x;
    const int r_lo = blockIdx.z * P.rows, r_hi = min(P.R, r_lo + P.rows);  // this CTA's rows
    const char* in0 = reinterpret_cast<const char*>(P.logits) + (size_t)b * P.in_b * ES;
    char* out0 = reinterpret_cast<char*>(P.out) + (size_t)b * P.out_b * ES;
    const uint32_t* allowed0 = MASK ? P.allowed + (size_t)b * P.R * P.mwords : nullptr;
    // Everything of the first round of loads is asked for at once: one after another, with barriers between, the lengths, the
    // history, the biases and the draft would take as long as the copy.
    const int32_t* h = P.history + (size_t)b * P.H;
    const int32_t hl_ = P.history_len ? __ldg(P.history_len + b) : P.H, pl = P.prompt_len ? __ldg(P.prompt_len + b) : 0;
    int32_t said[HU];
#pragma unroll
    for (int j = 0; j < HU; ++j) said[j] = t + j * NT < P.H ? __ldg(h + t + j * NT) : -1;
    const int32_t bias_t = t < P.nb ? __ldg(P.bias_tokens + (size_t)b * P.nb + t) : -1;
    const int32_t draft_t = t < P.N ? __ldg(P.tokens + (size_t)b * P.N + t) : -1;
    for (int i = t; i < (room + room / 32) / 4; i += NT) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    for (int i = (room + room / 32) / 4 * 4 + t; i < room + room / 32; i += NT) smem[i] = 0u;
    if (t == 0) ndraft = 0, nentry = 0, nbias = 0, nlist = 0, bad = 0;
    if (t < LMASK) same[t] = 0;
    __syncthreads();

    const int hl = min(max((int)hl_, 0), P.H);
    for (int i0 = t; i0 < hl; i0 += NT * HU) {
        if (i0 != t) {
#pragma unroll
            for (int j = 0; j < HU; ++j) said[j] = i0 + j * NT < hl ? __ldg(h + i0 + j * NT) : -1;
        }
#pragma unroll
        for (int j = 0; j < HU; ++j) {
            const uint32_t k = (uint32_t)(said[j] - v0);
            if (k < (uint32_t)nw && i0 + j * NT < hl) {
                if (i0 + j * NT < pl) atomicOr(&words[k], LW_SEEN);
                else atomicAdd(&words[k], 1u);
                atomicOr(&bits[k >> 5], 1u << (k & 31));
            }
        }
    }
    for (int i = t; i < P.nb; i += NT) {
        const uint32_t k = (uint32_t)((i == t ? bias_t : __ldg(P.bias_tokens + (size_t)b * P.nb + i)) - v0);
        if (k < (uint32_t)nw) {
            atomicOr(&words[k], LW_BIAS);
            atomicOr(&bits[k >> 5], 1u << (k & 31));
            bias[atomicAdd(&nbias, 1)] = (uint16_t)i;
        }
    }
    __syncthreads();
    // A drafted entry's word moves to `base` and makes room for the entry's number: the one thread that finds the
    // word unflagged does it.
    for (int i = t; i < P.N; i += NT) {
        const uint32_t k = (uint32_t)((i == t ? draft_t : __ldg(P.tokens + (size_t)b * P.N + i)) - v0);
        if (k < (uint32_t)nw) {
            const uint32_t was = atomicOr(&words[k], LW_DRAFT);
            draft[atomicAdd(&ndraft, 1)] = (uint16_t)i;
            if (!(was & LW_DRAFT)) {
                const int g = atomicAdd(&nentry, 1);
                base[g] = was;
                words[k] = LW_DRAFT | (uint32_t)g;
                atomicOr(&bits[k >> 5], 1u << (k & 31));
            }
        }
        if (P.parents && blockIdx.x == 0 && blockIdx.z == 0) {
            const int p = __ldg(P.parents + (size_t)b * P.N + i);
            if (p < -1 || p >= i) bad = 1;
        }
    }
    __syncthreads();
    if (P.row_status && blockIdx.x == 0 && blockIdx.z == 0 && t == 0) P.row_status[b] = bad ? ROW_BAD_PARENT : ROW_OK;
    const bool masks = ndraft <= LMASK && P.R <= LMASK_ROWS;
    if (masks && ndraft > 0) {
        if (t < ndraft) {
            const int v = __ldg(P.tokens + (size_t)b * P.N + draft[t]);
            atomicOr(reinterpret_cast<unsigned long long*>(&same[words[v - v0] & LW_COUNT]), 1ull << t);
        }
        for (int r = r_lo + t; r < r_hi; r += NT) {
            uint64_t m = 0;
            for (int node = r - 1; node >= 0;) {
                if (!P.parents) {
                    for (int i = 0; i < ndraft; ++i) m |= (uint64_t)(draft[i] <= node) << i;
                    break;
                }
                for (int i = 0; i < ndraft; ++i) m |= (uint64_t)(draft[i] == node) << i;
                const int p = __ldg(P.parents + (size_t)b * P.N + node);
                if (p >= node) break;  // out of range: the path ends here
                node = p;
            }
            row_path[r] = m;
        }
    }
    for (int i = t; i < room / 32; i += NT) {
        uint32_t left = bits[i];
        if (left) {
            int at = atomicAdd(&nlist, __popc(left));
            for (; left; left &= left - 1) list[at++] = (uint16_t)(i * 32 + __ffs(left) - 1);
        }
    }

    // the copy, with the mask
    if constexpr (VEC == 1) {
        for (int r = r_lo; r < r_hi; ++r) {
            const uint32_t* allowed = MASK ? allowed0 + (size_t)r * P.mwords : nullptr;
            for (int v = v0 + t; v < v0 + n; v += NT) {
                float x = load_one<DT>(in0 + (size_t)r * P.in_r * ES, v);
                if (MASK && !(__ldg(allowed + (v >> 5)) >> (v & 31) & 1u)) x = NEG_INF;
                store_one<DT>(out0 + (size_t)r * P.out_r * ES, v, x);
            }
        }
    } else {
        // slots: the vectors of a row that a thread may own in this run, threads apart
        const int slots = (n + VEC * NT - 1) / (VEC * NT);
        const char* in = in0 + (size_t)r_lo * P.in_r * ES;
        for (int r = r_lo, slot = 0; r < r_hi;) {
            uint4 w[LU];
            uint32_t ok[LU];
            char* to[LU];  // null: no vector
#pragma unroll
            for (int j = 0; j < LU; ++j) {
                to[j] = nullptr;
                ok[j] = 0xffffffffu;
                if (r < r_hi) {
                    const int s = lead_in<DT, VEC>(in);
                    const int first = s + ((v0 - s + VEC - 1) & ~(VEC - 1));  // the first vector that starts in the run
                    const int v = first + (slot * NT + t) * VEC;
                    if (v < v0 + n && v + VEC <= P.V) {
                        to[j] = out0 + ((size_t)r * P.out_r + v) * ES;
                        w[j] = __ldcs(reinterpret_cast<const uint4*>(in + (size_t)v * ES));
                        if constexpr (MASK) {
                            const uint32_t* a = allowed0 + (size_t)r * P.mwords + (v >> 5);
                            ok[j] = __ldg(a) >> (v & 31);
                            if ((v & 31) + VEC > 32) ok[j] |= __ldg(a + 1) << (32 - (v & 31));
                        }
                    }
                    if (++slot == slots) {
                        slot = 0;
                        ++r;
                        in += (size_t)P.in_r * ES;
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < LU; ++j) {
                if (!to[j]) continue;
                if constexpr (MASK) w[j] = masked_vec<DT>(w[j], ok[j]);
                __stcs(reinterpret_cast<uint4*>(to[j]), w[j]);
            }
        }
        // the entries before a row's first boundary and after its last whole vector: at most VEC - 1 each
        for (int f = t; f < (r_hi - r_lo) * 2 * VEC; f += NT) {
            const int r = r_lo + f / (2 * VEC), e = f % (2 * VEC);
            const char* row = in0 + (size_t)r * P.in_r * ES;
            const int s = min(lead_in<DT, VEC>(row), P.V);
            const int v = e < VEC ? e : s + ((P.V - s) & ~(VEC - 1)) + e - VEC;
            if ((e < VEC ? v < s : v < P.V) && v >= v0 && v < v0 + n) {
                float x = load_one<DT>(row, v);
                if (MASK && !(__ldg(allowed0 + (size_t)r * P.mwords + (v >> 5)) >> (v & 31) & 1u)) x = NEG_INF;
                store_one<DT>(out0 + (size_t)r * P.out_r * ES, v, x);
            }
        }
    }
    __syncthreads();

    // The touched entries.  In place they still hold their logits here: the copy wrote back what it read.
    q.ndraft = ndraft;
    q.nbias = nbias;
    q.words = words;
    q.draft = draft;
    q.bias = bias;
    q.base = base;
    q.same = masks ? same : nullptr;
    q.row_path = row_path;
    q.rep = P.repetition ? __ldg(P.repetition + b) : 1.0f;
    q.pres = P.presence ? __ldg(P.presence + b) : 0.0f;
    q.freq = P.frequency ? __ldg(P.frequency + b) : 0.0f;
    const int touched_n = nlist;
    const long long items = (long long)(r_hi - r_lo) * touched_n;
    constexpr int TU = 4;
    for (long long i0 = t; i0 < items; i0 += TU * NT) {
        float x[TU];
        int row[TU], at[TU];
#pragma unroll
        for (int j = 0; j < TU; ++j) {
            const long long i = i0 + j * NT;
            at[j] = -1;
            if (i < items) {
                const int k = items < (1LL << 31) ? (int)((uint32_t)i / (uint32_t)touched_n) : (int)(i / touched_n);
                const int r = row[j] = r_lo + k, v = v0 + list[(int)(i - (long long)k * touched_n)];
                const char* in = in0 + (size_t)r * P.in_r * ES;
                if (owns<VEC>(v, min(lead_in<DT, VEC>(in), P.V), P.V, v0, n) &&
                    !(MASK && !(__ldg(allowed0 + (size_t)r * P.mwords + (v >> 5)) >> (v & 31) & 1u))) {
                    at[j] = v;
                    x[j] = load_one<DT>(in, v);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < TU; ++j)
            if (at[j] >= 0) store_one<DT>(out0 + (size_t)row[j] * P.out_r * ES, at[j], touched(P, q, row[j], at[j], x[j]));
    }
}

template <auto K, int VEC>
cudaError_t launch_chunks(LogitsParams& P, int sms, cudaStream_t st)
{
    // The run length (and groups of rows) with the best of: few SM slots idle in the grid's last wave, and little time per run
    // spent on anything but its rows (reading the history, barriers, the touched entries: measured as long as some 24 KB of
    // rows).  At (B, R, V, H) = (64, 6, 128256, 2048) runs of 2048, 4096 and 8192 entries take 67, 65 and 79 us, at
    // (32, 65, 128256, 4000) 290, 335 and 398 us, at (200, 2, 128256, 2048) 110, 83 and 85 us.
    const auto smem = [&](int chunk) {
        return ((size_t)chunk + 32 + (chunk + 32) / 32 + P.N) * 4 + ((size_t)chunk + 32 + P.N + P.nb + 1) / 2 * 4;
    };
    static PerDevice kept;
    int& per_sm = kept.here();  // CTAs that the registers allow
    if (per_sm == 0) {
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, K);
        if (e != cudaSuccess) return e;
        const cudaError_t f = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, LOGITS_MAX_SMEM);
        if (f != cudaSuccess) return f;
        per_sm = max(1, min(2048 / NT, 65536 / (((a.numRegs + 7) / 8 * 8) * NT)));
    }
    constexpr int LEAST = NT * (VEC == 1 ? 4 : VEC);
    int best = LEAST, groups = 1;
    double most = 0.0;
    for (int chunk = 8192; chunk >= LEAST; chunk /= 2) {
        const long long slots = (long long)sms * min(per_sm, (int)(220000 / (smem(chunk) + 6144)));
        if (slots < 1) continue;
        const long long per = (long long)((P.V + chunk - 1) / chunk) * P.B;
        for (int g = 1; g <= 16 && g <= P.R; ++g) {
            // many rows are shared out where the shortest runs alone leave SMs idle ((4, 65, 128256, 4000): 83 to 48 us);
            // elsewhere more CTAs only repeat the history
            if (g > 1 && (chunk > LEAST || per * (g - 1) >= slots)) break;
            const int rows = (P.R + g - 1) / g;
            const long long ctas = per * ((P.R + rows - 1) / rows);
            const double full = (double)P.V * P.B * P.R / ((double)chunk * rows * ((ctas + slots - 1) / slots * slots));
            const double bytes = 2.0 * chunk * rows * (VEC == 4 ? 4 : 2), score = full * bytes / (bytes + 24576.0 + 4.0 * P.H);
            if (score > most) {
                most = score;
                best = chunk;
                groups = g;
            }
        }
    }
    P.rows = (P.R + groups - 1) / groups;
    P.chunk = best;
    const size_t bytes = smem(best);
    K<<<dim3((unsigned)((P.V + best - 1) / best), (unsigned)P.B, (unsigned)((P.R + P.rows - 1) / P.rows)), NT, bytes, st>>>(P);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_process_logits(LogitsParams& P, int dtype, int sms, cudaStream_t st)
{
    const size_t es = dtype == DT_BF16 ? 2 : 4;
    // vectors need every row of the output to lie on its 16-byte boundaries as its input does
    const auto off = [&](int64_t a, int64_t b) { return (a - b) * (int64_t)es % 16 == 0; };
    const bool vec = (reinterpret_cast<uintptr_t>(P.logits) - reinterpret_cast<uintptr_t>(P.out)) % 16 == 0 &&
                     (P.B == 1 || off(P.in_b, P.out_b)) && (P.R == 1 || off(P.in_r, P.out_r));
    const auto go = [&](auto dt, auto v, auto mask) {
        return launch_chunks<process_logits_kernel<dt.value, v.value, mask.value>, v.value>(P, sms, st);
    };
    const auto with = [&](auto dt, auto v) { return P.allowed ? go(dt, v, std::true_type{}) : go(dt, v, std::false_type{}); };
    using std::integral_constant;
    if (dtype == DT_BF16)
        return vec ? with(integral_constant<int, DT_BF16>{}, integral_constant<int, 8>{})
                   : with(integral_constant<int, DT_BF16>{}, integral_constant<int, 1>{});
    return vec ? with(integral_constant<int, DT_F32>{}, integral_constant<int, 4>{})
               : with(integral_constant<int, DT_F32>{}, integral_constant<int, 1>{});
}

}  // namespace sv
