// sv_sample.cu -- sample_logits: one token a row of logits, with temperature, top-k, top-p and min-p, from given uniforms.
//
// Every processor keeps the tokens whose stored logit lies at or above a threshold, ties and all, as the verify calls' do:
//   top-k   g = the k-th largest logit
//   top-p   of what top-k left, g = the largest logit with mass(x >= g) >= top_p * Z
//   min-p   g = max + T ln(min_p)
// and the token is the smallest v with u Z < C(v), C the cumulated mass of the kept tokens in ascending order (inverse CDF).
//
// Where a row lives.  With few rows a row is one thread-block cluster of CL CTAs that split it into slices, kept in shared memory:
// the logits are read from memory once, and the CTAs exchange a record a step through distributed shared memory behind a
// cluster barrier and take the same decisions from the same records.  With many rows a row is one CTA, which reads it again from
// L2 for each of its sweeps (RMEM): two rows an SM, no cluster barriers.  launch_type() has the rule and both sides' times.
//
// Arithmetic.  With c = log2(e) / T a token's mass is 2^(44 + x c - K), K the whole number nearest to max c, right to 2^-28 of
// itself (Mass) and rounded to a whole number, so sums do not depend on their order, a border is crossed by one token or the other,
// and a uniform falls as near to one as the masses are off once in some 10^4 draws among 50000 tokens.  Sums of 2^18 masses stay under
// 2^63.  The exponential unit alone is right to 2^-22: a kernel that summed with it, and drew the rows again whose decisions that left in
// doubt, took four times the code and was slower (512 rows of 152064 with top-p 407 us where a mass a logit of this kind took 300).
//
// Thresholds.  The logits that can matter are listed where they are few (LIST) and compared with one another, each with all: for
// top-k up to 512 those at or above a bound that the threads' maxima give, for min-p those that it keeps.  Otherwise a row of bf16 is
// counted by value (counted()).  In fp32 a histogram of masses (with the sum of all, in one sweep) or of counts brackets the threshold
// to a bin or so, whose logits are listed; a bracket with more of them gets bins of its own, and a group of ties is taken as one.
// Bisection over the row where that fails: a threshold under the bins.  Top-k's bins reach 32 under the largest logit, so it is what a
// row in fp32 gets whose mask, a large finite number, leaves fewer than k tokens: 64 rows of 50257 with k = 50 and three tokens left take
// 102 us, 13 without a mask and 11 with -inf, which the list leaves out (in bf16 29, 12 and 10).
//
// What bounds it.  With top-p the shared memory's atomics and lookups, one of each a logit at random places, and that SMs get
// three rows or four: 512 rows of 152064 take 108 us on the GPU (23 are the copy rate's), a row some 50 of which 18 are the first sweep, with the
// counts, and 15 the one that draws.  In fp32 the chain of a row's sweeps and steps behind the cluster's barriers, and
// clusters that last as long as their slowest row: 96 rows of 50257 with settings by row use 33% of the issue slots (30 to 45 instructions a
// logit in the sweep that forms the masses and the bins, 25 in the one that sums what lies over the bracket) and 6% of the
// memory's pace.  With top-k the chain of a row's steps: 64 rows of 128256 take 15 us on the GPU, 5 for the loads, 3 for the bound and the
// exchange, 3 for the list and 4 for what rank 0 does with it.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "sv_round.cuh"

namespace cg = cooperative_groups;

namespace sv {

namespace {

typedef unsigned long long u64;

constexpr int SNT = 512, SW = SNT / 32;
constexpr int LIST = 2 * SNT;      // candidates of a row that are compared with one another
constexpr int MAX_CL = 8;
constexpr int UNIT = SNT;          // vectors: a slice is a whole number of them, each warp's run one of 32
constexpr int STEPS = 32;          // of the exponential's table, an octave
constexpr int FINE = 4;            // bins a step: 128 an octave
constexpr int BINS = 6 * SNT;      // of the histogram: 24 octaves
constexpr int MAGS = 1 << 12;      // of bf16 magnitudes counted, for each sign: 31 octaves (see counted())
constexpr uint32_t GUESS = 0x4280; // bits of 64: the largest magnitude that the first sweep has places for
constexpr int BIN_ONE = 13;        // a mass in the middle of its bin counts 2^13: sums of 2^18 stay under 2^32

// 2^(j / 32) as pairs of floats
__constant__ float2 EXP2_STEPS[STEPS] = {
    {1.0f, 0.0f}, {1.0218972f, -4.81155986e-08f}, {1.04427373f, 4.83347016e-08f}, {1.06714046f, -5.93375198e-08f},
    {1.09050775f, -1.30775399e-08f}, {1.1143868f, -5.43554002e-08f}, {1.13878858f, 5.38622231e-08f}, {1.1637249f, -4.05144149e-08f},
    {1.18920708f, 3.79763527e-08f}, {1.21524739f, -3.26739489e-08f}, {1.24185777f, 4.4968381e-08f}, {1.26905096f, 1.41933332e-09f},
    {1.29683959f, -4.01899953e-08f}, {1.32523668f, -3.49637332e-08f}, {1.35425556f, -1.01233493e-08f}, {1.38390994f, -5.87557736e-08f},
    {1.41421354f, 2.4203235e-08f}, {1.44518077f, 3.32419994e-08f}, {1.47682619f, -4.50089885e-08f}, {1.50916445f, -2.49593732e-08f},
    {1.54221082f, 8.07090483e-09f}, {1.5759809f, -5.66102543e-08f}, {1.61049032f, 9.83621717e-09f}, {1.64575553f, -5.12497209e-08f},
    {1.68179286f, -2.47553267e-08f}, {1.71861935f, -4.8496176e-08f}, {1.75625217f, -9.23577037e-09f}, {1.79470909f, -1.14150449e-08f},
    {1.8340081f, -1.1239278e-08f}, {1.87416768f, -4.66300563e-08f}, {1.91520655f, 9.84532811e-09f}, {1.95714414f, -1.70218044e-08f},
};

__device__ __forceinline__ uint32_t key_of(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float float_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

__device__ __forceinline__ u64 f2_mul(u64 a, u64 b)
{
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 two(float x) { return f2_pack(x, x); }

// What depends on the logits' type: a vector's elements, and a threshold as the elements are compared with it.
template <int DT>
struct Vec;

template <>
struct Vec<DT_BF16> {
    static constexpr int N = 8, SIZE = 2;
    typedef uint32_t Bound;  // the smallest bf16 at or above a float, twice
    static __device__ __forceinline__ Bound bound(float g)
    {
        const uint32_t u = __float_as_uint(g);
        const uint32_t h = (u >> 16) + ((u & 0xffffu) && !(u >> 31) ? 1u : 0u);
        return h | h << 16;
    }
    static __device__ __forceinline__ uint32_t mask(uint32_t w, Bound g)
    {
        return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&g));
    }
    static __device__ __forceinline__ bool any(const uint4& v, Bound g) { return mask(v.x, g) | mask(v.y, g) | mask(v.z, g) | mask(v.w, g); }
    // the elements at or above g, -inf in the others' place; whether there are any
    static __device__ __forceinline__ bool keep(uint4& v, Bound g)
    {
        const uint32_t a = mask(v.x, g), b = mask(v.y, g), c = mask(v.z, g), d = mask(v.w, g), no = 0xff80ff80u;
        v = make_uint4((v.x & a) | (no & ~a), (v.y & b) | (no & ~b), (v.z & c) | (no & ~c), (v.w & d) | (no & ~d));
        return a | b | c | d;
    }
    // a bit for each element at or above g, and what a bit stands for
    static __device__ __forceinline__ uint32_t flags(const uint4& v, Bound g)
    {
        return (mask(v.x, g) & 0x10001u) | (mask(v.y, g) & 0x20002u) | (mask(v.z, g) & 0x40004u) | (mask(v.w, g) & 0x80008u);
    }
    static __device__ __forceinline__ int place(int bit) { return (bit & 3) * 2 + (bit >> 4); }
    static __device__ __forceinline__ float flagged(const uint4& v, int bit)
    {
        const uint32_t a = bit & 1 ? v.y : v.x, b = bit & 1 ? v.w : v.z, q = bit & 2 ? b : a;
        return bit & 16 ? bf16hi(q) : bf16lo(q);
    }
    static __device__ __forceinline__ float elem(const uint4& w, int e)
    {
        const uint32_t q = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
        return e & 1 ? bf16hi(q) : bf16lo(q);
    }
    static __device__ __forceinline__ float max_nan(const uint4& w)
    {
        const uint32_t m = bmax2_nan(bmax2_nan(w.x, w.y), bmax2_nan(w.z, w.w));
        return fmax_nan(bf16lo(m), bf16hi(m));
    }
    static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    static __device__ __forceinline__ void put(uint4& v, int e, const void* row, int t)
    {
        const uint32_t h = __ldg(reinterpret_cast<const unsigned short*>(row) + t);
        uint32_t* q = e < 2 ? &v.x : e < 4 ? &v.y : e < 6 ? &v.z : &v.w;
        *q = e & 1 ? (*q & 0xffffu) | h << 16 : (*q & 0xffff0000u) | h;
    }
};

template <>
struct Vec<DT_F32> {
    static constexpr int N = 4, SIZE = 4;
    typedef float Bound;
    static __device__ __forceinline__ Bound bound(float g) { return g; }
    static __device__ __forceinline__ float elem(const uint4& w, int e) { return __uint_as_float(e == 0 ? w.x : e == 1 ? w.y : e == 2 ? w.z : w.w); }
    static __device__ __forceinline__ bool any(const uint4& v, Bound g)
    {
        return fmaxf(fmaxf(elem(v, 0), elem(v, 1)), fmaxf(elem(v, 2), elem(v, 3))) >= g;
    }
    static __device__ __forceinline__ uint32_t flags(const uint4& v, Bound g)
    {
        return (uint32_t)(elem(v, 0) >= g) | (uint32_t)(elem(v, 1) >= g) << 1 | (uint32_t)(elem(v, 2) >= g) << 2 | (uint32_t)(elem(v, 3) >= g) << 3;
    }
    static __device__ __forceinline__ int place(int bit) { return bit; }
    static __device__ __forceinline__ float flagged(const uint4& v, int bit) { return elem(v, bit); }
    static __device__ __forceinline__ uint32_t one(uint32_t w, Bound g) { return __uint_as_float(w) >= g ? w : 0xff800000u; }
    static __device__ __forceinline__ bool keep(uint4& v, Bound g)
    {
        const bool some = any(v, g);
        v = make_uint4(one(v.x, g), one(v.y, g), one(v.z, g), one(v.w, g));
        return some;
    }
    static __device__ __forceinline__ float max_nan(const uint4& w)
    {
        return fmax_nan(fmax_nan(elem(w, 0), elem(w, 1)), fmax_nan(elem(w, 2), elem(w, 3)));
    }
    static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    static __device__ __forceinline__ void put(uint4& v, int e, const void* row, int t)
    {
        uint32_t* q = e == 0 ? &v.x : e == 1 ? &v.y : e == 2 ? &v.z : &v.w;
        *q = __ldg(reinterpret_cast<const uint32_t*>(row) + t);
    }
};

// A row's scale: c = log2(e) / T as a pair, K, and the origin that logits are taken from: 0, or the largest where |max c| is so
// large that it has to be (what counts then lies near it, and the difference is exact).  The product with c's second part comes behind J
// (see Mass): of a c of 16 bits that part is up to 2^-15 of it, and from 128 octaves (with the 46 that matter, 2^-7.5 at most) bf16 logits
// are taken from the largest.  (From 16384 octaves on, as in fp32, masses were off by up to 2^-15.)  A logit that has 2^-14 of the largest mass then
// lies within a ninth of it: the difference has 7 bits, and its product with 16 is exact.
template <int DT>
constexpr float FAR_OCTAVES = DT == DT_BF16 ? 128.0f : 16384.0f;
struct Scale {
    float hi, lo, origin;
    int K;
};

// units of 512 vectors of a row that begins anywhere in its first vector
constexpr int units_of(int V, int epv) { return ((V + 2 * epv - 2) / epv + UNIT - 1) / UNIT; }

// Masses as A 2^22 + B, each in the low bits of a float next to a power of two: sums of n of them in 32 bits.  A thread meets a
// vector a unit, of the widest row as one CTA 520 logits (516 in fp32), and a mass is 2^(44 + 1/2) at most, but for what K, rounded
// from c's first part, misses: 2^-8 of an octave (FAR_OCTAVES).
struct Part {
    static constexpr int MOST = units_of(SAMPLE_MAX_V, 8) * 8;
    static_assert(MOST >= units_of(SAMPLE_MAX_V, 4) * 4 && MOST * 1.42 * (1 << 22) < 0x1p32 && MOST * 0x1p21 < 0x1p31,
                  "A's sum, and B's, which has a sign");
    uint32_t a, b, n;
    __device__ __forceinline__ void add(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1)
    {
        a += a0 + a1;
        b += b0 + b1;
        n += 2;
    }
    __device__ __forceinline__ u64 whole() const { return ((u64)(a - n * 0x4b000000u) << 22) + (long long)(int)(b - n * 0x4b400000u); }
};

// The masses of two logits: x c as a pair of floats, J / 32 next to it, 2^(J / 32) from the table and e^z - 1 of the rest
// (|z| < 2^-6.1, with c's second part) as its series to z^4.  Of a mass that leaves the roundings of z, up to 2^-30 together, and of its
// product with the table's value, 2^-30: of 400,000 masses followed step by step the worst is off by 2^-28.5, the root of the mean square is 2^-31.
// Logits 80 octaves down are held there: no part of 2^-44.  The table stands in shared memory once a lane, so that a warp's loads meet no bank twice.
template <int DT>
struct Mass {
    u64 origin, hi, lo;
    float deep;
    uint32_t one;  // of a scale's exponent: bits of 2^-K
    const float* steps;  // this lane's: 2^(j / 32), and SECOND further the rest of it
    static constexpr float MAGIC = 12582912.0f;  // 1.5 * 2^23
    static constexpr int SECOND = STEPS * 32;
    __device__ __forceinline__ Mass(const Scale& c, const float* table)
        : origin(two(-c.origin)), hi(two(c.hi)), lo(two(c.lo)), deep(fmaxf(((float)c.K - 80.0f) / c.hi, -3.0e38f)),
          one((uint32_t)(127 - c.K) << 23), steps(table + (threadIdx.x & 31)) {}
    // A and B of each as bits; jx, jy: MAGIC + J as bits; r: the rest of x c
    __device__ __forceinline__ void pair(float x, float y, uint32_t (&ab)[4], uint32_t& jx, uint32_t& jy, u64& r) const
    {
        float dx, dy;
        f2_unpack(f2_add(f2_pack(x, y), origin), dx, dy);
        const u64 d = f2_pack(fmaxf(dx, deep), fmaxf(dy, deep)), th = f2_mul(d, hi);
        const u64 w = f2_fma(th, two((float)STEPS), two(MAGIC));
        r = f2_fma(f2_add(w, two(-MAGIC)), two(-1.0f / STEPS), th);
        // (a bf16 logit, or the difference of two, times a c of 16 bits is exact)
        if constexpr (DT == DT_F32) r = f2_add(r, f2_fma(d, hi, f2_mul(th, two(-1.0f))));
        r = f2_fma(d, lo, r);
        float wx, wy;
        f2_unpack(w, wx, wy);
        jx = __float_as_uint(wx);
        jy = __float_as_uint(wy);
        const float *ex = steps + jx % STEPS * 32, *ey = steps + jy % STEPS * 32;
        const u64 eh = f2_pack(ex[0], ey[0]), el = f2_pack(ex[SECOND], ey[SECOND]);
        // z = r ln 2
        const u64 z = f2_mul(r, f2_fma(r, f2_fma(r, f2_fma(r, two(0.00961812865f), two(0.0555041097f)), two(0.240226507f)), two(0.693147182f)));
        const u64 scale = f2_pack(__uint_as_float((jx << 18 & 0xff800000u) + one), __uint_as_float((jy << 18 & 0xff800000u) + one));
        const u64 v = f2_mul(eh, scale), more = f2_mul(f2_fma(eh, z, el), scale);
        // A next to (v + more) 2^22; what is left of v is exact, and so is its sum with `more`
        const u64 a = f2_fma(v, two(4194304.0f), f2_fma(more, two(4194304.0f), two(8388608.0f)));  // 2^22, 2^23
        const u64 b = f2_fma(f2_add(f2_add(v, f2_fma(a, two(-0x1p-22f), two(2.0f))), more), two(0x1p44f), two(MAGIC));
        float ax, ay, bx, by;
        f2_unpack(a, ax, ay);
        f2_unpack(b, bx, by);
        ab[0] = __float_as_uint(ax);
        ab[1] = __float_as_uint(ay);
        ab[2] = __float_as_uint(bx);
        ab[3] = __float_as_uint(by);
    }
    __device__ __forceinline__ u64 of(float x) const
    {
        uint32_t ab[4], jx, jy;
        u64 r;
        pair(x, x, ab, jx, jy, r);
        return Part{ab[0], ab[2], 1}.whole();
    }
    // the sum over a vector, onto m
    __device__ __forceinline__ void add(const uint4& v, Part& m) const
    {
#pragma unroll
        for (int e = 0; e < Vec<DT>::N; e += 2) {
            uint32_t ab[4], jx, jy;
            u64 r;
            pair(Vec<DT>::elem(v, e), Vec<DT>::elem(v, e + 1), ab, jx, jy, r);
            m.add(ab[0], ab[1], ab[2], ab[3]);
        }
    }
};

// floor(u * z) for u in [0, 1), exactly; `more`: the product is no whole number
__device__ __forceinline__ u64 scaled_floor(float u, u64 z, bool& more)
{
    const uint32_t b = __float_as_uint(u);
    const int e = (int)(b >> 23);
    const u64 m = e ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
    const int s = 150 - (e ? e : 1);  // u = m 2^-s, s >= 24
    const u64 hi = __umul64hi(m, z), lo = m * z;
    const u64 q = s < 64 ? hi << (64 - s) | lo >> s : s < 128 ? hi >> (s - 64) : 0ull;
    more = (s < 64 ? lo << (64 - s) : lo | (s < 128 ? hi & ((1ull << (s - 64)) - 1) : hi)) != 0;
    return q;
}

struct Rec {
    u64 a, b, c;
};

struct Lists {
    float lx[LIST];                // this CTA's candidates, or its logits of a bracket
    int lt[LIST];
    float gx[LIST];                // the row's
    int gt[LIST];
    union {                        // the bins have been read where the masses are formed
        u64 gm[LIST];
        alignas(8) uint32_t bins[BINS];
    };
};
struct Values {
    uint32_t n[2 * MAGS];          // logits of each value
    u64 group_mass[2 * MAGS / 32];
    uint32_t group_n[2 * MAGS / 32];
};
struct None {};

template <bool COUNTS>
struct Shared {
    Rec mine[2], all[MAX_CL];      // a step's record, the cluster's
    u64 warp[SW], sums[SW];
    uint32_t warp32[SW];
    float steps[2 * STEPS * 32];
    union {
        Lists l;
        typename std::conditional<COUNTS, Values, None>::type v;
    };
    int count, step;               // of the list; exchanges so far
    float least, bound[2];         // min-p's threshold; what jth() found
    int from, to;                  // bins of a threshold's bracket
};

// v's inclusive sums over the lanes
__device__ __forceinline__ u64 warp_scan(u64 v)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) >= o) v += y;
    }
    return v;
}

// Sum of v over the CTA, by way of `warp`.  (Out of line, as it is called from many places.)
__device__ __noinline__ u64 cta_sum(u64 v, u64* warp)
{
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = warp[threadIdx.x & (SW - 1)];
    __syncthreads();
#pragma unroll
    for (int o = SW / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int DT, bool RMEM>
struct Row {
    typedef Vec<DT> V;
    static constexpr int EPV = V::N;
    static constexpr bool COUNTS = DT == DT_BF16;  // see counted()
    typedef Shared<COUNTS> Sh;
    const SampleParams& P;
    Sh& sh;
    uint4* slice;
    const char* base;  // the row
    int tid, w, lane, rank, CL;
    int spw;           // segments of 32 vectors of a warp
    int vec0;          // this CTA's first vector; the row's begin at the 16-byte border at or before the row
    int head, whole0, whole1;  // elements of the first vector that are not the row's; vectors that are the row's altogether
    float top;
    Scale c;

    __device__ __forceinline__ Row(const SampleParams& p, Sh& s, uint4* sl, int row) : P(p), sh(s), slice(sl)
    {
        tid = threadIdx.x;
        w = tid >> 5;
        lane = tid & 31;
        rank = RMEM ? 0 : (int)cg::this_cluster().block_rank();
        CL = RMEM ? 1 : (int)cg::this_cluster().num_blocks();
        spw = P.units;
        vec0 = rank * P.units * UNIT;
        base = reinterpret_cast<const char*>(P.logits) + (int64_t)row * P.stride * V::SIZE;
        head = (int)(reinterpret_cast<uintptr_t>(base) % 16) / V::SIZE;
        whole0 = head > 0;
        whole1 = (head + P.V) / EPV;
    }

    __device__ __forceinline__ void cluster_sync() const
    {
        if constexpr (RMEM) __syncthreads();
        else cg::this_cluster().sync();
    }
    template <class X>
    __device__ __forceinline__ const X* of_rank(const X* p, int r) const { return RMEM ? p : cg::this_cluster().map_shared_rank(p, r); }

    // every CTA's record, in sh.all
    __device__ __forceinline__ void exchange(Rec r)
    {
        if constexpr (RMEM) {
            __syncthreads();
            if (tid == 0) sh.all[0] = r;
        } else {
            // two places in turn: a CTA writes one again only behind the barrier that follows the others' reads
            Rec* at = &sh.mine[sh.step & 1];
            if (tid == 0) *at = r;
            cluster_sync();
            if (tid == 0) ++sh.step;
            if (tid < CL) sh.all[tid] = *of_rank(at, tid);
        }
        __syncthreads();
    }
    __device__ __forceinline__ u64 block_sum(u64 v) { return cta_sum(v, sh.warp); }
    // sum of v over the cluster's threads
    __device__ __forceinline__ u64 cluster_sum(u64 v)
    {
        const u64 s = block_sum(v);
        if constexpr (RMEM) return s;
        exchange({s, 0, 0});
        u64 all = 0;
        for (int i = 0; i < CL; ++i) all += sh.all[i].a;
        return all;
    }

    // vector i of this CTA's part, from memory: what of it is not the row's is -inf
    __device__ __noinline__ static uint4 edge(const char* base, int i, int head, int V_)
    {
        uint4 v = V::nothing();
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const int t = i * EPV + e - head;
            if (t >= 0 && t < V_) V::put(v, e, base, t);
        }
        return v;
    }
    __device__ __forceinline__ uint4 load(int i) const
    {
        i += vec0;
        if (i >= whole0 && i < whole1) return __ldg(reinterpret_cast<const uint4*>(base - head * V::SIZE + (size_t)i * 16));
        return edge(base, i, head, P.V);
    }
    __device__ __forceinline__ uint4 vec(int i) const
    {
        if constexpr (RMEM) return load(i);
        else return slice[i];
    }
    // f on this thread's vectors, the next one on its way.  (One copy of f: unrolled, the kernel outgrew the instruction caches, and
    // what runs once or twice a row waited for every line of itself.)
    template <class F>
    __device__ __forceinline__ void sweep(F f) const
    {
        const int first = w * spw * 32 + lane;
        uint4 next = vec(first);
#pragma unroll 1
        for (int s = 0; s < spw; ++s) {
            const uint4 v = next;
            if (s + 1 < spw) next = vec(first + (s + 1) * 32);
            f(v, first + s * 32);
        }
    }
    __device__ __forceinline__ int token(int vec, int e) const { return (vec0 + vec) * EPV + e - head; }
    // the warp of this CTA whose run holds a token; another number for other CTAs' tokens
    __device__ __forceinline__ int warp_of(int token) const
    {
        const int i = (token + head) / EPV - vec0;
        return i < 0 ? -1 : i / (spw * 32);
    }

    // the largest g in [-inf, top] for which f(g) holds, f falling with g, f(-inf) taken to hold
    template <class F>
    __device__ __forceinline__ float largest(F f)
    {
        uint32_t lo = key_of(NEG_INF), hi = key_of(top) + 1;  // holds, does not
#pragma unroll 1
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            if (f(float_of(mid))) lo = mid;
            else hi = mid;
        }
        return float_of(lo);
    }
    // this thread's logits, or their mass, at or above g
    __device__ __forceinline__ u64 thread_sum(bool count, float g) const
    {
        const Mass<DT> mass(c, sh.steps);
        Part m = {0, 0, 0};
        u64 n = 0;
        const auto at = V::bound(g);
        sweep([&](uint4 v, int) {
            if (count) n += __popc(V::flags(v, at));
            else if (V::keep(v, at)) mass.add(v, m);
        });
        return count ? n : m.whole();
    }

    // The logits at or above `cut` (but -inf) to this CTA's list; their number in the cluster.
    __device__ __forceinline__ int collect(float cut)
    {
        if (tid == 0) sh.count = 0;
        __syncthreads();
        const auto bound = V::bound(fmaxf(cut, -3.4028235e38f));
        sweep([&](const uint4& v, int i) { list(v, i, V::flags(v, bound)); });
        __syncthreads();
        exchange({0, (u64)sh.count, 0});
        int n = 0;
        for (int i = 0; i < CL; ++i) n += (int)sh.all[i].b;
        return n;
    }
    __device__ __forceinline__ void list(const uint4& v, int i, uint32_t hits)
    {
#pragma unroll 1
        for (; hits; hits &= hits - 1) {
            const int bit = __ffs(hits) - 1, at = atomicAdd(&sh.count, 1);
            if (at < LIST) {
                sh.l.lx[at] = V::flagged(v, bit);
                sh.l.lt[at] = token(i, V::place(bit));
            }
        }
    }
    // The CTAs' lists (sh.all[].b logits each, LIST in all at most) in sh.l.gx and gt, their masses in sh.l.gm.
    __device__ __forceinline__ void gather(int n)
    {
        const Mass<DT> mass(c, sh.steps);
#pragma unroll 1
        for (int i = tid; i < n; i += SNT) {
            int at = i, r = 0;
            while (at >= (int)sh.all[r].b) at -= (int)sh.all[r++].b;
            const float x = of_rank(sh.l.lx, r)[at];
            sh.l.gx[i] = x;
            sh.l.gt[i] = of_rank(sh.l.lt, r)[at];
            sh.l.gm[i] = mass.of(x);
        }
        __syncthreads();
    }

    // Bins of the logits at or above g0: bin i holds those with rint((upper - x) * per) = i, or counts them.  A mass at the distance f
    // from its bin's middle is 2^(-f width) of the middle's, 1 - f width ln 2 to 2^-15; width: octaves of a bin.
    __device__ __forceinline__ void fill(bool count, float g0, float upper, float per, float width)
    {
        constexpr float UP = 8388608.0f;  // 2^23
        const u64 from = two(-upper), per2 = two(-per), fall = two((1 << BIN_ONE) * -0.693147181f * width);
        const auto cut = V::bound(fmaxf(g0, upper - (float)BINS / per));
        sweep([&](uint4 v, int) {
            if (!V::keep(v, cut)) return;
#pragma unroll
            for (int e = 0; e < EPV; e += 2) {
                const u64 d = f2_add(f2_pack(V::elem(v, e), V::elem(v, e + 1)), from), r = f2_fma(d, per2, two(UP));
                float rx, ry, qx, qy;
                f2_unpack(r, rx, ry);
                f2_unpack(f2_fma(f2_fma(d, per2, f2_fma(r, two(-1.0f), two(UP))), fall, two(UP + (1 << BIN_ONE))), qx, qy);
                const uint32_t ix = __float_as_uint(rx) - 0x4b000000u, iy = __float_as_uint(ry) - 0x4b000000u;
                if (ix < (uint32_t)BINS) atomicAdd(&sh.l.bins[ix], count ? 1u : __float_as_uint(qx) - 0x4b000000u);
                if (iy < (uint32_t)BINS) atomicAdd(&sh.l.bins[iy], count ? 1u : __float_as_uint(qy) - 0x4b000000u);
            }
        });
    }
    __device__ __forceinline__ void clear_bins()
    {
        for (int i = tid; i < BINS; i += SNT) sh.l.bins[i] = 0;
        __syncthreads();
    }
    // The mass of the logits at or above g0, and its bins of 1 / 128 octave, from 2^(K + 1) down, as the masses have them anyway.
    __device__ __forceinline__ u64 mass_and_bins(float g0)
    {
        clear_bins();
        const Mass<DT> mass(c, sh.steps);
        Part m = {0, 0, 0};
        const auto at = V::bound(g0);
        const uint32_t first = 0x4b400000u * (FINE + 1) + (uint32_t)((c.K + 1) * STEPS * FINE);
        sweep([&](uint4 v, int) {
            if (!V::keep(v, at)) return;
#pragma unroll
            for (int e = 0; e < EPV; e += 2) {
                uint32_t ab[4], jx, jy;
                u64 r;
                mass.pair(V::elem(v, e), V::elem(v, e + 1), ab, jx, jy, r);
                m.add(ab[0], ab[1], ab[2], ab[3]);
                const u64 f = f2_fma(r, two((float)(STEPS * FINE)), two(Mass<DT>::MAGIC));  // which of the step's bins
                float fx, fy, qx, qy;
                f2_unpack(f, fx, fy);
                r = f2_fma(f2_add(f, two(-Mass<DT>::MAGIC)), two(-1.0f / (STEPS * FINE)), r);
                f2_unpack(f2_fma(r, two((1 << BIN_ONE) * 0.693147181f), two(8388608.0f + (1 << BIN_ONE))), qx, qy);
                const uint32_t ix = first - FINE * jx - __float_as_uint(fx), iy = first - FINE * jy - __float_as_uint(fy);
                if (ix < (uint32_t)BINS) atomicAdd(&sh.l.bins[ix], __float_as_uint(qx) - 0x4b000000u);
                if (iy < (uint32_t)BINS) atomicAdd(&sh.l.bins[iy], __float_as_uint(qy) - 0x4b000000u);
            }
        });
        return cluster_sum(m.whole());
    }

    // The threshold of top-k (count: the largest logit with `want` logits at or above it) or of top-p (the largest with mass `want`
    // at or above it, whose bins mass_and_bins() has filled) among the logits from g0 on.  False, and nothing, where that takes
    // bisection.  For top-p the mass that is kept is in `kept`, and of each warp's run in sh.sums (0: neither is known).
    __device__ __forceinline__ bool bracket(bool count, float g0, u64 want, float& g, u64& kept)
    {
        float upper, per, width;  // the middle of bin 0, bins of a unit of x, octaves of a bin
        if (count) {
            upper = top;
            per = BINS / 32.0f;  // (a guess: a k-th logit more than 32 under the largest takes bisection)
        } else {
            upper = (float)(c.K + 1) / c.hi + c.origin;
            per = STEPS * FINE * c.hi;
        }
        u64 over0 = 0;  // what lies above the bins
#pragma unroll 1
        for (int level = 0; level < 4; ++level) {
            width = c.hi / per;
            if (count || level > 0) {
                clear_bins();
                fill(count, g0, upper, per, width);
            }
            exchange({0, 0, 0});
            // every CTA sums the cluster's bins: some consecutive ones a thread, then over the threads
            constexpr int BPT = BINS / SNT;
            float m[BPT], s = 0.0f;
#pragma unroll
            for (int k = 0; k < BPT; k += 2) {
                uint32_t n0 = 0, n1 = 0;
                for (int r = 0; r < CL; ++r) {
                    const uint2 n = *reinterpret_cast<const uint2*>(of_rank(sh.l.bins, r) + tid * BPT + k);
                    n0 += n.x;
                    n1 += n.y;
                }
                const float at = (float)(tid * BPT + k);
                m[k] = count ? (float)n0 : (float)n0 * ex2(-(float)BIN_ONE - at * width);
                m[k + 1] = count ? (float)n1 : (float)n1 * ex2(-(float)BIN_ONE - (at + 1.0f) * width);
                s += m[k] + m[k + 1];
            }
            float upto = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += y;
            }
            if (lane == 31) sh.warp32[w] = __float_as_uint(upto);
            if (tid == 0) sh.from = BINS, sh.to = -1, sh.count = 0;
            __syncthreads();
            float before = 0.0f;  // up to this warp's bins
#pragma unroll 1
            for (int i = 0; i < w; ++i) before += __uint_as_float(sh.warp32[i]);
            // A thread's sums go on from the very number at which its neighbour's end: summed in another order the two would differ
            // in their last bits, and a level between them be met by two threads or by none.
            const float end = before + upto, prev = __shfl_up_sync(0xffffffffu, end, 1);
            if (lane > 0) before = prev;
            // bins' masses are right to 2^-13 together; counts are exact
            const float left = (float)(want - over0), tol = count ? 0.0f : left * 0x1p-12f;
            // (of the mass in the middle of bin 0)
            const float unit = count ? 1.0f : ex2(-fmaf(upper - c.origin, c.hi, (float)-c.K)) * 0x1p-44f;
            const float lo = (left - tol) * unit, hi = (left + tol) * unit;
#pragma unroll
            for (int k = 0; k < BPT; ++k) {
                const float after = k < BPT - 1 ? before + m[k] : end;
                // (sums of rounded terms may fall by their last bits and meet a level twice; all CTAs have the same ones, and go the same way)
                if (before < lo && after >= lo) atomicMin(&sh.from, tid * BPT + k);
                if (before < hi && after >= hi) atomicMax(&sh.to, tid * BPT + k);
                before = after;
            }
            __syncthreads();
            const int from = sh.from, to = sh.to < 0 ? BINS - 1 : sh.to;
            if (from == BINS) return false;
            // What lies above the bracket, and the bracket's logits.  (A quarter of a bin more on either side: at a bin's border the
            // two roundings may differ.)
            const float x1 = from == 0 && level == 0 ? __int_as_float(0x7f800000) : upper - ((float)from - 0.75f) / per;
            const float x0 = fmaxf(fmaxf(g0, upper - ((float)to + 0.75f) / per), -3.4028235e38f);
            const auto at1 = V::bound(x1), at0 = V::bound(x0);
            u64 over = 0;
            uint32_t kmin = 0xffffffffu, kmax = 0;
            {
                const Mass<DT> mass(c, sh.steps);
                Part part = {0, 0, 0};
                sweep([&](uint4 v, int i) {
                    if (!V::any(v, at0)) return;
                    const uint32_t above = V::flags(v, at1), hits = V::flags(v, at0) & ~above;
                    for (uint32_t h = hits; h; h &= h - 1) {
                        const uint32_t k = key_of(V::flagged(v, __ffs(h) - 1));
                        kmin = min(kmin, k);
                        kmax = max(kmax, k);
                    }
                    list(v, i, hits);
                    if (count) over += __popc(above);
                    else if (V::keep(v, at1)) mass.add(v, part);
                });
                if (!count) over = part.whole();
            }
            // of each warp's run, of the CTA, of the cluster; the bracket's ends
            over = warp_sum(over);
            kmin = __reduce_min_sync(0xffffffffu, kmin);
            kmax = __reduce_max_sync(0xffffffffu, kmax);
            if (lane == 0) {
                sh.sums[w] = over;
                sh.warp[w] = (u64)kmax << 32 | kmin;
            }
            __syncthreads();
            over = 0;
#pragma unroll 1
            for (int i = 0; i < SW; ++i) {
                over += sh.sums[i];
                kmax = max(kmax, (uint32_t)(sh.warp[i] >> 32));
                kmin = min(kmin, (uint32_t)sh.warp[i]);
            }
            exchange({over, (u64)sh.count, (u64)kmax << 32 | kmin});
            over = 0;
            int members = 0;
            for (int i = 0; i < CL; ++i) {
                over += sh.all[i].a;
                members += (int)sh.all[i].b;
                kmax = max(kmax, (uint32_t)(sh.all[i].c >> 32));
                kmin = min(kmin, (uint32_t)sh.all[i].c);
            }
            if (over >= want) return false;
            if (members > LIST && kmin == kmax) {  // ties: the group that they are
                g = float_of(kmin);
                kept = 0;
                return over + (u64)members * (count ? 1ull : Mass<DT>(c, sh.steps).of(g)) >= want;
            }
            if (members > LIST) {  // the bracket's own bins
                over0 = over;
                upper = fminf(x1, top);
                if (!(upper > x0)) return false;
                per = (float)(BINS - 1) / (upper - x0);
                continue;
            }
            gather(members);
            // the least that is kept, by its key
            uint32_t least = 0xffffffffu;
            u64 mine = 0;
            bool keep[LIST / SNT];
#pragma unroll
            for (int q = 0; q < LIST / SNT; ++q) {
                const int i = tid + q * SNT;
                keep[q] = false;
                if (i < members) {
                    const float x = sh.l.gx[i];
                    u64 larger = over;
                    for (int j = 0; j < members; ++j)
                        if (sh.l.gx[j] > x) larger += count ? 1ull : sh.l.gm[j];
                    if (larger < want) {
                        keep[q] = true;
                        least = min(least, key_of(x));
                        mine += count ? 1ull : sh.l.gm[i];
                    }
                }
            }
            least = __reduce_min_sync(0xffffffffu, least);
            if (lane == 0) sh.warp32[w] = least;
            kept = over + block_sum(mine);
#pragma unroll 1
            for (int i = 0; i < SW; ++i) least = min(least, sh.warp32[i]);
            if (!count) {  // what is kept of the bracket, by warps' runs
#pragma unroll
                for (int q = 0; q < LIST / SNT; ++q) {
                    const int i = tid + q * SNT;
                    if (i < members && !keep[q]) sh.l.gm[i] = 0;
                }
                __syncthreads();
                u64 share = 0;
                for (int j = lane; j < members; j += 32)
                    if (warp_of(sh.l.gt[j]) == w) share += sh.l.gm[j];
                share = warp_sum(share);
                if (lane == 0) sh.sums[w] += share;
            }
            __syncthreads();
            // the bracket has to hold the threshold: something of it is kept, and there is enough
            if (least == 0xffffffffu || kept < want) return false;
            g = float_of(least);
            return true;
        }
        return false;
    }

    // Rank 0, all of its threads: top-k, top-p and min-p (g) among the row's n candidates, and the draw among those left.
    __device__ __forceinline__ void pick(int row, int n, int k, float p, float u, float g)
    {
        constexpr int PER = LIST / SNT;
        gather(n);
        bool keep[PER], more;
        u64 over[PER], mine = 0;  // mass of the larger ones; of this thread's that are kept
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int i = tid + q * SNT;
            keep[q] = false;
            over[q] = 0;
            if (i >= n) continue;
            const float x = sh.l.gx[i];
            int above = 0;
            for (int j = 0; j < n; ++j)
                if (sh.l.gx[j] > x) {
                    ++above;
                    over[q] += sh.l.gm[j];
                }
            keep[q] = k == 0 || above < k;
            if (keep[q]) mine += sh.l.gm[i];
        }
        if (p < 1.0f) {
            const u64 want = scaled_floor(p, block_sum(mine), more);
            mine = 0;
#pragma unroll
            for (int q = 0; q < PER; ++q) {
                keep[q] = keep[q] && over[q] < want + more;
                if (keep[q] && sh.l.gx[tid + q * SNT] >= g) mine += sh.l.gm[tid + q * SNT];
            }
        } else {
            mine = 0;
#pragma unroll
            for (int q = 0; q < PER; ++q)
                if (keep[q] && sh.l.gx[tid + q * SNT] >= g) mine += sh.l.gm[tid + q * SNT];
        }
        const u64 z = block_sum(mine);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int i = tid + q * SNT;
            keep[q] = keep[q] && sh.l.gx[i] >= g;
            if (i < n && !keep[q]) sh.l.gm[i] = 0;
        }
        __syncthreads();
        const u64 t = scaled_floor(u, z, more);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            if (!keep[q]) continue;
            const int i = tid + q * SNT, tok = sh.l.gt[i];
            u64 before = 0;
            for (int j = 0; j < n; ++j)
                if (sh.l.gt[j] < tok) before += sh.l.gm[j];
            if (before <= t && t < before + sh.l.gm[i]) emit(row, tok, sh.l.gx[i], z);
        }
    }

    // token and, with the kept tokens' mass z = m 2^e, its logprob ln 2 (x c - K + 44 - e) - ln m
    __device__ __forceinline__ void emit(int row, int tok, float x, u64 z) const
    {
        P.tokens[row] = tok;
        if (P.logprob) {
            const float d = x - c.origin, f = (float)z;
            const int e = (int)(__float_as_uint(f) >> 23) - 127 + (int)(__float_as_uint(f) >> 22 & 1u);  // m in [0.75, 1.5)
            const float o = fmaf(d, c.lo, fmaf(d, c.hi, (float)(44 - e - c.K)));
            P.logprob[row] = fmaf(o, 0.693147182f, -logf(f * exp2_int(-e)));
        }
    }

    // The j-th largest of this CTA's threads' values, in steps of 2^16 of its key: at least j of them lie at or above it.  Two j at a
    // time, a warp each.
    __device__ __forceinline__ void jth(float v, int j0, int j1)
    {
        sh.l.gt[tid] = (int)(key_of(v) >> 16);
        __syncthreads();
        if (w < 2) {
            const int j = w ? j1 : j0;
            uint32_t k[SNT / 32], lo = 0;
#pragma unroll
            for (int i = 0; i < SNT / 32; ++i) k[i] = (uint32_t)sh.l.gt[lane + 32 * i];
#pragma unroll 1
            for (int bit = 15; bit >= 0; --bit) {
                uint32_t n = 0;
#pragma unroll
                for (int i = 0; i < SNT / 32; ++i) n += k[i] >= (lo | 1u << bit);
                if ((int)__reduce_add_sync(0xffffffffu, n) >= j) lo |= 1u << bit;
            }
            const float g = float_of(lo << 16);
            if (lane == 0) sh.bound[w] = lo == 0 || !(g > NEG_INF) ? NEG_INF : g;  // (the key of a NaN lies under that of -inf)
        }
        __syncthreads();
    }
};

// The draw, with the masses of the warps' runs in sh.sums.  of(v): the mass of a vector's elements that are kept; one(x): of an
// element.  The run that holds the uniform's place is summed again, 32 vectors at a time, by all warps; warp 0 does the rest.
template <int DT, bool RMEM, class Of, class One>
__device__ __forceinline__ void draw_run(Row<DT, RMEM>& R, int row, float u, Of of, One one)
{
    constexpr int EPV = Vec<DT>::N;
    auto& sh = R.sh;
    bool more;
    __syncthreads();
    u64 cta = 0;
#pragma unroll 1
    for (int i = 0; i < SW; ++i) cta += sh.sums[i];
    R.exchange({cta, 0, 0});
    u64 z = 0, before = 0;
    for (int i = 0; i < R.CL; ++i) {
        if (i < R.rank) before += sh.all[i].a;
        z += sh.all[i].a;
    }
    const u64 t = scaled_floor(u, z, more);
    if (t < before || t >= before + cta) return;  // another CTA's
    int run = 0;
#pragma unroll 1
    for (u64 m; run < SW - 1 && t >= before + (m = sh.sums[run]); ++run) before += m;
    const int first = run * R.spw * 32 + R.lane;
#pragma unroll 1
    for (int s = R.w; s < R.spw; s += SW) {
        uint4 v = R.vec(first + s * 32);
        const u64 m = warp_sum(of(v));
        if (R.lane == 0) sh.l.gm[s] = m;
    }
    __syncthreads();
    if (R.w != 0) return;
    int s = 0;
#pragma unroll 1
    for (u64 m; s < R.spw - 1 && t >= before + (m = sh.l.gm[s]); ++s) before += m;
    uint4 v = R.vec(first + s * 32);
    const u64 own = of(v);
    u64 from = before + warp_scan(own) - own;
#pragma unroll 1
    for (int e = 0; from <= t && e < EPV; ++e) {
        const float x = Vec<DT>::elem(v, e);
        const u64 m = one(x);
        if (t < from + m) {
            R.emit(row, R.token(first + s * 32, e), x, z);
            break;
        }
        from += m;
    }
}

// top-p among the logits from gk on, then the draw among those that it and min-p (g) keep
template <int DT, bool RMEM>
__device__ __forceinline__ void draw(Row<DT, RMEM>& R, int row, float u, float p, float gk, float g)
{
    typedef Vec<DT> V;
    auto& sh = R.sh;
    u64 z = 0;
    bool have = false, more;  // z, and the warps' sums in sh.sums
    g = fmaxf(g, gk);
    if (p < 1.0f) {
        const u64 whole = R.mass_and_bins(gk);
        u64 want = scaled_floor(p, whole, more);
        want += more;  // a whole number is under p * whole where it is under this
        float gp;
        if (R.bracket(false, gk, want, gp, z)) have = z > 0 && gp >= g;
        else gp = R.largest([&](float at) { return R.cluster_sum(R.thread_sum(false, fmaxf(at, gk))) >= want; });
        g = fmaxf(g, gp);
    }
    if (!have) {
        const u64 mass = warp_sum(R.thread_sum(false, g));
        if (R.lane == 0) sh.sums[R.w] = mass;
    }
    const Mass<DT> mass(R.c, sh.steps);
    const auto at = V::bound(g);
    draw_run(
        R, row, u,
        [&](uint4& v) {
            Part part = {0, 0, 0};
            if (V::keep(v, at)) mass.add(v, part);
            return part.whole();
        },
        [&](float x) { return mass.of(x); });
}

// Rows of bf16: top-k, top-p and min-p (g) from the counts of the row's values, and the draw.
//
// A bf16 logit has one of 2^16 values, so what a sweep has to do is count: the masses are formed once a value, and sums over values are
// the sums over tokens that they were.  The values that have mass lie between `low` and the largest logit, and those of them within
// 31 octaves of the largest magnitude have a place each, [sign][MAGS]; smaller ones share place 0 with the zeros, and what is larger has no
// mass and place MAGS - 1.  The sweep for the largest logit counts by the way (`done`), as if it were 64; what does not fit is counted
// again.  Ranks go through them from the largest value on: rank r is place MAGS - 1 - r, or r; the zero of the second half is taken with
// the first's.  The CTAs of a cluster share the groups of 32 ranks out, each of which sums the counts of all for its own.  False, and nothing,
// where a logit in place 0 is no zero and may have mass.  `mass`: 2 MAGS of them, for the sweep that draws where a row is one CTA.
//
// (512 rows of 152064 with top-p: 111 us; 118 with loads that L1 may not keep, 132 with the counts as a sweep of their own and the
// loads of the drawing sweep one ahead, 300 with a mass a logit and the bracket of bins.  One row, by eight CTAs: 17 us; 35 where each
// of them sums all counts of all, 34 with the bracket.)
struct Places {
    uint32_t shift;
    __device__ __forceinline__ explicit Places(int base) : shift((uint32_t)(-base & 0xffff) * 0x10001u) {}
    // of a word's two logits
    __device__ __forceinline__ uint32_t of(uint32_t q) const
    {
        static_assert(MAGS == 0x8000 >> 3, "the sign's bit is the second half");
        return __viaddmin_s16x2_relu(q & 0x7fff7fffu, shift, (MAGS - 1) * 0x10001u) | (q & 0x80008000u) >> 3;
    }
    __device__ __forceinline__ void count(const uint4& v, uint32_t* n) const
    {
        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t at = of(q[e]);
            atomicAdd(n + (at & 0xffffu), 1u);
            atomicAdd(n + (at >> 16), 1u);
        }
    }
};
__host__ __device__ constexpr int base_of(uint32_t largest) { return (int)largest > MAGS - 2 ? (int)largest - (MAGS - 2) : 0; }

template <bool RMEM>
__device__ __forceinline__ bool counted(Row<DT_BF16, RMEM>& R, int row, float u, int k, float p, float g, bool done, u64* mass)
{
    typedef Vec<DT_BF16> V;
    auto& sh = R.sh;
    constexpr int GROUPS = 2 * MAGS / 32;
    const float low = ((float)R.c.K - 46.0f) / R.c.hi + R.c.origin;
    uint32_t largest = R.top > 0.0f ? __float_as_uint(R.top) >> 16 : 0u;
    if (low < 0.0f) largest = max(largest, (__float_as_uint(-low) >> 16) + 1);
    done = done && largest <= GUESS;
    const int base = base_of(done ? GUESS : largest);
    const Places places(base);
    const auto place_of = [](int r) { return r < MAGS ? MAGS - 1 - r : r; };
    const auto value_of = [&](int i) {  // of a place; place 0: zero
        return i % MAGS ? __uint_as_float((uint32_t)(i % MAGS + base) << 16 | (uint32_t)(i / MAGS) << 31) : 0.0f;
    };
    const auto dead = [](int i) { return i == MAGS || i % MAGS == MAGS - 1; };  // no value, or the zero that is counted elsewhere
    const auto owner = [&](int grp) { return RMEM ? 0 : grp / SW % R.CL; };
    if (!done) {
        R.exchange({0, 0, 0});  // the lists have been read
        for (int i = R.tid; i < 2 * MAGS; i += SNT) sh.v.n[i] = 0;
        __syncthreads();
        R.sweep([&](const uint4& v, int) { places.count(v, sh.v.n); });
        __syncthreads();
    }
    const uint32_t zeros = sh.v.n[0] + sh.v.n[MAGS];
    bool tiny = false;
    // (of place 0, magnitudes up to 2^16 base's: where the first sweep's places are for larger logits, all of the mass may lie in it)
    if (zeros && base > 0 && low <= __uint_as_float((uint32_t)base << 16)) {
        u64 all = 0;
        R.sweep([&](const uint4& v, int) {
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) all += (unsigned)((q[e] & 0x7fffu) == 0) + (unsigned)((q[e] & 0x7fff0000u) == 0);
        });
        tiny = R.block_sum(all) != zeros;
    }
    R.exchange({tiny, 0, 0});
    for (int r = 0; r < R.CL; ++r) tiny = tiny || sh.all[r].a;
    if (tiny) return false;
    // the masses, and the sums of 32 ranks; a group's counts are its owner's from here on
    {
        const Mass<DT_BF16> ms(R.c, sh.steps);
#pragma unroll 2
        for (int grp = R.rank * SW + R.w; grp < GROUPS; grp += SW * R.CL) {
            const int i = place_of(grp * 32 + R.lane);
            uint32_t n = 0;
            if constexpr (RMEM) {
                n = sh.v.n[i];
            } else {
#pragma unroll
                for (int r = 0; r < MAX_CL; ++r)
                    if (r < R.CL) n += R.of_rank(sh.v.n, r)[i];
            }
            if (i == 0)
                for (int r = 0; r < R.CL; ++r) n += R.of_rank(sh.v.n, r)[MAGS];
            if (dead(i)) n = 0;
            else if (!RMEM || i == 0) sh.v.n[i] = n;
            u64 m = 0, sum = 0;
            uint32_t ns = 0;
            if (__any_sync(0xffffffffu, n)) {
                m = n ? ms.of(value_of(i)) : 0;
                sum = warp_sum(m * n);
                ns = __reduce_add_sync(0xffffffffu, n);
            }
            if (R.lane == 0) sh.v.group_mass[grp] = sum, sh.v.group_n[grp] = ns;
            if constexpr (RMEM) mass[i] = m;
        }
    }
    if constexpr (RMEM) {
        __syncthreads();
    } else {
        R.exchange({0, 0, 0});
        if (R.tid < GROUPS && owner(R.tid) != R.rank) {
            sh.v.group_mass[R.tid] = R.of_rank(sh.v.group_mass, owner(R.tid))[R.tid];
            sh.v.group_n[R.tid] = R.of_rank(sh.v.group_n, owner(R.tid))[R.tid];
        }
        __syncthreads();
    }
    if (R.w == 0) {
        // top-k's last rank by the counts, then top-p's by the masses: the first up to which there are as many, or as much.  32 lanes have
        // the groups of ranks between them; then a group's ranks.
        constexpr int PER = GROUPS / 32;
        int end = 2 * MAGS - 1;
        u64 ms = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) ms += sh.v.group_mass[R.lane * PER + j];
        const u64 upto_m = warp_scan(ms);
        u64 z = __shfl_sync(0xffffffffu, upto_m, 31);  // of what is kept so far
#pragma unroll 1
        for (int step = k > 0 ? 0 : 1; step < (p < 1.0f ? 2 : 1); ++step) {
            const bool count = step == 0;
            u64 want = (u64)k, s = ms, upto = upto_m;
            if (count) {
                s = 0;
#pragma unroll
                for (int j = 0; j < PER; ++j) s += sh.v.group_n[R.lane * PER + j];
                upto = warp_scan(s);
            } else {
                bool more;
                want = scaled_floor(p, z, more);
                want += more;
            }
            const unsigned there = __ballot_sync(0xffffffffu, upto >= want);
            if (!there) continue;  // top-k ends among what has no mass
            const int src = __ffs(there) - 1;
            int grp = src * PER;
            u64 before = __shfl_sync(0xffffffffu, upto - s, src), before_m = __shfl_sync(0xffffffffu, upto_m - ms, src), n;
#pragma unroll 1
            for (; before + (n = count ? sh.v.group_n[grp] : sh.v.group_mass[grp]) < want; ++grp) {
                before += n;
                before_m += sh.v.group_mass[grp];
            }
            const int i = place_of(grp * 32 + R.lane);
            const uint32_t here = dead(i) ? 0 : R.of_rank(sh.v.n, owner(grp))[i];
            const u64 own = here * (RMEM ? mass[i] : Mass<DT_BF16>(R.c, sh.steps).of(value_of(i))), b = warp_scan(own),
                      a = count ? warp_scan(here) : b;
            const int l = __ffs(__ballot_sync(0xffffffffu, before + a >= want)) - 1;
            z = before_m + __shfl_sync(0xffffffffu, b, l);
            end = min(end, grp * 32 + l);
        }
        if (R.lane == 0) sh.to = end;
    }
    __syncthreads();
    const int end = sh.to;
    if (end < 2 * MAGS - 1) g = fmaxf(g, value_of(place_of(end)));
    if constexpr (!RMEM) {
        draw(R, row, u, 1.0f, g, g);
    } else {
        for (int r = R.tid; r < 2 * MAGS; r += SNT) {
            const int i = place_of(r);
            if (r > end || value_of(i) < g) mass[i] = 0;
        }
        __syncthreads();
        if (R.tid == 0) mass[MAGS] = mass[0];
        __syncthreads();
        const auto at = V::bound(g);
        const auto of = [&](const uint4& v) {
            u64 sum = 0;
            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t i = places.of(q[e]);
                sum += mass[i & 0xffffu] + mass[i >> 16];
            }
            return sum;
        };
        u64 sum = 0;
        {
            constexpr int LU = 4;
            const int first = R.w * R.spw * 32 + R.lane;
#pragma unroll 1
            for (int s = 0; s < R.spw; s += LU) {
                uint4 v[LU];
#pragma unroll
                for (int j = 0; j < LU; ++j)
                    if (s + j < R.spw) v[j] = R.load(first + (s + j) * 32);
#pragma unroll
                for (int j = 0; j < LU; ++j)
                    if (s + j < R.spw && V::any(v[j], at)) sum += of(v[j]);
            }
        }
        sum = warp_sum(sum);
        if (R.lane == 0) sh.sums[R.w] = sum;
        draw_run(R, row, u, of, [&](float x) { return mass[places.of(__float_as_uint(x) >> 16) & 0xffffu]; });
    }
    return true;
}

template <int DT, bool RMEM>
__global__ void __launch_bounds__(SNT, 2) sample_kernel(const __grid_constant__ SampleParams P)
{
    typedef Vec<DT> V;
    constexpr int EPV = V::N;
    extern __shared__ uint4 slice[];
    __shared__ typename Row<DT, RMEM>::Sh sh;
    constexpr bool COUNTS = Row<DT, RMEM>::COUNTS;
    const int row = RMEM ? blockIdx.x : blockIdx.x / cg::this_cluster().num_blocks();
    Row<DT, RMEM> R(P, sh, slice, row);
    const int tid = R.tid, CL = R.CL;
    for (int i = tid; i < STEPS * 32; i += SNT) {
        sh.steps[i] = EXP2_STEPS[i / 32].x;
        sh.steps[Mass<DT>::SECOND + i] = EXP2_STEPS[i / 32].y;
    }
    if (tid == 0) sh.step = 0;

    // ---- what was asked for
    const float u = __ldg(P.uniforms + row);
    const float T = P.temperature ? __ldg(P.temperature + row) : 1.0f;
    int k = P.top_k ? __ldg(P.top_k + row) : 0;
    const float p = P.top_p ? __ldg(P.top_p + row) : 1.0f, mp = P.min_p ? __ldg(P.min_p + row) : 0.0f;
    const bool bad_param = !(T >= 0.0f && T <= SAMPLE_MAX_T) || (T > 0.0f && T < SAMPLE_MIN_T) || k < 0 || !(p > 0.0f) ||
                           !(mp >= 0.0f && mp <= 1.0f);
    if (k >= P.V) k = 0;

    // ---- this thread's largest logit, NaN where it has met one
    float mine = NEG_INF;
    const bool few = k > 0 && k <= SNT && T > 0.0f;
    const bool count = COUNTS && (k > 0 || p < 1.0f) && !few && T > 0.0f;
    if constexpr (COUNTS)
        if (count) {
            for (int i = tid; i < 2 * MAGS; i += SNT) sh.v.n[i] = 0;
            __syncthreads();
        }
    {
        constexpr int LU = 4;  // vectors in flight
        const int first = R.w * R.spw * 32 + R.lane;
#pragma unroll 1
        for (int s = 0; s < R.spw; s += LU) {
            uint4 v[LU];
#pragma unroll
            for (int j = 0; j < LU; ++j)
                if (s + j < R.spw) v[j] = R.load(first + (s + j) * 32);
#pragma unroll
            for (int j = 0; j < LU; ++j)
                if (s + j < R.spw) {
                    if (!RMEM) slice[first + (s + j) * 32] = v[j];
                    if constexpr (COUNTS)
                        if (count) Places(base_of(GUESS)).count(v[j], sh.v.n);
                    mine = fmax_nan(mine, V::max_nan(v[j]));
                }
        }
    }

    // ---- the row's largest logit, and a bound under its k-th
    const bool odd = !(mine < __int_as_float(0x7f800000));  // NaN or +inf
    {
        const uint32_t kmax = __reduce_max_sync(0xffffffffu, odd ? key_of(__int_as_float(0x7f800000)) : key_of(mine));
        if (R.lane == 0) sh.warp32[R.w] = kmax;
    }
    __syncthreads();
    uint32_t ktop = 0;
    for (int i = 0; i < SW; ++i) ktop = max(ktop, sh.warp32[i]);
    float share = NEG_INF, local = NEG_INF;
    if (few) {
        // at least k logits lie at or above the k-th largest of one CTA's threads' maxima, and at or above the least of the
        // CTAs' (k / CL)-th largest
        R.jth(odd ? NEG_INF : mine, (k + CL - 1) / CL, k);
        share = sh.bound[0];
        local = sh.bound[1];
    }
    R.exchange({(u64)ktop << 32 | __float_as_uint(local), __float_as_uint(share), 0});
    float cut = __int_as_float(0x7f800000), cut2 = NEG_INF;
    ktop = 0;
    for (int i = 0; i < CL; ++i) {
        ktop = max(ktop, (uint32_t)(sh.all[i].a >> 32));
        cut2 = fmaxf(cut2, __uint_as_float((uint32_t)sh.all[i].a));
        cut = fminf(cut, __uint_as_float((uint32_t)sh.all[i].b));
    }
    cut = fmaxf(cut, cut2);
    const float top = R.top = float_of(ktop);
    int status = ROW_OK;
    if (!(top < __int_as_float(0x7f800000)) || !(top > NEG_INF)) status = ROW_NONFINITE;
    else if (!(u >= 0.0f && u < 1.0f)) status = ROW_BAD_UNIFORM;
    else if (bad_param) status = ROW_BAD_PARAM;
    if (R.rank == 0 && tid == 0) {
        if (P.row_status) P.row_status[row] = status;
        if (status != ROW_OK) {
            P.tokens[row] = -1;
            if (P.logprob) P.logprob[row] = __int_as_float(0x7fc00000);
        }
    }
    if (status != ROW_OK) {
        // nothing more
    } else if (T == 0.0f) {
        // ---- greedy: the first of the largest logits
        uint32_t at = 0xffffffffu;
        const auto bound = V::bound(top);
        R.sweep([&](const uint4& v, int i) {
            if (!V::any(v, bound)) return;
#pragma unroll
            for (int e = EPV - 1; e >= 0; --e)
                if (V::elem(v, e) == top) at = min(at, (uint32_t)R.token(i, e));
        });
        at = __reduce_min_sync(0xffffffffu, at);
        if (R.lane == 0) sh.warp32[R.w] = at;
        __syncthreads();
        for (int i = 0; i < SW; ++i) at = min(at, sh.warp32[i]);
        R.exchange({at, 0, 0});
        if (R.rank == 0 && tid == 0) {
            for (int i = 0; i < CL; ++i) at = min(at, (uint32_t)sh.all[i].a);
            P.tokens[row] = (int)at;
            if (P.logprob) P.logprob[row] = 0.0f;
        }
    } else {
        // ---- the scale: log2(e) as a pair, over T
        constexpr float E_HI = 1.44269502f, E_LO = 1.92596299e-8f;
        R.c.hi = __fdiv_rn(E_HI, T);
        if (DT == DT_BF16) R.c.hi = __uint_as_float(__float_as_uint(R.c.hi) & 0xffffff00u);  // 16 bits: see Mass
        R.c.lo = __fdiv_rn(__fadd_rn(fmaf(-R.c.hi, T, E_HI), E_LO), T);
        R.c.origin = fabsf(top * R.c.hi) < FAR_OCTAVES<DT> ? 0.0f : top;
        R.c.K = (int)rintf((top - R.c.origin) * R.c.hi);
        float g = NEG_INF;
        if (mp > 0.0f) {  // min-p
            if (tid == 0) sh.least = __double2float_ru((double)top + (double)T * log((double)mp));
            __syncthreads();
            g = fminf(sh.least, top);
        }
        int n = LIST + 1;
        if (few || (mp > 0.0f && k == 0 && p >= 1.0f)) n = R.collect(few ? cut : g);
        if (n <= LIST) {  // the rest is rank 0's
            if (R.rank == 0) R.pick(row, n, k, p, u, g);
        } else {
            bool drawn = false;
            if constexpr (COUNTS) drawn = (k > 0 || p < 1.0f) && counted(R, row, u, k, p, g, count, reinterpret_cast<u64*>(slice));
            if (!drawn) {
                float gk = NEG_INF;
                u64 all;
                if (k > 0 && !R.bracket(true, NEG_INF, (u64)k, gk, all))
                    gk = R.largest([&](float at) { return R.cluster_sum(R.thread_sum(true, at)) >= (u64)k; });
                draw(R, row, u, p, gk, g);
            }
        }
    }
    R.cluster_sync();  // no CTA leaves while another may read its records and lists
}

template <int DT>
cudaError_t launch_type(SampleParams& P, int sms, cudaStream_t st)
{
    constexpr int EPV = Vec<DT>::N;
    const int units = units_of(P.V, EPV);
    // with few rows as many CTAs as the GPU has room for
    const int room = sms / P.N;
    const int most_units = SAMPLE_UNITS - (DT == DT_BF16);  // beside the counts
    int cl = (units + most_units - 1) / most_units;
    cl = cl > room ? cl : room;
    cl = cl < units ? cl : units;
    cl = cl < MAX_CL ? cl : MAX_CL;
    // A row as one CTA: from three quarters of a row an SM on (96 rows of 50257 in fp32 with mixed settings take 37 us as clusters, 54 as a
    // CTA each; 100 of 152064 in bf16 without top-k and top-p 45 and 40).  In fp32 that border is too late for the widest rows, whose clusters
    // come in waves: with top-p 32, 64 and 113 rows of 152064, one CTA an SM, take 103, 172 and 280 us and 114 as a CTA each 100; of 128256
    // 53, 96 and 152, and 85; of 50257 26, 36 and 56, and 41.  Of bf16, where top-k or top-p may need the counts, also where the
    // clusters would come in two waves (64 rows of 152064 with top-p 44 us as clusters and 36 as a CTA each, 48 rows 30 and 43, one row 17
    // and 34), and some short rows, over which a cluster's steps are long (of 32000 48 rows 21 and 16, 32 rows 15 and 16, one row 13 and 15).
    const bool one = P.N >= sms - sms / 4 ||
                     (DT == DT_BF16 && (P.top_k || P.top_p) && (P.N * cl > 2 * sms || (units <= SAMPLE_UNITS - 1 && P.N >= sms / 4)));
    if (one) {
        P.units = units;
        const size_t table = DT == DT_BF16 ? 2 * MAGS * sizeof(u64) : 0;
        static PerDevice set;
        int& done = set.here();
        if (!done) {
            const cudaError_t e = cudaFuncSetAttribute(sample_kernel<DT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)table);
            if (e != cudaSuccess) return e;
            done = 1;
        }
        sample_kernel<DT, true><<<(unsigned)P.N, SNT, table, st>>>(P);
        return cudaGetLastError();
    }
    P.units = (units + cl - 1) / cl;
    cl = (units + P.units - 1) / P.units;
    const size_t smem = (size_t)P.units * UNIT * 16;
    auto* kern = sample_kernel<DT, false>;
    // (set once, to what the widest row takes: threads that call at once do not lower each other's)
    constexpr int WIDEST = units_of(SAMPLE_MAX_V, EPV), EACH = (WIDEST + MAX_CL - 1) / MAX_CL;
    constexpr int MOST = (EACH > SAMPLE_UNITS ? EACH : SAMPLE_UNITS) * UNIT * 16;
    static PerDevice kept;
    int& done = kept.here();
    if (!done) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST);
        if (e != cudaSuccess) return e;
        done = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(P.N * cl));
    cfg.blockDim = dim3(SNT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cl;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P);
}

}  // namespace

cudaError_t launch_sample_logits(SampleParams& P, int dtype, int sms, cudaStream_t st)
{
    return dtype == DT_BF16 ? launch_type<DT_BF16>(P, sms, st) : launch_type<DT_F32>(P, sms, st);
}

}  // namespace sv
