// sv_pages.cu -- kv_pages_reserve and kv_pages_release: page tables and slot maps from the requests' lengths.
//
// Free pages are a stack: free_pages[0 .. count).  With need_b = ceil((lens_b + n_new_b) / page) and grow_b = max(0, need_b -
// held_b), request b's new pages are the stack's entries count - 1 - (first_b + i), first_b = sum of grow_j over j < b: a prefix sum
// over the batch, so the tables do not depend on scheduling.  A request is served when first_b + grow_b <= count; the
// sums only grow, so what the served ones took is the top of the stack without a gap.  A release pushes in the same order.
//
// Nothing that a request reads is written by another one's work: new pages are read from the stack, never back from the
// table; held and count are written last.  A small batch is one CTA, which sums, writes and commits; otherwise every
// CTA sums what stands before its request (B words from L2) and writes its share, and a second kernel commits what
// all of them have read.
//
// What bounds it: latency, dependent reads and a prefix sum over the batch; with long prompts the slot map's writes.  On the GPU a
// reservation for 256 requests of a round and the release after it take 8 us, for 64 prompts (524,000 rows) and their release 14.  Past 1024
// requests every request's CTAs sum what stands before it, together half a square of the batch: 1024 requests take 21 us, 3000 40,
// 8192 161, 16384 516 and 65535 7 ms.
#include "sv_round.cuh"

namespace sv {

namespace {

constexpr int ONE_NT = 1024, FILL_NT = 256;
// What one CTA does alone: rows, beside four a request, of a reservation (with a release, as one CTA and as two kernels: 256 requests of
// 6 rows 6.3 and 8.0 us, 1024 of 7 10.9 and 13.2, 64 of 64 8.6 and 8.6, of 128 11.3 and 8.9, of 512 23.6 and 9.1), and a table's entries
// of a release, which as a rule gives few of them back (where 64 requests give back all of 512, with the reservation 14 us as one
// CTA and 11 as two kernels, whose second launch costs the host as much).
constexpr int ONE_ROWS = 1 << 12, ONE_ENTRIES = 1 << 16;

struct Grow {
    int len, rows, held, status;
    long long n;  // pages it takes (or gives back)
};

__device__ __forceinline__ Grow grow_of(const PagesParams& P, int b)
{
    Grow g;
    g.len = __ldg(P.lens + b);
    g.held = P.held[b];
    g.rows = P.n_new ? __ldg(P.n_new + b) : P.max_new;
    g.status = ROW_OK;
    g.n = 0;
    const long long have = ((long long)g.len + P.page - 1) >> P.page_shift;
    if (g.len < 0 || g.held < 0 || g.held > P.table_width || (P.release && have > g.held)) {
        g.status = ROW_BAD_LENGTH;
    } else if (P.release) {
        g.n = g.held - have;
    } else {
        const long long need = ((long long)g.len + g.rows + P.page - 1) >> P.page_shift;
        if (g.rows < 0 || g.rows > P.max_new || need > P.table_width) g.status = ROW_BAD_LENGTH;
        else if (need > g.held) g.n = need - g.held;
    }
    return g;
}

// pages that the stack has (a reservation), or has room for (a release)
__device__ __forceinline__ long long room_of(const PagesParams& P, int count)
{
    if (count < 0 || count > P.capacity) return 0;  // no stack: nobody is served
    return P.release ? P.capacity - count : count;
}

// inclusive sums over a CTA of NT threads
template <int NT>
__device__ long long block_scan(long long v, long long* sh)
{
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    if (lane == 31) sh[w] = v;
    __syncthreads();
    if (w == 0) {
        long long s = lane < NT / 32 ? sh[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += x;
        }
        if (lane < NT / 32) sh[lane] = s;
    }
    __syncthreads();
    if (w > 0) v += sh[w - 1];
    __syncthreads();
    return v;
}

// Row t of request b: its slot, and the table's entry where the row is the first of a new page.  (The pages of a length that passes
// those held begin before the new rows: the callers write these.)
__device__ __forceinline__ void reserve_row(const PagesParams& P, int b, int t, int len, int rows, int held, bool served, long long first, int count)
{
    long long slot = -1;
    if (served && t < rows) {
        const int pos = len + t, i = pos >> P.page_shift, in = pos & (P.page - 1);
        int page;
        if (i < held) {
            page = P.page_table[(size_t)b * P.table_width + i];
        } else {
            page = __ldg(P.free_in + (count - 1 - (first + i - held)));
            if (in == 0) P.page_table[(size_t)b * P.table_width + i] = page;
        }
        slot = (long long)page * P.page + in;
    }
    if (P.slots) P.slots[(size_t)b * P.max_new + t] = slot;
}

// the entry of new page i of a request
__device__ __forceinline__ void reserve_page(const PagesParams& P, int b, int i, int held, long long first, int count)
{
    P.page_table[(size_t)b * P.table_width + i] = __ldg(P.free_in + (count - 1 - (first + i - held)));
}

__device__ __forceinline__ void commit(const PagesParams& P, int b, const Grow& g, bool served)
{
    if (served && g.n) P.held[b] = g.held + (P.release ? -(int)g.n : (int)g.n);
    if (P.row_status) P.row_status[b] = g.status != ROW_OK ? g.status : served ? ROW_OK : ROW_NO_PAGES;
}

__global__ void __launch_bounds__(ONE_NT) pages_one_kernel(const __grid_constant__ PagesParams P)
{
    struct Req {
        int len, rows, held;
        int first;  // -1: not served
    };
    __shared__ Req req[ONE_NT];
    __shared__ long long sh[32];
    const int b = threadIdx.x, count = *P.count;
    Grow g = {};
    if (b < P.B) g = grow_of(P, b);
    const long long last = block_scan<ONE_NT>(g.n, sh), room = room_of(P, count);
    const bool served = g.status == ROW_OK && (g.n == 0 || last <= room);
    // first fits 32 bits where it is used: a served request's pages lie on the stack
    if (b < P.B) req[b] = {g.len, P.release ? (int)g.n : g.rows, g.held, served ? (int)(g.n ? last - g.n : 0) : -1};
    const long long moved = block_scan<ONE_NT>(served ? g.n : 0, sh);
    __syncthreads();
    if (P.release) {
        for (int r = threadIdx.x >> 5; r < P.B; r += ONE_NT / 32) {
            const Req q = req[r];
            if (q.first < 0) continue;
            const int32_t* from = P.page_table + (size_t)r * P.table_width + q.held - q.rows;
            int32_t* to = P.free_out + count + q.first;
#pragma unroll 4
            for (int i = threadIdx.x & 31; i < q.rows; i += 32) to[i] = __ldg(from + i);  // (a release writes no table)
        }
    } else {
        const unsigned items = (unsigned)P.B * (unsigned)P.max_new;
        for (unsigned i = threadIdx.x; i < items; i += ONE_NT) {
            const unsigned r = i / (unsigned)P.max_new;
            const Req q = req[r];
            reserve_row(P, (int)r, (int)(i - r * (unsigned)P.max_new), q.len, q.rows, q.held, q.first >= 0, q.first, count);
        }
        // lengths past the pages held, which are few if any: a warp's requests one by one
        const auto pages_of = [&](int len) { return (int)(((long long)len + P.page - 1) >> P.page_shift); };
        for (unsigned m = __ballot_sync(0xffffffffu, b < P.B && served && pages_of(g.len) > g.held); m; m &= m - 1) {
            const int r = (b & ~31) + __ffs(m) - 1;
            const Req q = req[r];
            for (int i = q.held + (b & 31); i < pages_of(q.len); i += 32) reserve_page(P, r, i, q.held, q.first, count);
        }
    }
    __syncthreads();  // held has been read by all
    if (b < P.B) commit(P, b, g, served);
    if (b == ONE_NT - 1 && moved) *P.count = count + (P.release ? (int)moved : -(int)moved);
}

// CTA (x, b): request b's share x
__global__ void __launch_bounds__(FILL_NT) pages_fill_kernel(const __grid_constant__ PagesParams P)
{
    __shared__ long long sh[FILL_NT / 32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = blockIdx.y, count = *P.count;
    long long before = 0;
    for (int j = threadIdx.x; j < b; j += FILL_NT) before += grow_of(P, j).n;
#pragma unroll
    for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = before;
    __syncthreads();
    before = 0;
#pragma unroll
    for (int w = 0; w < FILL_NT / 32; ++w) before += sh[w];
    const Grow g = grow_of(P, b);
    const bool served = g.status == ROW_OK && (g.n == 0 || before + g.n <= room_of(P, count));
    const int step = gridDim.x * FILL_NT, at = blockIdx.x * FILL_NT + threadIdx.x;
    if (P.release) {
        if (served)
            for (int i = at; i < g.n; i += step)
                P.free_out[count + before + i] = __ldg(P.page_table + (size_t)b * P.table_width + g.held - g.n + i);
    } else {
        for (int t = at; t < P.max_new; t += step) reserve_row(P, b, t, g.len, g.rows, g.held, served, before, count);
        if (served)
            for (long long i = g.held + at; i << P.page_shift < g.len; i += step) reserve_page(P, b, (int)i, g.held, before, count);
    }
}

__global__ void __launch_bounds__(ONE_NT) pages_commit_kernel(const __grid_constant__ PagesParams P)
{
    __shared__ long long sh[32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int count = *P.count;
    const long long room = room_of(P, count);
    long long before = 0, moved = 0;
    for (int b0 = 0; b0 < P.B; b0 += ONE_NT) {
        const int b = b0 + threadIdx.x;
        Grow g = {};
        if (b < P.B) g = grow_of(P, b);
        const long long last = before + block_scan<ONE_NT>(g.n, sh);
        const bool served = g.status == ROW_OK && (g.n == 0 || last <= room);
        const long long took = block_scan<ONE_NT>(served ? g.n : 0, sh);
        if (b < P.B) commit(P, b, g, served);
        // what the chunk's last thread has summed
        if (threadIdx.x == ONE_NT - 1) sh[0] = last, sh[1] = took;
        __syncthreads();
        before = sh[0];
        moved += sh[1];
        __syncthreads();
    }
    if (threadIdx.x == 0 && moved) *P.count = count + (P.release ? (int)moved : -(int)moved);
}

}  // namespace

cudaError_t launch_pages(const PagesParams& P, cudaStream_t st)
{
    const bool few = P.release ? (long long)P.B * P.table_width <= ONE_ENTRIES : (long long)P.B * P.max_new <= ONE_ROWS + 4LL * P.B;
    if (P.B <= ONE_NT && few) {
        pages_one_kernel<<<1, ONE_NT, 0, st>>>(P);
        return cudaGetLastError();
    }
    // up to four rows (or pages) a thread, and a thousand CTAs or so
    const long long each = P.release ? P.table_width : P.max_new;
    long long x = (each + 4 * FILL_NT - 1) / (4 * FILL_NT);
    if (x > 64) x = 64;
    pages_fill_kernel<<<dim3((unsigned)x, (unsigned)P.B), FILL_NT, 0, st>>>(P);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(ONE_NT);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, pages_commit_kernel, P);
}

}  // namespace sv
