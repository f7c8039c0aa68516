// kv8_pages_kernels.hip -- who holds which page of a pool, and copying pages.
#include "kv8_internal.h"

#include <limits.h>

namespace cfz {
namespace {

constexpr int kThreads = 256;

__device__ inline bool names_page(const Kv8Pages &p, int page) { return page >= 0 && page < p.pages; }

__device__ inline int64_t held_tokens(const Kv8Pages &p, int row)
{
    const int64_t n = p.len[row], most = (int64_t)p.width << p.log2page;
    return n < 0 ? 0 : (n > most ? most : n);
}

// What other threads wrote in this launch, read past the first-level cache (which atomics pass by).
__device__ inline int32_t fresh_load(const int32_t *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void fresh_store(int32_t *p, int32_t x)
{
    __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A thread's stores and atomics are done.  (A work-group's barrier by itself does not wait for them.)
__device__ inline void memory_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A thread a place.  The exchange makes a row that is listed twice let go of its pages once.
__global__ __launch_bounds__(kThreads) void kv8_free_kernel(Kv8Pages p, const int32_t *rows,
                                                            const int32_t *keep, int chunks)
{
    const int i = blockIdx.x / chunks;
    const int e = (int)(blockIdx.x % chunks) * kThreads + threadIdx.x;
    const int row = rows[i];
    if (row < 0 || row >= p.batch || e >= p.width)
        return;
    const int kept = keep ? (keep[i] < 0 ? 0 : keep[i]) : 0;
    if (e == 0)
        atomicMin(p.len + row, kept);
    if (((int64_t)e << p.log2page) < kept)
        return;
    const int page = atomicExch(p.table + (int64_t)row * p.width + e, -1);
    if (names_page(p, page))
        atomicSub(p.refs + page, 1);
}

// A thread a place of a child.  Which pairs count is decided by all of them, so that the order in
// which the work-groups run changes nothing: a child is written by one pair and is nobody's parent.  Every
// work-group looks through the whole list: 5 us for 1024 pairs, 15 for 4096, 0.53 ms for 32,000.
__global__ __launch_bounds__(kThreads) void kv8_fork_kernel(Kv8Pages p, int count,
                                                            const int32_t *parents,
                                                            const int32_t *children, int chunks)
{
    const int i = blockIdx.x / chunks;
    const int e = (int)(blockIdx.x % chunks) * kThreads + threadIdx.x;
    const int parent = parents[i], child = children[i];
    if (parent < 0 || parent >= p.batch || child < 0 || child >= p.batch)
        return;
    bool out = false;
    for (int j = threadIdx.x; j < count; j += kThreads)
        out |= parents[j] == child || (j < i && children[j] == child);
    if (__syncthreads_or(out) || e >= p.width)
        return;
    const int64_t n = held_tokens(p, parent);
    if (e == 0)
        p.len[child] = (int)n;
    int32_t *to = p.table + (int64_t)child * p.width + e;
    const int old = *to;
    int page = ((int64_t)e << p.log2page) < n ? p.table[(int64_t)parent * p.width + e] : -1;
    if (!names_page(p, page))
        page = -1;
    if (page == old)
        return;
    *to = page;
    if (page >= 0)
        atomicAdd(p.refs + page, 1);
    if (names_page(p, old))
        atomicSub(p.refs + old, 1);
}

// One work-group: which places need a page is a matter of a few thousand integers and of steps that
// wait for each other, which costs less in one launch than spread over the card and several.  The
// free pages are looked for from the front, kScan pages at a time, until there are enough.  96 rows, one token
// each, 32 of them forked: 9.3 us, most of it reads that wait for each other (length, table, count,
// holders); a scan step of 64 KB more for every 16,384 pages in use before the free ones, and 4 us for every 1024
// places (65,535 rows, a token each: 0.29 ms; 4096 rows of 4096 tokens: 1.05 ms).
constexpr int kWide = 1024, kWaves = kWide / 64, kPieces = 16, kScan = kWide * kPieces;

__global__ __launch_bounds__(kWide) void kv8_reserve_kernel(Kv8Pages p, Kv8Reserve r)
{
    __shared__ int found[kPieces * kWaves];
    __shared__ int sums[kWaves];
    __shared__ int list[kWide];  // the first free pages; more of them go through memory
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int b = tid; b < p.batch; b += kWide) {
        r.source[b] = r.target[b] = -1;
        if (r.left_out) {
            const int64_t room = ((int64_t)p.width << p.log2page) - held_tokens(p, b);
            const int64_t want = r.counts[b] < 0 ? 0 : r.counts[b];
            const int64_t most = r.max_new < room ? r.max_new : room;
            r.left_out[b] = (int)(want > most ? want - most : 0);
        }
    }

    // a place: its row, its place in the row, and the page it names (-1: none, -2: not written)
    const uint32_t span = (uint32_t)r.span;
    auto place = [&](int q, int &row, int &e, int64_t &held) {
        row = (int)((uint32_t)q / span);
        held = held_tokens(p, row);
        int64_t n = r.counts[row];
        n = n < 0 ? 0 : (n > r.max_new ? r.max_new : n);
        e = (int)(held >> p.log2page) + (q - row * r.span);
        if (e >= p.width || n == 0 || ((int64_t)e << p.log2page) >= held + n)
            return -2;
        const int page = p.table[(int64_t)row * p.width + e];
        return names_page(p, page) ? page : -1;
    };
    // the first free pages' counts are under way while the places are looked up
    int ahead[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
        const int64_t page = u * kWide + tid;
        ahead[u] = page < p.pages ? p.refs[page] : 1;
    }
    int row, e;
    int64_t held;
    // (a thread's first place is looked up once; few calls have more than one a thread)
    const int mine = tid < r.places ? place(tid, row, e, held) : -2;
    const int mine_refs = mine >= 0 ? p.refs[mine] : 0;
    auto look = [&](int64_t q, int &refs) {
        const int page = q == tid ? mine : place((int)q, row, e, held);
        refs = q == tid ? mine_refs : (page >= 0 ? p.refs[page] : 0);
        return page;
    };
    bool any = false;
    for (int64_t q = tid; q < r.places; q += kWide) {
        int refs;
        const int page = look(q, refs);
        if (refs > 1) {
            any = true;
            fresh_store(r.owner + page, INT_MAX);
            fresh_store(r.writers + page, 0);
        }
    }
    memory_done();
    if (__syncthreads_or(any)) {
        for (int64_t q = tid; q < r.places; q += kWide) {
            int refs;
            const int page = look(q, refs);
            if (refs > 1) {
                atomicMin(r.owner + page, (int)q);
                atomicAdd(r.writers + page, 1);
            }
        }
    }
    memory_done();
    __syncthreads();

    // ranks among the places that need a page
    int64_t total = 0;
    int mine_rank = -1;
    for (int64_t base = 0; base < r.places; base += kWide) {
        const int64_t q = base + tid;
        bool need = false;
        if (q < r.places) {
            int refs;
            const int page = look(q, refs);
            need = page == -1;
            if (refs > 1)
                need = !(refs <= fresh_load(r.writers + page) &&
                         fresh_load(r.owner + page) == (int)q);
        }
        const uint64_t votes = __ballot(need);
        if (lane == 0)
            sums[wave] = __popcll(votes);
        __syncthreads();
        int64_t before = total;
        for (int w = 0; w < kWaves; ++w) {
            before += w < wave ? sums[w] : 0;
            total += sums[w];
        }
        const int rank = need ? (int)(before + __popcll(votes & ((1ull << lane) - 1))) : -1;
        if (base == 0)
            mine_rank = rank;
        else if (q < r.places)
            r.rank[q] = rank;
        __syncthreads();
    }
    if (total == 0) {
        if (tid == 0)
            r.missing[0] = 0;
        return;
    }

    int64_t have = 0;
    for (int64_t base = 0; base < p.pages && have < total; base += kScan) {
        int refs[kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int64_t page = base + u * kWide + tid;
            refs[u] = base == 0 ? ahead[u] : (page < p.pages ? p.refs[page] : 1);
        }
        uint64_t votes[kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            votes[u] = __ballot(refs[u] <= 0);
            if (lane == 0)
                found[u * kWaves + wave] = __popcll(votes[u]);
        }
        __syncthreads();
        // the counts become how many free pages lie before, 4 a lane of every wave (each for itself, the first
        // writes them back)
        int c[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            c[j] = sum;
            sum += found[lane * 4 + j];
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d);
            incl += lane >= d ? o : 0;
        }
        const int all = __shfl(incl, 63);
        __syncthreads();
        if (wave == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                found[lane * 4 + j] = incl - sum + c[j];
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int64_t rank =
                have + found[u * kWaves + wave] + __popcll(votes[u] & ((1ull << lane) - 1));
            if (refs[u] <= 0 && rank < total) {
                const int page = (int)(base + u * kWide + tid);
                if (rank < kWide)
                    list[rank] = page;
                else
                    fresh_store(r.list + rank, page);
            }
        }
        have += all;
        memory_done();
        __syncthreads();
    }
    if (tid == 0)
        r.missing[0] = have < total ? (int)(total - have) : 0;
    if (have < total)
        return;
    for (int64_t q = tid; q < r.places; q += kWide) {
        const int rank = q == tid ? mine_rank : r.rank[q];
        if (rank < 0)
            continue;
        const int old = place((int)q, row, e, held);
        const int page = rank < kWide ? list[rank] : fresh_load(r.list + rank);
        p.table[(int64_t)row * p.width + e] = page;
        p.refs[page] = 1;
        if (old >= 0) {
            atomicSub(p.refs + old, 1);
            if (((int64_t)e << p.log2page) < held) {
                r.source[row] = old;
                r.target[row] = page;
            }
        }
    }
}

// ---- packing: pages in use of each chunk; lists of the moves; table and counts

__device__ inline int block_sum(int x, int *red)
{
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1)
        x += __shfl_xor(x, d);
    if ((threadIdx.x & 63) == 0)
        red[wave] = x;
    __syncthreads();
    x = red[0] + red[1] + red[2] + red[3];
    __syncthreads();
    return x;
}

__global__ __launch_bounds__(kThreads) void kv8_pack_count_kernel(Kv8Pages p, Kv8Compact k)
{
    __shared__ int red[4];
    const int64_t base = (int64_t)blockIdx.x * kKv8RefsChunk;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kKv8RefsChunk / kThreads; ++i) {
        const int64_t page = base + i * kThreads + threadIdx.x;
        n += page < p.pages && p.refs[page] > 0;
    }
    n = block_sum(n, red);
    if (threadIdx.x == 0)
        k.counts[blockIdx.x] = n;
}

// With n pages in use, the free pages below n in ascending order meet the pages in use from n on in
// descending order: both numbers follow from how many pages in use lie before a page.  One chunk
// counts itself.
__global__ __launch_bounds__(kWide) void kv8_pack_lists_kernel(Kv8Pages p, Kv8Compact k, int chunks)
{
    constexpr int N = kKv8RefsChunk / kWide;
    static_assert(N * kWaves == 64, "a lane of a wave a vote");
    __shared__ int red[2][kWaves];
    __shared__ int found[64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t base = (int64_t)blockIdx.x * kKv8RefsChunk;
    int refs[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t page = base + i * kWide + tid;
        refs[i] = page < p.pages ? p.refs[page] : 0;
    }
    int n = 0, before = 0;
    if (chunks > 1) {
        int all = 0, mine = 0;
        for (int i = tid; i < chunks; i += kWide) {
            const int c = k.counts[i];
            all += c;
            mine += i < (int)blockIdx.x ? c : 0;
        }
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) {
            all += __shfl_xor(all, d);
            mine += __shfl_xor(mine, d);
        }
        if (lane == 0) {
            red[0][wave] = all;
            red[1][wave] = mine;
        }
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) {
            n += red[0][w];
            before += red[1][w];
        }
    }
    uint64_t votes[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        votes[i] = __ballot(refs[i] > 0);
        if (lane == 0)
            found[i * kWaves + wave] = __popcll(votes[i]);
    }
    __syncthreads();
    const int own = found[lane];
    int incl = own;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        incl += lane >= d ? o : 0;
    }
    if (chunks == 1)
        n = __shfl(incl, 63);
    if (blockIdx.x == 0 && tid == 0) {
        k.live[0] = n;
        if (n == 0)
            k.moves[0] = 0;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int64_t page = base + i * kWide + tid;
        const bool used = refs[i] > 0;
        const int rank = before + __shfl(incl - own, i * kWaves + wave) +
                         __popcll(votes[i] & ((1ull << lane) - 1));
        if (page >= p.pages)
            continue;
        if (page < n) {
            if (!used)
                k.target[page - rank] = (int)page;
            if (page == n - 1)
                k.moves[0] = n - rank - used;
        } else {
            if (used)
                k.source[n - 1 - rank] = (int)page;
            k.where[page] = used ? n - 1 - rank : -1;
        }
    }
}

__global__ __launch_bounds__(kThreads) void kv8_pack_apply_kernel(Kv8Pages p, Kv8Compact k)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int n = k.live[0];
    if (i < (int64_t)p.batch * p.width) {
        const int page = p.table[i];
        if (page >= n && page < p.pages) {
            const int move = k.where[page];
            if (move >= 0)
                p.table[i] = k.target[move];
        }
    }
    if (i < k.moves[0]) {
        p.refs[k.target[i]] = p.refs[k.source[i]];
        p.refs[k.source[i]] = 0;
    }
}

// ---- copying: a page's codes and means lie side by side, so that a page is a few runs of bytes, cut
// into pieces of 16 KB.  984 pages of 135 KB in 54 us, 4.9 TB/s; 32 in 4.0 us.

constexpr int kPiece = 16384;

struct CopySizes {
    int64_t codes, mean;  // bytes of a page's keys (and of its values), and of its means
    int of_codes, of_mean, all;  // pieces
};

CopySizes copy_sizes(const Kv8Cache &c)
{
    CopySizes s;
    s.codes = (int64_t)c.heads * c.page * c.dim;
    s.mean = c.km ? (int64_t)c.heads * c.dim * 4 : 0;
    s.of_codes = (int)((s.codes + kPiece - 1) / kPiece);
    s.of_mean = (int)((s.mean + kPiece - 1) / kPiece);
    s.all = 2 * s.of_codes + s.of_mean + 1;
    return s;
}

__global__ __launch_bounds__(kThreads) void kv8_copy_kernel(Kv8Cache to, Kv8Cache from, CopySizes s,
                                                            int64_t count, const int32_t *source,
                                                            const int32_t *target,
                                                            const int32_t *used)
{
    const int64_t most = used && used[0] < count ? used[0] : count;
    for (int64_t w = blockIdx.x; w < most * s.all; w += gridDim.x) {
        const int64_t pair = w / s.all;
        int piece = (int)(w - pair * s.all);
        const int64_t a = source[pair], b = target[pair];
        if (a < 0 || a >= from.pages || b < 0 || b >= to.pages)
            continue;
        const uint8_t *x = from.k + a * s.codes;
        uint8_t *y = to.k + b * s.codes;
        int64_t bytes = s.codes;
        if (piece >= 2 * s.of_codes + s.of_mean) {
            for (int h = threadIdx.x; h < to.heads; h += kThreads) {
                to.ks[b * to.heads + h] = from.ks[a * to.heads + h];
                to.vs[b * to.heads + h] = from.vs[a * to.heads + h];
            }
            continue;
        }
        if (piece >= 2 * s.of_codes) {
            piece -= 2 * s.of_codes;
            x = (const uint8_t *)from.km + a * s.mean;
            y = (uint8_t *)to.km + b * s.mean;
            bytes = s.mean;
        } else if (piece >= s.of_codes) {
            piece -= s.of_codes;
            x = from.v + a * s.codes;
            y = to.v + b * s.codes;
        }
        const int64_t base = (int64_t)piece * kPiece;
        const uint4 *px = (const uint4 *)(x + base) + threadIdx.x;
        uint4 *py = (uint4 *)(y + base) + threadIdx.x;
        static_assert(kPiece == 4 * 16 * kThreads, "a piece is four vectors a thread");
        if (bytes - base >= kPiece) {
            const uint4 q0 = px[0], q1 = px[kThreads], q2 = px[2 * kThreads], q3 = px[3 * kThreads];
            py[0] = q0;
            py[kThreads] = q1;
            py[2 * kThreads] = q2;
            py[3 * kThreads] = q3;
        } else {
            for (int i = 0; i * kThreads + threadIdx.x < (bytes - base) / 16; ++i)
                py[i * kThreads] = px[i * kThreads];
        }
    }
}

}  // namespace

hipError_t launch_kv8_free(const Kv8Pages &p, int count, const int32_t *rows, const int32_t *keep,
                           hipStream_t st)
{
    const int chunks = (p.width + kThreads - 1) / kThreads;
    kv8_free_kernel<<<dim3((unsigned)(count * chunks)), kThreads, 0, st>>>(p, rows, keep, chunks);
    return hipGetLastError();
}

hipError_t launch_kv8_fork(const Kv8Pages &p, int count, const int32_t *parents,
                           const int32_t *children, hipStream_t st)
{
    const int chunks = (p.width + kThreads - 1) / kThreads;
    kv8_fork_kernel<<<dim3((unsigned)(count * chunks)), kThreads, 0, st>>>(p, count, parents,
                                                                           children, chunks);
    return hipGetLastError();
}

Kv8Reserve kv8_reserve_plan(const Kv8Pages &p, int64_t max_new)
{
    Kv8Reserve r{};
    const int64_t page = 1 << p.log2page, room = p.width * page;
    r.max_new = max_new < room ? max_new : room;
    // tokens that start inside a page reach one page more than they fill
    const int64_t span = r.max_new == 0 ? 0 : (r.max_new + page - 2) / page + 1;
    r.span = (int)(span < p.width ? span : p.width);
    r.places = (int64_t)p.batch * r.span;
    r.fresh = r.places < p.pages ? r.places : p.pages;
    return r;
}

int64_t kv8_reserve_ints(const Kv8Pages &p, const Kv8Reserve &r)
{
    return r.places + r.fresh + 2 * p.pages;
}

hipError_t launch_kv8_reserve(const Kv8Pages &p, const Kv8Reserve &r, hipStream_t st)
{
    kv8_reserve_kernel<<<dim3(1), kWide, 0, st>>>(p, r);
    return hipGetLastError();
}

int kv8_compact_chunks(const Kv8Pages &p)
{
    const int64_t n = (p.pages + kKv8RefsChunk - 1) / kKv8RefsChunk;
    return (int)(n < 1 ? 1 : n);
}

hipError_t launch_kv8_compact(const Kv8Pages &p, const Kv8Compact &k, hipStream_t st)
{
    const int chunks = kv8_compact_chunks(p);
    if (chunks > 1)
        kv8_pack_count_kernel<<<dim3((unsigned)chunks), kThreads, 0, st>>>(p, k);
    kv8_pack_lists_kernel<<<dim3((unsigned)chunks), kWide, 0, st>>>(p, k, chunks);
    const int64_t places = (int64_t)p.batch * p.width, moves = p.pages / 2;
    const int64_t n = ((places > moves ? places : moves) + kThreads - 1) / kThreads;  // (>= 1)
    kv8_pack_apply_kernel<<<dim3((unsigned)n), kThreads, 0, st>>>(p, k);
    return hipGetLastError();
}

hipError_t launch_kv8_copy(const Kv8Cache &to, const Kv8Cache &from, int64_t count,
                           const int32_t *source, const int32_t *target, const int32_t *used,
                           hipStream_t st)
{
    const CopySizes s = copy_sizes(to);
    const int64_t pieces = count * s.all;
    const int64_t groups = pieces < 2048 ? pieces : 2048;
    kv8_copy_kernel<<<dim3((unsigned)groups), kThreads, 0, st>>>(to, from, s, count, source, target,
                                                                 used);
    return hipGetLastError();
}

}  // namespace cfz
