// Page tables of the paged decode cache and the moves of its pages.
//
// A page belongs to one table entry or to none: owner[p] = slot * max_pages +
// entry, or -1. Sequences that share a prefix read it through a table row of
// its own, so no page needs a count of its users. Every operation below
// leaves a state that depends on its arguments alone: free pages are taken in
// ascending order, for the rows in the order of their list.
//
// reserve, fork and compact are index work: one block of 1024 threads, which
// reads the owners to count them and walks them 4096 at a time with a block
// scan. A reserve of one page for each of 256 rows takes 10 us in a pool of
// 8192 pages, 19 in one of 65536, 51 in 262144 and 199 in 1048576, where the
// one block's walk is what takes the time. It counts before it writes, so a
// call that cannot be served changes nothing but `info`. The bytes move in
// pages_copy, which the caller runs once for each layer's pool with the same list.
#include "paged.cuh"
#include "runtime.cuh"

namespace path {

namespace {

constexpr int NT = 1024;

// Exclusive prefix sum of x over the block; total in *sum. All threads call.
__device__ int block_scan(int x, int *sum)
{
    __shared__ int s_w[32];
    __shared__ int s_total;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) s_w[warp] = v;
    __syncthreads();
    if (warp == 0) {
        const int w = s_w[lane];
        int t = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        s_w[lane] = t - w;
        if (lane == 31) s_total = t;
    }
    __syncthreads();
    const int r = s_w[warp] + v - x;
    *sum = s_total;
    __syncthreads();  // s_w is free for the next call
    return r;
}

__device__ int block_sum(int x)
{
    int t;
    block_scan(x, &t);
    return t;
}

// Calls f(page, rank) for the pages of [lo, hi) whose owner is (used ? >= 0 :
// < 0), in ascending order of rank, until `limit` of them are found; returns
// how many were found (at most limit is called, more may be counted).
template <typename F>
__device__ int for_pages(const int *owner, int lo, int hi, bool used, int limit, F f)
{
    int found = 0;
    for (int base = lo; base < hi && found < limit; base += 4 * NT) {
        const int p0 = base + 4 * threadIdx.x;
        int o[4], cnt = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] = p0 + i < hi && (owner[p0 + i] >= 0) == used;
            cnt += o[i];
        }
        int total, rank = found + block_scan(cnt, &total);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (o[i]) {
                if (rank < limit) f(p0 + i, rank);
                ++rank;
            }
        found += total;
    }
    return found;
}

__device__ int count_used(const PageTables &t)
{
    int n = 0;
    for (int p = threadIdx.x; p < t.n_pages; p += NT) n += t.owner[p] >= 0;
    return block_sum(n);
}

__device__ __forceinline__ int pages_of(int tokens, int page_log2)
{
    return (int)(((long long)tokens + (1 << page_log2) - 1) >> page_log2);
}

__device__ void report(int *info, int status, int moves, int used, int given)
{
    if (threadIdx.x == 0) {
        info[0] = status;
        info[1] = moves;
        info[2] = used;
        info[3] = given;
    }
}

// off[i] is an ascending prefix sum; the last i with off[i] <= k
__device__ __forceinline__ int find_row(const int *off, int n, int k)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (off[mid] <= k)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// FORK: rows are the children, other the parents; else other is the token
// count that each row has to hold.
template <bool FORK>
__global__ void __launch_bounds__(NT) give_pages_kernel(PageTables t, const int *rows, const int *other,
                                                        int n, int *moves, int *info)
{
    __shared__ int s_off[PAGES_MAX_ROWS], s_row[PAGES_MAX_ROWS];
    const int used = count_used(t);
    for (int i = threadIdx.x; i < n; i += NT) s_row[i] = rows[i];
    __syncthreads();
    int bad = 0, total = 0;
    for (int base = 0; base < n; base += NT) {
        const int i = base + threadIdx.x;
        int need = 0;
        if (i < n && s_row[i] >= 0) {
            const int r = s_row[i];
            if (r >= t.n_slots) {
                bad = 1;
            } else if (FORK) {
                const int p = other[i];  // negative: a sequence without tokens of its own
                if (p >= t.n_slots || t.held[r] != 0 || (p >= 0 && t.lens[p] < 0)) {
                    bad = 1;
                } else if (p >= 0) {
                    need = pages_of(t.lens[p], t.page_log2);
                    if (need > t.held[p]) bad = 1;
                }
            } else {
                const int want = other[i];
                if (want < 0 || want > (long long)t.max_pages << t.page_log2 || t.held[r] < 0 ||
                    t.held[r] > t.max_pages)
                    bad = 1;
                else
                    need = max(0, pages_of(want, t.page_log2) - t.held[r]);
            }
            for (int j = 0; j < i; ++j) bad |= s_row[j] == r;  // a row twice
        }
        // a bad call gives nothing: keep the sums small
        need = min(need, t.max_pages);
        int sum, at = total + block_scan(need, &sum);
        if (i < n) s_off[i] = at;
        total += sum;
    }
    bad = block_sum(bad);
    if (bad || total > t.n_pages - used) {
        report(info, PATH_ERR_PAGE, 0, used, 0);
        return;
    }
    // everything that is read below of the rows' former state is read before the first write
    // to it: a child holds no pages, and its length is taken with its pages
    for_pages(t.owner, 0, t.n_pages, false, total, [&](int p, int k) {
        const int i = find_row(s_off, n, k);
        const int r = s_row[i], j = k - s_off[i] + (FORK ? 0 : t.held[r]);
        t.table[(long long)r * t.max_pages + j] = p;
        t.owner[p] = r * t.max_pages + j;
        if (FORK) {
            moves[2 * k] = t.table[(long long)other[i] * t.max_pages + j];
            moves[2 * k + 1] = p;
        }
    });
    __syncthreads();
    int len[PAGES_MAX_ROWS / NT];
#pragma unroll
    for (int c = 0; c < PAGES_MAX_ROWS / NT; ++c) {
        const int i = c * NT + threadIdx.x;
        len[c] = FORK && i < n && s_row[i] >= 0 && other[i] >= 0 ? t.lens[other[i]] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < PAGES_MAX_ROWS / NT; ++c) {
        const int i = c * NT + threadIdx.x;
        if (i < n && s_row[i] >= 0) {
            const int got = (i + 1 < n ? s_off[i + 1] : total) - s_off[i];
            t.held[s_row[i]] += got;
            if (FORK) t.lens[s_row[i]] = len[c];
        }
    }
    report(info, 0, FORK ? total : 0, used + total, total);
}

__global__ void __launch_bounds__(256) free_kernel(PageTables t, const int *rows)
{
    __shared__ int s_held;
    const int r = rows[blockIdx.x];
    if (r < 0 || r >= t.n_slots) return;
    if (threadIdx.x == 0) {
        s_held = atomicExch(&t.held[r], 0);  // a row named twice is freed once
        t.lens[r] = 0;
    }
    __syncthreads();
    const int n = min(s_held, t.max_pages);
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
        const int e = r * t.max_pages + j, p = t.table[e];
        if (p >= 0 && p < t.n_pages && t.owner[p] == e) t.owner[p] = -1;
        t.table[e] = -1;
    }
}

__global__ void __launch_bounds__(NT) compact_kernel(PageTables t, int *moves, int *info)
{
    const int used = count_used(t);
    const int n = for_pages(t.owner, used, t.n_pages, true, t.n_pages, [&](int p, int k) { moves[2 * k] = p; });
    for_pages(t.owner, 0, used, false, n, [&](int p, int k) { moves[2 * k + 1] = p; });
    __syncthreads();
    const int entries = t.n_slots * t.max_pages;
    int bad = 0;
    for (int k = threadIdx.x; k < n; k += NT) {
        const int e = t.owner[moves[2 * k]];
        bad |= e >= entries || e % t.max_pages >= t.held[e / t.max_pages] || t.table[e] != moves[2 * k];
    }
    bad = block_sum(bad);
    if (bad) {
        report(info, PATH_ERR_PAGE, 0, used, 0);
        return;
    }
    for (int k = threadIdx.x; k < n; k += NT) {
        const int src = moves[2 * k], dst = moves[2 * k + 1], e = t.owner[src];
        t.table[e] = dst;
        t.owner[dst] = e;
        t.owner[src] = -1;
    }
    report(info, 0, n, used, 0);
}

constexpr int COPY_THREADS = 256, COPY_VECS = 8;
constexpr int COPY_PIECE = COPY_THREADS * COPY_VECS * 16;  // bytes a block moves at a time

// One piece of at most COPY_PIECE bytes (a multiple of 16), all its loads before its stores.
__device__ __forceinline__ void copy_piece(const char *src, char *dst, int bytes)
{
    uint4 x[COPY_VECS];
#pragma unroll
    for (int i = 0; i < COPY_VECS; ++i) {
        const int o = (i * COPY_THREADS + threadIdx.x) * 16;
        if (o < bytes) x[i] = *reinterpret_cast<const uint4 *>(src + o);
    }
#pragma unroll
    for (int i = 0; i < COPY_VECS; ++i) {
        const int o = (i * COPY_THREADS + threadIdx.x) * 16;
        if (o < bytes) *reinterpret_cast<uint4 *>(dst + o) = x[i];
    }
}

// Pages of a move list: bound by HBM, each byte read and written once. Pieces of 32 KB keep
// 8 loads of a thread in flight (16 KB pieces: 4% slower; bulk copies through shared memory:
// within 2% of these). 32 sequences of 200 to 1500 tokens, 32 heads of 128: 151 us for 946 MB,
// 6.3 TB/s.
__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(PagesCopy a)
{
    const int n = min(a.info[1], a.max_moves);
    const int kv = (int)((a.kv_bytes + COPY_PIECE - 1) / COPY_PIECE);
    const int g = a.g ? (int)((a.g_bytes + COPY_PIECE - 1) / COPY_PIECE) : 0;
    const int per = 2 * kv + g;
    for (long long it = blockIdx.x; it < (long long)n * per; it += gridDim.x) {
        const int m = (int)(it / per), w = (int)(it % per);
        const int src = a.moves[2 * m], dst = a.moves[2 * m + 1];
        if (src < 0 || src >= a.n_pages || dst < 0 || dst >= a.n_pages) {
            if (threadIdx.x == 0) a.info[0] = PATH_ERR_PAGE;
            continue;
        }
        char *pool;
        long long bytes, at;
        if (w < 2 * kv) {
            const bool key = w < kv;
            pool = static_cast<char *>(key ? a.k : a.v);
            bytes = a.kv_bytes;
            at = (long long)(key ? w : w - kv) * COPY_PIECE;
        } else {
            pool = reinterpret_cast<char *>(a.g);
            bytes = a.g_bytes;
            at = (long long)(w - 2 * kv) * COPY_PIECE;
        }
        copy_piece(pool + src * bytes + at, pool + dst * bytes + at, (int)min((long long)COPY_PIECE, bytes - at));
    }
}

// One page of one head at a time: its rows are contiguous on both sides. Its keys and values
// are loaded together; what is read once is not kept in the caches. 8 x 24 heads of 64, 1 to
// 4096 tokens: 40 us for 217 MB, 5.4 TB/s (47 us one after the other and without the hints).
__global__ void __launch_bounds__(COPY_THREADS) store_kernel(PagesStore a)
{
    constexpr int VECS = 2, PIECE = COPY_THREADS * VECS * 16;
    const int page = 1 << a.c.page_log2;
    const long long items = (long long)a.B * a.pages * a.H;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int h = (int)(it % a.H), j = (int)(it / a.H % a.pages);
        const int b = (int)(it / a.H / a.pages);
        const int r = a.c.rows ? a.c.rows[b] : b;
        if (r < 0) continue;
        const int n = a.tokens[b];
        const int left = n - j * page;
        const bool ok = r < a.c.n_slots && n >= 0 && n <= a.capacity &&
                        n <= (long long)a.c.max_pages << a.c.page_log2;
        if (ok && left <= 0) continue;
        const int p = ok ? a.c.table[(long long)r * a.c.max_pages + j] : -1;
        if (p < 0 || p >= a.c.n_pages) {
            if (threadIdx.x == 0 && a.info) a.info[0] = PATH_ERR_PAGE;
            continue;
        }
        const int m = min(page, left);
        const long long from = ((long long)b * a.H + h) * a.capacity + j * page;
        const long long to = ((long long)p * a.H + h) * page;
        const int bytes = m * a.row_bytes;
        for (int at = threadIdx.x * 16; at - (int)threadIdx.x * 16 < bytes; at += PIECE) {
            uint4 x[2][VECS];
#pragma unroll
            for (int i = 0; i < 2 * VECS; ++i) {
                const int o = at + i / 2 * COPY_THREADS * 16;
                const char *src = static_cast<const char *>(i % 2 ? a.v_cache : a.k_cache) + from * a.row_bytes + o;
                if (o < bytes) x[i % 2][i / 2] = __ldcs(reinterpret_cast<const uint4 *>(src));
            }
#pragma unroll
            for (int i = 0; i < 2 * VECS; ++i) {
                const int o = at + i / 2 * COPY_THREADS * 16;
                char *dst = static_cast<char *>(i % 2 ? a.c.v : a.c.k) + to * a.row_bytes + o;
                if (o < bytes) __stcs(reinterpret_cast<uint4 *>(dst), x[i % 2][i / 2]);
            }
        }
        if (a.g_cache)
            for (int i = threadIdx.x; i < m; i += COPY_THREADS) a.c.g[to + i] = a.g_cache[from + i];
    }
}

// 32 x 32 heads of 128: 21 us for 134 MB (6.3 TB/s).
__global__ void __launch_bounds__(256) state_copy_kernel(float *state, float *g_state, const int *parents,
                                                         const int *children, int n_slots, int H, int d)
{
    const int i = blockIdx.x, h = blockIdx.y;
    const int p = parents[i], c = children[i];
    if (c < 0 || c >= n_slots || p >= n_slots || p == c) return;
    const int n4 = d * d / 4;
    float4 *dst = reinterpret_cast<float4 *>(state) + ((long long)c * H + h) * n4;
    if (p >= 0) {
        const float4 *src = reinterpret_cast<const float4 *>(state) + ((long long)p * H + h) * n4;
        for (int e = threadIdx.x; e < n4; e += 256) dst[e] = src[e];
    } else {  // a sequence that starts at the prefix's end: the identity
        for (int e = threadIdx.x; e < n4; e += 256) {
            const int r = 4 * e / d, c0 = 4 * e % d;
            dst[e] = make_float4(r == c0, r == c0 + 1, r == c0 + 2, r == c0 + 3);
        }
    }
    if (g_state && threadIdx.x == 0)
        g_state[(long long)c * H + h] = p >= 0 ? g_state[(long long)p * H + h] : 0.f;
}

}  // namespace

cudaError_t pages_reserve(const PageTables &t, const int *rows, const int *tokens, int n, int *info,
                          cudaStream_t st)
{
    give_pages_kernel<false><<<1, NT, 0, st>>>(t, rows, tokens, n, nullptr, info);
    count_launches();
    return cudaGetLastError();
}

cudaError_t pages_fork(const PageTables &t, const int *parents, const int *children, int n, int *moves,
                       int *info, cudaStream_t st)
{
    give_pages_kernel<true><<<1, NT, 0, st>>>(t, children, parents, n, moves, info);
    count_launches();
    return cudaGetLastError();
}

cudaError_t pages_free(const PageTables &t, const int *rows, int n, cudaStream_t st)
{
    free_kernel<<<n, 256, 0, st>>>(t, rows);
    count_launches();
    return cudaGetLastError();
}

cudaError_t pages_compact(const PageTables &t, int *moves, int *info, cudaStream_t st)
{
    compact_kernel<<<1, NT, 0, st>>>(t, moves, info);
    count_launches();
    return cudaGetLastError();
}

cudaError_t pages_copy(const PagesCopy &a, cudaStream_t st)
{
    copy_kernel<<<8 * sm_count(), COPY_THREADS, 0, st>>>(a);
    count_launches();
    return cudaGetLastError();
}

cudaError_t pages_store(const PagesStore &a, cudaStream_t st)
{
    const long long items = (long long)a.B * a.pages * a.H;
    const int blocks = (int)(items < 8LL * sm_count() ? items : 8LL * sm_count());
    store_kernel<<<blocks, COPY_THREADS, 0, st>>>(a);
    count_launches();
    return cudaGetLastError();
}

cudaError_t state_copy(float *state, float *g_state, const int *parents, const int *children, int n,
                       int n_slots, int H, int d, cudaStream_t st)
{
    state_copy_kernel<<<dim3(n, H), 256, 0, st>>>(state, g_state, parents, children, n_slots, H, d);
    count_launches();
    return cudaGetLastError();
}

}  // namespace path
