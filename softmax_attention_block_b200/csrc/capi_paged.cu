// C ABI of the paged decode cache: argument validation and launch sequences.
#include <math.h>

#include "paged.cuh"
#include "runtime.cuh"
#include "tc.cuh"

using namespace path;

namespace {

path_status launch_status(cudaError_t e) { return e == cudaSuccess ? PATH_OK : PATH_ERR_CUDA; }

#define TRY(x)                                          \
    do {                                                \
        cudaError_t e_ = (x);                           \
        if (e_ != cudaSuccess) return PATH_ERR_CUDA;    \
    } while (0)

bool kv_dtype_ok(path_dtype dt) { return dt == PATH_F32 || dt == PATH_BF16; }

// log2 of a page size the library handles, else -1
int page_log2(int page)
{
    for (int l = 4; l <= 10; ++l)
        if (page == 1 << l) return l;
    return -1;
}

bool aligned(const void *p, unsigned bytes) { return !(reinterpret_cast<uintptr_t>(p) & (bytes - 1)); }

// Row and entry numbers stay within 31 bits, a sequence's own with room for a tile behind it.
constexpr int MAX_ROWS = 1 << 30;  // of one sequence or prefix

bool pool_fits(int n_pages, int H, int page) { return (long long)n_pages * H * page < (1LL << 31); }
bool table_fits(int n_slots, int max_pages, int page)
{
    return (long long)n_slots * max_pages < (1LL << 31) && (long long)max_pages * page <= MAX_ROWS;
}

// Whether a table of this shape and its page size can be worked on.
path_status tables_ok(int n_slots, int max_pages, int n_pages, int page)
{
    if (n_slots <= 0 || max_pages <= 0 || n_pages <= 0) return PATH_ERR_INVALID_ARG;
    if (page_log2(page) < 0 || !table_fits(n_slots, max_pages, page)) return PATH_ERR_UNSUPPORTED;
    return PATH_OK;
}

// Checks of the two decode steps; fills what they have in common.
path_status step_args(const void *q, const void *k_new, const void *v_new, const void *w,
                      const float *beta, const float *log_f, float scale, int B, int H, int d,
                      path_dtype dt, void *k_pages, void *v_pages, float *g_pages, int n_pages,
                      int page, const int *table, int n_slots, int max_pages, const int *lens,
                      const int *rows, void *out, PagedStep &a)
{
    if (!q || !k_new || !v_new || !w || !beta || !k_pages || !v_pages || !table || !lens || !out)
        return PATH_ERR_INVALID_ARG;
    if ((log_f == nullptr) != (g_pages == nullptr)) return PATH_ERR_INVALID_ARG;
    if (B <= 0 || H <= 0 || !isfinite(scale) || (!rows && B > n_slots)) return PATH_ERR_INVALID_ARG;
    const path_status s = tables_ok(n_slots, max_pages, n_pages, page);
    if (s != PATH_OK) return s;
    if ((d != 64 && d != 128) || !kv_dtype_ok(dt) || (long long)B * H > 65535 || !pool_fits(n_pages, H, page))
        return PATH_ERR_UNSUPPORTED;
    // 16-byte vector access and bulk copies
    for (const void *p : {q, k_new, v_new, w, (const void *)k_pages, (const void *)v_pages, (const void *)g_pages})
        if (!aligned(p, 16)) return PATH_ERR_INVALID_ARG;
    a = PagedStep{};
    a.q = q;
    a.k_new = k_new;
    a.v_new = v_new;
    a.w = w;
    a.beta = beta;
    a.log_f = log_f;
    a.scale = scale;
    a.B = B;
    a.H = H;
    a.c = PagedCache{rows, n_slots, table, max_pages, lens, page_log2(page), n_pages, k_pages, v_pages, g_pages};
    a.out = out;
    a.withhold = withhold_kv_load();
    a.limit_ns = a.withhold ? 2000000ull : tc::WAIT_LIMIT_NS;
    return PATH_OK;
}

}  // namespace

extern "C" {

size_t path_decode_paged_workspace_bytes(int B, int H, int max_pages, int page, int d, path_dtype dt,
                                         int prefix_len)
{
    if (B <= 0 || H <= 0 || max_pages <= 0 || prefix_len < 0 || prefix_len > MAX_ROWS || page_log2(page) < 0 ||
        !table_fits(1, max_pages, page) || (d != 64 && d != 128) || !kv_dtype_ok(dt) ||
        (long long)B * H > 65535)
        return 0;
    PagedScratch s;
    const PagedPlan p = paged_plan(B, H, max_pages, page, d, (int)dt, prefix_len);
    return paged_carve(nullptr, p, B, H, d, s);
}

path_status path_decode_step_paged(const void *q, const void *k_new, const void *v_new, const void *w,
                                   const float *beta, const float *log_f, float scale, int B, int H,
                                   int d, path_dtype dt, void *k_pages, void *v_pages, float *g_pages,
                                   int n_pages, int page, const int *table, int n_slots, int max_pages,
                                   const int *lens, const int *rows, void *out, void *workspace,
                                   size_t workspace_bytes, path_stream_t stream)
{
    PagedStep a;
    const path_status st = step_args(q, k_new, v_new, w, beta, log_f, scale, B, H, d, dt, k_pages, v_pages,
                                     g_pages, n_pages, page, table, n_slots, max_pages, lens, rows, out, a);
    if (st != PATH_OK) return st;
    PagedScratch s;
    const PagedPlan p = paged_plan(B, H, max_pages, page, d, (int)dt, 0);
    if (!workspace || workspace_bytes < paged_carve(nullptr, p, B, H, d, s)) return PATH_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PATH_ERR_INVALID_ARG;
    paged_carve(workspace, p, B, H, d, s);
    return launch_status(decode_paged(a, (int)dt, d, false, p, s, reinterpret_cast<cudaStream_t>(stream)));
}

path_status path_decode_step_shared(const void *q, const void *k_new, const void *v_new, const void *w,
                                    const float *beta, const float *log_f, float scale, int B, int H,
                                    int d, path_dtype dt, void *k_pages, void *v_pages, float *g_pages,
                                    int n_pages, int page, const int *table, int n_slots, int max_pages,
                                    const int *lens, const int *rows, const int *prefix_table,
                                    int prefix_len, float *state, float *g_state, void *out,
                                    void *workspace, size_t workspace_bytes, path_stream_t stream)
{
    if (!prefix_table || !state || prefix_len <= 0) return PATH_ERR_INVALID_ARG;
    if ((log_f == nullptr) != (g_state == nullptr)) return PATH_ERR_INVALID_ARG;
    PagedStep a;
    const path_status st = step_args(q, k_new, v_new, w, beta, log_f, scale, B, H, d, dt, k_pages, v_pages,
                                     g_pages, n_pages, page, table, n_slots, max_pages, lens, rows, out, a);
    if (st != PATH_OK) return st;
    if (prefix_len > MAX_ROWS) return PATH_ERR_UNSUPPORTED;
    if (!aligned(state, 16)) return PATH_ERR_INVALID_ARG;
    a.prefix_table = prefix_table;
    a.prefix_len = prefix_len;
    a.state = state;
    a.g_state = g_state;
    PagedScratch s;
    const PagedPlan p = paged_plan(B, H, max_pages, page, d, (int)dt, prefix_len);
    if (!workspace || workspace_bytes < paged_carve(nullptr, p, B, H, d, s)) return PATH_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PATH_ERR_INVALID_ARG;
    paged_carve(workspace, p, B, H, d, s);
    cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    TRY(prefix_turn(a, (int)dt, d, p, s, cs));
    TRY(dt == PATH_BF16 ? prefix_attn_tc(a, d, p, s, cs) : prefix_attn_simt(a, d, p, s, cs));
    return launch_status(decode_paged(a, (int)dt, d, true, p, s, cs));
}

path_status path_pages_reserve(int *table, int *held, int *owner, int n_slots, int max_pages, int n_pages,
                               int page, const int *rows, const int *tokens, int n, int *info,
                               path_stream_t stream)
{
    if (!table || !held || !owner || !rows || !tokens || !info || n <= 0) return PATH_ERR_INVALID_ARG;
    const path_status s = tables_ok(n_slots, max_pages, n_pages, page);
    if (s != PATH_OK) return s;
    if (n > PAGES_MAX_ROWS) return PATH_ERR_UNSUPPORTED;
    const PageTables t{table, held, nullptr, owner, n_slots, max_pages, n_pages, page_log2(page)};
    return launch_status(pages_reserve(t, rows, tokens, n, info, reinterpret_cast<cudaStream_t>(stream)));
}

path_status path_pages_fork(int *table, int *held, int *lens, int *owner, int n_slots, int max_pages,
                            int n_pages, int page, const int *parents, const int *children, int n,
                            int *moves, int max_moves, int *info, path_stream_t stream)
{
    if (!table || !held || !lens || !owner || !parents || !children || !moves || !info || n <= 0)
        return PATH_ERR_INVALID_ARG;
    const path_status s = tables_ok(n_slots, max_pages, n_pages, page);
    if (s != PATH_OK) return s;
    if (n > PAGES_MAX_ROWS) return PATH_ERR_UNSUPPORTED;
    const long long most = (long long)n * max_pages;
    if (max_moves < (most < n_pages ? most : n_pages)) return PATH_ERR_INVALID_ARG;
    const PageTables t{table, held, lens, owner, n_slots, max_pages, n_pages, page_log2(page)};
    return launch_status(
        pages_fork(t, parents, children, n, moves, info, reinterpret_cast<cudaStream_t>(stream)));
}

path_status path_pages_free(int *table, int *held, int *lens, int *owner, int n_slots, int max_pages,
                            int n_pages, const int *rows, int n, path_stream_t stream)
{
    if (!table || !held || !lens || !owner || !rows || n <= 0) return PATH_ERR_INVALID_ARG;
    const path_status s = tables_ok(n_slots, max_pages, n_pages, 16);
    if (s != PATH_OK) return s;
    const PageTables t{table, held, lens, owner, n_slots, max_pages, n_pages, 0};
    return launch_status(pages_free(t, rows, n, reinterpret_cast<cudaStream_t>(stream)));
}

path_status path_pages_compact(int *table, const int *held, int *owner, int n_slots, int max_pages,
                               int n_pages, int *moves, int max_moves, int *info, path_stream_t stream)
{
    if (!table || !held || !owner || !moves || !info) return PATH_ERR_INVALID_ARG;
    const path_status s = tables_ok(n_slots, max_pages, n_pages, 16);
    if (s != PATH_OK) return s;
    if (max_moves < n_pages / 2) return PATH_ERR_INVALID_ARG;
    const PageTables t{table, const_cast<int *>(held), nullptr, owner, n_slots, max_pages, n_pages, 0};
    return launch_status(pages_compact(t, moves, info, reinterpret_cast<cudaStream_t>(stream)));
}

path_status path_pages_copy(const int *moves, int max_moves, int *info, void *k_pages, void *v_pages,
                            float *g_pages, int n_pages, int H, int page, int d, path_dtype dt,
                            path_stream_t stream)
{
    if (!moves || !info || !k_pages || !v_pages || max_moves < 0 || n_pages <= 0 || H <= 0)
        return PATH_ERR_INVALID_ARG;
    if (page_log2(page) < 0 || (d != 64 && d != 128) || !kv_dtype_ok(dt) || !pool_fits(n_pages, H, page))
        return PATH_ERR_UNSUPPORTED;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(g_pages, 16)) return PATH_ERR_INVALID_ARG;
    const long long rows = (long long)H * page;
    const PagesCopy a{moves, info, max_moves, k_pages, v_pages, g_pages, n_pages,
                      rows * d * (long long)dtype_size((int)dt), rows * 4};
    return launch_status(pages_copy(a, reinterpret_cast<cudaStream_t>(stream)));
}

path_status path_pages_store(const void *k_cache, const void *v_cache, const float *g_cache, int B, int H,
                             int d, int capacity, path_dtype dt, void *k_pages, void *v_pages,
                             float *g_pages, int n_pages, int page, const int *table, int n_slots,
                             int max_pages, const int *rows, const int *tokens, int *info,
                             path_stream_t stream)
{
    if (!k_cache || !v_cache || !k_pages || !v_pages || !table || !tokens) return PATH_ERR_INVALID_ARG;
    if ((g_cache == nullptr) != (g_pages == nullptr)) return PATH_ERR_INVALID_ARG;
    if (B <= 0 || H <= 0 || capacity <= 0 || (!rows && B > n_slots)) return PATH_ERR_INVALID_ARG;
    const path_status s = tables_ok(n_slots, max_pages, n_pages, page);
    if (s != PATH_OK) return s;
    if ((d != 64 && d != 128) || !kv_dtype_ok(dt) || (long long)B * H > 65535 || !pool_fits(n_pages, H, page))
        return PATH_ERR_UNSUPPORTED;
    for (const void *p : {k_cache, v_cache, (const void *)k_pages, (const void *)v_pages})
        if (!aligned(p, 16)) return PATH_ERR_INVALID_ARG;
    PagesStore a;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.g_cache = g_cache;
    a.B = B;
    a.H = H;
    a.capacity = capacity;
    a.row_bytes = d * (int)dtype_size((int)dt);
    a.pages = (int)(((long long)capacity + page - 1) / page);
    if (a.pages > max_pages) a.pages = max_pages;
    a.c = PagedCache{rows, n_slots, table, max_pages, nullptr, page_log2(page), n_pages, k_pages, v_pages, g_pages};
    a.tokens = tokens;
    a.info = info;
    return launch_status(pages_store(a, reinterpret_cast<cudaStream_t>(stream)));
}

path_status path_state_copy(float *state, float *g_state, int n_slots, int H, int d, const int *parents,
                            const int *children, int n, path_stream_t stream)
{
    if (!state || !parents || !children || n_slots <= 0 || H <= 0 || n <= 0 || !aligned(state, 16))
        return PATH_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || H > 65535) return PATH_ERR_UNSUPPORTED;
    return launch_status(
        state_copy(state, g_state, parents, children, n, n_slots, H, d, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
