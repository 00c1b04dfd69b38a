// Paged decode cache: kernels' arguments and launchers.
//
// A pool holds n_pages pages of `page` token rows for every head: keys and
// values [n_pages, H, page, d], gate biases [n_pages, H, page]. A slot r of
// the tables names the pages of one sequence, table[r * max_pages + j] for its
// rows j * page ...; lens[r] rows are filled. A batch row b works on slot
// rows[b] (b itself without `rows`); a negative slot is an idle batch row.
#pragma once
#include "common.cuh"

namespace path {

struct PagedCache {
    const int *rows;   // [B] slots, or null
    int n_slots;
    const int *table;  // [n_slots, max_pages]
    int max_pages;
    const int *lens;   // [n_slots]
    int page_log2, n_pages;
    void *k, *v;       // [n_pages, H, page, d]
    float *g;          // [n_pages, H, page], or null
};

struct PagedStep {
    const void *q, *k_new, *v_new, *w;  // [B, H, d]
    const float *beta, *log_f;          // [B, H]
    float scale;
    int B, H;
    PagedCache c;
    void *out;  // [B, H, d]
    // shared prefix (prefix_len > 0 or state set)
    const int *prefix_table;
    int prefix_len;
    float *state;    // [n_slots, H, d, d] products of the Householder factors
    float *g_state;  // [n_slots, H]
    unsigned long long limit_ns;  // of a wait on a barrier
    int withhold;  // test hook: one load of the first block never completes
};

// slot of batch row b: negative if idle, or invalid (see row_ok)
__device__ __forceinline__ int slot_of(const PagedCache &c, int b) { return c.rows ? c.rows[b] : b; }

// length of the sequence in `slot`; -1 if the slot or the length is out of range
__device__ __forceinline__ int length_of(const PagedCache &c, int slot)
{
    if (slot >= c.n_slots) return -1;
    const int n = c.lens[slot];
    return n >= 0 && n < (long long)c.max_pages << c.page_log2 ? n : -1;
}

// Rows of a granule of the own part: 8 KB of keys and values, or 16 rows (the smallest page).
constexpr int own_granule(int d, int size) { return d * size == 512 ? 8 : 16; }

// bf16 numbers whose sum is an fp32 number: 3 x 8 bits and more (a sum of two is off by 2^-17).
constexpr int PREFIX_PARTS = 3;

// What went wrong with a piece (bits of own_flag and pre_flag)
enum { PIECE_BAD_PAGE = 4, PIECE_GAVE_UP = 8 };

// Device error codes of a paged step (first word of the workspace)
constexpr int ERR_PAGE = 1000, ERR_PAGED_WAIT = 41;

// Scratch of a step, carved from the caller's workspace.
//
// Both parts deal a list of tiles (units in order, a unit's tiles in order)
// out to blocks in contiguous shares, so a unit may lie in several blocks and
// a block may hold several units. The piece of unit u that block i
// holds has the slot i + u: along the list i and u never fall and one of them
// rises at every piece, so no two pieces share a slot.
struct PagedScratch {
    int *err;          // [64]
    int *first, *last; // [B * H] blocks of a unit's first and last tile
    float *own;        // [own_slots, d + 2]: max (log2 domain), sum, accumulator
    int *own_flag;     // [own_slots] bits 2, 3: see PIECE_*
    // the queries turned back to the prefix's end, q_rows = q_tiles * q_tile of a head (zero past
    // the batch): [H, q_rows, d] fp32, or for the tensor cores [PREFIX_PARTS, H, q_rows, d] bf16
    float *qt;
    float *qg;         // [H, q_rows] the gate's bias since the prefix's end (log2 domain)
    float *pre;        // [pre_slots, q_tile, d] accumulators of the prefix part
    float *pre_ml;     // [pre_slots, 2, q_tile] max (log2 domain) and sum
    int *pre_flag;     // [pre_slots, 4] PIECE_* (one for each 16 queries)
};

struct PagedPlan {
    int own_blocks, own_slots;
    int q_tile, q_tiles, key_tile, key_tiles, pre_units, pre_blocks, pre_slots;
};

PagedPlan paged_plan(int B, int H, int max_pages, int page, int d, int dt, int prefix_len);
size_t paged_carve(void *base, const PagedPlan &p, int B, int H, int d, PagedScratch &s);

// state <- H state, and the queries the prefix sees (SHARED only)
cudaError_t prefix_turn(const PagedStep &a, int dt, int d, const PagedPlan &p, const PagedScratch &s,
                        cudaStream_t st);
// The batch's attention to the prefix: fp32 on CUDA cores, bf16 on the tensor cores.
cudaError_t prefix_attn_tc(const PagedStep &a, int d, const PagedPlan &p, const PagedScratch &s,
                           cudaStream_t st);
cudaError_t prefix_attn_simt(const PagedStep &a, int d, const PagedPlan &p,
                             const PagedScratch &s, cudaStream_t st);
// The sequences' own pages (in-place key update, softmax pieces), then the
// join of all pieces of a row, the prefix's included.
cudaError_t decode_paged(const PagedStep &a, int dt, int d, bool shared, const PagedPlan &p,
                         const PagedScratch &s, cudaStream_t st);

// ---------------------------------------------------------------- the tables
// info: [4] status (0 or PATH_ERR_PAGE), moves listed, pages in use, pages given
struct PageTables {
    int *table, *held, *lens, *owner;
    int n_slots, max_pages, n_pages, page_log2;
};

constexpr int PAGES_MAX_ROWS = 4096;  // rows of one reserve or fork call

cudaError_t pages_reserve(const PageTables &t, const int *rows, const int *tokens, int n, int *info,
                          cudaStream_t st);
cudaError_t pages_fork(const PageTables &t, const int *parents, const int *children, int n, int *moves,
                       int *info, cudaStream_t st);
cudaError_t pages_free(const PageTables &t, const int *rows, int n, cudaStream_t st);
cudaError_t pages_compact(const PageTables &t, int *moves, int *info, cudaStream_t st);

struct PagesCopy {
    const int *moves;  // [max_moves, 2] source, destination
    int *info;
    int max_moves;
    void *k, *v;
    float *g;
    int n_pages;
    long long kv_bytes, g_bytes;  // of one page
};

cudaError_t pages_copy(const PagesCopy &a, cudaStream_t st);

struct PagesStore {
    const void *k_cache, *v_cache;  // [B, H, capacity, d]
    const float *g_cache;           // [B, H, capacity]
    int B, H, capacity;
    int pages;                      // pages of a full cache, at most max_pages
    int row_bytes;                  // d elements
    PagedCache c;                   // lens unused
    const int *tokens;              // [B]
    int *info;
};

cudaError_t pages_store(const PagesStore &a, cudaStream_t st);
cudaError_t state_copy(float *state, float *g_state, const int *parents, const int *children, int n,
                       int n_slots, int H, int d, cudaStream_t st);

}  // namespace path
