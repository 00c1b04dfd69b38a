// Paged decode step: every batch row updates its own cached keys in place and
// attends to them (Paper-Notes "训练策略", inference paragraph), with lengths
// and pages read on the device. Per head, with n = lens[slot]:
//   k_j <- k_j - beta w (w^T k_j), g_j <- g_j + log f    (j < n, rounded to dt)
//   row n <- k_new, v_new, g = 0;  out = softmax_j(scale q^T k_j + g_j) V.
//
// Bound by HBM: it reads K and V once and writes K once (3 d elements a row and
// head) for about 8 d operations. Rows differ in length, so the (row, head)
// units are cut into tiles of OWN_TILE rows and the list of all tiles is dealt
// out to the blocks in equal contiguous shares (decode_own_kernel); pieces of a
// unit meet in decode_join_kernel, in block order, so results repeat exactly.
// The lengths are on the device: each block adds them up itself.
#include "paged.cuh"
#include "rowvec.cuh"
#include "runtime.cuh"
#include "tc.cuh"

namespace path {

namespace {

constexpr int NT = 256;
constexpr int UNROLL = 8;
constexpr float LOG2E = 1.4426950408889634f;

// tiles of one head of batch row b (0: idle or invalid; the new token is a row)
__device__ __forceinline__ int tiles_of(const PagedCache &c, int b)
{
    const int slot = slot_of(c, b);
    if (slot < 0) return 0;
    const int n = length_of(c, slot);
    return n < 0 ? 0 : n / OWN_TILE + 1;
}

__device__ long long block_scan(long long x, long long *total)
{
    __shared__ long long s_w[NT / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    long long v = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) s_w[warp] = v;
    __syncthreads();
    long long before = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
        if (i < warp) before += s_w[i];
        sum += s_w[i];
    }
    __syncthreads();
    *total = sum;
    return before + v - x;
}

template <typename T, int D, bool GATE, bool SHARED>
__global__ void __launch_bounds__(NT) decode_own_kernel(PagedStep a, PagedScratch s)
{
    constexpr int V = Vec<T>::N;
    constexpr int LPR = D / V;
    constexpr int G = NT / LPR;
    __shared__ float s_m[G], s_l[G];
    __shared__ float s_acc[G][D];
    __shared__ int s_row;
    __shared__ long long s_cum;
    const int tid = threadIdx.x, lane_in_row = tid % LPR, g = tid / LPR;
    const PagedCache &c = a.c;
    const int page = 1 << c.page_log2;

    // this block's share [t0, t1) of all tiles, and the batch row that t0 lies in
    long long total = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        long long sum;
        block_scan(b0 + tid < a.B ? (long long)tiles_of(c, b0 + tid) * a.H : 0, &sum);
        total += sum;
    }
    if (blockIdx.x == 0 && tid == 0) *s.err = 0;
    // no more blocks than tiles take part, so that no share is empty and the blocks that hold a
    // unit follow one another
    const long long nb = min((long long)gridDim.x, total);
    if (blockIdx.x >= nb) return;
    const long long t0 = total * blockIdx.x / nb, t1 = total * (blockIdx.x + 1) / nb;
    long long cum = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const long long mine = b0 + tid < a.B ? (long long)tiles_of(c, b0 + tid) * a.H : 0;
        long long sum;
        const long long at = cum + block_scan(mine, &sum);
        if (at <= t0 && t0 < at + mine) {
            s_row = b0 + tid;
            s_cum = at;
        }
        cum += sum;
    }
    __syncthreads();
    int b = s_row;
    cum = s_cum;
    int nt = tiles_of(c, b);
    const float scale2 = a.scale * LOG2E;

    for (long long t = t0; t < t1;) {
        while (t >= cum + (long long)nt * a.H) {  // next batch row with tiles
            cum += (long long)nt * a.H;
            nt = tiles_of(c, ++b);
        }
        const int slot = slot_of(c, b), n = length_of(c, slot);
        const int h = (int)((t - cum) / nt), tb = (int)((t - cum) % nt);
        const int te = (int)min((long long)nt, tb + (t1 - t));
        const int u = b * a.H + h;
        const int r1 = min(te * OWN_TILE, n + 1);
        float w[V], q[V];
        unpack<T>(reinterpret_cast<const uint4 *>(a.w)[(long long)u * LPR + lane_in_row], w);
        unpack<T>(reinterpret_cast<const uint4 *>(a.q)[(long long)u * LPR + lane_in_row], q);
        const float beta = a.beta[u];
        const float lf = GATE ? a.log_f[u] : 0.f;
        const int *tab = c.table + (long long)slot * c.max_pages;
        uint4 *K = static_cast<uint4 *>(c.k), *Vp = static_cast<uint4 *>(c.v);
        bool bad = false;
        float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.f;
        for (int rb = tb * OWN_TILE; rb < r1; rb += G * UNROLL) {
            uint4 kv[UNROLL], vv[UNROLL];
            long long at[UNROLL];  // row of the pool, or -1
            float gv[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const int r = rb + i * G + g;
                at[i] = -1;
                gv[i] = 0.f;
                kv[i] = vv[i] = make_uint4(0u, 0u, 0u, 0u);
                if (r < r1) {
                    const int p = tab[r >> c.page_log2];
                    if (p >= 0 && p < c.n_pages)
                        at[i] = ((long long)p * a.H + h) * page + (r & (page - 1));
                    else
                        bad = true;
                }
                if (at[i] >= 0) {
                    const bool fresh = r == n;
                    kv[i] = fresh ? static_cast<const uint4 *>(a.k_new)[(long long)u * LPR + lane_in_row]
                                  : K[at[i] * LPR + lane_in_row];
                    vv[i] = fresh ? static_cast<const uint4 *>(a.v_new)[(long long)u * LPR + lane_in_row]
                                  : Vp[at[i] * LPR + lane_in_row];
                    if (GATE && !fresh) gv[i] = c.g[at[i]] + lf;
                }
            }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const int r = rb + i * G + g;
                const bool valid = at[i] >= 0, fresh = r == n;
                float k[V], v[V];
                unpack<T>(kv[i], k);
                unpack<T>(vv[i], v);
                float wk = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) wk = fmaf(w[e], k[e], wk);
                const float coef = beta * group_sum<LPR>(wk);
                if (!fresh) {
#pragma unroll
                    for (int e = 0; e < V; ++e) k[e] = fmaf(-coef, w[e], k[e]);
                }
                if (valid) {
                    K[at[i] * LPR + lane_in_row] = fresh ? kv[i] : pack<T>(k);
                    if (fresh) Vp[at[i] * LPR + lane_in_row] = vv[i];
                    if (GATE && lane_in_row == 0) c.g[at[i]] = gv[i];
                }
                if (!fresh) round_to<T>(k);
                float z = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) z = fmaf(q[e], k[e], z);
                z = fmaf(group_sum<LPR>(z), scale2, gv[i] * LOG2E);
                if (valid) {
                    const float mn = fmaxf(m, z);
                    if (mn != -INFINITY) {  // all -inf so far: nothing to weigh
                        const float corr = tc::ex2(m - mn), p = tc::ex2(z - mn);
                        l = fmaf(l, corr, p);
#pragma unroll
                        for (int e = 0; e < V; ++e) acc[e] = fmaf(acc[e], corr, p * v[e]);
                        m = mn;
                    } else if (isnan(z)) {
                        l = z;
                    }
                }
            }
        }
        // join the row groups of this block
        if (lane_in_row == 0) {
            s_m[g] = m;
            s_l[g] = l;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) s_acc[g][lane_in_row * V + i] = acc[i];
        const bool any_bad = __syncthreads_or(bad);
        const bool whole = tb == 0 && te == nt;
        const long long piece = (long long)blockIdx.x + u;
        if (tid < D) {
            float M = -INFINITY;
            for (int j = 0; j < G; ++j) M = fmaxf(M, s_m[j]);
            float L = 0.f, A = 0.f;
            for (int j = 0; j < G; ++j) {
                const float f = s_m[j] == -INFINITY ? (s_l[j] == 0.f ? 0.f : 1.f) : tc::ex2(s_m[j] - M);
                L = fmaf(s_l[j], f, L);
                A = fmaf(s_acc[j][tid], f, A);
            }
            if (any_bad) M = L = A = __int_as_float(0x7fc00000);
            if (whole && !SHARED) {
                static_cast<T *>(a.out)[(long long)u * D + tid] = from_f<T>(A / L);
            } else {
                float *part = s.own + piece * (D + 2);
                part[2 + tid] = A;
                if (tid == 0) {
                    part[0] = M;
                    part[1] = L;
                }
            }
        }
        if (tid == 0) {
            s.own_flag[piece] = any_bad;
            if (tb == 0) s.first[u] = blockIdx.x;
            if (te == nt) s.last[u] = blockIdx.x;
        }
        __syncthreads();
        t += te - tb;
    }
}

// One (batch row, head): the pieces of its own part in block order, then the
// prefix's in block order. D threads.
template <typename T, int D, bool SHARED>
__global__ void __launch_bounds__(D) decode_join_kernel(PagedStep a, PagedScratch s, PagedPlan p)
{
    const int u = blockIdx.x, b = u / a.H, h = u % a.H, e = threadIdx.x;
    const int slot = slot_of(a.c, b);
    if (slot < 0) return;  // idle: out stays as it was
    T *out = static_cast<T *>(a.out) + (long long)u * D + e;
    bool bad = length_of(a.c, slot) < 0;
    if (a.c.rows) {  // two batch rows on one slot would update its keys twice
        for (int i = e; i < a.B; i += D) bad |= i != b && a.c.rows[i] == slot;
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        *out = from_f<T>(__int_as_float(0x7fc00000));
        if (e == 0) atomicMax(s.err, ERR_PAGE);
        return;
    }
    const int i0 = s.first[u], i1 = s.last[u];
    int flag = 0;
    for (int i = i0; i <= i1; ++i) flag |= s.own_flag[(long long)i + u];
    int j0 = 0, j1 = -1, row = 0;
    long long pu = 0;
    if (SHARED && a.prefix_len > 0) {
        // blocks of the prefix's units: block i holds tiles [total i / n, total (i + 1) / n)
        pu = (long long)h * p.q_tiles + b / p.q_tile;
        row = b % p.q_tile;
        const long long total = (long long)p.pre_units * p.key_tiles, t0 = pu * p.key_tiles;
        j0 = (int)(((t0 + 1) * p.pre_blocks - 1) / total);
        j1 = (int)(((t0 + p.key_tiles) * p.pre_blocks - 1) / total);
        for (int j = j0; j <= j1; ++j) flag |= s.pre_flag[j + pu];
    }
    if (flag && e == 0) atomicMax(s.err, ERR_PAGE);
    if (!SHARED && i0 == i1) return;  // one block held the whole unit and wrote out
    float M = -INFINITY;
    for (int i = i0; i <= i1; ++i) M = fmaxf(M, s.own[((long long)i + u) * (D + 2)]);
    for (int j = j0; j <= j1; ++j) M = fmaxf(M, s.pre_ml[(j + pu) * 2 * p.q_tile + row]);
    float L = 0.f, A = 0.f;
    for (int i = i0; i <= i1; ++i) {
        const float *x = s.own + ((long long)i + u) * (D + 2);
        const float f = x[0] == -INFINITY ? (x[1] == 0.f ? 0.f : 1.f) : tc::ex2(x[0] - M);
        L = fmaf(x[1], f, L);
        A = fmaf(x[2 + e], f, A);
    }
    for (int j = j0; j <= j1; ++j) {
        const float *ml = s.pre_ml + (j + pu) * 2 * p.q_tile + row;
        const float f = ml[0] == -INFINITY ? (ml[p.q_tile] == 0.f ? 0.f : 1.f) : tc::ex2(ml[0] - M);
        L = fmaf(ml[p.q_tile], f, L);
        A = fmaf(s.pre[((j + pu) * p.q_tile + row) * D + e], f, A);
    }
    if (flag) L = __int_as_float(0x7fc00000);
    *out = from_f<T>(A / L);
}

template <typename T, int D, bool SHARED>
cudaError_t run(const PagedStep &a, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    {
        Stage stage("decode_own", st);
        if (a.c.g)
            decode_own_kernel<T, D, true, SHARED><<<p.own_blocks, NT, 0, st>>>(a, s);
        else
            decode_own_kernel<T, D, false, SHARED><<<p.own_blocks, NT, 0, st>>>(a, s);
        count_launches();
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    Stage stage("decode_join", st);
    decode_join_kernel<T, D, SHARED><<<a.B * a.H, D, 0, st>>>(a, s, p);
    count_launches();
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t run(const PagedStep &a, bool shared, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    return shared ? run<T, D, true>(a, p, s, st) : run<T, D, false>(a, p, s, st);
}

}  // namespace

PagedPlan paged_plan(int B, int H, int max_pages, int page, int d, int dt, int prefix_len)
{
    PagedPlan p;
    const int sms = sm_count();
    const long long most = (long long)B * H * (((long long)max_pages * page - 1) / OWN_TILE + 1);
    long long blocks = 2LL * sms;
    if (blocks > OWN_MAX_BLOCKS) blocks = OWN_MAX_BLOCKS;
    if (blocks > most) blocks = most;
    p.own_blocks = (int)blocks;
    p.own_slots = p.own_blocks + B * H;
    p.q_tile = 32;
    p.key_tile = 64;
    p.q_tiles = ceil_div(B, p.q_tile);
    p.key_tiles = (int)(((long long)prefix_len + p.key_tile - 1) / p.key_tile);
    p.pre_units = p.q_tiles * H;
    const long long tiles = (long long)p.pre_units * p.key_tiles;
    p.pre_blocks = (int)(tiles < 2LL * sms ? tiles : 2LL * sms);
    p.pre_slots = prefix_len > 0 ? p.pre_blocks + p.pre_units : 0;
    return p;
}

size_t paged_carve(void *base, const PagedPlan &p, int B, int H, int d, PagedScratch &s)
{
    Carver c(base);
    const size_t nh = (size_t)B * H, own = p.own_slots, pre = p.pre_slots;
    s.err = c.take<int>(64);
    s.first = c.take<int>(nh);
    s.last = c.take<int>(nh);
    s.own = c.take<float>(own * (d + 2));
    s.own_flag = c.take<int>(own);
    s.qt = c.take<float>((size_t)p.q_tiles * p.q_tile * H * d);
    s.qg = c.take<float>((size_t)p.q_tiles * p.q_tile * H);
    s.pre = c.take<float>(pre * p.q_tile * d);
    s.pre_ml = c.take<float>(pre * 2 * p.q_tile);
    s.pre_flag = c.take<int>(pre);
    return c.bytes();
}

cudaError_t decode_paged(const PagedStep &a, int dt, int d, bool shared, const PagedPlan &p,
                         const PagedScratch &s, cudaStream_t st)
{
    if (d == 64) return dt == F32 ? run<float, 64>(a, shared, p, s, st) : run<bf16, 64>(a, shared, p, s, st);
    if (d == 128) return dt == F32 ? run<float, 128>(a, shared, p, s, st) : run<bf16, 128>(a, shared, p, s, st);
    return cudaErrorInvalidValue;
}

}  // namespace path
