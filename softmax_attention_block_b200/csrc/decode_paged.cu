// Paged decode step: every batch row updates its own cached keys in place and
// attends to them (Paper-Notes "训练策略", inference paragraph), with lengths
// and pages read on the device. Per head, with n = lens[slot]:
//   k_j <- k_j - beta w (w^T k_j), g_j <- g_j + log f    (j < n, rounded to dt)
//   row n <- k_new, v_new, g = 0;  out = softmax_j(scale q^T k_j + g_j) V.
//
// Bound by HBM: it reads K and V once and writes K once (3 d elements a row and
// head) for about 8 d operations. 48 rows of 500 to 6000 tokens, 24 heads of 64,
// bf16 with the gate: 250 us for 1475 MB, 5.9 TB/s (90% of a plain copy); 32 rows
// of 1 to 8192, 32 heads of 128: 580 us for 3331 MB, 5.7 TB/s (88%); fp32, 16 rows of
// 500 to 6000, 24 heads of 64: 172 us for 976 MB, 5.7 TB/s (87%). Another card was 3 to 8% slower.
//
// Rows differ in length, so the (row, head) units are cut into granules of 16 rows
// and the list of all granules is dealt out to the warps in equal contiguous shares
// (decode_own_kernel). A warp keeps its loads in flight across units, as bulk copies
// into a ring of its own: registers for loads in flight, as in the step over
// contiguous caches, left one block an SM here and took 1.7 to 3.5 times as long.
// Pieces of a unit meet in decode_join_kernel, in list order, so results repeat
// exactly. The lengths are on the device: each block adds them up itself.
#include "paged.cuh"
#include "rowvec.cuh"
#include "runtime.cuh"
#include "tc.cuh"

#include <type_traits>

namespace path {

namespace {

constexpr float LOG2E = 1.4426950408889634f;

// A warp's granule: GR rows of K and V (and gate biases) of one head, always inside one page.
// LPR lanes hold a row, 16 elements each as CPL 16-byte chunks; a pass takes 32 / LPR rows.
template <typename T, int D>
struct OwnCfg {
    // Warps of a block, and how many of them work when there is much to do. Rows of 128 bytes take
    // more instructions a byte, and the shares of short sequences wait for one another: twelve warps
    // instead of eight there (122 us instead of 129 for 96 rows of 0 to 512 tokens behind a prefix, 24
    // heads of 64). Long shares are bound by HBM, whose rate falls with the number of streams (288 us
    // instead of 250 for 48 rows of 500 to 6000). Even at about 45 granules for each of eight warps.
    static constexpr int WARPS = D * sizeof(T) == 128 ? 12 : 8, FEW = 8, NT = 32 * WARPS;
    static constexpr int LONG_SHARE = 40;
    static constexpr int LPR = D / 16, RPP = 32 / LPR;
    static constexpr int GR = own_granule(D, sizeof(T));
    static constexpr int PASSES = GR / RPP;
    static constexpr int CPL = sizeof(T);
    static constexpr int ROW_CHUNKS = D * (int)sizeof(T) / 16;
    static constexpr int TILE = GR * D * (int)sizeof(T);
    static constexpr int STAGES = 196608 / WARPS / (2 * TILE), MORE_STAGES = 196608 / FEW / (2 * TILE);  // of a warp
    static constexpr int GATE = GR * 4;
    static constexpr int ROW = D * (int)sizeof(T);
    // shared memory: the warps' rings of key and value tiles, then their units' q and w, then gate biases
    static constexpr int SLOTS = WARPS * STAGES > FEW * MORE_STAGES ? WARPS * STAGES : FEW * MORE_STAGES;
    static constexpr int SMEM = SLOTS * (2 * TILE + 2 * ROW + GATE);
    static_assert(GR % RPP == 0 && STAGES >= 3 && TILE % 128 == 0, "granule");
};

// Starting and ending a unit (one head of one batch row) takes a warp about as long as one
// granule, and the shares are dealt out with it: 96 rows of 0 to 512 tokens, 24 heads of 64, take
// 50 us instead of 67 without it and 51 with 2; long rows do not notice.
constexpr int UNIT_COST = 1;

// Cost of one head of batch row b (0: idle or invalid; the new token is a row).
template <int GR>
__device__ __forceinline__ int cost_of(const PagedCache &c, int b)
{
    const int slot = slot_of(c, b);
    if (slot < 0) return 0;
    const int n = length_of(c, slot);
    return n < 0 ? 0 : n / GR + 1 + UNIT_COST;
}

template <int WARPS>
__device__ long long block_scan(long long x, long long *total)
{
    __shared__ long long s_w[WARPS];
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
    for (int i = 0; i < WARPS; ++i) {
        if (i < warp) before += s_w[i];
        sum += s_w[i];
    }
    __syncthreads();
    *total = sum;
    return before + v - x;
}

// One 16-byte chunk to pairs, N of them.
template <typename T>
__device__ __forceinline__ void to_pairs(const uint4 &u, F2 *x)
{
    float f[Vec<T>::N];
    unpack<T>(u, f);
#pragma unroll
    for (int i = 0; i < Vec<T>::N / 2; ++i) x[i] = f2(f[2 * i], f[2 * i + 1]);
}

template <typename T>
__device__ __forceinline__ uint4 from_pairs(const F2 *x)
{
    float f[Vec<T>::N];
#pragma unroll
    for (int i = 0; i < Vec<T>::N / 2; ++i) split(x[i], f[2 * i], f[2 * i + 1]);
    return pack<T>(f);
}

__device__ __forceinline__ float dot16(const F2 *a, const F2 *b)
{
    F2 s0 = mul2(a[0], b[0]), s1 = mul2(a[1], b[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        s0 = fma2(a[i], b[i], s0);
        s1 = fma2(a[i + 1], b[i + 1], s1);
    }
    float x0, y0, x1, y1;
    split(s0, x0, y0);
    split(s1, x1, y1);
    return (x0 + y0) + (x1 + y1);
}

// Position in the list of all granules: unit (b, h), granule j of its nt. `left` is what
// remains of the warp's share, this granule included; nothing if it is not positive.
struct Cursor {
    int b, h, j, nt;
    int slot, n;
    long long left;

    template <int GR>
    __device__ __forceinline__ void at_row(const PagedCache &c, int row)
    {
        b = row;
        slot = slot_of(c, b);
        n = slot < 0 ? -1 : length_of(c, slot);
        nt = n < 0 ? 0 : n / GR + 1;
    }

    template <int GR>
    __device__ __forceinline__ void advance(const PagedStep &a)
    {
        --left;
        if (++j < nt) return;
        j = 0;
        left -= UNIT_COST;
        if (left <= 0 || ++h < a.H) return;
        h = 0;
        do {  // a row with granules follows, for something is left
            if (b + 1 >= a.B) {  // unless the lengths changed meanwhile
                left = 0;
                return;
            }
            at_row<GR>(a.c, b + 1);
        } while (nt == 0);
    }
};

// A unit's piece that a warp does not hold whole, for the block to put together.
template <int D>
struct Piece {
    int u, flags;  // unit; bit 0: from its first tile, bit 1: to its last, bits 2..: errors
    float m, l;
    float acc[D];
};
enum { FIRST = 1, LAST = 2, BAD_PAGE = PIECE_BAD_PAGE, GAVE_UP = PIECE_GAVE_UP };

template <typename T, int D, bool GATE, bool SHARED>
__global__ void __launch_bounds__(OwnCfg<T, D>::NT, 1) decode_own_kernel(PagedStep a, PagedScratch s)
{
    using C = OwnCfg<T, D>;
    constexpr int LPR = C::LPR, RPP = C::RPP, GR = C::GR, CPL = C::CPL, WARPS = C::WARPS, NT = C::NT;
    constexpr int VP = Vec<T>::N / 2;  // pairs of a chunk
    extern __shared__ __align__(128) char smem[];
    long long *s_cum = reinterpret_cast<long long *>(smem);  // before the rings are filled
    __shared__ uint64_t s_bar[WARPS][C::MORE_STAGES];
    __shared__ long long s_row[WARPS][C::MORE_STAGES];  // first row of the stage's granule in the pool, or -1
    __shared__ Piece<D> s_piece[WARPS][2];
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int lr = lane % LPR, grp = lane / LPR;
    const int odd = LPR == 4 ? grp & 1 : 0;
    const PagedCache &c = a.c;
    const int page = 1 << c.page_log2;

    release_next();
    if (lane == 0) {
        for (int i = 0; i < C::MORE_STAGES; ++i) tc::mbar_init(&s_bar[warp][i], 1);
        tc::mbar_fence_init();
        s_piece[warp][0].u = s_piece[warp][1].u = -1;
    }
    if (blockIdx.x == 0 && tid == 0) *s.err = 0;

    // this warp's share [t0, t1) of all cost, and the batch row that t0 lies in. A unit's cost
    // comes before its granules: a share that ends in it holds none of the unit's granules, one
    // that starts in it starts with its first. No share is empty, so the blocks between the
    // first and the last that hold granules of a unit hold some too.
    long long total = 0, mine = 0, at = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        long long sum;
        mine = b0 + tid < a.B ? (long long)cost_of<GR>(c, b0 + tid) * a.H : 0;
        at = block_scan<WARPS>(mine, &sum);
        total += sum;
    }
    const bool few = WARPS > C::FEW && total >= (long long)gridDim.x * C::FEW * C::LONG_SHARE;
    const int warps = few ? C::FEW : WARPS, S = few ? C::MORE_STAGES : C::STAGES;
    const long long nw = min((long long)gridDim.x * warps, total);
    const long long gw = warp < warps ? (long long)blockIdx.x * warps + warp : nw;
    const long long t0 = gw < nw ? total * gw / nw : total, t1 = gw < nw ? total * (gw + 1) / nw : total;
    Cursor cc{};
    long long cum = 0;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        long long sum = total;
        if (a.B > NT) {
            mine = b0 + tid < a.B ? (long long)cost_of<GR>(c, b0 + tid) * a.H : 0;
            at = block_scan<WARPS>(mine, &sum);
        }
        s_cum[tid] = cum + at;
        __syncthreads();
        if (t0 < t1 && cum <= t0 && t0 < cum + sum) {  // the last row whose tiles start at or before t0
            int lo = 0, hi = min(NT, a.B - b0) - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (s_cum[mid] <= t0)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            cc.at_row<GR>(c, b0 + lo);
            const long long off = t0 - s_cum[lo];
            const int at_unit = (int)(off % (cc.nt + UNIT_COST)) - UNIT_COST;
            cc.h = (int)(off / (cc.nt + UNIT_COST));
            cc.j = max(0, at_unit);
            cc.left = t1 - t0 + min(0, at_unit);
        }
        cum += sum;
        __syncthreads();
    }
    tc::fence_async_smem();  // s_cum's place now belongs to the copies
    if (a.withhold && blockIdx.x == 0 && tid == 0) tc::mbar_expect_more(&s_bar[0][1], 16);  // bytes that never come

    if (cc.left > 0) {
        const float scale2 = a.scale * LOG2E;
        char *ring = smem + warp * S * 2 * C::TILE, *head = smem + C::SLOTS * 2 * C::TILE + warp * S * 2 * C::ROW;
        float *gring = reinterpret_cast<float *>(smem + C::SLOTS * 2 * (C::TILE + C::ROW)) + warp * S * GR;
        T *K = static_cast<T *>(c.k), *Vp = static_cast<T *>(c.v);

        // The loads run ahead of the arithmetic by S granules, across units: a unit's first granule
        // brings q and w along (beta and log f wait in the stage's lane), its last one the new
        // token, which lands in the tile at its row.
        Cursor pc = cc;
        int tab_b = -1, tab_at = 0, tab = -1;  // 32 entries of row tab_b's table, one a lane
        // Values are not touched again before the next step; letting go of them first leaves L2 to the
        // keys on their way back (bf16, 32 rows of 32 heads of 128: 598 -> 580 us for 1 to 8192 tokens,
        // 161 -> 155 for 1 to 2000, 64.6 -> 65.0 for 1 to 700). At head dim 64 (251 -> 256 us for 48 rows
        // of 500 to 6000, 24 heads), at fp32 (16 rows of 500 to 6000: 172 -> 174 us for 24 heads of 64, 223
        // -> 224.5 for 16 of 128) or behind a prefix (202 -> 204) the hint costs more than it gives.
        constexpr bool HINT = sizeof(T) == 2 && D == 128 && !SHARED;
        const uint64_t once = HINT ? tc::l2_evict_first() : 0;
        bool begun = false;
        float p_beta = 0.f, p_lf = 0.f;
        auto load = [&](int st) {
            const int r0 = pc.j * GR, pg = r0 >> c.page_log2;
            if (pc.b != tab_b || pg < tab_at || pg >= tab_at + 32) {
                tab_b = pc.b;
                tab_at = pg;
                const int i = pg + lane;
                tab = i < c.max_pages ? c.table[(long long)pc.slot * c.max_pages + i] : -1;
            }
            const int p = __shfl_sync(0xffffffffu, tab, pg - tab_at);
            const bool ok = p >= 0 && p < c.n_pages, opens = pc.j == 0 || !begun;
            const long long row = ((long long)p * a.H + pc.h) * page + (r0 & (page - 1));
            const long long pu = (long long)pc.b * a.H + pc.h;
            if (opens && lane == st) {
                p_beta = a.beta[pu];
                if (GATE) p_lf = a.log_f[pu];
            }
            if (lane == 0) {
                s_row[warp][st] = ok ? row : -1;
                uint64_t *bar = &s_bar[warp][st];
                const int have = min(GR, pc.n - r0);  // cached rows of this granule
                const bool fresh = have < GR;
                const uint32_t bytes = have * C::ROW;
                char *tk = ring + st * 2 * C::TILE, *tv = tk + C::TILE;
                const uint32_t tx = (opens ? 2 * C::ROW : 0) +
                                    (ok ? 2 * bytes + (fresh ? 2 * C::ROW : 0) + (GATE ? C::GATE : 0) : 0);
                if (tx)
                    tc::mbar_expect_tx(bar, tx);
                else
                    tc::mbar_arrive(bar);
                if (opens) {
                    tc::bulk_load(head + st * 2 * C::ROW, static_cast<const T *>(a.q) + pu * D, C::ROW, bar);
                    tc::bulk_load(head + st * 2 * C::ROW + C::ROW, static_cast<const T *>(a.w) + pu * D, C::ROW, bar);
                }
                if (ok) {
                    if (bytes) {
                        tc::bulk_load(tk, K + row * D, bytes, bar);
                        if (HINT)
                            tc::bulk_load(tv, Vp + row * D, bytes, bar, once);
                        else
                            tc::bulk_load(tv, Vp + row * D, bytes, bar);
                    }
                    if (fresh) {
                        tc::bulk_load(tk + bytes, static_cast<const T *>(a.k_new) + pu * D, C::ROW, bar);
                        tc::bulk_load(tv + bytes, static_cast<const T *>(a.v_new) + pu * D, C::ROW, bar);
                    }
                    if (GATE) tc::bulk_load(gring + st * GR, c.g + row, C::GATE, bar);
                }
            }
            begun = true;
            pc.advance<GR>(a);
        };
        for (int i = 0; i < S && pc.left > 0; ++i) load(i);

        int st = 0, parity = 0, flags = 0, npiece = 0, u = -1, tb = 0;
        bool dead = false;
        float beta = 0.f, lf = 0.f, m = -INFINITY, l = 0.f;
        F2 q[8], w[8], acc[8];
        while (cc.left > 0) {
            if (!tc::mbar_wait(&s_bar[warp][st], parity, dead ? 0 : a.limit_ns)) {
                // Nothing more is worked on or loaded, but copies may still be on their way into this
                // block's memory: for this granule and the ring behind it (less of it at a share's end,
                // where the waits for the rest run out of time).
                if (!dead) {
#pragma unroll 1
                    for (int i = 0; i < S; ++i)
                        tc::mbar_wait(&s_bar[warp][(st + i) % S], st + i < S ? parity : parity ^ 1, a.limit_ns);
                }
                dead = true;
            }
            dead = __any_sync(0xffffffffu, dead);
            const long long row0 = s_row[warp][st];
            const int r0 = cc.j * GR, n = cc.n;
            if (u != cc.b * a.H + cc.h) {  // a new unit
                u = cc.b * a.H + cc.h;
                tb = cc.j;
                flags = 0;
                beta = __shfl_sync(0xffffffffu, p_beta, st);
                if (GATE) lf = __shfl_sync(0xffffffffu, p_lf, st);
                const uint4 *hq = reinterpret_cast<const uint4 *>(head + st * 2 * C::ROW);
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    const int x = lr + LPR * (j ^ odd);
                    to_pairs<T>(hq[x], q + j * VP);
                    to_pairs<T>(hq[C::ROW_CHUNKS + x], w + j * VP);
                }
                m = -INFINITY;
                l = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = 0ull;
            }
            if (dead) flags |= GAVE_UP;
            if (row0 < 0) flags |= BAD_PAGE;
            const uint4 *tk = reinterpret_cast<const uint4 *>(ring + st * 2 * C::TILE);
            const uint4 *tv = tk + C::TILE / 16;
            auto granule = [&](auto tail_tag) {
                constexpr bool TAIL = decltype(tail_tag)::value;
                float z[C::PASSES];
#pragma unroll
                for (int i = 0; i < C::PASSES; ++i) {
                    const int ri = i * RPP + grp, r = r0 + ri;
                    const bool valid = !TAIL || r <= n, fresh = TAIL && r == n;
                    uint4 kc[CPL];
                    F2 k[8];
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        const int x = lr + LPR * (j ^ odd);
                        kc[j] = tk[ri * C::ROW_CHUNKS + x];
                        to_pairs<T>(kc[j], k + j * VP);
                    }
                    const float nc = -(beta * group_sum<LPR>(dot16(w, k)));
                    const F2 nc2 = f2(nc, nc);
                    if (!TAIL || !fresh) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) k[e] = fma2(nc2, w[e], k[e]);
                    }
                    uint4 *dst = reinterpret_cast<uint4 *>(K + (row0 + ri) * D);
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        const int x = lr + LPR * (j ^ odd);
                        if (!TAIL || !fresh) kc[j] = from_pairs<T>(k + j * VP);
                        if (valid) dst[x] = kc[j];
                        if (sizeof(T) == 2) to_pairs<T>(kc[j], k + j * VP);  // the key as it is stored
                    }
                    float bias = 0.f;
                    if (GATE) {
                        bias = fresh ? 0.f : gring[st * GR + ri] + lf;
                        if (valid && lr == 0) c.g[row0 + ri] = bias;
                    }
                    z[i] = fmaf(group_sum<LPR>(dot16(q, k)), scale2, bias * LOG2E);
                    if (!valid) z[i] = -INFINITY;
                }
                float mn = m;
#pragma unroll
                for (int i = 0; i < C::PASSES; ++i) mn = fmaxf(mn, z[i]);
                const float base = mn == -INFINITY ? 0.f : mn;  // nothing weighs yet
                const float corr = tc::ex2(m - base);
                m = mn;
                l *= corr;
                const F2 c2 = f2(corr, corr);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = mul2(acc[e], c2);
#pragma unroll
                for (int i = 0; i < C::PASSES; ++i) {
                    const int ri = i * RPP + grp, r = r0 + ri;
                    const bool valid = !TAIL || r <= n, fresh = TAIL && r == n;
                    const float p = tc::ex2(z[i] - base);
                    l += p;
                    const F2 p2 = f2(p, p);
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        const int x = lr + LPR * (j ^ odd);
                        uint4 vc = make_uint4(0u, 0u, 0u, 0u);  // a row behind the last counts nothing
                        if (valid) vc = tv[ri * C::ROW_CHUNKS + x];
                        if (fresh) reinterpret_cast<uint4 *>(Vp + (row0 + ri) * D)[x] = vc;
                        F2 v[VP];
                        to_pairs<T>(vc, v);
#pragma unroll
                        for (int e = 0; e < VP; ++e) acc[j * VP + e] = fma2(p2, v[e], acc[j * VP + e]);
                    }
                }
            };
            if (row0 >= 0 && !dead) {
                if (r0 + GR > n)
                    granule(std::true_type{});
                else
                    granule(std::false_type{});
            }
            __syncwarp();  // the stage has been read
            if (pc.left > 0 && !dead) load(st);
            if (++st == S) {
                st = 0;
                parity ^= 1;
            }
            const bool ends = cc.j + 1 == cc.nt;
            const int u_done = u;
            const bool whole = ends && tb == 0;
            cc.advance<GR>(a);
            if (ends || cc.left <= 0) {  // the row groups join; then lanes 0 .. LPR - 1 hold the row
                float M = m;
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : tc::ex2(m - M);
                float L = l * f, x[16];
#pragma unroll
                for (int e = 0; e < 8; ++e) split(acc[e], x[2 * e], x[2 * e + 1]);
                if (LPR == 4) {  // odd rows hold neighbouring chunks in the other order
                    constexpr int N = Vec<T>::N;
#pragma unroll
                    for (int j = 0; j < CPL; j += 2)
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            const float y0 = x[j * N + e], y1 = x[(j + 1) * N + e];
                            x[j * N + e] = odd ? y1 : y0;
                            x[(j + 1) * N + e] = odd ? y0 : y1;
                        }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] *= f;
#pragma unroll
                for (int o = LPR; o < 32; o <<= 1) {
                    L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] += __shfl_xor_sync(0xffffffffu, x[e], o);
                }
                flags |= (tb == 0 ? FIRST : 0) | (ends ? LAST : 0);
                if (whole) {
                    const float nan = __int_as_float(0x7fc00000);
                    const long long piece = (long long)blockIdx.x + u_done;
                    const bool bad = flags & (BAD_PAGE | GAVE_UP);
                    if (lane < LPR) {
                        const float inv = bad ? nan : 1.f / L;
                        float *part = s.own + piece * (D + 2);
#pragma unroll
                        for (int j = 0; j < CPL; ++j) {
                            constexpr int N = Vec<T>::N;
                            const int ch = lane + LPR * j;
                            if (SHARED) {
#pragma unroll
                                for (int e = 0; e < N; e += 2)
                                    *reinterpret_cast<float2 *>(part + 2 + ch * N + e) =
                                        make_float2(x[j * N + e], x[j * N + e + 1]);
                            } else {
#pragma unroll
                                for (int e = 0; e < N; ++e) x[j * N + e] *= inv;
                                T *o = static_cast<T *>(a.out) + (long long)u_done * D + ch * N;
#pragma unroll
                                for (int e = 0; e < N; ++e) o[e] = from_f<T>(x[j * N + e]);
                            }
                        }
                        if (SHARED && lane == 0) {
                            part[0] = M;
                            part[1] = L;
                        }
                    }
                    if (lane == 0) {
                        s.own_flag[piece] = flags;
                        s.first[u_done] = s.last[u_done] = blockIdx.x;
                    }
                } else {
                    Piece<D> &pp = s_piece[warp][npiece++];
                    if (lane < LPR) {
#pragma unroll
                        for (int j = 0; j < CPL; ++j) {
                            constexpr int N = Vec<T>::N;
#pragma unroll
                            for (int e = 0; e < N; ++e) pp.acc[(lane + LPR * j) * N + e] = x[j * N + e];
                        }
                    }
                    if (lane == 0) {
                        pp.u = u_done;
                        pp.flags = flags;
                        pp.m = M;
                        pp.l = L;
                    }
                }
            }
        }
    }
    // this kernel needs nothing of the ones before it in the call, but completes after them
    if (SHARED && tid == 0) wait_previous();
    __syncthreads();

    // The pieces of the block's warps, in order: neighbours of one unit are put together.
    const Piece<D> *pieces = &s_piece[0][0];
    for (int i = 0; i < 2 * WARPS;) {
        const int u = pieces[i].u;
        if (u < 0) {
            ++i;
            continue;
        }
        int end = i, flags = 0;
        float M = -INFINITY;
        for (; end < 2 * WARPS && (pieces[end].u == u || pieces[end].u < 0); ++end) {
            if (pieces[end].u < 0) continue;
            flags |= pieces[end].flags;
            M = fmaxf(M, pieces[end].m);
        }
        const long long piece = (long long)blockIdx.x + u;
        if (tid < D) {
            float L = 0.f, A = 0.f;
            for (int k = i; k < end; ++k) {
                if (pieces[k].u < 0) continue;
                const float mk = pieces[k].m, lk = pieces[k].l;
                const float f = mk == -INFINITY ? (lk == 0.f ? 0.f : 1.f) : tc::ex2(mk - M);
                L = fmaf(lk, f, L);
                A = fmaf(pieces[k].acc[tid], f, A);
            }
            if (flags & (BAD_PAGE | GAVE_UP)) L = A = __int_as_float(0x7fc00000);
            if ((flags & FIRST) && (flags & LAST) && !SHARED) {
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
            s.own_flag[piece] = flags;
            if (flags & FIRST) s.first[u] = blockIdx.x;
            if (flags & LAST) s.last[u] = blockIdx.x;
        }
        i = end;
    }
}

// One (batch row, head): the pieces of its own part in block order, then the prefix's in block
// order. Their weights are worked out by the threads side by side, a batch of pieces at a time;
// then each thread adds up one output element over its share of them, its loads in flight together.
// NT = D threads where there are many units of few pieces, 256 where there are few units, which
// then have many (9 x 6, 33 pieces: 2 us less). Behind 8192 tokens, heads of 64, a step takes with
// D and with 256: 39.8 and 38.2 us at 192 units, 50.6 and 50.0 at 512, 59.4 and 58.6 at 768, 67.9 and
// 70.7 at 1152, 91.5 and 98.5 at 2048; heads of 128 or no prefix alike, within 2%.
template <typename T, int D, bool SHARED, int NT>
__global__ void __launch_bounds__(NT) decode_join_kernel(PagedStep a, PagedScratch s, PagedPlan p)
{
    constexpr int G = NT / D;  // threads of an output element
    __shared__ float s_f[NT], s_red[2][NT / 32], s_acc[NT];
    const int u = blockIdx.x, b = u / a.H, h = u % a.H, tid = threadIdx.x, e = tid % D, grp = tid / D;
    const int slot = slot_of(a.c, b);
    bool bad = slot >= 0 && length_of(a.c, slot) < 0;
    if (a.c.rows && slot >= 0) {  // two batch rows on one slot would update its keys twice
        for (int i = tid; i < a.B; i += NT) bad |= i != b && a.c.rows[i] == slot;
    }
    int j0 = 0, nj = 0, row = 0;
    long long pu = 0;
    if (SHARED) {
        // blocks of the prefix's units: block i holds tiles [total i / n, total (i + 1) / n)
        pu = (long long)h * p.q_tiles + b / p.q_tile;
        row = b % p.q_tile;
        const long long total = (long long)p.pre_units * p.key_tiles, t0 = pu * p.key_tiles;
        j0 = (int)(((t0 + 1) * p.pre_blocks - 1) / total);
        nj = (int)(((t0 + p.key_tiles) * p.pre_blocks - 1) / total) - j0 + 1;
    }
    wait_previous();
    bad = __syncthreads_or(bad);
    if (slot < 0) return;  // idle: out stays as it was
    T *out = static_cast<T *>(a.out) + (long long)u * D + e;
    if (bad) {
        if (grp == 0) *out = from_f<T>(__int_as_float(0x7fc00000));
        if (tid == 0) atomicMax(s.err, ERR_PAGE);
        return;
    }
    const int i0 = s.first[u], ni = s.last[u] - i0 + 1, np = ni + nj;
    // piece k: its maximum, sum, accumulator and flags
    auto ml = [&](int k, float &m, float &l, int &flag) {
        if (k < ni) {
            const long long x = (long long)i0 + k + u;
            m = s.own[x * (D + 2)];
            l = s.own[x * (D + 2) + 1];
            flag |= s.own_flag[x];
        } else {
            const long long x = (long long)j0 + k - ni + pu;
            m = s.pre_ml[x * 2 * p.q_tile + row];
            l = s.pre_ml[x * 2 * p.q_tile + p.q_tile + row];
            flag |= s.pre_flag[4 * x + row / 16];
        }
    };
    int flag = 0;
    float M = -INFINITY;
    if (!SHARED && ni == 1) {  // the block that held the whole unit wrote out
        flag = s.own_flag[(long long)i0 + u];
    } else {
        for (int k = tid; k < np; k += NT) {
            float m, l;
            ml(k, m, l, flag);
            M = fmaxf(M, m);
        }
    }
    flag &= BAD_PAGE | GAVE_UP;
    if (flag) atomicMax(s.err, flag & BAD_PAGE ? ERR_PAGE : ERR_PAGED_WAIT);
    if (!SHARED && ni == 1) return;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (tid % 32 == 0) s_red[0][tid / 32] = M;
    bad = __syncthreads_or(flag);
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) M = fmaxf(M, s_red[0][i]);
    float L = 0.f, A = 0.f;
    for (int k0 = 0; k0 < np; k0 += NT) {
        const int n = min(NT, np - k0), own = min(n, max(0, ni - k0));
        __syncthreads();
        if (tid < n) {
            float m, l;
            ml(k0 + tid, m, l, flag);
            const float f = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : tc::ex2(m - M);
            s_f[tid] = f;
            L = fmaf(l, f, L);
        }
        __syncthreads();
        const float *x = s.own + ((long long)i0 + k0 + u) * (D + 2) + 2 + e;
#pragma unroll 4
        for (int k = grp; k < own; k += G) A = fmaf(x[k * (D + 2)], s_f[k], A);
        if (SHARED) {
            const float *y = s.pre + ((j0 + k0 - ni + pu) * p.q_tile + row) * D + e;
#pragma unroll 8
            for (int k = own + grp; k < n; k += G) A = fmaf(y[(long long)k * p.q_tile * D], s_f[k], A);
        }
    }
    L = group_sum<32>(L);
    if (tid % 32 == 0) s_red[1][tid / 32] = L;
    s_acc[tid] = A;
    __syncthreads();
    if (grp > 0) return;
    L = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) L += s_red[1][i];
#pragma unroll
    for (int i = 1; i < G; ++i) A += s_acc[i * D + e];
    if (bad) L = __int_as_float(0x7fc00000);
    *out = from_f<T>(A / L);
}

template <typename T, int D, bool GATE, bool SHARED>
cudaError_t run_own(const PagedStep &a, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    auto k = decode_own_kernel<T, D, GATE, SHARED>;
    constexpr int smem = OwnCfg<T, D>::SMEM, NT = OwnCfg<T, D>::NT;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (SHARED) return launch_overlapped(k, p.own_blocks, NT, smem, st, a, s);
    k<<<p.own_blocks, NT, smem, st>>>(a, s);
    count_launches();
    return cudaGetLastError();
}

template <typename T, int D, bool SHARED>
cudaError_t run(const PagedStep &a, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    {
        Stage stage("decode_own", st);
        cudaError_t e = a.c.g ? run_own<T, D, true, SHARED>(a, p, s, st) : run_own<T, D, false, SHARED>(a, p, s, st);
        if (e != cudaSuccess) return e;
    }
    Stage stage("decode_join", st);
    const int units = a.B * a.H;
    if (units > 6 * sm_count()) return launch_overlapped(decode_join_kernel<T, D, SHARED, D>, units, D, 0, st, a, s, p);
    return launch_overlapped(decode_join_kernel<T, D, SHARED, 256>, units, 256, 0, st, a, s, p);
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
    const int gr = own_granule(d, (int)dtype_size(dt));
    const long long most = (long long)B * H * (((long long)max_pages * page - 1) / gr + 1);
    const long long blocks = (most + 7) / 8;  // eight warps or more
    p.own_blocks = (int)(blocks < sms ? blocks : sms);
    p.own_slots = p.own_blocks + B * H;
    // bf16: the prefix is read once for up to 64 queries (48 at d = 128: shared memory), tiles of even
    // size (their softmax is what can take longer than the loads); fp32: tiles of 32 on CUDA cores, of
    // 16 for few rows. Behind 16384 tokens, 8 heads, a step takes with 16 and with 32: at d = 128 72.5 and
    // 93.4 us for 12 rows, 73.0 and 95.2 for 16, 115.5 and 95.4 for 17; at d = 64 54.1 and 56.6 for 4
    // rows, 60.2 and 56.7 for 8, 73.0 and 59.5 for 16. Behind 2047 they are even at d = 64.
    if (dt == BF16)
        p.q_tile = ceil_div(ceil_div(B, ceil_div(B, d == 64 ? 64 : 48)), 16) * 16;
    else
        p.q_tile = B <= (d == 64 ? 4 : 16) ? 16 : 32;
    p.q_tiles = ceil_div(B, p.q_tile);
    p.key_tile = dt == BF16 ? 128 : 64;
    p.key_tiles = (int)(((long long)prefix_len + p.key_tile - 1) / p.key_tile);
    p.pre_units = p.q_tiles * H;
    const long long tiles = (long long)p.pre_units * p.key_tiles;
    const int most_blocks = dt == BF16 ? sms : 2 * sms;
    p.pre_blocks = (int)(tiles < most_blocks ? tiles : most_blocks);
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
    s.qt = reinterpret_cast<float *>(c.take<bf16>(PREFIX_PARTS * (size_t)p.q_tiles * p.q_tile * H * d));  // fp32: less
    s.qg = c.take<float>((size_t)p.q_tiles * p.q_tile * H);
    // room for the largest tile, so that a larger batch never needs less
    s.pre = c.take<float>(pre * 64 * d);
    s.pre_ml = c.take<float>(pre * 2 * 64);
    s.pre_flag = c.take<int>(4 * pre);
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
