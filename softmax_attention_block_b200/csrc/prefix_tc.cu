// Decode attention of a batch to one shared prefix on the tensor cores (bf16).
//
// The mathematics is that of prefix_attn.cu: queries qt = G^T q against the
// prefix's keys as they lie in the pages, one softmax per query. The prefix is
// read once for up to 64 queries, so the kernel is bound by HBM (4 d bytes a key
// and head) as long as the arithmetic hides behind the loads. Per tile of 128 keys
//   S^T [128 keys x queries] = K . qt^T        (A = K as stored, B = qt)
//   O^T [d x queries]       += V^T . P         (A = V transposed, B = P as written)
// keys lie along the 128 lanes of tensor memory: a thread holds one key, so the
// gate bias and the end of the prefix are one number a thread, and with few
// queries no lane idles (queries along the lanes would leave 3 of 4 empty at 32).
// Both products come out in the layout that the next step reads.
//
// bf16 operands alone would cost as much accuracy as the rounding of the output, and sums
// of two bf16 numbers (off by 2^-17) still show in the outputs' last bits. So qt and P are
// each split in three (hi + mid + lo), which hold an fp32 number's 24 bits: nothing of either
// is rounded. The products are S^T's D / 16 steps for each part, the small parts first, and
// 8 steps for O^T with the parts side by side as columns.
//
// A step cuts the sum so far to 24 bits instead of rounding it, so a long O^T would drift towards
// zero (832 steps: by 3.4e-5 of the weights' sum). Every 8 tiles (4 at D = 128) the softmax warps
// therefore add its parts to a total in tensor memory, in rounded fp32, and start them from zero
// (0.8e-6 every 8). For the step of 96 x 24 heads of 64 below, never, every 8 and every 4 tiles take
// 121, 123 and 126 us; at 32 x 32 of 128 156.2, 157.0 and 157.4, and 1.3, 0.62 and 0.37 e-4 of the
// output's norm differ from 64 bits rounded once.
//
// The running maximum of a query is a reference that moves only when a logit
// passes it by more than 2^8 (or at a unit's first tile): then the warps that
// hold the query agree on the new one and O^T joins its total, scaled. Otherwise a tile
// needs no maximum across threads at all: weights stay below 2^8 and sums and
// products are fp32. A thread keeps the sum of its own keys' weights per query;
// they are added up across threads at a unit's end.
//
// Warps: groups of four for the softmax of 16 queries each (they share nothing but the
// barriers towards the MMAs; the chain of one group, not its instructions, is what a tile
// waits for, and 16 columns a thread leave room for three or four groups), then one for the
// loads (a box of min(page, 128) rows a page, TMA) and one to issue each of the two products:
// a single warp takes longer to issue a tile's MMAs than the tensor cores to do them.
// Waits are bounded; one that gives up makes its pieces NaN and is reported.
//
// 32 queries, 32 heads of 128, 16384 keys: 58 us for 268 MB, DRAM 58% and the tensor pipe 23%
// busy (51 us with two parts). 96 queries, 24 heads of 64, gate: 59 us, DRAM 24%, tensor pipe 37%
// and half of the issue slots busy: nothing is full, a tile of keys and 48 queries takes 1.3 us, the
// chain of its logits, agreement, weights and product.
#include "paged.cuh"
#include "runtime.cuh"
#include "tc.cuh"

namespace path {

namespace {

using namespace tc;

constexpr int KT = 128;
constexpr int CN = 16;  // queries of a softmax group
constexpr int PARTS = PREFIX_PARTS;  // bf16 numbers that make an fp32 one
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LOW = -1e30f;  // reference of a query that has no weight yet
constexpr float SLACK = 8.f;

// GROUPS softmax groups: units of QT = 16 GROUPS queries, QN the distance of the two S^T.
template <int D, int GROUPS>
struct Cfg {
    static constexpr int PANELS = D / 64, QT = CN * GROUPS, QN = QT <= 32 ? 32 : 64;
    static constexpr int W_LOAD = 4 * GROUPS, W_S = W_LOAD + 1, W_O = W_S + 1, NT = 32 * (W_O + 1);
    static constexpr int TILE = KT * D * 2;             // one operand tile
    static constexpr int Q = PARTS * QT * D * 2;        // hi, mid, lo
    static constexpr int PP = KT * 128;                 // one panel of P: 64 columns
    static constexpr int P_PANELS = (PARTS * QT + 63) / 64, P = P_PANELS * PP;  // hi | mid | lo side by side
    static constexpr int NP = D == 128 && QT > 32 ? 1 : 2;  // buffers of P
    // buffers of keys and values: what is left
    static constexpr int NK = D == 64 ? P_PANELS == 3 ? 3 : 4 : QT == 16 ? 3 : 2, NV = D == 64 ? NK : 2, NG = NV + 1;
    static constexpr int K_OFF = 0, V_OFF = K_OFF + NK * TILE, Q_OFF = V_OFF + NV * TILE, P_OFF = Q_OFF + Q;
    static constexpr int G_OFF = P_OFF + NP * P, M_OFF = G_OFF + NG * KT * 4, F_OFF = M_OFF + QN * 4;
    static constexpr int RED_OFF = F_OFF + QN * 4, BAR_OFF = RED_OFF + 4 * QN * 4;
    static constexpr int NBAR = 2 * NK + 2 * NV + 9;
    static constexpr int SMEM = BAR_OFF + NBAR * 8 + 16 + 1024;
    static constexpr int T_S = 0, T_O = 2 * QN, T_T = T_O + PARTS * QT, T_END = T_T + QT;  // two S^T, O^T for hi | mid | lo, its total
    static constexpr int FOLD = D == 64 ? 8 : 4;  // tiles after which O^T's parts are added to its total
    static constexpr int TMEM = T_END <= 128 ? 128 : T_END <= 256 ? 256 : 512;
    static_assert(SMEM <= 232448, "shared memory");
};

// Barriers of one softmax group.
__device__ __forceinline__ void group_bar(int grp) { asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory"); }

__device__ __forceinline__ bool group_any(int grp, bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(1 + grp)
        : "memory");
    return r != 0;
}

// Sum or maximum over the warp's lanes of each of 16 values; lane i gets the i % 16-th. Halves of
// the values change places with halves of the lanes: 31 shuffles in all.
template <bool SUM>
__device__ __forceinline__ float warp_reduce(float (&v)[CN])
{
    auto both = [](float x, float y) { return SUM ? x + y : fmaxf(x, y); };
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i < CN; ++i) v[i] = both(v[i], __shfl_xor_sync(0xffffffffu, v[i], 16));
#pragma unroll
    for (int o = CN / 2; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float send = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = both(keep, __shfl_xor_sync(0xffffffffu, send, o));
        }
    }
    return v[0];
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int D, int GROUPS>
__global__ void __launch_bounds__(Cfg<D, GROUPS>::NT, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                     const __grid_constant__ CUtensorMap mV, PagedStep a, PagedScratch s, PagedPlan p)
{
    using C = Cfg<D, GROUPS>;
    constexpr int QT = C::QT, QN = C::QN;
    constexpr int NK = C::NK, NV = C::NV, NG = C::NG, NP = C::NP, PANELS = C::PANELS;
    constexpr int W_LOAD = C::W_LOAD, W_S = C::W_S, W_O = C::W_O;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + (1024 - (smem_u32(smraw) & 1023)) % 1024;
    uint64_t *k_full = reinterpret_cast<uint64_t *>(sm + C::BAR_OFF), *k_empty = k_full + NK;
    uint64_t *v_full = k_empty + NK, *v_empty = v_full + NV;
    uint64_t *q_full = v_empty + NV, *q_empty = q_full + 1, *s_full = q_full + 2, *p_full = q_full + 4;
    // P and its product: a barrier for each parity of the tile, since one group may be a tile ahead
    uint64_t *o_done = q_full + 6, *mma_done = q_full + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(q_full + 9);
    int *s_bad = reinterpret_cast<int *>(tmem_slot + 1);
    float *sG = reinterpret_cast<float *>(sm + C::G_OFF), *sM = reinterpret_cast<float *>(sm + C::M_OFF);
    float *sF = reinterpret_cast<float *>(sm + C::F_OFF), *sR = reinterpret_cast<float *>(sm + C::RED_OFF);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const bool gate = a.c.g != nullptr;

    release_next();
    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&p_full[i], 4 * GROUPS);  // a warp each
            mbar_init(&s_full[i], 3);  // the product, the warp that issued it, P's buffer
            mbar_init(&o_done[i], 1);
        }
        mbar_init(mma_done, 2);
        mbar_fence_init();
        if (a.withhold && blockIdx.x == 0) mbar_expect_more(&k_full[1], 16);  // bytes that never come
        *s_bad = 0;
    }
    if (warp == W_O) tmem_alloc(tmem_slot, C::TMEM);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tbase = *tmem_slot;

    // this block's share of all (unit, key tile) pairs; a segment is its part of one unit
    const long long total = (long long)p.pre_units * p.key_tiles;
    const long long t0 = total * blockIdx.x / gridDim.x, t1 = total * (blockIdx.x + 1) / gridDim.x;
    const int count = (int)(t1 - t0);
    const int q_rows = p.q_tiles * QT;

    if (warp == W_LOAD) {
        const int log2p = a.c.page_log2, page = 1 << log2p, box = page < KT ? page : KT, boxes = KT / box;
        const int npre = (a.prefix_len + page - 1) >> log2p;
        int tab = -1, tab_at = 0, tab_end = 0, issued_k = 0, issued_v = 0, seg = 0;
        bool ok = true;
        // position in the list, kept by hand: a division a tile would take longer than its loads
        int u = (int)(t0 / p.key_tiles), kt = (int)(t0 % p.key_tiles), h = u / p.q_tiles, qt = u % p.q_tiles;
        for (int n = 0; n < count && ok; ++n, ++kt) {
            if (kt == p.key_tiles) {
                kt = 0;
                if (++qt == p.q_tiles) {
                    qt = 0;
                    ++h;
                }
            }
            const int key0 = kt * KT;
            if (n == 0 || kt == 0) {
                // lanes may run out of time one by one: they go on, or leave, together
                ok = __all_sync(0xffffffffu, seg == 0 || mbar_wait(q_empty, (seg - 1) & 1, a.limit_ns));
                if (!ok) break;
                if (seg == 0) wait_previous();  // the queries; keys and values are nobody's output
                if (lane == 0) {
                    mbar_expect_tx(q_full, C::Q);
                    const int row = h * q_rows + qt * QT;
                    for (int x = 0; x < PARTS * PANELS; ++x)
                        tma_load_2d(sm + C::Q_OFF + x * QT * 128, &mQ, 64 * (x % PANELS), x / PANELS * a.H * q_rows + row, q_full);
                }
                ++seg;
            }
            // this lane's box: a page, or a part of a large one
            const int first = key0 >> log2p, key = key0 + lane * box;
            if (first < tab_at || first + boxes > tab_end) {
                tab_at = first;
                tab_end = first + 32;
                tab = first + lane < npre ? a.prefix_table[first + lane] : -1;
            }
            const int pid = __shfl_sync(0xffffffffu, tab, ((key >> log2p) - tab_at) & 31);
            const bool in = lane < boxes && key < a.prefix_len;
            const bool good = in && pid >= 0 && pid < a.c.n_pages;
            if (in && !good) *s_bad = 1;
            const int cnt = __popc(__ballot_sync(0xffffffffu, good));
            const int row = good ? (int)((((long long)pid * a.H + h) << log2p) + (key & (page - 1))) : 0;
            const uint32_t ks = (uint32_t)n % NK, vs = (uint32_t)n % NV, gs = (uint32_t)n % NG;
            if (n >= NK && !mbar_wait(&k_empty[ks], (n / NK - 1) & 1, a.limit_ns)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                // (a gate slot is free: tile n - NG = n - 1 - NV was done before V of tile n - 1 was loaded)
                if (cnt) mbar_expect_tx(&k_full[ks], cnt * box * (D * 2 + (gate ? 4 : 0)));
                else mbar_arrive(&k_full[ks]);
            }
            __syncwarp();
            if (good) {
                for (int x = 0; x < PANELS; ++x)
                    tma_load_2d(sm + C::K_OFF + ks * C::TILE + x * KT * 128 + lane * box * 128, &mK, 64 * x, row, &k_full[ks]);
                if (gate) bulk_load(sG + gs * KT + lane * box, a.c.g + row, box * 4, &k_full[ks]);
            }
            issued_k = n + 1;
            if (n >= NV && !mbar_wait(&v_empty[vs], (n / NV - 1) & 1, a.limit_ns)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                if (cnt) mbar_expect_tx(&v_full[vs], cnt * box * D * 2);
                else mbar_arrive(&v_full[vs]);
            }
            __syncwarp();
            if (good) {
                for (int x = 0; x < PANELS; ++x)
                    tma_load_2d(sm + C::V_OFF + vs * C::TILE + x * KT * 128 + lane * box * 128, &mV, 64 * x, row, &v_full[vs]);
            }
            issued_v = n + 1;
        }
        // leave no copy on its way into this block's memory: whoever waited for it may have given up
        for (int n = max(0, issued_k - NK); n < issued_k; ++n)
            mbar_wait(&k_full[n % NK], (n / NK) & 1, 8 * a.limit_ns);
        for (int n = max(0, issued_v - NV); n < issued_v; ++n)
            mbar_wait(&v_full[n % NV], (n / NV) & 1, 8 * a.limit_ns);
        if (seg > 0) mbar_wait(q_full, (seg - 1) & 1, 8 * a.limit_ns);
    } else if (warp == W_S) {
        // S^T = K . qt^T, lo, mid, hi: the sum that a step cuts is small until hi comes. The whole warp runs along, converged, and one lane issues:
        // descriptors stay uniform, and differ from a base by the address in their low bits.
        const uint32_t issue = lane == 0;
        constexpr uint32_t id = idesc_f16(128, QT, AB_BF16, 0, 0);
        const uint64_t k0 = desc_sw128(smem_u32(sm + C::K_OFF), 16, 1024), q0 = desc_sw128(smem_u32(sm + C::Q_OFF), 16, 1024);
        int kt = (int)(t0 % p.key_tiles), seg = 0;
        bool ok = true;
        for (int n = 0; n < count; ++n) {
            const uint32_t ks = (uint32_t)n % NK;
            if (n == 0 || kt == 0) ok = mbar_wait(q_full, seg++ & 1, a.limit_ns);
            ok = ok && mbar_wait(&k_full[ks], (n / NK) & 1, a.limit_ns);
            // the buffer of S^T was read before the weights of tile n - 2 were complete
            if (n >= 2) ok = ok && mbar_wait(&p_full[n & 1], ((n >> 1) - 1) & 1, a.limit_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fence_after_sync();
            const uint64_t kd = k0 + ks * (C::TILE >> 4);
            const uint32_t d = tbase + C::T_S + (n & 1) * QN;
#pragma unroll
            for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss_if(issue, d, kd + (((kk / 4) * KT * 128 + (kk % 4) * 32) >> 4),
                              q0 + (((part * PANELS + kk / 4) * QT * 128 + (kk % 4) * 32) >> 4), id, part < PARTS - 1 || kk > 0);
            commit_if(issue, &s_full[n & 1]);
            commit_if(issue, &k_empty[ks]);
            if (++kt == p.key_tiles) kt = 0;
            if (n + 1 == count || kt == 0) commit_if(issue, q_empty);
            // A wait costs a softmax warp 150 cycles even where there is nothing to wait for, so one
            // stands for three: tile n may be worked on once its logits are there, its gate biases (they
            // came with the keys, which this warp saw) and the buffer of its weights (free at first).
            if (lane == 0) {
                mbar_arrive(&s_full[n & 1]);
                if (n < NP) mbar_arrive(&s_full[n & 1]);
            }
        }
        // the tensor memory is freed after the issuing warps leave: no MMA may still be running then
        commit_if(issue, mma_done);
        mbar_wait(mma_done, 0, 8 * a.limit_ns);
    } else if (warp == W_O) {
        // O^T += V^T . P, hi | mid | lo as columns
        const uint32_t issue = lane == 0;
        constexpr uint32_t id = idesc_f16(D, PARTS * QT, AB_BF16, 1, 1);
        const uint64_t v0 = desc_sw128(smem_u32(sm + C::V_OFF), KT * 128, 1024), p0 = desc_sw128(smem_u32(sm + C::P_OFF), C::PP, 1024);
        int kt = (int)(t0 % p.key_tiles);
        bool ok = true;
        for (int n = 0; n < count; ++n) {
            const uint32_t vs = (uint32_t)n % NV;
            ok = mbar_wait(&v_full[vs], (n / NV) & 1, a.limit_ns) && mbar_wait(&p_full[n & 1], (n >> 1) & 1, a.limit_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            fence_after_sync();
            const uint64_t vd = v0 + vs * (C::TILE >> 4), pd = p0 + (n % NP) * (C::P >> 4);
            const bool fresh = n == 0 || kt == 0;
            if (++kt == p.key_tiles) kt = 0;
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk)
                mma_ss_if(issue, tbase + C::T_O, vd + (kk * 2048 >> 4), pd + (kk * 2048 >> 4), id, !fresh || kk > 0);
            commit_if(issue, &v_empty[vs]);
            commit_if(issue, &s_full[(n + NP) & 1]);  // tile n + NP may have this one's weights' place
            commit_if(issue, &o_done[n & 1]);
        }
        commit_if(issue, mma_done);
        mbar_wait(mma_done, 0, 8 * a.limit_ns);
    } else {
        // thread = key of the tile (a lane of S^T), queries c0 .. c0 + 15; then a row of O^T: dim gt,
        // or at D = 64 dim 16 (warp % 4) + lane in the lanes below 16. Waits that give up leave a mark
        // and go on (every address is fixed, every barrier is still met): the pieces become NaN.
        const int grp = warp / 4, gt = tid % 128, c0 = grp * CN;
        const uint32_t lane_off = (uint32_t)(32 * (warp % 4)) << 16;
        const float scale2 = a.scale * LOG2E;
        bool gave_up = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!mbar_try_wait(bar, parity) && !gave_up) gave_up = !mbar_wait(bar, parity, a.limit_ns);
            __syncwarp();
        };
        auto product_done = [&](int i) { wait(&o_done[i & 1], (i >> 1) & 1); };
        // this thread's row of P: where each part's first chunk of eight queries lies (the second is
        // its neighbour, 16 bytes off in one direction or the other)
        uint32_t p_at[PARTS];
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
            const int col = part * QT + c0;
            p_at[part] = col / 64 * C::PP + sw128_offset(gt, col % 64);
        }
        uint32_t gslot = 0;
        int n = 0, u = (int)(t0 / p.key_tiles), kb = (int)(t0 % p.key_tiles);
        int h = u / p.q_tiles, qt = u % p.q_tiles;
        while (n < count) {
            const int ke = min(p.key_tiles, kb + count - n);
            const int nq = min(CN, a.B - qt * QT - c0);  // queries of this unit and group
            float l[CN];
            bool folded = false;  // whether O^T's total holds anything
#pragma unroll
            for (int i = 0; i < CN; ++i) l[i] = 0.f;
            auto o_sum = [&](float (&o)[CN]) {  // the small parts first
                tmem_ld16_wait(tbase + C::T_O + (PARTS - 1) * QT + c0 + lane_off, o);
#pragma unroll 1
                for (int part = PARTS - 2; part >= (folded ? -1 : 0); --part) {
                    float x[CN];
                    tmem_ld16_wait(tbase + (part < 0 ? C::T_T : C::T_O + part * QT) + c0 + lane_off, x);
#pragma unroll
                    for (int i = 0; i < CN; ++i) o[i] += x[i];
                }
            };
            for (int kt = kb; kt < ke; ++kt, ++n) {
                const bool first = kt == kb, tail = (kt + 1) * KT > a.prefix_len;
                const bool live = !tail || kt * KT + gt < a.prefix_len;
                float v[CN], g = 0.f;
                float z[CN];
                auto minus_ref = [&]() {
#pragma unroll
                    for (int i = 0; i < CN; i += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(sM + c0 + i);
                        z[i] += m.x;
                        z[i + 1] += m.y;
                        z[i + 2] += m.z;
                        z[i + 3] += m.w;
                    }
                };
                wait(&s_full[n & 1], (n >> 1) & 1);
                if (gate) {
                    g = sG[gslot * KT + gt] * LOG2E;
                    if (++gslot == NG) gslot = 0;
                }
                fence_after_sync();
                tmem_ld16_wait(tbase + C::T_S + (n & 1) * QN + c0 + lane_off, v);
                auto logits = [&]() {
#pragma unroll
                    for (int i = 0; i < CN; ++i) z[i] = fmaf(v[i], scale2, g);
                    if (tail) {  // the page's rows behind the prefix hold anything
#pragma unroll
                        for (int i = 0; i < CN; ++i) z[i] = live ? z[i] : -INFINITY;
                    }
                };
                logits();
                float top = -INFINITY;
                if (!first) {
                    minus_ref();
#pragma unroll
                    for (int i = 0; i < CN; i += 2) asm("max.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(z[i]), "f"(z[i + 1]));
                }
                if (group_any(grp, first || n % C::FOLD == 0 || top > SLACK)) {
                    logits();
                    const float mine = warp_reduce<false>(z);
                    if (lane < CN) sR[(warp % 4) * QN + c0 + lane] = mine;
                    group_bar(grp);
                    if (gt < CN) {
                        const int c = c0 + gt;
                        const float old = first ? -INFINITY : -sM[c];
                        float x = fmaxf(fmaxf(sR[c], sR[QN + c]), fmaxf(sR[2 * QN + c], sR[3 * QN + c]));
                        x = fmaxf(fmaxf(old, x), LOW);
                        sM[c] = -x;
                        sF[c] = ex2(old - x);
                    }
                    group_bar(grp);
                    if (!first) {
                        product_done(n - 1);
                        fence_after_sync();
#pragma unroll
                        for (int i = 0; i < CN; ++i) l[i] *= sF[c0 + i];
                        float o[CN];
                        o_sum(o);
                        folded = true;
#pragma unroll
                        for (int i = 0; i < CN; i += 8) {
                            uint32_t r[8], zero[8] = {};
#pragma unroll
                            for (int e = 0; e < 8; ++e) r[e] = __float_as_uint(o[i + e] * sF[c0 + i + e]);
                            tmem_st8(tbase + C::T_T + c0 + i + lane_off, r);
#pragma unroll
                            for (int part = 0; part < PARTS; ++part)
                                tmem_st8(tbase + C::T_O + part * QT + c0 + i + lane_off, zero);
                        }
                        tmem_wait_st();
                    }
                    logits();
                    minus_ref();
                }
                // weights, split in three bf16 numbers; this thread's key is a row of P
                uint8_t *sP = sm + C::P_OFF + (n % NP) * C::P;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    uint32_t w[PARTS][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 8 * j + 2 * e;
                        float x = ex2(z[i]), y = ex2(z[i + 1]);
                        l[i] += x;
                        l[i + 1] += y;
#pragma unroll
                        for (int part = 0; part < PARTS; ++part) {
                            w[part][e] = pack_bf16(x, y);
                            x -= __uint_as_float(w[part][e] << 16);
                            y -= __uint_as_float(w[part][e] & 0xffff0000u);
                        }
                    }
#pragma unroll
                    for (int part = 0; part < PARTS; ++part)
                        *reinterpret_cast<uint4 *>(sP + (p_at[part] ^ (16 * j))) =
                            make_uint4(w[part][0], w[part][1], w[part][2], w[part][3]);
                }
                // values behind the prefix's end are whatever the page holds, and are weighed with
                // zero: make them zero too
                if (tail && grp == 0) {
                    wait(&v_full[n % NV], (n / NV) & 1);
                    if (!live) {
                        uint8_t *x = sm + C::V_OFF + (n % NV) * C::TILE + gt * 128;
#pragma unroll
                        for (int i = 0; i < PANELS * 8; ++i)
                            *reinterpret_cast<uint4 *>(x + (i / 8) * KT * 128 + (i % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_async_smem();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[n & 1]);
            }
            // the piece of this unit
            wait_previous();  // qg
            const float qg = gt < nq ? s.qg[(long long)h * q_rows + qt * QT + c0 + gt] : 0.f;
            product_done(n - 1);
            fence_after_sync();
            const long long piece = (long long)blockIdx.x + u;
            {
                const int dim = D == 128 ? gt : 16 * (warp % 4) + lane;
                float v[CN];
                o_sum(v);
                if (D == 128 || lane < 16) {
#pragma unroll
                    for (int i = 0; i < CN; ++i)
                        if (i < nq) s.pre[(piece * QT + c0 + i) * D + dim] = v[i];
                }
#pragma unroll
                for (int i = 0; i < CN; ++i) v[i] = l[i];
                const float sum = warp_reduce<true>(v);
                if (lane < CN) sR[(warp % 4) * QN + c0 + lane] = sum;
            }
            const bool failed = group_any(grp, gave_up);
            if (gt < nq) {
                // the gate since the prefix's end weighs every key of it alike; where it leaves
                // nothing (log f = -inf), neither the sum nor the values count
                const int c = c0 + gt;
                const float M = qg - sM[c];
                const float L = (sR[c] + sR[QN + c]) + (sR[2 * QN + c] + sR[3 * QN + c]);
                s.pre_ml[piece * 2 * QT + c] = M;
                s.pre_ml[piece * 2 * QT + QT + c] = M == -INFINITY && !isnan(L) ? 0.f : L;
            }
            if (gt == 0)
                s.pre_flag[4 * piece + grp] = (failed ? PIECE_GAVE_UP : 0) | (*(volatile int *)s_bad ? PIECE_BAD_PAGE : 0);
            group_bar(grp);
            kb = 0;
            ++u;
            if (++qt == p.q_tiles) {
                qt = 0;
                ++h;
            }
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == W_O) tmem_dealloc(tbase, C::TMEM);
}

template <int D, int GROUPS>
cudaError_t run(const PagedStep &a, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    using C = Cfg<D, GROUPS>;
    const int page = 1 << a.c.page_log2;
    const uint64_t rows = (uint64_t)a.c.n_pages * a.H * page;
    CUtensorMap mQ, mK, mV;
    if (!make_map_2d(&mQ, s.qt, BF16, D, (uint64_t)PARTS * a.H * p.q_tiles * p.q_tile, p.q_tile) ||
        !make_map_2d(&mK, a.c.k, BF16, D, rows, page < KT ? page : KT) ||
        !make_map_2d(&mV, a.c.v, BF16, D, rows, page < KT ? page : KT))
        return cudaErrorInvalidValue;
    auto k = prefix_tc_kernel<D, GROUPS>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_overlapped(k, p.pre_blocks, C::NT, C::SMEM, st, mQ, mK, mV, a, s, p);
}

template <int D>
cudaError_t run(const PagedStep &a, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    switch (p.q_tile / CN) {
    case 1: return run<D, 1>(a, p, s, st);
    case 2: return run<D, 2>(a, p, s, st);
    case 3: return run<D, 3>(a, p, s, st);
    default:
        if constexpr (D == 64) return run<D, 4>(a, p, s, st);
        return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t prefix_attn_tc(const PagedStep &a, int d, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    Stage stage("prefix_attn", st);
    return d == 64 ? run<64>(a, p, s, st) : run<128>(a, p, s, st);
}

}  // namespace path
