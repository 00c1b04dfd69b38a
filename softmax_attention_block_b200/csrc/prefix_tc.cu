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
// bf16 operands alone would cost as much accuracy as the rounding of the output,
// so qt and P are each split in two bf16 numbers (hi + lo, off by 2^-17) and
// multiplied twice; the tensor cores have the time (see the tile costs below).
//
// The running maximum of a query is a reference that moves only when a logit
// passes it by more than 2^8 (or at a unit's first tile): then all four warps
// agree on the new one and O^T is scaled in tensor memory. Otherwise a tile
// needs no maximum across threads at all: weights stay below 2^8 and sums and
// products are fp32. A thread keeps the sum of its own keys' weights per query;
// they are added up across threads at a unit's end.
//
// Warps 0-3 softmax, 4 loads (a box of min(page, 128) rows a page, TMA), 5 MMA.
// Waits are bounded; one that gives up makes its pieces NaN and is reported.
#include "paged.cuh"
#include "runtime.cuh"
#include "tc.cuh"

namespace path {

namespace {

using namespace tc;

constexpr int NT = 192, NSOFT = 128, W_LOAD = 4, W_MMA = 5;
constexpr int KT = 128;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LOW = -1e30f;  // reference of a query that has no weight yet
constexpr float SLACK = 8.f;

template <int D, int QN>
struct Cfg {
    static constexpr int PANELS = D / 64;
    static constexpr int TILE = KT * D * 2;             // one operand tile
    static constexpr int NK = D == 64 ? 4 : QN == 32 ? 3 : 2, NV = D == 64 ? 4 : 2, NG = NV + 1;
    static constexpr int Q = 2 * QN * D * 2;            // hi and lo
    static constexpr int PP = KT * 128;                 // one panel of P: 64 columns
    static constexpr int P = QN == 32 ? PP : 2 * PP;    // hi | lo side by side, or a panel each
    static constexpr int K_OFF = 0, V_OFF = K_OFF + NK * TILE, Q_OFF = V_OFF + NV * TILE, P_OFF = Q_OFF + Q;
    static constexpr int G_OFF = P_OFF + P, M_OFF = G_OFF + NG * KT * 4, F_OFF = M_OFF + QN * 4;
    static constexpr int RED_OFF = F_OFF + QN * 4, BAR_OFF = RED_OFF + 4 * QN * 4;
    static constexpr int NBAR = 2 * NK + 2 * NV + NG + 7;
    static constexpr int SMEM = BAR_OFF + NBAR * 8 + 16 + 1024;
    static constexpr int T_S = 0, T_O = 2 * QN, TMEM = QN == 32 ? 128 : 256;
    static_assert(SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ void soft_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ bool soft_any(bool x)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// Sum over the warp's lanes of each of 32 values; lane i gets the i-th.
__device__ __forceinline__ float warp_sums(float (&v)[32])
{
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int o = 16, n = 16; o > 0; o >>= 1, n >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    return v[0];
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int D, int QN>
__global__ void __launch_bounds__(NT, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                     const __grid_constant__ CUtensorMap mV, PagedStep a, PagedScratch s, PagedPlan p)
{
    using C = Cfg<D, QN>;
    constexpr int NK = C::NK, NV = C::NV, NG = C::NG, PANELS = C::PANELS;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + (1024 - (smem_u32(smraw) & 1023)) % 1024;
    uint64_t *k_full = reinterpret_cast<uint64_t *>(sm + C::BAR_OFF), *k_empty = k_full + NK;
    uint64_t *v_full = k_empty + NK, *v_empty = v_full + NV, *g_full = v_empty + NV;
    uint64_t *q_full = g_full + NG, *q_empty = q_full + 1, *s_full = q_full + 2, *p_full = q_full + 4;
    uint64_t *o_done = q_full + 5, *mma_done = q_full + 6;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(q_full + 7);
    int *s_bad = reinterpret_cast<int *>(tmem_slot + 1);
    float *sG = reinterpret_cast<float *>(sm + C::G_OFF), *sM = reinterpret_cast<float *>(sm + C::M_OFF);
    float *sF = reinterpret_cast<float *>(sm + C::F_OFF), *sR = reinterpret_cast<float *>(sm + C::RED_OFF);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const bool gate = a.c.g != nullptr;

    if (tid == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < NG; ++i) mbar_init(&g_full[i], 1);
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(&s_full[0], 1);
        mbar_init(&s_full[1], 1);
        mbar_init(p_full, NSOFT);
        mbar_init(o_done, 1);
        mbar_init(mma_done, 1);
        mbar_fence_init();
        *s_bad = 0;
    }
    if (warp == W_MMA) tmem_alloc(tmem_slot, C::TMEM);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tbase = *tmem_slot;

    // this block's share of all (unit, key tile) pairs; a segment is its part of one unit
    const long long total = (long long)p.pre_units * p.key_tiles;
    const long long t0 = total * blockIdx.x / gridDim.x, t1 = total * (blockIdx.x + 1) / gridDim.x;
    const int count = (int)(t1 - t0);
    const int q_rows = p.q_tiles * QN;

    if (warp == W_LOAD) {
        const int log2p = a.c.page_log2, page = 1 << log2p, box = page < KT ? page : KT, boxes = KT / box;
        const int npre = (a.prefix_len + page - 1) >> log2p;
        int tab = -1, tab_at = 0, tab_end = 0, issued_k = 0, issued_v = 0, seg = 0;
        bool ok = true;
        for (int n = 0; n < count && ok; ++n) {
            const long long t = t0 + n;
            const int u = (int)(t / p.key_tiles), kt = (int)(t % p.key_tiles);
            const int h = u / p.q_tiles, key0 = kt * KT;
            if (n == 0 || kt == 0) {
                if (seg > 0 && !mbar_wait(q_empty, (seg - 1) & 1, WAIT_LIMIT_NS)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    mbar_expect_tx(q_full, C::Q);
                    const int row = h * q_rows + (u % p.q_tiles) * QN;
                    for (int x = 0; x < PANELS; ++x) {
                        tma_load_2d(sm + C::Q_OFF + x * QN * 128, &mQ, 64 * x, row, q_full);
                        tma_load_2d(sm + C::Q_OFF + (PANELS + x) * QN * 128, &mQ, 64 * x, a.H * q_rows + row, q_full);
                    }
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
            const int ks = n % NK, vs = n % NV, gs = n % NG;
            if (n >= NK && !mbar_wait(&k_empty[ks], (n / NK - 1) & 1, WAIT_LIMIT_NS)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (lane == 0) {
                if (cnt) mbar_expect_tx(&k_full[ks], cnt * box * D * 2);
                else mbar_arrive(&k_full[ks]);
                if (gate) {
                    // the slot is free: tile n - NG = n - 1 - NV was done before V of tile n - 1 was loaded
                    if (cnt) mbar_expect_tx(&g_full[gs], cnt * box * 4);
                    else mbar_arrive(&g_full[gs]);
                }
            }
            __syncwarp();
            if (good) {
                for (int x = 0; x < PANELS; ++x)
                    tma_load_2d(sm + C::K_OFF + ks * C::TILE + x * KT * 128 + lane * box * 128, &mK, 64 * x, row, &k_full[ks]);
                if (gate) bulk_load(sG + gs * KT + lane * box, a.c.g + row, box * 4, &g_full[gs]);
            }
            issued_k = n + 1;
            if (n >= NV && !mbar_wait(&v_empty[vs], (n / NV - 1) & 1, WAIT_LIMIT_NS)) ok = false;
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
        if (!ok) {  // leave no copy on its way into this block's memory
            for (int n = max(0, issued_k - NK); n < issued_k; ++n) {
                mbar_wait(&k_full[n % NK], (n / NK) & 1, WAIT_LIMIT_NS);
                if (gate && n >= issued_k - NG) mbar_wait(&g_full[n % NG], (n / NG) & 1, WAIT_LIMIT_NS);
            }
            for (int n = max(0, issued_v - NV); n < issued_v; ++n)
                mbar_wait(&v_full[n % NV], (n / NV) & 1, WAIT_LIMIT_NS);
            if (seg > 0) mbar_wait(q_full, (seg - 1) & 1, WAIT_LIMIT_NS);
        }
    } else if (warp == W_MMA) {
        if (lane == 0) {
            // Tile costs at D = 128 in tensor-core cycles: S^T 8 steps x 2 (hi, lo) x 32, O^T
            // the same, 1024 in all, where the loads of a tile take 2800.
            constexpr uint32_t idS = idesc_f16(128, QN, AB_BF16, 0, 0), idO = idesc_f16(D, 64, AB_BF16, 1, 1);
            const uint32_t q_addr = smem_u32(sm + C::Q_OFF), p_addr = smem_u32(sm + C::P_OFF);
            int seg = 0;
            bool ok = true;
            auto issue_s = [&](int n) -> bool {
                const long long t = t0 + n;
                const int ks = n % NK;
                if (n == 0 || t % p.key_tiles == 0) {
                    if (!mbar_wait(q_full, seg & 1, WAIT_LIMIT_NS)) return false;
                    ++seg;
                }
                if (!mbar_wait(&k_full[ks], (n / NK) & 1, WAIT_LIMIT_NS)) return false;
                fence_after_sync();
                const uint32_t k_addr = smem_u32(sm + C::K_OFF + ks * C::TILE);
#pragma unroll
                for (int part = 0; part < 2; ++part)
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        mma_ss(tbase + C::T_S + (n & 1) * QN,
                               desc_sw128(k_addr + (kk / 4) * KT * 128 + (kk % 4) * 32, 16, 1024),
                               desc_sw128(q_addr + (part * PANELS + kk / 4) * QN * 128 + (kk % 4) * 32, 16, 1024),
                               idS, part + kk > 0);
                commit(&s_full[n & 1]);
                commit(&k_empty[ks]);
                if (n + 1 == count || (t + 1) % p.key_tiles == 0) commit(q_empty);
                return true;
            };
            ok = count > 0 && issue_s(0);
            for (int n = 0; ok && n < count; ++n) {
                // the buffer of S(n + 1) was read before P(n - 1) was complete
                if (n + 1 < count && !issue_s(n + 1)) break;
                const int vs = n % NV;
                if (!mbar_wait(&v_full[vs], (n / NV) & 1, WAIT_LIMIT_NS) || !mbar_wait(p_full, n & 1, WAIT_LIMIT_NS)) break;
                fence_after_sync();
                const uint32_t v_addr = smem_u32(sm + C::V_OFF + vs * C::TILE);
                const bool fresh = n == 0 || (t0 + n) % p.key_tiles == 0;
#pragma unroll
                for (int part = 0; part < C::P / C::PP; ++part)
#pragma unroll
                    for (int kk = 0; kk < KT / 16; ++kk)
                        mma_ss(tbase + C::T_O, desc_sw128(v_addr + kk * 2048, KT * 128, 1024),
                               desc_sw128(p_addr + part * C::PP + kk * 2048, C::PP, 1024), idO,
                               !fresh || part + kk > 0);
                commit(&v_empty[vs]);
                commit(o_done);
            }
            // the tensor memory is freed after this warp leaves: no MMA may still be running then
            commit(mma_done);
            mbar_wait(mma_done, 0, 8 * WAIT_LIMIT_NS);
        }
    } else {
        // thread = key of the tile (a lane of S^T), then a row of O^T: dim tid, or at D = 64
        // dim 16 warp + lane in the lanes below 16
        const uint32_t lane_off = (uint32_t)(32 * warp) << 16;
        const float scale2 = a.scale * LOG2E;
        uint8_t *sP = sm + C::P_OFF;
        bool ok = true;
        int n = 0;
        while (n < count) {
            const long long t = t0 + n;
            const int u = (int)(t / p.key_tiles), kb = (int)(t % p.key_tiles);
            const int ke = (int)min((long long)p.key_tiles, kb + (t1 - t));
            const int qt = u % p.q_tiles, h = u / p.q_tiles;
            const int nq = min(QN, a.B - qt * QN);  // queries of this unit
            float l[QN];
#pragma unroll
            for (int i = 0; i < QN; ++i) l[i] = 0.f;
            for (int kt = kb; kt < ke; ++kt, ++n) {
                const bool first = kt == kb;
                const bool live = kt * KT + tid < a.prefix_len;
                if (ok && !mbar_wait(&s_full[n & 1], (n >> 1) & 1, WAIT_LIMIT_NS)) ok = false;
                float g = 0.f;
                if (gate) {
                    if (ok && !mbar_wait(&g_full[n % NG], (n / NG) & 1, WAIT_LIMIT_NS)) ok = false;
                    if (ok) g = sG[(n % NG) * KT + tid] * LOG2E;
                }
                ok = __all_sync(0xffffffffu, ok);
                fence_after_sync();
                float z[QN];
                auto logits = [&](int c) {  // columns c .. c + 31
                    float v[32];
                    tmem_ld32(tbase + C::T_S + (n & 1) * QN + c + lane_off, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[c + i] = live ? fmaf(v[i], scale2, g) : -INFINITY;
                };
                auto minus_ref = [&](int c) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 m = *reinterpret_cast<const float4 *>(sM + c + i);
                        z[c + i] -= m.x;
                        z[c + i + 1] -= m.y;
                        z[c + i + 2] -= m.z;
                        z[c + i + 3] -= m.w;
                    }
                };
                float top = -INFINITY;
                if (ok) {
#pragma unroll
                    for (int c = 0; c < QN; c += 32) {
                        if (c >= nq) break;
                        logits(c);
                        if (!first) {
                            minus_ref(c);
#pragma unroll
                            for (int i = 0; i < 32; ++i) top = fmaxf(top, z[c + i]);
                        }
                    }
                }
                // P's buffer and O^T are free once the former tile's product is done
                if (ok && n > 0 && !mbar_wait(o_done, (n - 1) & 1, WAIT_LIMIT_NS)) ok = false;
                ok = __all_sync(0xffffffffu, ok);
                if (soft_any(first || top > SLACK)) {
                    if (ok) {
                        fence_after_sync();
#pragma unroll
                        for (int c = 0; c < QN; c += 32) {
                            if (c >= nq) break;
                            logits(c);
                            float mine = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float x = warp_max(z[c + i]);
                                if (lane == i) mine = x;
                            }
                            sR[warp * QN + c + lane] = mine;
                        }
                    }
                    soft_bar();
                    if (tid < QN) {
                        const float old = first ? -INFINITY : sM[tid];
                        float x = fmaxf(fmaxf(sR[tid], sR[QN + tid]), fmaxf(sR[2 * QN + tid], sR[3 * QN + tid]));
                        x = fmaxf(fmaxf(old, x), LOW);
                        sM[tid] = x;
                        sF[tid] = ex2(old - x);
                    }
                    soft_bar();
                    if (ok) {
                        if (!first) {
#pragma unroll
                            for (int i = 0; i < QN; ++i) l[i] *= sF[i];
#pragma unroll 1
                            for (int c = 0; c < 64; c += 32) {
                                float v[32];
                                tmem_ld32(tbase + C::T_O + c + lane_off, v);
#pragma unroll
                                for (int i = 0; i < 32; i += 8) {
                                    uint32_t r[8];
#pragma unroll
                                    for (int e = 0; e < 8; ++e)
                                        r[e] = __float_as_uint(v[i + e] * sF[(QN == 32 ? 0 : c) + i + e]);
                                    tmem_st8(tbase + C::T_O + c + i + lane_off, r);
                                }
                            }
                            tmem_wait_st();
                        }
#pragma unroll
                        for (int c = 0; c < QN; c += 32) {
                            if (c >= nq) break;
                            minus_ref(c);
                        }
                    }
                }
                if (ok) {
                    // weights, split in two bf16 numbers; this thread's key is a row of P
#pragma unroll
                    for (int c = 0; c < QN; c += 32) {
                        if (c >= nq) break;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t hi[4], lo[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x = ex2(z[c + i + 2 * e]), y = ex2(z[c + i + 2 * e + 1]);
                                l[c + i + 2 * e] += x;
                                l[c + i + 2 * e + 1] += y;
                                hi[e] = pack_bf16(x, y);
                                lo[e] = pack_bf16(x - __uint_as_float(hi[e] << 16),
                                                  y - __uint_as_float(hi[e] & 0xffff0000u));
                            }
                            *reinterpret_cast<uint4 *>(sP + sw128_offset(tid, c + i)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                            uint8_t *low = QN == 32 ? sP + sw128_offset(tid, 32 + i) : sP + C::PP + sw128_offset(tid, c + i);
                            *reinterpret_cast<uint4 *>(low) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        }
                    }
                    // values behind the prefix's end are whatever the page holds, and are weighed
                    // with zero: make them zero too
                    if ((kt + 1) * KT > a.prefix_len) {
                        if (!mbar_wait(&v_full[n % NV], (n / NV) & 1, WAIT_LIMIT_NS)) ok = false;
                        if (ok && !live) {
                            uint8_t *v = sm + C::V_OFF + (n % NV) * C::TILE + tid * 128;
#pragma unroll
                            for (int x = 0; x < PANELS; ++x)
#pragma unroll
                                for (int i = 0; i < 128; i += 16)
                                    *reinterpret_cast<uint4 *>(v + x * KT * 128 + i) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_async_smem();
                    fence_before_sync();
                    if (ok) mbar_arrive(p_full);
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            // the piece of this unit
            if (ok && !mbar_wait(o_done, (n - 1) & 1, WAIT_LIMIT_NS)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            fence_after_sync();
            const long long piece = (long long)blockIdx.x + u;
            const int dim = D == 128 ? tid : 16 * warp + lane;
#pragma unroll
            for (int c = 0; c < QN; c += 32) {
                if (c >= nq) break;
                float v[32], v2[32];
                if (ok) {
                    tmem_ld32(tbase + C::T_O + c + lane_off, v);
                    if (QN == 32) tmem_ld32(tbase + C::T_O + 32 + lane_off, v2);
                    if (D == 128 || lane < 16) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c + i < nq) s.pre[(piece * QN + c + i) * D + dim] = QN == 32 ? v[i] + v2[i] : v[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = l[c + i];
                sR[warp * QN + c + lane] = warp_sums(v);
            }
            const bool failed = soft_any(!ok);
            if (tid < nq) {
                // the gate since the prefix's end weighs every key of it alike; where it leaves
                // nothing (log f = -inf), neither the sum nor the values count
                const float M = sM[tid] + s.qg[(long long)h * q_rows + qt * QN + tid];
                const float L = (sR[tid] + sR[QN + tid]) + (sR[2 * QN + tid] + sR[3 * QN + tid]);
                s.pre_ml[piece * 2 * QN + tid] = M;
                s.pre_ml[piece * 2 * QN + QN + tid] = M == -INFINITY && !isnan(L) ? 0.f : L;
            }
            if (tid == 0) s.pre_flag[piece] = (failed ? PIECE_GAVE_UP : 0) | (*(volatile int *)s_bad ? PIECE_BAD_PAGE : 0);
            soft_bar();
        }
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == W_MMA) tmem_dealloc(tbase, C::TMEM);
}

template <int D, int QN>
cudaError_t run(const PagedStep &a, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    using C = Cfg<D, QN>;
    const int page = 1 << a.c.page_log2;
    const uint64_t rows = (uint64_t)a.c.n_pages * a.H * page;
    CUtensorMap mQ, mK, mV;
    if (!make_map_2d(&mQ, s.qt, BF16, D, 2ull * a.H * p.q_tiles * QN, QN) ||
        !make_map_2d(&mK, a.c.k, BF16, D, rows, page < KT ? page : KT) ||
        !make_map_2d(&mV, a.c.v, BF16, D, rows, page < KT ? page : KT))
        return cudaErrorInvalidValue;
    auto k = prefix_tc_kernel<D, QN>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    k<<<p.pre_blocks, NT, C::SMEM, st>>>(mQ, mK, mV, a, s, p);
    count_launches();
    return cudaGetLastError();
}

}  // namespace

cudaError_t prefix_attn_tc(const PagedStep &a, int d, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    Stage stage("prefix_attn", st);
    if (d == 64) return p.q_tile == 32 ? run<64, 32>(a, p, s, st) : run<64, 64>(a, p, s, st);
    return p.q_tile == 32 ? run<128, 32>(a, p, s, st) : run<128, 64>(a, p, s, st);
}

}  // namespace path
