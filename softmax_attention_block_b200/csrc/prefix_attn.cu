// Decode attention of a batch to one shared prefix, computed once for all.
//
// The keys of a prefix that many sequences continue cannot be updated in place:
// each sequence has its own factors. But the update is linear, and with
// G_t = H_t ... H_{P+1} (P the prefix's last position)
//   q_t^T (H_t ... H_{P+1}) k_j^{(P)} = (G_t^T q_t)^T k_j^{(P)}
// (from the logit equation, gist.science section 2), so the prefix's keys stay as
// they were when it ended and the query is turned back instead. A sequence
// carries G per head, d x d fp32, and one step costs it a rank-1 update:
//   y = G^T w;  G <- G - beta w y^T;  G_new^T q = G^T q - beta (q.w) y.
#include "paged.cuh"
#include "rowvec.cuh"
#include "runtime.cuh"
#include "tc.cuh"

namespace path {

namespace {

constexpr float LOG2E = 1.4426950408889634f;

// One (batch row, head): G read once and written once, bound by HBM (8 d^2
// bytes). A thread keeps D * D / 512 vectors of four columns in registers, so that a
// block's whole G is on its way at once, and only four partial sums of a column meet.
// 32 x 32 heads of 128: 21 us for 134 MB (6.3 TB/s), 27 us with 256 threads a block.
constexpr int TT = 128;

template <typename T, int D>
__global__ void __launch_bounds__(TT) turn_kernel(PagedStep a, PagedScratch s, int q_rows)
{
    constexpr int CG = D / 4;       // groups of four columns
    constexpr int RG = TT / CG;     // rows of a pass
    constexpr int R = D / RG;       // rows a thread keeps
    __shared__ float sw[D], sq[D];
    __shared__ float4 red[2][4][CG];
    const int u = blockIdx.x, b = u / a.H, h = u % a.H, tid = threadIdx.x;
    const int cg = tid % CG, rg = tid / CG, warp = tid / 32, lane = tid % 32;
    release_next();
    const int slot = b < a.B ? slot_of(a.c, b) : -1;
    const long long row = (long long)h * q_rows + b;
    float4 *qt = reinterpret_cast<float4 *>(s.qt) + row * CG;  // fp32
    uint2 *qb = reinterpret_cast<uint2 *>(s.qt) + row * CG;    // bf16, its parts one after the other
    const long long part = (long long)a.H * q_rows * CG;
    if (slot < 0 || length_of(a.c, slot) < 0) {  // past the batch, idle or invalid: a query of zeros
        if (tid < CG) {
            if (sizeof(T) == 4)
                qt[tid] = make_float4(0.f, 0.f, 0.f, 0.f);
            else
                for (int i = 0; i < PREFIX_PARTS; ++i) qb[i * part + tid] = make_uint2(0u, 0u);
        }
        if (tid == 0) s.qg[row] = 0.f;
        return;
    }
    float4 *G = reinterpret_cast<float4 *>(a.state) + ((long long)slot * a.H + h) * (D * CG);
    float4 x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = G[(i * RG + rg) * CG + cg];
    for (int i = tid; i < D; i += TT) {
        sw[i] = to_f(static_cast<const T *>(a.w)[(long long)u * D + i]);
        sq[i] = to_f(static_cast<const T *>(a.q)[(long long)u * D + i]);
    }
    const float beta = a.beta[u];
    __syncthreads();
    float qw = 0.f;
#pragma unroll
    for (int i = lane; i < D; i += 32) qw = fmaf(sq[i], sw[i], qw);
    qw = group_sum<32>(qw);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f), z = y;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float w = sw[i * RG + rg], q = sq[i * RG + rg];
        y.x = fmaf(w, x[i].x, y.x);
        y.y = fmaf(w, x[i].y, y.y);
        y.z = fmaf(w, x[i].z, y.z);
        y.w = fmaf(w, x[i].w, y.w);
        z.x = fmaf(q, x[i].x, z.x);
        z.y = fmaf(q, x[i].y, z.y);
        z.z = fmaf(q, x[i].z, z.z);
        z.w = fmaf(q, x[i].w, z.w);
    }
    if (CG == 16) {  // two rows of a pass in one warp
        float *f[2] = {&y.x, &z.x};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[i][e] += __shfl_xor_sync(0xffffffffu, f[i][e], 16);
    }
    red[0][warp][cg] = y;
    red[1][warp][cg] = z;
    __syncthreads();
    y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 t = red[0][i][cg];
        y.x += t.x;
        y.y += t.y;
        y.z += t.z;
        y.w += t.w;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float f = -beta * sw[i * RG + rg];
        x[i].x = fmaf(f, y.x, x[i].x);
        x[i].y = fmaf(f, y.y, x[i].y);
        x[i].z = fmaf(f, y.z, x[i].z);
        x[i].w = fmaf(f, y.w, x[i].w);
        G[(i * RG + rg) * CG + cg] = x[i];
    }
    if (rg == 0) {
        z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = red[1][i][cg];
            z.x += t.x;
            z.y += t.y;
            z.z += t.z;
            z.w += t.w;
        }
        const float f = -beta * qw;
        const float4 r = make_float4(fmaf(f, y.x, z.x), fmaf(f, y.y, z.y), fmaf(f, y.z, z.z), fmaf(f, y.w, z.w));
        if (sizeof(T) == 4) {
            qt[cg] = r;
        } else {  // r as a sum of bf16 numbers
            float v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int j = 0; j < PREFIX_PARTS; ++j) {
                __nv_bfloat162 b[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    b[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                    const float2 t = __bfloat1622float2(b[i]);
                    v[2 * i] -= t.x;
                    v[2 * i + 1] -= t.y;
                }
                qb[j * part + cg] = *reinterpret_cast<uint2 *>(b);
            }
        }
    }
    if (tid == 0) {
        float g = 0.f;
        if (a.g_state) {
            float *gs = a.g_state + (long long)slot * a.H + h;
            g = *gs + a.log_f[u];
            *gs = g;
        }
        s.qg[row] = g * LOG2E;
    }
}

// fp32 arithmetic on CUDA cores: QT queries (16 or 32) by 64 keys a tile, one pass
// over the keys with a running maximum and sum. A warp holds four queries, a lane
// two keys of the tile and then D / 32 dims of the output; queries and weights are
// read as broadcasts. Bound by shared-memory reads (12 for 32 products of logits, 5
// for 16 of outputs), or for few tiles by their latency. Where a key's row
// lies is looked up a tile ahead, so that the asynchronous copies of a tile wait
// for nothing; a tile's keys come in under the former tile's values, its values
// under its own keys. A step of 9 rows behind 2047 tokens (6 heads of 128), where a
// block has one tile: 26 us with 16 queries a tile, 33 with 32.
constexpr int KT = 64;

template <int D, int QT>
struct SimtCfg {
    static constexpr int NT = 8 * QT, LD = D + 4;
    static constexpr int Q = 0, K = Q + QT * LD, V = K + KT * LD, P = V + KT * D, G = P + QT * KT;
    static constexpr int SMEM = (G + 2 * KT) * 4;
};

// 16 bytes to shared memory, asynchronously; zeros where there is no source.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :
                 : "r"(tc::smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Largest value of a warp's lanes (NaN does not count).
__device__ __forceinline__ float warp_max(float x)
{
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

template <int D, int QT>
__global__ void __launch_bounds__(SimtCfg<D, QT>::NT) prefix_simt_kernel(PagedStep a, PagedScratch s, PagedPlan p)
{
    using C = SimtCfg<D, QT>;
    constexpr int LD = C::LD, NT = C::NT, DL = D / 32;  // dims a lane accumulates
    extern __shared__ float sm[];
    __shared__ long long s_row[2][KT];  // row of the pool that a key of the tile is, or -1
    float *sQ = sm + C::Q, *sK = sm + C::K, *sV = sm + C::V, *sP = sm + C::P, *sG = sm + C::G;
    const int tid = threadIdx.x, tx = tid % 32, ty = tid / 32;
    float *sW = sP + ty * 4 * KT;  // this warp's weights: four queries of a key side by side
    release_next();
    const int q_rows = p.q_tiles * QT;
    const float scale2 = a.scale * LOG2E;
    const long long total = (long long)p.pre_units * p.key_tiles;
    const long long t0 = total * blockIdx.x / gridDim.x, t1 = total * (blockIdx.x + 1) / gridDim.x;
    // where the keys of a tile lie, and their gate biases (-inf past the prefix)
    auto look_up = [&](int h, int kt) {
        bool bad = false;
        if (tid < KT) {
            const int key = kt * KT + tid;
            long long row = -1;
            float g = -INFINITY;
            if (key < a.prefix_len) {
                const int pg = a.prefix_table[key >> a.c.page_log2];
                bad = pg < 0 || pg >= a.c.n_pages;
                g = 0.f;
                if (!bad) {
                    row = (((long long)pg * a.H + h) << a.c.page_log2) + (key & ((1 << a.c.page_log2) - 1));
                    if (a.c.g) g = a.c.g[row] * LOG2E;
                }
            }
            s_row[kt & 1][tid] = row;
            sG[(kt & 1) * KT + tid] = g;
        }
        return bad;
    };
    auto load = [&](const void *pool, int kt, float *dst, int ld) {
        constexpr int LPR = D / 4;
#pragma unroll
        for (int i = tid; i < KT * LPR; i += NT) {
            const int r = i / LPR, x = i % LPR;
            const long long row = s_row[kt & 1][r];
            copy16(dst + r * ld + 4 * x, static_cast<const float *>(pool) + (row < 0 ? 0 : row) * D + 4 * x, row >= 0);
        }
        copies_commit();
    };
    for (long long t = t0; t < t1;) {
        const int u = (int)(t / p.key_tiles), kb = (int)(t % p.key_tiles);
        const int ke = (int)min((long long)p.key_tiles, kb + (t1 - t));
        const int qtile = u % p.q_tiles, h = u / p.q_tiles;
        bool bad = look_up(h, kb);
        __syncthreads();
        load(a.c.k, kb, sK, LD);
        load(a.c.v, kb, sV, D);
        if (t == t0) wait_previous();  // the queries; keys and values are nobody's output
        for (int i = tid; i < QT * D; i += NT) {
            const int r = i / D, e = i % D, b = qtile * QT + r;
            sQ[r * LD + e] = b < a.B ? s.qt[((long long)h * q_rows + b) * D + e] : 0.f;
        }
        float m[4], l[4], acc[4][DL];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < DL; ++e) acc[i][e] = 0.f;
        }
        for (int kt = kb; kt < ke; ++kt) {
            const int key0 = kt * KT;
            const float *g = sG + (kt & 1) * KT;
            copies_wait<1>();  // the keys
            __syncthreads();
            if (kt + 1 < ke) bad |= look_up(h, kt + 1);
            float z[4][2] = {};
#pragma unroll 2
            for (int e = 0; e < D; e += 4) {
                const float4 k0 = *reinterpret_cast<const float4 *>(sK + tx * LD + e);
                const float4 k1 = *reinterpret_cast<const float4 *>(sK + (tx + 32) * LD + e);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 q = *reinterpret_cast<const float4 *>(sQ + (4 * ty + i) * LD + e);
                    z[i][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, z[i][0]))));
                    z[i][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, z[i][1]))));
                }
            }
            float w[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    z[i][j] = key0 + tx + 32 * j < a.prefix_len ? fmaf(z[i][j], scale2, g[tx + 32 * j]) : -INFINITY;
                const float mx = fmaxf(m[i], warp_max(fmaxf(z[i][0], z[i][1])));
                const float base = mx == -INFINITY ? 0.f : mx;  // a row without a weight so far
                const float corr = tc::ex2(m[i] - base);
#pragma unroll
                for (int j = 0; j < 2; ++j) w[j][i] = tc::ex2(z[i][j] - base);
                l[i] = fmaf(l[i], corr, w[0][i] + w[1][i]);  // of this lane's keys
                m[i] = mx;
#pragma unroll
                for (int e = 0; e < DL; ++e) acc[i][e] *= corr;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
                *reinterpret_cast<float4 *>(sW + (tx + 32 * j) * 4) = make_float4(w[j][0], w[j][1], w[j][2], w[j][3]);
            copies_wait<0>();  // the values
            __syncthreads();
            if (kt + 1 < ke) load(a.c.k, kt + 1, sK, LD);
#pragma unroll 4
            for (int j = 0; j < KT; ++j) {
                const float4 pw = *reinterpret_cast<const float4 *>(sW + j * 4);
                const float *v = sV + j * D + DL * tx;
                float x[DL];
                if constexpr (DL == 4) {
                    const float4 y = *reinterpret_cast<const float4 *>(v);
                    x[0] = y.x;
                    x[1] = y.y;
                    x[2] = y.z;
                    x[3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2 *>(v);
                    x[0] = y.x;
                    x[1] = y.y;
                }
#pragma unroll
                for (int e = 0; e < DL; ++e) {
                    acc[0][e] = fmaf(pw.x, x[e], acc[0][e]);
                    acc[1][e] = fmaf(pw.y, x[e], acc[1][e]);
                    acc[2][e] = fmaf(pw.z, x[e], acc[2][e]);
                    acc[3][e] = fmaf(pw.w, x[e], acc[3][e]);
                }
            }
            __syncthreads();
            if (kt + 1 < ke) load(a.c.v, kt + 1, sV, D);
        }
        const long long piece = (long long)blockIdx.x + u;
        const bool any_bad = __syncthreads_or(bad);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * ty + i, b = qtile * QT + r;
            const float sum = group_sum<32>(l[i]);
            if (b < a.B) {
                float *o = s.pre + (piece * QT + r) * D + DL * tx;
#pragma unroll
                for (int e = 0; e < DL; e += 2) *reinterpret_cast<float2 *>(o + e) = make_float2(acc[i][e], acc[i][e + 1]);
                if (tx == 0) {
                    // the gate since the prefix's end weighs every key of it alike; where it
                    // leaves nothing (log f = -inf), neither the sum nor the values count
                    const float M = m[i] + s.qg[(long long)h * q_rows + b];
                    s.pre_ml[piece * 2 * QT + r] = M;
                    s.pre_ml[piece * 2 * QT + QT + r] = M == -INFINITY && !isnan(sum) ? 0.f : sum;
                }
            }
        }
        if (tid < 4) s.pre_flag[4 * piece + tid] = any_bad ? PIECE_BAD_PAGE : 0;
        t += ke - kb;
    }
}

template <int D, int QT>
cudaError_t run_simt(const PagedStep &a, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    using C = SimtCfg<D, QT>;
    auto k = prefix_simt_kernel<D, QT>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    return launch_overlapped(k, p.pre_blocks, C::NT, C::SMEM, st, a, s, p);
}

template <typename T, int D>
cudaError_t run_turn(const PagedStep &a, const PagedPlan &p, const PagedScratch &s, cudaStream_t st)
{
    const int q_rows = p.q_tiles * p.q_tile;
    turn_kernel<T, D><<<q_rows * a.H, TT, 0, st>>>(a, s, q_rows);
    count_launches();
    return cudaGetLastError();
}

}  // namespace

cudaError_t prefix_turn(const PagedStep &a, int dt, int d, const PagedPlan &p, const PagedScratch &s,
                        cudaStream_t st)
{
    Stage stage("prefix_turn", st);
    if (d == 64) return dt == F32 ? run_turn<float, 64>(a, p, s, st) : run_turn<bf16, 64>(a, p, s, st);
    if (d == 128) return dt == F32 ? run_turn<float, 128>(a, p, s, st) : run_turn<bf16, 128>(a, p, s, st);
    return cudaErrorInvalidValue;
}

cudaError_t prefix_attn_simt(const PagedStep &a, int d, const PagedPlan &p,
                             const PagedScratch &s, cudaStream_t st)
{
    Stage stage("prefix_attn", st);
    if (p.q_tile == 16) return d == 64 ? run_simt<64, 16>(a, p, s, st) : run_simt<128, 16>(a, p, s, st);
    return d == 64 ? run_simt<64, 32>(a, p, s, st) : run_simt<128, 32>(a, p, s, st);
}

}  // namespace path
