// sf_grouped.cu -- products grouped by expert on the tcgen05 tensor cores: forward, input gradient and
// weight gradient. The mathematics and the layouts are in include/sf.h.
//
// Forward and input gradient. Weights are the M operand (128 rows of the accumulator a CTA) and tokens the N
// operand, whose width is set per tile in steps of 16 or 32. So an expert's ragged end costs no more than its
// own tokens, a neighbour's rows inside a loaded box only feed accumulator columns that are never stored, and a
// handful of tokens still streams whole weight rows.
//   forward: M = rows r of W[e], K = columns c: W is K-major as it lies.
//   dx:      M = columns c,      K = rows r:    W is M-major as it lies; tcgen05 reads both.
// Weight gradient: M = r, N = c, K = the expert's tokens, both operands MN-major as they lie. The last 16-token
// step of an expert would also multiply the next expert's rows: those rows are cleared in shared memory, in both
// operands (a product of two zeros stays out of the sum whatever the neighbour holds).
#include <string.h>

#include <atomic>

#include "sf_common.cuh"
#include "sf_host.h"

namespace sf {
namespace {

constexpr int kMaxE = SF_GROUPED_MAX_EXPERTS;
constexpr int GK = 64;                        // elements of K per stage: 128 bytes, one swizzle row
constexpr int G_UMMA_K = 16;
constexpr int G_BOX_BYTES = 64 * GK * 2;      // a 64 x 64 box

// ---- tiles of CTA pairs: 256 accumulator rows x up to 256 columns, both CTAs' MMAs as one (cta_group::2) ----
constexpr int PM = 256;                       // accumulator rows of a pair, 128 in each CTA's TMEM
constexpr int PN = 256;                       // accumulator columns at most
constexpr int P_STAGES = 6;
constexpr int P_HALF_BYTES = 128 * GK * 2;    // one operand of a stage in one CTA: 16 KB
constexpr int P_STAGE_BYTES = 2 * P_HALF_BYTES;
constexpr int P_NBUF = 2;                     // accumulators: the MMAs fill one while the epilogue drains the other
constexpr int P_TMEM_COLS = P_NBUF * PN;
constexpr int P_EPI_WARPS = 8;                // two per TMEM lane quarter
constexpr int P_THREADS = 64 + 32 * P_EPI_WARPS;
constexpr size_t P_SMEM_BYTES = (size_t)P_STAGES * P_STAGE_BYTES + 1024;
constexpr int P_BAND = 8;                     // token tiles that share a pass over an expert's weights

// ---- single CTAs: 128 accumulator rows x up to 128 columns, K split over a cluster ----
constexpr int SM_ROWS = 128;
constexpr int S_EPI_WARPS = 4;
constexpr int S_THREADS = 64 + 32 * S_EPI_WARPS;
constexpr int S_W_BYTES = SM_ROWS * GK * 2;   // 16 KB
constexpr int S_MAX_STAGES = 12;

constexpr int W_CHUNK_STAGES = 1024 / GK;     // weight gradient: tokens summed by the tensor core before fp32 adds

struct GArgs {
    CUtensorMap tm_w;          // forward, dx: W as {C, R, E}; dw: A as {C, T}
    CUtensorMap tm_x;          // tokens: forward A, dx Y as {K, T}; dw: Y as {R, T}
    const int32_t *offsets;
    void *out;
    int64_t ld_out, stride_out;
    int32_t E, T, M, K, type;  // M: accumulator rows in all (forward R, dx C, dw R); K: forward C, dx R, dw C (its N)
    int32_t nb, stages, ksplit;      // single CTAs: token box, stages, CTAs of a cluster
    int32_t out_f32, accumulate;     // dw
};

__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// K-major: 128-byte rows, 8-row groups 1024 bytes apart (the leading offset is unused).
__device__ __forceinline__ uint64_t kmajor(uint32_t addr) { return sw128_desc(addr, 16, 1024); }
// MN-major: 64-element chunks a box apart, groups of 8 K rows 1024 bytes apart.
__device__ __forceinline__ uint64_t mnmajor(uint32_t addr) { return sw128_desc(addr, G_BOX_BYTES, 1024); }

// kind::f16: fp32 accumulator, A and B both bf16 or both fp16, their majors, N, M.
__device__ __forceinline__ uint32_t idesc(int type, bool a_mn, bool b_mn, int n, int m)
{
    const uint32_t t = type == SF_TYPE_BF16 ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// Token tiles of an expert: as few as `most` tokens each allow, evenly filled, in steps of `step` tokens.
__device__ __forceinline__ int tile_tokens(int cnt, int most, int step)
{
    const int n = (cnt + most - 1) / most;
    const int each = (cnt + n - 1) / n;
    return (each + step - 1) / step * step;
}

struct Plan {
    int off[kMaxE + 1];        // offsets
    int pre[kMaxE + 1];        // units of the experts before
    int scratch[33];
};

// Offsets and unit counts into shared memory. False (for every thread) when the offsets are not valid.
// per_expert(tokens) -> units. Contains __syncthreads.
template <typename F>
__device__ __forceinline__ bool load_plan(Plan &pl, const int32_t *offsets, int E, int T, F per_expert)
{
    int run = 0, bad = 0;
    for (int base = 0; base < E; base += blockDim.x) {
        const int e = base + threadIdx.x;
        int units = 0;
        if (e < E) {
            const int o0 = offsets[e], o1 = offsets[e + 1];
            if (o0 < 0 || o1 < o0 || o1 > T) bad = 1;
            else units = per_expert(o1 - o0);
            pl.off[e] = o0;
            if (e == E - 1) pl.off[E] = o1;
        }
        int total;
        const int at = block_exclusive_scan(units, pl.scratch, &total);
        if (e < E) pl.pre[e] = run + at;
        run += total;
    }
    if (threadIdx.x == 0) pl.pre[E] = run;
    return !__syncthreads_or(bad);
}

__device__ __forceinline__ int find_expert(const Plan &pl, int E, int u)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pl.pre[mid] <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b, int type)
{
    if (type == SF_TYPE_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(__uint_as_float(a), __uint_as_float(b));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Lane = feature, v[j] = token j: stores up to `n` tokens' rows. Neighbour lanes trade halves, so a lane stores two
// features of one token: even lanes the even tokens, odd lanes the odd ones (64 bytes of a row a warp).
template <int COLS>
__device__ __forceinline__ void store_tokens(const uint32_t (&v)[COLS], uint16_t *out, int64_t ld, int f, int M, int n,
                                             int type)
{
    const bool odd = f & 1;
#pragma unroll
    for (int j = 0; j < COLS; j += 2) {
        const uint32_t mine = pack2(v[j], v[j + 1], type);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
        const uint32_t w = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
        const int t = j + odd;
        if (t < n && f < M) *reinterpret_cast<uint32_t *>(out + (int64_t)t * ld + (f & ~1)) = w;
    }
}

// ------------------------------------------------------------------------------------------------
// forward and dx, CTA pairs
// ------------------------------------------------------------------------------------------------

struct PUnit {
    int e, m0, t0, n;          // expert, first accumulator row, first token, tokens
};

__device__ __forceinline__ PUnit pair_unit(const Plan &pl, const GArgs &g, int u)
{
    PUnit x;
    x.e = find_expert(pl, g.E, u);
    const int cnt = pl.off[x.e + 1] - pl.off[x.e];
    const int tile = tile_tokens(cnt, PN, 32), tiles = (cnt + tile - 1) / tile;
    const int m_tiles = (g.M + PM - 1) / PM;
    const int local = u - pl.pre[x.e];
    // token tiles in bands of P_BAND, all weight tiles of a band before the next band: pairs at work together
    // share weight tiles and a band's tokens in L2
    const int band = local / (m_tiles * P_BAND);
    const int in = local - band * m_tiles * P_BAND;
    const int width = min(P_BAND, tiles - band * P_BAND);
    const int mt = in / width, nt = band * P_BAND + in - mt * width;
    x.m0 = mt * PM;
    x.t0 = pl.off[x.e] + nt * tile;
    x.n = min(tile, cnt - nt * tile);
    return x;
}

template <bool TRANS>
__global__ void __launch_bounds__(P_THREADS, 1)
grouped_pair_kernel(const __grid_constant__ GArgs g, uint32_t *status)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_bar[P_STAGES], empty_bar[P_STAGES], tfull_bar[P_NBUF], tempty_bar[P_NBUF], drain_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_flag;
    __shared__ Plan pl;

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = cluster_ctarank();
    const bool leader = crank == 0;
    const int unit0 = blockIdx.x / 2, ustep = gridDim.x / 2;

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < P_STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int a = 0; a < P_NBUF; ++a) {
            mbar_init(&tfull_bar[a], 1);
            mbar_init(&tempty_bar[a], P_EPI_WARPS * 2);
        }
        mbar_init(&drain_bar, 1);
        fence_mbarrier_init();
        prefetch_tmap(&g.tm_w);
        prefetch_tmap(&g.tm_x);
    }
    const int m_tiles = (g.M + PM - 1) / PM;
    const bool valid = load_plan(pl, g.offsets, g.E, g.T, [&](int cnt) {
        if (cnt == 0) return 0;
        const int tile = tile_tokens(cnt, PN, 32);
        return (cnt + tile - 1) / tile * m_tiles;
    });
    if (!valid) {                                 // both CTAs of every pair see the same offsets
        if (blockIdx.x == 0 && tid == 0) set_status(status, SF_STATUS_BAD_OFFSET);
        return;
    }
    if (warp == 1) tmem_alloc_pair(&tmem_base_s, P_TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_s;
    const int total_units = pl.pre[g.E];
    const int nk = (g.K + GK - 1) / GK;

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool issued[P_STAGES] = {};
            uint32_t issued_parity[P_STAGES] = {};
            bool ok = true;
            for (int u = unit0; u < total_units && ok; u += ustep) {
                const PUnit x = pair_unit(pl, g, u);
                const int half_n = ((x.n + 31) & ~31) / 2;
                const int m = x.m0 + (int)crank * 128, t = x.t0 + (int)crank * half_n;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag)) { ok = false; break; }
                    uint8_t *sw = smem + stage * P_STAGE_BYTES, *sx = sw + P_HALF_BYTES;
                    if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * P_STAGE_BYTES);
                    if (TRANS) {
                        tma_load_3d_pair(sw, &g.tm_w, &full_bar[stage], m, kb * GK, x.e);
                        tma_load_3d_pair(sw + G_BOX_BYTES, &g.tm_w, &full_bar[stage], m + 64, kb * GK, x.e);
                    } else {
                        tma_load_3d_pair(sw, &g.tm_w, &full_bar[stage], kb * GK, m, x.e);
                    }
                    tma_load_2d_pair(sx, &g.tm_x, &full_bar[stage], kb * GK, t);
                    issued[stage] = true;
                    issued_parity[stage] = phase;
                    if (++stage == P_STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            {   // the MMA issuer commits drain_bar once it has finished or given up
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            }
            if ((!ok || abort_flag) && leader) {  // both CTAs' loads complete on the leader's barriers
                for (int s = 0; s < P_STAGES; ++s) {
                    if (!issued[s]) continue;
                    const uint64_t t0 = globaltimer_ns();
                    while (!mbar_try_wait(&full_bar[s], issued_parity[s]) && globaltimer_ns() - t0 < kWaitLimitNs) {}
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        if (lane == 0 && leader) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            for (int u = unit0; u < total_units && ok; u += ustep) {
                const PUnit x = pair_unit(pl, g, u);
                const uint32_t id = idesc(g.type, TRANS, false, (x.n + 31) & ~31, PM);
                const uint32_t d_tmem = tmem_base + (uint32_t)(buf * PN);
                if (!mbar_wait(&tempty_bar[buf], buf_phase ^ 1u, &abort_flag)) break;
                tc_fence_after();
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(&full_bar[stage], phase, &abort_flag)) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t sw = smem_u32(smem + stage * P_STAGE_BYTES), sx = sw + P_HALF_BYTES;
#pragma unroll
                    for (int k = 0; k < GK / G_UMMA_K; ++k)       // 16 of K: 32 bytes of a row, or 16 rows
                        mma_bf16_pair(d_tmem, TRANS ? mnmajor(sw + k * G_UMMA_K * 128) : kmajor(sw + k * 32),
                                      kmajor(sx + k * 32), id, (kb | k) != 0);
                    mma_commit_pair(&empty_bar[stage], 3);
                    if (++stage == P_STAGES) { stage = 0; phase ^= 1u; }
                }
                if (!ok) break;
                mma_commit_pair(&tfull_bar[buf], 3);
                if (++buf == P_NBUF) { buf = 0; buf_phase ^= 1u; }
            }
            mma_commit_pair(&drain_bar, 3);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
        }
    } else {
        // --------------------------- epilogue (warps 2..9) ---------------------------
        const int quad = warp & 3;              // TMEM lanes 32*quad .. 32*quad+31
        const int half = (warp - 2) >> 2;       // 32-token chunks half, half + 2, ...
        int buf = 0;
        uint32_t buf_phase = 0;
        for (int u = unit0; u < total_units; u += ustep) {
            const PUnit x = pair_unit(pl, g, u);
            const int f = x.m0 + (int)crank * 128 + quad * 32 + lane;
            const bool ready = __all_sync(0xffffffffu, mbar_wait(&tfull_bar[buf], buf_phase, &abort_flag));
            if (!ready) break;
            tc_fence_after();
            const uint32_t t_row = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * PN);
            for (int c = half * 32; c < x.n; c += 64) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(t_row + c, v);
                tmem_ld_wait();
                store_tokens<32>(v, static_cast<uint16_t *>(g.out) + (int64_t)(x.t0 + c) * g.ld_out, g.ld_out, f, g.M,
                                 x.n - c, g.type);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (leader) mbar_arrive(&tempty_bar[buf]);
                else mbar_arrive_remote(&tempty_bar[buf], 0);
            }
            if (++buf == P_NBUF) { buf = 0; buf_phase ^= 1u; }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();                             // neither CTA leaves while the pair's MMAs may run
    if (abort_flag && tid == 0) set_status(status, SF_STATUS_WAIT_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, P_TMEM_COLS);
    }
}

// ------------------------------------------------------------------------------------------------
// forward and dx, few tokens to an expert: one unit to a cluster, K split over its CTAs
// ------------------------------------------------------------------------------------------------

template <bool TRANS>
__global__ void __launch_bounds__(S_THREADS)
grouped_small_kernel(const __grid_constant__ GArgs g, uint32_t *status)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_bar[S_MAX_STAGES], empty_bar[S_MAX_STAGES], done_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_flag;
    __shared__ Plan pl;

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ks = g.ksplit, nb = g.nb, stages = g.stages;
    const int rank = ks > 1 ? (int)cluster_ctarank() : 0;
    const int u = blockIdx.x / ks;

    const int m_tiles = (g.M + SM_ROWS - 1) / SM_ROWS;
    const bool valid = load_plan(pl, g.offsets, g.E, g.T, [&](int cnt) {
        if (cnt == 0) return 0;
        const int tile = tile_tokens(cnt, nb, 16);
        return (cnt + tile - 1) / tile * m_tiles;
    });
    if (!valid) {
        if (blockIdx.x == 0 && tid == 0) set_status(status, SF_STATUS_BAD_OFFSET);
        return;
    }
    if (u >= pl.pre[g.E]) return;               // the whole cluster
    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        mbar_init(&done_bar, 1);
        fence_mbarrier_init();
        prefetch_tmap(&g.tm_w);
        prefetch_tmap(&g.tm_x);
    }
    const uint32_t tmem_cols = nb < 32 ? 32u : (uint32_t)nb;
    if (warp == 1) tmem_alloc(&tmem_base_s, tmem_cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_s;

    const int e = find_expert(pl, g.E, u);
    const int cnt = pl.off[e + 1] - pl.off[e];
    const int tile = tile_tokens(cnt, nb, 16), tiles = (cnt + tile - 1) / tile;
    const int local = u - pl.pre[e], mt = local / tiles, nt = local - mt * tiles;     // tiles of one weight tile adjoin
    const int m0 = mt * SM_ROWS, t0 = pl.off[e] + nt * tile, n = min(tile, cnt - nt * tile);
    const int nk_all = (g.K + GK - 1) / GK;
    const int k0 = (int)((int64_t)nk_all * rank / ks), nk = (int)((int64_t)nk_all * (rank + 1) / ks) - k0;
    const int stage_bytes = S_W_BYTES + nb * GK * 2;

    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, sent = 0;
            uint32_t phase = 0;
            for (int i = 0; i < nk; ++i) {
                if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag)) break;
                uint8_t *sw = smem + stage * stage_bytes, *sx = sw + S_W_BYTES;
                const int k = (k0 + i) * GK;
                mbar_arrive_expect_tx(&full_bar[stage], stage_bytes);
                if (TRANS) {
                    tma_load_3d(sw, &g.tm_w, &full_bar[stage], m0, k, e);
                    tma_load_3d(sw + G_BOX_BYTES, &g.tm_w, &full_bar[stage], m0 + 64, k, e);
                } else {
                    tma_load_3d(sw, &g.tm_w, &full_bar[stage], k, m0, e);
                }
                tma_load_2d(sx, &g.tm_x, &full_bar[stage], k, t0);
                ++sent;
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            const uint64_t begin = globaltimer_ns();
            while (!mbar_try_wait(&done_bar, 0) && globaltimer_ns() - begin < kWaitLimitNs) {}
            if (abort_flag) {                   // drain what was sent before the shared memory goes away
                for (int s = 0; s < stages && s < sent; ++s) {
                    const int last = (sent - 1 - s) / stages;        // the slot's last use
                    const uint64_t from = globaltimer_ns();
                    while (!mbar_try_wait(&full_bar[s], (uint32_t)(last & 1)) && globaltimer_ns() - from < kWaitLimitNs) {}
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            const uint32_t id = idesc(g.type, TRANS, false, (n + 15) & ~15, SM_ROWS);
            for (int i = 0; i < nk; ++i) {
                if (!mbar_wait(&full_bar[stage], phase, &abort_flag)) break;
                tc_fence_after();
                const uint32_t sw = smem_u32(smem + stage * stage_bytes), sx = sw + S_W_BYTES;
#pragma unroll
                for (int k = 0; k < GK / G_UMMA_K; ++k)
                    mma_bf16(tmem_base, TRANS ? mnmajor(sw + k * G_UMMA_K * 128) : kmajor(sw + k * 32), kmajor(sx + k * 32),
                             id, (i | k) != 0);
                mma_commit(&empty_bar[stage]);
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            mma_commit(&done_bar);
        }
    }
    __syncwarp();
    // Everyone waits for the MMAs (the producer has, in lane 0); a CTA that gave up tells its cluster.
    if (!mbar_wait(&done_bar, 0, &abort_flag)) abort_flag = 1;
    __syncthreads();
    const int quad = warp & 3;
    const int f = m0 + quad * 32 + lane;
    uint16_t *out = static_cast<uint16_t *>(g.out) + (int64_t)t0 * g.ld_out;
    tc_fence_after();
    const uint32_t t_row = tmem_base + ((uint32_t)(quad * 32) << 16);
    if (ks == 1) {
        if (warp >= 2 && !abort_flag) {
            for (int c = 0; c < n; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(t_row + c, v);
                tmem_ld_wait();
                store_tokens<16>(v, out + (int64_t)c * g.ld_out, g.ld_out, f, g.M, n - c, g.type);
            }
        }
    } else {
        // Rank q sums token columns q*own .. from the partial sums of ranks 0, 1, ... in that order. The partial
        // sums land in the stages, which are free in every CTA after the first barrier.
        const int own = nb / ks;
        if (tid == 0 && abort_flag)
            for (int q = 0; q < ks; ++q) st_cluster_u32(mapa_u32(smem_u32((const void *)&abort_flag), q), 1u);
        __syncwarp();
        cluster_sync();
        if (warp >= 2) {
            const uint32_t mine = smem_u32(smem) + (uint32_t)((rank * own * SM_ROWS + quad * 32 + lane) * 4);
            for (int c = 0; c < n; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(t_row + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int q = (c + j) / own, at = c + j - q * own;
                    if (c + j < n) st_cluster_u32(mapa_u32(mine + (uint32_t)(at * SM_ROWS * 4), q), v[j]);
                }
            }
        }
        cluster_sync();
        if (warp >= 2 && !abort_flag && f < g.M) {
            const float *part = reinterpret_cast<const float *>(smem) + quad * 32 + lane;
            for (int j = 0; j < own && rank * own + j < n; ++j) {
                float s = 0.0f;
                for (int q = 0; q < ks; ++q) s = __fadd_rn(s, part[(q * own + j) * SM_ROWS]);
                out[(int64_t)(rank * own + j) * g.ld_out + f] = (uint16_t)pack2(__float_as_uint(s), 0u, g.type);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (abort_flag && tid == 0) set_status(status, SF_STATUS_WAIT_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, tmem_cols);
    }
}

// ------------------------------------------------------------------------------------------------
// weight gradient, CTA pairs
// ------------------------------------------------------------------------------------------------

struct WUnit {
    int e, r0, c0, t0, cnt;
};

__device__ __forceinline__ WUnit dw_unit(const Plan &pl, const GArgs &g, int u)
{
    const int m_tiles = (g.M + PM - 1) / PM, n_tiles = (g.K + PN - 1) / PN;
    const int per = m_tiles * n_tiles;
    WUnit x;
    x.e = u / per;
    const int local = u - x.e * per, mt = local / n_tiles;
    x.r0 = mt * PM;
    x.c0 = (local - mt * n_tiles) * PN;
    x.t0 = pl.off[x.e];
    x.cnt = pl.off[x.e + 1] - x.t0;
    return x;
}

__global__ void __launch_bounds__(P_THREADS, 1)
grouped_dw_kernel(const __grid_constant__ GArgs g, uint32_t *status)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_bar[P_STAGES], empty_bar[P_STAGES], tfull_bar[P_NBUF], tempty_bar[P_NBUF], drain_bar;
    __shared__ uint64_t tail_bar[P_STAGES], clear_bar[P_STAGES];   // for the last stage of an expert, where rows are cleared
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_flag;
    __shared__ Plan pl;

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = cluster_ctarank();
    const bool leader = crank == 0;
    const int unit0 = blockIdx.x / 2, ustep = gridDim.x / 2;

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < P_STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
            mbar_init(&tail_bar[s], 1);           // this CTA's loads of the stage have landed
            mbar_init(&clear_bar[s], 2);          // the leader's: both CTAs have cleared their rows
        }
        for (int a = 0; a < P_NBUF; ++a) {
            mbar_init(&tfull_bar[a], 1);
            mbar_init(&tempty_bar[a], P_EPI_WARPS * 2);
        }
        mbar_init(&drain_bar, 1);
        fence_mbarrier_init();
        prefetch_tmap(&g.tm_w);
        prefetch_tmap(&g.tm_x);
    }
    const bool valid = load_plan(pl, g.offsets, g.E, g.T, [](int) { return 0; });
    if (!valid) {
        if (blockIdx.x == 0 && tid == 0) set_status(status, SF_STATUS_BAD_OFFSET);
        return;
    }
    if (warp == 1) tmem_alloc_pair(&tmem_base_s, P_TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_s;
    const int total_units = g.E * ((g.M + PM - 1) / PM) * ((g.K + PN - 1) / PN);

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool issued[P_STAGES] = {};
            uint32_t issued_parity[P_STAGES] = {};
            uint32_t tails = 0, tail_parity = 0;  // by stage: whether it held a tail, and the parity of its last one
            bool ok = true;
            for (int u = unit0; u < total_units && ok; u += ustep) {
                const WUnit x = dw_unit(pl, g, u);
                const int nk = (x.cnt + GK - 1) / GK;
                const int r = x.r0 + (int)crank * 128, c = x.c0 + (int)crank * 128;
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag)) { ok = false; break; }
                    uint8_t *sy = smem + stage * P_STAGE_BYTES, *sa = sy + P_HALF_BYTES;
                    const int t = x.t0 + kb * GK;
                    if (kb == nk - 1 && (x.cnt & (G_UMMA_K - 1))) {
                        // rows to clear: each CTA's loads complete on its own barrier, for the warp that clears them
                        if (leader) mbar_arrive(&full_bar[stage]);
                        mbar_arrive_expect_tx(&tail_bar[stage], P_STAGE_BYTES);
                        tma_load_2d(sy, &g.tm_x, &tail_bar[stage], r, t);
                        tma_load_2d(sy + G_BOX_BYTES, &g.tm_x, &tail_bar[stage], r + 64, t);
                        tma_load_2d(sa, &g.tm_w, &tail_bar[stage], c, t);
                        tma_load_2d(sa + G_BOX_BYTES, &g.tm_w, &tail_bar[stage], c + 64, t);
                        if (tails >> stage & 1u) tail_parity ^= 1u << stage;
                        tails |= 1u << stage;
                    } else {
                        if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * P_STAGE_BYTES);
                        tma_load_2d_pair(sy, &g.tm_x, &full_bar[stage], r, t);
                        tma_load_2d_pair(sy + G_BOX_BYTES, &g.tm_x, &full_bar[stage], r + 64, t);
                        tma_load_2d_pair(sa, &g.tm_w, &full_bar[stage], c, t);
                        tma_load_2d_pair(sa + G_BOX_BYTES, &g.tm_w, &full_bar[stage], c + 64, t);
                    }
                    issued[stage] = true;
                    issued_parity[stage] = phase;
                    if (++stage == P_STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            {
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            }
            if (!ok || abort_flag) {
                if (leader) {
                    for (int s = 0; s < P_STAGES; ++s) {
                        if (!issued[s]) continue;
                        const uint64_t t0 = globaltimer_ns();
                        while (!mbar_try_wait(&full_bar[s], issued_parity[s]) && globaltimer_ns() - t0 < kWaitLimitNs) {}
                    }
                }
                for (int s = 0; s < P_STAGES; ++s) {
                    if (!(tails >> s & 1u)) continue;
                    const uint64_t t0 = globaltimer_ns();
                    while (!mbar_try_wait(&tail_bar[s], tail_parity >> s & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {}
                }
            }
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader); clearing of rows behind an expert's end (both) ----------------
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0, tail_phase = 0;     // tail_phase: a bit a stage
        bool ok = true;
        for (int u = unit0; u < total_units && ok; u += ustep) {
            const WUnit x = dw_unit(pl, g, u);
            const int nk = (x.cnt + GK - 1) / GK;
            const uint32_t id = idesc(g.type, true, true, PN, PM);
            for (int kb = 0; kb < nk; ++kb) {
                const int in_chunk = kb % W_CHUNK_STAGES;
                const bool tail = kb == nk - 1 && (x.cnt & (G_UMMA_K - 1));
                uint8_t *sy = smem + stage * P_STAGE_BYTES;
                if (tail) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&tail_bar[stage], tail_phase >> stage & 1u, &abort_flag));
                    if (!ok) break;
                    const int from = x.cnt - kb * GK, upto = (from + G_UMMA_K - 1) & ~(G_UMMA_K - 1);
                    // a token is one 128-byte row of each of the stage's four boxes
                    for (int i = lane; i < (upto - from) * 8; i += 32)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4 *>(sy + q * G_BOX_BYTES + (from + (i >> 3)) * 128 + (i & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (leader) mbar_arrive(&clear_bar[stage]);
                        else mbar_arrive_remote(&clear_bar[stage], 0);
                    }
                }
                if (leader) {
                    if (lane == 0) {
                        if (in_chunk == 0) ok = mbar_wait(&tempty_bar[buf], buf_phase ^ 1u, &abort_flag);
                        if (ok) ok = mbar_wait(&full_bar[stage], phase, &abort_flag);
                        if (ok && tail) ok = mbar_wait_cluster(&clear_bar[stage], tail_phase >> stage & 1u, &abort_flag);
                        if (ok) {
                            tc_fence_after();
                            const uint32_t a = smem_u32(sy), bb = a + P_HALF_BYTES;
                            const uint32_t d_tmem = tmem_base + (uint32_t)(buf * PN);
                            const int steps = min(GK, x.cnt - kb * GK + G_UMMA_K - 1) / G_UMMA_K;
                            for (int k = 0; k < steps; ++k)
                                mma_bf16_pair(d_tmem, mnmajor(a + k * G_UMMA_K * 128), mnmajor(bb + k * G_UMMA_K * 128), id,
                                              (in_chunk | k) != 0);
                            mma_commit_pair(&empty_bar[stage], 3);
                            if (in_chunk == W_CHUNK_STAGES - 1 || kb == nk - 1) mma_commit_pair(&tfull_bar[buf], 3);
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    if (in_chunk == W_CHUNK_STAGES - 1 || kb == nk - 1)
                        if (++buf == P_NBUF) { buf = 0; buf_phase ^= 1u; }
                }
                if (tail) tail_phase ^= 1u << stage;
                if (++stage == P_STAGES) { stage = 0; phase ^= 1u; }
            }
        }
        if (leader && lane == 0) {
            mma_commit_pair(&drain_bar, 3);
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
        }
    } else {
        // --------------------------- epilogue (warps 2..9) ---------------------------
        const int quad = warp & 3;              // accumulator rows 32*quad .. 32*quad+31 of the CTA
        const int half = (warp - 2) >> 2;       // columns half*128 .. +127
        int buf = 0;
        uint32_t buf_phase = 0;
        for (int u = unit0; u < total_units; u += ustep) {
            const WUnit x = dw_unit(pl, g, u);
            const int nk = (x.cnt + GK - 1) / GK;
            if (nk == 0 && g.accumulate) continue;
            const int r = x.r0 + (int)crank * 128 + quad * 32 + lane, c0 = x.c0 + half * 128;
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
            bool ready = true;
            const int nchunks = (nk + W_CHUNK_STAGES - 1) / W_CHUNK_STAGES;
            for (int ch = 0; ch < nchunks; ++ch) {
                ready = __all_sync(0xffffffffu, mbar_wait(&tfull_bar[buf], buf_phase, &abort_flag));
                if (!ready) break;
                tc_fence_after();
                const uint32_t t_row = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * PN + half * 128);
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(t_row + cc * 32, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[cc * 32 + j] = __fadd_rn(acc[cc * 32 + j], __uint_as_float(v[j]));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(&tempty_bar[buf]);
                    else mbar_arrive_remote(&tempty_bar[buf], 0);
                }
                if (++buf == P_NBUF) { buf = 0; buf_phase ^= 1u; }
            }
            if (!ready) break;
            if (r >= g.M) continue;
            const int64_t at = (int64_t)x.e * g.stride_out + (int64_t)r * g.ld_out + c0;
            if (g.out_f32) {
                float *out = static_cast<float *>(g.out) + at;
#pragma unroll
                for (int j = 0; j < 128; j += 4) {
                    if (c0 + j >= g.K) break;
                    float4 v = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                    if (g.accumulate) {
                        const float4 o = *reinterpret_cast<const float4 *>(out + j);
                        v = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
                    }
                    *reinterpret_cast<float4 *>(out + j) = v;
                }
            } else {
                uint16_t *out = static_cast<uint16_t *>(g.out) + at;
#pragma unroll
                for (int j = 0; j < 128; j += 8) {
                    if (c0 + j >= g.K) break;
                    uint32_t w[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        w[q] = pack2(__float_as_uint(acc[j + 2 * q]), __float_as_uint(acc[j + 2 * q + 1]), g.type);
                    *reinterpret_cast<uint4 *>(out + j) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (abort_flag && tid == 0) set_status(status, SF_STATUS_WAIT_TIMEOUT);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, P_TMEM_COLS);
    }
}

// ------------------------------------ host side ------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn grouped_encode_fn()
{
    static std::atomic<EncodeTiledFn> cached{nullptr};
    EncodeTiledFn fn = cached.load(std::memory_order_relaxed);
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        fn = reinterpret_cast<EncodeTiledFn>(p);
        cached.store(fn, std::memory_order_relaxed);
    }
    return fn;
}

// 16-bit map over [depth x rows x cols] with 128-byte swizzled boxes of 64 columns by box_rows rows.
bool encode(CUtensorMap *m, int type, const void *base, int cols, int64_t rows, int64_t ld, int depth, int64_t stride,
            int box_rows)
{
    EncodeTiledFn fn = grouped_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)(rows > 0 ? rows : 1), (cuuint64_t)depth};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64u, (cuuint32_t)box_rows, 1u};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, type == SF_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              depth > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

int check_grouped(const sf_grouped *p, bool dw)
{
    if (!p) return SF_ERR_ARG;
    if (p->E < 1 || p->T < 0 || p->R <= 0 || p->C <= 0 || (p->R & 7) || (p->C & 7)) return SF_ERR_ARG;
    if (p->type != SF_TYPE_BF16 && p->type != SF_TYPE_F16) return SF_ERR_ARG;
    if (p->w_type != p->type && !(dw && p->w_type == SF_TYPE_F32)) return SF_ERR_ARG;
    if (!p->W || !p->offsets) return SF_ERR_ARG;
    if (p->ld_w < p->C || (p->E > 1 && p->stride_w < (int64_t)(p->R - 1) * p->ld_w + p->C)) return SF_ERR_ARG;
    const int w_unit = p->w_type == SF_TYPE_F32 ? 3 : 7;
    if (!aligned16(p->W) || (p->ld_w & w_unit) || (p->E > 1 && (p->stride_w & w_unit)) || ((uintptr_t)p->offsets & 3))
        return SF_ERR_ALIGN;
    if (p->T > 0) {
        if (!p->A || !p->Y || p->ld_a < p->C || p->ld_y < p->R) return SF_ERR_ARG;
        if (!aligned16(p->A) || !aligned16(p->Y) || (p->ld_a & 7) || (p->ld_y & 7)) return SF_ERR_ALIGN;
    }
    if (p->E > kMaxE) return SF_ERR_UNSUPPORTED;
    // byte strides a tensor map can hold (below 2^40), and tile counts that stay far inside 32 bits
    const int64_t far = (int64_t)1 << 38;
    if (p->ld_w > far || p->stride_w > far || p->ld_a > far || p->ld_y > far) return SF_ERR_UNSUPPORTED;
    const int64_t wide = (p->R > p->C ? p->R : p->C) / 128 + 1;
    const int64_t tall = (int64_t)p->T / 16 + p->E;
    if (wide * tall > (1 << 30) || (int64_t)p->E * ((p->R + PM - 1) / PM) * ((p->C + PN - 1) / PN) > (1 << 30))
        return SF_ERR_UNSUPPORTED;
    return SF_OK;
}

// CTA pairs that can be resident at once on the current device (the same for the three pair kernels: their
// threads and shared memory agree).
int pair_slots()
{
    constexpr int kDevs = 64;
    static std::atomic<int> cached[kDevs];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < kDevs) {
        const int n = cached[dev].load(std::memory_order_relaxed);
        if (n > 0) return n;
    }
    const int sms = sm_count();
    if (sms <= 0) return 0;
    if (cudaFuncSetAttribute(grouped_pair_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)P_SMEM_BYTES) != cudaSuccess)
        return 0;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * sms);
    cfg.blockDim = dim3(P_THREADS);
    cfg.dynamicSmemBytes = P_SMEM_BYTES;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, grouped_pair_kernel<false>, &cfg) != cudaSuccess || n <= 0) return 0;
    if (dev < kDevs) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <typename K>
int launch(K kernel, int grid, int cluster, int threads, size_t smem, const GArgs &g, uint32_t *status, sf_stream stream)
{
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return SF_ERR_CUDA;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = as_stream(stream);
    cfg.attrs = &attr;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, kernel, g, status) != cudaSuccess) return SF_ERR_CUDA;
    return launch_status();
}

// Pairs run when an expert has more than this many tokens on average.
#ifndef SF_GROUPED_PAIR_FROM
#define SF_GROUPED_PAIR_FROM 96
#endif

template <bool TRANS>
int grouped_product(const sf_grouped *p, uint32_t *status, sf_stream stream)
{
    int rc = check_grouped(p, false);
    if (rc != SF_OK) return rc;
    if (p->T == 0) return SF_OK;
    const int sms = sm_count();
    if (sms <= 0) return SF_ERR_NO_DEVICE;
    GArgs g;
    memset(&g, 0, sizeof(g));
    const bool fwd = !TRANS;
    g.offsets = p->offsets;
    g.out = fwd ? p->Y : p->A;
    g.ld_out = fwd ? p->ld_y : p->ld_a;
    g.E = p->E;
    g.T = p->T;
    g.M = fwd ? p->R : p->C;
    g.K = fwd ? p->C : p->R;
    g.type = p->type;
    const void *x = fwd ? p->A : p->Y;
    const int64_t ld_x = fwd ? p->ld_a : p->ld_y;
    const int64_t stride = p->E > 1 ? p->stride_w : (int64_t)p->R * p->ld_w;
    const int w_rows = fwd ? 128 : 64;
    const int nk = (g.K + GK - 1) / GK;

    if (p->T > (int64_t)SF_GROUPED_PAIR_FROM * p->E) {
        if (!encode(&g.tm_w, p->type, p->W, p->C, p->R, p->ld_w, p->E, stride, w_rows) ||
            !encode(&g.tm_x, p->type, x, g.K, p->T, ld_x, 0, 0, 128))
            return SF_ERR_CUDA;
        const int slots = pair_slots();
        if (slots <= 0) return SF_ERR_CUDA;
        const int64_t most = ((int64_t)p->T / 64 + p->E) * ((g.M + PM - 1) / PM);
        const int pairs = (int)(most < slots ? most : slots);
        return launch(grouped_pair_kernel<TRANS>, 2 * pairs, 2, P_THREADS, P_SMEM_BYTES, g, status, stream);
    }
    // a box of twice the average tokens holds nearly every expert in one tile
    const int avg = (p->T + p->E - 1) / p->E;
    int nb = 16;
    while (nb < 128 && nb < 2 * avg && nb < p->T) nb *= 2;
    g.nb = nb;
    const int stage_bytes = S_W_BYTES + nb * GK * 2;
    g.stages = 100 * 1024 / stage_bytes;                 // two CTAs to an SM
    if (g.stages > S_MAX_STAGES) g.stages = S_MAX_STAGES;
    const int64_t m_tiles = (g.M + SM_ROWS - 1) / SM_ROWS;
    const int64_t busy = p->E < p->T ? p->E : p->T;      // experts with a token, at most
    const int64_t units = (busy + p->T / nb) * m_tiles;  // tiles, at most
    int ks = 1;
    while (ks < 8 && busy * m_tiles * ks < 4 * sms && nk >= 8 * ks && nb / (2 * ks) >= 1) ks *= 2;
    g.ksplit = ks;
    if (!encode(&g.tm_w, p->type, p->W, p->C, p->R, p->ld_w, p->E, stride, w_rows) ||
        !encode(&g.tm_x, p->type, x, g.K, p->T, ld_x, 0, 0, nb))
        return SF_ERR_CUDA;
    return launch(grouped_small_kernel<TRANS>, (int)(units * ks), ks, S_THREADS, (size_t)g.stages * stage_bytes + 1024, g,
                  status, stream);
}

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" int sf_grouped_forward(const sf_grouped *p, uint32_t *dev_status, sf_stream stream)
{
    return grouped_product<false>(p, dev_status, stream);
}

extern "C" int sf_grouped_dx(const sf_grouped *p, uint32_t *dev_status, sf_stream stream)
{
    return grouped_product<true>(p, dev_status, stream);
}

extern "C" int sf_grouped_dw(const sf_grouped *p, int accumulate, uint32_t *dev_status, sf_stream stream)
{
    int rc = check_grouped(p, true);
    if (rc != SF_OK) return rc;
    if (accumulate && p->w_type != SF_TYPE_F32) return SF_ERR_ARG;
    if (sm_count() <= 0) return SF_ERR_NO_DEVICE;
    GArgs g;
    memset(&g, 0, sizeof(g));
    g.offsets = p->offsets;
    g.out = p->W;
    g.ld_out = p->ld_w;
    g.stride_out = p->E > 1 ? p->stride_w : 0;
    g.E = p->E;
    g.T = p->T;
    g.M = p->R;
    g.K = p->C;
    g.type = p->type;
    g.out_f32 = p->w_type == SF_TYPE_F32;
    g.accumulate = accumulate != 0;
    // without tokens nothing is loaded: any valid address makes the maps
    const void *a = p->T > 0 ? p->A : p->W, *y = p->T > 0 ? p->Y : p->W;
    const int64_t ld_a = p->T > 0 ? p->ld_a : p->C, ld_y = p->T > 0 ? p->ld_y : p->R;
    if (!encode(&g.tm_w, p->type, a, p->C, p->T, ld_a, 0, 0, 64) || !encode(&g.tm_x, p->type, y, p->R, p->T, ld_y, 0, 0, 64))
        return SF_ERR_CUDA;
    const int slots = pair_slots();
    if (slots <= 0) return SF_ERR_CUDA;
    const int64_t units = (int64_t)p->E * ((p->R + PM - 1) / PM) * ((p->C + PN - 1) / PN);
    return launch(grouped_dw_kernel, 2 * (int)(units < slots ? units : slots), 2, P_THREADS, P_SMEM_BYTES, g, dev_status,
                  stream);
}
