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
#include <stdlib.h>
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

// ---- tiles of CTA pairs: 256 accumulator rows x up to 512 columns, both CTAs' MMAs as one (cta_group::2). The columns
// are two halves of up to 256, two MMAs that share a stage's M operand: a stage of 48 KB in each SM then keeps the
// tensor cores busy for 1,024 cycles, so the ring's 4 cover the 2 us that a stage takes from its release to its next use
// (pairs of 256 x 256 with 32 KB stages: 512 cycles, and 1.4 us with nothing else on the memory system). ----
constexpr int PM = 256;                       // accumulator rows of a pair, 128 in each CTA's TMEM
constexpr int PN = 256;                       // columns of a half, at most
constexpr int P_HALF_BYTES = 128 * GK * 2;    // 128 rows of an operand, a stage, in one CTA: 16 KB
constexpr int P_TMEM_COLS = 2 * PN;
constexpr int P_EPI_WARPS = 8;                // two per TMEM lane quarter
constexpr int P_THREADS = 64 + 32 * P_EPI_WARPS;
constexpr int W_THREADS = P_THREADS + 32;     // weight gradient: and a warp that clears rows
constexpr int T_TOKENS = 2 * PN;              // columns of a tile, at most
constexpr int T_RING_BYTES = 4 * 3 * P_HALF_BYTES;
constexpr int T_MAX_STAGES = 8;
constexpr int T_OUT_BYTES = 32 * 128 * 2;     // forward, dx: 2 x 16 tokens' rows of the CTA's 128 features, on their way out
constexpr int W_OUT_BYTES = 32 * 128;         // weight gradient: 32 rows of 128 bytes of a warp's output
constexpr size_t T_SMEM_BYTES = (size_t)T_RING_BYTES + 2 * T_OUT_BYTES + 1024;
// weight gradient: 256 columns to a tile, two accumulators that the MMAs and the epilogue take in turn
constexpr int W_STAGES_NEW = 6, W_STAGES_FEW = 3;
constexpr int W_STAGE_BYTES = 2 * P_HALF_BYTES;
constexpr size_t W_SMEM_BYTES = (size_t)W_STAGES_NEW * W_STAGE_BYTES + P_EPI_WARPS * W_OUT_BYTES + 1024;
static_assert(W_SMEM_BYTES == (size_t)W_STAGES_FEW * W_STAGE_BYTES + P_EPI_WARPS * 4 * W_OUT_BYTES + 1024, "both divisions");
constexpr int T_AHEAD = 3;                    // stages of a unit whose first halves run before any second half
constexpr int T_BAND = 4;                     // token tiles that share a pass over an expert's weights

// ---- single CTAs: 128 accumulator rows x up to 256 columns ----
constexpr int SM_ROWS = 128;
constexpr int S_EPI_WARPS = 4;
constexpr int S_THREADS = 64 + 32 * S_EPI_WARPS;
constexpr int S_W_BYTES = SM_ROWS * GK * 2;   // 16 KB
constexpr int S_MAX_STAGES = 12;
constexpr int S_RING_BYTES = 200 * 1024;      // stages of a CTA that has its SM to itself, at most; half for two to an SM
constexpr size_t S_SMEM_BYTES = (size_t)S_RING_BYTES + 1024;
constexpr int D_THREADS = P_THREADS;          // weight gradient: TMA, MMA and eight epilogue warps
constexpr int D_STAGE_BYTES = 3 * P_HALF_BYTES;
constexpr int D_MAX_STAGES = 4;
constexpr size_t D_SMEM_BYTES = (size_t)D_MAX_STAGES * D_STAGE_BYTES + 1024;

// Weight gradient, fp32: tokens that the tensor core sums before the sums are added in fp32, in stages. It adds with
// truncation, so the error grows with the length (relative, normal values: 2.3e-7, 9.9e-7 and 9.1e-6 at 256, 1,024
// and 8,192 tokens); 960 keep it below 1e-6 at any length.
constexpr int W_CHUNK_STAGES = 960 / GK;
// In 16 bits, which round by up to 2^-8 or 2^-11 (4.9e-4): 8,192 tokens in single CTAs. Sums of one sign drift by 5.5e-9 a token,
// 4.5e-5 of those. Only the pairs and four slices have a place for their sums, in registers; calls that could make sums of more
// than 32,768 tokens in one or two slices (1.8e-4) take those (1032 x 520 over 200,000 tokens, two slices against pairs: 905 us
// and 5.6e-4 off on average, 1,195 us and 1.2e-5).
constexpr int W16_CHUNK_STAGES = 8192 / GK;
constexpr int W16_TOKENS = 32768;

// Tokens to a tile, at most, that the pair kernel chooses from.
constexpr int kCands = 15;
__device__ __forceinline__ int cand_tokens(int i) { return T_TOKENS - 32 * i; }      // 512 .. 64

struct GArgs {
    CUtensorMap tm_w;          // forward, dx: W as {C, R, E}; dw: A as {C, T}
    CUtensorMap tm_x;          // dw: Y as {R, T}
    CUtensorMap tm_out;        // dw: W as {C, R, E}, boxes of 128 bytes x 32 rows
    // forward, dx: tokens, A or Y as {K, T}, in boxes of as many rows as a tile needs (a box more costs more than its
    // rows): 32, 64, 96 and 128 for CTA pairs, 16, 32, 64 and 128 for single CTAs
    CUtensorMap tm_t[4];
    CUtensorMap tm_y;          // CTA pairs: the output as {M, T}, boxes of 128 features x 16 tokens
    const int32_t *offsets;
    void *out;
    int64_t ld_out, stride_out;
    int32_t E, T, M, K, type;  // M: accumulator rows in all (forward R, dx C, dw R); K: forward C, dx R, dw C (its N)
    int32_t nb, stages;              // single CTAs: token box, stages
    int32_t split;                   // single CTAs in slices: CTAs (a cluster) that share a unit's K
    int32_t out_f32, accumulate;     // dw
    int32_t whole;                   // dw: tm_t[0] (bit 0) and tm_t[1] (bit 1) have Y and A by chunks of 64 columns
    int32_t withhold_test;           // test hook: CTA 0's first stage never completes
};

// Arrivals that complete a phase of stage s's barriers. The test hook withholds one of the first stage's in CTA 0, so that the
// waits for that stage run out.
__device__ __forceinline__ uint32_t stage_arrivals(const GArgs &g, int s)
{
    return g.withhold_test && blockIdx.x == 0 && s == 0 ? 2 : 1;
}

// A CTA whose waits ran out leaves NaN in the place of its sums for the other CTAs of its cluster (none of its loads may be in
// flight), so that each of them sees it in the results and stores none. A NaN may also be right: whether a CTA gave up is only
// looked at then. Times as without it but for dw over clusters, 2% more; with the flags read ahead of the sums 4 to 11% more
// (64 x 4096 over 300 tokens 8.2 / 9.1 us, 128 x 128 over 65,536 31.3 / 33.0).
__device__ __noinline__ void leave_nan(uint8_t *sums, int n, int first, int step)
{
    for (int i = first; i < n; i += step) reinterpret_cast<volatile uint32_t *>(sums)[i] = 0x7FFFFFFFu;
}
__device__ __noinline__ bool cluster_gave_up(const volatile int *abort, int ctas)
{
    const uint32_t flag = smem_u32(const_cast<const int *>(abort));
    int any = 0;
    for (int c = 0; c < ctas; ++c) any |= ld_cluster_s32(flag, c);
    return any != 0;
}

__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}
// K-major: 128-byte rows, 8-row groups 1024 bytes apart (the leading offset is unused).
__device__ __forceinline__ uint64_t kmajor(uint32_t addr) { return sw128_desc(addr, 16, 1024); }
// MN-major: 64-element chunks a box apart, groups of 8 K rows 1024 bytes apart.
__device__ __forceinline__ uint64_t mnmajor(uint32_t addr) { return sw128_desc(addr, G_BOX_BYTES, 1024); }
// MN-major in 32-element chunks (64-byte rows, 64-byte swizzle) half a box apart.
__device__ __forceinline__ uint64_t mnmajor64(uint32_t addr)
{
    return (sw128_desc(addr, G_BOX_BYTES / 2, 512) & ~(7ull << 61)) | (4ull << 61);
}

// kind::f16: fp32 accumulator, A and B both bf16 or both fp16, their majors, N, M.
__device__ __forceinline__ uint32_t idesc(int type, bool a_mn, bool b_mn, int n, int m)
{
    const uint32_t t = type == SF_TYPE_BF16 ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// a / b for a >= 0, b > 0: below 2^24 both are exact in fp32 and the quotient of an approximate division is at most one
// off. The units' places are worked out again and again, and an integer division is a chain of ~150 cycles.
__device__ __forceinline__ int quot(int a, int b)
{
    if (a >= 1 << 24) return a / b;
    int q = (int)__fdividef((float)a, (float)b);
    const int r = a - q * b;
    q += (r >= b) - (r < 0);
    return q;
}
__device__ __forceinline__ int quot_up(int a, int b) { return quot(a + b - 1, b); }

// Token tiles of an expert: as few as `most` tokens each allow, evenly filled, in steps of `step` tokens (a power of 2).
__device__ __forceinline__ int tile_tokens(int cnt, int most, int step)
{
    return (quot_up(cnt, quot_up(cnt, most)) + step - 1) & -step;
}

struct Plan {
    int off[kMaxE + 1];        // offsets
    int pre[kMaxE + 1];        // units of the experts before, in the order below
    uint16_t order[kMaxE];     // experts in the order in which their units are numbered
    int scratch[33];
    float cand_time[kCands];
};

// Offsets into shared memory. False (for every thread) when they are not valid. Contains __syncthreads.
__device__ __forceinline__ bool load_offsets(Plan &pl, const int32_t *offsets, int E, int T)
{
    int bad = 0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const int o0 = offsets[e], o1 = offsets[e + 1];
        if (o0 < 0 || o1 < o0 || o1 > T) bad = 1;
        pl.off[e] = o0;
        if (e == E - 1) pl.off[E] = o1;
    }
    return !__syncthreads_or(bad);
}

// Experts by falling key (their own order among equals): long units first, so that the last ones to finish are
// short. Beyond kSortE experts the units are short beside the whole and keep the experts' order: ranking them, E
// reads a thread for each E / blockDim.x experts, would cost more than it evens out. Contains __syncthreads.
constexpr int kSortE = 256;
template <typename F>
__device__ __forceinline__ void order_experts(Plan &pl, int E, F key)
{
    int *keys = pl.pre;                       // free until the units are counted
    if (E <= kSortE)
        for (int e = threadIdx.x; e < E; e += blockDim.x) keys[e] = key(pl.off[e + 1] - pl.off[e]);
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int rank = e;
        if (E <= kSortE) {
            const int mine = keys[e];
            rank = 0;
            for (int k = 0; k < E; ++k) rank += keys[k] > mine || (keys[k] == mine && k < e);
        }
        pl.order[rank] = (uint16_t)e;
    }
    __syncthreads();
}

// Unit counts of the experts in order: per_expert(tokens) -> units. Contains __syncthreads.
template <typename F>
__device__ __forceinline__ void count_units(Plan &pl, int E, F per_expert)
{
    int run = 0;
    for (int base = 0; base < E; base += blockDim.x) {
        const int i = base + threadIdx.x;
        int units = 0;
        if (i < E) {
            const int e = pl.order[i];
            units = per_expert(pl.off[e + 1] - pl.off[e]);
        }
        int total;
        const int at = block_exclusive_scan(units, pl.scratch, &total);
        if (i < E) pl.pre[i] = run + at;
        run += total;
    }
    if (threadIdx.x == 0) pl.pre[E] = run;
    __syncthreads();
}

// The place in the order of the expert that unit u belongs to.
__device__ __forceinline__ int find_place(const Plan &pl, int E, int u)
{
    int lo = 0, hi = E - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pl.pre[mid] <= u) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Worker w of n takes units w, 2n-1-w, 2n+w, 4n-1-w, ...: with units that get shorter, what a worker gains in one
// round it gives back in the next. The unit of round i, which may be past the last one.
__device__ __forceinline__ int unit_of(int i, int w, int n) { return i * n + ((i & 1) ? n - 1 - w : w); }

__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b, int type)
{
    if (type == SF_TYPE_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __half2 h = __floats2half2_rn(__uint_as_float(a), __uint_as_float(b));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Lane = feature, w[j] = tokens 2j and 2j + 1, packed: stores up to `n` tokens' rows. Neighbour lanes trade halves, so a
// lane stores two features of one token: even lanes the even tokens, odd lanes the odd ones (64 bytes of a row a warp).
template <int COLS>
__device__ __forceinline__ void store_tokens(const uint32_t (&w)[COLS / 2], uint16_t *out, int64_t ld, int f, int M, int n)
{
    const bool odd = f & 1;
#pragma unroll
    for (int j = 0; j < COLS; j += 2) {
        const uint32_t mine = w[j / 2];
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
        const uint32_t both = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
        const int t = j + odd;
        if (t < n && f < M) *reinterpret_cast<uint32_t *>(out + (int64_t)t * ld + (f & ~1)) = both;
    }
}

// ------------------------------------------------------------------------------------------------
// forward and dx, CTA pairs
// ------------------------------------------------------------------------------------------------

struct PUnit {
    int e, m0, t0, n;          // expert, first accumulator row, first token, tokens
    int n0, n1;                // accumulator columns of the two halves (steps of 32; n1 may be 0)
};

__device__ __forceinline__ PUnit pair_unit(const Plan &pl, const GArgs &g, int most, int u)
{
    PUnit x;
    const int place = find_place(pl, g.E, u);
    x.e = pl.order[place];
    const int cnt = pl.off[x.e + 1] - pl.off[x.e];
    const int tile = tile_tokens(cnt, most, 32), tiles = quot_up(cnt, tile);
    const int m_tiles = (g.M + PM - 1) / PM;
    const int local = u - pl.pre[place];
    // token tiles in bands of T_BAND, all weight tiles of a band before the next band: pairs at work together
    // share weight tiles and a band's tokens in L2
    const int band = quot(local, m_tiles * T_BAND);
    const int in = local - band * m_tiles * T_BAND;
    const int width = min(T_BAND, tiles - band * T_BAND);
    const int mt = quot(in, width), nt = band * T_BAND + in - mt * width;
    x.m0 = mt * PM;
    x.t0 = pl.off[x.e] + nt * tile;
    x.n = min(tile, cnt - nt * tile);
    x.n0 = min((x.n + 31) & ~31, PN);
    x.n1 = ((x.n + 31) & ~31) - x.n0;
    return x;
}

// The accumulator of a unit's first half: a unit of one half takes the two in turn, so that its MMAs need not wait for the
// unit before to be drained.
__device__ __forceinline__ int accumulator_of(const PUnit &x, int &turn)
{
    if (x.n1) return 0;
    turn ^= 1;
    return turn ^ 1;
}

// The tile size for these offsets: the one whose rounds of units, at the mean cost of a unit, end first. A unit's time
// is about that of its accumulator columns and 128 more, for its weights and its ends (measured, 4 rounds of 4,096-long
// sums: 154, 204 and 248 us at 256, 384 and 512 tokens), so large tiles win unless they leave the last round empty.
// Counted in steps of 32 columns. A warp to a candidate, a lane to an expert; every thread gets the answer. Contains __syncthreads.
__device__ __forceinline__ int choose_tile(Plan &pl, const GArgs &g, int workers)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < kCands; i += P_THREADS / 32) {
        const int most = cand_tokens(i);
        int tiles = 0, cost = 0;
        for (int e = lane; e < g.E; e += 32) {
            const int cnt = pl.off[e + 1] - pl.off[e];
            if (cnt == 0) continue;
            const int tile = tile_tokens(cnt, most, 32), n = quot_up(cnt, tile);
            tiles += n;
            cost += (n - 1) * (tile / 32 + 4) + (cnt - (n - 1) * tile + 31) / 32 + 4;
        }
        tiles = __reduce_add_sync(0xffffffffu, tiles);
        cost = __reduce_add_sync(0xffffffffu, cost);
        if (lane == 0) {
            const float rounds = ceilf(__fdividef((float)tiles * (float)((g.M + PM - 1) / PM), (float)workers));
            pl.cand_time[i] = tiles ? rounds * __fdividef((float)cost, (float)tiles) : 0.0f;
        }
    }
    __syncthreads();
    const uint32_t t = lane < kCands ? __float_as_uint(pl.cand_time[lane]) : 0xffffffffu;     // not negative: ordered as bits
    const uint32_t best = __reduce_min_sync(0xffffffffu, t);
    return cand_tokens(__ffs(__ballot_sync(0xffffffffu, t == best)) - 1);
}

template <bool TRANS>
__global__ void __launch_bounds__(P_THREADS, 1)
grouped_pair_kernel(const __grid_constant__ GArgs g, uint32_t *status)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_bar[T_MAX_STAGES], empty_bar[T_MAX_STAGES], tfull_bar[2], tempty_bar[2], drain_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_flag;
    __shared__ Plan pl;

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = cluster_ctarank();
    const bool leader = crank == 0;
    const int worker = blockIdx.x / 2, workers = gridDim.x / 2;

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < T_MAX_STAGES; ++s) {
            mbar_init(&full_bar[s], stage_arrivals(g, s));
            mbar_init(&empty_bar[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull_bar[a], 1);
            mbar_init(&tempty_bar[a], P_EPI_WARPS * 2);
        }
        mbar_init(&drain_bar, 1);
        fence_mbarrier_init();
        prefetch_tmap(&g.tm_w);
        for (int b = 0; b < 4; ++b) prefetch_tmap(&g.tm_t[b]);
        prefetch_tmap(&g.tm_y);
    }
    griddep_wait();                             // what the launches before this one wrote is there from here on
    if (!load_offsets(pl, g.offsets, g.E, g.T)) {     // both CTAs of every pair see the same offsets
        if (blockIdx.x == 0 && tid == 0) set_status(status, SF_STATUS_BAD_OFFSET);
        return;
    }
    const int most = choose_tile(pl, g, workers);
    // The ring's stages hold what the tiles need: 8 of 24 KB, 6 of 32 KB or 4 of 48 KB. Tiles of up to 128 tokens are
    // bound by the requests to L2 (boxes asked for into L2 ahead of their loads cost 5 to 20% more time), so their token
    // boxes are as high as they need (half as high, when this was measured: 16 experts of 2048 x 2048 over 2048 tokens
    // 39.0 -> 35.7 us, 48 of 1416 x 2056 over 5000 77.6 -> 69.5 us, with an expert of half the tokens among them
    // 90.7 -> 78.3 us).
    const int stages = most <= 128 ? 8 : most <= PN ? 6 : 4, stage_bytes = T_RING_BYTES / stages;
    order_experts(pl, g.E, [&](int cnt) { return cnt > 0 ? tile_tokens(cnt, most, 32) : 0; });
    count_units(pl, g.E, [&](int cnt) { return cnt > 0 ? quot_up(cnt, tile_tokens(cnt, most, 32)) * ((g.M + PM - 1) / PM) : 0; });
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
            uint32_t issued = 0;                  // a bit a stage
            uint32_t issued_parity = 0;
            bool ok = true;
            for (int i = 0; i * workers < total_units && ok; ++i) {
                const int u = unit_of(i, worker, workers);
                if (u >= total_units) break;
                const PUnit x = pair_unit(pl, g, most, u);
                const int m = x.m0 + (int)crank * 128;
                const int ta = x.t0 + (int)crank * (x.n0 / 2), tb = x.t0 + x.n0 + (int)crank * (x.n1 / 2);
                // this CTA's half of a half's tokens, in quarters of 32 rows
                const int rows0 = (x.n0 / 2 + 31) / 32, rows1 = (x.n1 / 2 + 31) / 32;
                const uint32_t bytes = 2 * ((uint32_t)P_HALF_BYTES + (rows0 + rows1) * (P_HALF_BYTES / 4));
                for (int kb = 0; kb < nk; ++kb) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag)) { ok = false; break; }
                    uint8_t *sw = smem + stage * stage_bytes, *sx = sw + P_HALF_BYTES;
                    if (leader) mbar_arrive_expect_tx(&full_bar[stage], bytes);
                    if (TRANS) {
                        tma_load_3d_pair(sw, &g.tm_w, &full_bar[stage], m, kb * GK, x.e);
                        tma_load_3d_pair(sw + G_BOX_BYTES, &g.tm_w, &full_bar[stage], m + 64, kb * GK, x.e);
                    } else {
                        tma_load_3d_pair(sw, &g.tm_w, &full_bar[stage], kb * GK, m, x.e);
                    }
                    tma_load_2d_pair(sx, &g.tm_t[rows0 - 1], &full_bar[stage], kb * GK, ta);
                    if (x.n1) tma_load_2d_pair(sx + P_HALF_BYTES, &g.tm_t[rows1 - 1], &full_bar[stage], kb * GK, tb);
                    issued |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | phase << stage;
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
            }
            griddep_launch_dependents();        // the next launch may take what room is left
            {   // the MMA issuer commits drain_bar once it has finished or given up
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            }
            if ((!ok || abort_flag) && leader) {  // both CTAs' loads complete on the leader's barriers
                for (int s = 0; s < stages; ++s) {
                    if (!(issued >> s & 1u)) continue;
                    const uint64_t t0 = globaltimer_ns();
                    while (!mbar_try_wait(&full_bar[s], issued_parity >> s & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {}
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        if (leader) {
            int stage = 0;
            uint32_t phase = 0, half_phase = 0;   // half_phase: a bit an accumulator, flipped by each use of it
            int turn = 0;
            bool ok = true;
            const uint32_t s0 = smem_u32(smem);
            const uint64_t w0 = TRANS ? mnmajor(s0) : kmajor(s0), x0 = kmajor(s0 + P_HALF_BYTES);
            // one half's MMAs of a stage: 16 of K are 32 bytes of a K-major row, or 16 rows of 128 bytes
            auto half_stage = [&](int h, int acc, int st, uint32_t id, bool first, bool last, bool release) {
                const uint64_t dw = w0 + (uint64_t)(st * (stage_bytes >> 4));
                const uint64_t dx = x0 + (uint64_t)(st * (stage_bytes >> 4) + h * (P_HALF_BYTES >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < GK / G_UMMA_K; ++k)
                        mma_bf16_pair(tmem_base + acc * PN, dw + k * (TRANS ? 128 : 2), dx + k * 2, id, !first || k != 0);
                    if (last) mma_commit_pair(&tfull_bar[acc], 3);
                    if (release) mma_commit_pair(&empty_bar[st], 3);
                }
                __syncwarp();
            };
            for (int i = 0; i * workers < total_units && ok; ++i) {
                const int u = unit_of(i, worker, workers);
                if (u >= total_units) break;
                const PUnit x = pair_unit(pl, g, most, u);
                const uint32_t id0 = idesc(g.type, TRANS, false, x.n0, PM), id1 = idesc(g.type, TRANS, false, x.n1, PM);
                const int acc = accumulator_of(x, turn);
                ok = __all_sync(0xffffffffu, mbar_wait(&tempty_bar[acc], (half_phase >> acc & 1u) ^ 1u, &abort_flag));
                if (!ok) break;
                // The first stages of a unit run their first half alone, and then their second: that gives the epilogue
                // the time of T_AHEAD half stages to drain the second half of the unit before.
                const int ahead = x.n1 ? min(T_AHEAD, nk) : 0;
                int kb = 0;
                for (; kb < ahead && ok; ++kb) {
                    const int st = stage + kb < stages ? stage + kb : stage + kb - stages;
                    const uint32_t ph = stage + kb < stages ? phase : phase ^ 1u;
                    ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[st], ph, &abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    half_stage(0, 0, st, id0, kb == 0, kb == nk - 1, false);
                }
                if (ok && ahead) ok = __all_sync(0xffffffffu, mbar_wait(&tempty_bar[1], (half_phase >> 1) ^ 1u, &abort_flag));
                if (!ok) break;
                tc_fence_after();
                for (kb = 0; kb < ahead; ++kb) {
                    half_stage(1, 1, stage, id1, kb == 0, kb == nk - 1, true);
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
                for (; kb < nk; ++kb) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, &abort_flag));
                    if (!ok) break;
                    tc_fence_after();
                    half_stage(0, acc, stage, id0, kb == 0, kb == nk - 1, x.n1 == 0);
                    if (x.n1) half_stage(1, 1, stage, id1, false, kb == nk - 1, true);
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
                half_phase ^= x.n1 ? 3u : 1u << acc;
            }
            if (elect_one()) mma_commit_pair(&drain_bar, 3);
            __syncwarp();
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
        }
    } else {
        // --------------------------- epilogue (warps 2..9) ---------------------------
        const int quad = warp & 3;              // TMEM lanes 32*quad .. 32*quad+31
        const int part = (warp - 2) >> 2;       // each has half of a half's columns
        uint8_t *s_out = smem + T_RING_BYTES + part * T_OUT_BYTES;
        uint32_t half_phase = 0;
        int turn = 0;
        bool ready = true;
        for (int i = 0; i * workers < total_units && ready; ++i) {
            const int u = unit_of(i, worker, workers);
            if (u >= total_units) break;
            const PUnit x = pair_unit(pl, g, most, u);
            const int m = x.m0 + (int)crank * 128, bytes = 2 * min(128, g.M - m);
            const int first = accumulator_of(x, turn);
            for (int h = 0; h < (x.n1 ? 2 : 1); ++h) {
                const int acc = h + first;
                ready = mbar_wait(&tfull_bar[acc], half_phase >> acc & 1u, &abort_flag);
                ready = bar_all(1 + part, 128, ready);       // the part's warps go on together or not at all
                if (!ready) break;
                tc_fence_after();
                // all of this warp's columns, packed, into registers, so that the MMAs get the accumulator back at once
                const int n = h ? x.n1 : x.n0, c0 = part * ((n / 2 + 31) & ~31), cols = part ? n - c0 : min(n, (n / 2 + 31) & ~31);
                const uint32_t t_row = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(acc * PN + c0);
                uint32_t w[4][16];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q * 32 < cols) {
                        uint32_t v[32];
                        tmem_ld_32x32b_x32(t_row + q * 32, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[q][j] = pack2(v[2 * j], v[2 * j + 1], g.type);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(&tempty_bar[acc]);
                    else mbar_arrive_remote(&tempty_bar[acc], 0);
                }
                // Out through shared memory, 16 tokens at a time in two places in turn: the part's four warps lay down each
                // token's 128 features, 64 bytes a warp, neighbour lanes trading halves so that a lane has two features of a
                // token. 16 tokens leave as one box; at a tile's ragged end, each by its own bulk copy of a row. (8 experts of
                // 4096 x 256, 1,600 tokens each: 52 us; 63 with a copy a row, 32 tokens in one place.)
                const int t0 = h * PN + c0;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    if (q * 16 >= cols) break;
                    bulk_wait_read<1>();          // cols is a multiple of 32: the places take turns from half to half too
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory");
                    uint8_t *box = s_out + (q & 1) * (T_OUT_BYTES / 2);
                    uint32_t *slot = reinterpret_cast<uint32_t *>(box) + quad * 16 + (lane >> 1);
                    const bool odd = lane & 1;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t mine = w[q / 2][(q & 1) * 8 + j], other = __shfl_xor_sync(0xffffffffu, mine, 1);
                        slot[(2 * j + odd) * 64] = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
                    }
                    fence_proxy_async_smem();
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory");
                    const int row = quad * 4 + lane, t = t0 + q * 16 + row;
                    if (t0 + q * 16 + 16 <= x.n) {
                        if (quad == 0 && lane == 0 && bytes > 0) tma_store_2d(&g.tm_y, box, m, x.t0 + t0 + q * 16);
                    } else if (lane < 4 && t < x.n && bytes > 0) {
                        bulk_store(static_cast<uint16_t *>(g.out) + (int64_t)(x.t0 + t) * g.ld_out + m, box + row * 256, bytes);
                    }
                    bulk_commit();
                }
            }
            half_phase ^= x.n1 ? 3u : 1u << first;
        }
        bulk_wait_all();
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
// forward and dx, few tokens to an expert: single CTAs, two to an SM
//
// The time is that of the weights' way in, so what counts is that all SMs ask for them at once, early and without a
// pause: each CTA loads its next unit's weights while it multiplies and stores the one before. With few units, a unit is
// 128 / S accumulator rows and S slices of K: the M operand holds the same weight rows S times, slice j of K in rows
// j * 128 / S .., the N operand the tokens S times, slice j in columns j * nb ... The products of one slice with itself
// are the partial sums wanted; those of different slices are not read. S times the units, a S-th of the steps, and no
// exchange between CTAs. Where that still leaves most SMs without work, the slices of a unit lie in the CTAs of a cluster,
// S in each; every CTA adds up its own and then, out of the others' shared memory, its share of the unit's results. (In
// clusters alone, without the slices, a call with more units took 63 us where one slice took 27: 16 experts, 777 tokens,
// 2056 x 1416.)
// ------------------------------------------------------------------------------------------------

struct SUnit {
    int e, mt, t0, n;          // expert, tile of accumulator rows, first token, tokens; n = 0: no such unit
};

// Unit u of a call that has a unit to a CTA at most, found by each warp on its own (32 experts at a time): the experts
// are not ordered, and nothing is counted ahead.
__device__ __forceinline__ SUnit scan_unit(const int *off, int E, int nb, int u, int m_tiles)
{
    const int lane = threadIdx.x & 31;
    SUnit x;
    x.e = x.mt = x.t0 = x.n = 0;
    int run = 0;
    for (int base = 0; base < E && x.n == 0; base += 32) {
        const int e = base + lane;
        const int o0 = e < E ? off[e] : 0, cnt = e < E ? off[e + 1] - o0 : 0;
        const int tile = cnt ? tile_tokens(cnt, nb, 16) : 16, tiles = cnt ? quot_up(cnt, tile) : 0;
        const int units = tiles * m_tiles, inc = warp_inclusive_scan(units);
        const uint32_t past = __ballot_sync(0xffffffffu, run + inc > u);
        if (past) {
            const int l = __ffs(past) - 1;                   // the first expert whose units end behind u
            const int before = run + __shfl_sync(0xffffffffu, inc - units, l);
            const int first = __shfl_sync(0xffffffffu, o0, l), c = __shfl_sync(0xffffffffu, cnt, l);
            const int tl = __shfl_sync(0xffffffffu, tile, l), nt = __shfl_sync(0xffffffffu, tiles, l);
            x.e = base + l;
            x.mt = quot(u - before, nt);                     // the tiles of one weight tile adjoin
            const int t = u - before - x.mt * nt;
            x.t0 = first + t * tl;
            x.n = min(tl, c - t * tl);
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
    }
    return x;
}

// The same from the plan.
__device__ __forceinline__ SUnit plan_unit(const Plan &pl, int E, int nb, int u)
{
    SUnit x;
    const int place = find_place(pl, E, u);
    x.e = pl.order[place];
    const int cnt = pl.off[x.e + 1] - pl.off[x.e];
    const int tile = tile_tokens(cnt, nb, 16), nt = quot_up(cnt, tile);
    x.mt = quot(u - pl.pre[place], nt);
    const int t = u - pl.pre[place] - x.mt * nt;
    x.t0 = pl.off[x.e] + t * tile;
    x.n = min(tile, cnt - t * tile);
    return x;
}

// The sums of a cluster that are not numbers: right, unless one of its CTAs gave up.
template <int ROWS>
__device__ __noinline__ void store_odd(const GArgs &g, const volatile int *abort, uint32_t part, int mt, int t0, int n, int rank, int split)
{
    if (cluster_gave_up(abort, split)) return;
    for (int i = rank * S_THREADS + threadIdx.x; i < n * (ROWS / 2); i += split * S_THREADS) {
        const int t = i / (ROWS / 2), row = 2 * (i - t * (ROWS / 2)), m0 = mt * ROWS;
        float2 s = make_float2(0.0f, 0.0f);
        for (int c = 0; c < split; ++c) {
            const float2 a = ld_cluster_f32x2(part + (t * ROWS + row) * 4, c);
            s.x = __fadd_rn(s.x, a.x);
            s.y = __fadd_rn(s.y, a.y);
        }
        if (s.x != s.x && m0 + row < g.M)
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(g.out) + (int64_t)(t0 + t) * g.ld_out + m0 + row) =
                pack2(__float_as_uint(s.x), __float_as_uint(s.y), g.type);
    }
}

// ROUNDS: a CTA may have several units.
template <bool TRANS, int S, bool ROUNDS>
__global__ void __launch_bounds__(S_THREADS)
grouped_small_kernel(const __grid_constant__ GArgs g, uint32_t *status)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_bar[S_MAX_STAGES], empty_bar[S_MAX_STAGES], tfull_bar[2], tempty_bar[2], drain_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_flag;
    __shared__ Plan pl;

    constexpr int ROWS = SM_ROWS / S;           // accumulator rows of a unit
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nb = g.nb, stages = g.stages;
    const int buf_cols = S * nb;                // an accumulator; two where a CTA has several units
    const int tmem_cols = max(32, ROUNDS ? 2 * buf_cols : buf_cols);

    if (warp == 0 && lane == 0) {
        prefetch_tmap(&g.tm_w);
        for (int b = 0; 16 << b <= g.nb; ++b) prefetch_tmap(&g.tm_t[b]);
        abort_flag = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full_bar[s], stage_arrivals(g, s));
            mbar_init(&empty_bar[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull_bar[a], 1);
            mbar_init(&tempty_bar[a], S_EPI_WARPS);
        }
        mbar_init(&drain_bar, 1);
        fence_mbarrier_init();
    }
    if (warp == 1) tmem_alloc(&tmem_base_s, (uint32_t)tmem_cols);
    griddep_wait();                             // what the launches before this one wrote is there from here on
    tc_fence_before();
    const bool valid = load_offsets(pl, g.offsets, g.E, g.T);
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_s;
    const int m_tiles = (g.M + ROWS - 1) / ROWS;
    if (ROUNDS && valid) {
        order_experts(pl, g.E, [](int cnt) { return cnt; });
        count_units(pl, g.E, [&](int cnt) { return cnt > 0 ? quot_up(cnt, tile_tokens(cnt, nb, 16)) * m_tiles : 0; });
    }
    const int split = S > 1 ? g.split : 1, rank = S > 1 && split > 1 ? (int)cluster_ctarank() : 0;
    // steps of each slice (the last slices' may lie behind K: zeros)
    const int nk = ((g.K + GK - 1) / GK + S * split - 1) / (S * split);
    const int stage_bytes = S_W_BYTES + S * nb * GK * 2;
    // this CTA's i-th unit
    SUnit only;
    only.n = 0;
    if (!ROUNDS && valid) only = scan_unit(pl.off, g.E, nb, split > 1 ? blockIdx.x / split : blockIdx.x, m_tiles);
    auto unit = [&](int i) {
        SUnit x;
        x.n = 0;
        if (!ROUNDS) return i == 0 ? only : x;
        const int u = blockIdx.x + i * gridDim.x;
        return valid && u < pl.pre[g.E] ? plan_unit(pl, g.E, nb, u) : x;
    };

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        int stage = 0, sent = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int r = 0; ok; ++r) {
            const SUnit x = unit(r);
            if (x.n == 0) break;
            if (lane == 0) {
                const int m0 = x.mt * ROWS, high = x.n <= 16 ? 0 : x.n <= 32 ? 1 : x.n <= 64 ? 2 : 3;       // its token box
                const uint32_t bytes = S_W_BYTES + S * (16 << high) * GK * 2;
                for (int i = 0; i < nk; ++i) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag)) { ok = false; break; }
                    uint8_t *sw = smem + stage * stage_bytes, *sx = sw + S_W_BYTES;
                    mbar_arrive_expect_tx(&full_bar[stage], bytes);
#pragma unroll
                    for (int j = 0; j < S; ++j) {
                        const int k = ((rank * S + j) * nk + i) * GK;
                        if (TRANS && S == 1) {
                            tma_load_3d(sw, &g.tm_w, &full_bar[stage], m0, k, x.e);
                            tma_load_3d(sw + G_BOX_BYTES, &g.tm_w, &full_bar[stage], m0 + 64, k, x.e);
                        } else if (TRANS) {
                            tma_load_3d(sw + j * (S_W_BYTES / S), &g.tm_w, &full_bar[stage], m0, k, x.e);
                        } else {
                            tma_load_3d(sw + j * (S_W_BYTES / S), &g.tm_w, &full_bar[stage], k, m0, x.e);
                        }
                        tma_load_2d(sx + j * nb * GK * 2, &g.tm_t[high], &full_bar[stage], k, x.t0);
                    }
                    ++sent;
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
        if (lane == 0) {
            // The launch behind this one may take what room is left: now, when this CTA's time is nearly up (any sooner, its
            // CTAs crowd the SMs that this launch left room on: 8 experts of 1024 x 1024, 512 tokens: 11.1 us against 9.4).
            griddep_launch_dependents();
            const uint64_t begin = globaltimer_ns();
            while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - begin < kWaitLimitNs) {}
            if (abort_flag) {                   // drain what was sent before the shared memory goes away
                for (int s = 0; s < stages && s < sent; ++s) {
                    const int last = (sent - 1 - s) / stages;        // the slot's last use
                    const uint64_t from = globaltimer_ns();
                    while (!mbar_try_wait(&full_bar[s], (uint32_t)(last & 1)) && globaltimer_ns() - from < kWaitLimitNs) {}
                }
                if (S > 1) leave_nan(smem, only.n * ROWS, 0, 1);
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = true;
        const uint32_t s0 = smem_u32(smem);
        // M-major weights of four slices lie in 32-column boxes with 64-byte rows, otherwise in 64-column boxes
        const uint64_t w0 = !TRANS ? kmajor(s0) : S == 4 ? mnmajor64(s0) : mnmajor(s0), x0 = kmajor(s0 + S_W_BYTES);
        for (int r = 0; ok; ++r) {
            const SUnit x = unit(r);
            if (x.n == 0) break;
            const uint32_t id = idesc(g.type, TRANS, false, S == 1 ? (x.n + 15) & ~15 : S * nb, SM_ROWS);
            const uint32_t d_tmem = tmem_base + (uint32_t)(buf * buf_cols);
            ok = __all_sync(0xffffffffu, mbar_wait(&tempty_bar[buf], buf_phase ^ 1u, &abort_flag));
            if (!ok) break;
            for (int i = 0; i < nk; ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, &abort_flag));
                if (!ok) break;
                tc_fence_after();
                const uint64_t dw = w0 + (uint64_t)(stage * (stage_bytes >> 4)), dx = x0 + (uint64_t)(stage * (stage_bytes >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < GK / G_UMMA_K; ++k)
                        mma_bf16(d_tmem, dw + k * (!TRANS ? 2 : S == 4 ? 64 : 128), dx + k * 2, id, (i | k) != 0);
                    mma_commit(&empty_bar[stage]);
                    if (i == nk - 1) mma_commit(&tfull_bar[buf]);
                }
                __syncwarp();
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
        }
        if (elect_one()) mma_commit(&drain_bar);
        __syncwarp();
        const uint64_t begin = globaltimer_ns();
        while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - begin < kWaitLimitNs) {}
    } else {
        // --------------------------- epilogue (warps 2..5) ---------------------------
        const int quad = warp & 3;              // accumulator rows 32*quad .. 32*quad+31
        const int slice = quad * S / 4;         // the slice they belong to
        int buf = 0;
        uint32_t buf_phase = 0;
        for (int r = 0;; ++r) {
            const SUnit x = unit(r);
            if (x.n == 0) break;
            const int m0 = x.mt * ROWS;
            bool ready = mbar_wait(&tfull_bar[buf], buf_phase, &abort_flag);
            ready = bar_all(1, 32 * S_EPI_WARPS, ready);     // the four warps go on together or not at all
            if (!ready) {
                if (S > 1) leave_nan(smem, x.n * ROWS, tid - 64, 32 * S_EPI_WARPS);    // and the producer, when its loads are in
                break;
            }
            tc_fence_after();
            uint16_t *out = static_cast<uint16_t *>(g.out) + (int64_t)x.t0 * g.ld_out;
            const uint32_t t_row = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * buf_cols + slice * nb);
            float *part = reinterpret_cast<float *>(smem);    // S > 1, [slice][token][row]: the stages are free, it is the only unit
            for (int c = 0; c < x.n; c += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(t_row + c, v);
                tmem_ld_wait();
                if (S == 1) {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) w[j] = pack2(v[2 * j], v[2 * j + 1], g.type);
                    store_tokens<16>(w, out + (int64_t)c * g.ld_out, g.ld_out, m0 + quad * 32 + lane, g.M, x.n - c);
                } else {
                    float *mine = part + (slice * nb + c) * ROWS + quad * 32 + lane - slice * ROWS;
#pragma unroll
                    for (int j = 0; j < 16; ++j) mine[j * ROWS] = __uint_as_float(v[j]);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty_bar[buf]);
            if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            if (S > 1) {                        // the slices' sums, in their order; two rows of a token to a thread
                bar_all(1, 32 * S_EPI_WARPS, true);
                for (int i = tid - 64; i < x.n * (ROWS / 2); i += 32 * S_EPI_WARPS) {
                    const int t = i / (ROWS / 2), row = 2 * (i - t * (ROWS / 2));
                    float2 s = *reinterpret_cast<const float2 *>(part + t * ROWS + row);
#pragma unroll
                    for (int j = 1; j < S; ++j) {
                        const float2 a = *reinterpret_cast<const float2 *>(part + (j * nb + t) * ROWS + row);
                        s.x = __fadd_rn(s.x, a.x);
                        s.y = __fadd_rn(s.y, a.y);
                    }
                    if (split > 1)              // to be added up with the other CTAs'
                        *reinterpret_cast<float2 *>(part + t * ROWS + row) = s;
                    else if (m0 + row < g.M)
                        *reinterpret_cast<uint32_t *>(out + (int64_t)t * g.ld_out + m0 + row) =
                            pack2(__float_as_uint(s.x), __float_as_uint(s.y), g.type);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (S > 1 && split > 1) {                  // the CTAs' sums, in their order; each CTA has a share of the unit's results
        cluster_sync();
        const uint32_t part = smem_u32(smem);
        bool odd = false;
        for (int i = rank * S_THREADS + tid; i < only.n * (ROWS / 2); i += split * S_THREADS) {
            const int t = i / (ROWS / 2), row = 2 * (i - t * (ROWS / 2)), m0 = only.mt * ROWS;
            float2 s = make_float2(0.0f, 0.0f);
            for (int c = 0; c < split; ++c) {
                const float2 a = ld_cluster_f32x2(part + (t * ROWS + row) * 4, c);
                s.x = __fadd_rn(s.x, a.x);
                s.y = __fadd_rn(s.y, a.y);
            }
            odd |= s.x != s.x;
            if (s.x == s.x && m0 + row < g.M)
                *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(g.out) + (int64_t)(only.t0 + t) * g.ld_out + m0 + row) =
                    pack2(__float_as_uint(s.x), __float_as_uint(s.y), g.type);
        }
        if (odd) store_odd<ROWS>(g, &abort_flag, part, only.mt, only.t0, only.n, rank, split);
        __syncwarp();
        cluster_sync();                         // no CTA leaves while others read its sums
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, (uint32_t)tmem_cols);
    }
    if (tid == 0) {
        if (abort_flag) set_status(status, SF_STATUS_WAIT_TIMEOUT);
        if (!valid && blockIdx.x == 0) set_status(status, SF_STATUS_BAD_OFFSET);
    }
}

// ------------------------------------------------------------------------------------------------
// weight gradient, CTA pairs
// ------------------------------------------------------------------------------------------------

struct WUnit {
    int e, r0, c0, t0, cnt;    // expert, first row, first column, first token, tokens
    int nk, chunks, per;       // stages of 64 tokens, accumulation chunks, stages to a chunk
};

// Experts in the order of their numbers, or of `order` (falling stage counts) where there is one.
struct WPlan {
    uint16_t order[kSortE];
};

__device__ __forceinline__ WUnit dw_unit(const WPlan &pl, const GArgs &g, int u)
{
    const int n_tiles = (g.K + PN - 1) / PN, per = (g.M + PM - 1) / PM * n_tiles;
    WUnit x;
    const int place = quot(u, per), local = u - place * per, mt = quot(local, n_tiles);
    x.e = g.E <= kSortE ? pl.order[place] : place;
    x.r0 = mt * PM;
    x.c0 = (local - mt * n_tiles) * PN;
    x.t0 = __ldg(g.offsets + x.e);
    x.cnt = __ldg(g.offsets + x.e + 1) - x.t0;
    x.nk = (x.cnt + GK - 1) / GK;
    x.chunks = quot_up(x.nk, W_CHUNK_STAGES);
    x.per = x.chunks ? quot_up(x.nk, x.chunks) : 0;
    return x;
}

__device__ __forceinline__ bool has_tail(const WUnit &x) { return (x.cnt & (G_UMMA_K - 1)) != 0; }

// A pair sums 256 x 256 of W[e] over chunks of 960 tokens at most, in two accumulators in turn; the epilogue warps add the
// chunks' sums in registers. What bounds it is the traffic between L2 and the SMs: 64 KB a stage and pair, 10.3 TB/s into
// the SMs and 12.9 TB/s in all with the tensor cores 72% active (4 experts of 4096 x 4096 over 2,048 tokens each; the
// forward kernel's 512-column tiles take a quarter less and keep them 82% active). Wider tiles have no place for the sums:
// 256 x 512 of fp32 are an SM pair's whole register files.
// OLD: for gradients that are added to, over few tokens. What W holds comes into the output boxes by TMA while the MMAs
// run, is added there and goes out by TMA: the time is that of reading and writing W once, with fewer stages for the
// tokens and a place for all of a warp's boxes. Otherwise the addition is TMA's, at 2.4 TB/s of results.
// FEW: the same division of the shared memory for few tokens without OLD, where a unit's time is that of its way out.
template <bool OLD, bool FEW>
__global__ void __launch_bounds__(W_THREADS, 1)
grouped_dw_kernel(const __grid_constant__ GArgs g, uint32_t *status)
{
    static_assert(FEW || !OLD, "what W holds takes all of a warp's boxes");
    constexpr int W_STAGES = FEW ? W_STAGES_FEW : W_STAGES_NEW;
    constexpr int BOXES = FEW ? 4 : 1;          // output boxes of a warp in shared memory
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_bar[W_STAGES], empty_bar[W_STAGES], tfull_bar[2], tempty_bar[2], drain_bar;
    __shared__ uint64_t tail_bar[W_STAGES], clear_bar[W_STAGES];   // for the last stage of an expert, where rows are cleared
    __shared__ uint64_t old_bar[P_EPI_WARPS];   // OLD: what W holds has landed, by warp
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_flag;
    __shared__ WPlan pl;
    __shared__ int warp_busy[W_THREADS / 32];

    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = cluster_ctarank();
    const bool leader = crank == 0;
    const int worker = blockIdx.x / 2, workers = gridDim.x / 2;

    if (tid == 0) {
        abort_flag = 0;
        for (int s = 0; s < W_STAGES; ++s) {
            mbar_init(&full_bar[s], stage_arrivals(g, s));
            mbar_init(&empty_bar[s], 1);
            mbar_init(&tail_bar[s], stage_arrivals(g, s));      // this CTA's loads of the stage have landed
            mbar_init(&clear_bar[s], 2);          // the leader's: both CTAs have cleared their rows
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull_bar[a], 1);
            mbar_init(&tempty_bar[a], P_EPI_WARPS * 2);
        }
        mbar_init(&drain_bar, 1);
        for (int w = 0; w < P_EPI_WARPS; ++w) mbar_init(&old_bar[w], 1);
        fence_mbarrier_init();
        prefetch_tmap(&g.tm_w);
        prefetch_tmap(&g.tm_x);
        prefetch_tmap(&g.tm_out);
    }
    griddep_wait();                             // what the launches before this one wrote is there from here on
    int busy = 0;                               // experts with tokens
    {   // offsets: valid, and the experts' order
        int bad = 0, some = 0;
        int *keys = reinterpret_cast<int *>(smem);                  // before the stages are used
        for (int e = tid; e < g.E; e += W_THREADS) {
            const int o0 = g.offsets[e], o1 = g.offsets[e + 1];
            if (o0 < 0 || o1 < o0 || o1 > g.T) bad = 1;
            some += o1 > o0;
            if (g.E <= kSortE) keys[e] = (o1 - o0 + GK - 1) / GK;
        }
        some = __reduce_add_sync(0xffffffffu, some);
        if (lane == 0) warp_busy[warp] = some;
        if (__syncthreads_or(bad)) {
            if (blockIdx.x == 0 && tid == 0) set_status(status, SF_STATUS_BAD_OFFSET);
            return;
        }
        for (int w = 0; w < W_THREADS / 32; ++w) busy += warp_busy[w];
        if (g.E <= kSortE)
            for (int e = tid; e < g.E; e += W_THREADS) {
                const int mine = keys[e];
                int rank = 0;
                for (int k = 0; k < g.E; ++k) rank += keys[k] > mine || (keys[k] == mine && k < e);
                pl.order[rank] = (uint16_t)e;
            }
        __syncthreads();
        fence_proxy_async_smem();                                   // the stages are written by TMA from here on
    }
    if (warp == 1) tmem_alloc_pair(&tmem_base_s, P_TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_s;
    // experts without tokens are the last in the order; a gradient that is added to has nothing to do for them
    const int places = g.accumulate && g.E <= kSortE ? busy : g.E;
    const int total_units = places * ((g.M + PM - 1) / PM) * ((g.K + PN - 1) / PN);

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0;
            bool issued[W_STAGES] = {};
            uint32_t issued_parity[W_STAGES] = {};
            uint32_t tails = 0, tail_parity = 0;  // by stage: whether it held a tail, and the parity of its last one
            bool ok = true;
            for (int i = 0; i * workers < total_units && ok; ++i) {
                const int u = unit_of(i, worker, workers);
                if (u >= total_units) break;
                const WUnit x = dw_unit(pl, g, u);
                const int r = x.r0 + (int)crank * 128, c = x.c0 + (int)crank * 128;
                for (int kb = 0; kb < x.nk; ++kb) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag)) { ok = false; break; }
                    uint8_t *sy = smem + stage * W_STAGE_BYTES, *sa = sy + P_HALF_BYTES;
                    const int t = x.t0 + kb * GK;
                    if (kb == x.nk - 1 && has_tail(x)) {
                        // rows to clear: each CTA's loads complete on its own barrier, for the warp that clears them
                        if (leader) mbar_arrive(&full_bar[stage]);
                        mbar_arrive_expect_tx(&tail_bar[stage], W_STAGE_BYTES);
                        tma_load_2d(sy, &g.tm_x, &tail_bar[stage], r, t);
                        tma_load_2d(sy + G_BOX_BYTES, &g.tm_x, &tail_bar[stage], r + 64, t);
                        tma_load_2d(sa, &g.tm_w, &tail_bar[stage], c, t);
                        tma_load_2d(sa + G_BOX_BYTES, &g.tm_w, &tail_bar[stage], c + 64, t);
                        if (tails >> stage & 1u) tail_parity ^= 1u << stage;
                        tails |= 1u << stage;
                    } else {
                        if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * W_STAGE_BYTES);
                        if (g.whole & 1) {
                            tma_load_3d_pair(sy, &g.tm_t[0], &full_bar[stage], 0, t, r / 64);
                        } else {
                            tma_load_2d_pair(sy, &g.tm_x, &full_bar[stage], r, t);
                            tma_load_2d_pair(sy + G_BOX_BYTES, &g.tm_x, &full_bar[stage], r + 64, t);
                        }
                        if (g.whole & 2) {
                            tma_load_3d_pair(sa, &g.tm_t[1], &full_bar[stage], 0, t, c / 64);
                        } else {
                            tma_load_2d_pair(sa, &g.tm_w, &full_bar[stage], c, t);
                            tma_load_2d_pair(sa + G_BOX_BYTES, &g.tm_w, &full_bar[stage], c + 64, t);
                        }
                    }
                    issued[stage] = true;
                    issued_parity[stage] = phase;
                    if (++stage == W_STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            griddep_launch_dependents();
            {
                const uint64_t t0 = globaltimer_ns();
                while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
            }
            if (!ok || abort_flag) {
                if (leader) {
                    for (int s = 0; s < W_STAGES; ++s) {
                        if (!issued[s]) continue;
                        const uint64_t t0 = globaltimer_ns();
                        while (!mbar_try_wait(&full_bar[s], issued_parity[s]) && globaltimer_ns() - t0 < kWaitLimitNs) {}
                    }
                }
                for (int s = 0; s < W_STAGES; ++s) {
                    if (!(tails >> s & 1u)) continue;
                    const uint64_t t0 = globaltimer_ns();
                    while (!mbar_try_wait(&tail_bar[s], tail_parity >> s & 1u) && globaltimer_ns() - t0 < kWaitLimitNs) {}
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        if (leader) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0, clear_phase = 0;    // clear_phase: a bit a stage
            bool ok = true;
            const uint32_t s0 = smem_u32(smem);
            const uint64_t y0 = mnmajor(s0), a0 = mnmajor(s0 + P_HALF_BYTES);
            const uint32_t id = idesc(g.type, true, true, PN, PM);
            for (int i = 0; i * workers < total_units && ok; ++i) {
                const int u = unit_of(i, worker, workers);
                if (u >= total_units) break;
                const WUnit x = dw_unit(pl, g, u);
                for (int ch = 0, kb = 0; ch < x.chunks && ok; ++ch) {
                    const int end = min(x.nk, kb + x.per);
                    const uint32_t d_tmem = tmem_base + (uint32_t)(buf * PN);
                    ok = __all_sync(0xffffffffu, mbar_wait(&tempty_bar[buf], buf_phase ^ 1u, &abort_flag));
                    if (!ok) break;
                    for (bool first = true; kb < end; ++kb, first = false) {
                        const bool tail = kb == x.nk - 1 && has_tail(x);
                        bool there = mbar_wait(&full_bar[stage], phase, &abort_flag);
                        if (there && tail) there = mbar_wait_cluster(&clear_bar[stage], clear_phase >> stage & 1u, &abort_flag);
                        ok = __all_sync(0xffffffffu, there);
                        if (!ok) break;
                        if (tail) clear_phase ^= 1u << stage;
                        tc_fence_after();
                        const uint64_t dy = y0 + (uint64_t)(stage * (W_STAGE_BYTES >> 4));
                        const uint64_t da = a0 + (uint64_t)(stage * (W_STAGE_BYTES >> 4));
                        const int rest = x.cnt - kb * GK;
                        if (elect_one()) {
                            if (rest >= GK) {
#pragma unroll
                                for (int k = 0; k < GK / G_UMMA_K; ++k)
                                    mma_bf16_pair(d_tmem, dy + k * 128, da + k * 128, id, !first || k != 0);
                            } else {
                                for (int k = 0; k * G_UMMA_K < rest; ++k)
                                    mma_bf16_pair(d_tmem, dy + k * 128, da + k * 128, id, !first || k != 0);
                            }
                            mma_commit_pair(&empty_bar[stage], 3);
                            if (kb == end - 1) mma_commit_pair(&tfull_bar[buf], 3);
                        }
                        __syncwarp();
                        if (++stage == W_STAGES) { stage = 0; phase ^= 1u; }
                    }
                    if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
                }
            }
            if (elect_one()) mma_commit_pair(&drain_bar, 3);
            __syncwarp();
            const uint64_t t0 = globaltimer_ns();
            while (!mbar_try_wait(&drain_bar, 0) && globaltimer_ns() - t0 < kWaitLimitNs) {}
        }
    } else if (warp == 2 + P_EPI_WARPS) {
        // ---------------- clears the rows behind an expert's end, in this CTA's part of the stage ----------------
        int stage = 0;
        uint32_t tail_phase = 0;                // a bit a stage
        for (int i = 0; i * workers < total_units; ++i) {
            const int u = unit_of(i, worker, workers);
            if (u >= total_units) break;
            const WUnit x = dw_unit(pl, g, u);
            if (has_tail(x)) {
                const int st = (stage + x.nk - 1) % W_STAGES;
                if (!__all_sync(0xffffffffu, mbar_wait(&tail_bar[st], tail_phase >> st & 1u, &abort_flag))) break;
                tail_phase ^= 1u << st;
                const int from = x.cnt - (x.nk - 1) * GK, upto = (from + G_UMMA_K - 1) & ~(G_UMMA_K - 1);
                uint8_t *sy = smem + st * W_STAGE_BYTES;
                // a token is one 128-byte row of each of the stage's boxes
                for (int j = lane; j < (upto - from) * 8; j += 32)
#pragma unroll
                    for (int q = 0; q < W_STAGE_BYTES / G_BOX_BYTES; ++q)
                        *reinterpret_cast<uint4 *>(sy + q * G_BOX_BYTES + (from + (j >> 3)) * 128 + (j & 7) * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (leader) mbar_arrive(&clear_bar[st]);
                    else mbar_arrive_remote(&clear_bar[st], 0);
                }
            }
            stage = (stage + x.nk) % W_STAGES;
        }
    } else {
        // --------------------------- epilogue (warps 2..9) ---------------------------
        const int quad = warp & 3;              // accumulator rows 32*quad .. 32*quad+31 of the CTA
        const int part = (warp - 2) >> 2;       // columns part*128 .. +127
        uint8_t *s_warp = smem + W_STAGES * W_STAGE_BYTES + (warp - 2) * BOXES * W_OUT_BYTES;
        int buf = 0;
        uint32_t buf_phase = 0, old_phase = 0;
        for (int i = 0; i * workers < total_units; ++i) {
            const int u = unit_of(i, worker, workers);
            if (u >= total_units) break;
            const WUnit x = dw_unit(pl, g, u);
            if (x.nk == 0 && g.accumulate) continue;
            const int row0 = x.r0 + (int)crank * 128 + quad * 32, c0 = x.c0 + part * 128;
            const int boxes = row0 < g.M ? min(4, (g.K - c0 + 31) / 32) : 0;     // of 32 x 32 that W has here
            if (OLD && boxes > 0 && lane == 0) {
                bulk_wait_read<0>();
                mbar_arrive_expect_tx(&old_bar[warp - 2], boxes * W_OUT_BYTES);
                for (int q = 0; q < boxes; ++q)
                    tma_load_3d(s_warp + q * W_OUT_BYTES, &g.tm_out, &old_bar[warp - 2], c0 + q * 32, row0, x.e);
            }
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.0f;
            bool ready = true;
            for (int ch = 0; ch < x.chunks; ++ch) {
                ready = __all_sync(0xffffffffu, mbar_wait(&tfull_bar[buf], buf_phase, &abort_flag));
                if (!ready) break;
                tc_fence_after();
                const uint32_t t_row = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(buf * PN + part * 128);
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
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            }
            if (OLD && boxes > 0) {             // also where the MMAs gave up: these loads end in this shared memory
                const uint64_t from = globaltimer_ns();
                bool there = mbar_try_wait(&old_bar[warp - 2], old_phase);
                while (!there && globaltimer_ns() - from < kWaitLimitNs) there = mbar_try_wait(&old_bar[warp - 2], old_phase);
                if (!there) abort_flag = 1;
                ready = __all_sync(0xffffffffu, there) && ready;
                old_phase ^= 1u;
            }
            if (!ready) break;
            if (boxes <= 0) continue;
            // Out through shared memory, a box of 32 rows x 128 bytes at a time (16-byte units swizzled by row, as
            // the tensor map has it): what lies outside W the store leaves out.
            if (g.out_f32) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (q >= boxes) break;
                    uint8_t *s_out = s_warp + (FEW ? q * W_OUT_BYTES : 0);
                    float4 *slot = reinterpret_cast<float4 *>(s_out) + lane * 8;
                    if (!FEW || (!OLD && q == 0)) {
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float4 v = make_float4(acc[q * 32 + 4 * j], acc[q * 32 + 4 * j + 1], acc[q * 32 + 4 * j + 2], acc[q * 32 + 4 * j + 3]);
                        if (OLD) {
                            const float4 o = slot[j ^ (lane & 7)];
                            v = make_float4(__fadd_rn(o.x, v.x), __fadd_rn(o.y, v.y), __fadd_rn(o.z, v.z), __fadd_rn(o.w, v.w));
                        }
                        slot[j ^ (lane & 7)] = v;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        if (!OLD && g.accumulate) tma_add_3d(&g.tm_out, s_out, c0 + q * 32, row0, x.e);
                        else tma_store_3d(&g.tm_out, s_out, c0 + q * 32, row0, x.e);
                        bulk_commit();
                    }
                }
            } else if (!OLD) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (2 * q >= boxes) break;
                    uint8_t *s_out = s_warp + (FEW ? q * W_OUT_BYTES : 0);
                    uint4 *slot = reinterpret_cast<uint4 *>(s_out) + lane * 8;
                    if (!FEW || q == 0) {
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            w[k] = pack2(__float_as_uint(acc[q * 64 + 8 * j + 2 * k]), __float_as_uint(acc[q * 64 + 8 * j + 2 * k + 1]), g.type);
                        slot[j ^ (lane & 7)] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&g.tm_out, s_out, c0 + q * 64, row0, x.e);
                        bulk_commit();
                    }
                }
            }
        }
        if (lane == 0) bulk_wait_all();
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

// ------------------------------------------------------------------------------------------------
// weight gradient, few tokens to an expert or few tiles: a unit to a CTA, two CTAs to an SM
// ------------------------------------------------------------------------------------------------

// Adds a box of 32 rows x 128 bytes, laid down by its warp (lane = row, 16-byte units swizzled by row), to what W holds,
// four rows of 128 bytes at a time, so that each access is whole lines. (TMA's addition moves 2.4 TB/s of results where
// this moves 3.4: both read and write W.)
__device__ __forceinline__ void add_box(const uint4 *box, float *dst, int64_t ld, int rows, int cols, int lane)
{
    float4 old[8];
    const int col = (lane & 7) * 4;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + (lane >> 3);
        old[i] = row < rows && col < cols ? *reinterpret_cast<const float4 *>(dst + row * ld + col) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + (lane >> 3);
        const uint4 v = box[row * 8 + ((lane & 7) ^ (row & 7))];
        if (row < rows && col < cols)
            *reinterpret_cast<float4 *>(dst + row * ld + col) =
                make_float4(__fadd_rn(old[i].x, __uint_as_float(v.x)), __fadd_rn(old[i].y, __uint_as_float(v.y)),
                            __fadd_rn(old[i].z, __uint_as_float(v.z)), __fadd_rn(old[i].w, __uint_as_float(v.w)));
    }
}

// Four neighbouring sums into W, or added to what it holds.
__device__ __forceinline__ void put_weights(const GArgs &g, float *w32, uint16_t *w16, int r, int c, float4 s, bool add)
{
    if (g.out_f32) {
        float4 *dst = reinterpret_cast<float4 *>(w32 + r * g.ld_out + c);
        if (add) {
            const float4 o = *dst;
            s = make_float4(__fadd_rn(o.x, s.x), __fadd_rn(o.y, s.y), __fadd_rn(o.z, s.z), __fadd_rn(o.w, s.w));
        }
        *dst = s;
    } else {
        *reinterpret_cast<uint2 *>(w16 + r * g.ld_out + c) =
            make_uint2(pack2(__float_as_uint(s.x), __float_as_uint(s.y), g.type), pack2(__float_as_uint(s.z), __float_as_uint(s.w), g.type));
    }
}

// A unit is 128 / S rows x 256 / S columns of one expert's W and all its tokens, in S slices of tokens as in the small
// forward kernel: slice j in rows j * 128 / S .. of the M operand and columns j * 256 / S .. of the N operand, of whose
// products the S blocks on the diagonal are wanted. While one CTA of an SM waits for its tokens the other writes. As there,
// the slices of few units lie in the CTAs of a cluster, S in each (SPLIT).
template <int S, bool SPLIT>
__global__ void __launch_bounds__(D_THREADS, 2)
grouped_dw_small_kernel(const __grid_constant__ GArgs g, uint32_t *status)
{
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full_bar[D_MAX_STAGES], empty_bar[D_MAX_STAGES], done_bar;
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile int abort_flag;

    constexpr int ROWS = SM_ROWS / S, COLS = PN / S;
    constexpr int PITCH = COLS + 4;             // of the partial sums, in floats: rows start 4 banks apart
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int stages = g.stages;

    if (tid == 0) {
        prefetch_tmap(&g.tm_w);
        prefetch_tmap(&g.tm_x);
        abort_flag = 0;
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full_bar[s], stage_arrivals(g, s));
            mbar_init(&empty_bar[s], 1);
        }
        mbar_init(&done_bar, 1);
        fence_mbarrier_init();
    }
    if (warp == 1) tmem_alloc(&tmem_base_s, PN);
    griddep_wait();                             // as in the small forward kernel
    int bad = 0;
    for (int e = tid; e < g.E; e += D_THREADS) {
        const int o0 = g.offsets[e], o1 = g.offsets[e + 1];
        if (o0 < 0 || o1 < o0 || o1 > g.T) bad = 1;
    }
    tc_fence_before();
    bad = __syncthreads_or(bad);
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_s;

    const int n_tiles = (g.K + COLS - 1) / COLS, per = (g.M + ROWS - 1) / ROWS * n_tiles;
    const int split = SPLIT ? g.split : 1, rank = SPLIT ? (int)cluster_ctarank() : 0;
    const int u = SPLIT ? blockIdx.x / split : blockIdx.x;
    const int e = quot(u, per), local = u - e * per, mt = quot(local, n_tiles);
    const int r0 = mt * ROWS, c0 = (local - mt * n_tiles) * COLS;
    const int t0 = bad ? 0 : __ldg(g.offsets + e), cnt = bad ? 0 : __ldg(g.offsets + e + 1) - t0;
    const int rows = min(ROWS, g.M - r0), cols = min(COLS, g.K - c0);
    const int64_t at = (int64_t)e * g.stride_out + (int64_t)r0 * g.ld_out + c0;
    float *w32 = static_cast<float *>(g.out) + at;
    uint16_t *w16 = static_cast<uint16_t *>(g.out) + at;
    if (bad || cnt == 0) {
        if (bad) {
            if (blockIdx.x == 0 && tid == 0) set_status(status, SF_STATUS_BAD_OFFSET);
        } else if (!g.accumulate) {             // an expert without tokens: zeros, 16 bytes to a thread
            const int unit = g.out_f32 ? 4 : 8, line = cols / unit;
            for (int i = rank * D_THREADS + tid; i < rows * line; i += split * D_THREADS) {
                const int r = quot(i, line), c = (i - r * line) * unit;
                if (g.out_f32) *reinterpret_cast<uint4 *>(w32 + r * g.ld_out + c) = make_uint4(0u, 0u, 0u, 0u);
                else *reinterpret_cast<uint4 *>(w16 + r * g.ld_out + c) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
        __syncwarp();
        if (warp == 1) tmem_dealloc(tmem_base, PN);
        return;
    }
    if (g.accumulate)                           // what W holds, on its way while the MMAs run
        for (int i = rank * D_THREADS + tid; i < rows * (COLS / 32); i += split * D_THREADS) {
            const int r = i / (COLS / 32), c = (i - r * (COLS / 32)) * 32;
            if (c < cols) prefetch_l2(w32 + r * g.ld_out + c);
        }
    const int nk = ((cnt + GK - 1) / GK + S * split - 1) / (S * split);      // steps of each slice
    const int chunks = g.out_f32 ? quot_up(nk, W_CHUNK_STAGES) : S == 4 ? quot_up(nk, W16_CHUNK_STAGES) : 1, chunk = quot_up(nk, chunks);
    constexpr int HELD = S == 4 ? (SPLIT ? 1 : ROWS * (COLS / 4) / (32 * P_EPI_WARPS)) : 1;
    float4 held[HELD];                          // S == 4, 16 bits: the chunks' sums of this thread's results
    auto hold = [&](float4 s, int q, int ch) {  // true: the last chunk's are in
        held[q] = ch == 0 ? s : make_float4(__fadd_rn(held[q].x, s.x), __fadd_rn(held[q].y, s.y), __fadd_rn(held[q].z, s.z), __fadd_rn(held[q].w, s.w));
        return ch == chunks - 1;
    };
    // slice j's tokens in its step i, those of the slice's end and of the expert's end left out
    const int step0 = rank * S * nk;            // of the slices before this CTA's
    auto tokens_of = [&](int j, int i) { return min(GK, cnt - (step0 + j * nk + i) * GK); };
    int stage = 0, sent = 0;
    uint32_t phase = 0;
    bool drained = false;
    auto drain = [&]() {                        // by the thread that sent them: loads on their way into this shared memory
        for (int s = 0; s < stages && s < sent && !drained; ++s) {
            const int last = (sent - 1 - s) / stages;             // the slot's last use
            const uint64_t from = globaltimer_ns();
            while (!mbar_try_wait(&full_bar[s], (uint32_t)(last & 1)) && globaltimer_ns() - from < kWaitLimitNs) {}
        }
        drained = true;                         // nothing is sent behind it
    };
    for (int ch = 0; ch < chunks; ++ch) {
        const int begin = ch * chunk, end = min(nk, begin + chunk);
        if (warp == 0) {
            if (lane == 0) {
                for (int i = abort_flag ? end : begin; i < end; ++i) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1u, &abort_flag)) break;
                    uint8_t *sy = smem + stage * D_STAGE_BYTES, *sa = sy + P_HALF_BYTES;
                    mbar_arrive_expect_tx(&full_bar[stage], D_STAGE_BYTES);
#pragma unroll
                    for (int j = 0; j < S; ++j) {
                        // a step behind the end reads behind the last row: zeros
                        const int t = tokens_of(j, i) > 0 ? t0 + (step0 + j * nk + i) * GK : g.T;
                        if (S == 1 && (g.whole & 1)) {
                            tma_load_3d(sy, &g.tm_t[0], &full_bar[stage], 0, t, r0 / 64);
                        } else {
                            tma_load_2d(sy + j * (P_HALF_BYTES / S), &g.tm_x, &full_bar[stage], r0, t);
                            if (S == 1) tma_load_2d(sy + G_BOX_BYTES, &g.tm_x, &full_bar[stage], r0 + 64, t);
                        }
                        if (S == 1 && (g.whole & 2)) {
                            tma_load_3d(sa, &g.tm_t[1], &full_bar[stage], 0, t, c0 / 64);
                        } else {
#pragma unroll
                            for (int b = 0; b < COLS / 64; ++b)
                                tma_load_2d(sa + (j * (COLS / 64) + b) * G_BOX_BYTES, &g.tm_w, &full_bar[stage], c0 + 64 * b, t);
                        }
                    }
                    ++sent;
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                }
                if (end == nk) griddep_launch_dependents();
                const uint64_t from = globaltimer_ns();
                while (!mbar_try_wait(&done_bar, (uint32_t)(ch & 1)) && globaltimer_ns() - from < kWaitLimitNs) {}
            }
        } else if (warp == 1) {
            const uint32_t s0 = smem_u32(smem);
            const uint64_t y0 = S == 4 ? mnmajor64(s0) : mnmajor(s0), a0 = mnmajor(s0 + P_HALF_BYTES);
            const uint32_t id = idesc(g.type, true, true, S == 1 ? (cols + 15) & ~15 : PN, SM_ROWS);
            int i = begin;
            for (; i < end; ++i) {
                if (!__all_sync(0xffffffffu, mbar_wait(&full_bar[stage], phase, &abort_flag))) break;
                uint8_t *sy = smem + stage * D_STAGE_BYTES, *sa = sy + P_HALF_BYTES;
#pragma unroll
                for (int j = 0; j < S; ++j) {   // rows of the next expert, in the box that holds the end: cleared
                    const int n = tokens_of(j, i);
                    if (n <= 0 || n >= GK) continue;
                    constexpr int ROW = S == 4 ? 64 : 128;            // bytes of a token in a box of the M operand
                    for (int k = lane; k < (GK - n) * 8; k += 32) {
                        const int row = n + (k >> 3);
                        if ((k & 7) * 16 < ROW) {
                            *reinterpret_cast<uint4 *>(sy + j * (P_HALF_BYTES / S) + row * ROW + (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            if (S == 1)
                                *reinterpret_cast<uint4 *>(sy + G_BOX_BYTES + row * ROW + (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
#pragma unroll
                        for (int b = 0; b < COLS / 64; ++b)
                            *reinterpret_cast<uint4 *>(sa + (j * (COLS / 64) + b) * G_BOX_BYTES + row * 128 + (k & 7) * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                tc_fence_after();
                const uint64_t dy = y0 + (uint64_t)(stage * (D_STAGE_BYTES >> 4));
                const uint64_t da = a0 + (uint64_t)(stage * (D_STAGE_BYTES >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < GK / G_UMMA_K; ++k)
                        mma_bf16(tmem_base, dy + k * (S == 4 ? 64 : 128), da + k * 128, id, i != begin || k != 0);
                    mma_commit(&empty_bar[stage]);
                    if (i == end - 1) mma_commit(&done_bar);
                }
                __syncwarp();
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            if (i < end && elect_one()) mma_commit(&done_bar);    // gave up
        }
        __syncwarp();
        if (!mbar_wait(&done_bar, (uint32_t)(ch & 1), &abort_flag)) abort_flag = 1;
        __syncthreads();
        if (abort_flag && !SPLIT) break;    // the CTAs of a cluster go on together
        tc_fence_after();
        const bool add = g.accumulate || ch > 0;
        if (warp >= 2 && !(SPLIT && abort_flag)) {
            const int quad = warp & 3, part = (warp - 2) >> 2;
            const int slice = quad * S / 4;
            // this warp's 32 accumulator rows and its half of the slice's columns
            const uint32_t t_row = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(slice * COLS + part * (COLS / 2));
            if (S == 1) {
                // out through shared memory (the stages are free), a box of 32 rows x 128 bytes at a time
                uint8_t *s_out = smem + (warp - 2) * W_OUT_BYTES;
                uint4 *slot = reinterpret_cast<uint4 *>(s_out) + lane * 8;
                const int wrows = rows - quad * 32, wcols = cols - part * (COLS / 2);
                float *d32 = w32 + quad * 32 * g.ld_out + part * (COLS / 2);
                uint16_t *d16 = w16 + quad * 32 * g.ld_out + part * (COLS / 2);
                const int box = g.out_f32 ? 32 : 64;
                for (int c = 0; c < min(COLS / 2, wcols) && wrows > 0; c += box) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(t_row + c, v);
                    tmem_ld_wait();
                    if (g.out_f32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) slot[j ^ (lane & 7)] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                    } else {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (h == 1) {
                                tmem_ld_32x32b_x32(t_row + c + 32, v);
                                tmem_ld_wait();
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                slot[(4 * h + j) ^ (lane & 7)] =
                                    make_uint4(pack2(v[8 * j], v[8 * j + 1], g.type), pack2(v[8 * j + 2], v[8 * j + 3], g.type),
                                               pack2(v[8 * j + 4], v[8 * j + 5], g.type), pack2(v[8 * j + 6], v[8 * j + 7], g.type));
                        }
                    }
                    __syncwarp();
                    const uint4 *lines = reinterpret_cast<const uint4 *>(s_out);
                    if (add) {
                        add_box(lines, d32 + c, g.ld_out, wrows, wcols - c, lane);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int row = i * 4 + (lane >> 3), unit = lane & 7;
                            const uint4 w = lines[row * 8 + (unit ^ (row & 7))];
                            if (row >= wrows) continue;
                            if (g.out_f32) {
                                if (c + unit * 4 < wcols) *reinterpret_cast<uint4 *>(d32 + row * g.ld_out + c + unit * 4) = w;
                            } else if (c + unit * 8 < wcols) {
                                *reinterpret_cast<uint4 *>(d16 + row * g.ld_out + c + unit * 8) = w;
                            }
                        }
                    }
                    __syncwarp();
                }
            } else {
                // partial sums of the slices, [slice][row][column], then their sum in the slices' order
                float *part_sums = reinterpret_cast<float *>(smem);
                float *mine = part_sums + (quad * 32 + lane) * PITCH + part * (COLS / 2);
#pragma unroll
                for (int c = 0; c < COLS / 2; c += 32) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(t_row + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4 *>(mine + c + 4 * j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                }
                asm volatile("bar.sync 1, %0;" ::"r"(32 * P_EPI_WARPS) : "memory");
#pragma unroll (S == 4 ? 2 : 1)
                for (int q = 0; q < ROWS * (COLS / 4) / (32 * P_EPI_WARPS); ++q) {
                    const int i = tid - 64 + q * 32 * P_EPI_WARPS, r = i / (COLS / 4), c = (i - r * (COLS / 4)) * 4;
                    if (r >= rows || c >= cols) continue;
                    float4 s = *reinterpret_cast<const float4 *>(part_sums + r * PITCH + c);
#pragma unroll
                    for (int j = 1; j < S; ++j) {
                        const float4 a = *reinterpret_cast<const float4 *>(part_sums + (j * ROWS + r) * PITCH + c);
                        s = make_float4(__fadd_rn(s.x, a.x), __fadd_rn(s.y, a.y), __fadd_rn(s.z, a.z), __fadd_rn(s.w, a.w));
                    }
                    if (SPLIT) *reinterpret_cast<float4 *>(part_sums + r * PITCH + c) = s;    // to be added to the other CTAs'
                    else if (S != 4 || g.out_f32) put_weights(g, w32, w16, r, c, s, add);
                    else if (hold(s, SPLIT ? 0 : q, ch)) put_weights(g, w32, w16, r, c, held[SPLIT ? 0 : q], false);
                }
            }
        }
        if (SPLIT) {                            // the CTAs' sums, in their order; each CTA has a share of the unit's results
            if (abort_flag) {
                if (tid == 0) drain();
                __syncthreads();
                leave_nan(smem, ROWS * PITCH, tid, D_THREADS);
            }
            __syncwarp();
            cluster_sync();
            const uint32_t part_sums = smem_u32(smem);
            static_assert(!SPLIT || ROWS * (COLS / 4) <= 2 * D_THREADS, "a result to a thread");
            const int i = rank * D_THREADS + tid, r = i / (COLS / 4), c = (i - r * (COLS / 4)) * 4;
            if (i < ROWS * (COLS / 4) && r < rows && c < cols) {
                float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int o = 0; o < split; ++o) {
                    const uint32_t from = part_sums + (r * PITCH + c) * 4;
                    const float2 a = ld_cluster_f32x2(from, o), b = ld_cluster_f32x2(from + 8, o);
                    s = make_float4(__fadd_rn(s.x, a.x), __fadd_rn(s.y, a.y), __fadd_rn(s.z, b.x), __fadd_rn(s.w, b.y));
                }
                if (!g.out_f32 && hold(s, 0, ch)) s = held[0];
                if ((g.out_f32 || ch == chunks - 1) && !(s.x != s.x && cluster_gave_up(&abort_flag, split))) put_weights(g, w32, w16, r, c, s, add);
            }
            __syncwarp();
            cluster_sync();                     // no CTA goes on while others read its sums
        }
        tc_fence_before();
        if (ch + 1 < chunks) fence_proxy_async_smem();            // the stages go back to TMA
        __syncthreads();
        tc_fence_after();
    }
    __syncwarp();
    if (abort_flag && tid == 0) {               // before the shared memory goes away
        drain();
        set_status(status, SF_STATUS_WAIT_TIMEOUT);
    }
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, PN);
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

// Map over [depth x rows x cols] (depth 0: two dimensions) with boxes of box_bytes (128 or 64, swizzled, or 256, plain) by box_rows rows.
bool encode(CUtensorMap *m, int type, const void *base, int cols, int64_t rows, int64_t ld, int depth, int64_t stride,
            int box_rows, int box_bytes = 128)
{
    EncodeTiledFn fn = grouped_encode_fn();
    if (!fn) return false;
    const int size = type == SF_TYPE_F32 ? 4 : 2;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)(rows > 0 ? rows : 1), (cuuint64_t)depth};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * size, (cuuint64_t)stride * size};
    const cuuint32_t box[3] = {(cuuint32_t)(box_bytes / size), (cuuint32_t)box_rows, 1u};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, type == SF_TYPE_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                 : type == SF_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
              depth > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              box_bytes == 64    ? CU_TENSOR_MAP_SWIZZLE_64B
              : box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                 : CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Rows of whole chunks of 64 16-bit columns, as {64, rows, chunks}: a box is 64 rows of several chunks, each of which lies as a
// box of its own would.
bool encode_chunks(CUtensorMap *m, int type, const void *base, int cols, int64_t rows, int64_t ld, int chunks)
{
    EncodeTiledFn fn = grouped_encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(cols / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)ld * 2, 128};
    const cuuint32_t box[3] = {64, 64, (cuuint32_t)chunks}, estr[3] = {1, 1, 1};
    return fn(m, type == SF_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void *>(base),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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
    // The kernels round counts up to whole tiles, and add numbers of tiles to them, in 32 bits.
    const int most = 1 << 30;
    if (p->T > most || p->R > most || p->C > most) return SF_ERR_UNSUPPORTED;
    // byte strides a tensor map can hold (below 2^40), and tile counts that stay far inside 32 bits
    const int64_t far = (int64_t)1 << 38;
    if (p->ld_w > far || p->stride_w > far || p->ld_a > far || p->ld_y > far) return SF_ERR_UNSUPPORTED;
    const int64_t wide = (p->R > p->C ? p->R : p->C) / 128 + 1;
    const int64_t tall = (int64_t)p->T / 16 + p->E;
    if (wide * tall > (1 << 30) || (int64_t)p->E * ((p->R + PM - 1) / PM) * ((p->C + 63) / 64) > (1 << 30))
        return SF_ERR_UNSUPPORTED;
    if (p->T > 0 && (p->A == p->Y || p->A == p->W || p->Y == p->W)) return SF_ERR_ARG;      // one is written
    return SF_OK;
}

// Test hook for the bounded waits: with SF_TEST_GROUPED_WITHHOLD set in the environment, CTA 0's first stage never completes.
int withhold_test()
{
    const char *e = getenv("SF_TEST_GROUPED_WITHHOLD");
    return e && e[0] && e[0] != '0';
}

// CTA pairs that can be resident at once on the current device (the same for all pair kernels: a pair takes two
// whole SMs).
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
                             (int)T_SMEM_BYTES) != cudaSuccess)
        return 0;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * sms);
    cfg.blockDim = dim3(P_THREADS);
    cfg.dynamicSmemBytes = T_SMEM_BYTES;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, grouped_pair_kernel<false>, &cfg) != cudaSuccess || n <= 0) return 0;
    if (dev < kDevs) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Lets the kernel have the shared memory of the largest of its calls. The limit is one for all host threads, so it is never
// set to a call's own size, which another thread's launch may be above. Called before the tensor maps are made: in a host
// thread's first call it is what makes the device's context current, without which no map can be encoded.
template <typename K>
bool prepare_kernel(K kernel, size_t most)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) == cudaSuccess;
}

template <typename K>
int launch(K kernel, int grid, int cluster, int threads, size_t smem, const GArgs &g, uint32_t *status, sf_stream stream)
{
    // programmatic dependent launch: the kernels wait for their predecessor themselves, behind what they can do without it
    // (4.4 -> 3.4 us for the smallest calls back to back)
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = as_stream(stream);
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, g, status) != cudaSuccess) return SF_ERR_CUDA;
    return launch_status();
}

// Forward, dx: pairs run when an expert has more than this many tokens on average. At 96, 128 and 256 of them, single CTAs
// against pairs: 50.6 / 64.5, 70.6 / 65.9 and 98 / 76 us for 8 experts of 4096 x 4096; 69.8 / 74.4, 96 / 79 and 158 / 101 us
// for 48 of 1416 x 2056; 258 / 299, 308 / 340 and 455 / 369 us for 16 of 11008 x 4096. Short sums (nk steps of 64) have less
// to gain from large tiles: 8 experts of 4096 x 256 over 100, 200, 300 and 800 tokens each 9.6 / 13.5, 13.9 / 15.3, 18.0 /
// 19.3 and 33.9 / 32.5 us, 32 of 1376 x 512 over 128 and 300 15.8 / 18.8 and 25.6 / 30.5; 64 of 1024 x 1024 over 100, 160
// and 250 32.4 / 40.7, 40.9 / 43.8 and 50.6 / 51.0.
constexpr int64_t pair_from(int nk) { return nk <= 8 ? 512 : nk <= 16 ? 192 : 96; }
// dw that adds: below this many tokens to an expert, what W holds comes in by TMA and is added in shared memory; from there
// on the addition is TMA's. 4 experts of 11008 x 4096 over 64, 256, 512 and 900 tokens each: 250, 259, 313 and 509 us the
// one way, 322, 327, 330 and 418 us the other.
constexpr int64_t kDwOldBelow = 512;
// dw that does not add: below this many, fewer stages and a place for all of a warp's boxes too. At 16, 64, 128 and 512
// tokens, so against with the deep ring: 56 / 77, 61 / 78, 71 / 72 and 102 / 90 us for 16 experts of 2048 x 2048; 133 / 144,
// 140 / 147, 159 / 154 and 254 / 209 us for 4 of 11008 x 4096.
constexpr int64_t kDwFewBelow = 128;

// What a call takes.
struct Choice {
    int kernel;                // SF_GROUPED_*
    int slices, split;         // single CTAs: slices of the sums in a CTA, CTAs (a cluster) that share a unit's
    int nb, stages;            // single CTAs: token box (forward, dx), stages
    int64_t units;             // at most
};

Choice choose_product(const sf_grouped *p, bool fwd, int sms)
{
    Choice x = {};
    const int M = fwd ? p->R : p->C, nk = ((fwd ? p->C : p->R) + GK - 1) / GK;
    // A token box that holds most experts in one tile: up to 32 tokens, where the weights outweigh the box, twice the
    // average (a decode batch of 12 tokens each: 114.6 us against 116.5 with a box of 16), beyond that the average and
    // a quarter (49 tokens each: 26.7 us with a box of 64, 31.0 with 128).
    const int64_t avg = ((int64_t)p->T + p->E - 1) / p->E;
    int nb = 16;
    while (nb < 128 && nb < p->T && 4 * nb < (nb < 32 ? 8 * avg : 5 * avg)) nb *= 2;
    const int64_t busy = p->E < p->T ? p->E : p->T;      // experts with a token, at most
    const int64_t tiles = busy + p->T / nb;              // token tiles, at most
    const int64_t m_tiles = (M + SM_ROWS - 1) / SM_ROWS;
    const bool one_round = tiles * m_tiles <= 2 * sms;

    if (!one_round && p->T > pair_from(nk) * p->E) {
        x.kernel = SF_GROUPED_PAIRS;
        x.units = ((int64_t)p->T / 64 + p->E) * ((M + PM - 1) / PM);
        return x;
    }
    // K in slices while the units fit the device at once, two CTAs to an SM, with a token tile to an expert where most experts'
    // tokens fit one. Where they take several, only long sums that leave half of the SMs without work (one expert of 64 x 4096
    // over 300, 1,000 and 8,000 tokens: 23.8, 24.4 and 25.2 us without slices, 8.4, 9.2 and 15.3 with; 3 of 88 x 560 over 416
    // each 8.9 / 9.5, one of 184 x 9632 over 7,202 53 / 69).
    const bool one_tile = avg <= nb;
    int s = 1;
    while (s < 4 && (one_tile ? busy * m_tiles <= sms / s : tiles * m_tiles <= sms / (2 * s)) && nk >= (one_tile ? 4 : 10) * s && 2 * s * nb <= 256)
        s *= 2;
    // Several units to a CTA, planned ahead, where a unit is short (64 experts of 1024 x 1024 over 64 tokens each: 35.6 ->
    // 32.1 us); long ones come out more even as a CTA each (the decode batch above: 114.6 against 117.5 us).
    const bool rounds = s == 1 && tiles * m_tiles > 2 * sms && nk <= 24;
    const int stage_bytes = S_W_BYTES + s * nb * GK * 2;
    const int rows = SM_ROWS / s;
    x.units = tiles * ((M + rows - 1) / rows);
    // The slices over the CTAs of a cluster, too, while the units still fit and a CTA keeps two steps or more (alone against
    // in clusters: one expert of 64 x 4096 over 16 tokens 10.7 / 5.0 us, 512 x 11008 over 100 tokens 45.3 / 11.4, 4096 x 4096
    // over 2 tokens 11.0 / 8.9; with a step a CTA, 2 experts of 512 x 512 over 2 tokens each, 4.0 / 4.7).
    x.split = 1;
    while (s > 1 && x.split < 8 && x.units * 2 * x.split <= sms * 7 / 4 && nk >= 2 * 2 * x.split * s) x.split *= 2;
    // One CTA to an SM, or two. Clusters do not fill every SM (8 experts of 128 x 2048 over 2 tokens each, 144 CTAs in
    // clusters of 4: 7.9 us with one to an SM, 5.3 with two).
    x.stages = (x.units * x.split <= (x.split > 1 ? sms * 3 / 4 : sms) ? S_RING_BYTES : S_RING_BYTES / 2) / stage_bytes;
    if (x.stages > S_MAX_STAGES) x.stages = S_MAX_STAGES;
    x.nb = nb;
    x.slices = s;
    x.kernel = rounds ? SF_GROUPED_ROUNDS : x.split > 1 ? SF_GROUPED_CLUSTERS : s > 1 ? SF_GROUPED_SLICES : SF_GROUPED_SINGLE;
    return x;
}

Choice choose_dw(const sf_grouped *p, bool accumulate, int sms)
{
    Choice x = {};
    auto tiles = [&](int rows, int cols) {
        return (int64_t)((p->R + rows - 1) / rows) * ((p->C + cols - 1) / cols);
    };
    const int64_t busy = p->E < p->T ? p->E : p->T;      // experts with a token, at most
    // Pairs, unless they would be few, or one round of single CTAs does it all with short sums (8 experts of 1024 x 1024
    // over 128 tokens each: 11.1 us against 13.1; one of 2048 x 2048 over 4,096: 56 us against 30).
    const bool long16 = p->w_type != SF_TYPE_F32 && p->T > W16_TOKENS;
    const bool one_round = busy * tiles(SM_ROWS, PN) <= 2 * sms && p->T <= (int64_t)512 * p->E && !long16;
    // Tokens in slices while the units still fit the device at once (one expert of 512 x 512 over 8,192 tokens: 102, 43 and
    // 24 us with 1, 2 and 4 slices; where they do not fit, every slice more costs its share of the loads again).
    int s = 1;
    while (s < 4 && busy * tiles(SM_ROWS / (2 * s), PN / (2 * s)) <= 2 * sms && p->T > (int64_t)GK * s * p->E) s *= 2;
    if ((busy * tiles(PM, PN) >= sms / 4 && !one_round) || (long16 && s < 4)) {
        const bool few = p->T < (accumulate ? kDwOldBelow : kDwFewBelow) * p->E;
        x.kernel = !few ? SF_GROUPED_PAIRS : accumulate ? SF_GROUPED_PAIRS_ADD : SF_GROUPED_PAIRS_FEW;
        x.units = p->E * tiles(PM, PN);
        return x;
    }
    x.slices = s;
    // Four slices in each CTA of a cluster while the CTAs fit one to an SM and keep more than four steps (alone against in
    // clusters: one expert of 128 x 128 over 65,536 tokens 151 / 31 us, of 64 x 512 over 8,192 tokens 22.3 / 9.5; with
    // shorter sums or fewer slices clusters cost what they save).
    x.split = 1;
    x.units = p->E * tiles(SM_ROWS / s, PN / s);
    while (s == 4 && x.split < 8 && x.units * 2 * x.split <= sms && p->T > (int64_t)4 * GK * 4 * 2 * x.split * p->E) x.split *= 2;
    x.stages = x.units * x.split <= (x.split > 1 ? sms * 3 / 4 : sms) ? D_MAX_STAGES : D_MAX_STAGES / 2;       // one CTA to an SM, or two
    x.kernel = x.split > 1 ? SF_GROUPED_CLUSTERS : s > 1 ? SF_GROUPED_SLICES : SF_GROUPED_SINGLE;
    return x;
}

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
    g.withhold_test = withhold_test();
    const void *x = fwd ? p->A : p->Y;
    const int64_t ld_x = fwd ? p->ld_a : p->ld_y;
    const int64_t stride = p->E > 1 ? p->stride_w : (int64_t)p->R * p->ld_w;
    const Choice c = choose_product(p, fwd, sms);

    if (c.kernel == SF_GROUPED_PAIRS) {
        if (!prepare_kernel(grouped_pair_kernel<TRANS>, T_SMEM_BYTES)) return SF_ERR_CUDA;
        if (!encode(&g.tm_w, p->type, p->W, p->C, p->R, p->ld_w, p->E, stride, fwd ? 128 : 64) ||
            !encode(&g.tm_y, p->type, g.out, g.M, p->T, g.ld_out, 0, 0, 16, 256))
            return SF_ERR_CUDA;
        for (int b = 0; b < 4; ++b)
            if (!encode(&g.tm_t[b], p->type, x, g.K, p->T, ld_x, 0, 0, 32 * (b + 1))) return SF_ERR_CUDA;
        const int slots = pair_slots();
        if (slots <= 0) return SF_ERR_CUDA;
        const int pairs = (int)(c.units < slots ? c.units : slots);
        return launch(grouped_pair_kernel<TRANS>, 2 * pairs, 2, P_THREADS, T_SMEM_BYTES, g, status, stream);
    }
    const bool rounds = c.kernel == SF_GROUPED_ROUNDS;
    g.nb = c.nb;
    g.split = c.split;
    g.stages = c.stages;
    auto kernel = rounds ? grouped_small_kernel<TRANS, 1, true> : c.slices == 1 ? grouped_small_kernel<TRANS, 1, false>
                  : c.slices == 2 ? grouped_small_kernel<TRANS, 2, false> : grouped_small_kernel<TRANS, 4, false>;
    if (!prepare_kernel(kernel, S_SMEM_BYTES)) return SF_ERR_CUDA;
    const int box_rows = fwd ? SM_ROWS / c.slices : 64, box_bytes = !fwd && c.slices == 4 ? 64 : 128;
    if (!encode(&g.tm_w, p->type, p->W, p->C, p->R, p->ld_w, p->E, stride, box_rows, box_bytes)) return SF_ERR_CUDA;
    for (int b = 0; 16 << b <= c.nb; ++b)
        if (!encode(&g.tm_t[b], p->type, x, g.K, p->T, ld_x, 0, 0, 16 << b)) return SF_ERR_CUDA;
    const int grid = (int)(rounds ? 2 * sms : c.units * c.split);
    const size_t smem = (size_t)c.stages * (S_W_BYTES + c.slices * c.nb * GK * 2) + 1024;
    return launch(kernel, grid, c.split, S_THREADS, smem, g, status, stream);
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
    const int sms = sm_count();
    if (sms <= 0) return SF_ERR_NO_DEVICE;
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
    g.withhold_test = withhold_test();
    g.out_f32 = p->w_type == SF_TYPE_F32;
    g.accumulate = accumulate != 0;
    // without tokens nothing is loaded: any valid address makes the maps
    const void *a = p->T > 0 ? p->A : p->W, *y = p->T > 0 ? p->Y : p->W;
    const int64_t ld_a = p->T > 0 ? p->ld_a : p->C, ld_y = p->T > 0 ? p->ld_y : p->R;
    const int64_t stride = p->E > 1 ? p->stride_w : (int64_t)p->R * p->ld_w;
    const Choice c = choose_dw(p, accumulate != 0, sms);
    if (c.kernel >= SF_GROUPED_PAIRS) {
        auto kernel = c.kernel == SF_GROUPED_PAIRS     ? grouped_dw_kernel<false, false>
                      : c.kernel == SF_GROUPED_PAIRS_ADD ? grouped_dw_kernel<true, true>
                                                         : grouped_dw_kernel<false, true>;
        if (!prepare_kernel(kernel, W_SMEM_BYTES)) return SF_ERR_CUDA;
        if (!encode(&g.tm_w, p->type, a, p->C, p->T, ld_a, 0, 0, 64) || !encode(&g.tm_x, p->type, y, p->R, p->T, ld_y, 0, 0, 64) ||
            !encode(&g.tm_out, p->w_type, p->W, p->C, p->R, p->ld_w, p->E, stride, 32))
            return SF_ERR_CUDA;
        const int slots = pair_slots();
        if (slots <= 0) return SF_ERR_CUDA;
        // Where the columns are whole chunks of 64, one box takes two chunks: half the copies to issue (4 experts of 4096 x
        // 4096 over 1,024 tokens and more: 2% less).
        if (p->T > 0 && p->R % 64 == 0 && encode_chunks(&g.tm_t[0], p->type, y, p->R, p->T, ld_y, 2)) g.whole |= 1;
        if (p->T > 0 && p->C % 64 == 0 && encode_chunks(&g.tm_t[1], p->type, a, p->C, p->T, ld_a, 2)) g.whole |= 2;
        return launch(kernel, 2 * (int)(c.units < slots ? c.units : slots), 2, W_THREADS, W_SMEM_BYTES, g, dev_status, stream);
    }
    g.split = c.split;
    g.stages = c.stages;
    auto kernel = c.split > 1 ? grouped_dw_small_kernel<4, true> : c.slices == 1 ? grouped_dw_small_kernel<1, false>
                  : c.slices == 2 ? grouped_dw_small_kernel<2, false> : grouped_dw_small_kernel<4, false>;
    if (!prepare_kernel(kernel, D_SMEM_BYTES)) return SF_ERR_CUDA;
    if (!encode(&g.tm_w, p->type, a, p->C, p->T, ld_a, 0, 0, 64) ||
        !encode(&g.tm_x, p->type, y, p->R, p->T, ld_y, 0, 0, 64, c.slices == 4 ? 64 : 128))
        return SF_ERR_CUDA;
    // 2 copies a stage in place of 6 (8 experts of 1024 x 1024 over 128 tokens each: 11.7 -> 10.4 us; with slices no gain)
    if (p->T > 0 && c.slices == 1 && p->R % 64 == 0 && encode_chunks(&g.tm_t[0], p->type, y, p->R, p->T, ld_y, 2)) g.whole |= 1;
    if (p->T > 0 && c.slices == 1 && p->C % 64 == 0 && encode_chunks(&g.tm_t[1], p->type, a, p->C, p->T, ld_a, 4)) g.whole |= 2;
    return launch(kernel, (int)c.units * c.split, c.split, D_THREADS, (size_t)c.stages * D_STAGE_BYTES + 1024, g, dev_status, stream);
}

extern "C" int sf_grouped_kernel(const sf_grouped *p, int product, int accumulate)
{
    if (product != SF_GROUPED_FORWARD && product != SF_GROUPED_DX && product != SF_GROUPED_DW) return SF_ERR_ARG;
    const bool dw = product == SF_GROUPED_DW;
    int rc = check_grouped(p, dw);
    if (rc != SF_OK) return rc;
    if (dw && accumulate && p->w_type != SF_TYPE_F32) return SF_ERR_ARG;
    if (!dw && p->T == 0) return SF_GROUPED_NONE;
    const int sms = sm_count();
    if (sms <= 0) return SF_ERR_NO_DEVICE;
    return dw ? choose_dw(p, accumulate != 0, sms).kernel : choose_product(p, product == SF_GROUPED_FORWARD, sms).kernel;
}
