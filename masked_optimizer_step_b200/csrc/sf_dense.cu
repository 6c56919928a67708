// sf_dense.cu -- AdamW over many dense tensors at once, and the global gradient norm that clips it.
//
// The arithmetic is in include/sf.h. Both kernels are single passes over memory: the norm reads
// every gradient once, the step reads and writes every weight and moment once (28 bytes an element
// with fp32 moments, a bf16 gradient and a bf16 live copy; 16.06 with 8-bit moments).
//
// Layout of the work: a block of 256 elements (the unit that shares the 8-bit moments' scales) belongs to
// one warp, 8 consecutive elements to a lane, so every access is an 8-, 16- or 32-byte vector of a
// fully coalesced row and a block's largest magnitude is one warp-wide integer maximum. A unit is
// `per` blocks for each of a CTA's 8 warps; units of all tensors are numbered through. A CTA of the
// step takes one, a CTA of the norm every gridDim-th one.
#include <string.h>

#include <cuda_fp8.h>

#include "sf_common.cuh"
#include "sf_host.h"

namespace sf {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = SF_DENSE_BLOCK;
constexpr int kLaneElems = kBlock / 32;
static_assert(kLaneElems == 8, "eight elements to a lane");
constexpr int kMaxTensors = SF_DENSE_PER_LAUNCH;
constexpr int kMaxGridPerSm = 8;              // CTAs of the norm, to an SM
constexpr float kScaleFloor = 0x1p-100f;      // keeps 1 / scale finite
constexpr float kSmallestCode = 0x1p-9f;      // smallest positive e4m3 value

struct DenseDesc {
    int64_t n;
    void *p;
    const void *g;
    void *m, *v;
    float *m_scale, *v_scale;
    uint16_t *live;
    float decay;
    uint8_t p_type, g_type, state_type, pad;
};

// The tensors of a launch, as kernel parameters: a launch carries all of them, so there is a form for few, one for some
// and one for many (65 tensors: 13 us from call to call with 384 places, 8 with 96).
template <int N>
struct DenseBatch {
    int32_t n, units, per;                    // tensors, units in all, blocks of a unit per warp
    int32_t unit_begin[N];                    // units of the tensors before this one
    DenseDesc d[N];
};
static_assert(sizeof(DenseBatch<kMaxTensors>) <= 32000, "kernel parameter space");
constexpr int kFew = 16, kSome = 96;

// Two fp32 values in one 64-bit register pair, and the operations of sm_100 that take both at once, each rounded as
// its scalar form. The step with 8-bit moments is held up by the instructions it issues, not by memory alone.
typedef uint64_t pair_t;
__device__ __forceinline__ pair_t pair_of(float a, float b)
{
    pair_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 halves(pair_t p)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b)
{
    pair_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair_t add2(pair_t a, pair_t b)
{
    pair_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c)
{
    pair_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

struct StepArgs {
    pair_t beta1, beta2, omb1, omb2, eps, minus_lr;       // each value twice
    float lr, wd, clip;
    const float *bc1, *bc2;
    int32_t t_max, last;                      // last: this launch ends the call
    int32_t *step;
    const float *factor;
};

template <int N>
__device__ __forceinline__ int find_tensor(const DenseBatch<N> &b, int unit)
{
    int lo = 0, hi = b.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (b.unit_begin[mid] <= unit) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// Square roots by one step of Heron's iteration from the hardware's approximate reciprocal root y: with r = x y, the
// residual r r - x is exact in one fused operation, and r - (r r - x) y / 2 is the root to the last place (tests hold it
// to the correctly rounded one). The library's root, with its paths for numbers outside the normal ones, took a third of
// the step's instructions. Zero gives zero. The residual is a multiple of 2^-149, so it is off by up to 2^-150 and the
// root by up to 2^-150 y / 2, which is 2^-151 / x of it: nothing down to 2^-100, a quarter of a step at 2^-126. An infinite x,
// whose residual is not a number, gives infinity (a NaN does too: its moment and weight are NaN without the root).
__device__ __forceinline__ pair_t root2_of(pair_t x)
{
    const float2 v = halves(x);
    float ya, yb;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(ya) : "f"(fmaxf(v.x, 0x1p-149f)));
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(yb) : "f"(fmaxf(v.y, 0x1p-149f)));
    const pair_t y = pair_of(ya, yb), r = mul2(x, y);
    const pair_t off = fma2(r, r, mul2(x, pair_of(-1.0f, -1.0f)));
    const float2 root = halves(fma2(off, mul2(y, pair_of(-0.5f, -0.5f)), r));
    return pair_of(fminf(root.x, __int_as_float(0x7f800000)), fminf(root.y, __int_as_float(0x7f800000)));
}

// a / b within 2 units in the last place for the sizes that occur here (b normal, below 2^126).
__device__ __forceinline__ pair_t ratio2(pair_t a, pair_t b)
{
    const float2 v = halves(b);
    float ya, yb;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ya) : "f"(v.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(yb) : "f"(v.y));
    return mul2(a, pair_of(ya, yb));
}

// x between -limit and limit; a NaN stays one (fminf and fmaxf would take the limit in its place).
__device__ __forceinline__ float clamped(float x, float limit)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(-limit));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(r) : "f"(limit));
    return r;
}

// A lane's eight consecutive elements as they lie in memory: 16 bytes of 16-bit values, 32 of fp32. With FULL all eight
// are there; without, the first `cnt`, and the rest are zero.
struct Raw8 {
    uint4 a, b;
};

template <bool FULL>
__device__ __forceinline__ Raw8 load_raw(const void *base, int type, int64_t at, int cnt)
{
    Raw8 r;
    r.a = r.b = make_uint4(0u, 0u, 0u, 0u);
    if (type == SF_TYPE_F32) {
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
        if (FULL || cnt == 8) {
            r.a = __ldcs(src);
            r.b = __ldcs(src + 1);
        } else if (cnt > 0) {
            const uint32_t *w = reinterpret_cast<const uint32_t *>(src);
            r.a = make_uint4(w[0], cnt > 1 ? w[1] : 0u, cnt > 2 ? w[2] : 0u, cnt > 3 ? w[3] : 0u);
            r.b = make_uint4(cnt > 4 ? w[4] : 0u, cnt > 5 ? w[5] : 0u, cnt > 6 ? w[6] : 0u, 0u);
        }
    } else {
        const uint16_t *src = static_cast<const uint16_t *>(base) + at;
        if (FULL || cnt == 8) {
            r.a = __ldcs(reinterpret_cast<const uint4 *>(src));
        } else if (cnt > 0) {
            auto two = [&](int e) { return (e < cnt ? (uint32_t)src[e] : 0u) | (e + 1 < cnt ? (uint32_t)src[e + 1] << 16 : 0u); };
            r.a = make_uint4(two(0), two(2), two(4), two(6));
        }
    }
    return r;
}

__device__ __forceinline__ void to_pairs(pair_t (&x)[4], const Raw8 &r, int type)
{
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
    if (type == SF_TYPE_F32) {
        x[0] = pair_of(__uint_as_float(r.a.x), __uint_as_float(r.a.y));
        x[1] = pair_of(__uint_as_float(r.a.z), __uint_as_float(r.a.w));
        x[2] = pair_of(__uint_as_float(r.b.x), __uint_as_float(r.b.y));
        x[3] = pair_of(__uint_as_float(r.b.z), __uint_as_float(r.b.w));
    } else if (type == SF_TYPE_BF16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = pair_of(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
            x[e] = pair_of(h.x, h.y);
        }
    }
}

template <bool FULL>
__device__ __forceinline__ void store8_f32(float *dst, const pair_t (&x)[4], int cnt)
{
    const float2 a = halves(x[0]), b = halves(x[1]), c = halves(x[2]), d = halves(x[3]);
    if (FULL || cnt == 8) {
        __stcs(reinterpret_cast<float4 *>(dst), make_float4(a.x, a.y, b.x, b.y));
        __stcs(reinterpret_cast<float4 *>(dst) + 1, make_float4(c.x, c.y, d.x, d.y));
    } else {
        const float v[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < cnt) dst[e] = v[e];
    }
}

template <bool FULL>
__device__ __forceinline__ void store8_bf16(uint16_t *dst, const pair_t (&x)[4], int cnt)
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = halves(x[e]);
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        w[e] = *reinterpret_cast<const uint32_t *>(&h);
    }
    if (FULL || cnt == 8) {
        __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(w[0], w[1], w[2], w[3]));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < cnt) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}

// Eight e4m3 codes (zeros behind cnt) as two words.
template <bool FULL>
__device__ __forceinline__ uint2 load8_codes(const void *base, int64_t at, int cnt)
{
    const uint8_t *src = static_cast<const uint8_t *>(base) + at;
    if (FULL || cnt == 8) return __ldcs(reinterpret_cast<const uint2 *>(src));
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < cnt) w[e >> 2] |= (uint32_t)src[e] << (8 * (e & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode8(pair_t (&x)[4], uint2 codes, float scale)
{
    const pair_t s = pair_of(scale, scale);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = e < 2 ? codes.x : codes.y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (e & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[e] = mul2(pair_of(f.x, f.y), s);
    }
}

// Codes and scale of a block's values (this lane's eight); returns the scale. POSITIVE: no value is negative, and a value
// above zero keeps a code above zero.
template <bool FULL, bool POSITIVE>
__device__ __forceinline__ float encode8(const pair_t (&x)[4], void *base, int64_t at, int cnt, float *scale, int lane)
{
    uint32_t big = 0;                                // magnitudes order as their bits; a NaN is the largest
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 v = halves(x[e]);
        const uint32_t a = __float_as_uint(v.x), b = __float_as_uint(v.y);
        big = max(big, POSITIVE ? max(a, b) : max(a & 0x7FFFFFFFu, b & 0x7FFFFFFFu));
    }
    big = __reduce_max_sync(0xffffffffu, big);
    float sc = __fmul_rn(__uint_as_float(big), 1.0f / 448.0f);
    if (sc < kScaleFloor) sc = kScaleFloor;          // a NaN stays
    const float inv = __frcp_rn(sc);
    const pair_t inv2 = pair_of(inv, inv);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float2 v = halves(mul2(x[e], inv2));
        if (POSITIVE) {
            const float2 was = halves(x[e]);
            if (was.x > 0.0f) v.x = fmaxf(v.x, kSmallestCode);
            if (was.y > 0.0f) v.y = fmaxf(v.y, kSmallestCode);
        }
        w[e >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3) << (16 * (e & 1));
    }
    uint8_t *dst = static_cast<uint8_t *>(base) + at;
    if (FULL || cnt == 8) {
        __stcs(reinterpret_cast<uint2 *>(dst), make_uint2(w[0], w[1]));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < cnt) dst[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
    if (lane == 0) *scale = sc;
    return sc;
}

// A warp's way through its blocks of the CTA's unit, kWarps apart. The tensor comes from the CTA's number alone, so its
// description stays in uniform registers; only the warp's place in it is each lane's own (with the place worked out anew
// for each block the step took 502 instructions a block).
constexpr int kStride = kWarps * kBlock;

struct Place {
    int64_t at;                // this lane's first element
    int64_t blk;               // block of the tensor
    int left;                  // elements from the block's first one on, 2^30 at most
    int more;                  // blocks from here on

    __device__ __forceinline__ Place(const DenseDesc &d, int unit, int per)
    {
        blk = (int64_t)unit * per * kWarps + (threadIdx.x >> 5);
        at = blk * kBlock + (threadIdx.x & 31) * kLaneElems;
        left = (int)max((int64_t)0, min(d.n - blk * kBlock, (int64_t)1 << 30));
        more = min(per, (left + kStride - 1) / kStride);
    }
    __device__ __forceinline__ void next()
    {
        at += kStride;
        blk += kWarps;
        left -= kStride;
        --more;
    }
    __device__ __forceinline__ bool full() const { return left >= kBlock; }
    __device__ __forceinline__ int count() const { return max(0, min(8, left - (int)(threadIdx.x & 31) * kLaneElems)); }
};

// What a block's step reads, as it lies in memory.
template <bool CODED>
struct Block {
    Raw8 p, g, m, v;           // moments: fp32
    uint2 cm, cv;              // or codes

    __device__ __forceinline__ void load(const DenseDesc &d, const Place &w)
    {
        if (w.full()) load_from<true>(d, w, 8);
        else load_from<false>(d, w, w.count());
    }
    template <bool FULL>
    __device__ __forceinline__ void load_from(const DenseDesc &d, const Place &w, int cnt)
    {
        p = load_raw<FULL>(d.p, d.p_type, w.at, cnt);
        g = load_raw<FULL>(d.g, d.g_type, w.at, cnt);
        if (CODED) {
            cm = load8_codes<FULL>(d.m, w.at, cnt);
            cv = load8_codes<FULL>(d.v, w.at, cnt);
        } else {
            m = load_raw<FULL>(d.m, SF_TYPE_F32, w.at, cnt);
            v = load_raw<FULL>(d.v, SF_TYPE_F32, w.at, cnt);
        }
    }
};

// A block's lines into L2, ahead of its loads: a lane to a line of 128 bytes, 8 for an array of 32-bit values, 4 of 16, 2
// of 8.
struct Ahead {
    const char *line;          // this lane's line of the next block asked for
    int step, from;            // bytes from block to block; the line's first element in its block, 2^30 where there is none

    __device__ __forceinline__ Ahead(const DenseDesc &d, const Place &w)
    {
        const int lane = threadIdx.x & 31, type = lane < 8 ? d.p_type : lane < 16 ? d.g_type : d.state_type;
        const char *base = static_cast<const char *>(lane < 8 ? d.p : lane < 16 ? d.g : lane < 24 ? d.m : d.v);
        const int size = type == SF_TYPE_F32 ? 4 : type == SF_TYPE_E4M3 ? 1 : 2, l = lane & 7;
        line = base + w.blk * kBlock * size + l * 128;
        step = kStride * size;
        from = l < 2 * size ? l * 128 / size : 1 << 30;
    }
    // for the block that has `left` elements from its first one on
    __device__ __forceinline__ void ask(int left)
    {
        if (from < left) prefetch_l2(line);
        line += step;
    }
};

struct StepNow {
    pair_t bc1, root_bc2, factor;
};

// One block's step on what was loaded: this lane's eight elements. FULL: the block has all its 256.
template <bool CODED, bool CLIP, bool FULL>
__device__ __forceinline__ void step_block(const Block<CODED> &in, float sm, float sv, const DenseDesc &d, int64_t at, int64_t blk, int cnt,
                                           const StepArgs &a, const StepNow &now, pair_t &nan_sum)
{
    const int lane = threadIdx.x & 31;
    pair_t p[4], g[4], m[4], v[4];
    to_pairs(p, in.p, d.p_type);
    to_pairs(g, in.g, d.g_type);
    if (CODED) {
        decode8(m, in.cm, sm);
        decode8(v, in.cv, sv);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], v[e]);
    } else {
        to_pairs(m, in.m, SF_TYPE_F32);
        to_pairs(v, in.v, SF_TYPE_F32);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = mul2(g[e], now.factor);
    const pair_t zero = pair_of(0.0f, 0.0f);
    if (CLIP) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            nan_sum = fma2(g[e], zero, nan_sum);     // what is not finite is reported although the clamp makes an infinity finite
            const float2 x = halves(g[e]);
            g[e] = pair_of(clamped(x.x, a.clip), clamped(x.y, a.clip));
        }
    }
    const float wd = __fmul_rn(d.decay, __fmul_rn(a.lr, a.wd));
    const pair_t minus_wd = pair_of(-wd, -wd);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        m[e] = add2(mul2(m[e], a.beta1), mul2(g[e], a.omb1));
        v[e] = add2(mul2(v[e], a.beta2), mul2(mul2(g[e], g[e]), a.omb2));
        const pair_t root = root2_of(v[e]);
        const pair_t u = ratio2(mul2(m[e], now.bc1), fma2(root, now.root_bc2, a.eps));
        p[e] = fma2(minus_wd, p[e], fma2(a.minus_lr, u, p[e]));
        if (FULL) {                                  // x * 0 is 0 for every finite x, and NaN otherwise
            nan_sum = fma2(p[e], zero, nan_sum);
            if (!CODED) nan_sum = fma2(v[e], zero, nan_sum);
        } else {                                     // elements behind the end are not looked at
            const float2 x = halves(p[e]), y = halves(v[e]);
            nan_sum = fma2(pair_of(2 * e < cnt ? x.x : 0.0f, 2 * e + 1 < cnt ? x.y : 0.0f), zero, nan_sum);
            if (!CODED) nan_sum = fma2(pair_of(2 * e < cnt ? y.x : 0.0f, 2 * e + 1 < cnt ? y.y : 0.0f), zero, nan_sum);
        }
        if (CODED) v[e] = root;
    }
    if (d.p_type == SF_TYPE_F32) store8_f32<FULL>(static_cast<float *>(d.p) + at, p, cnt);
    else store8_bf16<FULL>(static_cast<uint16_t *>(d.p) + at, p, cnt);
    if (d.live) store8_bf16<FULL>(d.live + at, p, cnt);
    if (CODED) {                                     // a scale is the largest moment's: not finite where one of them is not
        const float new_sm = encode8<FULL, false>(m, d.m, at, cnt, d.m_scale + blk, lane);
        const float new_sv = encode8<FULL, true>(v, d.v, at, cnt, d.v_scale + blk, lane);
        nan_sum = fma2(pair_of(new_sm, new_sv), zero, nan_sum);
    } else {
        store8_f32<FULL>(static_cast<float *>(d.m) + at, m, cnt);
        store8_f32<FULL>(static_cast<float *>(d.v) + at, v, cnt);
    }
}

// With fp32 moments a block's loads (3.5 KB a warp) are issued behind the stores of the block before. With 8-bit moments
// they are 2 KB and the instructions (400 a block) take most of the memory's time, so four CTAs to an SM hide one another's
// waits: a block is loaded where it is used, its lines are asked for in L2 one block ahead, and the scales, which those
// lines leave out, are fetched for the whole unit at its beginning (2^26 elements over fp32 weights: 176 us, 203 with the
// scales loaded block by block, 6.1 TB/s against 5.3).
// CLIP: an element clip is on. It has instances of its own, so that steps without one do not pay for its registers (a 7B-shaped
// layer with fp32 moments 846 us; 852 with both in one).
template <int N, bool CODED, bool CLIP>
__global__ void __launch_bounds__(kThreads, CODED ? 4 : 3)
adamw_kernel(const __grid_constant__ DenseBatch<N> b, const __grid_constant__ StepArgs a, uint32_t *status)
{
    const int lane = threadIdx.x & 31, which = find_tensor(b, blockIdx.x);
    const DenseDesc &d = b.d[which];
    Place w(d, blockIdx.x - b.unit_begin[which], b.per);
    Ahead ahead(d, w);
    Block<CODED> in;
    griddep_wait();                                  // what the launches before this one wrote is there from here on
    float sms = 0.0f, svs = 0.0f;                    // 8-bit moments: lane k has the scales of the warp's k-th block
    if (CODED && lane < w.more) {
        sms = d.m_scale[w.blk + lane * kWarps];
        svs = d.v_scale[w.blk + lane * kWarps];
    }
    if (w.more > 0) {                                // before the step's own words, which take two trips to memory
        if (CODED) ahead.ask(w.left);
        else in.load(d, w);
    }
    const int t = a.step[0] + 1;
    const float f = a.factor ? a.factor[1] : 1.0f;
    if (!(f != 0.0f) || f != f) {                    // the gradient was not finite: leave everything
        if (blockIdx.x == 0 && threadIdx.x == 0) set_status(status, SF_STATUS_NONFINITE);
        return;
    }
    const int ti = t < 0 ? 0 : t < a.t_max ? t : a.t_max;
    const float bc1 = a.bc1[ti], root = __fsqrt_rn(a.bc2[ti]);
    const StepNow now = {pair_of(bc1, bc1), pair_of(root, root), pair_of(f, f)};
    pair_t nan_sum = pair_of(0.0f, 0.0f);            // stays 0 while everything is finite

    for (int k = 0; w.more > 0; ++k) {
        const int64_t at = w.at, blk = w.blk;
        const bool full = w.full();
        const int cnt = w.count();
        if (CODED) {
            if (w.more > 1) ahead.ask(w.left - kStride);
            in.load(d, w);
        }
        w.next();
        const float sm = CODED ? __shfl_sync(0xffffffffu, sms, k) : 0.0f, sv = CODED ? __shfl_sync(0xffffffffu, svs, k) : 0.0f;
        if (full) step_block<CODED, CLIP, true>(in, sm, sv, d, at, blk, 8, a, now, nan_sum);
        else step_block<CODED, CLIP, false>(in, sm, sv, d, at, blk, cnt, a, now, nan_sum);
        if (!CODED && w.more > 0) in.load(d, w);
    }
    griddep_launch_dependents();                     // the launch behind this one may take what room is left
    const float2 bad = halves(nan_sum);
    if (bad.x != 0.0f || bad.y != 0.0f) set_status(status, SF_STATUS_NONFINITE);
    // The last CTA to finish counts the step: by then every CTA has read the old count.
    if (a.last) {
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            if (atomicAdd(a.step + 1, 1) == (int)gridDim.x - 1) {
                a.step[0] = t;
                a.step[1] = 0;
            }
        }
    }
}

// A call with no elements still counts a step.
__global__ void count_step_kernel(int32_t *step, const float *factor, uint32_t *status)
{
    const float f = factor ? factor[1] : 1.0f;
    if (f != 0.0f && f == f) step[0] += 1;
    else set_status(status, SF_STATUS_NONFINITE);
}

// ws of the norm: [0] CTAs that have finished (int32, 0 between calls), then a double per CTA.
constexpr size_t kNormHeader = 16;

// This thread's elements' squares in fp64, in its order.
template <int N>
__device__ __forceinline__ double squares64(const DenseBatch<N> &b)
{
    double sum = 0.0;
    for (int unit = blockIdx.x; unit < b.units; unit += gridDim.x) {
        const int which = find_tensor(b, unit);
        const DenseDesc &d = b.d[which];
        Place w(d, unit - b.unit_begin[which], b.per);
        for (; w.more > 0; w.next()) {
            pair_t g[4];
            to_pairs(g, load_raw<false>(d.g, d.g_type, w.at, w.count()), d.g_type);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 x = halves(g[e]);
                sum = fma((double)x.x, (double)x.x, sum);
                sum = fma((double)x.y, (double)x.y, sum);
            }
        }
    }
    return sum;
}

// Sum of squares: fp32 over a lane's eight elements, fp64 from there. Every CTA leaves its sum in its own
// place; the last one of the call adds them in a fixed order. Where fp32 does not hold the squares (a thread's sum is not finite,
// or so small that squares of its elements may have been lost, and not all of them are zero), the thread sums its elements
// again in fp64. (2^26 x 3.1 bf16 elements: 74.5 us, 73.2 without the care, 77.7 with a check at each eight elements.)
template <int N>
__global__ void __launch_bounds__(kThreads)
grad_norm_kernel(const __grid_constant__ DenseBatch<N> b, int32_t *done, double *sums, int at0, int total_ctas,
                 float inv_scale, float max_norm, float *out, uint32_t *status)
{
    __shared__ double part[kWarps];
    __shared__ int is_last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double sum = 0.0;
    uint32_t any = 0;                                // a bit of some element
    griddep_wait();                                  // what the launches before this one wrote is there from here on
    for (int unit = blockIdx.x; unit < b.units; unit += gridDim.x) {
        const int which = find_tensor(b, unit);
        const DenseDesc &d = b.d[which];
        const int64_t first = ((int64_t)(unit - b.unit_begin[which]) * b.per * kWarps + warp) * kBlock + lane * kLaneElems;
        for (int k = 0; k < b.per; k += 4) {        // four blocks' loads at once
            Raw8 r[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t at = first + (int64_t)(k + q) * kStride;
                const int cnt = k + q < b.per ? (int)max((int64_t)0, min((int64_t)8, d.n - at)) : 0;
                r[q] = load_raw<false>(d.g, d.g_type, at, cnt);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                any |= r[q].a.x | r[q].a.y | r[q].a.z | r[q].a.w | r[q].b.x | r[q].b.y | r[q].b.z | r[q].b.w;
                pair_t g[4], s = pair_of(0.0f, 0.0f);
                to_pairs(g, r[q], d.g_type);
#pragma unroll
                for (int e = 0; e < 4; ++e) s = fma2(g[e], g[e], s);
                const float2 both = halves(s);
                sum += (double)__fadd_rn(both.x, both.y);
            }
        }
    }
    if (any && !(sum >= 0x1p-80 && sum <= 0x1p1000)) sum = squares64(b);
    griddep_launch_dependents();                     // the launch behind this one may take what room is left
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < kWarps; ++w) s += part[w];
        sums[at0 + blockIdx.x] = s;
        __threadfence();
        is_last = atomicAdd(done, 1) == total_ctas - 1;
    }
    __syncthreads();
    if (!is_last) return;
    __threadfence();
    sum = 0.0;
    for (int i = threadIdx.x; i < total_ctas; i += kThreads) sum += __ldcg(sums + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < kWarps; ++w) s += part[w];
        const float norm = (float)(sqrt(s) * (double)inv_scale);
        float f = inv_scale;
        if (max_norm > 0.0f) f = __fmul_rn(inv_scale, fminf(1.0f, __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f))));
        if (!isfinite(norm)) {
            f = 0.0f;
            set_status(status, SF_STATUS_NONFINITE);
        }
        out[0] = norm;
        out[1] = f;
        *done = 0;
    }
}

// ------------------------------------ host side ------------------------------------

// Elements of a call: units, of a block of 256 to a warp at least, are numbered in 32 bits. Looked at before the first launch,
// so that no call is refused half done.
constexpr int64_t kMaxElements = (int64_t)1 << 40;
static_assert(kMaxElements / (kWarps * kBlock) + SF_DENSE_PER_LAUNCH < 1 << 30, "units of a launch");

int check_dense(const sf_dense *t, int n, bool step)
{
    if (n < 0 || (n > 0 && !t)) return SF_ERR_ARG;
    int64_t room = kMaxElements;
    for (int i = 0; i < n; ++i) {
        const sf_dense &a = t[i];
        if (a.n < 0) return SF_ERR_ARG;
        if (a.n > room) return SF_ERR_UNSUPPORTED;
        room -= a.n;
        if (a.g_type != SF_TYPE_F32 && a.g_type != SF_TYPE_BF16 && a.g_type != SF_TYPE_F16) return SF_ERR_ARG;
        if (a.n > 0 && !a.g) return SF_ERR_ARG;
        if (!aligned16(a.g)) return SF_ERR_ALIGN;
        if (!step) continue;
        if (a.p_type != SF_TYPE_F32 && a.p_type != SF_TYPE_BF16) return SF_ERR_ARG;
        if (a.state_type != SF_TYPE_F32 && a.state_type != SF_TYPE_E4M3) return SF_ERR_ARG;
        if (a.n > 0 && (!a.p || !a.m || !a.v)) return SF_ERR_ARG;
        if (a.n > 0 && a.state_type == SF_TYPE_E4M3 && (!a.m_scale || !a.v_scale)) return SF_ERR_ARG;
        if (!aligned16(a.p) || !aligned16(a.m) || !aligned16(a.v) || !aligned16(a.live)) return SF_ERR_ALIGN;
        if (((uintptr_t)a.m_scale & 3) || ((uintptr_t)a.v_scale & 3)) return SF_ERR_ALIGN;
    }
    return SF_OK;
}

// Blocks of a unit per warp: what makes one round of four CTAs to an SM of a small call, and at most the kernel's own
// number. The step of 2^26 x 3.1 elements, with 2, 4, 8 and 16 blocks: fp32 moments and weights 884, 873, 890 and 907 us;
// 8-bit moments 526, 501, 514 and 528 us over fp32 weights, 457, 394, 352 and 344 us over bf16 ones, where the unit's
// beginning counts for more. The norm: 117, 76, 71 and 74 us.
constexpr int kStepBlocks = 4, kCodedBlocks = 8, kNormBlocks = 8;

int unit_blocks(const sf_dense *t, int n, int sms, int most)
{
    int64_t blocks = 0;
    for (int i = 0; i < n; ++i) blocks += (t[i].n + kBlock - 1) / kBlock;
    const int64_t round = (int64_t)sms * kWarps * 4, each = (blocks + blocks / 8 + round - 1) / round;
    return each >= most ? most : each >= 1 ? (int)each : 1;
}

// The next launch's tensors, from *at on: those with moments of the given type, or all (-1). Returns the units.
template <int N>
int64_t fill(DenseBatch<N> &b, const sf_dense *t, int n, int *at, int per, int state)
{
    b.n = 0;
    b.per = per;
    int64_t units = 0;
    for (; *at < n && b.n < N; ++*at) {
        const sf_dense &a = t[*at];
        if (a.n == 0 || (state >= 0 && a.state_type != state)) continue;
        b.unit_begin[b.n] = (int32_t)units;
        DenseDesc &d = b.d[b.n++];
        d.n = a.n;
        d.p = a.p;
        d.g = a.g;
        d.m = a.m;
        d.v = a.v;
        d.m_scale = a.m_scale;
        d.v_scale = a.v_scale;
        d.live = a.live;
        d.decay = a.decay;
        d.p_type = (uint8_t)a.p_type;
        d.g_type = (uint8_t)a.g_type;
        d.state_type = (uint8_t)a.state_type;
        d.pad = 0;
        units += (a.n + (int64_t)per * kWarps * kBlock - 1) / ((int64_t)per * kWarps * kBlock);
    }
    b.units = (int32_t)units;
    return units;
}

// Tensors with elements, with moments of the given type or of any (-1).
int full_tensors(const sf_dense *t, int n, int state)
{
    int full = 0;
    for (int i = 0; i < n; ++i) full += t[i].n > 0 && (state < 0 || t[i].state_type == state);
    return full;
}

int count_launches(const sf_dense *t, int n) { return (full_tensors(t, n, -1) + kMaxTensors - 1) / kMaxTensors; }

// Programmatic dependent launch: the kernels wait for their predecessor themselves, behind what they can do without it.
template <typename K, typename... Args>
int launch_early(K kernel, int grid, cudaStream_t stream, const Args &...args)
{
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) return SF_ERR_CUDA;
    return launch_status();
}

struct NormArgs {
    float inv_scale, max_norm;
    float *out;
    void *ws;
    uint32_t *status;
    cudaStream_t stream;
};

template <int N>
int launch_norm(const sf_dense *t, int n, int sms, const NormArgs &a)
{
    const int per = unit_blocks(t, n, sms, kNormBlocks);
    const int64_t cap = (int64_t)sms * kMaxGridPerSm;
    DenseBatch<N> b;
    // the CTAs of all launches, so that the last one of them knows itself
    int64_t total = 0;
    for (int at = 0, first = 1; first || at < n; first = 0) {
        const int64_t units = fill(b, t, n, &at, per, -1);
        if (units > 0 || first) total += units < cap ? (units > 0 ? units : 1) : cap;
    }
    int32_t *done = static_cast<int32_t *>(a.ws);
    double *sums = reinterpret_cast<double *>(static_cast<char *>(a.ws) + kNormHeader);
    int64_t placed = 0;
    for (int at = 0, first = 1; first || at < n; first = 0) {
        const int64_t units = fill(b, t, n, &at, per, -1);
        if (units == 0 && !first) continue;
        const int64_t grid = units < cap ? (units > 0 ? units : 1) : cap;
        const int rc = launch_early(grad_norm_kernel<N>, (int)grid, a.stream, b, done, sums, (int)placed, (int)total, a.inv_scale,
                                    a.max_norm, a.out, a.status);
        if (rc != SF_OK) return rc;
        placed += grid;
    }
    return SF_OK;
}

// The tensors with moments of one type; `last`: no launch of the call follows.
template <int N, bool CODED>
int launch_step(const sf_dense *t, int n, int per, bool last, StepArgs a, uint32_t *status, cudaStream_t stream)
{
    const int state = CODED ? SF_TYPE_E4M3 : SF_TYPE_F32;
    const int launches = (full_tensors(t, n, state) + N - 1) / N;
    DenseBatch<N> b;
    for (int at = 0, li = 0; li < launches; ++li) {
        const int64_t units = fill(b, t, n, &at, per, state);
        a.last = last && li == launches - 1;
        // a CTA to a unit: dealt out as SMs come free (a 7B-shaped layer with 8-bit moments, when this was chosen: 518 us
        // against 588 with eight CTAs to an SM that took units in turn)
        const int rc = launch_early(a.clip > 0.0f ? adamw_kernel<N, CODED, true> : adamw_kernel<N, CODED, false>, (int)units, stream, b, a, status);
        if (rc != SF_OK) return rc;
    }
    return SF_OK;
}

template <bool CODED>
int launch_steps(const sf_dense *t, int n, int per, bool last, const StepArgs &a, uint32_t *status, cudaStream_t stream)
{
    const int full = full_tensors(t, n, CODED ? SF_TYPE_E4M3 : SF_TYPE_F32);
    return full <= kFew ? launch_step<kFew, CODED>(t, n, per, last, a, status, stream)
           : full <= kSome ? launch_step<kSome, CODED>(t, n, per, last, a, status, stream)
                           : launch_step<kMaxTensors, CODED>(t, n, per, last, a, status, stream);
}

}  // namespace
}  // namespace sf

using namespace sf;

extern "C" size_t sf_grad_norm_ws_bytes(const sf_dense *t, int n)
{
    if (n < 0 || (n > 0 && !t)) return 0;
    const int launches = count_launches(t, n);
    // a place for every CTA of every launch, on a device of up to 256 SMs
    return kNormHeader + (size_t)(launches > 0 ? launches : 1) * 256 * kMaxGridPerSm * sizeof(double);
}

extern "C" int sf_grad_norm(const sf_dense *t, int n, float inv_scale, float max_norm, float *out, void *ws,
                            size_t ws_bytes, uint32_t *dev_status, sf_stream stream)
{
    int rc = check_dense(t, n, false);
    if (rc != SF_OK) return rc;
    if (!out || !ws || !(inv_scale > 0.0f) || max_norm != max_norm) return SF_ERR_ARG;
    if (ws_bytes < sf_grad_norm_ws_bytes(t, n)) return SF_ERR_ARG;
    if (!aligned16(ws) || ((uintptr_t)out & 3)) return SF_ERR_ALIGN;
    const int sms = sm_count();
    if (sms <= 0) return SF_ERR_NO_DEVICE;
    if (sms > 256) return SF_ERR_UNSUPPORTED;
    const NormArgs a = {inv_scale, max_norm, out, ws, dev_status, as_stream(stream)};
    const int full = full_tensors(t, n, -1);
    return full <= kFew ? launch_norm<kFew>(t, n, sms, a) : full <= kSome ? launch_norm<kSome>(t, n, sms, a)
                        : launch_norm<kMaxTensors>(t, n, sms, a);
}

extern "C" int sf_adamw_step(const sf_dense *t, int n, const sf_adam *hp, int32_t *step, const float *factor,
                             uint32_t *dev_status, sf_stream stream)
{
    int rc = check_dense(t, n, true);
    if (rc != SF_OK) return rc;
    if (!hp || !hp->bc1 || !hp->bc2 || hp->t_max < 1 || !step) return SF_ERR_ARG;
    if (((uintptr_t)step & 3) || ((uintptr_t)factor & 3)) return SF_ERR_ALIGN;
    const int sms = sm_count();
    if (sms <= 0) return SF_ERR_NO_DEVICE;
    StepArgs a;
    auto twice = [](float x) {
        uint32_t w;
        memcpy(&w, &x, 4);
        return (pair_t)w << 32 | w;
    };
    a.beta1 = twice(hp->beta1);
    a.beta2 = twice(hp->beta2);
    a.omb1 = twice(hp->one_minus_b1);
    a.omb2 = twice(hp->one_minus_b2);
    a.eps = twice(hp->eps);
    a.minus_lr = twice(-hp->lr);
    a.lr = hp->lr;
    a.wd = hp->wd;
    a.clip = hp->clip;
    a.bc1 = hp->bc1;
    a.bc2 = hp->bc2;
    a.t_max = hp->t_max;
    a.step = step;
    a.factor = factor;
    const int coded = full_tensors(t, n, SF_TYPE_E4M3), full = full_tensors(t, n, -1);
    if (full == 0) {
        count_step_kernel<<<1, 1, 0, as_stream(stream)>>>(step, factor, dev_status);
        return launch_status();
    }
    if (full > coded) {
        rc = launch_steps<false>(t, n, unit_blocks(t, n, sms, kStepBlocks), coded == 0, a, dev_status, as_stream(stream));
        if (rc != SF_OK) return rc;
    }
    return coded ? launch_steps<true>(t, n, unit_blocks(t, n, sms, kCodedBlocks), true, a, dev_status, as_stream(stream)) : SF_OK;
}
