// Gradient norm and AdamW over lists of tensors (include/rr.h: rr_grad_norm,
// rr_adamw, rr_adamw8).
//
// All three stream: every byte is touched once.  A launch takes its list of
// tensors by value in the kernel's parameters (no table in device memory to fill
// or keep; a small and a large table, as parameters are copied at each launch),
// cut into chunks of elements; a block finds a chunk's tensor by bisection.
//
// Times below are of one GB300 (152 SMs, measured copy 6.7 TB/s).
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <vector>

#include "rr_round.cuh"
#include "rr_spans.h"
#include "rr_step.h"

namespace rr {

namespace {

#define RR_TRY(expr)                  \
    do {                              \
        const rr_status st_ = (expr); \
        if (st_ != RR_OK) return st_; \
    } while (0)

constexpr int kThreads = 256;
constexpr int64_t kMaxSize = (int64_t)1 << 40;

// The chunk table of a launch.  head: elements before the first one at which
// every pointer of the tensor is aligned for a vector (kNoVector: there is none).
constexpr int kNoVector = -1;
template <int CAP>
struct Chunks {
    int64_t start[CAP + 1];  // first chunk of each tensor; start[count] = all
    int64_t size[CAP];
    int8_t head[CAP];
    int count;
    __device__ __forceinline__ int find(int64_t chunk) const
    {
        int lo = 0, hi = count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= chunk) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    // Blocks take equal stretches of chunks, so that a block's search is one
    // bisection and then a step now and then.
    __device__ __forceinline__ int64_t stretch(int64_t i) const { return start[count] * i / gridDim.x; }
};

// ---------------------------------------------------------------- gradient norm
constexpr int kNormCapSmall = 32, kNormCap = 1200;
constexpr int kNormUnroll = 8;
constexpr int kNormBlocks = 1024;  // most blocks of one launch, one partial sum each
// Up to so many chunks one block takes the list and finishes the norm itself.
constexpr int kNormAlone = 2;

struct GradNormEndArgs {
    const double *part;
    int64_t count;
    float inv_scale, max_norm;
    float *norm, *scale;
};

// Norm and scale from the sum of squares (one thread).
__device__ __forceinline__ void grad_norm_finish(const GradNormEndArgs &a, double sum)
{
    const float norm = (float)(sqrt(sum) * (double)a.inv_scale);
    const float clip = a.max_norm / (norm + 1e-6f);
    if (a.norm) *a.norm = norm;
    if (a.scale) *a.scale = isfinite(norm) ? a.inv_scale * fminf(1.0f, clip) : __int_as_float(0x7fc00000);
}

template <int CAP>
struct GradNormArgs {
    Chunks<CAP> list;
    const void *g[CAP];
    double *part;  // this launch's partial sums
    bool alone;    // its one block has the whole list: it finishes the norm itself
    GradNormEndArgs end;
};

// The sum of squares.  A thread takes 8 vectors of a chunk at once; their sum
// goes to a compensated sum, the threads' sums to binary64, the blocks' partial
// sums, in order, to a last block.
//
// Sums of squares in [2^-90, 2^90] are sound in binary32: every square that
// underflowed is below 2^-126 and lost in the sum's own rounding, and 2^30 such
// sums stay finite.  A thread's sum of a chunk that lies outside (zeros aside)
// is taken again in binary64; NaN fails the comparison and goes there too.
//
// Bound: HBM.  A layer of 233M bf16 gradients 69.7 us, the measured copy peak
// (with a range check for each vector and chunks dealt out in turn 120 and 74);
// 60M in 100 odd tensors 23 us (77 %: partial chunks at the tensors' ends); two
// tensors of 3584 4.4 us (latency, one launch).
__device__ __forceinline__ bool sound(float sum) { return sum >= 0x1p-90f && sum <= 0x1p90f; }

template <class T, int CAP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ GradNormArgs<CAP> a)
{
    stream_order();
    constexpr int E = 16 / (int)sizeof(T);
    constexpr int64_t C = (int64_t)kThreads * E * kNormUnroll;
    __shared__ double s[kThreads / 32];
    Compensated chunks;
    double wide = 0.0;
    const int64_t end = a.list.stretch(blockIdx.x + 1);
    int64_t chunk = a.list.stretch(blockIdx.x);
    for (int t = a.list.find(chunk); chunk < end; ++chunk) {
        while (chunk >= a.list.start[t + 1]) ++t;
        const T *g = static_cast<const T *>(a.g[t]);
        const int64_t n = a.list.size[t], c = chunk - a.list.start[t];
        const int head = a.list.head[t];
        const int64_t e0 = head + c * C + (int64_t)threadIdx.x * E;
        Pack<T, E> v[kNormUnroll];
        if (head + (c + 1) * C <= n) {
#pragma unroll
            for (int j = 0; j < kNormUnroll; ++j)
                v[j] = *reinterpret_cast<const Pack<T, E> *>(g + e0 + j * kThreads * E);
        } else {
#pragma unroll
            for (int j = 0; j < kNormUnroll; ++j) {
                const int64_t e = e0 + (int64_t)j * kThreads * E;
                if (e + E <= n) {
                    v[j] = *reinterpret_cast<const Pack<T, E> *>(g + e);
                } else {
#pragma unroll
                    for (int k = 0; k < E; ++k) v[j].v[k] = e + k < n ? g[e + k] : from_f32<T>(0.0f);
                }
            }
        }
        float2 acc[2] = {both(0.0f), both(0.0f)};
#pragma unroll
        for (int j = 0; j < kNormUnroll; ++j) {
#pragma unroll
            for (int k = 0; k < E; k += 2) {
                const float2 x = pair_f32(&v[j].v[k]);
                acc[j & 1] = fma2(x, x, acc[j & 1]);
            }
        }
        acc[0] = add2(acc[0], acc[1]);
        float sum = acc[0].x + acc[0].y;
        if (!sound(sum)) {
            sum = 0.0f;
            uint32_t any = 0;
#pragma unroll
            for (int j = 0; j < kNormUnroll; ++j) {
                const uint4 x = *reinterpret_cast<const uint4 *>(&v[j]);
                any |= x.x | x.y | x.z | x.w;
            }
            if (any & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu)) {
#pragma unroll
                for (int j = 0; j < kNormUnroll; ++j) {
#pragma unroll
                    for (int k = 0; k < E; ++k) wide += (double)to_f32(v[j].v[k]) * to_f32(v[j].v[k]);
                }
            }
        }
        if (c == 0 && (int)threadIdx.x < head && (int64_t)threadIdx.x < n) {
            const float x = to_f32(g[threadIdx.x]);
            if (sound(x * x)) sum = fmaf(x, x, sum);
            else wide += (double)x * x;
        }
        chunks.add(sum);
    }
    double d = wide + (double)chunks.hi + (double)chunks.lo;
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
        d = 0.0;
        for (int i = 0; i < kThreads / 32; ++i) d += s[i];
        if (a.alone) grad_norm_finish(a.end, d);
        else a.part[blockIdx.x] = d;
    }
}

__global__ void __launch_bounds__(kThreads) grad_norm_end_kernel(const __grid_constant__ GradNormEndArgs a)
{
    stream_order();
    __shared__ double s[kThreads / 32];
    double d = 0.0;
    for (int64_t i = threadIdx.x; i < a.count; i += kThreads) d += a.part[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = d;
    __syncthreads();
    if (threadIdx.x == 0) {
        d = 0.0;
        for (int i = 0; i < kThreads / 32; ++i) d += s[i];
        grad_norm_finish(a, d);
    }
}

// ---------------------------------------------------------------- AdamW
constexpr int kAdamCapSmall = 32, kAdamCap = 400;
constexpr int kUnit = 4;   // elements of a vector: 16 bytes of binary32, 8 of the 16-bit types
constexpr int kUnits = 4;  // vectors of a thread in a chunk
constexpr int64_t kAdamChunk = (int64_t)kThreads * kUnit * kUnits;

struct AdamScalars {
    float beta1, omb1, beta2, omb2;  // beta and 1 - beta
    float decay;                     // 1 - lr * weight_decay
    float inv_c2;                    // 1 / sqrt(1 - beta2^step)
    float step_size;                 // lr / (1 - beta1^step)
    float eps;
    float minus_zero;                // -0, for mul2_apart
    uint32_t one;                    // 1, where a multiply-add may not become an addition
    float root_most;                 // largest sqrt(v) of adamw8_block's fast quotients (-1: none)
    const float *scale;
};

template <int CAP>
struct AdamArgs {
    Chunks<CAP> list;
    void *p[CAP];
    const void *g[CAP];
    float *m[CAP], *v[CAP], *w[CAP];
    AdamScalars h;
};

// One element.  Every operation rounds by itself (no fused multiply-add), so
// that the result is the formula's, operation by operation, whatever the
// compiler contracts.
__device__ __forceinline__ float adam_element(const AdamScalars &h, float scale, float w, float g, float &m, float &v,
                                              float &root)
{
    g = __fmul_rn(g, scale);
    m = __fadd_rn(__fmul_rn(m, h.beta1), __fmul_rn(g, h.omb1));
    v = __fadd_rn(__fmul_rn(v, h.beta2), __fmul_rn(__fmul_rn(g, h.omb2), g));
    root = __fsqrt_rn(v);
    const float den = __fadd_rn(__fmul_rn(root, h.inv_c2), h.eps);
    return __fsub_rn(__fmul_rn(w, h.decay), __fmul_rn(__fdiv_rn(m, den), h.step_size));
}

// A thread has four vectors of four elements of a chunk; the loads of all streams
// are issued before the first is used.  Tensors whose pointers are not aligned
// alike go element by element.  Bound: HBM (7 streams with master weights).  One
// rank's shard of a layer, 29M bf16 weights with masters, 130 us, 6.3 TB/s, 93 % of
// the copy peak; 30M binary32 138 us (91 %); 7M in 61 tensors packed at any element
// 34.6 us (84 %); 30M whose pointers are not aligned alike 309 us with masters, 314
// in binary32 (40 %).  Two vectors a thread took 160 us for the shard.
template <class P, class G, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamArgs<CAP> a)
{
    stream_order();
    const AdamScalars &h = a.h;
    const float scale = h.scale ? *h.scale : 1.0f;
    if (scale != scale) return;
    const int64_t total = a.list.start[a.list.count];
    for (int64_t chunk = blockIdx.x; chunk < total; chunk += gridDim.x) {
        const int t = a.list.find(chunk);
        const int64_t n = a.list.size[t], c = chunk - a.list.start[t];
        const int head = a.list.head[t];
        P *p = static_cast<P *>(a.p[t]);
        const G *g = static_cast<const G *>(a.g[t]);
        float *m = a.m[t], *v = a.v[t], *w = MASTER ? a.w[t] : nullptr;
        auto one = [&](int64_t e) {
            float me = m[e], ve = v[e], root;
            const float x = adam_element(h, scale, MASTER ? w[e] : to_f32(p[e]), to_f32(g[e]), me, ve, root);
            m[e] = me;
            v[e] = ve;
            if (MASTER) w[e] = x;
            p[e] = from_f32<P>(x);
        };
        if (head == kNoVector) {
            const int64_t end = (c + 1) * kAdamChunk < n ? (c + 1) * kAdamChunk : n;
#pragma unroll 4
            for (int64_t e = c * kAdamChunk + threadIdx.x; e < end; e += kThreads) one(e);
            continue;
        }
        if (c == 0 && (int)threadIdx.x < head && (int64_t)threadIdx.x < n) one(threadIdx.x);
        const int64_t e0 = head + c * kAdamChunk + (int64_t)threadIdx.x * kUnit;
        Pack<P, kUnit> pv[kUnits];
        Pack<G, kUnit> gv[kUnits];
        Pack<float, kUnit> mv[kUnits], vv[kUnits], wv[kUnits];
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int64_t e = e0 + (int64_t)j * kThreads * kUnit;
            if (e + kUnit <= n) {
                if (MASTER) wv[j] = *reinterpret_cast<const Pack<float, kUnit> *>(w + e);
                else pv[j] = *reinterpret_cast<const Pack<P, kUnit> *>(p + e);
                gv[j] = *reinterpret_cast<const Pack<G, kUnit> *>(g + e);
                mv[j] = *reinterpret_cast<const Pack<float, kUnit> *>(m + e);
                vv[j] = *reinterpret_cast<const Pack<float, kUnit> *>(v + e);
            }
        }
#pragma unroll
        for (int j = 0; j < kUnits; ++j) {
            const int64_t e = e0 + (int64_t)j * kThreads * kUnit;
            if (e + kUnit <= n) {
#pragma unroll
                for (int k = 0; k < kUnit; ++k) {
                    float root;
                    const float x = adam_element(h, scale, MASTER ? wv[j].v[k] : to_f32(pv[j].v[k]), to_f32(gv[j].v[k]),
                                                 mv[j].v[k], vv[j].v[k], root);
                    if (MASTER) wv[j].v[k] = x;
                    pv[j].v[k] = from_f32<P>(x);
                }
                if (MASTER) *reinterpret_cast<Pack<float, kUnit> *>(w + e) = wv[j];
                *reinterpret_cast<Pack<P, kUnit> *>(p + e) = pv[j];
                *reinterpret_cast<Pack<float, kUnit> *>(m + e) = mv[j];
                *reinterpret_cast<Pack<float, kUnit> *>(v + e) = vv[j];
            } else {
                for (int64_t k = e; k < n; ++k) one(k);
            }
        }
    }
}

// ---------------------------------------------------------------- AdamW, 8-bit states
// A warp has one block of 256 elements, 8 to a lane: the block's largest
// magnitude is one warp-wide maximum, and states go from codes to codes in
// registers.
constexpr int kBlock = RR_ADAMW8_BLOCK;
constexpr int kLane = kBlock / 32;
constexpr int kAdam8Run = 16;  // most blocks of a run
// Blocks of a warp in flight or in use.  With 4-byte weights the 6 leave one
// thread block to an SM and are faster for it: 60M binary32 weights 160 us, with
// 5 (two thread blocks) 168; a bf16 layer 435 with 5, 446 with 4 or 6.
__host__ __device__ constexpr int adam8_stages(int weight_bytes) { return weight_bytes == 4 ? 6 : 5; }

template <int CAP>
struct Adam8Args {
    Chunks<CAP> list;  // chunk = block of kBlock elements
    void *p[CAP];
    const void *g[CAP];
    uint8_t *m[CAP], *r[CAP];
    float *ms[CAP], *rs[CAP], *w[CAP];
    AdamScalars h;
    uint32_t seed, first;  // first: index in the caller's list of this launch's first tensor
};

// Xor-shifts and odd multipliers: shifts and first multiplier after C. Wellons,
// "Prospecting for Hash Functions" (2018), with another second one.
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x7FEB352Du;
    x ^= x >> 15;
    x *= 0x68E31DA5u;
    return x ^ (x >> 16);
}

// Power-of-two scale of a block from the bits of its largest magnitude, as bits:
// the magnitude over the scale lies in [128, 256), or the scale is 2^-126.  Its
// reciprocal has the mirrored exponent.
__device__ __forceinline__ uint32_t scale_bits(uint32_t top) { return max(top & 0x7F800000u, 0x04000000u) - 0x03800000u; }
__device__ __forceinline__ float reciprocal(uint32_t scale) { return __uint_as_float(0x7F000000u - scale); }

// |x| / scale on the code's grid, up or down by the 16 random bits u: adding
// them just below the last kept mantissa bit and cutting there rounds up with
// the probability of the part cut off.  Below 2^-6 the grid is even, as that
// of values in [2^-6, 2^-5); lifting by 2^-6 makes it theirs.
__device__ __forceinline__ float round_to_code(float t, uint32_t u)
{
    const float lift = t < 0x1p-6f ? 0x1p-6f : 0.0f;
    const uint32_t bits = (__float_as_uint(__fadd_rn(t, lift)) + (u << 4) + 8u) & 0xFFF00000u;
    return __fsub_rn(__uint_as_float(bits), lift);
}
// The same for |x| / scale of at least 2^-6, sign and all.  `half`: 0x10 adds
// 16 times the low 16 bits of u, 0x1000 the high ones (a two-way dot product
// picks the half, shifts and adds at once); the 8 comes through a multiply-add,
// which runs beside the logic units that the rest of the rounding keeps busy.
__device__ __forceinline__ float cut_to_code(float t, uint32_t u, uint32_t half, const AdamScalars &h)
{
    return __uint_as_float(__dp2a_lo(u, half, __float_as_uint(t) * h.one + 8u) & 0xFFF00000u);
}
// A positive root is stored as no less than the smallest code.
__device__ __forceinline__ float floor_code(float t) { return t > 0.0f ? fmaxf(t, 0x1p-9f) : t; }
// 32 random bits of element `step` after the one whose product with kWeyl,
// plus the tensor's key, is `base`.  One multiplication makes each element's bits
// even over the seeds, not independent of other elements' of the same step: the
// high halves of elements 58678 apart correlate at 0.5, those 305 apart at 0.07.
constexpr uint32_t kWeyl = 0x9E3779B1u;
__device__ __forceinline__ uint32_t dither(uint32_t base, uint32_t step)
{
    uint32_t u = base + step * kWeyl;
    u ^= u >> 16;
    u *= 0x7FEB352Du;
    return u ^ (u >> 15);
}
__device__ __forceinline__ uint16_t to_codes(float lo, float hi)
{
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
    return c;
}
__device__ __forceinline__ float2 from_codes(uint16_t c)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// What a lane holds of a block: 8 elements in a row (VEC) or every 32nd, in
// memory's types until they are used, so that the next block's loads cost few
// registers.
template <class W, class G, bool VEC>
struct Lane8 {
    Pack<W, kLane> w;
    Pack<G, kLane> g;
    uint2 m, r;

    static __device__ __forceinline__ int element(int k, int lane) { return VEC ? lane * kLane + k : k * 32 + lane; }
    static __device__ __forceinline__ uint32_t after(int k) { return VEC ? k : k * 32; }  // element(k) - element(0)

    template <class T>
    static __device__ __forceinline__ void load(Pack<T, kLane> &x, const T *p, int lane, int left)
    {
        if (VEC) {
            constexpr int E = 16 / (int)sizeof(T);
            const Pack<T, E> *v = reinterpret_cast<const Pack<T, E> *>(p + lane * kLane);
#pragma unroll
            for (int j = 0; j < kLane / E; ++j) reinterpret_cast<Pack<T, E> *>(&x)[j] = v[j];
        } else {
#pragma unroll
            for (int k = 0; k < kLane; ++k) {
                const int e = element(k, lane);
                x.v[k] = e < left ? p[e] : from_f32<T>(0.0f);
            }
        }
    }
    static __device__ __forceinline__ uint2 load(const uint8_t *p, int lane, int left)
    {
        if (VEC) return *reinterpret_cast<const uint2 *>(p + lane * kLane);
        uint32_t c[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
            const int e = element(k, lane);
            c[k / 4] |= (e < left ? (uint32_t)p[e] : 0u) << 8 * (k % 4);
        }
        return make_uint2(c[0], c[1]);
    }
    template <class T>
    static __device__ __forceinline__ void store(T *p, const float2 (&x)[kLane / 2], int lane, int left)
    {
        if (VEC) {
            Pack<T, kLane> y;
#pragma unroll
            for (int k = 0; k < kLane; k += 2) pair_set(&y.v[k], x[k / 2]);
            constexpr int E = 16 / (int)sizeof(T);
            Pack<T, E> *v = reinterpret_cast<Pack<T, E> *>(p + lane * kLane);
#pragma unroll
            for (int j = 0; j < kLane / E; ++j) v[j] = reinterpret_cast<Pack<T, E> *>(&y)[j];
        } else {
#pragma unroll
            for (int k = 0; k < kLane; ++k) {
                const int e = element(k, lane);
                if (e < left) p[e] = from_f32<T>(k & 1 ? x[k / 2].y : x[k / 2].x);
            }
        }
    }
    static __device__ __forceinline__ void store(uint8_t *p, const float2 (&x)[kLane / 2], int lane, int left)
    {
        uint16_t c[kLane / 2];
#pragma unroll
        for (int k = 0; k < kLane / 2; ++k) c[k] = to_codes(x[k].x, x[k].y);
        if (VEC) {
            *reinterpret_cast<uint2 *>(p + lane * kLane) =
                make_uint2((uint32_t)c[0] | (uint32_t)c[1] << 16, (uint32_t)c[2] | (uint32_t)c[3] << 16);
        } else {
#pragma unroll
            for (int k = 0; k < kLane; ++k) {
                const int e = element(k, lane);
                if (e < left) p[e] = (uint8_t)(c[k / 2] >> 8 * (k & 1));
            }
        }
    }
    // W is the master weight's type where there is one, else the parameter's.
    __device__ __forceinline__ void load(const W *wp, const G *gp, const uint8_t *mp, const uint8_t *rp, int lane, int left)
    {
        load(w, wp, lane, left);
        load(g, gp, lane, left);
        m = load(mp, lane, left);
        r = load(rp, lane, left);
    }

    // Whole blocks come through a ring in shared memory, kStages blocks of a
    // warp's run deep: weights, gradients, codes, one after the other.
    static __device__ __forceinline__ constexpr int w_bytes() { return kBlock * (int)sizeof(W); }
    static __device__ __forceinline__ constexpr int g_bytes() { return kBlock * (int)sizeof(G); }
    static __device__ __forceinline__ constexpr int stage_bytes() { return w_bytes() + g_bytes() + 2 * kBlock; }
    static __device__ __forceinline__ void fetch(char *s, const W *wp, const G *gp, const uint8_t *mp, const uint8_t *rp,
                                                 int lane)
    {
#pragma unroll
        for (int j = 0; j < w_bytes(); j += 512) fetch16(s + j + lane * 16, reinterpret_cast<const char *>(wp) + j + lane * 16);
#pragma unroll
        for (int j = 0; j < g_bytes(); j += 512) fetch16(s + w_bytes() + j + lane * 16, reinterpret_cast<const char *>(gp) + j + lane * 16);
        fetch8(s + w_bytes() + g_bytes() + lane * 8, mp + lane * 8);
        fetch8(s + w_bytes() + g_bytes() + kBlock + lane * 8, rp + lane * 8);
    }
    __device__ __forceinline__ void take(const char *s, int lane)
    {
        load(w, reinterpret_cast<const W *>(s), lane, kBlock);
        load(g, reinterpret_cast<const G *>(s + w_bytes()), lane, kBlock);
        m = load(reinterpret_cast<const uint8_t *>(s + w_bytes() + g_bytes()), lane, kBlock);
        r = load(reinterpret_cast<const uint8_t *>(s + w_bytes() + g_bytes() + kBlock), lane, kBlock);
    }
};

__device__ __forceinline__ uint32_t warp_max(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
// max(|a|, |b|, |c|), NaN if one is; min(a, b, c) and min(|a|, |b|, |c|) of what is not NaN.
__device__ __forceinline__ float top3(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float low3(float a, float b, float c)
{
    float d;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float low3_abs(float a, float b, float c)
{
    float d;
    asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float2 codes_of(uint2 c, int k)
{
    const uint32_t word = k < 2 ? c.x : c.y;
    return from_codes((uint16_t)(k & 1 ? word >> 16 : word));
}

// One block of one tensor, loaded before: its step, weights and states stored.
template <class P, class W, class G, bool MASTER, bool VEC>
__device__ __forceinline__ void adamw8_block(const AdamScalars &h, float scale, uint32_t base, const Lane8<W, G, VEC> &in,
                                             float &mscale, float &rscale, P *p, float *master, uint8_t *mp, uint8_t *rp,
                                             int lane, int left)
{
    using L = Lane8<W, G, VEC>;
    float2 w[kLane / 2], m[kLane / 2], r[kLane / 2], v[kLane / 2];
    // A code times its power-of-two scale is exact.
    const float2 ms = both(mscale), rs = both(rscale), b1 = both(h.beta1), b2 = both(h.beta2), nz = both(h.minus_zero);
    float mtop = 0.0f, mlow = 3e38f, rtop = 0.0f, rlow = 3e38f;
#pragma unroll
    for (int k = 0; k < kLane / 2; ++k) {
        const float2 g = mul2(pair_f32(&in.g.v[2 * k]), both(scale));
        m[k] = add2(mul2_apart(mul2(codes_of(in.m, k), ms), b1, nz), mul2_apart(g, both(h.omb1), nz));
        r[k] = mul2(codes_of(in.r, k), rs);
        v[k] = add2(mul2_apart(mul2(r[k], r[k]), b2, nz), mul2_apart(mul2(g, both(h.omb2)), g, nz));
        mtop = top3(mtop, m[k].x, m[k].y);
        mlow = low3_abs(mlow, m[k].x, m[k].y);
        w[k] = pair_f32(&in.w.v[2 * k]);
        r[k] = root2(v[k], mul2(v[k], both(-1.0f)));
        rtop = top3(rtop, r[k].x, r[k].y);
        rlow = low3(rlow, r[k].x, r[k].y);
    }
    // The fast roots and quotients round as sqrt and / do while their operands
    // keep away from binary32's ends (a root that does not comes out as NaN,
    // below 2^-50 or above 2^50) and the quotient is normal: it is at most m over
    // the root, and at least 2^-100 over 2^25.  A lane with an operand that does
    // not, a v of 0 among them, takes sqrt and / for all 8.
    if (mlow < 0x1p-100f) {  // an m of 0 is no small one: its quotient is 0
        mlow = 3e38f;
#pragma unroll
        for (int k = 0; k < kLane / 2; ++k) {
            if (m[k].x != 0.0f) mlow = fminf(mlow, fabsf(m[k].x));
            if (m[k].y != 0.0f) mlow = fminf(mlow, fabsf(m[k].y));
        }
    }
    const float2 decay = both(h.decay), size = both(-h.step_size);
    if (rlow >= 0x1p-50f && rtop <= h.root_most && mlow >= 0x1p-100f && mtop <= fminf(rlow, 1.0f) * 0x1p100f) {
        const float2 nc2 = both(-h.inv_c2), neps = both(-h.eps);
#pragma unroll
        for (int k = 0; k < kLane / 2; ++k) {
            const float2 q = quotient2(m[k], add2(mul2_apart(r[k], nc2, nz), neps));
            w[k] = add2(mul2_apart(w[k], decay, nz), mul2_apart(q, size, nz));
        }
    } else {
        rtop = 0.0f;
#pragma unroll
        for (int k = 0; k < kLane / 2; ++k) {
            r[k] = make_float2(__fsqrt_rn(v[k].x), __fsqrt_rn(v[k].y));
            rtop = top3(rtop, r[k].x, r[k].y);
            const float2 den = add2(mul2_apart(r[k], both(h.inv_c2), nz), both(h.eps));
            w[k] = add2(mul2_apart(w[k], decay, nz), mul2_apart(make_float2(__fdiv_rn(m[k].x, den.x), __fdiv_rn(m[k].y, den.y)), size, nz));
        }
    }
    if (MASTER) L::store(master, w, lane, left);
    L::store(p, w, lane, left);

    // bits of magnitudes order as they do, NaN above all
    const uint32_t mbits = warp_max(__float_as_uint(mtop)), rbits = warp_max(__float_as_uint(rtop));
    const bool mfine = mbits < 0x7F800000u, rfine = rbits < 0x7F800000u;
    const uint32_t me = scale_bits(mbits), re = scale_bits(rbits);
    const float2 minv = both(reciprocal(me)), rinv = both(reciprocal(re));
    // (x / scale) on the code's grid: adding random bits just below the last
    // kept mantissa bit and cutting there rounds up with the probability of the
    // part cut off.  Signs stay out of it.
    float low = 3e38f;
    float2 mq[kLane / 2], rq[kLane / 2];
#pragma unroll
    for (int k = 0; k < kLane / 2; ++k) {
        m[k] = mul2(m[k], minv);
        r[k] = mul2(r[k], rinv);
        low = low3_abs(low3_abs(low, m[k].x, m[k].y), r[k].x, r[k].y);
        const uint32_t u0 = dither(base, L::after(2 * k)), u1 = dither(base, L::after(2 * k + 1));
        mq[k] = make_float2(cut_to_code(m[k].x, u0, 0x10u, h), cut_to_code(m[k].y, u1, 0x10u, h));
        rq[k] = make_float2(cut_to_code(r[k].x, u0, 0x1000u, h), cut_to_code(r[k].y, u1, 0x1000u, h));
    }
    // Below 2^-6 the grid is even; a lane with such a value (or a block that is
    // not finite) takes the long way.
    if (!(low >= 0x1p-6f) || !mfine || !rfine) {
#pragma unroll
        for (int k = 0; k < kLane / 2; ++k) {
            const uint32_t u0 = dither(base, L::after(2 * k)), u1 = dither(base, L::after(2 * k + 1));
            mq[k] = make_float2(copysignf(round_to_code(fabsf(m[k].x), u0 & 0xFFFFu), m[k].x),
                                copysignf(round_to_code(fabsf(m[k].y), u1 & 0xFFFFu), m[k].y));
            rq[k] = make_float2(round_to_code(floor_code(r[k].x), u0 >> 16), round_to_code(floor_code(r[k].y), u1 >> 16));
            if (!mfine) mq[k] = both(0.0f);
            if (!rfine) rq[k] = both(0.0f);
        }
    }
    L::store(mp, mq, lane, left);
    L::store(rp, rq, lane, left);
    const float nan = __int_as_float(0x7fc00000);
    mscale = mfine ? __uint_as_float(me) : nan;
    rscale = rfine ? __uint_as_float(re) : nan;
}

// Warps take equal stretches of the list's blocks, in runs of up to kAdam8Run of
// one tensor.  Lane i holds the scales of the run's block i, so that they are read
// and written together.
//
// Bound: instruction issue (74 % of the slots in use, about 55 instructions an
// element), then HBM.  A layer of 233M bf16 weights 437 us, 5.4 TB/s, 80 % of the
// copy peak: with sqrt and / of their own, one operation at a time, 906; those two
// at a time and corrected 594; the ring 455; the dither's halves by a dot product
// 446; runs in equal stretches 435; a look at the least m, and its code's scale
// apart from beta1, 2 more.  60M bf16 weights with masters 178 us (91 %), 60M
// binary32 156 us (92 %); runs of 32 dealt out in turn, uneven at the end, 185 and
// 161 (before that look).
//
// What a lane finds costs: 60M bf16 weights 121 us when a block's values are of one
// size, 135 when they spread log-normally (sigma 1), 141 with one value a hundred
// times the others in each block (values below 2^-6 of the code's range are rounded
// again), 315 when every tenth gradient has always been 0, 293 when all have (a v of
// 0 takes sqrt and / of their own).  Tensors off a 16-byte boundary go element by
// element: 175, with masters 236 (aligned 171), binary32 367 (158).
template <class P, class G, bool MASTER, int CAP>
__global__ void __launch_bounds__(kThreads) adamw8_kernel(const __grid_constant__ Adam8Args<CAP> a)
{
    stream_order();
    using W = typename std::conditional<MASTER, float, P>::type;
    using L = Lane8<W, G, true>;
    constexpr int kAdam8Stages = adam8_stages(sizeof(W));
    extern __shared__ uint4 s_ring[];
    const float scale = a.h.scale ? *a.h.scale : 1.0f;
    if (scale != scale) return;
    // one value in the warp, so that what follows from it is too
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
    char *const ring = reinterpret_cast<char *>(s_ring) + warp * kAdam8Stages * L::stage_bytes();
    const int64_t total = a.list.start[a.list.count], warps = (int64_t)gridDim.x * (kThreads / 32);
    const int64_t mine = (int64_t)blockIdx.x * (kThreads / 32) + warp, end = total * (mine + 1) / warps;
    int64_t from = total * mine / warps;
    for (int t = a.list.find(from); from < end;) {
        while (from >= a.list.start[t + 1]) ++t;
        const int64_t b = from - a.list.start[t], at = b * kBlock, left = a.list.size[t] - at;
        const int blocks = (int)min((int64_t)kAdam8Run, min(end, a.list.start[t + 1]) - from);
        const int whole = a.list.head[t] == 0 ? (int)min((int64_t)blocks, left / kBlock) : 0;
        from += blocks;
        P *p = static_cast<P *>(a.p[t]) + at;
        const G *g = static_cast<const G *>(a.g[t]) + at;
        uint8_t *m = a.m[t] + at, *r = a.r[t] + at;
        float *ms = a.ms[t] + b, *rs = a.rs[t] + b, *master = MASTER ? a.w[t] + at : nullptr;
        const W *w = MASTER ? reinterpret_cast<const W *>(master) : reinterpret_cast<const W *>(p);
        const uint32_t start = (uint32_t)at * kWeyl + mix32(a.seed + (a.first + (uint32_t)t + 1u) * 0x9E3779B9u);
        float mscales = 0.0f, rscales = 0.0f;
        if (lane < blocks) {
            mscales = ms[lane];
            rscales = rs[lane];
        }
        auto fetch = [&](int i) {
            if (i < whole) {
                const int e = i * kBlock;
                L::fetch(ring + i % kAdam8Stages * L::stage_bytes(), w + e, g + e, m + e, r + e, lane);
            }
            fetch_commit();
        };
#pragma unroll
        for (int i = 0; i < kAdam8Stages - 1; ++i) fetch(i);
        for (int i = 0; i < blocks; ++i) {
            const int e = i * kBlock;
            float msc = __shfl_sync(0xffffffffu, mscales, i), rsc = __shfl_sync(0xffffffffu, rscales, i);
            float *const master_at = MASTER ? master + e : nullptr;
            if (i < whole) {
                // block i has landed for every lane, and every lane is done with block i - 1
                fetch_wait<kAdam8Stages - 2>();
                __syncwarp();
                fetch(i + kAdam8Stages - 1);
                L cur;
                cur.take(ring + i % kAdam8Stages * L::stage_bytes(), lane);
                adamw8_block<P, W, G, MASTER, true>(a.h, scale, start + (e + L::element(0, lane)) * kWeyl, cur, msc, rsc, p + e,
                                                    master_at, m + e, r + e, lane, kBlock);
            } else {
                const int n = left - e < kBlock ? (int)(left - e) : kBlock;
                Lane8<W, G, false> cur;
                cur.load(w + e, g + e, m + e, r + e, lane, n);
                adamw8_block<P, W, G, MASTER, false>(a.h, scale, start + (e + Lane8<W, G, false>::element(0, lane)) * kWeyl,
                                                     cur, msc, rsc, p + e, master_at, m + e, r + e, lane, n);
            }
            if (lane == i) {
                mscales = msc;
                rscales = rsc;
            }
        }
        if (lane < blocks) {
            ms[lane] = mscales;
            rs[lane] = rscales;
        }
        __syncwarp();  // the next run refills the ring
    }
}

// ---------------------------------------------------------------- host side
rr_status check_list(const int64_t *sizes, int count)
{
    if (count < 0) return step_fail(RR_ERR_INVALID_ARG, "num_tensors %d", count);
    if (count > 0 && !sizes) return step_fail(RR_ERR_INVALID_ARG, "sizes is NULL");
    for (int i = 0; i < count; ++i)
        if (sizes[i] < 0 || sizes[i] > kMaxSize)
            return step_fail(RR_ERR_INVALID_ARG, "sizes[%d] is %lld", i, (long long)sizes[i]);
    return RR_OK;
}
rr_status check_pointers(const char *name, const void *const *p, const int64_t *sizes, int count, int bytes)
{
    if (count > 0 && !p) return step_fail(RR_ERR_INVALID_ARG, "%s is NULL", name);
    for (int i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        if (!p[i]) return step_fail(RR_ERR_INVALID_ARG, "%s[%d] is NULL", name, i);
        if (!aligned_to(p[i], bytes))
            return step_fail(RR_ERR_ALIGNMENT, "%s[%d] not aligned to its %d-byte element", name, i, bytes);
    }
    return RR_OK;
}
template <class T>
const void *const *plain(T *const *p) { return reinterpret_cast<const void *const *>(p); }

// Elements before p's first `unit`-element boundary.
int elements_before(const void *p, int bytes, int unit)
{
    const int past = (int)(reinterpret_cast<uintptr_t>(p) % (uintptr_t)(bytes * unit));
    return past == 0 ? 0 : (bytes * unit - past) / bytes;
}

rr_status check_hyper(const rr_adamw_hyper *h)
{
    if (!h) return step_fail(RR_ERR_INVALID_ARG, "hyper is NULL");
    if (!(h->beta1 >= 0.0 && h->beta1 < 1.0)) return step_fail(RR_ERR_INVALID_ARG, "beta1 %g", h->beta1);
    if (!(h->beta2 >= 0.0 && h->beta2 < 1.0)) return step_fail(RR_ERR_INVALID_ARG, "beta2 %g", h->beta2);
    if (!(h->lr >= 0.0)) return step_fail(RR_ERR_INVALID_ARG, "lr %g", h->lr);
    if (!(h->eps >= 0.0)) return step_fail(RR_ERR_INVALID_ARG, "eps %g", h->eps);
    if (!(h->weight_decay >= 0.0)) return step_fail(RR_ERR_INVALID_ARG, "weight_decay %g", h->weight_decay);
    if (h->step < 1) return step_fail(RR_ERR_INVALID_ARG, "step %lld: steps count from 1", (long long)h->step);
    return RR_OK;
}
AdamScalars scalars(const rr_adamw_hyper &h, const float *scale)
{
    AdamScalars s;
    s.beta1 = (float)h.beta1;
    s.omb1 = (float)(1.0 - h.beta1);
    s.beta2 = (float)h.beta2;
    s.omb2 = (float)(1.0 - h.beta2);
    s.decay = (float)(1.0 - h.lr * h.weight_decay);
    s.inv_c2 = (float)(1.0 / std::sqrt(1.0 - std::pow(h.beta2, (double)h.step)));
    s.step_size = (float)(h.lr / (1.0 - std::pow(h.beta1, (double)h.step)));
    s.eps = (float)h.eps;
    s.minus_zero = -0.0f;
    s.one = 1;
    // keeps sqrt(v) * inv_c2 + eps at 2^25 or below
    s.root_most = s.eps <= 0x1p24f ? std::fmin(0x1p50f, 0x1p24f / s.inv_c2) : -1.0f;
    s.scale = scale;
    return s;
}

int64_t chunks_of(int64_t size, int head, int64_t chunk)
{
    if (size == 0) return 0;
    const int64_t body = size - (head > 0 ? head : 0);
    return body <= 0 ? 1 : (body + chunk - 1) / chunk;
}

template <int CAP>
rr_status norm_lists(const void *const *grads, const int64_t *sizes, int count, rr_dtype dtype, int sms,
                     GradNormEndArgs &end, double *part, cudaStream_t stream)
{
    const int eb = float_bytes(dtype), E = 16 / eb;
    const int64_t chunk = (int64_t)kThreads * E * kNormUnroll;
    const void *fn = dtype == RR_FP32   ? (const void *)grad_norm_kernel<float, CAP>
                     : dtype == RR_BF16 ? (const void *)grad_norm_kernel<__nv_bfloat16, CAP>
                                        : (const void *)grad_norm_kernel<__half, CAP>;
    int fit = 0;
    RR_TRY(step_fit(fn, kThreads, 0, &fit));
    const int64_t most = std::min<int64_t>((int64_t)fit * sms, kNormBlocks);
    GradNormArgs<CAP> a;
    for (int i = 0; i < count;) {
        int k = 0;
        a.list.start[0] = 0;
        for (; i < count && k < CAP; ++i) {
            if (sizes[i] == 0) continue;
            a.g[k] = grads[i];
            a.list.size[k] = sizes[i];
            a.list.head[k] = (int8_t)elements_before(grads[i], eb, E);
            a.list.start[k + 1] = a.list.start[k] + chunks_of(sizes[i], a.list.head[k], chunk);
            ++k;
        }
        if (k == 0) break;
        a.list.count = k;
        a.alone = i == count && end.count == 0 && a.list.start[k] <= kNormAlone;
        const int64_t grid = a.alone ? 1 : std::min(a.list.start[k], most);
        a.part = part + end.count;
        a.end = end;
        RR_TRY(step_launch(fn, grid, kThreads, 0, &a, stream));
        if (a.alone) return RR_OK;
        end.count += grid;
    }
    return step_launch((const void *)grad_norm_end_kernel, 1, kThreads, 0, &end, stream);
}

// Kernels by parameter type, gradient type and master weights.
template <class P, class G, int CAP>
const void *adamw_fn(bool master)
{
    return master ? (const void *)adamw_kernel<P, G, true, CAP> : (const void *)adamw_kernel<P, G, false, CAP>;
}
template <class P, class G, int CAP>
const void *adamw8_fn(bool master)
{
    return master ? (const void *)adamw8_kernel<P, G, true, CAP> : (const void *)adamw8_kernel<P, G, false, CAP>;
}
#define RR_BY_TYPES(fn)                                                                                    \
    template <class P, int CAP>                                                                            \
    const void *fn##_for(rr_dtype g, bool master)                                                          \
    {                                                                                                      \
        return g == RR_FP32   ? fn<P, float, CAP>(master)                                                  \
               : g == RR_BF16 ? fn<P, __nv_bfloat16, CAP>(master) : fn<P, __half, CAP>(master);            \
    }                                                                                                      \
    template <int CAP>                                                                                     \
    const void *fn##_for(rr_dtype p, rr_dtype g, bool master)                                              \
    {                                                                                                      \
        return p == RR_FP32   ? fn##_for<float, CAP>(g, master)                                            \
               : p == RR_BF16 ? fn##_for<__nv_bfloat16, CAP>(g, master) : fn##_for<__half, CAP>(g, master); \
    }
RR_BY_TYPES(adamw_fn)
RR_BY_TYPES(adamw8_fn)
#undef RR_BY_TYPES

template <int CAP>
rr_status adamw_lists(void *const *params, const void *const *grads, float *const *m, float *const *v,
                      float *const *master, const int64_t *sizes, int count, rr_dtype pd, rr_dtype gd,
                      const AdamScalars &h, int sms, cudaStream_t stream)
{
    const int pb = float_bytes(pd), gb = float_bytes(gd);
    AdamArgs<CAP> a;
    a.h = h;
    const void *fn = adamw_fn_for<CAP>(pd, gd, master != nullptr);
    int fit = 0;
    RR_TRY(step_fit(fn, kThreads, 0, &fit));
    for (int i = 0; i < count;) {
        int k = 0;
        a.list.start[0] = 0;
        for (; i < count && k < CAP; ++i) {
            if (sizes[i] == 0) continue;
            a.p[k] = params[i];
            a.g[k] = grads[i];
            a.m[k] = m[i];
            a.v[k] = v[i];
            a.w[k] = master ? master[i] : nullptr;
            const int head = elements_before(params[i], pb, kUnit);
            const bool together = elements_before(grads[i], gb, kUnit) == head && elements_before(m[i], 4, kUnit) == head &&
                                  elements_before(v[i], 4, kUnit) == head &&
                                  (!master || elements_before(master[i], 4, kUnit) == head);
            a.list.head[k] = (int8_t)(together ? head : kNoVector);
            a.list.size[k] = sizes[i];
            a.list.start[k + 1] = a.list.start[k] + chunks_of(sizes[i], a.list.head[k], kAdamChunk);
            ++k;
        }
        if (k == 0) break;
        a.list.count = k;
        RR_TRY(step_launch(fn, std::min<int64_t>(a.list.start[k], (int64_t)fit * sms), kThreads, 0, &a, stream));
    }
    return RR_OK;
}

template <int CAP>
rr_status adamw8_lists(void *const *params, const void *const *grads, uint8_t *const *m, float *const *ms,
                       uint8_t *const *r, float *const *rs, float *const *master, const int64_t *sizes, int count,
                       rr_dtype pd, rr_dtype gd, const AdamScalars &h, uint32_t seed, int sms, cudaStream_t stream)
{
    Adam8Args<CAP> a;
    a.h = h;
    a.seed = seed;
    const void *fn = adamw8_fn_for<CAP>(pd, gd, master != nullptr);
    int fit = 0;
    const int wb = master ? 4 : float_bytes(pd);
    const int smem = kThreads / 32 * adam8_stages(wb) * kBlock * (wb + float_bytes(gd) + 2);
    RR_TRY(step_fit(fn, kThreads, smem, &fit));
    // Tensors keep their place in the caller's list (it enters the random
    // bits), so empty ones stay in the table with no chunks.
    for (int i = 0; i < count;) {
        int k = 0;
        a.first = (uint32_t)i;
        a.list.start[0] = 0;
        for (; i < count && k < CAP; ++i, ++k) {
            a.p[k] = params[i];
            a.g[k] = grads[i];
            a.m[k] = m[i];
            a.ms[k] = ms[i];
            a.r[k] = r[i];
            a.rs[k] = rs[i];
            a.w[k] = master ? master[i] : nullptr;
            a.list.head[k] = (int8_t)(aligned_to(params[i], 16) && aligned_to(grads[i], 16) && aligned_to(m[i], 8) &&
                                              aligned_to(r[i], 8) && (!master || aligned_to(master[i], 16))
                                          ? 0 : kNoVector);
            a.list.size[k] = sizes[i];
            a.list.start[k + 1] = a.list.start[k] + (sizes[i] + kBlock - 1) / kBlock;
        }
        a.list.count = k;
        if (a.list.start[k] == 0) continue;
        const int64_t want = (a.list.start[k] + kThreads / 32 - 1) / (kThreads / 32);
        RR_TRY(step_launch(fn, std::min<int64_t>(want, (int64_t)fit * sms), kThreads, smem, &a, stream));
    }
    return RR_OK;
}

int64_t norm_launches(int count) { return count <= kNormCap ? 1 : (count + kNormCap - 1) / kNormCap; }

rr_status check_types(rr_dtype pd, rr_dtype gd)
{
    if (!float_bytes(pd)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "param_dtype %d", (int)pd);
    if (!float_bytes(gd)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "grad_dtype %d", (int)gd);
    return RR_OK;
}

bool nothing_to_do(const int64_t *sizes, int count)
{
    for (int i = 0; i < count; ++i)
        if (sizes[i] > 0) return false;
    return true;
}

}  // namespace

}  // namespace rr

using namespace rr;

extern "C" rr_status rr_grad_norm_workspace(int num_tensors, size_t *bytes)
{
    if (!bytes) return step_fail(RR_ERR_INVALID_ARG, "bytes is NULL");
    if (num_tensors < 0) return step_fail(RR_ERR_INVALID_ARG, "num_tensors %d", num_tensors);
    *bytes = (size_t)(norm_launches(num_tensors) * kNormBlocks) * sizeof(double);
    return step_ok();
}

extern "C" rr_status rr_grad_norm(const void *const *grads, const int64_t *sizes, int num_tensors, rr_dtype dtype,
                                  float inv_scale, float max_norm, float *norm, float *scale, void *workspace,
                                  size_t workspace_bytes, cudaStream_t stream)
try {
    if (!float_bytes(dtype)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
    RR_TRY(check_list(sizes, num_tensors));
    if (!(inv_scale > 0.0f && std::isfinite(inv_scale))) return step_fail(RR_ERR_INVALID_ARG, "inv_scale %g", (double)inv_scale);
    if (!(max_norm >= 0.0f)) return step_fail(RR_ERR_INVALID_ARG, "max_norm %g", (double)max_norm);
    if (!norm && !scale) return step_fail(RR_ERR_INVALID_ARG, "norm and scale are both NULL");
    RR_TRY(check_pointers("grads", grads, sizes, num_tensors, float_bytes(dtype)));
    if (!aligned_to(norm, 4)) return step_fail(RR_ERR_ALIGNMENT, "norm not 4-byte aligned");
    if (!aligned_to(scale, 4)) return step_fail(RR_ERR_ALIGNMENT, "scale not 4-byte aligned");
    if (!workspace) return step_fail(RR_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned_to(workspace, 16)) return step_fail(RR_ERR_ALIGNMENT, "workspace not 16-byte aligned");
    size_t need = 0;
    RR_TRY(rr_grad_norm_workspace(num_tensors, &need));
    if (workspace_bytes < need)
        return step_fail(RR_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    static thread_local Spans spans;
    spans.all.clear();
    for (int i = 0; i < num_tensors; ++i) spans.add(grads[i], sizes[i] * float_bytes(dtype), false);
    spans.add(workspace, (int64_t)need, true);
    spans.add(norm, 4, true);
    spans.add(scale, 4, true);
    if (spans.touch()) return step_fail(RR_ERR_ALIAS, "norm, scale or workspace overlaps another argument");

    int sms = 0;
    RR_TRY(step_sms(&sms));
    double *part = static_cast<double *>(workspace);
    GradNormEndArgs end{part, 0, inv_scale, max_norm, norm, scale};
    RR_TRY(num_tensors <= kNormCapSmall ? norm_lists<kNormCapSmall>(grads, sizes, num_tensors, dtype, sms, end, part, stream)
                                        : norm_lists<kNormCap>(grads, sizes, num_tensors, dtype, sms, end, part, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}

extern "C" rr_status rr_adamw(void *const *params, const void *const *grads, float *const *exp_avg,
                              float *const *exp_avg_sq, float *const *master, const int64_t *sizes,
                              int num_tensors, rr_dtype param_dtype, rr_dtype grad_dtype,
                              const rr_adamw_hyper *hyper, const float *grad_scale, cudaStream_t stream)
try {
    RR_TRY(check_types(param_dtype, grad_dtype));
    RR_TRY(check_list(sizes, num_tensors));
    RR_TRY(check_hyper(hyper));
    const int pb = float_bytes(param_dtype), gb = float_bytes(grad_dtype);
    RR_TRY(check_pointers("params", plain(params), sizes, num_tensors, pb));
    RR_TRY(check_pointers("grads", grads, sizes, num_tensors, gb));
    RR_TRY(check_pointers("exp_avg", plain(exp_avg), sizes, num_tensors, 4));
    RR_TRY(check_pointers("exp_avg_sq", plain(exp_avg_sq), sizes, num_tensors, 4));
    if (master) RR_TRY(check_pointers("master", plain(master), sizes, num_tensors, 4));
    if (!aligned_to(grad_scale, 4)) return step_fail(RR_ERR_ALIGNMENT, "grad_scale not 4-byte aligned");
    static thread_local Spans spans;
    spans.all.clear();
    for (int i = 0; i < num_tensors; ++i) spans.add(params[i], sizes[i] * pb, true);
    for (int i = 0; i < num_tensors; ++i) spans.add(grads[i], sizes[i] * gb, false);
    for (int i = 0; i < num_tensors; ++i) spans.add(exp_avg[i], sizes[i] * 4, true);
    for (int i = 0; i < num_tensors; ++i) spans.add(exp_avg_sq[i], sizes[i] * 4, true);
    for (int i = 0; master && i < num_tensors; ++i) spans.add(master[i], sizes[i] * 4, true);
    spans.add(grad_scale, 4, false);
    if (spans.touch()) return step_fail(RR_ERR_ALIAS, "a parameter, state or master weight overlaps another argument");
    if (nothing_to_do(sizes, num_tensors)) return step_ok();

    int sms = 0;
    RR_TRY(step_sms(&sms));
    const AdamScalars h = scalars(*hyper, grad_scale);
    RR_TRY(num_tensors <= kAdamCapSmall
               ? adamw_lists<kAdamCapSmall>(params, grads, exp_avg, exp_avg_sq, master, sizes, num_tensors, param_dtype,
                                            grad_dtype, h, sms, stream)
               : adamw_lists<kAdamCap>(params, grads, exp_avg, exp_avg_sq, master, sizes, num_tensors, param_dtype,
                                       grad_dtype, h, sms, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}

extern "C" rr_status rr_adamw8(void *const *params, const void *const *grads, uint8_t *const *exp_avg,
                               float *const *exp_avg_scale, uint8_t *const *exp_avg_sq,
                               float *const *exp_avg_sq_scale, float *const *master, const int64_t *sizes,
                               int num_tensors, rr_dtype param_dtype, rr_dtype grad_dtype,
                               const rr_adamw_hyper *hyper, uint32_t seed, const float *grad_scale,
                               cudaStream_t stream)
try {
    RR_TRY(check_types(param_dtype, grad_dtype));
    RR_TRY(check_list(sizes, num_tensors));
    RR_TRY(check_hyper(hyper));
    const int pb = float_bytes(param_dtype), gb = float_bytes(grad_dtype);
    RR_TRY(check_pointers("params", plain(params), sizes, num_tensors, pb));
    RR_TRY(check_pointers("grads", grads, sizes, num_tensors, gb));
    RR_TRY(check_pointers("exp_avg", plain(exp_avg), sizes, num_tensors, 1));
    RR_TRY(check_pointers("exp_avg_scale", plain(exp_avg_scale), sizes, num_tensors, 4));
    RR_TRY(check_pointers("exp_avg_sq", plain(exp_avg_sq), sizes, num_tensors, 1));
    RR_TRY(check_pointers("exp_avg_sq_scale", plain(exp_avg_sq_scale), sizes, num_tensors, 4));
    if (master) RR_TRY(check_pointers("master", plain(master), sizes, num_tensors, 4));
    if (!aligned_to(grad_scale, 4)) return step_fail(RR_ERR_ALIGNMENT, "grad_scale not 4-byte aligned");
    static thread_local Spans spans;
    spans.all.clear();
    auto blocks = [](int64_t n) { return (n + kBlock - 1) / kBlock; };
    for (int i = 0; i < num_tensors; ++i) spans.add(params[i], sizes[i] * pb, true);
    for (int i = 0; i < num_tensors; ++i) spans.add(grads[i], sizes[i] * gb, false);
    for (int i = 0; i < num_tensors; ++i) spans.add(exp_avg[i], sizes[i], true);
    for (int i = 0; i < num_tensors; ++i) spans.add(exp_avg_scale[i], blocks(sizes[i]) * 4, true);
    for (int i = 0; i < num_tensors; ++i) spans.add(exp_avg_sq[i], sizes[i], true);
    for (int i = 0; i < num_tensors; ++i) spans.add(exp_avg_sq_scale[i], blocks(sizes[i]) * 4, true);
    for (int i = 0; master && i < num_tensors; ++i) spans.add(master[i], sizes[i] * 4, true);
    spans.add(grad_scale, 4, false);
    if (spans.touch()) return step_fail(RR_ERR_ALIAS, "a parameter, state or master weight overlaps another argument");
    if (nothing_to_do(sizes, num_tensors)) return step_ok();

    int sms = 0;
    RR_TRY(step_sms(&sms));
    const AdamScalars h = scalars(*hyper, grad_scale);
    RR_TRY(num_tensors <= kAdamCapSmall
               ? adamw8_lists<kAdamCapSmall>(params, grads, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, master,
                                             sizes, num_tensors, param_dtype, grad_dtype, h, seed, sms, stream)
               : adamw8_lists<kAdamCap>(params, grads, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, master,
                                        sizes, num_tensors, param_dtype, grad_dtype, h, seed, sms, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}
