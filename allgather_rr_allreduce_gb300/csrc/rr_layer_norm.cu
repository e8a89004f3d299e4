// Layer norm and its gradient (include/rr.h: rr_layer_norm,
// rr_layer_norm_backward).
//
// Both are bound by HBM: a row is read once into registers, its statistics are
// reduced over the warps that share it, and the result is written from the
// same registers.  A row belongs to G warps of one block, EL elements to a
// lane; with G = 1 the warps of a block work on rows of their own and meet
// nowhere.  Blocks stay for many rows, so weights are loaded once and the
// weight's gradient is summed in registers over a block's rows; the blocks'
// partial sums go to the workspace and a second kernel adds them in order.
//
// Times below are of one GB300 (152 SMs, measured copy 6.7 TB/s), rows x columns.
#include <map>
#include <mutex>
#include <tuple>

#include "rr_step.h"

namespace rr {

namespace {

constexpr int kMaxPartials = 608;  // blocks whose partial weight gradients are kept
constexpr int kWidePartials = 152;  // of them, of the kernels of long rows

struct NormArgs {
    const void *x, *w, *b;
    void *y;
    float *mean, *rstd;
    int64_t rows, cols, xs, ys;
    float eps;
    int wdtype;
};

struct NormGradArgs {
    const void *dy, *x, *w;
    const float *mean, *rstd;
    void *dx;
    float *part;   // [2][P][cols] partial dweight, dbias; null: not wanted
    float2 *coef;  // [rows], the two row means (columns kernel only)
    int64_t rows, cols, dys, xs, dxs;
    int wdtype;
    int P;
};

// One lane's EL elements of a row.  Warp g of the row has columns
// [g * 32 * EL, (g + 1) * 32 * EL).  VEC: its 16-byte vectors in turn, vector v
// of the lane at column ((g * NV + v) * 32 + lane) * EN; else its single
// elements in turn, element k at column (g * EL + k) * 32 + lane.  Columns past
// the row read as zero and are not written.
template <class T, int EL, bool VEC>
struct Slice {
    static constexpr int EN = 16 / (int)sizeof(T);
    static constexpr int NV = EL / EN;
    static constexpr int kStep = VEC ? 32 * EN : 32;  // columns from a lane's vector (element) to its next
    static constexpr int kRing = NV * 32;             // 16-byte slots of a warp in one stage of a ring
    Pack<T, EN> raw[NV];

    // The lane's first column; column of its k-th element.
    static __device__ __forceinline__ int first(int g, int lane) { return g * 32 * EL + (VEC ? lane * EN : lane); }
    static __device__ __forceinline__ int col(int k, int g, int lane)
    {
        return first(g, lane) + (VEC ? k / EN * kStep + k % EN : k * kStep);
    }
    // p: address of the lane's first column; c: that column.
    __device__ __forceinline__ void load(const T *p, int c, int cols)
    {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (VEC) {
                if (c + v * kStep < cols) {
                    raw[v] = *reinterpret_cast<const Pack<T, EN> *>(p + v * kStep);
                } else {
                    *reinterpret_cast<uint4 *>(&raw[v]) = make_uint4(0, 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int j = 0; j < EN; ++j) {
                    const int k = v * EN + j;
                    raw[v].v[j] = c + k * kStep < cols ? p[k * kStep] : from_f32<T>(0.0f);
                }
            }
        }
    }
    // The same through the lane's own slots of a ring in shared memory (VEC
    // only).  Slots past the row are zeroed once and never fetched.
    static __device__ __forceinline__ void fetch(uint4 *slot, const T *p, int c, int cols)
    {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (c + v * kStep < cols) fetch16(slot + v * 32, p + v * kStep);
    }
    static __device__ __forceinline__ void clear(uint4 *slot, int c, int cols)
    {
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (c + v * kStep >= cols) slot[v * 32] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void take(const uint4 *slot)
    {
#pragma unroll
        for (int v = 0; v < NV; ++v) *reinterpret_cast<uint4 *>(&raw[v]) = slot[v * 32];
    }
    __device__ __forceinline__ float2 pair(int k) const { return pair_f32(&raw[k / EN].v[k % EN]); }
    __device__ __forceinline__ void set(int k, float2 x) { pair_set(&raw[k / EN].v[k % EN], x); }
    __device__ __forceinline__ void store(T *p, int c, int cols) const
    {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            if (VEC) {
                if (c + v * kStep < cols) *reinterpret_cast<Pack<T, EN> *>(p + v * kStep) = raw[v];
            } else {
#pragma unroll
                for (int j = 0; j < EN; ++j) {
                    const int k = v * EN + j;
                    if (c + k * kStep < cols) p[k * kStep] = raw[v].v[j];
                }
            }
        }
    }
};

// A lane's pairs of a vector of weights as binary32; zero past the row.
template <class S, int EL>
__device__ __forceinline__ void load_weights(float2 (&w)[EL / 2], const void *p, int dtype, float absent, int cols, int g,
                                             int lane)
{
#pragma unroll
    for (int k = 0; k < EL; ++k) {
        const int c = S::col(k, g, lane);
        const float v = c < cols ? (p ? load_any(p, c, dtype) : absent) : 0.0f;
        if (k & 1) w[k / 2].y = v;
        else w[k / 2].x = v;
    }
}

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// E weights from column c on as binary32 (`aligned`: their address is a
// multiple of 16 bytes wherever c is one of E).
template <int E>
__device__ __forceinline__ void weights_at(float (&w)[E], const void *p, int64_t c, int dtype, bool aligned, float absent)
{
    if (!p) {
#pragma unroll
        for (int k = 0; k < E; ++k) w[k] = absent;
    } else if (E == 1 || !aligned) {
#pragma unroll
        for (int k = 0; k < E; ++k) w[k] = load_any(p, c + k, dtype);
    } else if (dtype == RR_FP32) {
        const Pack<float, E> v = *reinterpret_cast<const Pack<float, E> *>(static_cast<const float *>(p) + c);
#pragma unroll
        for (int k = 0; k < E; ++k) w[k] = v.v[k];
    } else if (dtype == RR_BF16) {
        const Pack<__nv_bfloat16, E> v = *reinterpret_cast<const Pack<__nv_bfloat16, E> *>(static_cast<const __nv_bfloat16 *>(p) + c);
#pragma unroll
        for (int k = 0; k < E; ++k) w[k] = to_f32(v.v[k]);
    } else {
        const Pack<__half, E> v = *reinterpret_cast<const Pack<__half, E> *>(static_cast<const __half *>(p) + c);
#pragma unroll
        for (int k = 0; k < E; ++k) w[k] = to_f32(v.v[k]);
    }
}

// Sum over a block's G warps of what lane i % 2 * half holds for warp i (half:
// the largest power of two below G, 0 for one warp); every lane gets it.
__device__ __forceinline__ float group_sum(float x, int half)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (half >= o) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ __forceinline__ int half_of(int G) { return G > 1 ? 1 << (31 - __clz(G - 1)) : 0; }

// Row statistics: each warp takes the sum of its part and the squares centred
// on its own mean, and the warps' parts are joined around the common mean, so
// nothing is subtracted from a large sum of squares and one barrier serves.
// GROUP: the block's G warps share a row (else the warp has it alone).
// VEC (even rows: whole, aligned 16-byte vectors): rows come through a ring of
// ring_rows() rows in shared memory, each thread fetching and reading only its
// own vectors, so no barrier guards it; else one row is held ahead in registers.
//
// Bound: HBM.  32768 x 3584 bf16 with statistics 75.7 us, 6.2 TB/s, 93 % of the
// copy peak (one row ahead in registers 104; 2 blocks to an SM in place of 3,
// 93-100; divisions where the parts are joined, 193).  65536 x 1024 50 us (80 %),
// 8192 x 8192 45 us (88 %), 8 rows of 3584 2.7 us (latency).  Uneven rows are bound
// by instructions, an element to each load and store: 20011 x 1027 fp16 28.8 us.
__host__ __device__ constexpr int ring_rows(int el, int eb) { return el * eb > 64 ? 3 : 4; }  // 512 threads' rings fit an SM
template <class T, int EL, bool VEC, bool GROUP>
__global__ void __launch_bounds__(EL == 8 ? 1024 : EL == 16 ? 256 : 512, EL == 16 ? (VEC ? 3 : 2) : 1) norm_rows_kernel(const __grid_constant__ NormArgs a)
{
    stream_order();
    using S = Slice<T, EL, VEC>;
    constexpr int kStages = ring_rows(EL, sizeof(T));
    __shared__ float2 s_part[2][32];
    __shared__ float2 s_count[32];  // columns of each warp and the reciprocal
    extern __shared__ uint4 s_ring[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int G = GROUP ? warps : 1, g = GROUP ? warp : 0;
    const int64_t step = GROUP ? gridDim.x : (int64_t)gridDim.x * warps;
    int64_t row = GROUP ? blockIdx.x : (int64_t)blockIdx.x * warps + warp;
    const int cols = (int)a.cols, half = half_of(G), c0 = S::first(g, lane);

    // Ring: stage s of this lane at ring + s * round.
    uint4 *const ring = s_ring + warp * S::kRing + lane;
    const int round = warps * S::kRing;
    // rows to come, to reduce and to fetch: fewer than 2^31, as more than 2^31 rows fill the grid
    int left = row < a.rows ? (int)((a.rows - row + step - 1) / step) : 0, far = left;
    const T *src = static_cast<const T *>(a.x) + row * a.xs + c0;
    const int64_t src_step = step * a.xs;
    if (VEC) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) S::clear(ring + s * round, c0, cols);
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            if (far > 0) S::fetch(ring + s * round, src, c0, cols);
            fetch_commit();
            src += src_step;
            --far;
        }
    }
    float2 w[EL / 2], b[EL / 2];
    load_weights<S, EL>(w, a.w, a.wdtype, 1.0f, cols, g, lane);
    load_weights<S, EL>(b, a.b, a.wdtype, 0.0f, cols, g, lane);
    float mine = 0.0f;
#pragma unroll
    for (int k = 0; k < EL; ++k) mine += S::col(k, g, lane) < cols ? 1.0f : 0.0f;
    const float count = warp_sum(mine);
    const float inv_count = count > 0.0f ? 1.0f / count : 0.0f, inv_n = 1.0f / (float)cols;
    float2 part_count = make_float2(0.0f, 0.0f);
    const int peer = half ? lane & (2 * half - 1) : 0;
    if (GROUP) {
        if (lane == 0) s_count[g] = make_float2(count, inv_count);
        __syncthreads();
        if (peer < G) part_count = s_count[peer];
    }

    T *dst = static_cast<T *>(a.y) + row * a.ys + c0;
    const int64_t dst_step = step * a.ys;
    S next;
    if (!VEC && left > 0) next.load(src, c0, cols);
    int stage = 0;
    for (int it = 0; left > 0; --left, it ^= 1) {
        S cur;
        if (VEC) {
            if (far > 0) S::fetch(ring + (stage == 0 ? kStages - 1 : stage - 1) * round, src, c0, cols);
            fetch_commit();
            src += src_step;
            --far;
            fetch_wait<kStages - 1>();
            cur.take(ring + stage * round);
            stage = stage == kStages - 1 ? 0 : stage + 1;
        } else {
            cur = next;
            src += src_step;
            if (left > 1) next.load(src, c0, cols);
        }
        float2 d[EL / 2];
        float2 acc = both(0.0f);
#pragma unroll
        for (int k = 0; k < EL / 2; ++k) {
            d[k] = cur.pair(2 * k);
            acc = add2(acc, d[k]);
        }
        const float sum = warp_sum(acc.x + acc.y);
        float shift = sum * inv_count;  // the warp's mean
        acc = both(0.0f);
#pragma unroll
        for (int k = 0; k < EL / 2; ++k) {
            d[k] = add2(d[k], both(-shift));
            if (VEC) {  // whole vectors lie inside the row or past it
                if (S::col(2 * k, g, lane) < cols) acc = fma2(d[k], d[k], acc);
            } else {
                float2 in = d[k];
                if (S::col(2 * k, g, lane) >= cols) in.x = 0.0f;
                if (S::col(2 * k + 1, g, lane) >= cols) in.y = 0.0f;
                acc = fma2(in, in, acc);
            }
        }
        float m2 = warp_sum(acc.x + acc.y), mean = shift;
        if (GROUP) {
            if (lane == 0) s_part[it][g] = make_float2(sum, m2);
            __syncthreads();
            const float2 p = peer < G ? s_part[it][peer] : make_float2(0.0f, 0.0f);
            mean = group_sum(p.x, half) * inv_n;
            const float off = fmaf(p.x, part_count.y, -mean);
            m2 = group_sum(fmaf(part_count.x * off, off, p.y), half);
        }
        // (x - mean) * rstd from x less the warp's mean: both terms are of the
        // spread's size, however large the mean
        const float rstd = rsqrtf(fmaf(m2, inv_n, a.eps));
        const float2 r2 = both(rstd), move = both((shift - mean) * rstd);
#pragma unroll
        for (int k = 0; k < EL / 2; ++k) cur.set(2 * k, fma2(fma2(d[k], r2, move), w[k], b[k]));
        cur.store(dst, c0, cols);
        if (g == 0 && lane == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        dst += dst_step;
        row += step;
    }
}

// Rows too long for registers: a block per row, three passes over it, the
// second and third out of L1 or L2.  EVEN: rows of whole, aligned 16-byte
// vectors, E elements at a time; else one at a time.  Bound by the latency of the
// passes and their two block sums: 4096 x 18944 bf16 83 us (56 % of the copy peak;
// 92 without the next row's way to L2).
//
// A thread's sums go to a compensated one after each kPart elements: the rounding
// of a row's sums does not grow with its length.
template <class T, bool EVEN>
constexpr int kWidth = EVEN ? 16 / (int)sizeof(T) : 1;
constexpr int kPart = 64;

__device__ __forceinline__ float block_sum(float x, float *s)
{
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) t += s[i];
    return t;
}

// A thread's two sums of a row from column c on: `sum` of each stretch, the
// stretches by compensated sums.  Rows of one stretch (up to 32768 columns of
// vectors, 65536 single ones) take `sum` alone: 83 us for 4096 x 18944 bf16, in one
// loop over the stretches 89.
template <class F>
__device__ __forceinline__ float2 in_parts(int64_t c, int64_t cols, int64_t stretch, F sum)
{
    if (cols <= stretch) return sum(c, cols);
    Compensated x, y;
    for (; c < cols; c += stretch) {
        const float2 part = sum(c, min(cols, c + stretch));
        x.add(part.x);
        y.add(part.y);
    }
    return make_float2(x.value(), y.value());
}

// Vectors: 83 us for 4096 x 18944 bf16 forward with 512 threads, 119 with 1024;
// single elements: 275 and 197 for 2000 x 40001 (before rows were brought to L2).
__host__ __device__ constexpr int long_threads(bool even) { return even ? 512 : 1024; }
template <class T, bool EVEN>
__global__ void __launch_bounds__(long_threads(EVEN)) norm_long_kernel(const __grid_constant__ NormArgs a)
{
    stream_order();
    constexpr int E = kWidth<T, EVEN>, kLongThreads = long_threads(EVEN);
    __shared__ float s[32];
    const int64_t first = (int64_t)threadIdx.x * E, next = (int64_t)kLongThreads * E, stretch = kPart / E * next;
    const bool waligned = aligned16(a.w), baligned = aligned16(a.b);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + row * a.xs;
        T *y = static_cast<T *>(a.y) + row * a.ys;
        const float sum = in_parts(first, a.cols, stretch, [&](int64_t c, int64_t end) {
            float part = 0.0f;
#pragma unroll 4
            for (; c < end; c += next) {
                const Pack<T, E> v = *reinterpret_cast<const Pack<T, E> *>(x + c);
#pragma unroll
                for (int k = 0; k < E; ++k) part += to_f32(v.v[k]);
            }
            return make_float2(part, 0.0f);
        }).x;
        if (row + gridDim.x < a.rows) {  // the next row into L2, 128 bytes to a thread
            const char *far = reinterpret_cast<const char *>(x + gridDim.x * a.xs);
            for (int64_t l = threadIdx.x * 128; l < a.cols * (int64_t)sizeof(T); l += kLongThreads * 128) prefetch_l2(far + l);
        }
        const float mean = block_sum(sum, s) / (float)a.cols;
        const float m2 = in_parts(first, a.cols, stretch, [&](int64_t c, int64_t end) {
            float part = 0.0f;
#pragma unroll 4
            for (; c < end; c += next) {
                const Pack<T, E> v = *reinterpret_cast<const Pack<T, E> *>(x + c);
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const float d = to_f32(v.v[k]) - mean;
                    part = fmaf(d, d, part);
                }
            }
            return make_float2(part, 0.0f);
        }).x;
        const float rstd = rsqrtf(block_sum(m2, s) / (float)a.cols + a.eps);
#pragma unroll 4
        for (int64_t c = first; c < a.cols; c += next) {
            Pack<T, E> v = *reinterpret_cast<const Pack<T, E> *>(x + c);
            float w[E], b[E];
            weights_at<E>(w, a.w, c, a.wdtype, waligned, 1.0f);
            weights_at<E>(b, a.b, c, a.wdtype, baligned, 0.0f);
#pragma unroll
            for (int k = 0; k < E; ++k) v.v[k] = from_f32<T>(fmaf((to_f32(v.v[k]) - mean) * rstd, w[k], b[k]));
            *reinterpret_cast<Pack<T, E> *>(y + c) = v;
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// ---------------------------------------------------------------- gradient
// Each row needs two sums over its columns, sum(w dy) and sum(w dy xhat),
// before its dx; dweight and dbias are sums over rows and stay in registers.
//
// What bounds a block is the chain of one row (load, sum, shuffles, barrier,
// store), so rows of up to 256 columns go two at once, and grad_stages() steps
// fill the ring in shared memory.  Row statistics come 32 rows at a time, one to
// a lane: fetched row by row they cost about 10 us of 128.
//
// 32768 x 3584 bf16 114 us, 6.2 TB/s, 92 % of the copy peak with the join (two
// rows at once spill and take 130; three blocks to an SM spill, 163).  65536 x
// 1024 68 us (89 %), 8192 x 8192 79 us (76 %: one block of 227 registers to an SM),
// 131072 x 256 37 us (83 %), 1024 x 3584 14.5 us (the chain, and partial sums).
//
// Past its end a row reads as x = dy = 0, which leaves 0 * infinity in sum(w dy
// xhat) where mean * rstd overflows; such a row's sum is taken again without
// those columns.
__device__ __forceinline__ bool product_overflows(float mean, float rstd)
{
    return !(fabsf(mean * rstd) < __int_as_float(0x7f800000));
}
__host__ __device__ constexpr int grad_rows(int el, bool vec) { return vec && el == 8 ? 2 : 1; }
__host__ __device__ constexpr int grad_stages(int el) { return el == 8 ? 2 : 3; }
template <class T, int EL, bool VEC, bool GROUP>
__global__ void __launch_bounds__(EL == 32 ? 256 : 512, EL == 8 ? 1 : 0) norm_grad_rows_kernel(const __grid_constant__ NormGradArgs a)
{
    stream_order();
    using S = Slice<T, EL, VEC>;
    constexpr int R = grad_rows(EL, VEC), kStages = grad_stages(EL);
    __shared__ float2 s_part[2][R][16];
    extern __shared__ uint4 s_ring[];  // the ring of rows; at the end the sums that join a block's warps
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int G = GROUP ? warps : 1, g = GROUP ? warp : 0;
    const int64_t step = GROUP ? gridDim.x : (int64_t)gridDim.x * warps;
    const int64_t row = GROUP ? blockIdx.x : (int64_t)blockIdx.x * warps + warp;
    const int cols = (int)a.cols, half = half_of(G), c0 = S::first(g, lane);
    const float inv_n = 1.0f / (float)cols;
    const int peer = half ? lane & (2 * half - 1) : 0;

    uint4 *const ring = s_ring + warp * 2 * S::kRing + lane;  // of each row, dy's slots and then x's
    const int round = warps * 2 * S::kRing;
    // rows of this group: fewer than 2^31, as more than 2^31 rows fill the grid
    const int count = row < a.rows ? (int)((a.rows - row + step - 1) / step) : 0;
    int far = count;
    const T *gdy = static_cast<const T *>(a.dy) + row * a.dys + c0, *gx = static_cast<const T *>(a.x) + row * a.xs + c0;
    const int64_t dy_step = step * a.dys, x_step = step * a.xs;
    auto fetch = [&](uint4 *slot) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (far > i) {
                S::fetch(slot + i * round, gdy, c0, cols);
                S::fetch(slot + i * round + S::kRing, gx, c0, cols);
            }
            gdy += dy_step;
            gx += x_step;
        }
        fetch_commit();
        far -= R;
    };
    if (VEC) {
#pragma unroll
        for (int s = 0; s < kStages * R; ++s) {
            S::clear(ring + s * round, c0, cols);
            S::clear(ring + s * round + S::kRing, c0, cols);
        }
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) fetch(ring + s * R * round);
    }
    float means = 0.0f, rstds = 0.0f, next_means = 0.0f, next_rstds = 0.0f;  // of rows i .. i + 31, and the 32 after
    auto statistics = [&](int i) {
        if (i + lane < count) {
            next_means = a.mean[row + (i + lane) * step];
            next_rstds = a.rstd[row + (i + lane) * step];
        }
    };
    statistics(0);
    float2 w[EL / 2], dw[EL / 2], db[EL / 2];
    load_weights<S, EL>(w, a.w, a.wdtype, 1.0f, cols, g, lane);
#pragma unroll
    for (int k = 0; k < EL / 2; ++k) dw[k] = db[k] = both(0.0f);
    T *dst = static_cast<T *>(a.dx) + (a.dx ? row * a.dxs + c0 : 0);
    const int64_t dst_step = step * a.dxs;
    S ndy, nx;
    if (!VEC && count > 0) {
        ndy.load(gdy, c0, cols);
        nx.load(gx, c0, cols);
    }
    int stage = 0, it = 0;
    for (int i = 0; i < count; i += R, it ^= 1) {
        if ((i & 31) == 0) {
            means = next_means;
            rstds = next_rstds;
            statistics(i + 32);
        }
        S dy[R], x[R];
        if (VEC) {
            fetch(ring + (stage == 0 ? kStages - 1 : stage - 1) * R * round);
            fetch_wait<kStages - 1>();
#pragma unroll
            for (int j = 0; j < R; ++j) {
                dy[j].take(ring + (stage * R + j) * round);
                x[j].take(ring + (stage * R + j) * round + S::kRing);
            }
            stage = stage == kStages - 1 ? 0 : stage + 1;
        } else {
            dy[0] = ndy;
            x[0] = nx;
            gdy += dy_step;
            gx += x_step;
            if (i + 1 < count) {
                ndy.load(gdy, c0, cols);
                nx.load(gx, c0, cols);
            }
        }
        // With xhat = (x - mean) rstd: db += dy, dw += dy xhat, and the row's sums
        // are c1 of w dy and c2 of w dy xhat, from which
        //   dx = w dy rstd - (c1 rstd / n + xhat c2 rstd / n).
        // Neither rstd^2 nor dy rstd is taken by itself: they may leave binary32's
        // range where dx and dw do not.
        float mean[R], rstd[R], c1[R], c2[R];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            // past the last row nothing is kept; past a row's columns dy = w = 0
            const bool in = R == 1 || i + j < count;
            mean[j] = __shfl_sync(0xffffffffu, means, (i & 31) + j);
            rstd[j] = in ? __shfl_sync(0xffffffffu, rstds, (i & 31) + j) : 0.0f;
            const float2 r2 = both(rstd[j]), shift = both(-mean[j]);
            float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
            for (int k = 0; k < EL / 2; ++k) {
                const float2 d = dy[j].pair(2 * k), xhat = mul2(add2(x[j].pair(2 * k), shift), r2), wd = mul2(w[k], d);
                if (in) db[k] = add2(db[k], d);
                if (in) dw[k] = fma2(d, xhat, dw[k]);
                s1 = add2(s1, wd);
                s2 = fma2(wd, xhat, s2);
            }
            if (product_overflows(mean[j], rstd[j])) {  // without the columns past the row
                s2 = both(0.0f);
#pragma unroll
                for (int k = 0; k < EL / 2; ++k) {
                    const float2 xhat = mul2(add2(x[j].pair(2 * k), shift), r2), wd = mul2(w[k], dy[j].pair(2 * k));
                    if (S::col(2 * k, g, lane) < cols) s2.x = fmaf(wd.x, xhat.x, s2.x);
                    if (S::col(2 * k + 1, g, lane) < cols) s2.y = fmaf(wd.y, xhat.y, s2.y);
                }
            }
            c1[j] = s1.x + s1.y;
            c2[j] = s2.x + s2.y;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                c1[j] += __shfl_xor_sync(0xffffffffu, c1[j], o);
                c2[j] += __shfl_xor_sync(0xffffffffu, c2[j], o);
            }
        }
        if (GROUP) {
            if (lane == 0) {
#pragma unroll
                for (int j = 0; j < R; ++j) s_part[it][j][g] = make_float2(c1[j], c2[j]);
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const float2 p = peer < G ? s_part[it][j][peer] : make_float2(0.0f, 0.0f);
                c1[j] = group_sum(p.x, half);
                c2[j] = group_sum(p.y, half);
            }
        }
        if (a.dx) {
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const float2 r2 = both(rstd[j]), shift = both(-mean[j]);
                const float2 k1 = both(-c1[j] * inv_n * rstd[j]), k2 = both(-c2[j] * inv_n * rstd[j]);
#pragma unroll
                for (int k = 0; k < EL / 2; ++k) {
                    const float2 xhat = mul2(add2(x[j].pair(2 * k), shift), r2), wd = mul2(w[k], dy[j].pair(2 * k));
                    x[j].set(2 * k, fma2(wd, r2, fma2(xhat, k2, k1)));
                }
                if (R == 1 || i + j < count) x[j].store(dst, c0, cols);
                dst += dst_step;
            }
        }
    }
    if (!a.part) return;
    float *out = a.part + (int64_t)blockIdx.x * cols;
    const int64_t other = (int64_t)a.P * cols;  // from a column's dw to its db
    if (GROUP) {
#pragma unroll
        for (int k = 0; k < EL; ++k) {
            const int c = S::col(k, g, lane);
            if (c < cols) {
                out[c] = k & 1 ? dw[k / 2].y : dw[k / 2].x;
                out[c + other] = k & 1 ? db[k / 2].y : db[k / 2].x;
            }
        }
    } else {
        // join the block's warps in order: [warp][element][lane], the ring's memory
        float2 *s_sum = reinterpret_cast<float2 *>(s_ring);
        if (VEC) fetch_wait<0>();
        __syncthreads();
#pragma unroll
        for (int k = 0; k < EL; ++k)
            s_sum[(warp * EL + k) * 32 + lane] = k & 1 ? make_float2(dw[k / 2].y, db[k / 2].y) : make_float2(dw[k / 2].x, db[k / 2].x);
        __syncthreads();
        for (int k = warp; k < EL; k += warps) {
            float2 t = s_sum[k * 32 + lane];
            for (int i = 1; i < warps; ++i) t = add2(t, s_sum[(i * EL + k) * 32 + lane]);
            const int c = S::col(k, 0, lane);
            if (c < cols) {
                out[c] = t.x;
                out[c + other] = t.y;
            }
        }
    }
}

// Rows of more than a block's registers hold beside the sums: a block per row
// and two passes over it, the second out of L1, the weight's gradient in
// registers, EL columns to a thread, kAtOnce of them loaded together.  While a
// row's second pass runs, the next row comes into L2 (4096 x 18944 bf16 150 us,
// 46 % of the copy peak; without that 190).  One block of 16 warps to an SM: bound by
// the latency of its loads and by instructions; 48 columns to a thread spill 16 to
// 104 bytes of its 128 registers.
constexpr int kWideThreads = 512, kAtOnce = 8;
template <class T, int EL, bool EVEN>
__global__ void __launch_bounds__(kWideThreads) norm_grad_wide_kernel(const __grid_constant__ NormGradArgs a)
{
    stream_order();
    constexpr int E = kWidth<T, EVEN>, kWarps = kWideThreads / 32;
    __shared__ float2 s[2][kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cols = (int)a.cols;
    const float inv_n = 1.0f / (float)cols;
    const bool waligned = aligned16(a.w);
    // element k of the thread is at column c0 + column(k)
    const int c0 = threadIdx.x * E;
    auto column = [](int k) { return k / E * (kWideThreads * E) + k % E; };
    float2 dw[EL / 2], db[EL / 2];
#pragma unroll
    for (int k = 0; k < EL / 2; ++k) dw[k] = db[k] = both(0.0f);
    int it = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, it ^= 1) {
        const T *dy = static_cast<const T *>(a.dy) + row * a.dys + c0, *x = static_cast<const T *>(a.x) + row * a.xs + c0;
        const float mean = a.mean[row], rstd = a.rstd[row];
        const float2 r2 = both(rstd), shift = both(-mean);
        float g[kAtOnce], xv[kAtOnce], w[kAtOnce];  // elements k0 and on; 0 past the row
        auto load = [&](int k0) {
            Pack<T, E> pd[kAtOnce / E], px[kAtOnce / E];
#pragma unroll
            for (int j = 0; j < kAtOnce / E; ++j) {
                const int c = column(k0 + j * E);
                float wj[E];
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    pd[j].v[k] = px[j].v[k] = from_f32<T>(0.0f);
                    wj[k] = 0.0f;
                }
                if (c0 + c < cols) {
                    pd[j] = *reinterpret_cast<const Pack<T, E> *>(dy + c);
                    px[j] = *reinterpret_cast<const Pack<T, E> *>(x + c);
                    weights_at<E>(wj, a.w, c0 + c, a.wdtype, waligned, 1.0f);
                }
#pragma unroll
                for (int k = 0; k < E; ++k) w[j * E + k] = wj[k];
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; k += 2) {
                if (E > 1) {
                    const float2 gk = pair_f32(&pd[k / E].v[k % E]), xk = pair_f32(&px[k / E].v[k % E]);
                    g[k] = gk.x;
                    g[k + 1] = gk.y;
                    xv[k] = xk.x;
                    xv[k + 1] = xk.y;
                } else {
                    g[k] = to_f32(pd[k / E].v[k % E]);
                    g[k + 1] = to_f32(pd[(k + 1) / E].v[(k + 1) % E]);
                    xv[k] = to_f32(px[k / E].v[k % E]);
                    xv[k + 1] = to_f32(px[(k + 1) / E].v[(k + 1) % E]);
                }
            }
        };
        float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int k0 = 0; k0 < EL; k0 += kAtOnce) {
            load(k0);
#pragma unroll
            for (int k = 0; k < kAtOnce; k += 2) {
                const float2 wd = mul2(make_float2(w[k], w[k + 1]), make_float2(g[k], g[k + 1]));
                s1 = add2(s1, wd);
                s2 = fma2(wd, mul2(add2(make_float2(xv[k], xv[k + 1]), shift), r2), s2);
            }
        }
        if (product_overflows(mean, rstd)) {  // without the columns past the row
            s2 = both(0.0f);
#pragma unroll 1
            for (int c = threadIdx.x; c < cols; c += kWideThreads)
                s2.x = fmaf((a.w ? load_any(a.w, c, a.wdtype) : 1.0f) * to_f32(dy[c - c0]), (to_f32(x[c - c0]) - mean) * rstd, s2.x);
        }
        float c1 = warp_sum(s1.x + s1.y), c2 = warp_sum(s2.x + s2.y);
        if (lane == 0) s[it][warp] = make_float2(c1, c2);
        __syncthreads();
        const float2 p = s[it][lane % kWarps];
        const float2 k1 = both(-group_sum(p.x, kWarps / 2) * inv_n * rstd), k2 = both(-group_sum(p.y, kWarps / 2) * inv_n * rstd);
        if (row + gridDim.x < a.rows) {  // the next row, 128 bytes to a thread
            const char *fd = reinterpret_cast<const char *>(dy - c0 + gridDim.x * a.dys);
            const char *fx = reinterpret_cast<const char *>(x - c0 + gridDim.x * a.xs);
            for (int l = threadIdx.x * 128; l < cols * (int)sizeof(T); l += kWideThreads * 128) {
                prefetch_l2(fd + l);
                prefetch_l2(fx + l);
            }
        }
        T *dx = static_cast<T *>(a.dx) + (a.dx ? row * a.dxs + c0 : 0);
#pragma unroll
        for (int k0 = 0; k0 < EL; k0 += kAtOnce) {
            load(k0);
            Pack<T, E> out[kAtOnce / E];
#pragma unroll
            for (int k = 0; k < kAtOnce; k += 2) {
                const int i = (k0 + k) / 2;
                const float2 gk = make_float2(g[k], g[k + 1]), xhat = mul2(add2(make_float2(xv[k], xv[k + 1]), shift), r2);
                db[i] = add2(db[i], gk);
                dw[i] = fma2(gk, xhat, dw[i]);
                const float2 y = fma2(mul2(make_float2(w[k], w[k + 1]), gk), r2, fma2(xhat, k2, k1));
                if (E > 1) {
                    pair_set(&out[k / E].v[k % E], y);
                } else {
                    out[k / E].v[k % E] = from_f32<T>(y.x);
                    out[(k + 1) / E].v[(k + 1) % E] = from_f32<T>(y.y);
                }
            }
            if (a.dx) {
#pragma unroll
                for (int j = 0; j < kAtOnce / E; ++j) {
                    const int c = column(k0 + j * E);
                    if (c0 + c < cols) *reinterpret_cast<Pack<T, E> *>(dx + c) = out[j];
                }
            }
        }
    }
    if (!a.part) return;
    float *out = a.part + (int64_t)blockIdx.x * cols;
    const int64_t other = (int64_t)a.P * cols;
#pragma unroll
    for (int k = 0; k < EL; ++k) {
        const int c = c0 + column(k);
        if (c < cols) {
            out[c] = k & 1 ? dw[k / 2].y : dw[k / 2].x;
            out[c + other] = k & 1 ? db[k / 2].y : db[k / 2].x;
        }
    }
}

// Rows too long for that: the two row means first (two blocks to an SM: 2000 x
// 40001 bf16, both kernels 348 us, with one 440) ...
template <class T, bool EVEN>
__global__ void __launch_bounds__(long_threads(EVEN), 2) norm_grad_means_kernel(const __grid_constant__ NormGradArgs a)
{
    stream_order();
    constexpr int E = kWidth<T, EVEN>, kLongThreads = long_threads(EVEN);
    __shared__ float2 s[2][32];
    const bool waligned = aligned16(a.w);
    const int64_t next = (int64_t)kLongThreads * E, stretch = kPart / E * next;
    int it = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, it ^= 1) {
        const T *dy = static_cast<const T *>(a.dy) + row * a.dys;
        const T *x = static_cast<const T *>(a.x) + row * a.xs;
        const float mean = a.mean[row], rstd = a.rstd[row];
        const float2 sums = in_parts((int64_t)threadIdx.x * E, a.cols, stretch, [&](int64_t c, int64_t end) {
            float2 part = both(0.0f);
#pragma unroll 4
            for (; c < end; c += next) {
                const Pack<T, E> d = *reinterpret_cast<const Pack<T, E> *>(dy + c), v = *reinterpret_cast<const Pack<T, E> *>(x + c);
                float w[E];
                weights_at<E>(w, a.w, c, a.wdtype, waligned, 1.0f);
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const float wd = w[k] * to_f32(d.v[k]);
                    part.x += wd;
                    part.y = fmaf(wd, (to_f32(v.v[k]) - mean) * rstd, part.y);
                }
            }
            return part;
        });
        float c1 = warp_sum(sums.x), c2 = warp_sum(sums.y);
        if ((threadIdx.x & 31) == 0) s[it][threadIdx.x >> 5] = make_float2(c1, c2);
        __syncthreads();
        if (threadIdx.x < 32) {
            const float2 p = threadIdx.x < kLongThreads / 32 ? s[it][threadIdx.x] : make_float2(0.0f, 0.0f);
            c1 = warp_sum(p.x);
            c2 = warp_sum(p.y);
            if (threadIdx.x == 0) a.coef[row] = make_float2(c1 / (float)a.cols, c2 / (float)a.cols);
        }
    }
}

// ... then dx and the weight's gradient by columns: block p * tiles + i has
// tile i of the columns, E to a thread, and every P-th row, kTileRows at once
// and the next ones' loads under way.  There are fewer P the longer the rows, so
// a thread's sums go to a compensated sum after each kPart rows, in shared
// memory (20000 x 32776 bf16, both kernels 2530 us; in registers, which leave two
// blocks to an SM in place of three, 3334).  Single elements go two steps at a time
// (2000 x 40001 348 us, one by one 366).
constexpr int kTileThreads = 128, kTileRows = 4;
template <class T, bool EVEN>
struct TileRows {
    static constexpr int E = kWidth<T, EVEN>;
    Pack<T, E> d[kTileRows], x[kTileRows];
    float2 m[kTileRows];
    float mean[kTileRows], rstd[kTileRows];
    __device__ __forceinline__ void load(const NormGradArgs &a, int64_t row, int64_t c)
    {
#pragma unroll
        for (int j = 0; j < kTileRows; ++j) {
            const int64_t r = row + (int64_t)j * a.P;
            if (r < a.rows) {
                d[j] = *reinterpret_cast<const Pack<T, E> *>(static_cast<const T *>(a.dy) + r * a.dys + c);
                x[j] = *reinterpret_cast<const Pack<T, E> *>(static_cast<const T *>(a.x) + r * a.xs + c);
                m[j] = a.coef[r];
                mean[j] = a.mean[r];
                rstd[j] = a.rstd[r];
            }
        }
    }
};
template <class T, bool EVEN>
__global__ void __launch_bounds__(kTileThreads, EVEN ? 3 : 6) norm_grad_columns_kernel(const __grid_constant__ NormGradArgs a)
{
    stream_order();
    constexpr int E = kWidth<T, EVEN>;
    const int64_t tiles = (a.cols + kTileThreads * E - 1) / (kTileThreads * E);
    const int64_t c = (blockIdx.x % tiles * kTileThreads + threadIdx.x) * E;
    const int p = (int)(blockIdx.x / tiles);
    if (c >= a.cols) return;
    float w[E], dw[E], db[E];
    weights_at<E>(w, a.w, c, a.wdtype, false, 1.0f);
#pragma unroll
    for (int k = 0; k < E; ++k) dw[k] = db[k] = 0.0f;
    __shared__ float2 s_all[2 * E][kTileThreads];  // each thread its own
#pragma unroll
    for (int k = 0; k < 2 * E; ++k) s_all[k][threadIdx.x] = make_float2(0.0f, 0.0f);
    auto flush = [&](float &x, float2 &all) {
        Compensated t{all.x, all.y};
        t.add(x);
        all = make_float2(t.hi, t.lo);
        x = 0.0f;
        return t.value();
    };
    TileRows<T, EVEN> cur, next;
    const int64_t step = (int64_t)kTileRows * a.P;
    next.load(a, p, c);
    for (int64_t row = p; row < a.rows;) {
        const int64_t end = min(a.rows, row + kPart / kTileRows * step);
#pragma unroll (EVEN ? 1 : 2)
        for (; row < end; row += step) {
            cur = next;
            next.load(a, row + step, c);
#pragma unroll
            for (int j = 0; j < kTileRows; ++j) {
                const int64_t r = row + (int64_t)j * a.P;
                if (r >= a.rows) break;
#pragma unroll
                for (int k = 0; k < E; ++k) {
                    const float g = to_f32(cur.d[j].v[k]), xhat = (to_f32(cur.x[j].v[k]) - cur.mean[j]) * cur.rstd[j];
                    dw[k] = fmaf(g, xhat, dw[k]);
                    db[k] += g;
                    cur.x[j].v[k] = from_f32<T>((w[k] * g - cur.m[j].x - xhat * cur.m[j].y) * cur.rstd[j]);
                }
                if (a.dx) *reinterpret_cast<Pack<T, E> *>(static_cast<T *>(a.dx) + r * a.dxs + c) = cur.x[j];
            }
        }
#pragma unroll
        for (int k = 0; k < E; ++k) {
            flush(dw[k], s_all[k][threadIdx.x]);
            flush(db[k], s_all[E + k][threadIdx.x]);
        }
    }
    if (!a.part) return;
#pragma unroll
    for (int k = 0; k < E; ++k) {
        a.part[(int64_t)p * a.cols + c + k] = flush(dw[k], s_all[k][threadIdx.x]);
        a.part[((int64_t)a.P + p) * a.cols + c + k] = flush(db[k], s_all[E + k][threadIdx.x]);
    }
}

// The blocks' partial sums, added in order: 32 columns to a block, every
// kJoinWarps-th partial to a warp, then the warps' sums.  304 partials of 3584
// columns: 7 us from cold, in latency.
struct NormJoinArgs {
    const float *part;
    void *dweight, *dbias;
    int64_t cols;
    int P, wdtype;
};
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps) norm_grad_join_kernel(const __grid_constant__ NormJoinArgs a)
{
    stream_order();
    __shared__ float2 s[kJoinWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float2 t = both(0.0f);
    if (c < a.cols) {
#pragma unroll 8
        for (int p = warp; p < a.P; p += kJoinWarps)
            t = add2(t, make_float2(a.part[(int64_t)p * a.cols + c], a.part[((int64_t)a.P + p) * a.cols + c]));
    }
    s[warp][lane] = t;
    __syncthreads();
    // column `warp` of the block by warp: its kJoinWarps sums in a fixed tree
    t = s[lane][warp];
    t.x = warp_sum(t.x);
    t.y = warp_sum(t.y);
    const int64_t mine = (int64_t)blockIdx.x * 32 + warp;
    if (lane == 0 && mine < a.cols) {
        if (a.dweight) store_any(a.dweight, mine, a.wdtype, t.x);
        if (a.dbias) store_any(a.dbias, mine, a.wdtype, t.y);
    }
}

// ---------------------------------------------------------------- host side
std::mutex g_mu;
std::map<int, int> g_sms;
std::map<std::tuple<int, const void *, int, int>, int> g_fit;  // device, kernel, threads, shared memory

// Blocks of the columns kernel for each SM: what fits at once with vectors, more
// with single elements (before the sums in stretches, both kernels: 4096 x 18944
// bf16 210 us, with 8 blocks 227; 2000 x 12001 118, with 3 blocks 171).
constexpr int tile_blocks(bool even) { return even ? 3 : 16; }
template <class T>
const void *norm_long_fn(bool even)
{
    return even ? (const void *)norm_long_kernel<T, true> : (const void *)norm_long_kernel<T, false>;
}
template <class T>
void norm_grad_long_fn(bool even, const void **means, const void **columns)
{
    *means = even ? (const void *)norm_grad_means_kernel<T, true> : (const void *)norm_grad_means_kernel<T, false>;
    *columns = even ? (const void *)norm_grad_columns_kernel<T, true> : (const void *)norm_grad_columns_kernel<T, false>;
}

template <class T, bool EVEN>
const void *norm_grad_wide_fn(int el)
{
    return el == 32   ? (const void *)norm_grad_wide_kernel<T, 32, EVEN>
           : el == 40 ? (const void *)norm_grad_wide_kernel<T, 40, EVEN> : (const void *)norm_grad_wide_kernel<T, 48, EVEN>;
}
template <class T>
const void *norm_grad_wide_fn(int el, bool even)
{
    return even ? norm_grad_wide_fn<T, true>(el) : norm_grad_wide_fn<T, false>(el);
}

// Kernels of the shapes that row_shape gives.
template <class T>
const void *norm_rows_fn(int el, bool vec, bool group)
{
    if (!vec && el == 32) return (const void *)norm_rows_kernel<T, 32, false, true>;
    if (!vec && el == 16) return (const void *)norm_rows_kernel<T, 16, false, false>;
    if (!vec) return group ? (const void *)norm_rows_kernel<T, 8, false, true> : (const void *)norm_rows_kernel<T, 8, false, false>;
    if (el == 8) return group ? (const void *)norm_rows_kernel<T, 8, true, true> : (const void *)norm_rows_kernel<T, 8, true, false>;
    if (el == 16) return group ? (const void *)norm_rows_kernel<T, 16, true, true> : (const void *)norm_rows_kernel<T, 16, true, false>;
    return group ? (const void *)norm_rows_kernel<T, 32, true, true> : (const void *)norm_rows_kernel<T, 32, true, false>;
}
template <class T>
const void *norm_grad_fn(int el, bool vec, bool group)
{
    if (!vec && el == 32) return (const void *)norm_grad_rows_kernel<T, 32, false, true>;
    if (!vec && el == 16) return (const void *)norm_grad_rows_kernel<T, 16, false, false>;
    if (!vec) return group ? (const void *)norm_grad_rows_kernel<T, 8, false, true> : (const void *)norm_grad_rows_kernel<T, 8, false, false>;
    if (el == 8) return group ? (const void *)norm_grad_rows_kernel<T, 8, true, true> : (const void *)norm_grad_rows_kernel<T, 8, true, false>;
    if (el == 16) return group ? (const void *)norm_grad_rows_kernel<T, 16, true, true> : (const void *)norm_grad_rows_kernel<T, 16, true, false>;
    return group ? (const void *)norm_grad_rows_kernel<T, 32, true, true> : (const void *)norm_grad_rows_kernel<T, 32, true, false>;
}

// Elements to a lane and warps to a row.  Even rows: one warp with 8 or 16 elements
// a lane up to 512 columns; up to 1024 two warps with 16 while there are fewer than
// 8 rows for each SM, then one with 32; from there 16 a lane up to 8 warps (12 for
// the gradient), then 32; with fewer rows than SMs, where nothing but one row's
// latency counts, 8 a lane.  Both sides, 16 and 32 a lane, in us:
//   1024 columns of bf16, 257 rows: forward 2.8, 4.3, gradient 7.4, 7.9; 1000 rows:
//   4.2, 4.6 and 9.4, 7.8; 16384 rows: 14.9, 16.6 and 29.6, 23.0.  The border is late
//   for the gradient (32 is ahead from 608 rows) and early for the forward.
//   Gradient, 8192 rows of bf16: 4608 columns 56, 67; 5120 58, 68; 6144 63, 72 (300
//   rows 14.7, 15.6); binary32 5120 84, 81; 6144 107, 106.  8192 columns 85, 79.
// Uneven rows take 8 a lane while its warps allow (8000 x 5001 bf16 forward 60 us,
// with 16 66), except one warp a row with 16 for 257 to 512 columns (65536 x 301
// bf16: 30 against 35, gradient 49 against 81), then 32 (it spills, but reads a row
// once: 4000 x 12001 94 us, the long-row kernel 120).  warps > 0 where a kernel of
// that shape takes the row (most[]: the warps its launch bounds allow with 8, 16
// and 32 elements a lane), else 0.
void row_shape(int64_t rows, int64_t cols, bool even, int sms, const int *most, int *el, int *warps)
{
    auto need = [&](int e) { return (cols + 32 * e - 1) / (32 * e); };
    if (!even) *el = cols > 256 && cols <= 512 ? 16 : need(8) <= most[0] ? 8 : 32;
    else if (cols <= 256 || (rows <= sms && need(8) <= most[0])) *el = 8;
    else if (cols <= 512) *el = 16;
    else if (cols <= 1024) *el = rows < 8 * sms ? 16 : 32;
    else *el = need(16) <= most[1] ? 16 : 32;
    const int64_t n = need(*el);
    *warps = n <= most[*el == 8 ? 0 : *el == 16 ? 1 : 2] ? (int)n : 0;
}

constexpr int kNormWarps[3] = {32, 8, 16}, kNormGradWarps[3] = {16, 12, 8};

struct Rows {
    const char *name;
    const void *p;
    int64_t stride;
};

// Whether two row layouts (bytes) touch each other's elements.
bool rows_touch(uintptr_t a, int64_t as, uintptr_t b, int64_t bs, int64_t rows, int64_t len)
{
    const uintptr_t a1 = a + (uintptr_t)((rows - 1) * as + len), b1 = b + (uintptr_t)((rows - 1) * bs + len);
    if (a >= b1 || b >= a1) return false;
    if (as != bs || as <= 0) return true;
    const int64_t d = (int64_t)(a > b ? a - b : b - a) % as;  // interleaved rows of one buffer
    return !(d >= len && as - d >= len);
}
bool ranges_touch(const void *a, int64_t an, const void *b, int64_t bn)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

rr_status check_sizes(int64_t rows, int64_t cols, rr_dtype dtype, rr_dtype wdtype)
{
    if (!float_bytes(dtype)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
    if (!float_bytes(wdtype)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "weight_dtype %d", (int)wdtype);
    if (rows < 0 || rows > ((int64_t)1 << 40)) return step_fail(RR_ERR_INVALID_ARG, "rows %lld", (long long)rows);
    if (cols < 1 || cols > ((int64_t)1 << 31)) return step_fail(RR_ERR_INVALID_ARG, "cols %lld", (long long)cols);
    return RR_OK;
}
rr_status check_stride(const char *name, int64_t stride, int64_t rows, int64_t cols, bool written)
{
    if (stride < 0 || stride > ((int64_t)1 << 40) || (written && rows > 1 && stride < cols))
        return step_fail(RR_ERR_INVALID_ARG, "%s %lld with cols %lld", name, (long long)stride, (long long)cols);
    if (rows > 0 && stride > 0 && rows > ((int64_t)1 << 60) / stride)
        return step_fail(RR_ERR_INVALID_ARG, "%s %lld with rows %lld", name, (long long)stride, (long long)rows);
    return RR_OK;
}
rr_status check_element(const char *name, const void *p, int bytes)
{
    if (!aligned_to(p, bytes)) return step_fail(RR_ERR_ALIGNMENT, "%s not aligned to its %d-byte element", name, bytes);
    return RR_OK;
}

#define RR_TRY(expr)                            \
    do {                                        \
        const rr_status st_ = (expr);           \
        if (st_ != RR_OK) return st_;           \
    } while (0)

// Most partial weight gradients of a call: what the workspace has room for, so a
// function of the sizes alone.  Up to the 8192 columns that row_shape has warps for,
// a block's; of longer rows one for each SM of a GB300 where norm_grad_wide_kernel
// may take them, else what gives norm_grad_columns_kernel tile_blocks() to each of
// those SMs.  A device with more SMs leaves some of them without.
int64_t most_partials(int64_t rows, int64_t cols)
{
    int64_t most = kMaxPartials;
    if (cols > kNormGradWarps[2] * 1024) {
        most = kWidePartials;
        if (cols > kWideThreads * 48) {
            most = 1;
            for (int e : {1, 4, 8}) {  // single elements, vectors of binary32, of the 16-bit types
                const int64_t tiles = (cols + kTileThreads * e - 1) / (kTileThreads * e);
                const int64_t p = (tile_blocks(e > 1) * (int64_t)kWidePartials + tiles - 1) / tiles;
                if (p > most) most = p;
            }
        }
    }
    return rows < most ? rows : most;
}

int64_t row_span(int64_t rows, int64_t stride, int64_t cols) { return (rows - 1) * stride + cols; }

bool vector_rows(const void *p, int64_t stride, int64_t rows, int eb)
{
    return aligned_to(p, 16) && (rows <= 1 || stride * eb % 16 == 0);
}

}  // namespace

// Most dynamic shared memory of a block: the 227 KB of an SM less room for
// the kernels' few static words.
constexpr int kMaxDynamic = 224 * 1024;

rr_status step_fit(const void *fn, int threads, int smem, int *out)
{
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return step_cuda_fail(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lock(g_mu);
    const auto key = std::make_tuple(dev, fn, threads, smem);
    auto it = g_fit.find(key);
    if (it == g_fit.end()) {
        int fit = 0;
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic);
        if (e != cudaSuccess) return step_cuda_fail(e, "cudaFuncSetAttribute(maxDynamicSharedMemorySize)");
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, fn, threads, smem);
        if (e != cudaSuccess) return step_cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
        if (fit < 1) return step_fail(RR_ERR_CUDA, "a block of %d threads does not fit the device", threads);
        it = g_fit.emplace(key, fit).first;
    }
    *out = it->second;
    return RR_OK;
}

rr_status step_sms(int *sms)
{
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return step_cuda_fail(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lock(g_mu);
    auto it = g_sms.find(dev);
    if (it == g_sms.end()) {
        int n = 0;
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return step_cuda_fail(e, "cudaDeviceGetAttribute(multiProcessorCount)");
        it = g_sms.emplace(dev, n).first;
    }
    *sms = it->second;
    return RR_OK;
}

rr_status step_launch(const void *fn, int64_t grid, int threads, int smem, void *args, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *params[1] = {args};
    cudaError_t e = cudaLaunchKernelExC(&cfg, fn, params);
    if (e != cudaSuccess) return step_cuda_fail(e, "cudaLaunchKernelExC");
    return RR_OK;
}

}  // namespace rr

using namespace rr;

extern "C" rr_status rr_layer_norm(const void *x, const void *weight, const void *bias, void *y, float *mean,
                                   float *rstd, int64_t rows, int64_t cols, int64_t x_stride,
                                   int64_t y_stride, float eps, rr_dtype dtype, rr_dtype weight_dtype,
                                   cudaStream_t stream)
try {
    RR_TRY(check_sizes(rows, cols, dtype, weight_dtype));
    RR_TRY(check_stride("x_stride", x_stride, rows, cols, false));
    RR_TRY(check_stride("y_stride", y_stride, rows, cols, true));
    if (!(eps >= 0.0f)) return step_fail(RR_ERR_INVALID_ARG, "eps %g", (double)eps);
    if (rows == 0) return step_ok();
    if (!x || !y) return step_fail(RR_ERR_INVALID_ARG, "%s is NULL", x ? "y" : "x");
    const int eb = float_bytes(dtype), wb = float_bytes(weight_dtype);
    RR_TRY(check_element("x", x, eb));
    RR_TRY(check_element("y", y, eb));
    RR_TRY(check_element("weight", weight, wb));
    RR_TRY(check_element("bias", bias, wb));
    RR_TRY(check_element("mean", mean, 4));
    RR_TRY(check_element("rstd", rstd, 4));
    const int64_t ybytes = row_span(rows, y_stride, cols) * eb, xbytes = row_span(rows, x_stride, cols) * eb;
    if (!(x == y && (x_stride == y_stride || rows == 1)) &&
        rows_touch(reinterpret_cast<uintptr_t>(x), x_stride * eb, reinterpret_cast<uintptr_t>(y), y_stride * eb, rows,
                   cols * eb))
        return step_fail(RR_ERR_ALIAS, "y overlaps x");
    if (ranges_touch(y, ybytes, weight, cols * wb) || ranges_touch(y, ybytes, bias, cols * wb) ||
        ranges_touch(y, ybytes, mean, rows * 4) || ranges_touch(y, ybytes, rstd, rows * 4))
        return step_fail(RR_ERR_ALIAS, "y overlaps another argument");
    for (const float *stat : {mean, rstd})
        if (ranges_touch(stat, rows * 4, x, xbytes) || ranges_touch(stat, rows * 4, weight, cols * wb) ||
            ranges_touch(stat, rows * 4, bias, cols * wb))
            return step_fail(RR_ERR_ALIAS, "a statistic overlaps an input");
    if (ranges_touch(mean, rows * 4, rstd, rows * 4)) return step_fail(RR_ERR_ALIAS, "mean overlaps rstd");

    int sms = 0;
    RR_TRY(step_sms(&sms));
    NormArgs a{x, weight, bias, y, mean, rstd, rows, cols, x_stride, y_stride, eps, (int)weight_dtype};
    int el = 0, warps = 0;
    const bool vec = cols * eb % 16 == 0 && vector_rows(x, x_stride, rows, eb) && vector_rows(y, y_stride, rows, eb);
    row_shape(rows, cols, vec, sms, kNormWarps, &el, &warps);
    const void *fn;
    int threads, smem = 0;
    int64_t blocks;
    if (warps == 0) {
        fn = dtype == RR_FP32   ? norm_long_fn<float>(vec)
             : dtype == RR_BF16 ? norm_long_fn<__nv_bfloat16>(vec) : norm_long_fn<__half>(vec);
        threads = long_threads(vec);
        blocks = rows;
    } else {
        const bool group = warps > 1;
        fn = dtype == RR_FP32 ? norm_rows_fn<float>(el, vec, group)
             : dtype == RR_BF16 ? norm_rows_fn<__nv_bfloat16>(el, vec, group) : norm_rows_fn<__half>(el, vec, group);
        const int64_t per = group ? 1 : rows >= 8 * (int64_t)sms ? 8 : (rows + sms - 1) / sms;  // rows a block has at once
        threads = 32 * (group ? warps : (int)per);
        smem = vec ? ring_rows(el, eb) * threads * el * eb : 0;
        blocks = (rows + per - 1) / per;
    }
    int fit = 0;
    RR_TRY(step_fit(fn, threads, smem, &fit));
    const int64_t most = (int64_t)fit * sms;
    RR_TRY(step_launch(fn, blocks < most ? blocks : most, threads, smem, &a, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}

extern "C" rr_status rr_layer_norm_backward_workspace(int64_t rows, int64_t cols, size_t *bytes)
{
    if (!bytes) return step_fail(RR_ERR_INVALID_ARG, "bytes is NULL");
    RR_TRY(check_sizes(rows, cols, RR_FP32, RR_FP32));
    *bytes = (size_t)(((rows * 8 + 15) & ~(int64_t)15) + 2 * most_partials(rows, cols) * cols * 4);
    return step_ok();
}

extern "C" rr_status rr_layer_norm_backward(const void *dy, const void *x, const void *weight, const float *mean,
                                            const float *rstd, void *dx, void *dweight, void *dbias,
                                            int64_t rows, int64_t cols, int64_t dy_stride, int64_t x_stride,
                                            int64_t dx_stride, rr_dtype dtype, rr_dtype weight_dtype,
                                            void *workspace, size_t workspace_bytes, cudaStream_t stream)
try {
    RR_TRY(check_sizes(rows, cols, dtype, weight_dtype));
    RR_TRY(check_stride("dy_stride", dy_stride, rows, cols, false));
    RR_TRY(check_stride("x_stride", x_stride, rows, cols, false));
    if (dx) RR_TRY(check_stride("dx_stride", dx_stride, rows, cols, true));
    if (!dx && !dweight && !dbias) return step_fail(RR_ERR_INVALID_ARG, "dx, dweight and dbias are all NULL");
    if (rows > 0 && (!dy || !x || !mean || !rstd))
        return step_fail(RR_ERR_INVALID_ARG, "%s is NULL", !dy ? "dy" : !x ? "x" : !mean ? "mean" : "rstd");
    const int eb = float_bytes(dtype), wb = float_bytes(weight_dtype);
    RR_TRY(check_element("dy", dy, eb));
    RR_TRY(check_element("x", x, eb));
    RR_TRY(check_element("dx", dx, eb));
    RR_TRY(check_element("weight", weight, wb));
    RR_TRY(check_element("dweight", dweight, wb));
    RR_TRY(check_element("dbias", dbias, wb));
    RR_TRY(check_element("mean", mean, 4));
    RR_TRY(check_element("rstd", rstd, 4));
    size_t need = 0;
    RR_TRY(rr_layer_norm_backward_workspace(rows, cols, &need));
    if (rows > 0) {
        if (!workspace) return step_fail(RR_ERR_INVALID_ARG, "workspace is NULL");
        if (!aligned_to(workspace, 16)) return step_fail(RR_ERR_ALIGNMENT, "workspace not 16-byte aligned");
        if (workspace_bytes < need)
            return step_fail(RR_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
        const int64_t len = cols * eb;
        struct {
            const char *name;
            const void *p;
            int64_t bytes;
        } in[] = {{"weight", weight, cols * wb}, {"mean", mean, rows * 4}, {"rstd", rstd, rows * 4},
                  {"dy", dy, row_span(rows, dy_stride, cols) * eb}, {"x", x, row_span(rows, x_stride, cols) * eb}},
          out[] = {{"dweight", dweight, cols * wb}, {"dbias", dbias, cols * wb}, {"workspace", workspace, (int64_t)need},
                   {"dx", dx, row_span(rows, dx_stride, cols) * eb}};
        for (int i = 0; i < 4; ++i) {
            for (int j = 0; j < (i == 3 ? 3 : 5); ++j)
                if (ranges_touch(out[i].p, out[i].bytes, in[j].p, in[j].bytes))
                    return step_fail(RR_ERR_ALIAS, "%s overlaps %s", out[i].name, in[j].name);
            for (int j = 0; j < i; ++j)
                if (ranges_touch(out[i].p, out[i].bytes, out[j].p, out[j].bytes))
                    return step_fail(RR_ERR_ALIAS, "%s overlaps %s", out[i].name, out[j].name);
        }
        for (const Rows &r : {Rows{"dy", dy, dy_stride}, Rows{"x", x, x_stride}})
            if (dx && !(dx == r.p && (dx_stride == r.stride || rows == 1)) &&
                rows_touch(reinterpret_cast<uintptr_t>(dx), dx_stride * eb, reinterpret_cast<uintptr_t>(r.p),
                           r.stride * eb, rows, len))
                return step_fail(RR_ERR_ALIAS, "dx overlaps %s", r.name);
    } else if (ranges_touch(dweight, cols * wb, dbias, cols * wb)) {
        return step_fail(RR_ERR_ALIAS, "dbias overlaps dweight");
    }
    if (rows == 0 && !dweight && !dbias) return step_ok();

    int sms = 0;
    RR_TRY(step_sms(&sms));
    const bool sums = dweight || dbias;
    float2 *coef = static_cast<float2 *>(workspace);
    float *part = sums ? reinterpret_cast<float *>(static_cast<char *>(workspace) + ((rows * 8 + 15) & ~(int64_t)15)) : nullptr;
    NormGradArgs a{dy, x, weight, mean, rstd, dx, part, coef, rows, cols, dy_stride, x_stride, dx_stride,
                   (int)weight_dtype, 0};
    if (rows > 0) {
        int el = 0, warps = 0;
        const bool vec = cols * eb % 16 == 0 && vector_rows(dy, dy_stride, rows, eb) &&
                         vector_rows(x, x_stride, rows, eb) && (!dx || vector_rows(dx, dx_stride, rows, eb));
        row_shape(rows, cols, vec, sms, kNormGradWarps, &el, &warps);
        const int64_t most = most_partials(rows, cols);
        // Long rows: one pass over HBM once each SM has a few of them, else the two
        // kernels that share a row among blocks.  Both sides in us: 18944 columns of
        // bf16, 304 rows 43, 23; 608 rows 52, 35; 1216 rows 69, 72; 2432 rows 104,
        // 135.  12288 of binary32, 608 rows 34, 28; 912 rows 43, 43.  12001 uneven, 152
        // rows 15, 17; 608 rows 30, 41; 2432 rows 82, 137.
        if (warps == 0 && cols <= kWideThreads * 48 && rows >= 4 * (int64_t)sms) {
            const int wide = cols <= kWideThreads * 32 ? 32 : cols <= kWideThreads * 40 ? 40 : 48;
            const void *fn = dtype == RR_FP32   ? norm_grad_wide_fn<float>(wide, vec)
                             : dtype == RR_BF16 ? norm_grad_wide_fn<__nv_bfloat16>(wide, vec) : norm_grad_wide_fn<__half>(wide, vec);
            a.P = (int)(sms < most ? sms : most);
            RR_TRY(step_launch(fn, a.P, kWideThreads, 0, &a, stream));
        } else if (warps == 0) {
            const void *means, *columns;
            if (dtype == RR_FP32) norm_grad_long_fn<float>(vec, &means, &columns);
            else if (dtype == RR_BF16) norm_grad_long_fn<__nv_bfloat16>(vec, &means, &columns);
            else norm_grad_long_fn<__half>(vec, &means, &columns);
            const int64_t two = 2 * (int64_t)sms;
            const int64_t tile = kTileThreads * (vec ? 16 / eb : 1), tiles = (cols + tile - 1) / tile;
            RR_TRY(step_launch(means, rows < two ? rows : two, long_threads(vec), 0, &a, stream));
            int64_t P = (tile_blocks(vec) * (int64_t)sms + tiles - 1) / tiles;
            if (P > most) P = most;
            a.P = (int)P;
            RR_TRY(step_launch(columns, P * tiles, kTileThreads, 0, &a, stream));
        } else {
            const bool group = warps > 1;
            const void *fn = dtype == RR_FP32 ? norm_grad_fn<float>(el, vec, group)
                             : dtype == RR_BF16 ? norm_grad_fn<__nv_bfloat16>(el, vec, group)
                                                : norm_grad_fn<__half>(el, vec, group);
            const int64_t per = group ? 1 : rows >= 8 * (int64_t)sms ? 8 : (rows + sms - 1) / sms;
            const int threads = 32 * (group ? warps : (int)per);
            const int ring = vec ? 2 * grad_stages(el) * grad_rows(el, vec) * threads * el * eb : 0, sums_bytes = group ? 0 : threads * el * 8;
            const int smem = ring > sums_bytes ? ring : sums_bytes;
            int fit = 0;
            RR_TRY(step_fit(fn, threads, smem, &fit));
            int64_t blocks = (rows + per - 1) / per;
            if (blocks > (int64_t)fit * sms) blocks = (int64_t)fit * sms;
            // A block's partial sums are written and read again, so it should have
            // 8 rows to itself where that leaves one block to an SM (1024 x 3584
            // bf16: 14.8 us, with every block that fits 19.2).
            const int64_t busy = rows / 8 / per > sms ? rows / 8 / per : sms;
            if (blocks > busy) blocks = busy;
            if (blocks > most) blocks = most;
            a.P = (int)blocks;
            RR_TRY(step_launch(fn, blocks, threads, smem, &a, stream));
        }
    }
    if (sums) {
        NormJoinArgs j{part, dweight, dbias, cols, a.P, (int)weight_dtype};
        RR_TRY(step_launch((const void *)norm_grad_join_kernel, (cols + 31) / 32, 32 * kJoinWarps, 0, &j, stream));
    }
    return step_ok();
} catch (...) {
    return step_no_memory();
}
