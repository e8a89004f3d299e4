// Log-probabilities of tokens, the clipped policy loss and the preference loss,
// with their gradients (include/rr.h: rr_token_logp, rr_token_logp_backward,
// rr_policy_loss, rr_preference_loss).
//
// All of them are row operators over logits x of `vocab` elements: with
// z = x / temperature, M = max(x), s = sum of exp(z - M / temperature),
//   logp = (x_t - M) / temperature - log(s),
//   d logp / d x_j = (1[j = t] - exp(z_j - M / temperature) / s) / temperature.
// A row's maximum and sum are taken in one pass (each thread keeps its own and
// joins them at the end); a gradient needs them first, so it is a second pass
// over the row, which then comes mostly out of the L2.
//
// Bound: HBM.  12288 x 50021 fp16 log-probabilities 192 us (89 % of the copy peak), the
// gradient of 4096 x 32768 bf16 84 (92 %), a policy loss with its gradient of 8192 x
// 131072 bf16 838 (74 % by one read and a write; some rows are read twice, a quarter of
// 2048 in a profile), a preference loss of 4821 rows x 131072, 3866 of them counted, 551
// (two reads and a write, 89 %).  Rows of 1000 to 4096 columns are far from it: a block
// has a few vectors a thread and two joins to wait for (65536 x 1000 bf16
// log-probabilities 252 us, 8 %, and with the policy's gradient 402; 65536 x 4096 310 and
// 526).
//
// Times below are of one GB300 (152 SMs, measured copy 6.7 TB/s).
#include <cmath>
#include <cooperative_groups.h>

#include "rr_step.h"

namespace rr {

namespace {

namespace cg = cooperative_groups;

#define RR_TRY(expr)                  \
    do {                              \
        const rr_status st_ = (expr); \
        if (st_ != RR_OK) return st_; \
    } while (0)

constexpr int kThreads = 256;
constexpr int kBlocks = 4;      // blocks of an SM: one's loads run while another joins its sums
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;      // vectors a thread has in flight
constexpr int kMostCluster = 8; // blocks that share a row
constexpr int64_t kMaxVocab = (int64_t)1 << 31;
constexpr int64_t kMaxRows = (int64_t)1 << 40;
constexpr int kMaxPairs = 1 << 24;
// So that neither 1 / (temperature * log(2)) nor a log-sum times the temperature
// leaves binary32's range.
constexpr float kMinInvT = 0x1p-120f, kMaxInvT = 0x1p127f;

enum Mode { kLogp, kPolicy, kPreference };

struct RowArgs {
    const void *x;
    const int64_t *target;
    int64_t rows, vocab, stride;
    float inv_t, log2_scale;  // 1 / temperature, and that over log(2)
    float *logp, *lse;
    // policy loss
    const float *old_logp, *ref_logp, *advantage, *weight;
    float low, high, kl, grad_scale;
    float *token_loss;
    void *dx;
    int64_t dx_stride;
    // preference loss: rows of [offsets[0], offsets[last]) only; what the gradient takes
    // probabilities from
    const int64_t *offsets;
    int last;
    float *base, *over;
};

// loss = sum / count, in one order.
struct SumArgs {
    const float *part;
    int64_t n;
    double count;
    float *loss;
};
struct GradArgs {
    const void *x;
    const int64_t *target;
    const float *lse;          // or each row's maximum and 1 / sum:
    const float *base, *over;
    const float *dlogp;
    void *dx;
    int64_t rows, vocab, stride, dx_stride;
    float inv_t, log2_scale;
    const int64_t *offsets;  // NULL: all rows
    int last;
    SumArgs sum;             // of the pairs' losses, by the first block; loss NULL: none
};

// A product in which a factor of 0 leaves out what it multiplies, also where that is
// infinite (a masked target, or what binary32 does not hold).  NaN stays NaN.
__device__ __forceinline__ float times(float x, float y)
{
    const float p = x * y;
    return (x == 0.0f && y == y) || (y == 0.0f && x == x) ? 0.0f : p;
}

// An offset kept to the rows on both sides: what rows are counted from must not
// wrap where a thread's number or a stretch of rows is added to it.
__device__ __forceinline__ int64_t row_within(int64_t offset, int64_t rows) { return min(max(offset, (int64_t)0), rows); }

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A maximum and the sum of exponentials relative to it.  An empty part, or one
// of -inf alone, has maximum -inf and sum 0.
struct Stat {
    float top, sum;
};
// What exponents are taken relative to: -inf - -inf is no number.
__device__ __forceinline__ float base_of(float top) { return top == -INFINITY ? 0.0f : top; }
__device__ __forceinline__ Stat join(Stat a, Stat b, float scale)
{
    const float top = fmaxf(a.top, b.top), base = base_of(top);
    return Stat{top, a.sum * exp2_fast((a.top - base) * scale) + b.sum * exp2_fast((b.top - base) * scale)};
}

// The largest of a thread's elements (a NaN among them may be passed over: the sum
// of exponentials keeps it).
__device__ __forceinline__ float largest(const Pack<float, 4> (&v)[kUnroll])
{
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, v[j].v[k]);
    return top;
}
template <class T2, class T>
__device__ __forceinline__ float largest_pairs(const Pack<T, 8> (&v)[kUnroll])
{
    T2 top = *reinterpret_cast<const T2 *>(v[0].v);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
#pragma unroll
        for (int k = j == 0 ? 2 : 0; k < 8; k += 2) top = __hmax2(top, *reinterpret_cast<const T2 *>(v[j].v + k));
    return fmaxf(to_f32(top.x), to_f32(top.y));
}
__device__ __forceinline__ float largest(const Pack<__half, 8> (&v)[kUnroll]) { return largest_pairs<__half2>(v); }
__device__ __forceinline__ float largest(const Pack<__nv_bfloat16, 8> (&v)[kUnroll]) { return largest_pairs<__nv_bfloat162>(v); }

template <class T, int E>
__device__ __forceinline__ void take(Stat &s, const Pack<T, E> (&v)[kUnroll], float scale)
{
    const float top = fmaxf(s.top, largest(v));
    const float base = base_of(top);
    float2 sum = make_float2(s.sum * exp2_fast((s.top - base) * scale), 0.0f);
    const float2 less = both(-base), by = both(scale);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
#pragma unroll
        for (int k = 0; k < E; k += 2) {
            const float2 t = mul2(add2(pair_f32(v[j].v + k), less), by);
            sum = add2(sum, make_float2(exp2_fast(t.x), exp2_fast(t.y)));
        }
    s.top = top;
    s.sum = sum.x + sum.y;
}
__device__ __forceinline__ void take(Stat &s, float x, float scale) { s = join(s, Stat{x, 1.0f}, scale); }

// A row's elements as a block of a cluster takes them: vectors of 16 bytes where
// they are aligned, single elements before and behind.
struct Slice {
    uint32_t first, last;  // this block's elements
    uint32_t v0, v1;       // of which whole aligned vectors lie in [v0, v1)
};
template <class T>
__device__ __forceinline__ Slice slice_of(const T *row, int64_t vocab, int part, int parts)
{
    constexpr int E = 16 / (int)sizeof(T);
    uint32_t head = (16 - (int)(reinterpret_cast<uintptr_t>(row) & 15)) % 16 / (int)sizeof(T);
    if (head > (uint32_t)vocab) head = (uint32_t)vocab;
    const uint32_t n = ((uint32_t)vocab - head) / E, each = n / parts, more = n % parts;
    Slice s;
    s.v0 = head + (part * each + min((uint32_t)part, more)) * E;
    s.v1 = s.v0 + (each + ((uint32_t)part < more ? 1 : 0)) * E;
    s.first = part == 0 ? 0 : s.v0;
    s.last = part == parts - 1 ? (uint32_t)vocab : s.v1;
    return s;
}

template <class T>
__device__ __forceinline__ Stat row_stat(const T *row, const Slice &s, float scale)
{
    constexpr int E = 16 / (int)sizeof(T);
    constexpr uint32_t step = kThreads * E * kUnroll;
    Stat st{-INFINITY, 0.0f};
    Pack<T, E> v[kUnroll];
    uint32_t e = s.v0 + threadIdx.x * E;
    for (; e + (kUnroll - 1) * kThreads * E < s.v1; e += step) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) v[j] = *reinterpret_cast<const Pack<T, E> *>(row + e + j * kThreads * E);
        take(st, v, scale);
    }
    if (e < s.v1) {
#pragma unroll
        for (int j = 0; j < kUnroll; ++j) {
            if (e + j * kThreads * E < s.v1) {
                v[j] = *reinterpret_cast<const Pack<T, E> *>(row + e + j * kThreads * E);
            } else {
#pragma unroll
                for (int k = 0; k < E; ++k) v[j].v[k] = from_f32<T>(-INFINITY);
            }
        }
        take(st, v, scale);
    }
    // fewer than a vector each
    if (s.first + threadIdx.x < s.v0) take(st, to_f32(row[s.first + threadIdx.x]), scale);
    if (s.v1 + threadIdx.x < s.last) take(st, to_f32(row[s.v1 + threadIdx.x]), scale);
    return st;
}

// 16 bytes that lie `by` bytes into 32: by is a multiple of 2, the same for all lanes.
__device__ __forceinline__ uint4 cut_out(uint4 x, uint4 y, uint32_t by)
{
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    if (by & 8) {
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
    }
    if (by & 4) {
#pragma unroll
        for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
    }
    const uint32_t bits = (by & 2) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

// dx_j = -slope * exp2((x_j - base) * scale) * over, plus slope at the target.
// LAST: rows of other blocks wait in the L2 for this pass, so what it has read and
// written leaves the L2 first (policy loss of 8192 x 131072 bf16 935 -> 837 us; the
// gradient by itself is slower for it, 547 -> 559 us of a preference loss).
template <bool LAST, class T>
__device__ __forceinline__ void row_grad(const T *row, T *out, const Slice &s, int64_t vocab, int64_t target, float base,
                                         float scale, float slope, float over)
{
    constexpr int E = 16 / (int)sizeof(T);
    const float factor = -slope * over;
    const uint32_t t = (uint32_t)target;
    auto one = [&](uint32_t i) {
        const float g = exp2_fast((to_f32(row[i]) - base) * scale) * factor;
        out[i] = from_f32<T>(i == t ? g + slope : g);
    };
    const float2 less = both(-base), by = both(scale), f = both(factor);
    auto vector = [&](Pack<T, E> &v, uint32_t at) {
#pragma unroll
        for (int k = 0; k < E; k += 2) {
            const float2 z = mul2(add2(pair_f32(v.v + k), less), by);
            pair_set(v.v + k, mul2(make_float2(exp2_fast(z.x), exp2_fast(z.y)), f));
        }
        if (t - at < E) {  // the target's place, from its own element
#pragma unroll
            for (int k = 0; k < E; ++k)
                if (t - at == k) v.v[k] = from_f32<T>(exp2_fast((to_f32(row[t]) - base) * scale) * factor + slope);
        }
        if (LAST) __stcs(reinterpret_cast<uint4 *>(out + at), *reinterpret_cast<const uint4 *>(v.v));
        else *reinterpret_cast<Pack<T, E> *>(out + at) = v;
    };
    const uint32_t shift = (uint32_t)(reinterpret_cast<uintptr_t>(row) - reinterpret_cast<uintptr_t>(out)) & 15;
    constexpr uint32_t step = kThreads * E * kUnroll;
    if (shift == 0) {
        for (uint32_t e = s.v0 + threadIdx.x * E; e < s.v1; e += step) {
            Pack<T, E> v[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j)
                if (e + j * kThreads * E < s.v1) {
                    if (LAST) *reinterpret_cast<uint4 *>(v[j].v) = __ldcs(reinterpret_cast<const uint4 *>(row + e + j * kThreads * E));
                    else v[j] = *reinterpret_cast<const Pack<T, E> *>(row + e + j * kThreads * E);
                }
#pragma unroll
            for (int j = 0; j < kUnroll; ++j)
                if (e + j * kThreads * E < s.v1) vector(v[j], e + j * kThreads * E);
        }
        if (s.first + threadIdx.x < s.v0) one(s.first + threadIdx.x);
        if (s.v1 + threadIdx.x < s.last) one(s.v1 + threadIdx.x);
        return;
    }
    // The rows are aligned to different places: whole vectors of the output are cut out
    // of two neighbours of the input (2049 x 50021 fp16: element by element 184 us, so
    // 102).  In place it does not come here.
    const Slice o = slice_of(out + s.first, s.last - s.first, 0, 1);  // this block's part, from its first element on
    uint32_t v0 = s.first + o.v0, v1 = s.first + o.v1;
    // both neighbours have to lie in the row
    const uint32_t lead = shift / (uint32_t)sizeof(T);
    if (v0 < lead && v0 < v1) v0 += E;
    while (v0 < v1 && v1 + (E - lead) > (uint32_t)vocab) v1 -= E;
    constexpr int U = kUnroll / 2;
    for (uint32_t e = v0 + threadIdx.x * E; e < v1; e += kThreads * E * U) {
        uint4 x[U], y[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (e + j * kThreads * E < v1) {
                x[j] = *reinterpret_cast<const uint4 *>(row + (e + j * kThreads * E - lead));
                y[j] = *reinterpret_cast<const uint4 *>(row + (e + j * kThreads * E - lead + E));
            }
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (e + j * kThreads * E < v1) {
                const uint4 q = cut_out(x[j], y[j], shift);
                Pack<T, E> v = *reinterpret_cast<const Pack<T, E> *>(&q);
                vector(v, e + j * kThreads * E);
            }
    }
    for (uint32_t i = s.first + threadIdx.x; i < v0; i += kThreads) one(i);
    for (uint32_t i = v1 + threadIdx.x; i < s.last; i += kThreads) one(i);
}

template <class T>
__device__ __forceinline__ void row_zero(T *out, int64_t vocab, int part, int parts)
{
    constexpr int E = 16 / (int)sizeof(T);
    const Slice s = slice_of(out, vocab, part, parts);
    if (s.first + threadIdx.x < s.v0) out[s.first + threadIdx.x] = from_f32<T>(0.0f);
    for (uint32_t e = s.v0 + threadIdx.x * E; e < s.v1; e += kThreads * E)
        *reinterpret_cast<uint4 *>(out + e) = make_uint4(0, 0, 0, 0);
    if (s.v1 + threadIdx.x < s.last) out[s.v1 + threadIdx.x] = from_f32<T>(0.0f);
}

// A row to a cluster of blocks (of one, mostly).  The policy loss spills 20 to 40 bytes
// a thread at its 64 registers.
template <class T, Mode MODE>
__global__ void __launch_bounds__(kThreads, kBlocks) row_kernel(const __grid_constant__ RowArgs a)
{
    stream_order();
    const cg::cluster_group cluster = cg::this_cluster();
    const int parts = (int)cluster.num_blocks(), part = (int)cluster.block_rank();
    __shared__ Stat of_warp[2][kWarps];
    __shared__ Stat of_block[2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t row = blockIdx.x / parts, end = a.rows;
    const int64_t every = gridDim.x / parts;
    if (MODE == kPreference) {
        const int64_t first = row_within(a.offsets[0], a.rows);
        end = row_within(a.offsets[a.last], a.rows);
        if (first > row) row += (first - row + every - 1) / every * every;
    }
    int turn = 0;
    for (; row < end; row += every) {
        const T *x = static_cast<const T *>(a.x) + row * a.stride;
        T *dx = a.dx ? static_cast<T *>(a.dx) + row * a.dx_stride : nullptr;
        const int64_t target = a.target[row];
        if (target < 0 || target >= a.vocab) {  // the same for every block of the cluster
            if (part == 0 && threadIdx.x == 0) {
                a.logp[row] = 0.0f;
                if (MODE == kLogp && a.lse) a.lse[row] = 0.0f;
                if (MODE == kPolicy) a.token_loss[row] = 0.0f;
            }
            if (MODE == kPolicy && dx) row_zero(dx, a.vocab, part, parts);
            continue;
        }
        const float xt = to_f32(x[target]);
        const Slice slice = slice_of(x, a.vocab, part, parts);
        Stat s = row_stat(x, slice, a.log2_scale);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s = join(s, Stat{__shfl_xor_sync(~0u, s.top, o), __shfl_xor_sync(~0u, s.sum, o)}, a.log2_scale);
        if (lane == 0) of_warp[turn][warp] = s;
        __syncthreads();
        s = lane < kWarps ? of_warp[turn][lane] : Stat{-INFINITY, 0.0f};
#pragma unroll
        for (int o = 16; o; o >>= 1)
            s = join(s, Stat{__shfl_xor_sync(~0u, s.top, o), __shfl_xor_sync(~0u, s.sum, o)}, a.log2_scale);
        if (parts > 1) {
            if (threadIdx.x == 0) of_block[turn] = s;
            cluster.sync();
            s = lane < parts ? *cluster.map_shared_rank(&of_block[turn], lane) : Stat{-INFINITY, 0.0f};
#pragma unroll
            for (int o = kMostCluster / 2; o; o >>= 1)
                s = join(s, Stat{__shfl_xor_sync(~0u, s.top, o), __shfl_xor_sync(~0u, s.sum, o)}, a.log2_scale);
            s.top = __shfl_sync(~0u, s.top, 0);
            s.sum = __shfl_sync(~0u, s.sum, 0);
        }
        turn ^= 1;
        const float log_sum = logf(s.sum), logp = (xt - s.top) * a.inv_t - log_sum;
        const bool first = part == 0 && threadIdx.x == 0;
        if (first) {
            a.logp[row] = logp;
            if (MODE == kLogp && a.lse) a.lse[row] = s.top * a.inv_t + log_sum;
            if (MODE == kPreference) {
                a.base[row] = base_of(s.top);
                a.over[row] = 1.0f / s.sum;
            }
        }
        if (MODE == kPolicy) {
            const float weight = a.weight ? a.weight[row] : 1.0f, adv = a.advantage[row];
            const float ratio = a.old_logp ? expf(logp - a.old_logp[row]) : 1.0f;
            const float free = times(ratio, adv), held = times(fminf(fmaxf(ratio, a.low), a.high), adv);
            const bool passes = !(free > held);  // NaN passes
            const float loss = passes ? -free : -held, slope = passes ? -free : 0.0f;
            float apart = 0.0f, pull = 0.0f;  // of the KL term
            if (a.ref_logp) {
                const float gap = a.ref_logp[row] - logp, back = expm1f(gap);
                apart = times(a.kl, back < INFINITY ? back - gap : back);  // of a masked target both are infinite
                pull = times(a.kl, back);
            }
            // without a factor the parts are 0 each: infinite ones do not meet first
            if (first)
                a.token_loss[row] = weight == 0.0f ? times(loss, 0.0f) + times(apart, 0.0f) : (loss + apart) * weight;
            if (dx)
                row_grad<true>(x, dx, slice, a.vocab, target, base_of(s.top), a.log2_scale,
                               weight == 0.0f || a.grad_scale == 0.0f ? times(slope, 0.0f) + times(pull, 0.0f)
                                                                      : (slope - pull) * weight * a.grad_scale * a.inv_t,
                               1.0f / s.sum);
        }
    }
    if (parts > 1) cluster.sync();  // a block's shared memory stays until the others have read it
}

__device__ __forceinline__ void take_sum(const SumArgs &a, double *s)
{
    double sum = 0.0;
    for (int64_t i = threadIdx.x; i < a.n; i += kThreads) sum += (double)a.part[i];
    sum = block_sum64<kWarps>(sum, s);
    if (threadIdx.x == 0) *a.loss = (float)(sum / a.count);
}

// The gradient of log-probabilities whose sums are known: a row to a block, or
// to `parts` blocks that do not meet.  exp(z - lse) carries lse's rounding, 1e-5 of
// a probability where logits lie around 1000; it is what rr_token_logp_backward's
// caller hands over.  The preference loss keeps the maximum and the sum apart
// (3e-7 wherever logits lie).
template <class T>
__global__ void __launch_bounds__(kThreads, kBlocks) row_grad_kernel(const __grid_constant__ GradArgs a, int parts)
{
    stream_order();
    __shared__ double s[kWarps];
    if (blockIdx.x == 0 && a.sum.loss) take_sum(a.sum, s);
    int64_t first = 0, end = a.rows;
    if (a.offsets) {
        first = row_within(a.offsets[0], a.rows);
        end = row_within(a.offsets[a.last], a.rows);
    }
    const int64_t every = gridDim.x / parts;
    const int part = (int)(blockIdx.x % parts);
    // From the last row on: the sums' pass has read it last, so it may still be in the L2.
    for (int64_t row = end - 1 - blockIdx.x / parts; row >= first; row -= every) {
        const T *x = static_cast<const T *>(a.x) + row * a.stride;
        T *dx = static_cast<T *>(a.dx) + row * a.dx_stride;
        const int64_t target = a.target[row];
        if (target < 0 || target >= a.vocab)
            row_zero(dx, a.vocab, part, parts);
        else
            row_grad<false>(x, dx, slice_of(x, a.vocab, part, parts), a.vocab, target,
                            a.lse ? a.lse[row] / a.inv_t : a.base[row], a.log2_scale, a.dlogp[row] * a.inv_t,
                            a.lse ? 1.0f : a.over[row]);
    }
}

// ---------------------------------------------------------------- pairs of sequences
struct PairArgs {
    const float *logp, *ref;
    const int64_t *target, *offsets;
    int64_t rows, vocab;
    int pairs;
    float beta, smoothing, margin, grad_scale;
    bool average;
    float *seq_logp, *loss, *slope;  // of each sequence, pair and row
};

// log(1 + exp(x)) without overflow.
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }

// A block a pair: sums of log-probabilities, the pair's loss, the slope of every row.
__global__ void __launch_bounds__(kThreads) pair_kernel(const __grid_constant__ PairArgs a)
{
    stream_order();
    __shared__ double s[kWarps];
    const int p = blockIdx.x;
    int64_t lo[2], hi[2];
    double mean[2], count[2];
    for (int k = 0; k < 2; ++k) {
        const int q = p + k * a.pairs;
        lo[k] = row_within(a.offsets[q], a.rows);
        hi[k] = row_within(a.offsets[q + 1], a.rows);
        double sum = 0.0, n = 0.0;
        for (int64_t i = lo[k] + threadIdx.x; i < hi[k]; i += kThreads) {
            const int64_t t = a.target[i];
            if (t >= 0 && t < a.vocab) {
                sum += (double)a.logp[i];
                n += 1.0;
            }
        }
        sum = block_sum64<kWarps>(sum, s);
        count[k] = a.average ? fmax(1.0, block_sum64<kWarps>(n, s)) : 1.0;
        mean[k] = sum / count[k];
        if (threadIdx.x == 0) a.seq_logp[q] = (float)mean[k];
    }
    double gap = mean[0] - mean[1];
    if (a.ref) gap -= (double)a.ref[p] - (double)a.ref[p + a.pairs];
    const float h = (float)((double)a.beta * gap - (double)a.margin);
    if (threadIdx.x == 0) a.loss[p] = times(1.0f - a.smoothing, softplus(-h)) + times(a.smoothing, softplus(h));
    if (!a.slope) return;
    // d loss / d h = smoothing * sigmoid(h) - (1 - smoothing) * sigmoid(-h)
    const float e = expf(-fabsf(h)), small = e / (1.0f + e), large = 1.0f / (1.0f + e);
    const float up = h >= 0.0f ? large : small, down = h >= 0.0f ? small : large;
    const float dh = (a.smoothing * up - (1.0f - a.smoothing) * down) * a.beta / (float)a.pairs * a.grad_scale;
    for (int k = 0; k < 2; ++k) {
        const float slope = (k ? -dh : dh) / (float)count[k];
        for (int64_t i = lo[k] + threadIdx.x; i < hi[k]; i += kThreads) a.slope[i] = slope;
    }
}

__global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ SumArgs a)
{
    stream_order();
    __shared__ double s[kWarps];
    take_sum(a, s);
}

// ---------------------------------------------------------------- host side
struct Range {
    const char *name;
    const void *p;
    int64_t bytes;
};
bool ranges_touch(const Range &a, const Range &b)
{
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
// Nothing written may overlap anything else.
template <size_t N, size_t M>
rr_status check_apart(const Range (&out)[N], const Range (&in)[M])
{
    for (size_t i = 0; i < N; ++i) {
        for (size_t j = 0; j < M; ++j)
            if (ranges_touch(out[i], in[j])) return step_fail(RR_ERR_ALIAS, "%s overlaps %s", out[i].name, in[j].name);
        for (size_t j = 0; j < i; ++j)
            if (ranges_touch(out[i], out[j])) return step_fail(RR_ERR_ALIAS, "%s overlaps %s", out[i].name, out[j].name);
    }
    return RR_OK;
}

rr_status check_rows(int64_t rows, int64_t vocab, int64_t stride, float inv_t, rr_dtype dtype)
{
    if (!float_bytes(dtype)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "dtype %d", (int)dtype);
    if (rows < 0 || rows > kMaxRows) return step_fail(RR_ERR_INVALID_ARG, "rows %lld", (long long)rows);
    if (vocab < 1 || vocab > kMaxVocab) return step_fail(RR_ERR_INVALID_ARG, "vocab %lld", (long long)vocab);
    if (rows > 1 && (stride < vocab || stride > kMaxRows))
        return step_fail(RR_ERR_INVALID_ARG, "logits_stride %lld, vocab %lld", (long long)stride, (long long)vocab);
    if (rows > 1 && rows > INT64_MAX / 8 / stride) return step_fail(RR_ERR_INVALID_ARG, "rows %lld of logits_stride %lld", (long long)rows, (long long)stride);
    if (!(inv_t >= kMinInvT && inv_t <= kMaxInvT)) return step_fail(RR_ERR_INVALID_ARG, "inv_temperature %g", (double)inv_t);
    return RR_OK;
}
rr_status check_grad(const void *logits, const void *dlogits, int64_t rows, int64_t vocab, int64_t stride,
                     int64_t dstride, int eb)
{
    if (rows > 1 && (dstride < vocab || dstride > kMaxRows || rows > INT64_MAX / 8 / dstride))
        return step_fail(RR_ERR_INVALID_ARG, "dlogits_stride %lld, vocab %lld", (long long)dstride, (long long)vocab);
    if (!aligned_to(dlogits, eb)) return step_fail(RR_ERR_ALIGNMENT, "dlogits not %d-byte aligned", eb);
    const bool in_place = dlogits == logits && (dstride == stride || rows <= 1);
    const Range out[] = {{"dlogits", dlogits, ((rows - 1) * dstride + vocab) * eb}};
    const Range in[] = {{"logits", in_place ? nullptr : logits, ((rows - 1) * stride + vocab) * eb}};
    return check_apart(out, in);
}
rr_status check_word(const char *name, const void *p, int bytes, bool needed)
{
    if (needed && !p) return step_fail(RR_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned_to(p, bytes)) return step_fail(RR_ERR_ALIGNMENT, "%s not %d-byte aligned", name, bytes);
    return RR_OK;
}

template <Mode MODE>
const void *row_fn(rr_dtype d)
{
    return d == RR_FP32 ? (const void *)row_kernel<float, MODE>
           : d == RR_BF16 ? (const void *)row_kernel<__nv_bfloat16, MODE> : (const void *)row_kernel<__half, MODE>;
}

// Blocks that share a row: as many as all fit at once where rows are few; with a
// second pass (the policy loss's gradient) at least so many that the rows under way
// stay in the L2 until then (without a gradient too: the loss is the same).  8192 x
// 131072 bf16: 85 MB of them 837 us, 160 MB 904, 43 MB 1039 (blocks that share a row
// wait for one another).  The border rests on that one vocabulary: bf16 rows of 73297
// columns and more get two blocks (8192 x 100000 658 us, 74 % of the copy peak by one
// read and a write; x 146000 1012, 71 %), of 146594 and more four, which is too many
// (x 152064 1405, 53 %; x 200064 1861), and binary32 rows of 73297 and more as well
// (4096 x 65536 419, 77 %; x 128256 1139, 55 %).
constexpr int64_t kRowsInL2 = (int64_t)85 << 20;
int blocks_to_a_row(int64_t rows, int64_t vocab, int eb, int64_t blocks, bool again)
{
    int parts = 1;
    while (parts < kMostCluster && vocab * eb / (parts * 2) >= 8192 &&
           (rows * parts * 2 <= blocks || (again && blocks / parts * vocab * eb > kRowsInL2)))
        parts *= 2;
    return parts;
}

rr_status launch_rows(const void *fn, RowArgs &a, rr_dtype dtype, bool again, cudaStream_t stream)
{
    int sms = 0, fit = 0;
    RR_TRY(step_sms(&sms));
    RR_TRY(step_fit(fn, kThreads, 0, &fit));
    const int parts = blocks_to_a_row(a.rows, a.vocab, float_bytes(dtype), (int64_t)fit * sms, again);
    int64_t clusters = a.rows;
    if (clusters > (int64_t)fit * sms / parts) clusters = (int64_t)fit * sms / parts;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    void *args[] = {&a};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    return e == cudaSuccess ? RR_OK : step_cuda_fail(e, "kernel launch");
}

rr_status launch_grad(GradArgs &a, rr_dtype dtype, cudaStream_t stream)
{
    const void *fn = dtype == RR_FP32   ? (const void *)row_grad_kernel<float>
                     : dtype == RR_BF16 ? (const void *)row_grad_kernel<__nv_bfloat16> : (const void *)row_grad_kernel<__half>;
    int sms = 0, fit = 0;
    RR_TRY(step_sms(&sms));
    RR_TRY(step_fit(fn, kThreads, 0, &fit));
    int parts = blocks_to_a_row(a.rows, a.vocab, float_bytes(dtype), (int64_t)fit * sms, false);
    int64_t teams = a.rows;
    if (teams * parts > (int64_t)fit * sms) teams = (int64_t)fit * sms / parts;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(teams * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    void *args[] = {&a, &parts};
    const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
    return e == cudaSuccess ? RR_OK : step_cuda_fail(e, "kernel launch");
}

float log2_scale(float inv_t) { return (float)((double)inv_t * 1.4426950408889634); }
int64_t span(int64_t rows, int64_t stride, int64_t vocab, int eb) { return ((rows - 1) * stride + vocab) * eb; }

rr_status launch_sum(const float *part, int64_t n, double count, float *loss, cudaStream_t stream)
{
    SumArgs a{part, n, count, loss};
    return step_launch((const void *)sum_kernel, 1, kThreads, 0, &a, stream);
}

// Workspace of the preference loss: each row's maximum, 1 / sum and slope, each pair's loss.
int64_t padded(int64_t floats) { return (floats + 3) & ~(int64_t)3; }

}  // namespace

}  // namespace rr

using namespace rr;

extern "C" rr_status rr_token_logp(const void *logits, const int64_t *targets, float *logp, float *lse, int64_t rows,
                                   int64_t vocab, int64_t logits_stride, float inv_temperature, rr_dtype dtype,
                                   cudaStream_t stream)
try {
    RR_TRY(check_rows(rows, vocab, logits_stride, inv_temperature, dtype));
    if (rows == 0) return step_ok();
    const int eb = float_bytes(dtype);
    RR_TRY(check_word("logits", logits, eb, true));
    RR_TRY(check_word("targets", targets, 8, true));
    RR_TRY(check_word("logp", logp, 4, true));
    RR_TRY(check_word("lse", lse, 4, false));
    const Range out[] = {{"logp", logp, rows * 4}, {"lse", lse, rows * 4}};
    const Range in[] = {{"logits", logits, span(rows, logits_stride, vocab, eb)}, {"targets", targets, rows * 8}};
    RR_TRY(check_apart(out, in));
    RowArgs a = {};
    a.x = logits;
    a.target = targets;
    a.rows = rows;
    a.vocab = vocab;
    a.stride = logits_stride;
    a.inv_t = inv_temperature;
    a.log2_scale = log2_scale(inv_temperature);
    a.logp = logp;
    a.lse = lse;
    RR_TRY(launch_rows(row_fn<kLogp>(dtype), a, dtype, false, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}

extern "C" rr_status rr_token_logp_backward(const void *logits, const int64_t *targets, const float *lse,
                                            const float *dlogp, void *dlogits, int64_t rows, int64_t vocab,
                                            int64_t logits_stride, int64_t dlogits_stride, float inv_temperature,
                                            rr_dtype dtype, cudaStream_t stream)
try {
    RR_TRY(check_rows(rows, vocab, logits_stride, inv_temperature, dtype));
    if (rows == 0) return step_ok();
    const int eb = float_bytes(dtype);
    RR_TRY(check_word("logits", logits, eb, true));
    RR_TRY(check_word("targets", targets, 8, true));
    RR_TRY(check_word("lse", lse, 4, true));
    RR_TRY(check_word("dlogp", dlogp, 4, true));
    RR_TRY(check_word("dlogits", dlogits, eb, true));
    RR_TRY(check_grad(logits, dlogits, rows, vocab, logits_stride, dlogits_stride, eb));
    const Range out[] = {{"dlogits", dlogits, span(rows, dlogits_stride, vocab, eb)}};
    const Range in[] = {{"targets", targets, rows * 8}, {"lse", lse, rows * 4}, {"dlogp", dlogp, rows * 4}};
    RR_TRY(check_apart(out, in));
    GradArgs a{logits, targets, lse, nullptr, nullptr, dlogp, dlogits, rows, vocab, logits_stride, dlogits_stride, inv_temperature,
               log2_scale(inv_temperature), nullptr, 0, {}};
    RR_TRY(launch_grad(a, dtype, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}

extern "C" rr_status rr_policy_loss(const void *logits, const int64_t *targets, const float *old_logp,
                                    const float *ref_logp, const float *advantages, const float *weights, float *loss,
                                    float *token_loss, float *logp, void *dlogits, int64_t rows, int64_t vocab,
                                    int64_t logits_stride, int64_t dlogits_stride, const rr_policy_hyper *hyper,
                                    rr_dtype dtype, cudaStream_t stream)
try {
    if (!hyper) return step_fail(RR_ERR_INVALID_ARG, "hyper is NULL");
    const float inv_t = (float)hyper->inv_temperature;
    RR_TRY(check_rows(rows, vocab, logits_stride, inv_t, dtype));
    if (!(hyper->clip_low >= 0.0 && hyper->clip_high >= 0.0))
        return step_fail(RR_ERR_INVALID_ARG, "clip_low %g, clip_high %g", hyper->clip_low, hyper->clip_high);
    if (!std::isfinite((float)hyper->kl_coef)) return step_fail(RR_ERR_INVALID_ARG, "kl_coef %g", hyper->kl_coef);
    if (!std::isfinite((float)hyper->grad_scale)) return step_fail(RR_ERR_INVALID_ARG, "grad_scale %g", hyper->grad_scale);
    RR_TRY(check_word("loss", loss, 4, false));
    if (rows == 0) {
        if (loss) RR_TRY(launch_sum(nullptr, 0, 1.0, loss, stream));
        return step_ok();
    }
    const int eb = float_bytes(dtype);
    RR_TRY(check_word("logits", logits, eb, true));
    RR_TRY(check_word("targets", targets, 8, true));
    RR_TRY(check_word("old_logp", old_logp, 4, false));
    RR_TRY(check_word("ref_logp", ref_logp, 4, false));
    RR_TRY(check_word("advantages", advantages, 4, true));
    RR_TRY(check_word("weights", weights, 4, false));
    RR_TRY(check_word("token_loss", token_loss, 4, true));
    RR_TRY(check_word("logp", logp, 4, true));
    if (dlogits) RR_TRY(check_grad(logits, dlogits, rows, vocab, logits_stride, dlogits_stride, eb));
    const Range out[] = {{"loss", loss, 4}, {"token_loss", token_loss, rows * 4}, {"logp", logp, rows * 4}};
    const Range in[] = {{"logits", logits, span(rows, logits_stride, vocab, eb)}, {"targets", targets, rows * 8},
                        {"old_logp", old_logp, rows * 4}, {"ref_logp", ref_logp, rows * 4},
                        {"advantages", advantages, rows * 4}, {"weights", weights, rows * 4},
                        {"dlogits", dlogits, dlogits ? span(rows, dlogits_stride, vocab, eb) : 0}};
    RR_TRY(check_apart(out, in));
    const Range dout[] = {{"dlogits", dlogits, dlogits ? span(rows, dlogits_stride, vocab, eb) : 0}};
    const Range din[] = {in[1], in[2], in[3], in[4], in[5]};
    RR_TRY(check_apart(dout, din));
    RowArgs a = {};
    a.x = logits;
    a.target = targets;
    a.rows = rows;
    a.vocab = vocab;
    a.stride = logits_stride;
    a.inv_t = inv_t;
    a.log2_scale = log2_scale(inv_t);
    a.logp = logp;
    a.old_logp = old_logp;
    a.ref_logp = ref_logp;
    a.advantage = advantages;
    a.weight = weights;
    a.low = (float)(1.0 - hyper->clip_low);
    a.high = (float)(1.0 + hyper->clip_high);
    a.kl = (float)hyper->kl_coef;
    a.grad_scale = (float)hyper->grad_scale;
    a.token_loss = token_loss;
    a.dx = dlogits;
    a.dx_stride = dlogits_stride;
    RR_TRY(launch_rows(row_fn<kPolicy>(dtype), a, dtype, true, stream));
    if (loss) RR_TRY(launch_sum(token_loss, rows, 1.0, loss, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}

extern "C" rr_status rr_preference_loss_workspace(int64_t rows, int pairs, size_t *bytes)
{
    if (!bytes) return step_fail(RR_ERR_INVALID_ARG, "bytes is NULL");
    if (rows < 0 || rows > kMaxRows) return step_fail(RR_ERR_INVALID_ARG, "rows %lld", (long long)rows);
    if (pairs < 1 || pairs > kMaxPairs) return step_fail(RR_ERR_INVALID_ARG, "pairs %d", pairs);
    *bytes = (size_t)(3 * padded(rows) + padded(pairs)) * 4;
    return step_ok();
}

extern "C" rr_status rr_preference_loss(const void *logits, const int64_t *targets, const int64_t *offsets,
                                        const float *ref_logp, float *loss, float *seq_logp, float *logp, void *dlogits,
                                        int64_t rows, int64_t vocab, int64_t logits_stride, int64_t dlogits_stride,
                                        int pairs, const rr_preference_hyper *hyper, rr_dtype dtype, void *workspace,
                                        size_t workspace_bytes, cudaStream_t stream)
try {
    if (!hyper) return step_fail(RR_ERR_INVALID_ARG, "hyper is NULL");
    const float inv_t = (float)hyper->inv_temperature;
    RR_TRY(check_rows(rows, vocab, logits_stride, inv_t, dtype));
    size_t need = 0;
    RR_TRY(rr_preference_loss_workspace(rows, pairs, &need));
    if (!std::isfinite((float)hyper->beta)) return step_fail(RR_ERR_INVALID_ARG, "beta %g", hyper->beta);
    if (!(hyper->label_smoothing >= 0.0 && hyper->label_smoothing <= 1.0))
        return step_fail(RR_ERR_INVALID_ARG, "label_smoothing %g", hyper->label_smoothing);
    if (!std::isfinite((float)hyper->margin)) return step_fail(RR_ERR_INVALID_ARG, "margin %g", hyper->margin);
    if (!std::isfinite((float)hyper->grad_scale)) return step_fail(RR_ERR_INVALID_ARG, "grad_scale %g", hyper->grad_scale);
    const int eb = float_bytes(dtype);
    RR_TRY(check_word("logits", logits, eb, rows > 0));
    RR_TRY(check_word("targets", targets, 8, rows > 0));
    RR_TRY(check_word("offsets", offsets, 8, true));
    RR_TRY(check_word("ref_logp", ref_logp, 4, false));
    RR_TRY(check_word("loss", loss, 4, true));
    RR_TRY(check_word("seq_logp", seq_logp, 4, true));
    RR_TRY(check_word("logp", logp, 4, rows > 0));
    if (!workspace) return step_fail(RR_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned_to(workspace, 16)) return step_fail(RR_ERR_ALIGNMENT, "workspace not 16-byte aligned");
    if (workspace_bytes < need)
        return step_fail(RR_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if (rows > 0 && dlogits) RR_TRY(check_grad(logits, dlogits, rows, vocab, logits_stride, dlogits_stride, eb));
    const int64_t seqs = 2 * (int64_t)pairs, in_bytes = rows > 0 ? span(rows, logits_stride, vocab, eb) : 0;
    const int64_t out_bytes = rows > 0 && dlogits ? span(rows, dlogits_stride, vocab, eb) : 0;
    const Range out[] = {{"loss", loss, 4}, {"seq_logp", seq_logp, seqs * 4}, {"logp", logp, rows * 4},
                         {"workspace", workspace, (int64_t)need}};
    const Range in[] = {{"logits", logits, in_bytes}, {"targets", targets, rows * 8}, {"offsets", offsets, (seqs + 1) * 8},
                        {"ref_logp", ref_logp, seqs * 4}, {"dlogits", dlogits, out_bytes}};
    RR_TRY(check_apart(out, in));
    const Range dout[] = {{"dlogits", dlogits, out_bytes}};
    const Range din[] = {in[1], in[2], in[3]};
    RR_TRY(check_apart(dout, din));

    float *base = static_cast<float *>(workspace), *over = base + padded(rows), *slope = over + padded(rows);
    float *pair_loss = slope + padded(rows);
    if (rows > 0) {
        RowArgs a = {};
        a.x = logits;
        a.target = targets;
        a.rows = rows;
        a.vocab = vocab;
        a.stride = logits_stride;
        a.inv_t = inv_t;
        a.log2_scale = log2_scale(inv_t);
        a.logp = logp;
        a.base = base;
        a.over = over;
        a.offsets = offsets;
        a.last = (int)seqs;
        RR_TRY(launch_rows(row_fn<kPreference>(dtype), a, dtype, false, stream));
    }
    PairArgs p{logp, ref_logp, targets, offsets, rows, vocab, pairs, (float)hyper->beta, (float)hyper->label_smoothing,
               (float)hyper->margin, (float)hyper->grad_scale, hyper->average != 0, seq_logp, pair_loss,
               dlogits ? slope : nullptr};
    RR_TRY(step_launch((const void *)pair_kernel, pairs, kThreads, 0, &p, stream));
    if (rows == 0 || !dlogits) {
        RR_TRY(launch_sum(pair_loss, pairs, (double)pairs, loss, stream));
    } else {
        GradArgs g{logits, targets, nullptr, base, over, slope, dlogits, rows, vocab, logits_stride, dlogits_stride, inv_t,
                   log2_scale(inv_t), offsets, (int)seqs, {pair_loss, pairs, (double)pairs, loss}};
        RR_TRY(launch_grad(g, dtype, stream));
    }
    return step_ok();
} catch (...) {
    return step_no_memory();
}
