// Orthogonalisation of matrices by Newton-Schulz products and the Muon step
// (include/rr.h: rr_orthogonalize, rr_muon).
//
// With X the matrix or its transpose, whichever has the fewer rows, divided by
// its Frobenius norm, each iteration is three products on the short side m:
//   A = X X',  B = a I + b A + c A A,  X <- B X.
// They run on the tensor cores (tcgen05, accumulators in TMEM) over a list of
// matrices at once: a launch takes one product of every matrix of the list.
//
// Operands are pairs of binary16 pieces, v * scale = hi + lo, 22 bits together,
// and a product is hi hi + hi lo + lo hi: the iteration amplifies what small
// singular values are off by some hundred times, so that one bf16 piece (8 bits)
// leaves 1 to 7 % in the result, one fp16 piece 0.2 to 0.9 %, and the pairs
// about 1e-6, as binary32 products do.
//
// The tensor cores' accumulator drops what lies below its last bit at every
// instruction of 16 values (measured 4.6e-8 of the sum each, all one way: 1.5e-4
// after the 18944 of a long row).  So it sums 64 values only, the small products
// first, and is then added to sums in registers, rounded to nearest, while the next
// 64 go to a second accumulator.
//
// Next to products in binary32 that leaves fewer bits in three places: operands have
// 22 bits for 24, the product of the two low pieces is dropped, and what lies below
// 2^-36 is (half the smallest binary16 over the scale: elements of X under 1e-4 lose
// bits).  Results are 0.5 to 2.2 times as far from 64 bits as binary32 products leave
// them (4e-6 at most on drawn matrices of 32 to 8192 a side).
//
// Operands live in the workspace in blocks of 128 rows x 64 columns, both pieces
// one after the other (16 KB each), rows of 128 bytes with their 16-byte pieces
// permuted as the tensor cores' 128-byte swizzle wants them.  A block comes to
// shared memory by one plain bulk copy, and the same bytes serve as an operand
// along either side: rows of K values for X X' and, column by column, K rows for
// B X.  Sizes are padded with zeros to whole tiles of 128.
//
// Times below are of one GB300 (152 SMs, measured 2.01 PFLOP/s bf16).
#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "rr_ring.h"
#include "rr_spans.h"
#include "rr_step.h"

namespace rr {

namespace {

#define RR_TRY(expr)                  \
    do {                              \
        const rr_status st_ = (expr); \
        if (st_ != RR_OK) return st_; \
    } while (0)

constexpr int kThreads = 256;     // of the kernels that stream
constexpr int kTile = 128;        // rows and columns of a block's tile in memory
constexpr int kK = 64;            // columns of a block of an operand: the depth of a stage
constexpr int kPiece = kTile * kK * 2;  // bytes of one piece of a block
constexpr int kBlock = 2 * kPiece;
constexpr int kSumWarps = 8;      // warps that sum the stages' products and write results
constexpr int kGemmThreads = 32 * (kSumWarps + 4);  // and one that copies, one that multiplies, two idle
// Registers of a summing warp's threads and of the others': the launch has 168 each.
// (128 sums and 16 values on their way do not fit 168 with what else a thread holds:
// they spilled, and a stage's sums took 2500 cycles where the products take 1536.)
constexpr int kSumRegisters = 216, kOtherRegisters = 72;
static_assert(kSumWarps * kSumRegisters + 4 * kOtherRegisters <= (kSumWarps + 4) * 168, "more than the launch has");
constexpr int kDesk = 32 * 128;   // bytes of a summing warp's own: 32 x 32 sums

enum Kind { kSums, kSplit, kGram256, kNext256, kGram128, kNext128, kKinds };

// A pair of blocks works on 256 rows x N columns.  256 columns read least; 128
// where there are few tiles, or where they fill the last wave of pairs better.
template <int N>
struct Shape {
    static constexpr int half = N / 2;                       // columns of the right operand that a block holds
    static constexpr int right = half * kK * 4;              // bytes of them, both pieces
    static constexpr int stage = kBlock + right;
    static constexpr int stages = N == 256 ? 3 : 4;
    static constexpr int desks = stages * stage, barriers = desks + kSumWarps * kDesk;
    static constexpr int smem = barriers + 256 + 1024;       // 1024 to start on a swizzle's boundary
    static constexpr __device__ int units(bool next) { return N == 256 ? (next ? kNext256 : kGram256) : (next ? kNext128 : kGram128); }
};
constexpr int kSumBlocks = 1024;  // most partial sums of a matrix's norm
constexpr int kCapSmall = 16, kCap = 160;
constexpr int64_t kMaxSide = (int64_t)1 << 20;
constexpr int kMaxSteps = 64;
// Scales of the pieces: X, A and B hold values up to 32 in magnitude, and values
// of 1e-4 still have all 22 bits.
constexpr float kScale = 0x1p11f, kUnscale = 0x1p-11f;

enum Stage { kStageGram, kStageSquare, kStageNext, kStageLast };

struct Item {
    const void *src;   // the matrix, or its gradient
    float *momentum;   // NULL: no step, the matrix itself is orthogonalised
    void *out;         // result or parameter
    float *master;
    char *x, *y, *a, *b;  // blocked operands; X and its successor swap
    double *part;
    int64_t size;
    int m, n;          // short and long side
    int mt, nt;        // tiles of them
    float scale;       // of the step
    bool tall;         // the matrix has n rows: X is its transpose
};

template <int CAP>
struct Args {
    Item item[CAP];
    int start[kKinds][CAP + 1];  // first unit of work of each matrix; start[.][count] = all
    int count;
    int src_dtype, out_dtype;
    double eps;
    float momentum, fresh, keep;  // beta; 1 - beta and 1 - lr * weight_decay, formed in binary64
    bool nesterov;
    const float *grad_scale;
    float ca, cb, cc;      // this iteration's coefficients
    int stage, swap;       // swap: X is in y
    __device__ __forceinline__ int find(int kind, int unit) const
    {
        int lo = 0, hi = count;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[kind][mid] <= unit) lo = mid;
            else hi = mid;
        }
        return lo;
    }
};

// ---------------------------------------------------------------- norm and momentum
__host__ __device__ __forceinline__ int sum_blocks(int64_t size)
{
    const int64_t n = (size + 16383) / 16384;
    return (int)(n < kSumBlocks ? n : kSumBlocks);
}
__device__ __forceinline__ float update_of(float g, float m, float beta, float fresh, bool nesterov)
{
    return nesterov ? fresh * g + beta * m : m;
}

// Four consecutive elements, aligned to their size.
__device__ __forceinline__ void load4(float *v, const void *p, int64_t i, int dtype)
{
    if (dtype == RR_FP32) {
        const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p) + i);
        const uint32_t w[2] = {x.x, x.y};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 f = dtype == RR_BF16 ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[k]))
                                              : __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            v[2 * k] = f.x;
            v[2 * k + 1] = f.y;
        }
    }
}
__device__ __forceinline__ bool aligned4(const void *p, int dtype)
{
    return (reinterpret_cast<uintptr_t>(p) & (dtype == RR_FP32 ? 15 : 7)) == 0;
}

// A step whose gradient scale is NaN is skipped: every kernel of it leaves at once,
// and reads and writes nothing else.
//
// The new momentum, and the sum of squares of what is orthogonalised.  Eight
// squares are added in binary32; such a sum outside [2^-90, 2^90] (zero aside) is
// taken again in binary64, and so is the sum of the sums.  Bound: HBM.
template <int CAP>
__global__ void __launch_bounds__(kThreads) sums_kernel(const __grid_constant__ Args<CAP> a)
{
    stream_order();
    __shared__ double s[kThreads / 32];
    const int i = a.find(kSums, blockIdx.x);
    const Item &it = a.item[i];
    const int b = blockIdx.x - a.start[kSums][i], blocks = sum_blocks(it.size);
    const int64_t lo = it.size * b / blocks & ~(int64_t)7, hi = b + 1 == blocks ? it.size : it.size * (b + 1) / blocks & ~(int64_t)7;
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const bool step = it.momentum != nullptr;
    if (step && isnan(gs)) return;
    const bool vec = aligned4(it.src, a.src_dtype) && aligned4(it.momentum, RR_FP32);
    double sum = 0.0;
    for (int64_t e = lo + (vec ? 4 * threadIdx.x : threadIdx.x); e < hi; e += 8 * kThreads) {
        float v[8], m[8];
        float part = 0.0f;
        const bool whole = vec && e + 4 * kThreads + 4 <= hi;
        auto at = [&](int j) { return e + (vec ? (j & 3) + (j >> 2) * 4 * kThreads : (int64_t)j * kThreads); };
        if (whole) {
            load4(v, it.src, e, a.src_dtype);
            load4(v + 4, it.src, e + 4 * kThreads, a.src_dtype);
            if (step) {
                load4(m, it.momentum, e, RR_FP32);
                load4(m + 4, it.momentum, e + 4 * kThreads, RR_FP32);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = at(j) < hi ? load_any(it.src, at(j), a.src_dtype) : 0.0f;
                m[j] = step && at(j) < hi ? it.momentum[at(j)] : 0.0f;
            }
        }
        if (step) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float g = v[j] * gs;
                m[j] = a.momentum * m[j] + a.fresh * g;
                v[j] = update_of(g, m[j], a.momentum, a.fresh, a.nesterov);
            }
            if (whole) {
                *reinterpret_cast<float4 *>(it.momentum + e) = make_float4(m[0], m[1], m[2], m[3]);
                *reinterpret_cast<float4 *>(it.momentum + e + 4 * kThreads) = make_float4(m[4], m[5], m[6], m[7]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (at(j) < hi) it.momentum[at(j)] = m[j];
            }
        }
        bool zero = true;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            part = fmaf(v[j], v[j], part);
            zero = zero && v[j] == 0.0f;
        }
        if (zero || (part >= 0x1p-90f && part <= 0x1p90f)) {
            sum += (double)part;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += (double)v[j] * (double)v[j];
        }
    }
    sum = block_sum64<kThreads / 32>(sum, s);
    if (threadIdx.x == 0) it.part[b] = sum;
}

// ---------------------------------------------------------------- operands
__device__ __forceinline__ uint32_t halves(float2 v)
{
    const __half2 h = __float22half2_rn(v);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 floats(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }
// Eight scaled values as two pieces of 16 bytes.
__device__ __forceinline__ void split8(const float2 (&v)[4], uint4 &hi, uint4 &lo)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        h[k] = halves(v[k]);
        const float2 f = floats(h[k]);
        l[k] = halves(add2(v[k], make_float2(-f.x, -f.y)));
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// Where columns [8 c, 8 c + 8) of row r of a block's piece lie.
__device__ __forceinline__ int chunk_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// X = update / (norm + eps) as pieces, a block of 128 x 64 at a time.  Bound: HBM.
template <int CAP>
__global__ void __launch_bounds__(kThreads) split_kernel(const __grid_constant__ Args<CAP> a)
{
    stream_order();
    __shared__ float tile[kK][kTile + 1];  // of a matrix whose transpose is X
    __shared__ double s[kThreads / 32];
    const int i = a.find(kSplit, blockIdx.x);
    const Item &it = a.item[i];
    const int u = blockIdx.x - a.start[kSplit][i], nb = it.nt * 2;
    const int r0 = u / nb * kTile, c0 = u % nb * kK;
    const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
    const bool step = it.momentum != nullptr;
    if (step && isnan(gs)) return;
    const int blocks = sum_blocks(it.size);
    double total = 0.0;
    for (int k = threadIdx.x; k < blocks; k += kThreads) total += it.part[k];
    total = block_sum64<kThreads / 32>(total, s);
    const double divisor = sqrt(total) + a.eps;
    const float by = (float)divisor;
    const bool plain = by >= 0x1p-100f && by <= 0x1p100f;
    auto scaled = [&](float g, float m) {
        const float v = step ? update_of(g * gs, m, a.momentum, a.fresh, a.nesterov) : g;
        return (plain ? v / by : (float)((double)v / divisor)) * kScale;
    };
    char *block = it.x + (int64_t)u * kBlock;
    const bool vec = it.n % 8 == 0 && !it.tall && aligned4(it.src, a.src_dtype) && aligned4(it.momentum, RR_FP32);
    if (it.tall) {  // neighbouring threads along the matrix's own rows
        for (int k0 = threadIdx.x; k0 < kTile * kK; k0 += 8 * kThreads) {
            float v[8], m[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = k0 + j * kThreads, r = k % kTile, c = k / kTile;
                const bool in = r0 + r < it.m && c0 + c < it.n;
                const int64_t at = (int64_t)(c0 + c) * it.m + r0 + r;
                v[j] = in ? load_any(it.src, at, a.src_dtype) : 0.0f;
                m[j] = in && step ? it.momentum[at] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = k0 + j * kThreads, r = k % kTile, c = k / kTile;
                tile[c][r] = r0 + r < it.m && c0 + c < it.n ? scaled(v[j], m[j]) : 0.0f;
            }
        }
        __syncthreads();
    }
#pragma unroll 2
    for (int k = threadIdx.x; k < kTile * 8; k += kThreads) {
        const int r = k >> 3, c = k & 7, col = c0 + 8 * c;
        float v[8];
        if (it.tall) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = tile[8 * c + e][r];
        } else {
            const bool row = r0 + r < it.m;
            const int64_t at = (int64_t)(r0 + r) * it.n + col;
            float m[8];
            if (vec && row && col < it.n) {
                load4(v, it.src, at, a.src_dtype);
                load4(v + 4, it.src, at + 4, a.src_dtype);
                if (step) {
                    load4(m, it.momentum, at, RR_FP32);
                    load4(m + 4, it.momentum, at + 4, RR_FP32);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const bool in = row && col + e < it.n;
                    v[e] = in ? load_any(it.src, at + e, a.src_dtype) : 0.0f;
                    m[e] = in && step ? it.momentum[at + e] : 0.0f;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = row && col + e < it.n ? scaled(v[e], m[e]) : 0.0f;
        }
        uint4 hi, lo;
        split8({make_float2(v[0], v[1]), make_float2(v[2], v[3]), make_float2(v[4], v[5]), make_float2(v[6], v[7])}, hi, lo);
        *reinterpret_cast<uint4 *>(block + chunk_at(r, c)) = hi;
        *reinterpret_cast<uint4 *>(block + kPiece + chunk_at(r, c)) = lo;
    }
    asm volatile("fence.proxy.async.global;" ::: "memory");  // the products fetch it by bulk copies
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ uint32_t smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// Arrive at the barrier of the pair's first block.  Nothing but accumulators and
// bulk copies is ordered by it, so it takes no wider scope (a release to the
// cluster waits for the thread's stores: with it a layer's attention weights took 5.8
// ms where they took 4.7 without).
__device__ __forceinline__ void mbar_arrive_first(uint32_t bar)
{
    asm volatile("{\n\t.reg .b32 first;\n\tmapa.shared::cluster.u32 first, %0, 0;\n\t"
                 "mbarrier.arrive.shared::cluster.b64 _, [first];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, int bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, int parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Waits end after two seconds: the block then stops, and its tiles become NaN.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, int parity, volatile int *dead)
{
    if (mbar_test(bar, parity)) return true;
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
    for (uint32_t spins = 1; !mbar_test(bar, parity); ++spins) {
        if ((spins & 63u) == 0) {
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
            if (*dead || t - t0 > 2000000000ull) {
                *dead = 1;
                return false;
            }
        }
    }
    return true;
}
__device__ __forceinline__ void bulk_load(uint32_t to, const void *from, int bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
                 "l"(from), "r"(bytes), "r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// An operand in shared memory, 128-byte swizzle.  Rows of K values: groups of 8
// rows lie 1024 bytes apart.  Columns (K rows of 64 values): groups of 8 K rows
// lie 1024 bytes apart, the next 64 columns 8192.
__device__ __forceinline__ uint64_t operand(uint32_t at, bool columns)
{
    const uint64_t leading = columns ? 8192 >> 4 : 1, stride = 1024 >> 4;
    return (uint64_t)((at & 0x3FFFF) >> 4) | leading << 16 | stride << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
// fp16 operands, each by rows or by columns, binary32 accumulators, 256 x N over
// two blocks.
template <int N>
__device__ __forceinline__ uint32_t instruction(bool left_columns, bool right_columns)
{
    return 1u << 4 | (left_columns ? 1u << 15 : 0u) | (right_columns ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 |
           (uint32_t)(2 * kTile >> 4) << 24;
}
__device__ __forceinline__ void mma(uint32_t acc, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(acc), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
// Arrives at both blocks' barriers when the products issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3) : "memory");
}
// 16 columns of this warp's 32 rows.
__device__ __forceinline__ void tmem_load(float (&v)[16], uint32_t at)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at) : "memory");
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
}

// A pair's tile of a product: which matrix, which 256 rows and N columns, how deep.
struct Job {
    const Item *it;
    int ti, tj, depth;
};
template <int N, int CAP>
__device__ __forceinline__ Job job_of(const Args<CAP> &a, int unit)
{
    const bool next = a.stage >= kStageNext;
    const int kind = Shape<N>::units(next), i = a.find(kind, unit);
    const Item &it = a.item[i];
    const int u = unit - a.start[kind][i], tiles = (it.mt + 1) / 2;
    Job j;
    j.it = &it;
    if (next) {
        j.ti = u % tiles;
        j.tj = u / tiles;
    } else {  // a symmetric product's squares of 256 on and below the diagonal, N columns at a time
        constexpr int per = 256 / N;
        const int t = u / per;
        j.ti = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
        while (j.ti * (j.ti + 1) / 2 > t) --j.ti;
        while ((j.ti + 1) * (j.ti + 2) / 2 <= t) ++j.ti;
        j.tj = (t - j.ti * (j.ti + 1) / 2) * per + u % per;
    }
    j.depth = ((a.stage == kStageGram ? it.n : it.m) + kK - 1) / kK;
    return j;
}

// ---------------------------------------------------------------- a tile's results
// A warp holds 32 rows of a tile, a row to a lane.  Lines of memory hold a row's 64
// values of a piece, so lanes that went to memory each for itself would touch 32
// lines at a time (17 to 25 thousand cycles a tile, and 100 thousand for row-major
// results).  Values pass through the warp's desk instead, 32 x 32 at a time: value of
// row r, column c at r * 32 + (c ^ r), free of conflicts along both.  What is left is
// the rate at which an SM stores, some 32 bytes a cycle: 4 to 5 thousand cycles for the
// 128 KB of a tile of 256 columns, against 86 thousand of products at a depth of 3584.

// 32 x 32 results to row-major memory, neighbouring lanes along its rows.
template <class T>
__device__ __forceinline__ void store_result(const Item &it, float keep, int row0, int col0, const float *desk, int lane)
{
    // the matrix's own rows and columns
    const int64_t wide = it.tall ? it.m : it.n, first = it.tall ? col0 : row0, along = (it.tall ? row0 : col0) + lane;
    const int most = along < wide ? (int)min((int64_t)32, (it.tall ? it.n : it.m) - first) : 0;
    // row k of the desk, this lane's column, or the other way round
    const int base = it.tall ? lane * 32 : 0, by = it.tall ? 0 : 32;
    T *out = static_cast<T *>(it.out) + first * wide + along;
    if (!it.momentum) {
#pragma unroll 4
        for (int k = 0; k < most; ++k, out += wide) *out = from_f32<T>(desk[base + k * by + (k ^ lane)] * (kUnscale * kUnscale));
        return;
    }
    float *master = it.master ? it.master + first * wide + along : nullptr;
    const float step = it.scale * (kUnscale * kUnscale);
#pragma unroll 1
    for (int k0 = 0; k0 < most; k0 += 8) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k0 + i < most) w[i] = master ? master[i * wide] : to_f32(out[i * wide]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k0 + i < most) {
                w[i] = keep * w[i] - step * desk[base + (k0 + i) * by + ((k0 + i) ^ lane)];
                if (master) master[i * wide] = w[i];
                out[i * wide] = from_f32<T>(w[i]);
            }
        out += 8 * wide;
        if (master) master += 8 * wide;
    }
}

// 32 x 32 sums to a block, as pieces; of a square, c * sum + b * A + a * I.
// Four lanes have 64 bytes of a row.
template <int CAP>
__device__ __forceinline__ void store_pieces(const Args<CAP> &a, const Item &it, char *to, int64_t at, int chunk0, int diagonal,
                                             const float *desk, int lane)
{
    const bool square = a.stage == kStageSquare;
    const float2 by = both(square ? a.cc * kUnscale : kUnscale), cb = both(a.cb);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2), c = (lane & 3) * 8;
        const int64_t e = at + chunk_at(r, chunk0 + (lane & 3));  // rows begin at a multiple of 8
        uint4 hi, lo;
        if (square) {
            hi = *reinterpret_cast<const uint4 *>(it.a + e);
            lo = *reinterpret_cast<const uint4 *>(it.a + e + kPiece);
        }
        const float *row = desk + r * 32;
        float2 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(make_float2(row[(c + 2 * k) ^ r], row[(c + 2 * k + 1) ^ r]), by);
        if (square) {
            const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = fma2(add2(floats(h[k]), floats(l[k])), cb, v[k]);
            if (diagonal == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (r == c + 2 * k) v[k].x += a.ca * kScale;
                    if (r == c + 2 * k + 1) v[k].y += a.ca * kScale;
                }
            }
        }
        split8(v, hi, lo);
        *reinterpret_cast<uint4 *>(to + e) = hi;
        *reinterpret_cast<uint4 *>(to + e + kPiece) = lo;
    }
}

// Sums of 32 rows (from row0 on) and M columns (from block column cb0 on) of a
// product to where the stage puts them.
template <int M, int CAP>
__device__ __forceinline__ void finish(const Args<CAP> &a, const Item &it, float (&v)[M], int row0, int cb0, int wide, float *desk,
                                       int lane)
{
    if (a.stage == kStageLast && row0 >= it.m) return;
    char *to = a.stage == kStageGram ? it.a : a.stage == kStageSquare ? it.b : a.swap ? it.x : it.y;
    const int64_t block0 = ((int64_t)(row0 / kTile) * wide * 2 + cb0) * kBlock + row0 % kTile * 128;
#pragma unroll 1
    for (int g = 0; g < M / 32; ++g) {
        if (cb0 + g / 2 >= wide * 2) break;
        __syncwarp();
#pragma unroll
        for (int h = 0; h < M / 32; ++h)
            if (g == h) {
#pragma unroll
                for (int k = 0; k < 32; ++k) desk[lane * 32 + (k ^ lane)] = v[32 * h + k];
            }
        __syncwarp();
        const int col0 = cb0 * kK + 32 * g;
        if (a.stage != kStageLast)
            store_pieces(a, it, to, block0 + g / 2 * kBlock, g % 2 * 4, col0 - row0, desk, lane);
        else if (a.out_dtype == RR_FP32)
            store_result<float>(it, a.keep, row0, col0, desk, lane);
        else if (a.out_dtype == RR_BF16)
            store_result<__nv_bfloat16>(it, a.keep, row0, col0, desk, lane);
        else
            store_result<__half>(it, a.keep, row0, col0, desk, lane);
    }
}

// Of a symmetric matrix the squares of 256 on and below the diagonal are stored.  The
// rows of such a square `band`, columns of K block k, that lie above are the transpose
// of some below: they are fetched by columns.
__device__ __forceinline__ bool above(int band, int k) { return band < k / 4; }
// Both pieces of R rows (64 or 128, the `at`th such) and a K block, from a blocked
// matrix `wide` tiles across.
template <int R>
__device__ __forceinline__ void fetch_rows(uint32_t to, const char *m, int wide, int at, int k, uint32_t bar)
{
    constexpr int per = kTile / R;
    const char *from = m + ((int64_t)(at / per) * wide * 2 + k) * kBlock + at % per * (R * 128);
    if (R == kTile) {
        bulk_load(to, from, kBlock, bar);
    } else {
        bulk_load(to, from, R * 128, bar);
        bulk_load(to + R * 128, from + kPiece, R * 128, bar);
    }
}
// The same of its transpose: 64 of a block's rows are the depth, and R columns are
// one block or two side by side; each piece apart.
template <int R>
__device__ __forceinline__ void fetch_columns(uint32_t to, const char *m, int wide, int at, int k, uint32_t bar)
{
    constexpr int cbs = R / kK;
    const char *from = m + ((int64_t)(k >> 1) * wide * 2 + at * cbs) * kBlock + (k & 1) * (kPiece / 2);
#pragma unroll
    for (int q = 0; q < 2 * cbs; ++q)
        bulk_load(to + q * (kPiece / 2), from + q % cbs * kBlock + q / cbs * kPiece, kPiece / 2, bar);
}

// Bound: the tensor cores.  Both sides of a feed-forward product (3584 x 18944): X X'
// 0.82 ms, 1.90 PFLOP/s of binary16 products (of 2.01 measured for cuBLAS in bf16); the
// square 0.17; B X 1.54 ms, 1.89 PFLOP/s: launches by themselves, at 2.07 GHz.  Five steps
// take 13.5 ms so, and 15.0 call after call, at the 1.6 GHz that the power limit leaves
// (1.63 PFLOP/s, cuBLAS 1.77).  Sums in registers run beside the products
// (three stages of 64 KB come from the L2 at 43 bytes a cycle); results do not, see above.
//
// Two blocks of a cluster work on a tile of 256 x N, each on 128 rows of it.
// Each has its rows of the first operand and half the second one's columns in
// shared memory; the first block's thread issues the products of both.
template <int N, int CAP>
__global__ void __cluster_dims__(2) __launch_bounds__(kGemmThreads, 1) product_kernel(const __grid_constant__ Args<CAP> a)
{
    using S = Shape<N>;
    extern __shared__ char raw[];
    char *base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const uint32_t smem = smem_u32(base), bars = smem + S::barriers;
    uint32_t *tmem_base = reinterpret_cast<uint32_t *>(base + S::barriers + 192);
    volatile int *dead = reinterpret_cast<volatile int *>(base + S::barriers + 196);
    // full: a stage's copies are here, in the first block the second one's too; empty:
    // the products have read it; done, free: an accumulator's products are complete,
    // have been added up
    const uint32_t full = bars, empty = full + 8 * S::stages, done = empty + 8 * S::stages, free = done + 16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::stages; ++s) {
            mbar_init(full + 8 * s, rank == 0 ? 2 : 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(done + 8 * s, 1);
            mbar_init(free + 8 * s, 2 * kSumWarps);
        }
        *dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    cluster_sync();
    if (blockIdx.x / 2 < a.start[S::units(a.stage >= kStageNext)][a.count]) {
        // the table of matrices comes to the SM while the stage before runs
        const Job j = job_of<N>(a, blockIdx.x / 2);
        asm volatile("" ::"l"(j.it->x), "l"(j.it->b), "l"(j.it->out), "r"(j.ti + j.tj + j.depth));
    }
    stream_order();
    // Only now: accumulators held while waiting could be what a kernel before waits for.
    // (The first block's products wait for the second's copies, whose arrival the warp
    // that has made room there passes on.)
    if (warp == kSumWarps + 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bars + 192), "n"(2 * N) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    fence_tmem_before();
    __syncthreads();
    fence_tmem_after();
    const uint32_t tmem = *tmem_base;
    const bool next = a.stage >= kStageNext;
    const int units = a.start[S::units(next)][a.count], first_unit = blockIdx.x / 2, every = gridDim.x / 2;

    // (Read here: on its way while the accumulators are made it cost every launch 0.1 us.)
    if (a.grad_scale && isnan(*a.grad_scale)) {
        // a step that is skipped
    } else if (warp < kSumWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegisters));
        const int half = warp >> 2;  // of the tile's columns
        float *desk = reinterpret_cast<float *>(base + S::desks + warp * kDesk);
        const uint32_t mine = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * S::half;
        Turn<2> acc(0);
        bool ok = true;
        for (int unit = first_unit; unit < units; unit += every) {
            float v[S::half];
#pragma unroll
            for (int k = 0; k < S::half; ++k) v[k] = 0.0f;
            ok = take_turns(
                ok, acc, job_of<N>(a, unit).depth,
                [&](const Turn<2> &t) { return mbar_wait(done + 8 * t.at, t.phase, dead); },
                [&](const Turn<2> &t) {
                    fence_tmem_after();
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < S::half / 16; ++q) {
                        float x[16];
                        tmem_load(x, mine + t.at * N + q * 16);
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[q * 16 + e] += x[e];
                    }
                    fence_tmem_before();
                    __syncwarp();
                },
                [&](const Turn<2> &t) {  // by lane 0 for the warp
                    if (lane == 0) mbar_arrive_first(free + 8 * t.at);
                });
            if (!ok) {
#pragma unroll
                for (int k = 0; k < S::half; ++k) v[k] = __int_as_float(0x7fc00000);
            }
            const Job j = job_of<N>(a, unit);
            const Item &it = *j.it;
            const int rt = j.ti * 2 + (int)rank, cb = (j.tj * 2 + half) * (S::half / kK), wide = next ? it.nt : it.mt;
            if (rt < it.mt && cb < wide * 2) finish(a, it, v, rt * kTile + (warp & 3) * 32, cb, wide, desk, lane);
        }
        asm volatile("fence.proxy.async.global;" ::: "memory");  // the next product fetches it by bulk copies
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegisters));
        if (warp == kSumWarps && lane == 0) {
            asm volatile("fence.proxy.async.global;" ::: "memory");
            Turn<S::stages> turn(1);
            bool ok = true;
            for (int unit = first_unit; unit < units && ok; unit += every) {
                const Job j = job_of<N>(a, unit);
                const Item &it = *j.it;
                const char *x = a.swap ? it.y : it.x, *sq = a.stage == kStageSquare ? it.a : it.b;
                // the last tile may have one half: the other one's place takes what is at hand
                const int rows = min(j.ti * 2 + (int)rank, it.mt - 1);
                // columns of the right operand by S::half
                const int cols = min(j.tj * 2 + (int)rank, (next ? it.nt : it.mt) * (kTile / S::half) - 1);
                for (int k = 0; k < j.depth; ++k, turn.next()) {
                    ok = mbar_wait(empty + 8 * turn.at, turn.phase, dead);
                    if (!ok) break;
                    const uint32_t left = smem + turn.at * S::stage, right = left + kBlock, bar = full + 8 * turn.at;
                    mbar_expect(bar, S::stage);
                    if (a.stage == kStageGram) fetch_rows<kTile>(left, x, it.nt, rows, k, bar);
                    else if (above(j.ti, k)) fetch_columns<kTile>(left, sq, it.mt, rows, k, bar);
                    else fetch_rows<kTile>(left, sq, it.mt, rows, k, bar);
                    if (a.stage == kStageGram) fetch_rows<S::half>(right, x, it.nt, cols, k, bar);
                    else if (next) fetch_columns<S::half>(right, x, it.nt, cols, k, bar);
                    else if (above(j.tj * N / 256, k)) fetch_columns<S::half>(right, sq, it.mt, cols, k, bar);
                    else fetch_rows<S::half>(right, sq, it.mt, cols, k, bar);
                }
            }
            // a block waits for its copies before its shared memory goes, whichever thread gave up
            for (int s = 0; s < S::stages; ++s, turn.next()) {
                volatile int late = 0;
                mbar_wait(full + 8 * turn.at, turn.phase, &late);
            }
        } else if (warp == kSumWarps + 1 && lane == 0 && rank == 1) {
            // tells the first block what has come here
            Turn<S::stages> turn(0);
            bool ok = true;
            for (int unit = first_unit; unit < units && ok; unit += every) {
                const Job j = job_of<N>(a, unit);
                for (int k = 0; k < j.depth && ok; ++k, turn.next()) {
                    ok = mbar_wait(full + 8 * turn.at, turn.phase, dead);
                    if (ok) mbar_arrive_first(full + 8 * turn.at);
                }
            }
        } else if (warp == kSumWarps + 1 && lane == 0) {
            Turn<S::stages> turn(0);
            Turn<2> acc(1);
            bool ok = true;
            for (int unit = first_unit; unit < units && ok; unit += every) {
                const Job j = job_of<N>(a, unit);
                for (int k = 0; k < j.depth; ++k, turn.next(), acc.next()) {
                    const bool lc = a.stage != kStageGram && above(j.ti, k);
                    const bool rc = next || (a.stage == kStageSquare && above(j.tj * N / 256, k));
                    const uint32_t left = smem + turn.at * S::stage, right = left + kBlock, sums = tmem + acc.at * N;
                    const uint32_t idesc = instruction<N>(lc, rc);
                    const uint64_t lh = operand(left, lc), ll = operand(left + kPiece, lc), rh = operand(right, rc),
                                   rl = operand(right + S::right / 2, rc);
                    const int lstep = (lc ? 2048 : 32) >> 4, rstep = (rc ? 2048 : 32) >> 4;  // 16 values on
                    ok = mbar_wait(free + 8 * acc.at, acc.phase, dead) && mbar_wait(full + 8 * turn.at, turn.phase, dead);
                    if (!ok) break;
                    fence_tmem_after();
#pragma unroll
                    for (int q = 0; q < kK / 16; ++q) {
                        mma(sums, lh + q * lstep, rl + q * rstep, idesc, q > 0);
                        mma(sums, ll + q * lstep, rh + q * rstep, idesc, true);
                    }
#pragma unroll
                    for (int q = 0; q < kK / 16; ++q) mma(sums, lh + q * lstep, rh + q * rstep, idesc, true);
                    mma_commit(empty + 8 * turn.at);
                    mma_commit(done + 8 * acc.at);
                }
            }
            // what is in flight reads shared memory: the last stages' releases show its end
            for (int s = 0; s < S::stages; ++s, turn.next()) {
                volatile int late = 0;
                mbar_wait(empty + 8 * turn.at, turn.phase ^ 1, &late);
            }
        }
    }
    __syncwarp();
    fence_tmem_before();
    __syncthreads();
    cluster_sync();  // neither block's shared memory or barriers go before the other is done
    if (warp == kSumWarps + 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(2 * N) : "memory");
}

// ---------------------------------------------------------------- host side
struct Sizes {
    int m, n, mt, nt;
    int64_t x, sq, part;  // bytes of X, of a square, of the partial sums
    int64_t all() const { return 2 * x + 2 * sq + part; }
};
Sizes sizes_of(int64_t rows, int64_t cols)
{
    Sizes s;
    s.m = (int)std::min(rows, cols);
    s.n = (int)std::max(rows, cols);
    s.mt = (s.m + kTile - 1) / kTile;
    s.nt = (s.n + kTile - 1) / kTile;
    s.x = (int64_t)s.mt * s.nt * 2 * kBlock;
    s.sq = (int64_t)s.mt * s.mt * 2 * kBlock;
    s.part = kSumBlocks * 8;
    return s;
}

// A matrix's units of work in each kind of launch.
struct Units {
    int64_t of[kKinds];
};
Units units_of(const Sizes &s)
{
    const int64_t mp = (s.mt + 1) / 2, np = (s.nt + 1) / 2;  // pairs' tiles
    return {{sum_blocks((int64_t)s.m * s.n), (int64_t)s.mt * s.nt * 2, mp * (mp + 1) / 2, mp * np, mp * (mp + 1), mp * s.nt}};
}

rr_status check_shapes(const int64_t *rows, const int64_t *cols, int count)
{
    if (count < 0) return step_fail(RR_ERR_INVALID_ARG, "num_tensors %d", count);
    if (count > 0 && (!rows || !cols)) return step_fail(RR_ERR_INVALID_ARG, "%s is NULL", rows ? "cols" : "rows");
    for (int i = 0; i < count; ++i) {
        if (rows[i] < 0 || rows[i] > kMaxSide) return step_fail(RR_ERR_INVALID_ARG, "rows[%d] is %lld", i, (long long)rows[i]);
        if (cols[i] < 0 || cols[i] > kMaxSide) return step_fail(RR_ERR_INVALID_ARG, "cols[%d] is %lld", i, (long long)cols[i]);
    }
    return RR_OK;
}
// The list as run_lists works through it, kCap matrices at a time (empty ones aside):
// whether each table's launches can count their units; bytes: of the largest table's
// workspace, as the tables come one after the other.
rr_status check_list(const int64_t *rows, const int64_t *cols, int count, size_t *bytes)
{
    Units all = {};
    int64_t sum = 0, most = 0;
    for (int i = 0, k = 0; i < count; ++i) {
        if (rows[i] * cols[i] == 0) continue;
        if (k++ % kCap == 0) {
            all = {};
            sum = 0;
        }
        const Sizes s = sizes_of(rows[i], cols[i]);
        const Units units = units_of(s);
        bool fits = true;
        for (int q = 0; q < kKinds; ++q) fits = fits && (all.of[q] += units.of[q]) <= INT32_MAX;
        sum += s.all();  // of fewer than 2^31 blocks
        most = std::max(most, sum);
        if (!fits) return step_fail(RR_ERR_INVALID_ARG, "the list's matrices are too large for one call");
    }
    *bytes = (size_t)most;
    return RR_OK;
}
rr_status check_pointers(const char *name, const void *const *p, const int64_t *rows, const int64_t *cols, int count,
                         int bytes)
{
    if (count > 0 && !p) return step_fail(RR_ERR_INVALID_ARG, "%s is NULL", name);
    for (int i = 0; i < count; ++i) {
        if (rows[i] * cols[i] == 0) continue;
        if (!p[i]) return step_fail(RR_ERR_INVALID_ARG, "%s[%d] is NULL", name, i);
        if (!aligned_to(p[i], bytes))
            return step_fail(RR_ERR_ALIGNMENT, "%s[%d] not aligned to its %d-byte element", name, i, bytes);
    }
    return RR_OK;
}
rr_status check_iteration(const double *coefs, int steps, double eps)
{
    if (steps < 0 || steps > kMaxSteps) return step_fail(RR_ERR_INVALID_ARG, "steps %d", steps);
    if (steps == 0) return step_fail(RR_ERR_INVALID_ARG, "steps 0: there is nothing to iterate");
    if (!coefs) return step_fail(RR_ERR_INVALID_ARG, "coefs is NULL");
    for (int i = 0; i < 3 * steps; ++i)
        if (!(std::fabs(coefs[i]) <= 1e6)) return step_fail(RR_ERR_INVALID_ARG, "coefs[%d] is %g", i, coefs[i]);
    if (!(eps >= 0.0 && std::isfinite(eps))) return step_fail(RR_ERR_INVALID_ARG, "eps %g", eps);
    return RR_OK;
}
rr_status check_workspace(const int64_t *rows, const int64_t *cols, int count, const void *workspace, size_t bytes,
                          size_t *need)
{
    RR_TRY(rr_orthogonalize_workspace(rows, cols, count, need));
    if (*need == 0) return RR_OK;
    if (!workspace) return step_fail(RR_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned_to(workspace, 16)) return step_fail(RR_ERR_ALIGNMENT, "workspace not 16-byte aligned");
    if (bytes < *need) return step_fail(RR_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", bytes, *need);
    return RR_OK;
}

// What both entries hand over, checked.
struct Call {
    const void *const *src;
    void *const *out;
    float *const *momentum;  // NULL: no step
    float *const *master;
    const int64_t *rows, *cols;
    int count;
    rr_dtype src_dtype, out_dtype;
    const double *coefs;
    int steps;
    double eps;
    const rr_muon_hyper *hyper;
    const float *grad_scale;
    char *workspace;
};

// The products' kernel takes nearly all of an SM's shared memory, more than
// step_fit asks for; asked for once on each device.
template <int N, int CAP>
rr_status product_ready()
{
    static std::mutex mu;
    static std::vector<char> ready;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return step_cuda_fail(e, "cudaGetDevice");
    std::lock_guard<std::mutex> lock(mu);
    if ((int)ready.size() <= dev) ready.resize(dev + 1, 0);
    if (!ready[dev]) {
        e = cudaFuncSetAttribute((const void *)product_kernel<N, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<N>::smem);
        if (e != cudaSuccess) return step_cuda_fail(e, "cudaFuncSetAttribute(maxDynamicSharedMemorySize)");
        ready[dev] = 1;
    }
    return RR_OK;
}
template <int N, int CAP>
rr_status launch_product(Args<CAP> &a, int64_t units, int64_t pairs, cudaStream_t stream)
{
    return step_launch((const void *)product_kernel<N, CAP>, 2 * std::min(units, pairs), kGemmThreads, Shape<N>::smem, &a, stream);
}
// Whether tiles of 128 columns take less: a wave of them is 0.77 of a wave of 256
// (they read more for each product).  Five steps of square matrices, us at 256 and 128
// columns throughout: four of 512 260, 203; 1024 351, 283; 2048 586, 601 (518 as chosen
// here); 2560 888, 1189; 3584 2001, 2649; eight of 1024 x 4096 1703, 2074.
bool narrow_tiles(int64_t wide_units, int64_t narrow_units, int64_t pairs)
{
    return 77 * ((narrow_units + pairs - 1) / pairs) < 100 * ((wide_units + pairs - 1) / pairs);
}

template <int CAP>
rr_status run_lists(const Call &c, int sms, cudaStream_t stream)
{
    Args<CAP> a;
    a.src_dtype = (int)c.src_dtype;
    a.out_dtype = (int)c.out_dtype;
    a.eps = c.eps;
    a.momentum = c.hyper ? (float)c.hyper->momentum : 0.0f;
    a.fresh = c.hyper ? (float)(1.0 - c.hyper->momentum) : 0.0f;
    a.keep = c.hyper ? (float)(1.0 - c.hyper->lr * c.hyper->weight_decay) : 0.0f;
    a.nesterov = c.hyper && c.hyper->nesterov;
    a.grad_scale = c.grad_scale;
    a.stage = a.swap = 0;
    a.ca = a.cb = a.cc = 0.0f;
    RR_TRY((product_ready<256, CAP>()));
    RR_TRY((product_ready<128, CAP>()));
    const int64_t pairs = std::max(1, sms / 2);
    for (int i = 0; i < c.count;) {
        int k = 0;
        char *at = c.workspace;
        for (int q = 0; q < kKinds; ++q) a.start[q][0] = 0;
        for (; i < c.count && k < CAP; ++i) {
            if (c.rows[i] * c.cols[i] == 0) continue;
            const Sizes s = sizes_of(c.rows[i], c.cols[i]);
            Item &it = a.item[k];
            it.src = c.src[i];
            it.out = c.out[i];
            it.momentum = c.momentum ? c.momentum[i] : nullptr;
            it.master = c.master ? c.master[i] : nullptr;
            it.x = at;
            it.y = it.x + s.x;
            it.a = it.y + s.x;
            it.b = it.a + s.sq;
            it.part = reinterpret_cast<double *>(it.b + s.sq);
            at += s.all();
            it.size = c.rows[i] * c.cols[i];
            it.m = s.m;
            it.n = s.n;
            it.mt = s.mt;
            it.nt = s.nt;
            it.tall = c.rows[i] > c.cols[i];
            it.scale = 0.0f;
            if (c.hyper) {
                const double r = (double)c.rows[i], l = (double)c.cols[i];
                it.scale = (float)(c.hyper->lr * (c.hyper->adjust == RR_MUON_RMS ? 0.2 * std::sqrt(std::max(r, l))
                                                                                 : std::sqrt(std::max(1.0, r / l))));
            }
            const Units units = units_of(s);
            for (int q = 0; q < kKinds; ++q) a.start[q][k + 1] = (int)(a.start[q][k] + units.of[q]);  // see check_list
            ++k;
        }
        if (k == 0) break;
        a.count = k;
        RR_TRY(step_launch((const void *)sums_kernel<CAP>, a.start[kSums][k], kThreads, 0, &a, stream));
        RR_TRY(step_launch((const void *)split_kernel<CAP>, a.start[kSplit][k], kThreads, 0, &a, stream));
        for (int step = 0; step < c.steps; ++step) {
            a.ca = (float)c.coefs[3 * step];
            a.cb = (float)c.coefs[3 * step + 1];
            a.cc = (float)c.coefs[3 * step + 2];
            a.swap = step & 1;
            for (int q = 0; q < 3; ++q) {
                a.stage = q < 2 ? q : step + 1 < c.steps ? kStageNext : kStageLast;
                const int64_t wide = a.start[q < 2 ? kGram256 : kNext256][k], narrow = a.start[q < 2 ? kGram128 : kNext128][k];
                RR_TRY((narrow_tiles(wide, narrow, pairs) ? launch_product<128>(a, narrow, pairs, stream)
                                                          : launch_product<256>(a, wide, pairs, stream)));
            }
        }
    }
    return RR_OK;
}

rr_status run(const Call &c, cudaStream_t stream)
{
    int sms = 0;
    RR_TRY(step_sms(&sms));
    return c.count <= kCapSmall ? run_lists<kCapSmall>(c, sms, stream) : run_lists<kCap>(c, sms, stream);
}

template <class T>
const void *const *plain(T *const *p) { return reinterpret_cast<const void *const *>(p); }

}  // namespace

}  // namespace rr

using namespace rr;

extern "C" rr_status rr_orthogonalize_workspace(const int64_t *rows, const int64_t *cols, int num_tensors, size_t *bytes)
{
    if (!bytes) return step_fail(RR_ERR_INVALID_ARG, "bytes is NULL");
    RR_TRY(check_shapes(rows, cols, num_tensors));
    RR_TRY(check_list(rows, cols, num_tensors, bytes));
    return step_ok();
}

extern "C" rr_status rr_orthogonalize(const void *const *x, void *const *y, const int64_t *rows, const int64_t *cols,
                                      int num_tensors, rr_dtype x_dtype, rr_dtype y_dtype, const double *coefs, int steps,
                                      double eps, void *workspace, size_t workspace_bytes, cudaStream_t stream)
try {
    if (!float_bytes(x_dtype)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "x_dtype %d", (int)x_dtype);
    if (!float_bytes(y_dtype)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "y_dtype %d", (int)y_dtype);
    RR_TRY(check_shapes(rows, cols, num_tensors));
    RR_TRY(check_iteration(coefs, steps, eps));
    const int xb = float_bytes(x_dtype), yb = float_bytes(y_dtype);
    RR_TRY(check_pointers("x", x, rows, cols, num_tensors, xb));
    RR_TRY(check_pointers("y", plain(y), rows, cols, num_tensors, yb));
    size_t need = 0;
    RR_TRY(check_workspace(rows, cols, num_tensors, workspace, workspace_bytes, &need));
    static thread_local Spans spans;
    spans.all.clear();
    // y[i] == x[i] of one type works in place: the matrix has been read before the result is written
    for (int i = 0; i < num_tensors; ++i)
        if (!(x[i] == y[i] && x_dtype == y_dtype)) spans.add(x[i], rows[i] * cols[i] * xb, false);
    for (int i = 0; i < num_tensors; ++i) spans.add(y[i], rows[i] * cols[i] * yb, true);
    spans.add(workspace, (int64_t)need, true);
    if (spans.touch()) return step_fail(RR_ERR_ALIAS, "a result or the workspace overlaps another argument");
    if (need == 0) return step_ok();
    const Call c{x, y, nullptr, nullptr, rows, cols, num_tensors, x_dtype, y_dtype, coefs, steps, eps, nullptr, nullptr,
                 static_cast<char *>(workspace)};
    RR_TRY(run(c, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}

extern "C" rr_status rr_muon(void *const *params, const void *const *grads, float *const *momentum, float *const *master,
                             const int64_t *rows, const int64_t *cols, int num_tensors, rr_dtype param_dtype,
                             rr_dtype grad_dtype, const rr_muon_hyper *hyper, const double *coefs, int steps,
                             const float *grad_scale, void *workspace, size_t workspace_bytes, cudaStream_t stream)
try {
    if (!float_bytes(param_dtype)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "param_dtype %d", (int)param_dtype);
    if (!float_bytes(grad_dtype)) return step_fail(RR_ERR_UNSUPPORTED_DTYPE, "grad_dtype %d", (int)grad_dtype);
    RR_TRY(check_shapes(rows, cols, num_tensors));
    if (!hyper) return step_fail(RR_ERR_INVALID_ARG, "hyper is NULL");
    if (!(hyper->lr >= 0.0 && std::isfinite(hyper->lr))) return step_fail(RR_ERR_INVALID_ARG, "lr %g", hyper->lr);
    if (!(hyper->momentum >= 0.0 && hyper->momentum < 1.0)) return step_fail(RR_ERR_INVALID_ARG, "momentum %g", hyper->momentum);
    if (!(hyper->weight_decay >= 0.0 && std::isfinite(hyper->weight_decay)))
        return step_fail(RR_ERR_INVALID_ARG, "weight_decay %g", hyper->weight_decay);
    if (hyper->adjust != RR_MUON_SPECTRAL && hyper->adjust != RR_MUON_RMS)
        return step_fail(RR_ERR_INVALID_ARG, "adjust %d", hyper->adjust);
    RR_TRY(check_iteration(coefs, steps, hyper->eps));
    const int pb = float_bytes(param_dtype), gb = float_bytes(grad_dtype);
    RR_TRY(check_pointers("params", plain(params), rows, cols, num_tensors, pb));
    RR_TRY(check_pointers("grads", grads, rows, cols, num_tensors, gb));
    RR_TRY(check_pointers("momentum", plain(momentum), rows, cols, num_tensors, 4));
    if (master) RR_TRY(check_pointers("master", plain(master), rows, cols, num_tensors, 4));
    if (!aligned_to(grad_scale, 4)) return step_fail(RR_ERR_ALIGNMENT, "grad_scale not 4-byte aligned");
    size_t need = 0;
    RR_TRY(check_workspace(rows, cols, num_tensors, workspace, workspace_bytes, &need));
    static thread_local Spans spans;
    spans.all.clear();
    for (int i = 0; i < num_tensors; ++i) spans.add(params[i], rows[i] * cols[i] * pb, true);
    for (int i = 0; i < num_tensors; ++i) spans.add(grads[i], rows[i] * cols[i] * gb, false);
    for (int i = 0; i < num_tensors; ++i) spans.add(momentum[i], rows[i] * cols[i] * 4, true);
    for (int i = 0; master && i < num_tensors; ++i) spans.add(master[i], rows[i] * cols[i] * 4, true);
    spans.add(grad_scale, 4, false);
    spans.add(workspace, (int64_t)need, true);
    if (spans.touch()) return step_fail(RR_ERR_ALIAS, "a parameter, state, master weight or the workspace overlaps another argument");
    if (need == 0) return step_ok();
    const Call c{grads, params, momentum, master, rows, cols, num_tensors, grad_dtype, param_dtype, coefs, steps,
                 hyper->eps, hyper, grad_scale, static_cast<char *>(workspace)};
    RR_TRY(run(c, stream));
    return step_ok();
} catch (...) {
    return step_no_memory();
}
