// Compares rr_round.cuh with the device's rounded square root and division:
// square roots and reciprocals for every mantissa (both exponent parities, at
// several exponents), quotients for random
// operands with a normal quotient.  Prints the mismatches
// and exits 1 if a square root or a quotient differs.
#include <cstdio>

#include "rr_round.cuh"

namespace rr {

__device__ unsigned long long bad[3];

// Every float of the two binades from `bits` up.
__global__ void roots(unsigned bits)
{
    const unsigned i = blockIdx.x * blockDim.x + threadIdx.x;  // 2^23 threads, two values each
    const float2 v = make_float2(__uint_as_float(bits + i), __uint_as_float(bits + (1u << 23) + i));
    const float2 r = root2(v, make_float2(-v.x, -v.y));
    if (r.x != __fsqrt_rn(v.x)) atomicAdd(&bad[0], 1ull);
    if (r.y != __fsqrt_rn(v.y)) atomicAdd(&bad[0], 1ull);
}

__device__ bool normal(float x) { return fabsf(x) >= 0x1p-126f && fabsf(x) < 0x1p127f; }

__device__ unsigned draw(unsigned long long &s)
{
    s = s * 6364136223846793005ull + 1442695040888963407ull;
    return (unsigned)(s >> 32);
}

// Every mantissa as divisor, against `rounds` random dividends each.
__global__ void quotients(unsigned bits, int rounds, unsigned seed)
{
    const unsigned i = blockIdx.x * blockDim.x + threadIdx.x;
    unsigned long long s = ((unsigned long long)seed << 32) + i * 2654435761ull;
    const float d = __uint_as_float(bits + i);
    for (int k = 0; k < rounds; ++k) {
        const unsigned a = draw(s), b = draw(s);
        float2 m;  // signs, exponents in [-100, 100), mantissas
        m.x = __uint_as_float((a & 0x807FFFFFu) | (27u + (b >> 23 & 0xFFu) % 200u) << 23);
        m.y = k == 0 ? 1.0f : __uint_as_float((b & 0x807FFFFFu) | (27u + (a >> 23 & 0xFFu) % 200u) << 23);
        const float2 q = quotient2(m, make_float2(-d, -d)), want = make_float2(__fdiv_rn(m.x, d), __fdiv_rn(m.y, d));
        if (normal(want.x) && q.x != want.x) atomicAdd(&bad[1], 1ull);
        if (normal(want.y) && q.y != want.y) atomicAdd(&bad[k == 0 ? 2 : 1], 1ull);
    }
}

}  // namespace rr

int main()
{
    const int exponents[] = {27, 64, 126, 127, 190, 225};  // biased: 2^-100 ... 2^98
    for (int e : exponents) rr::roots<<<1 << 15, 256>>>((unsigned)e << 23);
    for (int e : exponents) rr::quotients<<<1 << 15, 256>>>((unsigned)e << 23, 64, (unsigned)e);
    unsigned long long bad[3];
    const cudaError_t e = cudaMemcpyFromSymbol(bad, rr::bad, sizeof bad);
    if (e != cudaSuccess) {
        std::printf("%s\n", cudaGetErrorString(e));
        return 2;
    }
    std::printf("square roots off: %llu, quotients off: %llu, reciprocals off: %llu\n", bad[0], bad[1], bad[2]);
    return bad[0] || bad[1] || bad[2] ? 1 : 0;
}
