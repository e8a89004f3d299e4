// Shared by the training-step operators (rr_layer_norm.cu, rr_optim.cu):
// errors, launches, element loads and reductions.  Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cstring>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "rr.h"

namespace rr {

// ---------------------------------------------------------------- host side
// The calling thread's rr_last_error (rr_api.cu).
rr_status step_fail(rr_status s, const char *fmt, ...);
rr_status step_cuda_fail(cudaError_t e, const char *what);
rr_status step_ok();
// What a C entry returns for a C++ exception, which can only be host memory's.
inline rr_status step_no_memory() { return step_fail(RR_ERR_CUDA, "host memory ran out"); }

inline int float_bytes(rr_dtype d) { return d == RR_FP32 ? 4 : d == RR_BF16 || d == RR_FP16 ? 2 : 0; }
inline bool aligned_to(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

// SMs of the current device; blocks of a kernel that fit one of them.
rr_status step_sms(int *sms);
rr_status step_fit(const void *fn, int threads, int smem, int *blocks);

// One programmatic launch: the grid may start while the previous kernel in
// the stream drains; every kernel here begins with stream_order().
rr_status step_launch(const void *fn, int64_t grid, int threads, int smem, void *args, cudaStream_t stream);

#if defined(__CUDACC__)
// ---------------------------------------------------------------- device side
// Wait for the previous grid in the stream (its writes are visible after
// this), then let the next one be scheduled early.  Every thread of every
// kernel calls it before it touches memory or exits.
__device__ __forceinline__ void stream_order()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// One element of a float type known only at run time.
__device__ __forceinline__ float load_any(const void *p, int64_t i, int dtype)
{
    if (dtype == RR_FP32) return static_cast<const float *>(p)[i];
    if (dtype == RR_BF16) return to_f32(static_cast<const __nv_bfloat16 *>(p)[i]);
    return to_f32(static_cast<const __half *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int64_t i, int dtype, float x)
{
    if (dtype == RR_FP32) static_cast<float *>(p)[i] = x;
    else if (dtype == RR_BF16) static_cast<__nv_bfloat16 *>(p)[i] = from_f32<__nv_bfloat16>(x);
    else static_cast<__half *>(p)[i] = from_f32<__half>(x);
}

// N consecutive elements at an address aligned to their N * sizeof(T) bytes
// (4, 8 or 16 bytes at a time).
template <class T, int N>
struct alignas(N * sizeof(T) > 16 ? 16 : N * sizeof(T)) Pack {
    T v[N];
};

// Two binary32 operations in one instruction.  The assembler contracts a mul2
// whose result only an add2 takes into one fused operation, whatever its flags
// say; where the product's own rounding matters, see mul2_apart.
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
// A product rounded by itself: fused with an addend of -0 that the compiler
// cannot see (a kernel argument), it equals the product, and no later addition
// can be contracted with it.
__device__ __forceinline__ float2 mul2_apart(float2 a, float2 b, float2 minus_zero) { return fma2(a, b, minus_zero); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Two neighbouring elements between memory's type and binary32.
__device__ __forceinline__ float2 pair_f32(const float *p) { return make_float2(p[0], p[1]); }
__device__ __forceinline__ float2 pair_f32(const __half *p) { return __half22float2(*reinterpret_cast<const __half2 *>(p)); }
__device__ __forceinline__ float2 pair_f32(const __nv_bfloat16 *p)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
}
__device__ __forceinline__ void pair_set(float *p, float2 x)
{
    p[0] = x.x;
    p[1] = x.y;
}
__device__ __forceinline__ void pair_set(__half *p, float2 x) { *reinterpret_cast<__half2 *>(p) = __float22half2_rn(x); }
__device__ __forceinline__ void pair_set(__nv_bfloat16 *p, float2 x)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __float22bfloat162_rn(x);
}

// 16 bytes from global to shared memory, past the registers; groups complete
// in order.  A thread reads back only what it fetched, so nothing else waits.
__device__ __forceinline__ void fetch16(void *s, const void *g)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(s))),
                 "l"(g) : "memory");
}
__device__ __forceinline__ void fetch8(void *s, const void *g)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(s))),
                 "l"(g) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void fetch_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A sum that keeps what each addition rounds off (Knuth's two-sum), so that its
// own rounding does not grow with the number of parts.
struct Compensated {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = __fadd_rn(hi, x), z = __fsub_rn(t, hi);
        lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, z)), __fsub_rn(x, z));
        hi = t;
    }
    // Of a sum that is not finite nothing was rounded off.
    __device__ __forceinline__ float value() const { return fabsf(hi) < __int_as_float(0x7f800000) ? hi + lo : hi; }
};

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
#endif

}  // namespace rr
