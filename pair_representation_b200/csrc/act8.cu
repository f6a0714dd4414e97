// act8.cu - activations kept in 8 bits between the forward and the backward:
// bf16 to E4M3 codes with one E8M0 scale per 32 channels, and back
// (include/linear.h has the format).
//
// Both directions are one pass over the array, bound by memory: 2 + 33/32 bytes per
// value (589824 x 128, one call on inputs cold in L2: packing 45 us, unpacking 41, 5.1 and 5.6 TB/s; one after the
// other 79, where unpacking finds part of the codes in L2). The array is flat (channels are a
// multiple of 32, so blocks never cross a row): a thread takes 8 consecutive values, four
// threads a block, so that a warp's loads are 512 contiguous bytes of bf16 and 256 of codes,
// and kUnroll such pieces are in flight per thread. The block's largest value is an unsigned
// 16-bit maximum over the sign-cleared bf16 patterns (they order like their values), joined
// over the four threads by two shuffles; its exponent field gives the scale.
#include <cuda_fp8.h>

#include "kernels.h"
#include "linear_act.cuh"

namespace trimul {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

// The largest of two packed pairs of unsigned 16-bit values.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    asm("max.u16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return a;
}

// |w| with infinities and NaNs as 0.
__device__ __forceinline__ uint32_t finite_size(uint32_t w) {
    const uint32_t m = w & 0x7FFF7FFFu;
    return ((m & 0xFFFFu) >= 0x7F80u ? 0u : m & 0xFFFFu) | ((m >> 16) >= 0x7F80u ? 0u : m & 0xFFFF0000u);
}

__device__ __forceinline__ float element(uint32_t w, int hi) {
    const uint32_t bits = hi ? w & 0xFFFF0000u : w << 16;
    // An infinity would saturate to a finite code: keep it as NaN.
    return (bits & 0x7F800000u) == 0x7F800000u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(bits);
}

__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, float inv) {
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(element(w0, 0) * inv, element(w0, 1) * inv), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(element(w1, 0) * inv, element(w1, 1) * inv), __NV_SATFINITE, __NV_E4M3);
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

__global__ void __launch_bounds__(kThreads) act8_pack_kernel(const uint4 *__restrict__ x, uint2 *__restrict__ codes,
                                                             uint8_t *__restrict__ scales, long long pieces) {
    // pieces = 8-value pieces, a multiple of 4: the four threads of a block are always
    // all inside or all outside.
    const long long step = (long long)gridDim.x * kThreads * kUnroll;
    for (long long base = (long long)blockIdx.x * kThreads * kUnroll + threadIdx.x; base - threadIdx.x < pieces;
         base += step) {
        uint4 v[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long i = base + (long long)u * kThreads;
            v[u] = i < pieces ? x[i] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long i = base + (long long)u * kThreads;
            uint32_t m = max_u16x2(max_u16x2(v[u].x & 0x7FFF7FFFu, v[u].y & 0x7FFF7FFFu),
                                   max_u16x2(v[u].z & 0x7FFF7FFFu, v[u].w & 0x7FFF7FFFu));
            m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
            uint32_t top = max(m & 0xFFFFu, m >> 16);
            if (__any_sync(0xffffffffu, top >= 0x7F80u)) {  // an infinity or NaN: the largest finite value instead
                m = max_u16x2(max_u16x2(finite_size(v[u].x), finite_size(v[u].y)),
                              max_u16x2(finite_size(v[u].z), finite_size(v[u].w)));
                m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, 2));
                top = max(m & 0xFFFFu, m >> 16);
            }
            const int s = max((int)(top >> 7) - 8, 0);  // e + 127; 0 too for a block of zeros
            const float inv = __uint_as_float((uint32_t)(254 - s) << 23);  // 2^-e, exact
            if (i < pieces) {
                codes[i] = make_uint2(codes4(v[u].x, v[u].y, inv), codes4(v[u].z, v[u].w, inv));
                if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)s;
            }
        }
    }
}

__device__ __forceinline__ uint32_t value2(uint32_t code2, float size) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)code2, __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16x2(f.x * size, f.y * size);
}

__global__ void __launch_bounds__(kThreads) act8_unpack_kernel(const uint2 *__restrict__ codes,
                                                               const uint8_t *__restrict__ scales,
                                                               uint4 *__restrict__ x, long long pieces, bool more) {
    if (more) next_kernel_may_start();
    const long long step = (long long)gridDim.x * kThreads * kUnroll;
    for (long long base = (long long)blockIdx.x * kThreads * kUnroll + threadIdx.x; base < pieces; base += step) {
        uint2 c[kUnroll];
        uint32_t s[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long i = base + (long long)u * kThreads;
            c[u] = make_uint2(0u, 0u);
            s[u] = 0u;
            if (i < pieces) {
                c[u] = codes[i];
                s[u] = __ldg(scales + (i >> 2));
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const long long i = base + (long long)u * kThreads;
            const float size = e8m0_value(s[u]);
            if (i < pieces)
                x[i] = make_uint4(value2(c[u].x & 0xFFFFu, size), value2(c[u].x >> 16, size),
                                  value2(c[u].y & 0xFFFFu, size), value2(c[u].y >> 16, size));
        }
    }
}

// 32 blocks for each SM at most: five waves, whose ends overlap (8 a SM, one wave and a part, 86 us both ways
// at 589824 x 128; 32 80, without a limit 81). Loads and stores leave the caches as they are: evicting what
// streams past gained 1 us in the packing alone and cost 4 where the values are taken back soon (80 -> 76;
// call after call on the same array, as the figures before it).
int grid_for(long long pieces, int sms) {
    const long long need = (pieces + kThreads * kUnroll - 1) / (kThreads * kUnroll), most = (long long)sms * 32;
    return (int)(need < most ? need : most);
}

}  // namespace

cudaError_t launch_act8_pack(const void *x, void *codes, void *scales, long long values, int sms, cudaStream_t s) {
    act8_pack_kernel<<<grid_for(values / 8, sms), kThreads, 0, s>>>(
        static_cast<const uint4 *>(x), static_cast<uint2 *>(codes), static_cast<uint8_t *>(scales), values / 8);
    return cudaGetLastError();
}

cudaError_t launch_act8_unpack(const void *codes, const void *scales, void *x, long long values, int sms, bool more,
                               cudaStream_t s) {
    act8_unpack_kernel<<<grid_for(values / 8, sms), kThreads, 0, s>>>(
        static_cast<const uint2 *>(codes), static_cast<const uint8_t *>(scales), static_cast<uint4 *>(x), values / 8, more);
    return cudaGetLastError();
}

}  // namespace trimul
