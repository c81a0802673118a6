// Pieces shared by the gated delta rule's kernels: row addressing and gate values.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "delta.h"

namespace hla {
namespace delta {

using bf16 = __nv_bfloat16;

// Row index of token t of (b, head) among `heads` heads, in either layout.
__device__ __forceinline__ long long row_of(bool bthd, int b, int head, int heads, int t, int T) {
    return bthd ? (static_cast<long long>(b) * T + t) * heads + head
                : (static_cast<long long>(b) * heads + head) * T + t;
}
// Rows between two tokens of one head.
__device__ __forceinline__ int row_step(bool bthd, int heads) { return bthd ? heads : 1; }

__device__ __forceinline__ int length_of(const int* lengths, int b, int T) {
    if (!lengths) return T;
    const int n = lengths[b];
    return n < 0 ? 0 : (n > T ? T : n);
}

// A log decay below -120 counts as -120 (exp(-120) is 0 in fp32): differences of sums of decays
// then stay finite where a head starts anew.  NaN stays NaN.
__device__ __forceinline__ float gate(float g) { return g < -120.f ? -120.f : g; }

__device__ __forceinline__ void store_elem(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_elem(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// Four consecutive elements at p (16-byte aligned for fp32, 8-byte for bf16).
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(bf16* p, const float (&x)[4]) {
    __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    uint2 u;
    u.x = *reinterpret_cast<uint32_t*>(&a);
    u.y = *reinterpret_cast<uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&x)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xffff0000u);
}

}  // namespace delta
}  // namespace hla
