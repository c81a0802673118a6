// Warp-level matrix pieces of the gated delta rule's chunk kernels.
//
// fp32 values enter the bf16 tensor-core products as a sum of bf16 terms, x = x1 + x2 (+ x3), each
// the rounding of what the earlier ones leave: 8 bits a term, so three terms hold an fp32 value
// to 2^-24 and two to 2^-16.  A product of an AT-term and a BT-term operand keeps the pairs (i, j)
// with i + j < max(AT, BT); what is left out is of the size of the last term's own rounding.
// bf16 inputs are one exact term.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "delta_common.cuh"
#include "ptx.cuh"

namespace hla {
namespace delta {

constexpr int C = 32;   // tokens of a chunk

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
    const int n = on ? 16 : 0;   // 0: sixteen zero bytes
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// c[n] += A B(n-tile n) for 2 NP tiles; b[np][t] = {tile 2 np k-low, k-high, tile 2 np + 1 k-low, k-high}.
// The tiles of one pair of terms follow one another, so a tile's own chain of sums does not stall
// them; the smallest products come first, since each sum is cut at the accumulator's last bit.
template <int AT, int BT, int NP>
__device__ __forceinline__ void prod(float (&c)[2 * NP][4], const uint32_t (&a)[AT][4], const uint32_t (&b)[NP][BT][4]) {
    constexpr int M = AT > BT ? AT : BT;
#pragma unroll
    for (int d = M - 1; d >= 0; --d)
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            const int j = d - i;
            if (j >= 0 && j < BT) {
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    mma16816(c[2 * p], a[i], b[p][j][0], b[p][j][1]);
                    mma16816(c[2 * p + 1], a[i], b[p][j][2], b[p][j][3]);
                }
            }
        }
}
template <int AT, int BT>
__device__ __forceinline__ void prod2(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[AT][4],
                                      const uint32_t (&b)[BT][4]) {
    constexpr int M = AT > BT ? AT : BT;
#pragma unroll
    for (int d = M - 1; d >= 0; --d)
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            const int j = d - i;
            if (j >= 0 && j < BT) {
                mma16816(c0, a[i], b[j][0], b[j][1]);
                mma16816(c1, a[i], b[j][2], b[j][3]);
            }
        }
}

// The same with the leading products and the small ones summed apart (add the two at the end): a long
// axis then cuts at the large sum's last bit once a step, not once a product.
template <int AT, int BT>
__device__ __forceinline__ void prod2(float (&h0)[4], float (&h1)[4], float (&l0)[4], float (&l1)[4],
                                      const uint32_t (&a)[AT][4], const uint32_t (&b)[BT][4]) {
    constexpr int M = AT > BT ? AT : BT;
#pragma unroll
    for (int d = M - 1; d > 0; --d)
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            const int j = d - i;
            if (j >= 0 && j < BT) {
                mma16816(l0, a[i], b[j][0], b[j][1]);
                mma16816(l1, a[i], b[j][2], b[j][3]);
            }
        }
    mma16816(h0, a[0], b[0][0], b[0][1]);
    mma16816(h1, a[0], b[0][2], b[0][3]);
}

// S = f S + W, rounded once: a carried state is not itself an accumulator of the products, which would
// cut it at its last bit once a product, always towards zero, so that a state that forgets slowly lost
// 1e-4 of itself in 512 chunks.
template <int NT>
__device__ __forceinline__ void decay_and_add(float (*S)[4], float f, const float (&W)[NT][4]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) S[n][j] = fmaf(S[n][j], f, W[n][j]);
}

// The bf16 terms of a pair, packed (x0 in the low half).
template <int N>
__device__ __forceinline__ void split(float x0, float x1, uint32_t (&t)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        t[i] = ptx::pack_bf16(x0, x1);
        if (i + 1 < N) {
            x0 -= __uint_as_float(t[i] << 16);
            x1 -= __uint_as_float(t[i] & 0xffff0000u);
        }
    }
}
// Two neighbouring 16 x 8 accumulator tiles as the A operand (16 x 16) of the next product: the
// accumulator layout of m16n8 is the A layout of m16k16 taken two tiles at a time.
template <int N>
__device__ __forceinline__ void split_a(const float (&lo)[4], const float (&hi)[4], uint32_t (&a)[N][4]) {
    uint32_t t[N];
    split<N>(lo[0], lo[1], t);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i][0] = t[i];
    split<N>(lo[2], lo[3], t);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i][1] = t[i];
    split<N>(hi[0], hi[1], t);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i][2] = t[i];
    split<N>(hi[2], hi[3], t);
#pragma unroll
    for (int i = 0; i < N; ++i) a[i][3] = t[i];
}

// A NaN or an infinity of one token must not reach the tokens before it, but 0 x NaN is NaN, and the
// triangular products multiply every token of a 16 x 16 block with the zeros above the diagonal.  Where a
// warp finds such a value in the tokens' axis of an operand (x: accumulator tiles, tile n's tokens
// 8 n + 2 (lane % 4) + (j & 1), columns lane / 4 + 8 (j >> 1)), it takes the product of the cleaned operand
// and makes NaN of the tokens from the first bad one on, column by column.
template <int N>
__device__ __forceinline__ bool any_bad(const float (&x)[N][4]) {       // of the warp's: 0 x is NaN then
    float s[4] = {};
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = fmaf(x[n][j], 0.f, s[j]);
    return __any_sync(0xffffffffu, (s[0] + s[1]) + (s[2] + s[3]) != 0.f);
}
__device__ __forceinline__ bool bad(float x) { return !(fabsf(x) <= 3.4028235e38f); }
template <int N>
__device__ __forceinline__ void first_bad(const float (&x)[N][4], int lane, int (&first)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int f = 8 * N;
#pragma unroll
        for (int n = N - 1; n >= 0; --n)
#pragma unroll
            for (int j = 1; j >= 0; --j)
                if (bad(x[n][2 * h + j])) f = 8 * n + 2 * (lane & 3) + j;
        f = min(f, __shfl_xor_sync(0xffffffffu, f, 1));
        first[h] = min(f, __shfl_xor_sync(0xffffffffu, f, 2));
    }
}
template <int N>
__device__ __forceinline__ void clean(float (&x)[N][4]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[n][j] = bad(x[n][j]) ? 0.f : x[n][j];
}
template <int N>
__device__ __forceinline__ void spoil(float (&x)[N][4], int lane, const int (&first)[2]) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (8 * n + 2 * (lane & 3) + (j & 1) >= first[j >> 1]) x[n][j] = __int_as_float(0x7fffffff);
}

// Byte offset of 16-byte piece c of row r in a bf16 tile with rows of RB bytes, swizzled so that
// eight rows of one piece (an ldmatrix) and eight pieces of one row fall on all banks.
template <int RB>
__device__ __forceinline__ uint32_t piece(int r, int c) {
    if constexpr (RB >= 128) return static_cast<uint32_t>(r * RB + ((c ^ (r & 7)) << 4));
    else if constexpr (RB == 64) return static_cast<uint32_t>(r * RB + ((c ^ ((r >> 1) & 3)) << 4));
    else return static_cast<uint32_t>(r * RB + ((c ^ ((r >> 2) & 1)) << 4));
}

// Addresses of the four 8 x 8 matrices of one ldmatrix.x4, for this lane.
// A operand, or B operand whose k axis is the rows (transposed load): rows r0.., pieces c0, c0+1.
template <int RB>
__device__ __forceinline__ uint32_t at_rows_first(uint32_t tile, int r0, int c0, int lane) {
    return tile + piece<RB>(r0 + ((lane >> 3) & 1) * 8 + (lane & 7), c0 + (lane >> 4));
}
// B operand whose n axis is the rows: rows r0.., pieces c0 (k low) and c0+1 (k high).
template <int RB>
__device__ __forceinline__ uint32_t at_pieces_first(uint32_t tile, int r0, int c0, int lane) {
    return tile + piece<RB>(r0 + (lane >> 4) * 8 + (lane & 7), c0 + ((lane >> 3) & 1));
}

}  // namespace delta
}  // namespace hla
