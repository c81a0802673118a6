// Roles shared by the forward and the reverse walk of the gated delta rule: the loader, the
// decayed products K K^T and Q K^T of a chunk, and the inverse of its unit triangular system.
//
// A block walks the chunks (32 tokens) of one head for CS value columns, a warp or two to a role,
// each role one chunk ahead of the next, one block barrier a step:
//     load (c)  ->  products (c)  ->  inverse (c)  ->  state (c)  ->  output (c)
#pragma once
#include "delta_mma.cuh"

namespace hla {
namespace delta {

constexpr int kMS = 36;                      // floats of a row of the transposed system

// Values of a chunk's decays: c = sum of g up to the token as hi + lo (differences of two such
// sums keep 2^-24 of the gap however large the sums are), e^c, e^(c_last - c), beta.
struct Gates {
    float2 sum[C];
    float since[C], left[C], beta[C];
    float all;                               // e^(c_last)
    float pad[3];
};

// Which chunk a role works on in step s: PIPE, each role `ahead` of the state's chunk s; else the
// roles take turns, four steps a chunk.
template <bool PIPE>
__device__ __forceinline__ int chunk_of(int s, int ahead, int turn) {
    if constexpr (PIPE) return s + ahead;
    return (s & 3) == turn ? (s >> 2) : -1;
}

// 32 rows of D elements into KT swizzled bf16 tiles, by NT threads; rows >= `rows` become zeros.
template <int D, int KT, int NT>
__device__ __forceinline__ void load_tile(uint32_t tile, const bf16* src, long long step, int rows, int tid) {
    static_assert(KT == 1, "bf16 inputs are one term");
    constexpr int P = D / 8;
    for (int i = tid; i < C * P; i += NT) {
        const int r = i / P, c = i % P;
        const bool on = r < rows;
        cp_async16(tile + piece<D * 2>(r, c), src + (on ? r * step : 0) + c * 8, on);
    }
}
template <int D, int KT, int NT>
__device__ __forceinline__ void load_tile(uint32_t tile, const float* src, long long step, int rows, int tid) {
    constexpr int P = D / 4;                  // four floats at a time
    constexpr int N = (C * P + NT - 1) / NT;
    constexpr int U = N < 8 ? N : 8;
    for (int base = 0; base < N; base += U) {
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tid + (base + u) * NT, r = i / P, c = i % P;
            x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < C * P && r < rows) x[u] = *reinterpret_cast<const float4*>(src + r * step + c * 4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tid + (base + u) * NT, r = i / P, c = i % P;
            if (i >= C * P) continue;
            uint32_t a[KT], b[KT];
            split<KT>(x[u].x, x[u].y, a);
            split<KT>(x[u].z, x[u].w, b);
#pragma unroll
            for (int t = 0; t < KT; ++t)
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(tile + t * (C * D * 2) + piece<D * 2>(r, c >> 1) + (c & 1) * 8),
                             "r"(a[t]), "r"(b[t]) : "memory");
        }
    }
}

// 32 rows of CS columns as they are (the values, or the gradients of the outputs).
template <int CS, int NT>
__device__ __forceinline__ void load_cols(uint32_t tile, const bf16* src, long long step, int rows, int tid) {
    constexpr int P = CS / 8;
    for (int i = tid; i < C * P; i += NT) {
        const int r = i / P, c = i % P;
        const bool on = r < rows;
        cp_async16(tile + piece<CS * 2>(r, c), src + (on ? r * step : 0) + c * 8, on);
    }
}
template <int CS, int NT>
__device__ __forceinline__ void load_cols(uint32_t tile, const float* src, long long step, int rows, int tid) {
    constexpr int P = CS / 4;                 // rows of CS + 4 floats: columns of eight rows on all banks
    for (int i = tid; i < C * P; i += NT) {
        const int r = i / P, c = i % P;
        const bool on = r < rows;
        cp_async16(tile + (r * (CS + 4) + c * 4) * 4, src + (on ? r * step : 0) + c * 4, on);
    }
}
template <typename E, int CS>
constexpr int cols_bytes() { return sizeof(E) == 2 ? C * CS * 2 : C * (CS + 4) * 4; }

// A 16-column x 8-token accumulator pair of tiles (tokens n0.., n0 + 8..) read transposed.
template <int CS>
__device__ __forceinline__ void cols_t(const bf16*, uint32_t tile, int col0, int n0, int lane, float (&x)[4], float (&y)[4]) {
    uint32_t r[4];
    // matrices: tokens n0.. cols 0-7, cols 8-15; tokens n0 + 8.. cols 0-7, cols 8-15
    ldsm4t(r, tile + piece<CS * 2>(n0 + (lane >> 4) * 8 + (lane & 7), col0 / 8 + ((lane >> 3) & 1)));
    x[0] = __uint_as_float(r[0] << 16); x[1] = __uint_as_float(r[0] & 0xffff0000u);
    x[2] = __uint_as_float(r[1] << 16); x[3] = __uint_as_float(r[1] & 0xffff0000u);
    y[0] = __uint_as_float(r[2] << 16); y[1] = __uint_as_float(r[2] & 0xffff0000u);
    y[2] = __uint_as_float(r[3] << 16); y[3] = __uint_as_float(r[3] & 0xffff0000u);
}
template <int CS>
__device__ __forceinline__ float lds(uint32_t a) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(a) : "memory");
    return x;
}
template <int CS>
__device__ __forceinline__ void cols_t(const float*, uint32_t tile, int col0, int n0, int lane, float (&x)[4], float (&y)[4]) {
    const int col = col0 + (lane >> 2), tok = n0 + 2 * (lane & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = tile + ((tok + (j & 1)) * (CS + 4) + col + (j >> 1) * 8) * 4;
        x[j] = lds<CS>(a);
        y[j] = lds<CS>(a + 8 * (CS + 4) * 4);
    }
}

// Gate values of one chunk from each lane's g and beta (lane = token; idle tokens: 0 and 0).
__device__ __forceinline__ void finish_gates(Gates* s, float g, float beta, int lane) {
    double c = gate(g);
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, c, w);
        if (lane >= w) c += o;
    }
    const double last = __shfl_sync(0xffffffffu, c, 31);
    const float hi = static_cast<float>(c);
    s->sum[lane] = make_float2(hi, static_cast<float>(c - static_cast<double>(hi)));
    s->since[lane] = expf(hi);
    s->left[lane] = expf(static_cast<float>(last - c));
    s->beta[lane] = beta;
    if (lane == 31) s->all = expf(hi);
}

// Products of a chunk, warp p of two: rows 16p.. of M = strict_low(D o K K^T) with a beta factor, to
// mt[j][i] (transposed), and of P = scale low(D o Q K^T) as PT bf16 terms.  ROWBETA: beta_i, else beta_j.
template <int DK, int KT, int PT, bool QUERY, bool ROWBETA>
__device__ __forceinline__ void products(uint32_t kt, uint32_t qt, const Gates* s, float* mt, uint8_t* pt, float scale,
                                         int p, int lane) {
    constexpr int RB = DK * 2, TERM = C * DK * 2;
    float kk[4][4] = {}, qk[4][4] = {};
#pragma unroll
    for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t a[KT][4], aq[KT][4];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            ldsm4(a[t], at_rows_first<RB>(kt + t * TERM, 16 * p, 2 * ks, lane));
            if (QUERY) ldsm4(aq[t], at_rows_first<RB>(qt + t * TERM, 16 * p, 2 * ks, lane));
        }
#pragma unroll
        for (int np = 0; np < 2; ++np) {
            if (np > p) continue;
            uint32_t b[KT][4];
#pragma unroll
            for (int t = 0; t < KT; ++t) ldsm4(b[t], at_pieces_first<RB>(kt + t * TERM, 16 * np, 2 * ks, lane));
            prod2<KT, KT>(kk[2 * np], kk[2 * np + 1], a, b);
            if (QUERY) prod2<KT, KT>(qk[2 * np], qk[2 * np + 1], aq, b);
        }
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        if (nt > 2 * p + 1) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * p + (lane >> 2) + 8 * h, j0 = 8 * nt + 2 * (lane & 3);
            const float2 ci = s->sum[i];
            const float bi = s->beta[i];
            float pr[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = j0 + e;
                const float2 cj = s->sum[j];
                const float D = j <= i ? expf((ci.x - cj.x) + (ci.y - cj.y)) : 0.f;
                mt[j * kMS + i] = j < i ? D * kk[nt][2 * h + e] * (ROWBETA ? bi : s->beta[j]) : 0.f;
                pr[e] = j <= i ? scale * D * qk[nt][2 * h + e] : 0.f;
            }
            if (QUERY) {
                uint32_t t[PT];
                split<PT>(pr[0], pr[1], t);
#pragma unroll
                for (int n = 0; n < PT; ++n)
                    *reinterpret_cast<uint32_t*>(pt + n * (C * C * 2) + piece<C * 2>(i, j0 >> 3) + (j0 & 7) * 2) = t[n];
            }
        }
    }
}

// X = (I + L)^-1 of the strictly lower L (mt[j][i] = L_ij), column `lane` by forward substitution
// in fp32, to three bf16 terms [i][j].
__device__ __forceinline__ void invert(const float* mt, uint8_t* xt, int lane) {
    float x[C];
#pragma unroll
    for (int i = 0; i < C; ++i) x[i] = i == lane ? 1.f : 0.f;
#pragma unroll
    for (int j = 0; j < C - 1; ++j) {
#pragma unroll
        for (int i4 = (j + 1) / 4 * 4; i4 < C; i4 += 4) {
            const float4 m = *reinterpret_cast<const float4*>(mt + j * kMS + i4);
            if (i4 + 0 > j) x[i4 + 0] = fmaf(-m.x, x[j], x[i4 + 0]);
            if (i4 + 1 > j) x[i4 + 1] = fmaf(-m.y, x[j], x[i4 + 1]);
            if (i4 + 2 > j) x[i4 + 2] = fmaf(-m.z, x[j], x[i4 + 2]);
            if (i4 + 3 > j) x[i4 + 3] = fmaf(-m.w, x[j], x[i4 + 3]);
        }
    }
#pragma unroll
    for (int i = 0; i < C; i += 2) {
        uint32_t t[3];
        split<3>(x[i], x[i + 1], t);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            uint8_t* q = xt + n * (C * C * 2) + (lane & 7) * 2;
            *reinterpret_cast<uint16_t*>(q + piece<C * 2>(i, lane >> 3)) = static_cast<uint16_t>(t[n]);
            *reinterpret_cast<uint16_t*>(q + piece<C * 2>(i + 1, lane >> 3)) = static_cast<uint16_t>(t[n] >> 16);
        }
    }
}

}  // namespace delta
}  // namespace hla
