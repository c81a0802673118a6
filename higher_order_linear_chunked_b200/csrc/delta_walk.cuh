// Pieces of the gated delta rule's chunk kernels: what a chunk needs that does not depend on the
// carried state (its decayed products, the inverse of its unit triangular system, its gate values:
// a record in the workspace, written by delta_prepare.cu for all chunks at once), and the loaders
// of the kernels that walk the chunks.
#pragma once
#include "delta_mma.cuh"

#include <atomic>

namespace hla {
namespace delta {

// Dynamic shared memory of a kernel, asked for once a device (the attribute stays with the device), and
// all of an SM's memory as shared memory: blocks of another kernel fit beside this one's only where the
// split between shared memory and cache leaves them room, and the split of a busy SM stays as it is.
template <auto KERNEL>
inline cudaError_t allow_smem(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Two kernels that do not need one another run side by side: the second one is a programmatic dependent
// of the first, launched once every block of the first has passed next_may_start(), and waits for the
// first one's end at its own (previous_done()), so that whatever follows finds both complete.  What the
// first one follows is an ordinary dependency of the first, complete before any of its blocks starts.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void previous_done() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename A, typename... Args>
inline cudaError_t launch_beside(void (*kernel)(A, Args...), int blocks, int threads, int smem, cudaStream_t st, A a, Args... more) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, more...);
}

constexpr int kMS = 36;                      // floats of a row of the transposed system

// Gate values of a chunk: e^c, e^(c_last - c), beta, e^(c_last); c = sum of g up to the token.
struct Gates {
    float since[C], left[C], beta[C];
    float all;
    float pad[31];
};
static_assert(sizeof(Gates) == 512, "a record's last piece");

// Bytes of a chunk's record: `inverses` inverses and P, in three terms each, and the gates.
constexpr int kXBytes = 3 * C * C * 2;
constexpr int record_bytes(int inverses) { return (inverses + 1) * kXBytes + 512; }

__device__ __forceinline__ float ex2(float x) {      // 2^x to 2^-22, below 2^-126 zero
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^x, the whole part apart from the rest: a rounding of a large x costs nothing
__device__ __forceinline__ float ex2_long(double x) {
    const float n = rintf(static_cast<float>(x));
    return ex2(static_cast<float>(x - static_cast<double>(n))) * ex2(n);
}

// 32 rows of D elements into KT swizzled bf16 tiles, by NT threads; rows >= `rows` become zeros.
template <int D, int KT, int NT>
__device__ __forceinline__ void load_tile(uint32_t tile, const bf16* src, long long step, int rows, int tid) {
    static_assert(KT == 1, "bf16 inputs are one term");
    constexpr int P = D / 8;
    const int c = tid % P;
    src += c * 8;
#pragma unroll 4
    for (int r = tid / P; r < C; r += NT / P) {
        const bool on = r < rows;
        cp_async16(tile + piece<D * 2>(r, c), src + (on ? r * step : 0), on);
    }
}
template <int D, int KT, int NT>
__device__ __forceinline__ void load_tile(uint32_t tile, const float* src, long long step, int rows, int tid) {
    constexpr int P = D / 4;                  // four floats at a time
    constexpr int N = (C * P + NT - 1) / NT;
    constexpr int U = N < 8 ? N : 8;
#pragma unroll 1
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
// N bytes as they are (a record's piece), by NT threads.
template <int N, int NT>
__device__ __forceinline__ void load_bytes(uint32_t to, const uint8_t* src, int tid) {
#pragma unroll 4
    for (int i = tid; i < N / 16; i += NT) cp_async16(to + i * 16, src + i * 16, true);
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

// Gate values of one chunk from each lane's g and beta (lane = token; idle tokens: 0 and 0), and
// sum[i] = c_i / ln 2 as hi + lo: the difference of two such sums keeps 2^-24 of the gap however
// large the sums are.
__device__ __forceinline__ void finish_gates(Gates* s, float2* sum, float g, float beta, int lane) {
    double c = static_cast<double>(gate(g)) * 1.4426950408889634;   // 1 / ln 2
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, c, w);
        if (lane >= w) c += o;
    }
    const double last = __shfl_sync(0xffffffffu, c, 31);
    const float hi = static_cast<float>(c);
    sum[lane] = make_float2(hi, static_cast<float>(c - static_cast<double>(hi)));
    const float since = ex2_long(c);
    s->since[lane] = since;
    s->left[lane] = ex2_long(last - c);
    s->beta[lane] = beta;
    s->pad[lane < 31 ? lane : 30] = 0.f;
    if (lane == 31) s->all = since;
}

// 16 rows (16p..) of a chunk's decayed products with the keys, one warp.
//   keys:  M = strict_low(D o K K^T) with a beta factor (rowbeta: beta_i, else beta_j), to mt[j][i]
//   else:  P = scale low(D o Q K^T) as three bf16 terms, to pt
template <int DK, int KT>
__device__ __forceinline__ void products(bool keys, bool rowbeta, uint32_t kt, uint32_t at, const float2* sum, const float* beta,
                                         float* mt, uint8_t* pt, float scale, int p, int lane) {
    constexpr int RB = DK * 2, TERM = C * DK * 2;
    float acc[4][4] = {}, low[4][4] = {};
#pragma unroll(DK > 32 ? 2 : 1)
    for (int ks = 0; ks < DK / 16; ++ks) {
        uint32_t a[KT][4];
#pragma unroll
        for (int t = 0; t < KT; ++t) ldsm4(a[t], at_rows_first<RB>(at + t * TERM, 16 * p, 2 * ks, lane));
#pragma unroll
        for (int np = 0; np < 2; ++np) {
            if (np > p) continue;
            uint32_t b[KT][4];
#pragma unroll
            for (int t = 0; t < KT; ++t) ldsm4(b[t], at_pieces_first<RB>(kt + t * TERM, 16 * np, 2 * ks, lane));
            if constexpr (KT == 1) prod2<KT, KT>(acc[2 * np], acc[2 * np + 1], a, b);
            else prod2<KT, KT>(acc[2 * np], acc[2 * np + 1], low[2 * np], low[2 * np + 1], a, b);
        }
    }
    if constexpr (KT > 1) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] += low[n][j];
    }
    float2 ci[2];
    float fi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int i = 16 * p + (lane >> 2) + 8 * h;
        ci[h] = sum[i];
        fi[h] = keys ? (rowbeta ? beta[i] : 1.f) : scale;
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        if (nt > 2 * p + 1) continue;
        const int j0 = 8 * nt + 2 * (lane & 3);
        const float4 cj = *reinterpret_cast<const float4*>(&sum[j0]);
        float2 fj = make_float2(1.f, 1.f);
        if (!rowbeta && keys) fj = *reinterpret_cast<const float2*>(&beta[j0]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * p + (lane >> 2) + 8 * h;
            const float x0 = fi[h] * fj.x * acc[nt][2 * h] * ex2((ci[h].x - cj.x) + (ci[h].y - cj.y));
            const float x1 = fi[h] * fj.y * acc[nt][2 * h + 1] * ex2((ci[h].x - cj.z) + (ci[h].y - cj.w));
            if (keys) {
                mt[j0 * kMS + i] = j0 < i ? x0 : 0.f;
                mt[(j0 + 1) * kMS + i] = j0 + 1 < i ? x1 : 0.f;
            } else {
                uint32_t t[3];
                split<3>(j0 <= i ? x0 : 0.f, j0 + 1 <= i ? x1 : 0.f, t);
#pragma unroll
                for (int n = 0; n < 3; ++n)
                    *reinterpret_cast<uint32_t*>(pt + n * (C * C * 2) + piece<C * 2>(i, j0 >> 3) + (j0 & 7) * 2) = t[n];
            }
        }
    }
}

// X = (I + L)^-1 of the strictly lower L (mt[j][i] = L_ij) as three bf16 terms [i][j], one warp.
// The two 16 x 16 blocks on the diagonal by forward substitution in fp32, a column a lane; below
// them X21 = -X22 L21 X11 in two products of three-term operands, transposed so that the first
// one's accumulators are the second one's A operand.
__device__ __forceinline__ void invert(const float* mt, uint8_t* xt, int lane) {
    constexpr int TERM = C * C * 2;
    const int blk = lane >> 4, col = lane & 15;
    const float* m = mt + 16 * blk * (kMS + 1);
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == col ? 1.f : 0.f;
#pragma unroll
    for (int j = 0; j < 15; ++j) {
#pragma unroll
        for (int i4 = (j + 1) / 4 * 4; i4 < 16; i4 += 4) {
            const float4 f = *reinterpret_cast<const float4*>(m + j * kMS + i4);
            if (i4 + 0 > j) x[i4 + 0] = fmaf(-f.x, x[j], x[i4 + 0]);
            if (i4 + 1 > j) x[i4 + 1] = fmaf(-f.y, x[j], x[i4 + 1]);
            if (i4 + 2 > j) x[i4 + 2] = fmaf(-f.z, x[j], x[i4 + 2]);
            if (i4 + 3 > j) x[i4 + 3] = fmaf(-f.w, x[j], x[i4 + 3]);
        }
    }
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        uint32_t t[3];
        split<3>(x[i], x[i + 1], t);
#pragma unroll
        for (int n = 0; n < 3; ++n) {
            uint8_t* q = xt + n * TERM + (lane & 7) * 2;
            *reinterpret_cast<uint16_t*>(q + piece<C * 2>(16 * blk + i, lane >> 3)) = static_cast<uint16_t>(t[n]);
            *reinterpret_cast<uint16_t*>(q + piece<C * 2>(16 * blk + i + 1, lane >> 3)) = static_cast<uint16_t>(t[n] >> 16);
        }
    }
    __syncwarp();
    const uint32_t xb = ptx::smem_u32(xt);
    // Z^T [col][i] = X11^T L21^T
    uint32_t a[3][4], b[3][4];
#pragma unroll
    for (int t = 0; t < 3; ++t)   // X11 is stored [j][col]: transposed 8 x 8 blocks, rows of A = columns
        ldsm4t(a[t], xb + t * TERM + piece<C * 2>((lane >> 4) * 8 + (lane & 7), (lane >> 3) & 1));
#pragma unroll
    for (int n = 0; n < 4; ++n) {  // n-tile n >> 1, k half n & 1
        const float* l = mt + (2 * (lane & 3) + 8 * (n & 1)) * kMS + 16 + 8 * (n >> 1) + (lane >> 2);
        uint32_t t[3];
        split<3>(-l[0], -l[kMS], t);
        b[0][n] = t[0]; b[1][n] = t[1]; b[2][n] = t[2];
    }
    float z[2][4] = {};
    prod2<3, 3>(z[0], z[1], a, b);
    const bool spoilt = any_bad(z);
    int first[2];
    if (spoilt) {
        first_bad(z, lane, first);
        clean(z);
    }
    // X21^T [col][i] = -Z^T X22^T
    split_a<3>(z[0], z[1], a);
#pragma unroll
    for (int t = 0; t < 3; ++t) ldsm4(b[t], at_pieces_first<C * 2>(xb + t * TERM, 16, 2, lane));
    float y[2][4] = {};
    prod2<3, 3>(y[0], y[1], a, b);
    if (spoilt) spoil(y, lane, first);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c0 = (lane >> 2) + 8 * h, i = 16 + 8 * n + 2 * (lane & 3);
            uint32_t t[3];
            split<3>(y[n][2 * h], y[n][2 * h + 1], t);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                uint8_t* q = xt + k * TERM + (c0 & 7) * 2;
                *reinterpret_cast<uint16_t*>(q + piece<C * 2>(i, c0 >> 3)) = static_cast<uint16_t>(t[k]);
                *reinterpret_cast<uint16_t*>(q + piece<C * 2>(i + 1, c0 >> 3)) = static_cast<uint16_t>(t[k] >> 16);
            }
        }
}

}  // namespace delta
}  // namespace hla
