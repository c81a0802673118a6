// The gated delta rule over a sequence: the forward walk.
//
// Within a chunk of C tokens from the carried state S0, with c the running sum of the log decays,
// D_ij = e^(c_i - c_j), M = strict_low(D o K K^T), P = scale low(D o Q K^T):
//     R = (I + M diag(beta))^-1 (V - diag(e^c) K S0)      (each token's error v - S^T k)
//     U = diag(beta) R
//     O = scale diag(e^c) Q S0 + P U
//     S = e^(c_C) S0 + K^T diag(e^(c_C - c)) U
// A block owns CS = 16 NG value columns of one head (S's columns do not mix).  Two warps hold the
// state of 16 columns transposed in registers, half of the key axis each, so S^T, Y^T and U^T are
// in turn the A operand of the next product and only the partial K S0 passes through shared memory.
#include "delta_walk.cuh"

namespace hla {
namespace delta {
namespace {

enum Mode { OUT = 0, SUMMARY = 1, STORE = 2 };

struct WalkArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    const float* start;       // states before each segment [BH][segments][d][dv], or one per head, or null
    const int* lengths;
    void* o;
    float* state_out;         // after the last segment, or null
    float* sums;              // SUMMARY: [BH][segments - 1][d][dv + d]
    int Hk, H, T, dv, bthd;
    int segments, seg_chunks; // chunks of a segment
    float scale;
};

template <typename E, int DK_, int NG_, Mode MODE_>
struct Cfg {
    using Elem = E;
    static constexpr int DK = DK_, NG = NG_, CS = 16 * NG_;
    static constexpr Mode MODE = MODE_;
    static constexpr bool BF = sizeof(E) == 2;
    static constexpr int KT = BF ? 1 : 3;             // terms of q, k
    static constexpr int OT = BF ? 2 : 3;             // terms of S0, U and P in the outputs: twice the
                                                      // 8 bits that a bf16 output keeps
    static constexpr bool PIPE = BF || DK_ < 128;     // fp32 at d = 128 has no room for that
    static constexpr int NST = PIPE ? (BF ? 6 : 5) : 2;
    static constexpr int NLD = BF ? 1 : 4;            // loader warps (fp32 tiles are split on the way)
    static constexpr int W_STATE = 2 * NG_, W_OUT = 2, W_PROD = 2;
    static constexpr int WARPS = W_STATE + W_OUT + W_PROD + 1 + NLD;
    static constexpr int KTILE = KT * C * DK_ * 2;
    static constexpr int VTILE = cols_bytes<E, CS>();
    static constexpr int NP = PIPE ? 4 : 1, N2 = PIPE ? 2 : 1;
    // shared memory, bytes
    static constexpr int k = 0;
    static constexpr int q = k + NST * KTILE;
    static constexpr int v = q + (MODE_ == OUT ? NST * KTILE : 0);
    static constexpr int gates = v + NST * VTILE;
    static constexpr int m = gates + NST * static_cast<int>(sizeof(Gates));
    static constexpr int p = m + N2 * C * kMS * 4;
    static constexpr int PB = OT * C * C * 2;
    static constexpr int x = p + (MODE_ == OUT ? NP * PB : 0);
    static constexpr int XB = 3 * C * C * 2;
    static constexpr int sf = x + N2 * XB;
    static constexpr int SB = NG_ * (DK_ / 16) * OT * 512;
    static constexpr int uf = sf + (MODE_ == OUT ? N2 * SB : 0);
    static constexpr int UB = NG_ * 2 * OT * 512;
    static constexpr int ex = uf + (MODE_ == OUT ? N2 * UB : 0);
    static constexpr int bytes = ex + W_STATE * 2048;
};

template <typename F>
__global__ void __launch_bounds__(F::WARPS * 32, 1) k_delta_walk(const WalkArgs a) {
    using E = typename F::Elem;
    constexpr int DK = F::DK, DH = DK / 2, NG = F::NG, CS = F::CS, KT = F::KT, OT = F::OT;
    constexpr bool PIPE = F::PIPE;
    constexpr Mode MODE = F::MODE;
    extern __shared__ __align__(128) uint8_t sm[];
    const uint32_t sb = ptx::smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // block -> (head, segment, columns)
    const int vslices = a.dv / CS;
    const int slices = MODE == SUMMARY ? vslices + DK / CS : vslices;
    const int walked = MODE == SUMMARY ? a.segments - 1 : a.segments;
    const int slice = blockIdx.x % slices, seg = (blockIdx.x / slices) % walked, bh = blockIdx.x / slices / walked;
    const bool unit = MODE == SUMMARY && slice >= vslices;      // columns of the transition: v = 0, S = I
    const int col0 = (unit ? slice - vslices : slice) * CS;
    if (unit && seg == 0) return;                               // the first segment starts from the given state
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int T = length_of(a.lengths, b, a.T);
    const int t_first = seg * a.seg_chunks * C;
    const int t_last = seg + 1 == a.segments ? a.T : min(a.T, t_first + a.seg_chunks * C);   // rows of this segment
    const int t_end = min(T, t_last);
    const int chunks = t_end > t_first ? (t_end - t_first + C - 1) / C : 0;

    const int kstep = row_step(a.bthd, a.Hk), vstep = row_step(a.bthd, a.H);
    const long long krow = row_of(a.bthd, b, hk, a.Hk, t_first, a.T);
    const long long vrow = row_of(a.bthd, b, h, a.H, t_first, a.T);

    // roles
    const int w_out = F::W_STATE, w_prod = w_out + F::W_OUT, w_inv = w_prod + F::W_PROD, w_load = w_inv + 1;
    const int grp = warp >> 1, half = warp & 1;                 // state warps
    float S[DH / 8][4];
    if (warp < F::W_STATE) {
        // S^T: this lane's columns col, col + 8, keys 8 n + 2 (lane % 4), + 1 of its half
        const int col = col0 + 16 * grp + (lane >> 2), key = half * DH + 2 * (lane & 3);
        const float* from = nullptr;
        if (a.start && !unit && (MODE != SUMMARY || seg == 0))
            from = a.start + (MODE == SUMMARY ? bh : static_cast<long long>(bh) * a.segments + seg) * DK * a.dv;
#pragma unroll
        for (int n = 0; n < DH / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int kk = key + 8 * n + (j & 1), cc = col + 8 * (j >> 1);
                S[n][j] = unit ? (kk == cc ? 1.f : 0.f) : (from ? from[static_cast<long long>(kk) * a.dv + cc] : 0.f);
            }
    }
    float next_g = 0.f, next_beta = 0.f;

    const int s0 = -4, s1 = PIPE ? chunks : 4 * chunks - 1;
    if (chunks > 0)
    for (int s = s0; s <= s1; ++s) {
        if (warp < F::W_STATE) {
            // ------------------------------------------------ state
            const int c = chunk_of<PIPE>(s, 0, 2);
            if (c >= 0 && c < chunks) {
                const int st = c % F::NST, c2 = c % F::N2;
                const Gates* G = reinterpret_cast<const Gates*>(sm + F::gates) + st;
                const uint32_t kt = sb + F::k + st * F::KTILE, vt = sb + F::v + st * F::VTILE;
                const uint32_t xt = sb + F::x + c2 * F::XB;
                uint4* sf = reinterpret_cast<uint4*>(sm + F::sf + c2 * F::SB);
                uint4* uf = reinterpret_cast<uint4*>(sm + F::uf + c2 * F::UB);
                float y[4][4] = {};
                // this half's part of S0^T K^T
#pragma unroll
                for (int ks = 0; ks < DH / 16; ++ks) {
                    uint32_t as[3][4];
                    split_a<3>(S[2 * ks], S[2 * ks + 1], as);
                    if (MODE == OUT) {
#pragma unroll
                        for (int t = 0; t < OT; ++t)
                            sf[((grp * (DK / 16) + half * (DH / 16) + ks) * OT + t) * 32 + lane] =
                                make_uint4(as[t][0], as[t][1], as[t][2], as[t][3]);
                    }
#pragma unroll
                    for (int np = 0; np < 2; ++np) {
                        uint32_t bk[KT][4];
#pragma unroll
                        for (int t = 0; t < KT; ++t)
                            ldsm4(bk[t], at_pieces_first<DK * 2>(kt + t * (C * DK * 2), 16 * np, half * (DH / 8) + 2 * ks, lane));
                        prod2<3, KT>(y[2 * np], y[2 * np + 1], as, bk);
                    }
                }
                float4* ex = reinterpret_cast<float4*>(sm + F::ex);
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    ex[((grp * 2 + half) * 4 + n) * 32 + lane] = make_float4(y[n][0], y[n][1], y[n][2], y[n][3]);
                ptx::named_sync(1 + grp, 64);
                // Y^T = V^T - (S0^T K^T) e^c
#pragma unroll
                for (int np = 0; np < 2; ++np) {
                    float v0[4] = {}, v1[4] = {};
                    if (!unit) cols_t<CS>(static_cast<const E*>(nullptr), vt, 16 * grp, 16 * np, lane, v0, v1);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int n = 2 * np + e;
                        const float4 o = ex[((grp * 2 + (half ^ 1)) * 4 + n) * 32 + lane];
                        const float2 f = *reinterpret_cast<const float2*>(&G->since[8 * n + 2 * (lane & 3)]);
                        const float (&vv)[4] = e ? v1 : v0;
                        y[n][0] = fmaf(-f.x, y[n][0] + o.x, vv[0]);
                        y[n][1] = fmaf(-f.y, y[n][1] + o.y, vv[1]);
                        y[n][2] = fmaf(-f.x, y[n][2] + o.z, vv[2]);
                        y[n][3] = fmaf(-f.y, y[n][3] + o.w, vv[3]);
                    }
                }
                // R^T = Y^T X^T, X lower triangular: tokens 16.. of the sum reach tokens 16.. alone
                float r[4][4] = {};
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t ay[3][4];
                    split_a<3>(y[2 * kk], y[2 * kk + 1], ay);
#pragma unroll
                    for (int np = kk; np < 2; ++np) {
                        uint32_t bx[3][4];
#pragma unroll
                        for (int t = 0; t < 3; ++t) ldsm4(bx[t], at_pieces_first<C * 2>(xt + t * (C * C * 2), 16 * np, 2 * kk, lane));
                        prod2<3, 3>(r[2 * np], r[2 * np + 1], ay, bx);
                    }
                }
                // U^T, for the outputs, and U^T e^(c_C - c), for the state
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 be = *reinterpret_cast<const float2*>(&G->beta[8 * n + 2 * (lane & 3)]);
                    r[n][0] *= be.x; r[n][1] *= be.y; r[n][2] *= be.x; r[n][3] *= be.y;
                }
                if (MODE == OUT) {
                    uint32_t au[OT][4];
                    if (half == 0) split_a<OT>(r[0], r[1], au);
                    else split_a<OT>(r[2], r[3], au);
#pragma unroll
                    for (int t = 0; t < OT; ++t)
                        uf[((grp * 2 + half) * OT + t) * 32 + lane] = make_uint4(au[t][0], au[t][1], au[t][2], au[t][3]);
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 f = *reinterpret_cast<const float2*>(&G->left[8 * n + 2 * (lane & 3)]);
                    r[n][0] *= f.x; r[n][1] *= f.y; r[n][2] *= f.x; r[n][3] *= f.y;
                }
                const float all = G->all;
#pragma unroll
                for (int n = 0; n < DH / 8; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[n][j] *= all;
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t au[3][4];
                    split_a<3>(r[2 * kk], r[2 * kk + 1], au);
#pragma unroll
                    for (int np = 0; np < DH / 16; ++np) {
                        uint32_t bk[KT][4];
#pragma unroll
                        for (int t = 0; t < KT; ++t)
                            ldsm4t(bk[t], at_rows_first<DK * 2>(kt + t * (C * DK * 2), 16 * kk, half * (DH / 8) + 2 * np, lane));
                        prod2<3, KT>(S[2 * np], S[2 * np + 1], au, bk);
                    }
                }
            }
        } else if (warp < w_prod) {
            // ------------------------------------------------ output: 16 tokens a warp
            const int c = chunk_of<PIPE>(s, -1, 3);
            if (MODE == OUT && c >= 0 && c < chunks) {
                const int st = c % F::NST, c2 = c % F::N2, i0 = 16 * (warp - w_out);
                const Gates* G = reinterpret_cast<const Gates*>(sm + F::gates) + st;
                const uint32_t qt = sb + F::q + st * F::KTILE, pt = sb + F::p + (c % F::NP) * F::PB;
                const uint4* sf = reinterpret_cast<const uint4*>(sm + F::sf + c2 * F::SB);
                const uint4* uf = reinterpret_cast<const uint4*>(sm + F::uf + c2 * F::UB);
                float acc[2 * NG][4] = {};
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    uint32_t aq[KT][4];
#pragma unroll
                    for (int t = 0; t < KT; ++t) ldsm4(aq[t], at_rows_first<DK * 2>(qt + t * (C * DK * 2), i0, 2 * ks, lane));
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        uint32_t bs[OT][4];
#pragma unroll
                        for (int t = 0; t < OT; ++t) {
                            const uint4 u = sf[((g * (DK / 16) + ks) * OT + t) * 32 + lane];
                            bs[t][0] = u.x; bs[t][1] = u.z; bs[t][2] = u.y; bs[t][3] = u.w;
                        }
                        prod2<KT, OT>(acc[2 * g], acc[2 * g + 1], aq, bs);
                    }
                }
                const int r0 = i0 + (lane >> 2);
                const float f0 = a.scale * G->since[r0], f1 = a.scale * G->since[r0 + 8];
#pragma unroll
                for (int n = 0; n < 2 * NG; ++n) {
                    acc[n][0] *= f0; acc[n][1] *= f0; acc[n][2] *= f1; acc[n][3] *= f1;
                }
                for (int kk = 0; kk <= warp - w_out; ++kk) {
                    uint32_t ap[OT][4];
#pragma unroll
                    for (int t = 0; t < OT; ++t) ldsm4(ap[t], at_rows_first<C * 2>(pt + t * (C * C * 2), i0, 2 * kk, lane));
#pragma unroll
                    for (int g = 0; g < NG; ++g) {
                        uint32_t bu[OT][4];
#pragma unroll
                        for (int t = 0; t < OT; ++t) {
                            const uint4 u = uf[((g * 2 + kk) * OT + t) * 32 + lane];
                            bu[t][0] = u.x; bu[t][1] = u.z; bu[t][2] = u.y; bu[t][3] = u.w;
                        }
                        prod2<OT, OT>(acc[2 * g], acc[2 * g + 1], ap, bu);
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tok = c * C + r0 + 8 * e;              // within the segment
                    if (t_first + tok >= t_last) continue;
                    const bool on = t_first + tok < t_end;
                    E* o = static_cast<E*>(a.o) + (vrow + static_cast<long long>(tok) * vstep) * a.dv + col0 + 2 * (lane & 3);
#pragma unroll
                    for (int n = 0; n < 2 * NG; ++n) {
                        const float x0 = on ? acc[n][2 * e] : 0.f, x1 = on ? acc[n][2 * e + 1] : 0.f;
                        if constexpr (F::BF) *reinterpret_cast<uint32_t*>(o + 8 * n) = ptx::pack_bf16(x0, x1);
                        else *reinterpret_cast<float2*>(o + 8 * n) = make_float2(x0, x1);
                    }
                }
            }
        } else if (warp < w_inv) {
            // ------------------------------------------------ products
            const int c = chunk_of<PIPE>(s, 2, 0);
            if (c >= 0 && c < chunks) {
                const int st = c % F::NST;
                products<DK, KT, OT, MODE == OUT, false>(
                    sb + F::k + st * F::KTILE, sb + F::q + st * F::KTILE, reinterpret_cast<const Gates*>(sm + F::gates) + st,
                    reinterpret_cast<float*>(sm + F::m) + (c % F::N2) * C * kMS, sm + F::p + (c % F::NP) * F::PB, a.scale,
                    warp - w_prod, lane);
            }
        } else if (warp < w_load) {
            // ------------------------------------------------ inverse
            const int c = chunk_of<PIPE>(s, 1, 1);
            if (c >= 0 && c < chunks)
                invert(reinterpret_cast<const float*>(sm + F::m) + (c % F::N2) * C * kMS, sm + F::x + (c % F::N2) * F::XB, lane);
        } else {
            // ------------------------------------------------ load: bf16 tiles are asked for four chunks
            // ahead and there three ahead; fp32 tiles are loaded and split three ahead
            const int lt = (warp - w_load) * 32 + lane;
            constexpr int LT = F::NLD * 32;
            const int c = PIPE ? (F::BF ? s + 4 : s + 3) : ((s & 3) == 0 ? (s >> 2) + 1 : -1);
            const float g_was = next_g, beta_was = next_beta;
            if (c >= 0 && c < chunks) {
                const int st = c % F::NST, rows = min(C, t_end - t_first - c * C);
                const long long kr = krow + static_cast<long long>(c) * C * kstep, vr = vrow + static_cast<long long>(c) * C * vstep;
                const long long ks = static_cast<long long>(kstep) * DK, vs = static_cast<long long>(vstep) * a.dv;
                load_tile<DK, KT, LT>(sb + F::k + st * F::KTILE, static_cast<const E*>(a.k) + kr * DK, ks, rows, lt);
                if (MODE == OUT) load_tile<DK, KT, LT>(sb + F::q + st * F::KTILE, static_cast<const E*>(a.q) + kr * DK, ks, rows, lt);
                if (!unit) load_cols<CS, LT>(sb + F::v + st * F::VTILE, static_cast<const E*>(a.v) + vr * a.dv + col0, vs, rows, lt);
                if (warp == w_load) {
                    const bool on = lane < rows;
                    next_g = on ? a.g[vr + static_cast<long long>(lane) * vstep] : 0.f;
                    next_beta = on ? a.beta[vr + static_cast<long long>(lane) * vstep] : 0.f;
                    if (!(PIPE && F::BF)) finish_gates(reinterpret_cast<Gates*>(sm + F::gates) + st, next_g, next_beta, lane);
                }
            }
            cp_commit();
            if constexpr (PIPE && F::BF) {
                cp_wait<1>();
                if (c - 1 >= 0 && c - 1 < chunks)
                    finish_gates(reinterpret_cast<Gates*>(sm + F::gates) + (c - 1) % F::NST, g_was, beta_was, lane);
            } else {
                cp_wait<0>();
            }
        }
        __syncthreads();
    }

    if (warp < F::W_STATE) {
        const int col = col0 + 16 * grp + (lane >> 2), key = half * DH + 2 * (lane & 3);
        float* to = nullptr;
        long long width = a.dv;
        if (MODE == SUMMARY) {
            width = a.dv + DK;
            to = a.sums + (static_cast<long long>(bh) * walked + seg) * DK * width + (unit ? a.dv : 0);
        } else if (a.state_out && seg + 1 == a.segments) {
            to = a.state_out + static_cast<long long>(bh) * DK * a.dv;
        }
        if (to)
#pragma unroll
            for (int n = 0; n < DH / 8; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    to[static_cast<long long>(key + 8 * n + (j & 1)) * width + col + 8 * (j >> 1)] = S[n][j];
    }
    if (MODE == OUT) {
        // rows behind the sequence's end that no chunk covers
        for (int i = t_first + chunks * C + tid / (CS / 4); i < t_last; i += F::WARPS * 32 / (CS / 4)) {
            const float zero[4] = {};
            store4(static_cast<E*>(a.o) + (vrow + static_cast<long long>(i - t_first) * vstep) * a.dv + col0 + 4 * (tid % (CS / 4)), zero);
        }
    }
}

template <typename F>
cudaError_t start(const WalkArgs& a, int blocks, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(k_delta_walk<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::bytes);
    if (e != cudaSuccess) return e;
    k_delta_walk<F><<<blocks, F::WARPS * 32, F::bytes, st>>>(a);
    return cudaGetLastError();
}

template <typename E, int DK>
cudaError_t walk(const Problem& p, cudaStream_t st) {
    constexpr int NG = sizeof(E) == 2 ? 2 : 1;
    using F = Cfg<E, DK, NG, OUT>;
    static_assert(F::bytes <= 227 * 1024, "shared memory of a block");
    const int BH = p.B * p.H, NC = (p.T + C - 1) / C;
    WalkArgs a{p.q, p.k, p.v, p.g, p.beta, p.state_in, p.lengths, p.o, p.state_out, nullptr,
               p.Hk, p.H, p.T, p.dv, p.bthd ? 1 : 0, 1, NC, p.scale};
    return start<F>(a, BH * (p.dv / F::CS), st);
}

}  // namespace

cudaError_t forward(const Problem& p, cudaStream_t st) {
    if (p.bf16) {
        if (p.d == 32) return walk<bf16, 32>(p, st);
        if (p.d == 64) return walk<bf16, 64>(p, st);
        return walk<bf16, 128>(p, st);
    }
    if (p.d == 32) return walk<float, 32>(p, st);
    if (p.d == 64) return walk<float, 64>(p, st);
    return walk<float, 128>(p, st);
}

}  // namespace delta
}  // namespace hla
