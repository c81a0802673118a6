// Gradients of the gated delta rule.
//
// With a chunk's terms as in delta_forward.cu, dS the gradient at the state behind the chunk, and
//     dU = P^T dO + diag(e^(c_C - c)) K dS
//     H  = ((I + diag(beta) M)^-1)^T dU        (the gradient at U with all that U feeds)
//     Z  = diag(beta) H                        (the gradient at R, and at V)
// the gradient at the state before the chunk is
//     dS0 = e^(c_C) dS + (scale e^c Q)^T dO - (e^c K)^T Z.
// Three passes: the forward walk again, which keeps the states before blocks of chunks and R; beside it this
// reverse walk, which keeps dS behind the blocks and H; and one kernel over all blocks, which has
// then everything for dq, dk, dv, dbeta and dg.  R and H are per token, not per chunk (R is a token's
// error, H the gradient at what it writes), so the blocks need not be the walks' chunks.
#include <type_traits>

#include "delta_walk.cuh"

namespace hla {
namespace delta {
namespace {

// ------------------------------------------------------------------ reverse walk
struct ReverseArgs {
    const void *q, *k, *dout;
    const uint8_t* records;   // gradients' form
    const float* behind;      // dS behind each segment [BH][segments][d][dv]; SUMMARY: behind the last one
                              // [BH][d][dv]; or null
    const int* lengths;
    float* dstate_in;         // [BH][d][dv] or null
    float* dstates;           // [BH][blocks][d][dv]: dS behind each block
    float* H;                 // [BH][T][dv]
    float* back;              // SUMMARY: [BH][segments][d][dv], dS before each segment from zero behind it
    int Hk, Hv, T, dv, bthd, block_chunks;
    int segments, seg_chunks;
    float scale;
};

// SUMMARY: only dS before each segment but the first, from zero (behind the last: from what is given).
template <typename E, int DK_, int NG_, bool SUMMARY_>
struct Rev {
    static constexpr bool SUMMARY = SUMMARY_;
    using Elem = E;
    static constexpr int DK = DK_, CS = 16 * NG_;
    static constexpr bool BF = sizeof(E) == 2;
    static constexpr int KT = BF ? 1 : 3;
    // state warps of 16 columns, as in the forward walk, but four at d = 128: it has half again as many
    // products between its exchanges (16 heads of 4096x128: four 246 us, two 256)
    static constexpr int NH = DK_ == 128 ? 4 : (BF || DK_ == 32 ? 1 : 2);
    // with one state warp a group, another one takes the outputs' share of dS, a chunk ahead of it
    static constexpr int W_SIDE = NH == 1 ? NG_ : 0;
    static constexpr int AHEAD = (BF ? 2 : 1) + (W_SIDE ? 1 : 0), NS = AHEAD + 1, NLD = BF ? 2 : 4;
    static constexpr int W_STATE = NH * NG_, WARPS = W_STATE + W_SIDE + NLD;
    static constexpr int KTILE = KT * C * DK_ * 2, OTILE = KT * C * CS * 2, PB = 3 * C * C * 2;
    // a stage
    static constexpr int k = 0, q = k + KTILE, x = q + KTILE, p = x + kXBytes, dO = p + PB, gates = dO + OTILE;
    static constexpr int STAGE = (gates + 512 + 255) / 256 * 256;
    static constexpr int ex = NS * STAGE;               // partial sums, then the decayed Z
    static constexpr int YB = 2 * 3 * 512;
    static constexpr int yf = ex + W_STATE * 2048;      // dU as an A operand
    static constexpr int wf = yf + NG_ * YB;            // scale e^c dO as an A operand
    static constexpr int side = ex;                     // or the outputs' share of two chunks
    static constexpr int SIDE = NG_ * (DK_ / 8) * 512;
    static constexpr int bytes = NH > 1 ? wf + NG_ * YB : side + 2 * SIDE;
    static constexpr int BLOCKS = bytes <= 113 * 1024 ? 2 : 1;   // of an SM
};

template <typename F>
__global__ void __launch_bounds__(F::WARPS * 32, F::BLOCKS) k_delta_reverse(const ReverseArgs a) {
    using E = typename F::Elem;
    constexpr int DK = F::DK, NH = F::NH, DH = DK / NH, TN = 4 / (NH == 1 ? 2 : NH), CS = F::CS, KT = F::KT;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = ptx::smem_u32(sm);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = tid >> 5;
    const int slices = a.dv / CS, walked = F::SUMMARY ? a.segments - 1 : a.segments;
    const int col0 = (blockIdx.x % slices) * CS, bh = blockIdx.x / slices / walked;
    const int seg = (blockIdx.x / slices) % walked + (F::SUMMARY ? 1 : 0);
    const int b = bh / a.Hv, h = bh % a.Hv, hk = h / (a.Hv / a.Hk);
    const int T = length_of(a.lengths, b, a.T);
    const int all_chunks = (a.T + C - 1) / C, live_chunks = (T + C - 1) / C;
    const int c_first = seg * a.seg_chunks, c_end = min(live_chunks, c_first + a.seg_chunks);
    const int chunks = max(0, c_end - c_first);
    const int blocks = (all_chunks + a.block_chunks - 1) / a.block_chunks;
    const int kstep = row_step(a.bthd, a.Hk), vstep = row_step(a.bthd, a.Hv);
    constexpr int w_side = F::W_STATE, w_load = w_side + F::W_SIDE;
    const int grp = warp / NH, part = warp % NH;

    float S[DH / 8][4];                                 // dS^T, as the forward walk holds S^T
    const int own_col = col0 + 16 * grp + (lane >> 2), own_key = part * DH + 2 * (lane & 3);
    if (warp < w_side) {
        const float* from = nullptr;
        if (a.behind && !F::SUMMARY) from = a.behind + (static_cast<long long>(bh) * a.segments + seg) * DK * a.dv;
        if (a.behind && F::SUMMARY && seg == a.segments - 1) from = a.behind + static_cast<long long>(bh) * DK * a.dv;
#pragma unroll
        for (int n = 0; n < DH / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                S[n][j] = from ? from[static_cast<long long>(own_key + 8 * n + (j & 1)) * a.dv + own_col + 8 * (j >> 1)] : 0.f;
    }
    constexpr int ALL = F::WARPS * 32;
    const auto step_end = [] { ptx::named_sync(15, ALL); };
    if (chunks > 0 && warp < w_side) {
        const uint32_t k_n = at_pieces_first<DK * 2>(sb + F::k, 0, part * (DH / 8), lane);
        const uint32_t k_t = at_rows_first<DK * 2>(sb + F::k, 0, part * (DH / 8), lane);
        const uint32_t q_t = at_rows_first<DK * 2>(sb + F::q, 0, part * (DH / 8), lane);
        float4* const ex = reinterpret_cast<float4*>(sm + F::ex) + grp * NH * 128 + lane;
        uint8_t* const yf = sm + F::yf + grp * F::YB;
        uint8_t* const wf = sm + F::wf + grp * F::YB;
        uint8_t* const vf = reinterpret_cast<uint8_t*>(ex - lane);
        int stage = 0;
        for (int s = -F::AHEAD; s < 0; ++s) step_end();
        for (int c = c_end - 1; c >= c_first; --c) {
            const uint32_t so = stage * F::STAGE;
            const Gates* G = reinterpret_cast<const Gates*>(sm + stage * F::STAGE + F::gates);
            if (!F::SUMMARY && (c % a.block_chunks == a.block_chunks - 1 || c == live_chunks - 1)) {
                float* to = a.dstates + (static_cast<long long>(bh) * blocks + c / a.block_chunks) * DK * a.dv +
                            static_cast<long long>(own_key) * a.dv + own_col;
#pragma unroll
                for (int n = 0; n < DH / 8; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) to[static_cast<long long>(8 * n + (j & 1)) * a.dv + 8 * (j >> 1)] = S[n][j];
            }
            if constexpr (NH == 1) {
                // one warp has the whole key axis: everything stays in its registers
                float y[4][4] = {};
#pragma unroll
                for (int ks = 0; ks < DK / 16; ++ks) {
                    uint32_t bk[2][KT][4], as[3][4];
#pragma unroll
                    for (int np = 0; np < 2; ++np)
#pragma unroll
                        for (int t = 0; t < KT; ++t)
                            ldsm4(bk[np][t], ((k_n + so) ^ (ks << 5)) + t * (C * DK * 2) + np * 16 * DK * 2);
                    split_a<3>(S[2 * ks], S[2 * ks + 1], as);
                    prod<3, KT, 2>(y, as, bk);
                }
                // dU^T = dO^T P + (dS^T K^T) e^(c_C - c); P[i][j] is zero for j > i
                uint32_t ao[2][KT][4];
                float z[4][4] = {};
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                    for (int t = 0; t < KT; ++t)
                        ldsm4t(ao[kk][t], sb + F::dO + so + t * (C * CS * 2) +
                                              piece<CS * 2>(16 * kk + (lane >> 4) * 8 + (lane & 7), 2 * grp + ((lane >> 3) & 1)));
#pragma unroll
                    for (int np = 0; np <= kk; ++np) {
                        uint32_t bp[3][4];
#pragma unroll
                        for (int t = 0; t < 3; ++t)
                            ldsm4t(bp[t], at_rows_first<C * 2>(sb + F::p + so + t * (C * C * 2), 16 * kk, 2 * np, lane));
                        prod2<KT, 3>(z[2 * np], z[2 * np + 1], ao[kk], bp);
                    }
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 f = *reinterpret_cast<const float2*>(&G->left[8 * n + 2 * (lane & 3)]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) z[n][j] = fmaf((j & 1) ? f.y : f.x, y[n][j], z[n][j]);
                }
                // H^T = dU^T X'; X'[j][i] is zero for j < i
                float r[4][4] = {};
#pragma unroll
                for (int kk = 1; kk >= 0; --kk) {
                    uint32_t ay[3][4];
                    split_a<3>(z[2 * kk], z[2 * kk + 1], ay);
#pragma unroll
                    for (int np = 0; np <= kk; ++np) {
                        uint32_t bx[3][4];
#pragma unroll
                        for (int t = 0; t < 3; ++t)
                            ldsm4t(bx[t], at_rows_first<C * 2>(sb + F::x + so + t * (C * C * 2), 16 * kk, 2 * np, lane));
                        prod2<3, 3>(r[2 * np], r[2 * np + 1], ay, bx);
                    }
                }
                if (!F::SUMMARY) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int tok = c * C + 8 * n + 2 * (lane & 3);
                        float* to = a.H + (static_cast<long long>(bh) * a.T + tok) * a.dv + own_col;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (tok + (j & 1) < T) to[(j & 1) * a.dv + 8 * (j >> 1)] = r[n][j];
                    }
                }
                // dS0^T: the outputs' share from the side warp, and -(e^c K)^T Z, transposed
                uint32_t au[2][3][4];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 f = *reinterpret_cast<const float2*>(&G->since[16 * kk + 8 * e + 2 * (lane & 3)]);
                        const float2 be = *reinterpret_cast<const float2*>(&G->beta[16 * kk + 8 * e + 2 * (lane & 3)]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[2 * kk + e][j] *= (j & 1) ? -f.y * be.y : -f.x * be.x;
                    }
                    split_a<3>(r[2 * kk], r[2 * kk + 1], au[kk]);
                }
                const float4* sd = reinterpret_cast<const float4*>(sm + F::side + (c & 1) * F::SIDE) + grp * (DK / 8) * 32 + lane;
#pragma unroll
                for (int g = 0; g < DK / 32; ++g) {
                    float W[4][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const float4 x = sd[(4 * g + n) * 32];
                        W[n][0] = x.x; W[n][1] = x.y; W[n][2] = x.z; W[n][3] = x.w;
                    }
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        uint32_t bt[2][KT][4];
#pragma unroll
                        for (int np = 0; np < 2; ++np)
#pragma unroll
                            for (int t = 0; t < KT; ++t)
                                ldsm4t(bt[np][t], ((k_t + so) ^ ((2 * g + np) << 5)) + t * (C * DK * 2) + kk * 16 * DK * 2);
                        prod<3, KT, 2>(W, au[kk], bt);
                    }
                    decay_and_add(S + 4 * g, G->all, W);
                }
            } else {
            // this part's share of dS^T K^T, all tokens
            float y[4][4] = {};
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
                uint32_t bk[2][KT][4];
#pragma unroll
                for (int np = 0; np < 2; ++np)
#pragma unroll
                    for (int t = 0; t < KT; ++t)
                        ldsm4(bk[np][t], ((k_n + so) ^ (ks << 5)) + t * (C * DK * 2) + np * 16 * DK * 2);
                uint32_t as[3][4];
                split_a<3>(S[2 * ks], S[2 * ks + 1], as);
                prod<3, KT, 2>(y, as, bk);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n / TN != part) ex[(part * 4 + n) * 32] = make_float4(y[n][0], y[n][1], y[n][2], y[n][3]);
            // meanwhile, for the tokens of this part: dO^T P, and scale e^c dO^T for the state
            float2 since[TN], beta[TN], left[TN];
            float z[TN][4];
            uint32_t ao[2][KT][4];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < KT; ++t)      // [col][token] out of rows of tokens: transposed 8 x 8 blocks
                    ldsm4t(ao[kk][t], sb + F::dO + so + t * (C * CS * 2) +
                                          piece<CS * 2>(16 * kk + (lane >> 4) * 8 + (lane & 7), 2 * grp + ((lane >> 3) & 1)));
#pragma unroll
            for (int e = 0; e < TN; ++e) {
                const int n = part * TN + e, tok = 8 * n + 2 * (lane & 3);
                since[e] = *reinterpret_cast<const float2*>(&G->since[tok]);
                beta[e] = *reinterpret_cast<const float2*>(&G->beta[tok]);
                left[e] = *reinterpret_cast<const float2*>(&G->left[tok]);
                uint32_t bp[3][4];
#pragma unroll
                for (int t = 0; t < 3; ++t)       // P[i][j], i the summed axis: all four blocks of rows of piece n
                    ldsm4t(bp[t], sb + F::p + so + t * (C * C * 2) + piece<C * 2>(lane, n));
                float r[2][4] = {};
                constexpr int M = 3;
#pragma unroll
                for (int i = 0; i < KT; ++i)
#pragma unroll
                    for (int j = 0; j < 3; ++j)
                        if (i + j < M) {
                            mma16816(r[1], ao[1][i], bp[j][2], bp[j][3]);
                            if (n < 2) mma16816(r[0], ao[0][i], bp[j][0], bp[j][1]);
                        }
                // the outputs' gradients of this tile themselves, in the accumulators' layout
                float o[4] = {};
#pragma unroll
                for (int t = KT - 1; t >= 0; --t) {
                    // registers 0, 1: the first tile of 16 tokens, 2, 3: the second (constant indexes only)
                    const uint32_t lo = n < 2 ? ((n & 1) ? ao[0][t][2] : ao[0][t][0]) : ((n & 1) ? ao[1][t][2] : ao[1][t][0]);
                    const uint32_t hi = n < 2 ? ((n & 1) ? ao[0][t][3] : ao[0][t][1]) : ((n & 1) ? ao[1][t][3] : ao[1][t][1]);
                    o[0] += __uint_as_float(lo << 16); o[1] += __uint_as_float(lo & 0xffff0000u);
                    o[2] += __uint_as_float(hi << 16); o[3] += __uint_as_float(hi & 0xffff0000u);
                }
                uint32_t t0[3], t1[3];
                const float f0 = a.scale * since[e].x, f1 = a.scale * since[e].y;
                split<3>(o[0] * f0, o[1] * f1, t0);
                split<3>(o[2] * f0, o[3] * f1, t1);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    reinterpret_cast<uint2*>(wf)[((n >> 1) * 3 + t) * 64 + lane * 2 + (n & 1)] = make_uint2(t0[t], t1[t]);
#pragma unroll
                for (int j = 0; j < 4; ++j) z[e][j] = r[0][j] + r[1][j];
            }
            uint32_t bx[TN][3][4];
#pragma unroll
            for (int e = 0; e < TN; ++e)
#pragma unroll
                for (int t = 0; t < 3; ++t)       // X'[j][i], j the summed axis
                    ldsm4t(bx[e][t], sb + F::x + so + t * (C * C * 2) + piece<C * 2>(lane, part * TN + e));
            float mine[TN][4];
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n / TN == part)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mine[n % TN][j] = y[n][j];
            ptx::named_sync(1 + grp, NH * 32);
#pragma unroll
            for (int e = 0; e < TN; ++e) {
                const int n = part * TN + e;
                float w[4] = {mine[e][0], mine[e][1], mine[e][2], mine[e][3]};
#pragma unroll
                for (int o = 1; o < NH; ++o) {
                    const float4 x = ex[((part ^ o) * 4 + n) * 32];
                    w[0] += x.x; w[1] += x.y; w[2] += x.z; w[3] += x.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) z[e][j] = fmaf((j & 1) ? left[e].y : left[e].x, w[j], z[e][j]);
                uint32_t t0[3], t1[3];
                split<3>(z[e][0], z[e][1], t0);
                split<3>(z[e][2], z[e][3], t1);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    reinterpret_cast<uint2*>(yf)[((n >> 1) * 3 + t) * 64 + lane * 2 + (n & 1)] = make_uint2(t0[t], t1[t]);
            }
            float W[DH / 8][4] = {};
            ptx::named_sync(1 + grp, NH * 32);
            // scale (e^c Q)^T dO, transposed: all parts have shared theirs by now
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t au[3][4], bq[DH / 16][KT][4];
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const uint4 u = reinterpret_cast<const uint4*>(wf)[(kk * 3 + t) * 32 + lane];
                    au[t][0] = u.x; au[t][1] = u.y; au[t][2] = u.z; au[t][3] = u.w;
                }
#pragma unroll
                for (int np = 0; np < DH / 16; ++np)
#pragma unroll
                    for (int t = 0; t < KT; ++t)
                        ldsm4t(bq[np][t], ((q_t + so) ^ (np << 5)) + t * (C * DK * 2) + kk * 16 * DK * 2);
                prod<3, KT, DH / 16>(W, au, bq);
            }
            // H^T = dU^T X' for the tokens of this part; X'[j][i] is zero above the diagonal (j < i)
            uint32_t ay[2][3][4];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const uint4 u = reinterpret_cast<const uint4*>(yf)[(kk * 3 + t) * 32 + lane];
                    ay[kk][t][0] = u.x; ay[kk][t][1] = u.y; ay[kk][t][2] = u.z; ay[kk][t][3] = u.w;
                }
#pragma unroll
            for (int e = 0; e < TN; ++e) {
                const int n = part * TN + e;
                float r[4][4] = {};
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int j = 0; j < 3 - i; ++j) {
                        mma16816(r[2 + ((i + j) & 1)], ay[1][i], bx[e][j][2], bx[e][j][3]);
                        if (n < 2) mma16816(r[(i + j) & 1], ay[0][i], bx[e][j][0], bx[e][j][1]);
                    }
                float u[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = (r[0][j] + r[1][j]) + (r[2][j] + r[3][j]);
                const int tok = c * C + 8 * n + 2 * (lane & 3);
                float* to = a.H + (static_cast<long long>(bh) * a.T + tok) * a.dv + own_col;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (!F::SUMMARY && tok + (j & 1) < T) to[(j & 1) * a.dv + 8 * (j >> 1)] = u[j];
                const float f0 = -since[e].x * beta[e].x, f1 = -since[e].y * beta[e].y;
                uint32_t t0[3], t1[3];
                split<3>(u[0] * f0, u[1] * f1, t0);
                split<3>(u[2] * f0, u[3] * f1, t1);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    reinterpret_cast<uint2*>(vf)[((n >> 1) * 3 + t) * 64 + lane * 2 + (n & 1)] = make_uint2(t0[t], t1[t]);
            }
            ptx::named_sync(1 + grp, NH * 32);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t au[3][4], bt[DH / 16][KT][4];
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const uint4 u = reinterpret_cast<const uint4*>(vf)[(kk * 3 + t) * 32 + lane];
                    au[t][0] = u.x; au[t][1] = u.y; au[t][2] = u.z; au[t][3] = u.w;
                }
#pragma unroll
                for (int np = 0; np < DH / 16; ++np)
#pragma unroll
                    for (int t = 0; t < KT; ++t)
                        ldsm4t(bt[np][t], ((k_t + so) ^ (np << 5)) + t * (C * DK * 2) + kk * 16 * DK * 2);
                prod<3, KT, DH / 16>(W, au, bt);
            }
            decay_and_add(S, G->all, W);
            }
            if (++stage == F::NS) stage = 0;
            step_end();
        }
    } else if (chunks > 0 && warp < w_load) {
        // scale (e^c Q)^T dO, transposed: what the outputs of a chunk add to dS, a step before the state
        const int g = warp - w_side;
        const uint32_t q_t = at_rows_first<DK * 2>(sb + F::q, 0, 0, lane);
        int stage = 0;
        for (int s = -F::AHEAD; s < -1; ++s) step_end();
        for (int c = c_end - 1; c >= c_first; --c) {
            const uint32_t so = stage * F::STAGE;
            const Gates* G = reinterpret_cast<const Gates*>(sm + stage * F::STAGE + F::gates);
            float W[DK / 8][4] = {};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t ao[KT][4], au[3][4], bt[DK / 16][KT][4];
                float w[2][4];
#pragma unroll
                for (int t = 0; t < KT; ++t)
                    ldsm4t(ao[t], sb + F::dO + so + t * (C * CS * 2) +
                                      piece<CS * 2>(16 * kk + (lane >> 4) * 8 + (lane & 7), 2 * g + ((lane >> 3) & 1)));
#pragma unroll
                for (int np = 0; np < DK / 16; ++np)
#pragma unroll
                    for (int t = 0; t < KT; ++t)
                        ldsm4t(bt[np][t], ((q_t + so) ^ (np << 5)) + t * (C * DK * 2) + kk * 16 * DK * 2);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 f = *reinterpret_cast<const float2*>(&G->since[16 * kk + 8 * e + 2 * (lane & 3)]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {     // registers 2 e + h: columns + 8 h of tile e
                        float x0 = 0.f, x1 = 0.f;
#pragma unroll
                        for (int t = KT - 1; t >= 0; --t) {
                            x0 += __uint_as_float(ao[t][2 * e + h] << 16);
                            x1 += __uint_as_float(ao[t][2 * e + h] & 0xffff0000u);
                        }
                        w[e][2 * h] = a.scale * f.x * x0;
                        w[e][2 * h + 1] = a.scale * f.y * x1;
                    }
                }
                split_a<3>(w[0], w[1], au);
                prod<3, KT, DK / 16>(W, au, bt);
            }
            float4* sd = reinterpret_cast<float4*>(sm + F::side + (c & 1) * F::SIDE) + g * (DK / 8) * 32 + lane;
#pragma unroll
            for (int n = 0; n < DK / 8; ++n) sd[n * 32] = make_float4(W[n][0], W[n][1], W[n][2], W[n][3]);
            if (++stage == F::NS) stage = 0;
            step_end();
        }
        step_end();
    } else if (chunks > 0) {
        const int lt = (warp - w_load) * 32 + lane;
        constexpr int LT = F::NLD * 32, REC = record_bytes(2);
        const long long ks = static_cast<long long>(kstep) * DK, vs = static_cast<long long>(vstep) * a.dv;
        const E* kp = static_cast<const E*>(a.k) + row_of(a.bthd, b, hk, a.Hk, 0, a.T) * DK;
        const E* qp = static_cast<const E*>(a.q) + row_of(a.bthd, b, hk, a.Hk, 0, a.T) * DK;
        const E* op = static_cast<const E*>(a.dout) + row_of(a.bthd, b, h, a.Hv, 0, a.T) * a.dv + col0;
        const uint8_t* rec = a.records + static_cast<long long>(bh) * all_chunks * REC;
        int stage = 0;
        for (int i = 0; i < chunks + F::AHEAD; ++i) {
            const int c = c_end - 1 - i;
            if (c >= c_first) {
                const uint32_t sg = sb + stage * F::STAGE;
                const int rows = min(C, T - c * C);
                const uint8_t* from = rec + static_cast<long long>(c) * REC + kXBytes;
                load_bytes<kXBytes + F::PB, LT>(sg + F::x, from, lt);      // X' and P lie one behind the other
                load_bytes<512, LT>(sg + F::gates, from + kXBytes + F::PB, lt);
                load_tile<CS, KT, LT>(sg + F::dO, op + static_cast<long long>(c) * C * vs, vs, rows, lt);
                load_tile<DK, KT, LT>(sg + F::k, kp + static_cast<long long>(c) * C * ks, ks, rows, lt);
                load_tile<DK, KT, LT>(sg + F::q, qp + static_cast<long long>(c) * C * ks, ks, rows, lt);
                if (++stage == F::NS) stage = 0;
            }
            cp_commit();
            cp_wait<F::AHEAD - 1 - (F::W_SIDE ? 1 : 0)>();
            step_end();
        }
    }
    float* const to = F::SUMMARY ? a.back + (static_cast<long long>(bh) * a.segments + seg) * DK * a.dv
                                 : (a.dstate_in && seg == 0 ? a.dstate_in + static_cast<long long>(bh) * DK * a.dv : nullptr);
    if (warp < w_side && to) {
#pragma unroll
        for (int n = 0; n < DH / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                to[static_cast<long long>(own_key + 8 * n + (j & 1)) * a.dv + own_col + 8 * (j >> 1)] = S[n][j];
    }
    previous_done();
}

// ------------------------------------------------------------------ gradients of a block
// A block of N tokens (c, D, e^c from the block's first token), S0 before it, dS behind it, two warps
// to 16 tokens, one for the terms of dP = dO U^T and of dS, one for those of dM = -Z U^T (each has
// the pairs of a row and of a column of blocks, five blocks of 16 x 16 in all whatever its tokens):
//     dq  = scale e^c dO S0^T + (scale D dO U^T) K
//     dk  = -e^c Z S0^T + (-D Z U^T) K                                  (as a row of M)
//         + e^(c_N - c) U dS^T + (scale D dO U^T)^T Q + (-D Z U^T)^T K    (as a column)
// A pair (i, j) depends on the decays through e^(c_i - c_j), that is on g of the tokens j < t <= i.
// With x_ij what the pair contributes to the loss's logarithmic derivative, e_i the same of token i
// against S0 and x_j of token j against dS,
//     dg_t = sum_{j < t <= i} x_ij + sum_{i >= t} e_i + sum_{j < t} x_j + e^(c_N) <dS, S0>.
// The first sum is the running sum of (row sum - column sum) of x: both from the same numbers, so
// that what cancels there does so to the last bit (from q.dq - k.dk, the same in theory, dg came out
// ten times less exact).
struct BlockArgs {
    const void *q, *k, *dout;
    const float *g, *beta, *states, *dstates, *R, *H;
    const int* lengths;
    void *dq, *dk, *dv;       // dq, dk: gradients, or with shared heads fp32 [BH][T][d] (PARTIAL)
    float *dg, *dbeta;
    int B, Hk, Hv, T, blocks, bthd;
    float scale;
};

template <typename E, int DK_, int DV_, int N_>
struct Blk {
    using Elem = E;
    static constexpr int DK = DK_, DV = DV_, N = N_, WARPS = N_ / 16, NT = 2 * WARPS * 32;
    static constexpr int KT = sizeof(E) == 2 ? 1 : 3;
    static constexpr int SW = 32;                       // value columns of a state at a time
    static constexpr int KTERM = N * DK * 2, OTERM = N * DV * 2, STERM = DK * SW * 2;
    static constexpr int k = 0, q = k + KT * KTERM, o = q + KT * KTERM, u = o + KT * OTERM, z = u + 3 * OTERM;
    static constexpr int s = z + 3 * OTERM;
    static constexpr int sum = s + 2 * 3 * STERM, since = sum + N * 8, left = since + N * 4, beta = left + N * 4;
    static constexpr int dc = beta + N * 4, xj = dc + 2 * N * 4, cols = xj + N * 4, red = cols + 2 * WARPS * N * 4;
    static constexpr int bytes = red + 32 * 4;
    static_assert(N * DK * 4 <= 2 * 3 * STERM, "a half of dk passes through the slices' place");
    // two blocks an SM where shared memory and 128 registers a thread let them
    static constexpr int BLOCKS = DK <= 64 && bytes <= 113 * 1024 ? 2 : 1;
};

// R rows x D columns of fp32 into three swizzled bf16 terms.
template <int RB, int R, int D, int NT>
__device__ __forceinline__ void load_split(uint32_t tile, uint32_t term, const float* src, long long step, int rows, int tid) {
    constexpr int P = D / 4, U = 4;
#pragma unroll 1
    for (int i0 = tid; i0 < R * P; i0 += NT * U) {
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * NT, r = i / P, c = i % P;
            x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < R * P && r < rows) x[u] = *reinterpret_cast<const float4*>(src + r * step + c * 4);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * NT, r = i / P, c = i % P;
            if (i >= R * P) continue;
            uint32_t lo[3], hi[3];
            split<3>(x[u].x, x[u].y, lo);
            split<3>(x[u].z, x[u].w, hi);
#pragma unroll
            for (int t = 0; t < 3; ++t)
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(tile + t * term + piece<RB>(r, c >> 1) + (c & 1) * 8),
                             "r"(lo[t]), "r"(hi[t]) : "memory");
        }
    }
}

// N rows of E into KT swizzled terms.
template <int N, int D, int KT, int NT>
__device__ __forceinline__ void load_rows(uint32_t tile, const bf16* src, long long step, int rows, int tid) {
    constexpr int P = D / 8;
#pragma unroll 4
    for (int i = tid; i < N * P; i += NT) {
        const int r = i / P, c = i % P;
        const bool on = r < rows;
        cp_async16(tile + piece<D * 2>(r, c), src + (on ? r * step : 0) + c * 8, on);
    }
}
template <int N, int D, int KT, int NT>
__device__ __forceinline__ void load_rows(uint32_t tile, const float* src, long long step, int rows, int tid) {
    load_split<D * 2, N, D, NT>(tile, N * D * 2, src, step, rows, tid);
}

// sum over this lane's columns of acc[row] * tile[row], rows r0 + lane / 4 (+ 8); all four lanes get it
template <int D, int KT>
__device__ __forceinline__ void row_dots(const float (&acc)[D / 8][4], const uint8_t* tile, int term, int r0, int lane,
                                         float (&out)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = r0 + (lane >> 2) + 8 * h;
        float s = 0.f;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            float x0 = 0.f, x1 = 0.f;
#pragma unroll
            for (int t = KT - 1; t >= 0; --t) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + t * term + piece<D * 2>(r, n) + (lane & 3) * 4);
                x0 += __uint_as_float(w << 16);
                x1 += __uint_as_float(w & 0xffff0000u);
            }
            s = fmaf(acc[n][2 * h], x0, s);
            s = fmaf(acc[n][2 * h + 1], x1, s);
        }
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        out[h] = s + __shfl_xor_sync(0xffffffffu, s, 2);
    }
}

// A slice of SW columns of a state, from device memory into registers and from there into shared
// memory as three terms.
template <typename F>
struct Slice {
    static constexpr int P = F::SW / 4, U = F::DK * P / F::NT;
    static_assert(F::DK * P % F::NT == 0, "whole rounds");
    float4 x[U];
    __device__ __forceinline__ void load(const float* state, int tid) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tid + u * F::NT;
            x[u] = *reinterpret_cast<const float4*>(state + (i / P) * F::DV + (i % P) * 4);
        }
    }
    __device__ __forceinline__ void put(uint32_t to, int tid) const {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tid + u * F::NT, r = i / P, c = i % P;
            uint32_t lo[3], hi[3];
            split<3>(x[u].x, x[u].y, lo);
            split<3>(x[u].z, x[u].w, hi);
#pragma unroll
            for (int t = 0; t < 3; ++t)
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to + t * F::STERM + piece<F::SW * 2>(r, c >> 1) + (c & 1) * 8),
                             "r"(lo[t]), "r"(hi[t]) : "memory");
        }
    }
    __device__ __forceinline__ float dot(const Slice& o) const {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
            s += (x[u].x * o.x[u].x + x[u].y * o.x[u].y) + (x[u].z * o.x[u].z + x[u].w * o.x[u].w);
        return s;
    }
};

// acc[16 tokens][DK] += columns c0.. of the rows at `at` (AT terms) x (slice at `st`)^T
template <typename F, int AT>
__device__ __forceinline__ void with_slice(float (&acc)[F::DK / 8][4], uint32_t at, uint32_t st, int c0, int r0, int lane) {
    constexpr int DK = F::DK, DV = F::DV, SW = F::SW;
#pragma unroll
    for (int ks = 0; ks < SW / 16; ++ks) {
        uint32_t x[AT][4];
#pragma unroll
        for (int t = 0; t < AT; ++t) ldsm4(x[t], at_rows_first<DV * 2>(at + t * F::OTERM, r0, c0 / 8 + 2 * ks, lane));
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
            // a fresh sum, its smallest products first: every step cuts at the sum's last bit
            uint32_t y[3][4];
            float w[2][4] = {};
#pragma unroll
            for (int t = 0; t < 3; ++t) ldsm4(y[t], at_pieces_first<SW * 2>(st + t * F::STERM, 16 * np, 2 * ks, lane));
            prod2<AT, 3>(w[0], w[1], x, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[2 * np][j] += w[0][j];
                acc[2 * np + 1][j] += w[1][j];
            }
        }
    }
}

// acc += (f D o (X Y^T)) B over the 16 x 16 blocks of one side of the diagonal: X the rows of this
// warp's tokens, Y and B rows of the whole block.  ROWS: this warp's tokens are i (D_ij counts for
// j <= i, for j < i when STRICT), else they are j.
// With ROWS also x = (f D o (X Y^T)) o (G B^T) for the rows G at `gt`: its row sums onto `rows`
// and its column sums to cols[warp][..].
template <typename F, int AT, int YT, bool ROWS, bool STRICT>
__device__ __forceinline__ void with_pairs(float (&acc)[F::DK / 8][4], uint32_t sb, const float2* sum, int at, int yt, int bt,
                                           float f, int lane, int warp, int gt = 0, float* rows = nullptr, float* cols = nullptr) {
    constexpr int DK = F::DK, DV = F::DV, KT = F::KT;
    const int r0 = warp * 16;
    const float2 own[2] = {sum[r0 + (lane >> 2)], sum[r0 + 8 + (lane >> 2)]};
#pragma unroll 1
    for (int jb = ROWS ? 0 : warp; jb <= (ROWS ? warp : F::WARPS - 1); ++jb) {
        float w[2][4] = {}, low[2][4] = {};
#pragma unroll 2
        for (int ks = 0; ks < DV / 16; ++ks) {
            uint32_t x[AT][4], y[YT][4];
#pragma unroll
            for (int t = 0; t < AT; ++t) ldsm4(x[t], at_rows_first<DV * 2>(sb + at + t * F::OTERM, r0, 2 * ks, lane));
#pragma unroll
            for (int t = 0; t < YT; ++t) ldsm4(y[t], at_pieces_first<DV * 2>(sb + yt + t * F::OTERM, 16 * jb, 2 * ks, lane));
            prod2<AT, YT>(w[0], w[1], low[0], low[1], x, y);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) w[0][j] += low[0][j], w[1][j] += low[1][j];
        const bool diagonal = jb == warp;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const float4 his = *reinterpret_cast<const float4*>(&sum[16 * jb + 8 * n + 2 * (lane & 3)]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 other = (j & 1) ? make_float2(his.z, his.w) : make_float2(his.x, his.y);
                const float gap = (own[j >> 1].x - other.x) + (own[j >> 1].y - other.y);
                w[n][j] *= f * ex2(ROWS ? gap : -gap);
                // this lane's row and column within the block: off the diagonal block all count
                const int lead = (lane >> 2) + 8 * (j >> 1) - (8 * n + 2 * (lane & 3) + (j & 1));
                if (diagonal && !(ROWS ? (STRICT ? lead > 0 : lead >= 0) : (STRICT ? lead < 0 : lead <= 0))) w[n][j] = 0.f;
            }
        }
        if constexpr (ROWS) {
            float g[2][4] = {}, glow[2][4] = {};
#pragma unroll 2
            for (int ks = 0; ks < DK / 16; ++ks) {
                uint32_t x[KT][4], y[KT][4];
#pragma unroll
                for (int t = 0; t < KT; ++t) ldsm4(x[t], at_rows_first<DK * 2>(sb + gt + t * F::KTERM, r0, 2 * ks, lane));
#pragma unroll
                for (int t = 0; t < KT; ++t) ldsm4(y[t], at_pieces_first<DK * 2>(sb + bt + t * F::KTERM, 16 * jb, 2 * ks, lane));
                if constexpr (KT == 1) prod2<KT, KT>(g[0], g[1], x, y);
                else prod2<KT, KT>(g[0], g[1], glow[0], glow[1], x, y);
            }
            if constexpr (KT > 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j) g[0][j] += glow[0][j], g[1][j] += glow[1][j];
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    g[n][j] *= w[n][j];
                    rows[j >> 1] += g[n][j];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float c = g[n][e] + g[n][2 + e];
#pragma unroll
                    for (int m = 4; m < 32; m <<= 1) c += __shfl_xor_sync(0xffffffffu, c, m);
                    float* to = cols + warp * F::N + 16 * jb + 8 * n + 2 * lane + e;
                    if (lane < 4) *to = c;
                }
            }
        }
        uint32_t x[3][4];
        split_a<3>(w[0], w[1], x);
#pragma unroll
        for (int np = 0; np < DK / 16; ++np) {
            uint32_t y[KT][4];
#pragma unroll
            for (int t = 0; t < KT; ++t) ldsm4t(y[t], at_rows_first<DK * 2>(sb + bt + t * F::KTERM, 16 * jb, 2 * np, lane));
            float v[2][4] = {};
            prod2<3, KT>(v[0], v[1], x, y);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[2 * np][j] += v[0][j];
                acc[2 * np + 1][j] += v[1][j];
            }
        }
    }
}

template <int NT_>
__device__ __forceinline__ void clear(float (&acc)[NT_][4]) {
#pragma unroll
    for (int n = 0; n < NT_; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
}
// acc[row] *= f of[row], rows r0 + lane / 4 (+ 8)
template <int NT_>
__device__ __forceinline__ void by_row(float (&acc)[NT_][4], const float* of, float f, int r0, int lane) {
    const float x = f * of[r0 + (lane >> 2)], y = f * of[r0 + 8 + (lane >> 2)];
#pragma unroll
    for (int n = 0; n < NT_; ++n) {
        acc[n][0] *= x; acc[n][1] *= x; acc[n][2] *= y; acc[n][3] *= y;
    }
}
// rows r0 + lane / 4 (+ 8) of acc to rows of `to` (`step` elements apart); zeros from `rows` on
template <typename O, int NT_>
__device__ __forceinline__ void write_rows(const float (&acc)[NT_][4], O* to, long long step, int r0, int rows, int out_rows, int lane) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = r0 + (lane >> 2) + 8 * e;
        if (r >= out_rows) continue;
#pragma unroll
        for (int n = 0; n < NT_; ++n) {
            const float x0 = r < rows ? acc[n][2 * e] : 0.f, x1 = r < rows ? acc[n][2 * e + 1] : 0.f;
            O* at = to + r * step + 8 * n + 2 * (lane & 3);
            if constexpr (sizeof(O) == 2) *reinterpret_cast<uint32_t*>(at) = ptx::pack_bf16(x0, x1);
            else *reinterpret_cast<float2*>(at) = make_float2(x0, x1);
        }
    }
}

template <typename F, bool PARTIAL>
__global__ void __launch_bounds__(F::NT, F::BLOCKS) k_delta_block_grads(const BlockArgs a) {
    using E = typename F::Elem;
    constexpr int DK = F::DK, DV = F::DV, N = F::N, KT = F::KT, NT = F::NT, SW = F::SW;
    extern __shared__ __align__(1024) uint8_t sm[];
    const uint32_t sb = ptx::smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, tile = warp % F::WARPS, r0 = 16 * tile;
    const bool of_m = warp >= F::WARPS;
    const int bh = blockIdx.x / a.blocks, blk = blockIdx.x % a.blocks;
    const int b = bh / a.Hv, h = bh % a.Hv, hk = h / (a.Hv / a.Hk);
    const int t0 = blk * N, T = length_of(a.lengths, b, a.T);
    const int rows = max(0, min(N, T - t0)), out_rows = min(N, a.T - t0);
    const int kstep = row_step(a.bthd, a.Hk), vstep = row_step(a.bthd, a.Hv);
    const long long kr = row_of(a.bthd, b, hk, a.Hk, t0, a.T), vr = row_of(a.bthd, b, h, a.Hv, t0, a.T);
    float2* sum = reinterpret_cast<float2*>(sm + F::sum);
    float* since = reinterpret_cast<float*>(sm + F::since);
    float* left = reinterpret_cast<float*>(sm + F::left);
    float* beta = reinterpret_cast<float*>(sm + F::beta);
    float* dc = reinterpret_cast<float*>(sm + F::dc);
    float* xj = reinterpret_cast<float*>(sm + F::xj);
    float* cols = reinterpret_cast<float*>(sm + F::cols);
    float* red = reinterpret_cast<float*>(sm + F::red);
    const float* R = a.R + (static_cast<long long>(bh) * a.T + t0) * DV;
    const float* H = a.H + (static_cast<long long>(bh) * a.T + t0) * DV;
    const float* S0 = a.states + (static_cast<long long>(bh) * a.blocks + blk) * DK * DV;
    const float* dS = a.dstates + (static_cast<long long>(bh) * a.blocks + blk) * DK * DV;

    if (rows > 0) {
        load_rows<N, DK, KT, NT>(sb + F::k, static_cast<const E*>(a.k) + kr * DK, static_cast<long long>(kstep) * DK, rows, tid);
        load_rows<N, DK, KT, NT>(sb + F::q, static_cast<const E*>(a.q) + kr * DK, static_cast<long long>(kstep) * DK, rows, tid);
        load_rows<N, DV, KT, NT>(sb + F::o, static_cast<const E*>(a.dout) + vr * DV, static_cast<long long>(vstep) * DV, rows, tid);
        cp_commit();
    }
    if (warp == 0) {
        double c = 0.0, last = 0.0, keep[N / 32];
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {
            const int r = 32 * i + lane;
            const bool on = r < rows;
            beta[r] = on ? a.beta[vr + static_cast<long long>(r) * vstep] : 0.f;
            c = on ? static_cast<double>(gate(a.g[vr + static_cast<long long>(r) * vstep])) * 1.4426950408889634 : 0.0;
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const double x = __shfl_up_sync(0xffffffffu, c, w);
                if (lane >= w) c += x;
            }
            c += last;
            last = __shfl_sync(0xffffffffu, c, 31);
            keep[i] = c;
        }
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {
            const int r = 32 * i + lane;
            const float hi = static_cast<float>(keep[i]);
            sum[r] = make_float2(hi, static_cast<float>(keep[i] - static_cast<double>(hi)));
            since[r] = ex2_long(keep[i]);
            left[r] = ex2_long(last - keep[i]);
        }
    }
    __syncthreads();
    if (rows <= 0) {
        for (int i = tid; i < out_rows * DK; i += NT) {
            const int r = i / DK, c = i % DK;
            if (PARTIAL) {
                const long long at = (static_cast<long long>(bh) * a.T + t0 + r) * DK + c;
                static_cast<float*>(a.dq)[at] = 0.f;
                static_cast<float*>(a.dk)[at] = 0.f;
            } else {
                const long long at = (kr + static_cast<long long>(r) * kstep) * DK + c;
                store_elem(static_cast<E*>(a.dq) + at, 0.f);
                store_elem(static_cast<E*>(a.dk) + at, 0.f);
            }
        }
        for (int i = tid; i < out_rows * DV; i += NT)
            store_elem(static_cast<E*>(a.dv) + (vr + static_cast<long long>(i / DV) * vstep) * DV + i % DV, 0.f);
        for (int r = tid; r < out_rows; r += NT) {
            a.dg[vr + static_cast<long long>(r) * vstep] = 0.f;
            a.dbeta[vr + static_cast<long long>(r) * vstep] = 0.f;
        }
        return;
    }
    Slice<F> s0, ds;
    s0.load(S0, tid);
    ds.load(dS, tid);
    // U = beta R and Z = beta H for the products, dv = Z, dbeta = R . H (DV / 4 lanes a row)
    {
        constexpr int P = DV / 4, U = N * P / NT < 4 ? N * P / NT : 4;
        static_assert(N * P % (NT * U) == 0, "whole rounds");
#pragma unroll 1
        for (int i0 = tid; i0 < N * P; i0 += NT * U) {
            float4 x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * NT, r = i / P;
                x[u] = y[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < rows) {
                    x[u] = *reinterpret_cast<const float4*>(R + i * 4);
                    y[u] = *reinterpret_cast<const float4*>(H + i * 4);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * NT, r = i / P, c = i % P;
                const float w = beta[r];
                float dot = (x[u].x * y[u].x + x[u].y * y[u].y) + (x[u].z * y[u].z + x[u].w * y[u].w);
#pragma unroll
                for (int m = 1; m < P; m <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
                const float z[4] = {w * y[u].x, w * y[u].y, w * y[u].z, w * y[u].w};
                if (r < out_rows) {
                    store4(static_cast<E*>(a.dv) + (vr + static_cast<long long>(r) * vstep) * DV + c * 4, z);
                    if (c == 0) a.dbeta[vr + static_cast<long long>(r) * vstep] = dot;
                }
                const uint32_t at = piece<DV * 2>(r, c >> 1) + (c & 1) * 8;
                uint32_t lo[3], hi[3];
                split<3>(z[0], z[1], lo);
                split<3>(z[2], z[3], hi);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(sb + F::z + t * F::OTERM + at), "r"(lo[t]), "r"(hi[t]) : "memory");
                split<3>(w * x[u].x, w * x[u].y, lo);
                split<3>(w * x[u].z, w * x[u].w, hi);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(sb + F::u + t * F::OTERM + at), "r"(lo[t]), "r"(hi[t]) : "memory");
            }
        }
    }
    cp_wait<0>();

    // where dq and dk go: the gradients, or this value head's share of them
    using O = std::conditional_t<PARTIAL, float, E>;
    const long long out_at = (PARTIAL ? static_cast<long long>(bh) * a.T + t0 : kr) * DK;
    const long long out_step = static_cast<long long>(PARTIAL ? 1 : kstep) * DK;
    O* const dq = static_cast<O*>(a.dq) + out_at;
    O* const dk = static_cast<O*>(a.dk) + out_at;
    float acc[DK / 8][4], acc_q[DK / 8][4];          // a part of dk; dq
    float cross = 0.f;
    clear(acc);
    clear(acc_q);
    const uint32_t st0 = sb + F::s, st1 = st0 + 3 * F::STERM;
#pragma unroll 1
    for (int n = 0; n < DV / SW; ++n) {
        s0.put(st0, tid);
        ds.put(st1, tid);
        cross += ds.dot(s0);
        __syncthreads();
        if (n + 1 < DV / SW) {                     // the next slices are on their way meanwhile
            s0.load(S0 + (n + 1) * SW, tid);
            ds.load(dS + (n + 1) * SW, tid);
        }
        if (of_m) {
            with_slice<F, 3>(acc, sb + F::z, st0, n * SW, r0, lane);
        } else {
            with_slice<F, KT>(acc_q, sb + F::o, st0, n * SW, r0, lane);
            with_slice<F, 3>(acc, sb + F::u, st1, n * SW, r0, lane);
        }
        __syncthreads();
    }
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) cross += __shfl_xor_sync(0xffffffffu, cross, w);
    if (lane == 0) red[warp] = cross;
    float4* const pass = reinterpret_cast<float4*>(sm + F::s) + tile * (DK / 8) * 32 + lane;
    float state_part[2], pairs[2] = {};
    if (of_m) {
        by_row(acc, since, -1.f, r0, lane);
        row_dots<DK, KT>(acc, sm + F::k, F::KTERM, r0, lane, state_part);
        with_pairs<F, 3, 3, true, true>(acc, sb, sum, F::z, F::u, F::k, -1.f, lane, tile, F::k, pairs, cols + F::WARPS * N);
        with_pairs<F, 3, 3, false, true>(acc, sb, sum, F::u, F::z, F::k, -1.f, lane, tile);
#pragma unroll
        for (int n = 0; n < DK / 8; ++n) pass[n * 32] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
    } else {
        by_row(acc_q, since, a.scale, r0, lane);
        row_dots<DK, KT>(acc_q, sm + F::q, F::KTERM, r0, lane, state_part);
        with_pairs<F, KT, 3, true, false>(acc_q, sb, sum, F::o, F::u, F::k, a.scale, lane, tile, F::q, pairs, cols);
        write_rows(acc_q, dq, out_step, r0, rows, out_rows, lane);
        float xs[2];
        by_row(acc, left, 1.f, r0, lane);
        row_dots<DK, KT>(acc, sm + F::k, F::KTERM, r0, lane, xs);
        with_pairs<F, 3, KT, false, false>(acc, sb, sum, F::u, F::o, F::q, a.scale, lane, tile);
        if ((lane & 3) == 0) {
#pragma unroll
            for (int e = 0; e < 2; ++e) xj[r0 + (lane >> 2) + 8 * e] = xs[e];
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        pairs[e] += __shfl_xor_sync(0xffffffffu, pairs[e], 1);
        pairs[e] += __shfl_xor_sync(0xffffffffu, pairs[e], 2);
        if ((lane & 3) == 0) dc[(of_m ? N : 0) + r0 + (lane >> 2) + 8 * e] = pairs[e] + state_part[e];
    }
    __syncthreads();
    if (!of_m) {
#pragma unroll
        for (int n = 0; n < DK / 8; ++n) {
            const float4 x = pass[n * 32];
            acc[n][0] += x.x; acc[n][1] += x.y; acc[n][2] += x.z; acc[n][3] += x.w;
        }
        write_rows(acc, dk, out_step, r0, rows, out_rows, lane);
    }
    if (warp == F::WARPS) {
        float cross_all = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * F::WARPS; ++i) cross_all += red[i];
        float tail = 0.f, head = since[N - 1] * cross_all, above[N / 32];
#pragma unroll
        for (int i = 0; i < N / 32; ++i) {                 // sums over j < t
            const int r = 32 * i + lane;
            float x = xj[r];
            const float own = x;
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, x, w);
                if (lane >= w) x += y;
            }
            above[i] = head + (x - own);
            head += __shfl_sync(0xffffffffu, x, 31);
        }
#pragma unroll
        for (int i = N / 32 - 1; i >= 0; --i) {            // sums over i >= t
            const int r = 32 * i + lane;
            float x = dc[r] + dc[N + r];
#pragma unroll
            for (int w = 0; w < F::WARPS; ++w)
                if (w >= r / 16) x -= cols[w * N + r] + cols[(F::WARPS + w) * N + r];
#pragma unroll
            for (int w = 1; w < 32; w <<= 1) {
                const float y = __shfl_down_sync(0xffffffffu, x, w);
                if (lane + w < 32) x += y;
            }
            x += tail;
            tail = __shfl_sync(0xffffffffu, x, 0);
            if (r < out_rows) a.dg[vr + static_cast<long long>(r) * vstep] = r < rows ? x + above[i] : 0.f;
        }
    }
}

// Shared heads: dq, dk of a key head are the sums over its value heads, in their order.
template <typename E>
__global__ void __launch_bounds__(256) k_delta_share(const float* dq, const float* dk, E* oq, E* ok, int B, int Hk, int share,
                                                     int T, int d, int bthd) {
    const long long per = static_cast<long long>(T) * d / 4, n = static_cast<long long>(B) * Hk * per;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<long long>(gridDim.x) * 256) {
        const long long bhk = i / per, at = (i % per) * 4;
        const int b = static_cast<int>(bhk / Hk), hk = static_cast<int>(bhk % Hk);
        const int t = static_cast<int>(at / d), c = static_cast<int>(at % d);
        float x[4] = {}, y[4] = {};
        for (int s = 0; s < share; ++s) {
            const long long from = ((static_cast<long long>(b) * Hk + hk) * share + s) * T * d + at;
            float u[4], w[4];
            load4(dq + from, u);
            load4(dk + from, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] += u[j], y[j] += w[j];
        }
        const long long to = row_of(bthd, b, hk, Hk, t, T) * d + c;
        store4(oq + to, x);
        store4(ok + to, y);
    }
}

// ------------------------------------------------------------------ host
// Tokens of a block: 64, or 32 where the fp32 tiles of 64 do not fit.
int block_tokens(const Problem& p) { return !p.bf16 && (p.d == 128 || p.dv == 128) ? 32 : 64; }

struct Space {   // the workspace's pieces, bytes from its start
    size_t records, states, dstates, R, H, dq, dk, sums, starts, back, behind, end;
};
Space space(const Problem& p) {
    const size_t BH = static_cast<size_t>(p.B) * p.H, blocks = (p.T + block_tokens(p) - 1) / block_tokens(p);
    const size_t state = BH * blocks * p.d * p.dv * 4, rows = BH * p.T * p.dv * 4;
    const size_t part = p.H != p.Hk ? BH * p.T * p.d * 4 : 0;
    Space s;
    s.records = 0;
    s.states = s.records + records_bytes(p, true);
    s.dstates = s.states + state;
    s.R = s.dstates + state;
    s.H = s.R + rows;
    s.dq = s.H + rows;
    s.dk = s.dq + part;
    const Segments g = segments(p, true);
    s.sums = s.dk + part;
    s.starts = s.sums + g.sums * 4;
    s.back = s.starts + g.starts * 4;
    s.behind = s.back + g.starts * 4;
    s.end = s.behind + g.starts * 4;
    return s;
}

template <typename F>
cudaError_t start(const ReverseArgs& a, bool beside, int blocks, cudaStream_t st) {
    static_assert(F::bytes <= 227 * 1024, "shared memory of a block");
    const cudaError_t e = allow_smem<k_delta_reverse<F>>(F::bytes);
    if (e != cudaSuccess) return e;
    if (beside) return launch_beside(k_delta_reverse<F>, blocks, F::WARPS * 32, F::bytes, st, a);
    k_delta_reverse<F><<<blocks, F::WARPS * 32, F::bytes, st>>>(a);
    return cudaGetLastError();
}

// The two walks.  Neither needs the other, so the reverse walk mostly runs beside the forward one, and so do
// their summaries and folds where there are segments (the linear part of a segment backwards is the
// transpose of the forward walk's A).  All gradients, side by side and one after the
// other: bf16 4x16x4096x64 588 and 679 us, fp32 2x8x4096x32 (in segments) 168 and 205, 2x16x512x32 50 and 68.
template <typename E, int DK>
cudaError_t walks(const Problem& p, const Gradients& gr, char* ws, const Space& s, cudaStream_t st) {
    constexpr int NG = sizeof(E) == 2 ? 2 : 1;
    const Segments g = segments(p, true);
    const int slices = p.dv / (16 * NG), BH = p.B * p.H;
    const uint8_t* records = reinterpret_cast<uint8_t*>(ws + s.records);
    const float* first = p.state_in;
    float* back = reinterpret_cast<float*>(ws + s.back);
    float* behind = reinterpret_cast<float*>(ws + s.behind);
    ReverseArgs a{p.q, p.k, gr.dout, reinterpret_cast<uint8_t*>(ws + s.records), gr.dstate_out, p.lengths, gr.dstate_in,
                  reinterpret_cast<float*>(ws + s.dstates), reinterpret_cast<float*>(ws + s.H), back,
                  p.Hk, p.H, p.T, p.dv, p.bthd ? 1 : 0, block_tokens(p) / C, g.count, g.chunks, p.scale};
    cudaError_t e = cudaSuccess;
    if (g.count > 1) {
        float* sums = reinterpret_cast<float*>(ws + s.sums);
        float* starts = reinterpret_cast<float*>(ws + s.starts);
        e = summarize(p, g, records, sums, st);
        if (e == cudaSuccess) e = start<Rev<E, DK, NG, true>>(a, true, BH * (g.count - 1) * slices, st);
        if (e == cudaSuccess) e = fold(p, g, sums, nullptr, p.state_in, starts, st);
        if (e == cudaSuccess) e = fold(p, g, sums, back, gr.dstate_out, behind, st);
        a.behind = behind;
        first = starts;
    }
    if (e == cudaSuccess)
        e = store_states(p, g, records, first, reinterpret_cast<float*>(ws + s.states), reinterpret_cast<float*>(ws + s.R),
                         block_tokens(p) / C, st);
    if (e != cudaSuccess) return e;
    if constexpr (sizeof(E) == 2 && DK <= 64)
        if (gradient_columns(p, static_cast<long long>(p.B) * p.H * g.count) == 64) return start<Rev<E, DK, 4, false>>(a, true, BH * g.count * (p.dv / 64), st);
    const int blocks = BH * g.count * slices;
    return start<Rev<E, DK, NG, false>>(a, gradient_walks_beside(p, blocks), blocks, st);
}

template <typename E, int DK, int DV>
cudaError_t block_grads(const Problem& p, const Gradients& gr, char* ws, const Space& s, cudaStream_t st) {
    constexpr int N = sizeof(E) == 4 && (DK == 128 || DV == 128) ? 32 : 64;
    using F = Blk<E, DK, DV, N>;
    static_assert(F::bytes <= 227 * 1024, "shared memory of a block");
    const bool shared = p.H != p.Hk;
    const int blocks = (p.T + N - 1) / N;
    const BlockArgs a{p.q, p.k, gr.dout, p.g, p.beta, reinterpret_cast<float*>(ws + s.states),
                      reinterpret_cast<float*>(ws + s.dstates), reinterpret_cast<float*>(ws + s.R),
                      reinterpret_cast<float*>(ws + s.H), p.lengths, shared ? ws + s.dq : gr.dq, shared ? ws + s.dk : gr.dk,
                      gr.dv, gr.dg, gr.dbeta, p.B, p.Hk, p.H, p.T, blocks, p.bthd ? 1 : 0, p.scale};
    const cudaError_t e = shared ? allow_smem<k_delta_block_grads<F, true>>(F::bytes) : allow_smem<k_delta_block_grads<F, false>>(F::bytes);
    if (e != cudaSuccess) return e;
    if (shared) k_delta_block_grads<F, true><<<p.B * p.H * blocks, F::NT, F::bytes, st>>>(a);
    else k_delta_block_grads<F, false><<<p.B * p.H * blocks, F::NT, F::bytes, st>>>(a);
    return cudaGetLastError();
}

template <typename E, int DK>
cudaError_t all(const Problem& p, const Gradients& gr, char* ws, cudaStream_t st) {
    const Space s = space(p);
    uint8_t* records = reinterpret_cast<uint8_t*>(ws + s.records);
    cudaError_t e = prepare(p, true, records, st);
    if (e == cudaSuccess) e = walks<E, DK>(p, gr, ws, s, st);
    if (e == cudaSuccess) {
        if (p.dv == 32) e = block_grads<E, DK, 32>(p, gr, ws, s, st);
        else if (p.dv == 64) e = block_grads<E, DK, 64>(p, gr, ws, s, st);
        else e = block_grads<E, DK, 128>(p, gr, ws, s, st);
    }
    if (e == cudaSuccess && p.H != p.Hk) {
        const long long n = static_cast<long long>(p.B) * p.Hk * p.T * p.d / 4;
        const long long want = (n + 255) / 256;
        k_delta_share<E><<<static_cast<unsigned>(want < 148 * 16 ? want : 148 * 16), 256, 0, st>>>(
            reinterpret_cast<float*>(ws + s.dq), reinterpret_cast<float*>(ws + s.dk), static_cast<E*>(gr.dq),
            static_cast<E*>(gr.dk), p.B, p.Hk, p.H / p.Hk, p.T, p.d, p.bthd ? 1 : 0);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace

size_t backward_bytes(const Problem& p) { return space(p).end; }
int backward_launches(const Problem& p) { return (p.H != p.Hk ? 5 : 4) + (segments(p, true).count > 1 ? 4 : 0); }

cudaError_t backward(const Problem& p, const Gradients& gr, void* ws, cudaStream_t st) {
    char* w = static_cast<char*>(ws);
    if (p.bf16) {
        if (p.d == 32) return all<bf16, 32>(p, gr, w, st);
        if (p.d == 64) return all<bf16, 64>(p, gr, w, st);
        return all<bf16, 128>(p, gr, w, st);
    }
    if (p.d == 32) return all<float, 32>(p, gr, w, st);
    if (p.d == 64) return all<float, 64>(p, gr, w, st);
    return all<float, 128>(p, gr, w, st);
}

}  // namespace delta
}  // namespace hla
