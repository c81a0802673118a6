// The gated delta rule over a sequence: the forward walk.
//
// Within a chunk of C tokens from the carried state S0, with c the running sum of the log decays,
// D_ij = e^(c_i - c_j), M = strict_low(D o K K^T), P = scale low(D o Q K^T):
//     R = (I + M diag(beta))^-1 (V - diag(e^c) K S0)      (each token's error v - S^T k)
//     U = diag(beta) R
//     O = scale diag(e^c) Q S0 + P U
//     S = e^(c_C) S0 + K^T diag(e^(c_C - c)) U
// A block owns CS = 16 NG value columns of one head (S's columns do not mix).  NH warps hold the
// state of 16 columns transposed in registers, each a part of the key axis; between the products
// they share the chunk's Y and U, each splitting the tokens of its part once, through shared memory.
//
// One head's chunks follow one another, so few long heads leave most of the machine idle.  Then the
// sequence is cut into segments (delta_fold.cu): a first walk takes each segment from a zero state and
// also takes the unit matrix through it without values, which gives S_end = A S_start + B; the states
// between the segments follow from those, and the second walk has all segments at once.
#include "delta_walk.cuh"

namespace hla {
namespace delta {
namespace {

enum Mode { OUT = 0, SUMMARY = 1, STORE = 2 };

struct WalkArgs {
    const void *q, *k, *v;
    const uint8_t* records;   // [BH][chunks][record], see delta_walk.cuh
    const float* start;       // states before each segment [BH][segments][d][dv], or one per head, or null
    const int* lengths;
    void* o;
    float* state_out;         // after the last segment, or null
    float* sums;              // SUMMARY: [BH][segments - 1][d][dv + d]
    float* states;            // STORE: [BH][blocks][d][dv], the state before each block of block_chunks chunks
    float* errors;            // STORE: [BH][T][dv], R
    int block_chunks;
    int Hk, H, T, dv, bthd;
    int segments, seg_chunks; // chunks of a segment
    float scale;
};

// GR: the records have the gradients' form.
template <typename E, int DK_, int NG_, Mode MODE_, bool GR>
struct Cfg {
    using Elem = E;
    static constexpr int DK = DK_, CS = 16 * NG_;
    static constexpr Mode MODE = MODE_;
    static constexpr bool BF = sizeof(E) == 2;
    static constexpr int KT = BF ? 1 : 3;             // terms of q, k
    // terms of S0, U and P in the outputs: fp32's 24 bits for either type, since an output may be far
    // smaller than its terms (with two, 16 bits, 4x16x4096x64 bf16 took 184 us, not 194, and 2x16x4096x128
    // 230, not 265)
    static constexpr int OT = 3;
    static constexpr int INV = GR ? 2 : 1;
    static constexpr int AHEAD = BF ? 2 : 1;          // chunks between a tile's request and its use
    static constexpr int NLD = BF ? 2 : 4;            // loader warps (fp32 tiles are split on the way)
    // state warps of 16 columns: one holds 64 keys' part of the state and the chunk's terms in its
    // registers (bf16: 4x16x4096x64 the same with one and two, with half the warps); twice the keys, or
    // the six products of fp32 terms, are worth the exchanges (2x16x4096x128: four are 3% slower than two)
    static constexpr int NH = DK_ == 128 || (!BF && DK_ == 64) ? 2 : 1;
    static constexpr int W_STATE = NH * NG_, W_OUT = MODE_ == OUT ? NG_ : 0;
    static constexpr int WARPS = W_STATE + W_OUT + NLD;
    static constexpr int KTILE = KT * C * DK_ * 2;
    // ring of AHEAD + 1 stages: keys, inverse, values
    static constexpr int NS = AHEAD + 1;
    static constexpr int k = 0, x = k + KTILE, v = x + kXBytes;
    static constexpr int STAGE = (v + cols_bytes<E, CS>() + 255) / 256 * 256;
    // ring of AHEAD + 2: gates, which the outputs need a chunk behind the state
    static constexpr int NG_STAGES = AHEAD + 2;
    static constexpr int gates = NS * STAGE;
    // ring of AHEAD + 1: for the outputs, queries and P, asked for a chunk behind the rest
    static constexpr int behind = gates + NG_STAGES * 512;
    static constexpr int q = 0, p = q + KTILE;
    static constexpr int OSTAGE = MODE_ == OUT ? p + kXBytes : 0;
    // S0 and U of the last two chunks for the outputs (fp32: the output warps, which have the time, split
    // them), the partial sums
    static constexpr int sf = behind + NS * OSTAGE;
    static constexpr int SB = NG_ * (DK_ / 8) * 512;
    static constexpr int uf = sf + (MODE_ == OUT ? 2 * SB : 0);
    static constexpr int UB = NG_ * 4 * 512;
    static constexpr int ex = uf + (MODE_ == OUT ? 2 * UB : 0);
    static constexpr int yf = ex + (NH > 1 ? W_STATE * 2048 : 0);    // Y of the chunk as an A operand; the decayed U
    static constexpr int YB = 2 * 3 * 512;            // takes the partial sums' place
    static constexpr int bytes = yf + (NH > 1 ? NG_ * YB : 0);
    // of an SM; summaries of narrow bf16 heads are four warps and 38 kB, so that 128 registers a thread let
    // four share one (1x4x16384x64: 110 us, with three 126)
    static constexpr int BLOCKS = MODE_ == SUMMARY && BF && DK_ <= 64 ? 4 : bytes <= 113 * 1024 ? 2 : 1;
};

// Two neighbouring tiles of S0 or U, transposed as the state warps hold them, as a B operand.
template <int N>
__device__ __forceinline__ void operand(const float (&x)[4], const float (&y)[4], uint32_t (&b)[N][4]) {
    uint32_t a[N][4];
    split_a<N>(x, y, a);
#pragma unroll
    for (int t = 0; t < N; ++t) {
        b[t][0] = a[t][0]; b[t][1] = a[t][2]; b[t][2] = a[t][1]; b[t][3] = a[t][3];
    }
}

template <typename F>
__global__ void __launch_bounds__(F::WARPS * 32, F::BLOCKS) k_delta_walk(const WalkArgs a) {
    using E = typename F::Elem;
    constexpr int DK = F::DK, NH = F::NH, DH = DK / NH, TN = 4 / (NH == 1 ? 2 : NH), CS = F::CS, KT = F::KT, OT = F::OT;
    constexpr Mode MODE = F::MODE;
    extern __shared__ __align__(1024) uint8_t sm[];   // swizzles are exclusive ors of address bits
    const uint32_t sb = ptx::smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // block -> (head, segment, columns)
    const int vslices = a.dv / CS;
    const int slices = MODE == SUMMARY ? vslices + DK / CS : vslices;
    const int walked = MODE == SUMMARY ? a.segments - 1 : a.segments;
    const int slice = blockIdx.x % slices, seg = (blockIdx.x / slices) % walked, bh = blockIdx.x / slices / walked;
    if (MODE != OUT) next_may_start();                          // the reverse walk of the same kind, if there is one
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
    constexpr int w_out = F::W_STATE, w_load = w_out + F::W_OUT;
    const int grp = warp / NH, part = warp % NH;                // state warps
    float S[DH / 8][4];
    if (warp < F::W_STATE) {
        // S^T: this lane's columns col, col + 8, keys 8 n + 2 (lane % 4), + 1 of its half
        const int col = col0 + 16 * grp + (lane >> 2), key = part * DH + 2 * (lane & 3);
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
    // Step s: tiles of chunk s + AHEAD asked for, state over chunk s, outputs of chunk s - 1; one
    // barrier of the whole block a step, each role in a loop of its own.
    constexpr int ALL = F::WARPS * 32;
    const auto step_end = [] { ptx::named_sync(15, ALL); };
    if (chunks > 0 && warp < F::W_STATE) {
        // ---------------------------------------------------- state
        // this lane's places in a stage's keys and inverse
        const uint32_t k_n = at_pieces_first<DK * 2>(sb + F::k, 0, part * (DH / 8), lane);
        const uint32_t k_t = at_rows_first<DK * 2>(sb + F::k, 0, part * (DH / 8), lane);
        float4* const ex = reinterpret_cast<float4*>(sm + F::ex) + grp * NH * 128 + lane;
        uint8_t* const yf = sm + F::yf + grp * F::YB;
        uint8_t* const vf = reinterpret_cast<uint8_t*>(ex - lane);
        int stage = 0, gstage = 0;
        for (int s = -F::AHEAD; s < 0; ++s) step_end();
        for (int c = 0; c < chunks; ++c) {
            const uint32_t so = stage * F::STAGE;
            const Gates* G = reinterpret_cast<const Gates*>(sm + F::gates + gstage * 512);
            float4* const sf = reinterpret_cast<float4*>(sm + F::sf + (c & 1) * F::SB) + (grp * (DK / 8) + part * (DH / 8)) * 32 + lane;
            float4* const uf = reinterpret_cast<float4*>(sm + F::uf + (c & 1) * F::UB) + grp * 4 * 32 + lane;
            if (MODE == OUT) {
#pragma unroll
                for (int n = 0; n < DH / 8; ++n) sf[n * 32] = make_float4(S[n][0], S[n][1], S[n][2], S[n][3]);
            }
            if (MODE == STORE) {
                const int chunk = t_first / C + c;
                if (chunk % a.block_chunks == 0) {
                    const int blocks = ((a.T + C - 1) / C + a.block_chunks - 1) / a.block_chunks;
                    float* to = a.states + (static_cast<long long>(bh) * blocks + chunk / a.block_chunks) * DK * a.dv +
                                static_cast<long long>(part * DH + 2 * (lane & 3)) * a.dv + col0 + 16 * grp + (lane >> 2);
#pragma unroll
                    for (int n = 0; n < DH / 8; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) to[static_cast<long long>(8 * n + (j & 1)) * a.dv + 8 * (j >> 1)] = S[n][j];
                }
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
                        for (int t = 0; t < KT; ++t)   // a step of 16 keys changes the piece by two: its swizzle is an exclusive or
                            ldsm4(bk[np][t], ((k_n + so) ^ (ks << 5)) + t * (C * DK * 2) + np * 16 * DK * 2);
                    split_a<3>(S[2 * ks], S[2 * ks + 1], as);
                    prod<3, KT, 2>(y, as, bk);
                }
                // Y^T = V^T - (S0^T K^T) e^c
                float v[4][4] = {};
                if (!unit) {
                    cols_t<CS>(static_cast<const E*>(nullptr), sb + F::v + so, 16 * grp, 0, lane, v[0], v[1]);
                    cols_t<CS>(static_cast<const E*>(nullptr), sb + F::v + so, 16 * grp, 16, lane, v[2], v[3]);
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 f = *reinterpret_cast<const float2*>(&G->since[8 * n + 2 * (lane & 3)]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) y[n][j] = fmaf((j & 1) ? -f.y : -f.x, y[n][j], v[n][j]);
                }
                // R^T = Y^T X^T; X is lower triangular
                const uint32_t x_n = at_pieces_first<C * 2>(sb + F::x + so, 0, 0, lane);
                float r[4][4];
                const auto solve = [&] {
                    uint32_t ay[3][4], bx[2][3][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[n][j] = 0.f;
#pragma unroll
                    for (int np = 0; np < 2; ++np)
#pragma unroll
                        for (int t = 0; t < 3; ++t) ldsm4(bx[np][t], x_n + t * (C * C * 2) + np * 16 * C * 2);
                    split_a<3>(y[0], y[1], ay);
                    prod<3, 3, 2>(r, ay, bx);
#pragma unroll
                    for (int t = 0; t < 3; ++t) ldsm4(bx[0][t], (x_n ^ 32) + t * (C * C * 2) + 16 * C * 2);
                    split_a<3>(y[2], y[3], ay);
                    prod2<3, 3>(r[2], r[3], ay, bx[0]);
                };
                solve();
                float2 be[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) be[n] = *reinterpret_cast<const float2*>(&G->beta[8 * n + 2 * (lane & 3)]);
                if constexpr (MODE == OUT) {
                    if (any_bad(y)) {              // found while the products are under way; then once more, cleaned
                        int first[2];
                        first_bad(y, lane, first);
                        clean(y);
                        solve();
                        spoil(r, lane, first);
                    }
                }
                if (MODE == STORE) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int tok = t_first + c * C + 8 * n + 2 * (lane & 3);
                        float* to = a.errors + (static_cast<long long>(bh) * a.T + tok) * a.dv + col0 + 16 * grp + (lane >> 2);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (tok + (j & 1) < t_end) to[(j & 1) * a.dv + 8 * (j >> 1)] = r[n][j];
                    }
                }
                // U^T for the outputs, and U^T e^(c_C - c) for the state
                uint32_t au[2][3][4];
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
                    for (int n = 2 * kk; n < 2 * kk + 2; ++n) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[n][j] *= (j & 1) ? be[n].y : be[n].x;
                    }
                    if (MODE == OUT) {
#pragma unroll
                        for (int n = 2 * kk; n < 2 * kk + 2; ++n) uf[n * 32] = make_float4(r[n][0], r[n][1], r[n][2], r[n][3]);
                    }
#pragma unroll
                    for (int n = 2 * kk; n < 2 * kk + 2; ++n) {
                        const float2 f = *reinterpret_cast<const float2*>(&G->left[8 * n + 2 * (lane & 3)]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) r[n][j] *= (j & 1) ? f.y : f.x;
                    }
                    split_a<3>(r[2 * kk], r[2 * kk + 1], au[kk]);
                }
                // 32 keys at a time: four tiles cover a product's latency
#pragma unroll
                for (int g = 0; g < DK / 32; ++g) {
                    float W[4][4] = {};
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
            // this part's share of S0^T K^T, all tokens
            float y[4][4] = {};
#pragma unroll
            for (int ks = 0; ks < DH / 16; ++ks) {
                uint32_t bk[2][KT][4];
#pragma unroll
                for (int np = 0; np < 2; ++np)
#pragma unroll
                    for (int t = 0; t < KT; ++t)   // a step of 16 keys changes the piece by two: its swizzle is an exclusive or
                        ldsm4(bk[np][t], ((k_n + so) ^ (ks << 5)) + t * (C * DK * 2) + np * 16 * DK * 2);
                uint32_t as[3][4];
                split_a<3>(S[2 * ks], S[2 * ks + 1], as);
                prod<3, KT, 2>(y, as, bk);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n / TN != part) ex[(part * 4 + n) * 32] = make_float4(y[n][0], y[n][1], y[n][2], y[n][3]);
            // meanwhile: V, gates and the inverse for the tokens of this part
            float v[2][4] = {};
            if (!unit) cols_t<CS>(static_cast<const E*>(nullptr), sb + F::v + so, 16 * grp, part * TN * 8 / 16 * 16, lane, v[0], v[1]);
            float2 since[TN], beta[TN], left[TN];
            uint32_t bx[TN][3][4];
#pragma unroll
            for (int e = 0; e < TN; ++e) {
                const int n = part * TN + e, tok = 8 * n + 2 * (lane & 3);
                since[e] = *reinterpret_cast<const float2*>(&G->since[tok]);
                beta[e] = *reinterpret_cast<const float2*>(&G->beta[tok]);
                left[e] = *reinterpret_cast<const float2*>(&G->left[tok]);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    ldsm4(bx[e][t], sb + F::x + so + t * (C * C * 2) + piece<C * 2>(8 * n + (lane & 7), lane >> 3));
            }
            const float all = G->all;
            float mine[TN][4];
#pragma unroll
            for (int n = 0; n < 4; ++n)                   // (register arrays take constant indexes only)
                if (n / TN == part)
#pragma unroll
                    for (int j = 0; j < 4; ++j) mine[n % TN][j] = y[n][j];
            ptx::named_sync(1 + grp, NH * 32);
            // Y^T = V^T - (S0^T K^T) e^c for the tokens of this part
            float z[TN][4];
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
                for (int j = 0; j < 4; ++j) z[e][j] = fmaf((j & 1) ? -since[e].y : -since[e].x, w[j], v[e][j]);
                uint32_t t0[3], t1[3];
                split<3>(z[e][0], z[e][1], t0);
                split<3>(z[e][2], z[e][3], t1);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    reinterpret_cast<uint2*>(yf)[((n >> 1) * 3 + t) * 64 + lane * 2 + (n & 1)] = make_uint2(t0[t], t1[t]);
            }
            ptx::named_sync(1 + grp, NH * 32);
            // R^T = Y^T X^T for the tokens of this part; X is lower triangular
            uint32_t ay[2][3][4];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const uint4 u = reinterpret_cast<const uint4*>(yf)[(kk * 3 + t) * 32 + lane];
                    ay[kk][t][0] = u.x; ay[kk][t][1] = u.y; ay[kk][t][2] = u.z; ay[kk][t][3] = u.w;
                }
            float u[TN][4];
            const auto solve = [&] {
#pragma unroll
            for (int e = 0; e < TN; ++e) {
                const int n = part * TN + e;
                float r[4][4] = {};
#pragma unroll
                for (int i = 0; i < 3; ++i)
#pragma unroll
                    for (int j = 0; j < 3 - i; ++j) {
                        mma16816(r[(i + j) & 1], ay[0][i], bx[e][j][0], bx[e][j][1]);
                        if (n >= 2) mma16816(r[2 + ((i + j) & 1)], ay[1][i], bx[e][j][2], bx[e][j][3]);
                    }
#pragma unroll
                for (int j = 0; j < 4; ++j) u[e][j] = (r[0][j] + r[1][j]) + (r[2][j] + r[3][j]);
            }
            };
            solve();
            if (MODE == STORE) {
#pragma unroll
                for (int e = 0; e < TN; ++e) {
                    const int n = part * TN + e;
                    const int tok = t_first + c * C + 8 * n + 2 * (lane & 3);
                    float* to = a.errors + (static_cast<long long>(bh) * a.T + tok) * a.dv + col0 + 16 * grp + (lane >> 2);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (tok + (j & 1) < t_end) to[(j & 1) * a.dv + 8 * (j >> 1)] = u[e][j];
                }
            }
            if constexpr (MODE == OUT) {
                if (any_bad(z)) {
                    // once more with this half's share cleaned; the other half's stays as it is, since all of this
                    // half comes behind what is bad there
                    int first[2];
                    first_bad(z, lane, first);
                    clean(z);
                    if (part == 0) split_a<3>(z[0], z[1], ay[0]);
                    else split_a<3>(z[0], z[1], ay[1]);
                    solve();
                    spoil(u, lane, first);
                }
            }
            // U^T for the outputs, and U^T e^(c_C - c) for the state
#pragma unroll
            for (int e = 0; e < TN; ++e)
#pragma unroll
                for (int j = 0; j < 4; ++j) u[e][j] *= (j & 1) ? beta[e].y : beta[e].x;
#pragma unroll
            for (int e = 0; e < TN; ++e) {
                const int n = part * TN + e;
                uint32_t t0[3], t1[3];
                split<3>(u[e][0] * left[e].x, u[e][1] * left[e].y, t0);
                split<3>(u[e][2] * left[e].x, u[e][3] * left[e].y, t1);
#pragma unroll
                for (int t = 0; t < 3; ++t)
                    reinterpret_cast<uint2*>(vf)[((n >> 1) * 3 + t) * 64 + lane * 2 + (n & 1)] = make_uint2(t0[t], t1[t]);
                if (MODE == OUT) uf[n * 32] = make_float4(u[e][0], u[e][1], u[e][2], u[e][3]);
            }
            uint32_t bt[2][DH / 16][KT][4];
            if constexpr (KT == 1) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int np = 0; np < DH / 16; ++np)
                        ldsm4t(bt[kk][np][0], ((k_t + so) ^ (np << 5)) + kk * 16 * DK * 2);
            }
            ptx::named_sync(1 + grp, NH * 32);
            float W[DH / 8][4] = {};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t au[3][4];
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const uint4 u = reinterpret_cast<const uint4*>(vf)[(kk * 3 + t) * 32 + lane];
                    au[t][0] = u.x; au[t][1] = u.y; au[t][2] = u.z; au[t][3] = u.w;
                }
                if constexpr (KT > 1) {
#pragma unroll
                    for (int np = 0; np < DH / 16; ++np)
#pragma unroll
                        for (int t = 0; t < KT; ++t)
                            ldsm4t(bt[kk][np][t], ((k_t + so) ^ (np << 5)) + t * (C * DK * 2) + kk * 16 * DK * 2);
                }
                prod<3, KT, DH / 16>(W, au, bt[kk]);
            }
            decay_and_add(S, all, W);
            }
            if (++stage == F::NS) stage = 0;
            if (++gstage == F::NG_STAGES) gstage = 0;
            step_end();
        }
        step_end();
    } else if (chunks > 0 && warp < w_load) {
        // ---------------------------------------------------- output: 16 columns a warp
        const int g = warp - w_out;
        const uint32_t q_a = at_rows_first<DK * 2>(sb + F::behind + F::q, 0, 0, lane);
        const uint32_t p_a = at_rows_first<C * 2>(sb + F::behind + F::p, 0, 0, lane);
        E* o = static_cast<E*>(a.o) + (vrow + static_cast<long long>(lane >> 2) * vstep) * a.dv + col0 + 16 * g + 2 * (lane & 3);
        const long long next8 = static_cast<long long>(8) * vstep * a.dv;
        int ostage = 0, gstage = 0;
        for (int s = -F::AHEAD; s < 1; ++s) step_end();
        for (int c = 0; c < chunks; ++c) {
            const uint32_t so = ostage * F::OSTAGE;
            const Gates* G = reinterpret_cast<const Gates*>(sm + F::gates + gstage * 512);
            const float4* sf = reinterpret_cast<const float4*>(sm + F::sf + (c & 1) * F::SB) + g * (DK / 8) * 32 + lane;
            const float4* uf = reinterpret_cast<const float4*>(sm + F::uf + (c & 1) * F::UB) + g * 4 * 32 + lane;
            float acc[2][2][4] = {};          // [16 tokens][8 columns]
            float U[4][4];
#pragma unroll
            for (int n = 0; n < 4; ++n) load4(reinterpret_cast<const float*>(uf + n * 32), U[n]);
            // bad writes are cleaned, and the outputs from their tokens on spoilt below; looked for where it measured
            // faster (behind the state's products 195 and 277 us at 4x16x4096x64 and 2x16x4096x128, before them 198 and 269)
            bool spoilt;
            int first[2];
            const auto look = [&] {
                spoilt = any_bad(U);
                if (spoilt) {
                    first_bad(U, lane, first);
                    clean(U);
                }
            };
            if (DK == 128) look();
#pragma unroll
            for (int ks = 0; ks < DK / 16; ++ks) {
                uint32_t aq[2][KT][4], bs[1][OT][4];
                float x[2][4];
                load4(reinterpret_cast<const float*>(sf + 2 * ks * 32), x[0]);
                load4(reinterpret_cast<const float*>(sf + (2 * ks + 1) * 32), x[1]);
                operand<OT>(x[0], x[1], bs[0]);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
#pragma unroll
                    for (int t = 0; t < KT; ++t) ldsm4(aq[m][t], ((q_a + so) ^ (ks << 5)) + t * (C * DK * 2) + m * 16 * DK * 2);
                    prod<KT, OT, 1>(acc[m], aq[m], bs);
                }
            }
            if (DK < 128) look();
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const float f[2] = {a.scale * G->since[16 * m + (lane >> 2)], a.scale * G->since[16 * m + 8 + (lane >> 2)]};
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[m][n][j] *= f[j >> 1];
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t ap[OT][4], bu[1][OT][4];
                operand<OT>(U[2 * kk], U[2 * kk + 1], bu[0]);
#pragma unroll
                for (int m = kk; m < 2; ++m) {     // P is lower triangular
#pragma unroll
                    for (int t = 0; t < OT; ++t) ldsm4(ap[t], ((p_a + so) ^ (kk << 5)) + t * (C * C * 2) + m * 16 * C * 2);
                    prod<OT, OT, 1>(acc[m], ap, bu);
                }
            }
            if (spoilt) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {            // the column's first bad token, from the lanes that have it
                        const int from = __shfl_sync(0xffffffffu, first[n], 4 * (2 * (lane & 3) + (j & 1)));
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            if (16 * m + (lane >> 2) + 8 * (j >> 1) >= from) acc[m][n][j] = __int_as_float(0x7fffffff);
                    }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int tok = t_first + c * C + (lane >> 2) + 8 * e;
                if (tok >= t_last) continue;
                const bool on = tok < t_end;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float x0 = on ? acc[e >> 1][n][2 * (e & 1)] : 0.f, x1 = on ? acc[e >> 1][n][2 * (e & 1) + 1] : 0.f;
                    if constexpr (F::BF) *reinterpret_cast<uint32_t*>(o + e * next8 + 8 * n) = ptx::pack_bf16(x0, x1);
                    else *reinterpret_cast<float2*>(o + e * next8 + 8 * n) = make_float2(x0, x1);
                }
            }
            o += 4 * next8;
            if (++ostage == F::NS) ostage = 0;
            if (++gstage == F::NG_STAGES) gstage = 0;
            step_end();
        }
    } else if (chunks > 0) {
        // ---------------------------------------------------- load
        const int lt = (warp - w_load) * 32 + lane;
        constexpr int LT = F::NLD * 32;
        const long long ks = static_cast<long long>(kstep) * DK, vs = static_cast<long long>(vstep) * a.dv;
        const E* kp = static_cast<const E*>(a.k) + krow * DK;
        const E* qp = static_cast<const E*>(a.q) + krow * DK;
        const E* vp = static_cast<const E*>(a.v) + vrow * a.dv + col0;
        constexpr int REC = record_bytes(F::INV);
        const uint8_t* rec = a.records + (static_cast<long long>(bh) * ((a.T + C - 1) / C) + t_first / C) * REC;
        const uint8_t* behind = rec;
        int stage = 0, ostage = 0, gstage = 0;
        for (int c = 0; c <= chunks + F::AHEAD; ++c) {
            if (c < chunks) {
                const uint32_t sg = sb + stage * F::STAGE;
                const int rows = min(C, t_end - t_first - c * C);
                load_bytes<kXBytes, LT>(sg + F::x, rec, lt);
                load_bytes<512, LT>(sb + F::gates + gstage * 512, rec + (F::INV + 1) * kXBytes, lt);
                if (!unit) load_cols<CS, LT>(sg + F::v, vp, vs, rows, lt);
                load_tile<DK, KT, LT>(sg + F::k, kp, ks, rows, lt);
                kp += C * ks; vp += C * vs;
                rec += REC;
                if (++stage == F::NS) stage = 0;
                if (++gstage == F::NG_STAGES) gstage = 0;
            }
            if (MODE == OUT && c > 0 && c <= chunks) {      // queries and P of the chunk before
                const uint32_t so = sb + F::behind + ostage * F::OSTAGE;
                load_bytes<kXBytes, LT>(so + F::p, behind + F::INV * kXBytes, lt);
                load_tile<DK, KT, LT>(so + F::q, qp, ks, min(C, t_end - t_first - (c - 1) * C), lt);
                qp += C * ks; behind += REC;
                if (++ostage == F::NS) ostage = 0;
            }
            cp_commit();
            cp_wait<F::AHEAD - 1>();
            step_end();
        }
    }

    if (warp < F::W_STATE) {
        const int col = col0 + 16 * grp + (lane >> 2), key = part * DH + 2 * (lane & 3);
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
    cudaError_t e = allow_smem<k_delta_walk<F>>(F::bytes);
    if (e != cudaSuccess) return e;
    k_delta_walk<F><<<blocks, F::WARPS * 32, F::bytes, st>>>(a);
    return cudaGetLastError();
}

template <typename E, int DK, bool GR>
cudaError_t summaries(const Problem& p, const Segments& g, const uint8_t* records, float* sums, cudaStream_t st) {
    using F = Cfg<E, DK, sizeof(E) == 2 ? 2 : 1, SUMMARY, GR>;
    static_assert(F::bytes <= 227 * 1024, "shared memory of a block");
    const WalkArgs a{p.q, p.k, p.v, records, p.state_in, p.lengths, nullptr, nullptr, sums, nullptr, nullptr, 1,
                     p.Hk, p.H, p.T, p.dv, p.bthd ? 1 : 0, g.count, g.chunks, p.scale};
    return start<F>(a, p.B * p.H * (g.count - 1) * ((p.dv + DK) / F::CS), st);
}

template <typename E, int DK>
cudaError_t walk(const Problem& p, void* ws, cudaStream_t st) {
    constexpr int NG = sizeof(E) == 2 ? 2 : 1;
    using F = Cfg<E, DK, NG, OUT, false>;
    static_assert(F::bytes <= 227 * 1024, "shared memory of a block");
    const int BH = p.B * p.H;
    char* w = static_cast<char*>(ws);
    uint8_t* records = reinterpret_cast<uint8_t*>(w);
    const Segments g = segments(p, false);
    float* sums = reinterpret_cast<float*>(w + records_bytes(p, false));
    float* starts = sums + g.sums;
    cudaError_t e = prepare(p, false, records, st);
    if (e == cudaSuccess && g.count > 1) e = summaries<E, DK, false>(p, g, records, sums, st);
    if (e == cudaSuccess && g.count > 1) e = fold(p, g, sums, nullptr, p.state_in, starts, st);
    if (e != cudaSuccess) return e;
    WalkArgs a{p.q, p.k, p.v, records, g.count > 1 ? starts : p.state_in, p.lengths, p.o, p.state_out, nullptr, nullptr,
               nullptr, 1, p.Hk, p.H, p.T, p.dv, p.bthd ? 1 : 0, g.count, g.chunks, p.scale};
    return start<F>(a, BH * g.count * (p.dv / F::CS), st);
}

template <typename E, int DK, int NG>
cudaError_t walk_store(const Problem& p, const Segments& g, const uint8_t* records, const float* first, float* states,
                       float* errors, int block_chunks, cudaStream_t st) {
    using F = Cfg<E, DK, NG, STORE, true>;
    static_assert(F::bytes <= 227 * 1024, "shared memory of a block");
    WalkArgs a{p.q, p.k, p.v, records, first, p.lengths, nullptr, nullptr, nullptr, states,
               errors, block_chunks, p.Hk, p.H, p.T, p.dv, p.bthd ? 1 : 0, g.count, g.chunks, p.scale};
    return start<F>(a, p.B * p.H * g.count * (p.dv / F::CS), st);
}

}  // namespace

cudaError_t summarize(const Problem& p, const Segments& g, const uint8_t* records, float* sums, cudaStream_t st) {
    if (p.bf16) {
        if (p.d == 32) return summaries<bf16, 32, true>(p, g, records, sums, st);
        if (p.d == 64) return summaries<bf16, 64, true>(p, g, records, sums, st);
        return summaries<bf16, 128, true>(p, g, records, sums, st);
    }
    if (p.d == 32) return summaries<float, 32, true>(p, g, records, sums, st);
    if (p.d == 64) return summaries<float, 64, true>(p, g, records, sums, st);
    return summaries<float, 128, true>(p, g, records, sums, st);
}

cudaError_t store_states(const Problem& p, const Segments& g, const uint8_t* records, const float* first, float* states,
                         float* errors, int block_chunks, cudaStream_t st) {
    if (p.bf16) {
        const bool wide = gradient_columns(p, static_cast<long long>(p.B) * p.H * g.count) == 64;
        if (p.d == 32)
            return wide ? walk_store<bf16, 32, 4>(p, g, records, first, states, errors, block_chunks, st)
                        : walk_store<bf16, 32, 2>(p, g, records, first, states, errors, block_chunks, st);
        if (p.d == 64)
            return wide ? walk_store<bf16, 64, 4>(p, g, records, first, states, errors, block_chunks, st)
                        : walk_store<bf16, 64, 2>(p, g, records, first, states, errors, block_chunks, st);
        return walk_store<bf16, 128, 2>(p, g, records, first, states, errors, block_chunks, st);
    }
    if (p.d == 32) return walk_store<float, 32, 1>(p, g, records, first, states, errors, block_chunks, st);
    if (p.d == 64) return walk_store<float, 64, 1>(p, g, records, first, states, errors, block_chunks, st);
    return walk_store<float, 128, 1>(p, g, records, first, states, errors, block_chunks, st);
}

size_t forward_bytes(const Problem& p) {
    const Segments g = segments(p, false);
    return records_bytes(p, false) + sizeof(float) * (g.sums + g.starts);
}
int forward_launches(const Problem& p) { return segments(p, false).count > 1 ? 4 : 2; }

cudaError_t forward(const Problem& p, void* ws, cudaStream_t st) {
    if (p.bf16) {
        if (p.d == 32) return walk<bf16, 32>(p, ws, st);
        if (p.d == 64) return walk<bf16, 64>(p, ws, st);
        return walk<bf16, 128>(p, ws, st);
    }
    if (p.d == 32) return walk<float, 32>(p, ws, st);
    if (p.d == 64) return walk<float, 64>(p, ws, st);
    return walk<float, 128>(p, ws, st);
}

}  // namespace delta
}  // namespace hla
