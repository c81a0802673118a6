// One token of the gated delta rule (decoding).
//
//   y = S^T k, z = S^T q (both of the old S, one pass over it)
//   u = beta (v - a y),  S <- a S + k u^T,  o = scale (a z + (q.k) u)        a = exp(g)
//
// A CTA owns CV value columns of one head: S never leaves its registers between the read and the
// write, so a step moves each state element once each way, which is all that bounds it (7 flops
// per 8 bytes; 193x16 heads of 128x128 take 63 us, 98% of the copy rate).
#include "delta_common.cuh"

namespace hla {
namespace delta {
namespace {

struct StepArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    float* state;            // [B*H][d][dv], in place
    void* o;
    int share;               // value heads of a key head
    float scale;
};

// DV is known at compile time so that a thread's rows are one address and offsets: with an address a row,
// kept from the loads to the stores, some of S left the registers (193x16 heads of 128x128 in bf16: 66 us, not 63).
template <typename E, int DK, int DV, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_delta_step(const StepArgs a) {
    constexpr int CV = DV < 64 ? DV : 64;
    constexpr int LPR = CV / 4;           // lanes per state row (four columns each)
    constexpr int RPP = NT / LPR;         // rows per pass
    constexpr int NP = DK / RPP;          // passes: rows of one thread
    constexpr int NW = NT / 32;
    static_assert(DK % RPP == 0 && 32 % LPR == 0, "rows must divide over the threads");
    __shared__ float s_k[DK], s_q[DK];
    __shared__ float4 s_y[NW][LPR], s_z[NW][LPR];
    __shared__ float s_qk[NW];

    constexpr int slices = DV / CV;
    const int bh = blockIdx.x / slices, col0 = (blockIdx.x % slices) * CV;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c4 = tid % LPR, r0 = tid / LPR;
    const long long krow = static_cast<long long>(bh / a.share) * DK;      // H is a multiple of Hk: b and hk in one
    const long long vat = static_cast<long long>(bh) * DV + col0 + 4 * c4;
    float* const state = a.state + (static_cast<long long>(bh) * DK + r0) * DV + col0 + 4 * c4;

    float S[NP][4], vv[4];
#pragma unroll
    for (int i = 0; i < NP; ++i) load4(state + i * RPP * DV, S[i]);
    for (int i = tid; i < DK; i += NT) {
        s_k[i] = to_f32(static_cast<const E*>(a.k)[krow + i]);
        s_q[i] = to_f32(static_cast<const E*>(a.q)[krow + i]);
    }
    const float decay = expf(gate(a.g[bh])), beta = a.beta[bh];
    load4(static_cast<const E*>(a.v) + vat, vv);
    __syncthreads();
    float y[4] = {}, z[4] = {}, qk = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const float kk = s_k[r0 + i * RPP], qq = s_q[r0 + i * RPP];
        qk = fmaf(kk, qq, qk);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = fmaf(kk, S[i][j], y[j]);
            z[j] = fmaf(qq, S[i][j], z[j]);
        }
    }
#pragma unroll
    for (int w = LPR; w < 32; w <<= 1) {
        qk += __shfl_xor_sync(0xffffffffu, qk, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] += __shfl_xor_sync(0xffffffffu, y[j], w);
            z[j] += __shfl_xor_sync(0xffffffffu, z[j], w);
        }
    }
    if (lane < LPR) {
        s_y[warp][lane] = make_float4(y[0], y[1], y[2], y[3]);
        s_z[warp][lane] = make_float4(z[0], z[1], z[2], z[3]);
        if (lane == 0) s_qk[warp] = qk;
    }
    __syncthreads();
    float u[4] = {}, tz[4] = {}, tqk = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float4 fy = s_y[w][c4], fz = s_z[w][c4];
        u[0] += fy.x; u[1] += fy.y; u[2] += fy.z; u[3] += fy.w;
        tz[0] += fz.x; tz[1] += fz.y; tz[2] += fz.z; tz[3] += fz.w;
        tqk += s_qk[w];
    }
    float out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        u[j] = beta * (vv[j] - decay * u[j]);
        out[j] = a.scale * fmaf(decay, tz[j], tqk * u[j]);
    }
    if (r0 == 0) store4(static_cast<E*>(a.o) + vat, out);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const float kk = s_k[r0 + i * RPP];
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] = fmaf(kk, u[j], decay * S[i][j]);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) store4(state + i * RPP * DV, S[i]);
}

template <typename E, int DK>
cudaError_t launch(const Problem& p, const StepArgs& a, cudaStream_t st) {
    constexpr int NT = DK == 128 ? 256 : 128;
    const int BH = p.B * p.H;
    if (p.dv == 32) k_delta_step<E, DK, 32, 128><<<BH, 128, 0, st>>>(a);
    else if (p.dv == 64) k_delta_step<E, DK, 64, NT><<<BH, NT, 0, st>>>(a);
    else k_delta_step<E, DK, 128, NT><<<2 * BH, NT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t step(const Problem& p, cudaStream_t st) {
    const StepArgs a{p.q, p.k, p.v, p.g, p.beta, p.state_out, p.o, p.H / p.Hk, p.scale};
    if (p.bf16) {
        if (p.d == 32) return launch<bf16, 32>(p, a, st);
        if (p.d == 64) return launch<bf16, 64>(p, a, st);
        return launch<bf16, 128>(p, a, st);
    }
    if (p.d == 32) return launch<float, 32>(p, a, st);
    if (p.d == 64) return launch<float, 64>(p, a, st);
    return launch<float, 128>(p, a, st);
}

}  // namespace delta
}  // namespace hla
