// The gated delta rule token by token (decoding).
//
//   y = S^T k, z = S^T q (both of the old S, one pass over it)
//   u = beta (v - a y),  S <- a S + k u^T,  o = scale (a z + (q.k) u)        a = exp(g)
//
// A CTA owns CV value columns of one head: S never leaves its registers between the read and the
// write, so a step moves each state element once each way, which is all that bounds it (7 flops
// per 8 bytes).
#include "delta_common.cuh"

namespace hla {
namespace delta {
namespace {

struct RecurArgs {
    const void *q, *k, *v;
    const float *g, *beta, *state_in;
    const int* lengths;
    void* o;
    float* state_out;
    int Hk, H, T, dv, bthd;
    float scale;
};

template <typename E, int DK, int CV, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) k_delta_recur(const RecurArgs a) {
    constexpr int LPR = CV / 4;           // lanes per state row (four columns each)
    constexpr int RPP = NT / LPR;         // rows per pass
    constexpr int NP = DK / RPP;          // passes: rows of one thread
    constexpr int NW = NT / 32;
    static_assert(DK % RPP == 0 && 32 % LPR == 0, "rows must divide over the threads");
    __shared__ float s_k[2][DK], s_q[2][DK];
    __shared__ float4 s_y[2][NW][LPR], s_z[2][NW][LPR];
    __shared__ float s_qk[2][NW];

    const int slices = a.dv / CV;
    const int bh = blockIdx.x / slices, col0 = (blockIdx.x % slices) * CV;
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c4 = tid % LPR, r0 = tid / LPR;
    const int T = length_of(a.lengths, b, a.T);
    const long long krow = row_of(a.bthd, b, hk, a.Hk, 0, a.T), vrow = row_of(a.bthd, b, h, a.H, 0, a.T);
    const int kstep = row_step(a.bthd, a.Hk), vstep = row_step(a.bthd, a.H);
    const E* q = static_cast<const E*>(a.q) + krow * DK;
    const E* k = static_cast<const E*>(a.k) + krow * DK;
    const E* v = static_cast<const E*>(a.v) + vrow * a.dv + col0 + 4 * c4;
    E* o = static_cast<E*>(a.o) + vrow * a.dv + col0 + 4 * c4;
    const long long sbase = (static_cast<long long>(bh) * DK) * a.dv + col0 + 4 * c4;

    float S[NP][4];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        if (a.state_in) {
            load4(a.state_in + sbase + static_cast<long long>(r0 + i * RPP) * a.dv, S[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = 0.f;
        }
    }
    for (int t = 0; t < T; ++t) {
        const int p = t & 1;
        for (int i = tid; i < DK; i += NT) {
            s_k[p][i] = to_f32(k[static_cast<long long>(t) * kstep * DK + i]);
            s_q[p][i] = to_f32(q[static_cast<long long>(t) * kstep * DK + i]);
        }
        const long long row = vrow + static_cast<long long>(t) * vstep;
        const float decay = expf(gate(a.g[row])), beta = a.beta[row];
        float vv[4];
        load4(v + static_cast<long long>(t) * vstep * a.dv, vv);
        __syncthreads();
        float y[4] = {}, z[4] = {}, qk = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float kk = s_k[p][r0 + i * RPP], qq = s_q[p][r0 + i * RPP];
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
            s_y[p][warp][lane] = make_float4(y[0], y[1], y[2], y[3]);
            s_z[p][warp][lane] = make_float4(z[0], z[1], z[2], z[3]);
            if (lane == 0) s_qk[p][warp] = qk;
        }
        __syncthreads();
        float ty[4] = {}, tz[4] = {}, tqk = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float4 fy = s_y[p][w][c4], fz = s_z[p][w][c4];
            ty[0] += fy.x; ty[1] += fy.y; ty[2] += fy.z; ty[3] += fy.w;
            tz[0] += fz.x; tz[1] += fz.y; tz[2] += fz.z; tz[3] += fz.w;
            tqk += s_qk[p][w];
        }
        float out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = beta * (vv[j] - decay * ty[j]);
            out[j] = a.scale * fmaf(decay, tz[j], tqk * u);
            ty[j] = u;
        }
        if (r0 == 0) store4(o + static_cast<long long>(t) * vstep * a.dv, out);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const float kk = s_k[p][r0 + i * RPP];
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = fmaf(kk, ty[j], decay * S[i][j]);
        }
    }
    if (r0 == 0) {
        const float zero[4] = {};
        for (int t = T; t < a.T; ++t) store4(o + static_cast<long long>(t) * vstep * a.dv, zero);
    }
    if (a.state_out) {
#pragma unroll
        for (int i = 0; i < NP; ++i) store4(a.state_out + sbase + static_cast<long long>(r0 + i * RPP) * a.dv, S[i]);
    }
}

template <typename E, int DK>
cudaError_t launch(const Problem& p, const RecurArgs& a, cudaStream_t st) {
    const int BH = p.B * p.H;
    if (p.dv == 32) {
        k_delta_recur<E, DK, 32, 128><<<BH, 128, 0, st>>>(a);
    } else {
        constexpr int NT = DK == 128 ? 256 : 128;
        k_delta_recur<E, DK, 64, NT><<<BH * (p.dv / 64), NT, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t recur(const Problem& p, cudaStream_t st) {
    const RecurArgs a{p.q, p.k, p.v, p.g, p.beta, p.state_in, p.lengths, p.o, p.state_out,
                      p.Hk, p.H, p.T, p.dv, p.bthd ? 1 : 0, p.scale};
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
