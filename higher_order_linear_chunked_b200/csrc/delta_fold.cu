// Segments of long sequences: how many, and the states between them.
#include "delta_walk.cuh"

namespace hla {
namespace delta {
namespace {

struct FoldArgs {
    const float *sums, *back, *first;
    float* out;
    int dv, count;
};

// S <- A S + B from segment to segment (REV: S <- A^T S + G, from the last to the first), 8 columns of
// one head a block; a thread has four columns of one row.  A segment's A and B are on their way while
// the one before is worked on: what is left of a segment is 2 d d 8 flops a block on the CUDA cores (fp32)
// and two barriers, about 0.4 us at d = 64.
template <int DK, bool REV>
__global__ void __launch_bounds__(DK * 2) k_delta_fold(const FoldArgs a) {
    constexpr int NT = DK * 2, LD = DK + 1, U = DK * DK / 4 / NT;      // float4 of A a thread
    extern __shared__ __align__(16) float sm[];
    float* As = sm;                                                    // [k][row]
    float4* Ss = reinterpret_cast<float4*>(sm + (DK * LD + 3) / 4 * 4);   // [k][2 x 4 columns]
    const int slices = a.dv / 8, bh = blockIdx.x / slices, col0 = (blockIdx.x % slices) * 8;
    const int tid = threadIdx.x, r = tid % DK, cg = tid / DK, width = a.dv + DK;
    const int N = a.count;
    const auto A = [&](int s) { return a.sums + (static_cast<long long>(bh) * (N - 1) + s) * DK * width + a.dv; };
    const auto add = [&](int s) {
        return REV ? a.back + ((static_cast<long long>(bh) * N + s) * DK + r) * a.dv + col0 + 4 * cg
                   : a.sums + ((static_cast<long long>(bh) * (N - 1) + s) * DK + r) * width + col0 + 4 * cg;
    };
    const auto put = [&](int s, const float (&x)[4]) {
        store4(a.out + ((static_cast<long long>(bh) * N + s) * DK + r) * a.dv + col0 + 4 * cg, x);
    };
    const int step = REV ? -1 : 1, s0 = REV ? N - 1 : 0, last = REV ? 0 : N - 1;
    float4 next[U];
    float plus[4];
    const auto ask = [&](int s) {
        if (s == last) return;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tid + u * NT;
            next[u] = *reinterpret_cast<const float4*>(A(s) + (i / (DK / 4)) * width + (i % (DK / 4)) * 4);
        }
        load4(add(s), plus);
    };
    ask(s0 + step);
    float cur[4] = {};
    if (a.first) load4(a.first + (static_cast<long long>(bh) * DK + r) * a.dv + col0 + 4 * cg, cur);
    put(s0, cur);
    load4(add(s0), cur);
    put(s0 + step, cur);
    for (int s = s0 + step; s != last; s += step) {
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = tid + u * NT, row = i / (DK / 4), c = (i % (DK / 4)) * 4;
            const float x[4] = {next[u].x, next[u].y, next[u].z, next[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) As[REV ? row * LD + c + j : (c + j) * LD + row] = x[j];
        }
        Ss[r * 2 + cg] = make_float4(cur[0], cur[1], cur[2], cur[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) cur[j] = plus[j];
        __syncthreads();
        ask(s + step);
        float odd[4] = {};
#pragma unroll 16
        for (int k = 0; k < DK; k += 2) {
            const float x0 = As[k * LD + r], x1 = As[(k + 1) * LD + r];
            const float4 y0 = Ss[k * 2 + cg], y1 = Ss[(k + 1) * 2 + cg];
            cur[0] = fmaf(x0, y0.x, cur[0]); odd[0] = fmaf(x1, y1.x, odd[0]);
            cur[1] = fmaf(x0, y0.y, cur[1]); odd[1] = fmaf(x1, y1.y, odd[1]);
            cur[2] = fmaf(x0, y0.z, cur[2]); odd[2] = fmaf(x1, y1.z, odd[2]);
            cur[3] = fmaf(x0, y0.w, cur[3]); odd[3] = fmaf(x1, y1.w, odd[3]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) cur[j] += odd[j];
        put(s + step, cur);
    }
}

template <int DK, bool REV>
cudaError_t run(const Problem& p, const FoldArgs& a, cudaStream_t st) {
    constexpr int bytes = ((DK * (DK + 1) + 3) / 4 * 4 + DK * 8) * 4;
    const cudaError_t e = allow_smem<k_delta_fold<DK, REV>>(bytes);
    if (e != cudaSuccess) return e;
    k_delta_fold<DK, REV><<<p.B * p.H * (p.dv / 8), DK * 2, bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// Steps of chunks one after another, in units of one walk step: without segments, all chunks of a head
// as often as the heads' column slices fill the SMs (two blocks an SM where they fit, a step of which
// takes 1.25 times one block's); with them, the summaries' walk (no outputs: about 0.85 of a step, two
// blocks an SM), the fold (0.4 a segment at d = 64, by d squared) and the second walk.  Taken when a
// tenth is gained.  Forward at bf16, without and with the segments that it takes: 1x4x16384x64 578 and
// 135 us (10 segments), 1x8x4096x64 154 and 74, 2x16x4096x64 168 and 159; 4x16x4096x64 fills the
// machine: 188 without, 254 with three.
Segments segments(const Problem& p) {
    constexpr int SMS = 148;
    const long long BH = static_cast<long long>(p.B) * p.H;
    const int NC = (p.T + C - 1) / C, CS = p.bf16 ? 32 : 16, fit = p.bf16 ? (p.d <= 64 ? 2 : 1) : (p.d == 32 ? 2 : 1);
    const auto waves = [&](long long blocks, int fit) {
        const long long rest = blocks % (SMS * fit);
        return (fit == 2 ? 1.25 : 1.0) * static_cast<double>(blocks / (SMS * fit)) + (rest == 0 ? 0.0 : rest <= SMS ? 1.0 : 1.25);
    };
    const double fold_step = 0.4 * (p.d / 64.0) * (p.d / 64.0) + 0.1;
    int best = 1;
    double cost = 0.9 * waves(BH * p.dv / CS, fit) * NC;
    for (int n = 2; n <= 64 && n <= NC / 4; ++n) {
        const int chunks = (NC + n - 1) / n;
        if ((NC + chunks - 1) / chunks != n) continue;
        const long long summaries = BH * (static_cast<long long>(n - 2) * (p.dv + p.d) + p.dv) / CS;
        const double c = 0.85 * chunks * waves(summaries, 2) + fold_step * n + 8 + chunks * waves(BH * n * p.dv / CS, fit);
        if (c < cost) cost = c, best = n;
    }
    Segments g{best, (NC + best - 1) / best, 0, 0};
    if (best > 1) {
        g.sums = static_cast<size_t>(BH) * (best - 1) * p.d * (p.dv + p.d);
        g.starts = static_cast<size_t>(BH) * best * p.d * p.dv;
    }
    return g;
}

cudaError_t fold(const Problem& p, const Segments& g, const float* sums, const float* back, const float* first,
                 float* out, cudaStream_t st) {
    const FoldArgs a{sums, back, first, out, p.dv, g.count};
    if (back) return p.d == 32 ? run<32, true>(p, a, st) : p.d == 64 ? run<64, true>(p, a, st) : run<128, true>(p, a, st);
    return p.d == 32 ? run<32, false>(p, a, st) : p.d == 64 ? run<64, false>(p, a, st) : run<128, false>(p, a, st);
}

}  // namespace delta
}  // namespace hla
