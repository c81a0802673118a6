// Segments of long sequences: how many, and the states between them.
#include "delta_walk.cuh"

namespace hla {
namespace delta {
namespace {

constexpr int kSMs = 148;

struct FoldArgs {
    const float *sums, *back, *first;
    float* out;
    int dv, count;
};

// S <- A S + B from segment to segment (REV: S <- A^T S + G, from the last to the first), 8 columns of
// one head a block; a thread has four columns of one row.  A and B of the next two segments are on
// their way into a ring of three; a segment then costs 2 d d 8 flops a block on the CUDA cores (fp32)
// and one barrier: 0.8 us at d = 64, bound by the four warps' own latency (four lanes to a row, with
// 16 warps, took 1.1: the barrier and the copies weigh more than the products).
template <int DK>
struct FoldSmem {
    static constexpr int LD = DK + 4, A = DK * LD, STAGE = A + DK * 8, S = 3 * STAGE, floats = S + 2 * DK * 8;
};

template <int DK, bool REV>
__global__ void __launch_bounds__(DK * 2) k_delta_fold(const FoldArgs a) {
    using M = FoldSmem<DK>;
    constexpr int NT = DK * 2, LD = M::LD;
    extern __shared__ __align__(16) float sm[];
    const uint32_t sb = ptx::smem_u32(sm);
    const int slices = a.dv / 8, bh = blockIdx.x / slices, col0 = (blockIdx.x % slices) * 8;
    const int tid = threadIdx.x, r = tid % DK, cg = tid / DK, width = a.dv + DK;
    const int N = a.count, step = REV ? -1 : 1, s0 = REV ? N - 1 : 0, last = REV ? 0 : N - 1;
    const auto added = [&](int s) {      // B or G of segment s, this block's columns
        return REV ? a.back + (static_cast<long long>(bh) * N + s) * DK * a.dv + col0
                   : a.sums + (static_cast<long long>(bh) * (N - 1) + s) * DK * width + col0;
    };
    const int bstep = REV ? a.dv : width;
    const auto put = [&](int s, const float (&x)[4]) {
        store4(a.out + ((static_cast<long long>(bh) * N + s) * DK + r) * a.dv + col0 + 4 * cg, x);
    };
    const auto ask = [&](int n) {        // the n-th segment of the fold into its stage
        const int s = s0 + n * step;
        if (n < N - 1) {
            const uint32_t to = sb + (n % 3) * M::STAGE * 4;
            const float* A = a.sums + (static_cast<long long>(bh) * (N - 1) + s) * DK * width + a.dv;
#pragma unroll
            for (int i = tid; i < DK * DK / 4; i += NT)
                cp_async16(to + ((i / (DK / 4)) * LD + (i % (DK / 4)) * 4) * 4, A + (i / (DK / 4)) * width + (i % (DK / 4)) * 4, true);
            cp_async16(to + (M::A + r * 8 + 4 * cg) * 4, added(s) + r * bstep + 4 * cg, true);
        }
        cp_commit();
    };
    next_may_start();                    // REV runs beside the fold from the first segment on
    ask(1);
    ask(2);
    float cur[4] = {};
    if (a.first) load4(a.first + (static_cast<long long>(bh) * DK + r) * a.dv + col0 + 4 * cg, cur);
    put(s0, cur);
    load4(added(s0) + r * bstep + 4 * cg, cur);
    put(s0 + step, cur);
    for (int n = 1; s0 + n * step != last; ++n) {
        float4* Ss = reinterpret_cast<float4*>(sm + M::S + (n & 1) * DK * 8);
        const float* As = sm + (n % 3) * M::STAGE;
        Ss[r * 2 + cg] = make_float4(cur[0], cur[1], cur[2], cur[3]);
        cp_wait<1>();
        __syncthreads();
        ask(n + 2);                      // its stage was last read before this barrier
        load4(As + M::A + r * 8 + 4 * cg, cur);
        float odd[4] = {};
#pragma unroll 16
        for (int k = 0; k < DK; k += 4) {
            float x[4];
            if (REV) {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = As[(k + j) * LD + r];
            } else {
                load4(As + r * LD + k, x);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 y = Ss[(k + j) * 2 + cg];
                float (&to)[4] = (j & 1) ? odd : cur;
                to[0] = fmaf(x[j], y.x, to[0]);
                to[1] = fmaf(x[j], y.y, to[1]);
                to[2] = fmaf(x[j], y.z, to[2]);
                to[3] = fmaf(x[j], y.w, to[3]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) cur[j] += odd[j];
        put(s0 + (n + 1) * step, cur);
    }
    cp_wait<0>();
    if (REV) previous_done();
}

template <int DK, bool REV>
cudaError_t run(const Problem& p, const FoldArgs& a, cudaStream_t st) {
    constexpr int bytes = FoldSmem<DK>::floats * 4;
    static_assert(bytes <= 227 * 1024, "shared memory of a block");
    const cudaError_t e = allow_smem<k_delta_fold<DK, REV>>(bytes);
    if (e != cudaSuccess) return e;
    const int blocks = p.B * p.H * (p.dv / 8);
    if (REV) return launch_beside(k_delta_fold<DK, REV>, blocks, DK * 2, bytes, st, a);
    k_delta_fold<DK, REV><<<blocks, DK * 2, bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

// A block of one walk beside a block of the other on an SM costs both as much as one after the other,
// a block of twice the columns only a quarter more: 64 columns where both walks' blocks then have an SM
// each and blocks of 32 would not.  4x16x4096x64, all gradients: the walks one after the other 679 us, side by
// side 735 with 32 columns and 588 with 64.
int gradient_columns(const Problem& p, long long walked) {
    if (!p.bf16) return 16;
    const long long walks = 2 * walked;
    return p.d <= 64 && p.dv % 64 == 0 && walks * (p.dv / 32) > kSMs && walks * (p.dv / 64) <= kSMs ? 64 : 32;
}

// Side by side the walks are faster or the same for all widths and types (bf16 5x8x2048x128: 668 us, one after
// the other 728; fp32 16x16x512x32: 232 and 252), but not for bf16 with d = 64 where one walk alone has a
// block or two for every SM: two reverse blocks leave an SM no room for a forward one, and the second walk's
// last blocks come late (5x16x2048x64: 504 us, one after the other 471; 9x16x1024x64 360 and 337; 8x16x2048x64
// 639 and 606; with more blocks the same again, 16x16x1024x64 574 and 575).
bool gradient_walks_beside(const Problem& p, long long blocks) {
    return !(p.bf16 && p.d == 64 && blocks > kSMs && blocks <= 2 * kSMs);
}

// Steps of chunks one after another, in units of one walk step: without segments, all chunks of a head
// as often as the heads' column slices fill the SMs (two blocks an SM where they fit, a step of which
// takes 1.25 times one block's); with them, the summaries' walk (no outputs: about 0.85 of a step, two
// blocks an SM), the fold (0.5 a segment at d = 64) and the second walk.  Taken when a
// tenth is gained.  Forward at bf16, without and with the segments that it takes: 1x4x16384x64 612 and
// 102 us, 1x8x4096x64 161 and 58, 2x16x4096x64 178 and 160; 4x16x4096x64 fills the machine: 196
// without, 273 with.
// The gradients have two such walks side by side, a reverse step 1.3; on SMs of their own that is all,
// with 64 columns a block 1.25 times it, on shared ones 1.35 a wave (between 1.2 and 1.75 eight shapes
// of ten chose the same, the two others best here): 2x16x4096x64 needs no segments, 367 us with the rest of
// the gradients, not 423.
Segments segments(const Problem& p, bool gradients) {
    const long long BH = static_cast<long long>(p.B) * p.H;
    const int NC = (p.T + C - 1) / C, CS = p.bf16 ? 32 : 16, fit = p.bf16 ? (p.d <= 64 ? 2 : 1) : (p.d == 32 ? 2 : 1);
    const auto waves = [&](long long blocks, int fit) {
        const long long rest = blocks % (kSMs * fit);
        return (fit == 2 ? 1.25 : 1.0) * static_cast<double>(blocks / (kSMs * fit)) + (rest == 0 ? 0.0 : rest <= kSMs ? 1.0 : 1.25);
    };
    const auto walk_waves = [&](long long blocks) {
        if (!gradients) return waves(blocks, fit);
        if (2 * blocks <= kSMs) return 1.3;
        if (gradient_columns(p, blocks * CS / p.dv) == 64) return 1.3 * 1.25;
        return 1.3 * 1.35 * waves(blocks, fit);
    };
    const double fold_step = 0.4 * (p.d / 64.0) * (p.d / 64.0) + 0.1;
    int best = 1;
    double cost = 0.9 * walk_waves(BH * p.dv / CS) * NC;
    for (int n = 2; n <= 64 && n <= NC / 4; ++n) {
        const int chunks = (NC + n - 1) / n;
        if ((NC + chunks - 1) / chunks != n) continue;
        const long long summaries = BH * (static_cast<long long>(n - 2) * (p.dv + p.d) + p.dv) / CS;
        const double c = 0.85 * chunks * waves(summaries, 2) * (gradients ? 1.5 : 1.0) + fold_step * n + 8 +
                         chunks * walk_waves(BH * n * p.dv / CS);
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
