// What the chunks of the gated delta rule need before any state is known, a block a chunk:
//     M = strict_low(D o K K^T),  P = scale low(D o Q K^T),  X = (I + M diag(beta))^-1
// and, for the gradients, X' = (I + diag(beta) M)^-1; written to the chunk's record with its gate
// values, as the shared-memory images that the walks copy.  All chunks of all heads are independent
// here.  8192 chunks (4x16x4096x64, bf16) read 67 MB and write 105 MB, 155 for the gradients: 41 and 57
// us, 64% and 60% of the copy rate; what is left is a chunk's own chain of products, substitution and
// copies at the ten to eighteen warps an SM that shared memory lets in.  Forward, one warp takes P and
// another X; for the gradients one warp takes all three in turn, each in the place of what it no
// longer needs (57 us; two warps with the larger footprint 70).
#include "delta_walk.cuh"

namespace hla {
namespace delta {
namespace {

struct PrepArgs {
    const void *q, *k;
    const float *g, *beta;
    const int* lengths;
    uint8_t* records;          // [B*H][chunks][record]
    int* status;
    int B, Hk, H, T, chunks, bthd;
    float scale;
};

template <typename E, int DK_, int INV_>
struct Prep {
    using Elem = E;
    static constexpr int DK = DK_, INV = INV_, KT = sizeof(E) == 2 ? 1 : 3;
    static constexpr int TILE = KT * C * DK * 2;
    static constexpr int REC = record_bytes(INV);
    static constexpr int WARPS = INV == 1 ? 2 : 1;
    // shared memory: with one warp the inverses take the queries' place once P is there
    static constexpr int k = 0, q = k + TILE, x = WARPS == 2 ? q + TILE : q;
    static constexpr int m = WARPS == 2 ? x + kXBytes : q + (TILE > kXBytes ? TILE : kXBytes), p = m + C * kMS * 4;
    static constexpr int TAIL = kXBytes + 512, sum = p + TAIL;
    static constexpr int bytes = sum + C * 8;
};

// The blocks above the diagonal of three terms' images, which the products do not write: by one warp.
__device__ __forceinline__ void clear_above(uint8_t* to, int lane) {
    for (int t = 0; t < 3; ++t)
        *reinterpret_cast<uint4*>(to + t * (C * C * 2) + piece<C * 2>(lane & 15, 2 + (lane >> 4))) = make_uint4(0u, 0u, 0u, 0u);
}
template <int N>
__device__ __forceinline__ void copy_out(uint8_t* to, const uint8_t* from, int lane) {
#pragma unroll 4
    for (int i = lane; i < N / 16; i += 32) reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(from)[i];
}

template <typename F>
__global__ void __launch_bounds__(F::WARPS * 32) k_delta_prepare(const PrepArgs a) {
    using E = typename F::Elem;
    constexpr int DK = F::DK, KT = F::KT;
    extern __shared__ __align__(128) uint8_t sm[];
    const uint32_t sb = ptx::smem_u32(sm);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bh = blockIdx.x / a.chunks, c = blockIdx.x % a.chunks;
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int rows = min(C, length_of(a.lengths, b, a.T) - c * C);
    if (blockIdx.x == 0 && tid == 0) *a.status = DEV_OK;               // no kernel of these calls sets it
    if (rows <= 0) return;                                              // no walk reads this chunk
    const int kstep = row_step(a.bthd, a.Hk), vstep = row_step(a.bthd, a.H);
    const long long kr = row_of(a.bthd, b, hk, a.Hk, c * C, a.T), vr = row_of(a.bthd, b, h, a.H, c * C, a.T);
    const long long ks = static_cast<long long>(kstep) * DK;
    load_tile<DK, KT, F::WARPS * 32>(sb + F::k, static_cast<const E*>(a.k) + kr * DK, ks, rows, tid);
    load_tile<DK, KT, F::WARPS * 32>(sb + F::q, static_cast<const E*>(a.q) + kr * DK, ks, rows, tid);
    cp_commit();
    uint8_t* const pt = sm + F::p;
    Gates* const gates = reinterpret_cast<Gates*>(pt + kXBytes);
    float2* const sum = reinterpret_cast<float2*>(sm + F::sum);
    uint8_t* const rec = a.records + static_cast<long long>(blockIdx.x) * F::REC;
    float* const mt = reinterpret_cast<float*>(sm + F::m);
    uint8_t* const xt = sm + F::x;
    if (warp == 0) {
        const bool on = lane < rows;
        const float g = on ? a.g[vr + static_cast<long long>(lane) * vstep] : 0.f;
        const float beta = on ? a.beta[vr + static_cast<long long>(lane) * vstep] : 0.f;
        finish_gates(gates, sum, g, beta, lane);
        clear_above(pt, lane);
    }
    if (F::WARPS == 2 && warp == 1) clear_above(xt, lane);
    cp_wait<0>();
    __syncthreads();
    // queries with keys for P, keys with keys for X, then for X'
    const int first = warp, end = F::WARPS == 2 ? warp + 1 : 1 + F::INV;
#pragma unroll 1
    for (int part = first; part < end; ++part) {
#pragma unroll 1
        for (int w = 0; w < 2; ++w)
            products<DK, KT>(part > 0, part == 2, sb + F::k, sb + (part > 0 ? F::k : F::q), sum, gates->beta, mt, pt,
                                 a.scale, w, lane);
        __syncwarp();
        if (part > 0) {
            invert(mt, xt, lane);
            __syncwarp();
            copy_out<kXBytes>(rec + (part - 1) * kXBytes, xt, lane);
            __syncwarp();
        } else {
            copy_out<F::TAIL>(rec + F::INV * kXBytes, pt, lane);
            if (F::WARPS == 1) clear_above(xt, lane);                   // the queries are done with
        }
    }
}

template <typename E, int DK, int INV>
cudaError_t launch(const Problem& p, uint8_t* records, cudaStream_t st) {
    using F = Prep<E, DK, INV>;
    static_assert(F::bytes <= 227 * 1024, "shared memory of a block");
    const int chunks = (p.T + C - 1) / C;
    const PrepArgs a{p.q, p.k, p.g, p.beta, p.lengths, records, p.status, p.B, p.Hk, p.H, p.T, chunks, p.bthd ? 1 : 0, p.scale};
    const cudaError_t e = allow_smem<k_delta_prepare<F>>(F::bytes);
    if (e != cudaSuccess) return e;
    k_delta_prepare<F><<<p.B * p.H * chunks, F::WARPS * 32, F::bytes, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t records_bytes(const Problem& p, bool gradients) {
    return static_cast<size_t>(p.B) * p.H * ((p.T + C - 1) / C) * record_bytes(gradients ? 2 : 1);
}

template <typename E, int INV>
static cudaError_t by_width(const Problem& p, uint8_t* records, cudaStream_t st) {
    if (p.d == 32) return launch<E, 32, INV>(p, records, st);
    if (p.d == 64) return launch<E, 64, INV>(p, records, st);
    return launch<E, 128, INV>(p, records, st);
}

cudaError_t prepare(const Problem& p, bool gradients, uint8_t* records, cudaStream_t st) {
    if (p.bf16) return gradients ? by_width<bf16, 2>(p, records, st) : by_width<bf16, 1>(p, records, st);
    return gradients ? by_width<float, 2>(p, records, st) : by_width<float, 1>(p, records, st);
}

}  // namespace delta
}  // namespace hla
