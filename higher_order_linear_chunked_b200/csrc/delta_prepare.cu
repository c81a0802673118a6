// What the chunks of the gated delta rule need before any state is known, one warp a chunk:
//     M = strict_low(D o K K^T),  P = scale low(D o Q K^T),  X = (I + M diag(beta))^-1
// and, for the gradients, X' = (I + diag(beta) M)^-1; written to the chunk's record with its gate
// values, as the shared-memory images that the walks copy.  All chunks of all heads are independent
// here; reading the keys and queries and writing the records bounds it.
#include "delta_walk.cuh"

namespace hla {
namespace delta {
namespace {

struct PrepArgs {
    const void *q, *k;
    const float *g, *beta;
    const int* lengths;
    uint8_t* records;          // [B*H][chunks][record]
    int B, Hk, H, T, chunks, bthd;
    float scale;
};

template <typename E, int DK_, int PT_, int INV_>
struct Prep {
    using Elem = E;
    static constexpr int DK = DK_, PT = PT_, INV = INV_, KT = sizeof(E) == 2 ? 1 : 3;
    static constexpr int TILE = KT * C * DK * 2;
    static constexpr int REC = record_bytes(INV, PT);
    // shared memory of one warp: the inverse takes the queries' place once P is there, one inverse
    // at a time; what the record has beside the inverses is staged behind
    static constexpr int k = 0, q = k + TILE, x = q, m = q + (TILE > kXBytes ? TILE : kXBytes), p = m + C * kMS * 4;
    static constexpr int TAIL = PT * C * C * 2 + 512, sum = p + TAIL;
    static constexpr int bytes = (sum + C * 8 + 127) / 128 * 128;
    static constexpr int WARPS = 2;              // small blocks: ten warps an SM at d = 64, bf16
};

template <typename F>
__global__ void __launch_bounds__(F::WARPS * 32) k_delta_prepare(const PrepArgs a) {
    using E = typename F::Elem;
    constexpr int DK = F::DK, KT = F::KT, PT = F::PT;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31;
    uint8_t* sm = smem + (threadIdx.x >> 5) * F::bytes;
    const uint32_t sb = ptx::smem_u32(sm);
    const long long n = static_cast<long long>(blockIdx.x) * F::WARPS + (threadIdx.x >> 5);
    if (n >= static_cast<long long>(a.B) * a.H * a.chunks) return;      // warps do not meet
    const int bh = static_cast<int>(n / a.chunks), c = static_cast<int>(n % a.chunks);
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int rows = min(C, length_of(a.lengths, b, a.T) - c * C);
    if (rows <= 0) return;                                              // no walk reads this chunk
    const int kstep = row_step(a.bthd, a.Hk), vstep = row_step(a.bthd, a.H);
    const long long kr = row_of(a.bthd, b, hk, a.Hk, c * C, a.T), vr = row_of(a.bthd, b, h, a.H, c * C, a.T);
    const long long ks = static_cast<long long>(kstep) * DK;
    load_tile<DK, KT, 32>(sb + F::k, static_cast<const E*>(a.k) + kr * DK, ks, rows, lane);
    load_tile<DK, KT, 32>(sb + F::q, static_cast<const E*>(a.q) + kr * DK, ks, rows, lane);
    cp_commit();
    const bool on = lane < rows;
    const float g = on ? a.g[vr + static_cast<long long>(lane) * vstep] : 0.f;
    const float beta = on ? a.beta[vr + static_cast<long long>(lane) * vstep] : 0.f;
    uint8_t* const pt = sm + F::p;
    uint8_t* const xt = sm + F::x;
    Gates* gates = reinterpret_cast<Gates*>(pt + PT * C * C * 2);
    float2* sum = reinterpret_cast<float2*>(sm + F::sum);
    float* mt = reinterpret_cast<float*>(sm + F::m);
    uint8_t* const rec = a.records + n * F::REC;
    finish_gates(gates, sum, g, beta, lane);
    // the blocks above the diagonal, which the products do not write
    const auto clear_above = [&](uint8_t* to, int terms) {
        for (int t = 0; t < terms; ++t)
            *reinterpret_cast<uint4*>(to + t * (C * C * 2) + piece<C * 2>(lane & 15, 2 + (lane >> 4))) = make_uint4(0u, 0u, 0u, 0u);
    };
    clear_above(pt, PT);
    cp_wait<0>();
    __syncwarp();
#pragma unroll 1
    for (int w = 0; w < 2; ++w)
        products<DK, KT, PT>(false, false, sb + F::k, sb + F::q, sum, gates->beta, mt, pt, a.scale, w, lane);
    __syncwarp();
    clear_above(xt, 3);
    uint4* to = reinterpret_cast<uint4*>(rec + F::INV * kXBytes);
#pragma unroll 4
    for (int i = lane; i < F::TAIL / 16; i += 32) to[i] = reinterpret_cast<const uint4*>(pt)[i];
#pragma unroll 1
    for (int x = 0; x < F::INV; ++x) {
#pragma unroll 1
        for (int w = 0; w < 2; ++w)
            products<DK, KT, PT>(true, x == 1, sb + F::k, sb + F::k, sum, gates->beta, mt, pt, a.scale, w, lane);
        __syncwarp();
        invert(mt, xt, lane);
        __syncwarp();
        to = reinterpret_cast<uint4*>(rec + x * kXBytes);
#pragma unroll 4
        for (int i = lane; i < kXBytes / 16; i += 32) to[i] = reinterpret_cast<const uint4*>(xt)[i];
        __syncwarp();
    }
}

template <typename E, int DK, int PT, int INV>
cudaError_t launch(const Problem& p, uint8_t* records, cudaStream_t st) {
    using F = Prep<E, DK, PT, INV>;
    static_assert(F::bytes * F::WARPS <= 227 * 1024, "shared memory of a block");
    const int chunks = (p.T + C - 1) / C;
    const PrepArgs a{p.q, p.k, p.g, p.beta, p.lengths, records, p.B, p.Hk, p.H, p.T, chunks, p.bthd ? 1 : 0, p.scale};
    cudaError_t e = allow_smem<k_delta_prepare<F>>(F::bytes * F::WARPS);
    if (e != cudaSuccess) return e;
    const long long n = static_cast<long long>(p.B) * p.H * chunks;
    k_delta_prepare<F><<<static_cast<unsigned>((n + F::WARPS - 1) / F::WARPS), F::WARPS * 32, F::bytes * F::WARPS, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t records_bytes(const Problem& p, bool gradients) {
    const int rec = gradients ? record_bytes(2, 3) : record_bytes(1, p.bf16 ? 2 : 3);
    return static_cast<size_t>(p.B) * p.H * ((p.T + C - 1) / C) * rec;
}

template <typename E, int PT, int INV>
static cudaError_t by_width(const Problem& p, uint8_t* records, cudaStream_t st) {
    if (p.d == 32) return launch<E, 32, PT, INV>(p, records, st);
    if (p.d == 64) return launch<E, 64, PT, INV>(p, records, st);
    return launch<E, 128, PT, INV>(p, records, st);
}

cudaError_t prepare(const Problem& p, bool gradients, uint8_t* records, cudaStream_t st) {
    if (p.bf16) return gradients ? by_width<bf16, 3, 2>(p, records, st) : by_width<bf16, 2, 1>(p, records, st);
    return gradients ? by_width<float, 3, 2>(p, records, st) : by_width<float, 3, 1>(p, records, st);
}

}  // namespace delta
}  // namespace hla
