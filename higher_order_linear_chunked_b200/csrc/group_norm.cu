// Group norm with an activation over channels-last rows, forward and backward.
//
//   n = (x - m) r, r = 1/sqrt(mean((x-m)^2) + eps);  z = n w + b;  y = act(z) or z act(gate)
// Backward, with dz the gradient at z and e = dz w:
//   dx = r (e - n mean(e n) - [m subtracted] mean(e)),  dw = sum_rows dz n,  db = sum_rows dz
//
// The groups of all rows lie one behind another in memory, so a group is a piece of `width`
// elements: L lanes (a power of two) hold it in registers, 16 bytes a lane where the width allows,
// and the statistics are shuffles among those lanes.  Every element is read once and written once;
// device memory bounds it (about ten flops an element).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "delta.h"

namespace hla {
namespace gnorm {
namespace {

using bf16 = __nv_bfloat16;

template <int BYTES> struct Raw;
template <> struct Raw<16> { using type = uint4; };
template <> struct Raw<8> { using type = uint2; };
template <> struct Raw<4> { using type = uint32_t; };
template <> struct Raw<2> { using type = uint16_t; };

// VEC elements as one load or store.
template <typename E, int VEC>
struct Pack {
    using R = typename Raw<sizeof(E) * VEC>::type;
    R r;
    __device__ __forceinline__ void load(const E* p) { r = *reinterpret_cast<const R*>(p); }
    __device__ __forceinline__ void clear() { r = R{}; }
    __device__ __forceinline__ void get(float (&x)[VEC]) const {
        union { R r; E e[VEC]; } u;
        u.r = r;
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = to_f32(u.e[i]);
    }
};
__device__ __forceinline__ void round_to(float& e, float x) { e = x; }
__device__ __forceinline__ void round_to(bf16& e, float x) { e = __float2bfloat16_rn(x); }
template <typename E, int VEC>
__device__ __forceinline__ void store(E* p, const float (&x)[VEC]) {
    using R = typename Raw<sizeof(E) * VEC>::type;
    union U { R r; E e[VEC]; __device__ U() {} } u;
#pragma unroll
    for (int i = 0; i < VEC; ++i) round_to(u.e[i], x[i]);
    *reinterpret_cast<R*>(p) = u.r;
}
// VEC floats of a per-channel vector (4-byte aligned only when VEC is 1; its base is 16-byte aligned
// when `wide`), or `none` where there is no vector.
template <int VEC>
__device__ __forceinline__ void channel(const float* p, int at, bool wide, float none, float (&x)[VEC]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = none;
    } else if (VEC % 4 == 0 && wide) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + at + i);
            x[i] = v.x; x[i + 1 < VEC ? i + 1 : i] = v.y; x[i + 2 < VEC ? i + 2 : i] = v.z; x[i + 3 < VEC ? i + 3 : i] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) x[i] = p[at + i];
    }
}

__device__ __forceinline__ float lanes_sum(float x, int L) {
    for (int w = 1; w < L; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    return x;
}
// 1 / (1 + e^-a): for fp32 by the library's exponential and division, for bf16 (a result of eight
// bits) by the approximate ones, whose 2^-21 it does not see.
template <typename E>
__device__ __forceinline__ float sigmoid(float a) {
    if constexpr (sizeof(E) == 2) return __fdividef(1.f, 1.f + __expf(-a));
    else return 1.f / (1.f + expf(-a));
}

// n of one group in place of x; returns r.  Lanes past the width hold zeros before and after.
template <int VEC, int IT>
__device__ __forceinline__ float normalise(float (&x)[IT][VEC], const bool (&on)[IT], int L, int width, float eps,
                                           int center) {
    const float inv = 1.f / static_cast<float>(width);
    if (center) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) s += x[i][j];
        const float m = lanes_sum(s, L) * inv;
#pragma unroll
        for (int i = 0; i < IT; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) x[i][j] = on[i] ? x[i][j] - m : 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(x[i][j], x[i][j], ss);
    const float r = 1.f / sqrtf(lanes_sum(ss, L) * inv + eps);
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[i][j] *= r;
    return r;
}

constexpr int kThreads = 256;

// Two groups to a group of lanes, half the grid apart in memory order (both in flight at once).
template <typename E, int VEC, int IT>
__global__ void __launch_bounds__(kThreads) k_group_norm(const Args a, int L, bool wide) {
    constexpr int U = IT * VEC <= 8 ? 2 : 1;
    const int width = a.C / a.groups;
    const long long total = a.rows * a.groups;
    const int lane = threadIdx.x & 31;
    const int sub = lane / L, in = lane % L;
    const int per = 32 / L;                                  // groups of lanes in a warp
    const long long first = (static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (per * U) + sub;
    Pack<E, VEC> rx[U][IT], rt[U][IT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const long long gi = first + u * per;
            const int e = (i * L + in) * VEC;
            if (gi < total && e < width) {
                rx[u][i].load(static_cast<const E*>(a.x) + gi * width + e);
                if (a.gate) rt[u][i].load(static_cast<const E*>(a.gate) + gi * width + e);
            } else {
                rx[u][i].clear();
            }
        }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long gi = first + u * per;
        const bool live = gi < total;                        // every lane takes part in the shuffles
        const int wbase = static_cast<int>((live ? gi : 0) % a.groups) * width;
        float x[IT][VEC];
        bool on[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            on[i] = live && (i * L + in) * VEC < width;
            rx[u][i].get(x[i]);
        }
        normalise<VEC, IT>(x, on, L, width, a.eps, a.center);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (!on[i]) continue;
            const int e = (i * L + in) * VEC;
            float out[VEC], t[VEC], w[VEC], b[VEC];
            channel<VEC>(a.weight, wbase + e, wide, 1.f, w);
            channel<VEC>(a.bias, wbase + e, wide, 0.f, b);
            if (a.gate) rt[u][i].get(t);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float z = fmaf(x[i][j], w[j], b[j]);
                const float hot = a.gate ? t[j] : z;
                const float act = a.silu ? hot * sigmoid<E>(hot) : hot;
                out[j] = a.gate ? z * act : act;
            }
            store<E, VEC>(static_cast<E*>(a.y) + gi * width + e, out);
        }
    }
}

// A group of lanes keeps one group column and walks the rows slot, slot + slots, ..., the next row on
// its way while it works on one; its sums over those rows go to row `slot` of the partial sums.
template <typename E, int VEC, int IT>
__global__ void __launch_bounds__(kThreads) k_group_norm_grad(const Args a, int L, int slots, bool wide) {
    const int width = a.C / a.groups;
    const int lane = threadIdx.x & 31;
    const int sub = lane / L, in = lane % L;
    const long long sw = (static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (32 / L) + sub;
    const long long slot = sw / a.groups;
    const int wbase = static_cast<int>(sw % a.groups) * width;
    const bool mine = slot < slots;
    float w[IT][VEC], bb[IT][VEC], dw[IT][VEC], db[IT][VEC];
    bool on[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int e = (i * L + in) * VEC;
        on[i] = mine && e < width;
        channel<VEC>(on[i] ? a.weight : nullptr, wbase + e, wide, 1.f, w[i]);
        channel<VEC>(on[i] ? a.bias : nullptr, wbase + e, wide, 0.f, bb[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.f;
    }
    const float inv = 1.f / static_cast<float>(width);
    // every group of lanes of a warp makes the same number of rounds: shuffles need every lane
    const long long rounds = (a.rows + slots - 1) / slots;
    Pack<E, VEC> rx[IT], rd[IT], rt[IT];
    const auto ask = [&](long long row) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (on[i] && row < a.rows) {
                const long long at = row * a.C + wbase + (i * L + in) * VEC;
                rx[i].load(static_cast<const E*>(a.x) + at);
                rd[i].load(static_cast<const E*>(a.dy) + at);
                if (a.gate) rt[i].load(static_cast<const E*>(a.gate) + at);
            } else {
                rx[i].clear();
                rd[i].clear();
                rt[i].clear();
            }
        }
    };
    ask(slot);
    for (long long n = 0; n < rounds; ++n) {
        const long long row = n * slots + slot;
        const long long base = row * a.C + wbase;
        float x[IT][VEC], t[IT][VEC], dz[IT][VEC];
        bool here[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            here[i] = on[i] && row < a.rows;
            rx[i].get(x[i]);
            rd[i].get(dz[i]);
            if (a.gate) rt[i].get(t[i]);
        }
        ask(row + slots);
        const float r = normalise<VEC, IT>(x, here, L, width, a.eps, a.center);
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float dg[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float z = fmaf(x[i][j], w[i][j], bb[i][j]);
                const float hot = a.gate ? t[i][j] : z;
                float act = hot, slope = 1.f;
                if (a.silu) {
                    const float s = sigmoid<E>(hot);
                    act = hot * s;
                    slope = s * (1.f + hot * (1.f - s));
                }
                if (a.gate) {
                    dg[j] = dz[i][j] * z * slope;
                    dz[i][j] *= act;
                } else {
                    dz[i][j] *= slope;
                }
                if (here[i]) {
                    dw[i][j] = fmaf(dz[i][j], x[i][j], dw[i][j]);
                    db[i][j] += dz[i][j];
                }
                dz[i][j] = here[i] ? dz[i][j] * w[i][j] : 0.f;
                c1 = fmaf(dz[i][j], x[i][j], c1);
                c2 += dz[i][j];
            }
            if (a.gate && here[i]) store<E, VEC>(static_cast<E*>(a.dgate) + base + (i * L + in) * VEC, dg);
        }
        c1 = lanes_sum(c1, L) * inv;
        c2 = a.center ? lanes_sum(c2, L) * inv : 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (!here[i]) continue;
            float dx[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) dx[j] = r * (dz[i][j] - x[i][j] * c1 - c2);
            store<E, VEC>(static_cast<E*>(a.dx) + base + (i * L + in) * VEC, dx);
        }
    }
    if (!a.partial || !mine) return;
    float* pw = a.partial + slot * 2 * a.C + wbase;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int e = (i * L + in) * VEC;
        if (!on[i]) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            pw[e + j] = dw[i][j];
            pw[a.C + e + j] = db[i][j];
        }
    }
}

// Column sums of the partial rows, in a fixed order: 32 columns a block, 8 threads a column.
__global__ void __launch_bounds__(256) k_group_norm_columns(const float* partial, int slots, int C, float* dweight,
                                                            float* dbias) {
    __shared__ float s[8][33];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
    float* out = c < C ? dweight : dbias;
    const int col = c < C ? c : c - C;
    float sum = 0.f;
    if (c < 2 * C && out)
        for (int r = part; r < slots; r += 8) sum += partial[static_cast<long long>(r) * 2 * C + c];
    s[part][threadIdx.x & 31] = sum;
    __syncthreads();
    if (part == 0 && c < 2 * C && out) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t += s[i][threadIdx.x & 31];
        out[col] = t;
    }
}

struct Shape { int vec, it, L; };

// 16 bytes a lane where the width is a multiple of that, else 8 bytes, else single elements; the
// fewest lanes that hold the group with IT vectors each.
Shape shape_of(bool is_bf16, int width) {
    const int full = is_bf16 ? 8 : 4;
    Shape s;
    s.vec = width % full == 0 ? full : (is_bf16 && width % 4 == 0 ? 4 : 1);
    const int n = (width + s.vec - 1) / s.vec;
    s.it = n <= 32 ? 1 : (n <= 128 ? 4 : 16);
    s.L = 1;
    while (s.L < 32 && s.L * s.it < n) s.L *= 2;
    return s;
}

// weight and bias on 16 bytes (the C ABI asks for 4 only)
bool wide_channels(const Args& a) {
    return ((reinterpret_cast<uintptr_t>(a.weight) | reinterpret_cast<uintptr_t>(a.bias)) & 15u) == 0;
}

template <typename E, int VEC, int IT>
void run_forward(const Args& a, int L, cudaStream_t st) {
    const long long per = (kThreads / 32) * (32 / L) * (IT * VEC <= 8 ? 2 : 1);
    const long long blocks = (a.rows * a.groups + per - 1) / per;
    k_group_norm<E, VEC, IT><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a, L, wide_channels(a));
}
template <typename E, int VEC, int IT>
void run_backward(const Args& a, int L, int slots, cudaStream_t st) {
    const long long per = (kThreads / 32) * (32 / L);
    const long long blocks = (static_cast<long long>(slots) * a.groups + per - 1) / per;
    k_group_norm_grad<E, VEC, IT><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a, L, slots, wide_channels(a));
}

template <typename F>
void pick(bool is_bf16, const Shape& s, F f) {
    if (is_bf16) {
        if (s.vec == 8) { if (s.it == 1) f.template go<bf16, 8, 1>(); else f.template go<bf16, 8, 4>(); }
        else if (s.vec == 4) { if (s.it == 1) f.template go<bf16, 4, 1>(); else f.template go<bf16, 4, 4>(); }
        else if (s.it == 1) f.template go<bf16, 1, 1>();
        else if (s.it == 4) f.template go<bf16, 1, 4>();
        else f.template go<bf16, 1, 16>();
    } else {
        if (s.vec == 4) { if (s.it == 1) f.template go<float, 4, 1>(); else f.template go<float, 4, 4>(); }
        else if (s.it == 1) f.template go<float, 1, 1>();
        else if (s.it == 4) f.template go<float, 1, 4>();
        else f.template go<float, 1, 16>();
    }
}

struct Forward {
    const Args& a;
    int L;
    cudaStream_t st;
    template <typename E, int VEC, int IT> void go() { run_forward<E, VEC, IT>(a, L, st); }
};
struct Backward {
    const Args& a;
    int L, slots;
    cudaStream_t st;
    template <typename E, int VEC, int IT> void go() { run_backward<E, VEC, IT>(a, L, slots, st); }
};

}  // namespace

cudaError_t forward(const Args& a, bool is_bf16, cudaStream_t st) {
    const Shape s = shape_of(is_bf16, a.C / a.groups);
    pick(is_bf16, s, Forward{a, s.L, st});
    return cudaGetLastError();
}

// About four blocks an SM walk the rows (a partial row costs 8 C bytes twice), never more slots
// than rows.
int partial_rows(bool is_bf16, long long rows, int C, int groups) {
    const Shape s = shape_of(is_bf16, C / groups);
    const long long lanes = 148LL * 4 * kThreads;
    long long slots = lanes / (static_cast<long long>(s.L) * groups);
    if (slots < 1) slots = 1;
    return static_cast<int>(slots < rows ? slots : rows);
}

cudaError_t backward(const Args& a, bool is_bf16, cudaStream_t st) {
    const Shape s = shape_of(is_bf16, a.C / a.groups);
    const int slots = partial_rows(is_bf16, a.rows, a.C, a.groups);
    pick(is_bf16, s, Backward{a, s.L, slots, st});
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.partial) return e;
    k_group_norm_columns<<<(2 * a.C + 31) / 32, 256, 0, st>>>(a.partial, slots, a.C, a.dweight, a.dbias);
    return cudaGetLastError();
}

}  // namespace gnorm
}  // namespace hla
