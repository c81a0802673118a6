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
// 1 / (1 + e^-a).  Also for bf16 to fp32's bits, since the gradients of weight and bias are fp32 results:
// there with the approximate reciprocal (one unit in the last place; zero below a = -87.3, where silu is
// under 4e-37), which the division's own steps would slow down (16384 x 1024 gradients: 47 us, not 58).
template <typename E>
__device__ __forceinline__ float sigmoid(float a) {
    const float d = 1.f + expf(-a);
    if constexpr (sizeof(E) == 2) {
        float s;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(d));
        return s;
    } else {
        return 1.f / d;
    }
}

// n of one group in place of x; returns r.  inv: 1 / width.  Lanes past the width hold zeros before
// and after.
template <int VEC, int IT>
__device__ __forceinline__ float normalise(float (&x)[IT][VEC], const bool (&on)[IT], int L, float inv, float eps,
                                           bool center) {
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
    const float r = rsqrtf(lanes_sum(ss, L) * inv + eps);
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[i][j] *= r;
    return r;
}

constexpr int kThreads = 256;

// What a call asks for: known at compile time (FLAGS = GATE + SILU + CENTER) for the widths that come
// most, 16 bytes a lane in one vector; else (FLAGS < 0) tested as it runs.
enum { GATE = 1, SILU = 2, CENTER = 4 };
template <int FLAGS>
struct Form {
    bool gate, silu, center;
    __device__ __forceinline__ explicit Form(const Args& a)
        : gate(FLAGS < 0 ? a.gate != nullptr : (FLAGS & GATE) != 0),
          silu(FLAGS < 0 ? a.silu != 0 : (FLAGS & SILU) != 0),
          center(FLAGS < 0 ? a.center != 0 : (FLAGS & CENTER) != 0) {}
};

// Two groups to a group of lanes (2^lg lanes), both in flight at once.  I: the index type that holds
// every group's number.
template <typename E, int VEC, int IT, int FLAGS, typename I>
__global__ void __launch_bounds__(kThreads) k_group_norm(const Args a, int lg, bool wide) {
    constexpr int U = IT * VEC <= 8 ? 2 : 1;
    const Form<FLAGS> form(a);
    const I groups = static_cast<I>(a.groups), total = static_cast<I>(a.rows) * groups;
    const int width = a.width;
    const int lane = threadIdx.x & 31;
    const int L = 1 << lg, sub = lane >> lg, in = lane & (L - 1);
    const int per = 32 >> lg;                                // groups of lanes in a warp
    const I first = (static_cast<I>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (per * U) + sub;
    int column = static_cast<int>(first % groups);           // the group's place in its row
    Pack<E, VEC> rx[U][IT], rt[U][IT];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const I gi = first + u * per;
            const int e = (i * L + in) * VEC;
            if (gi < total && e < width) {
                const long long at = static_cast<long long>(gi) * width + e;
                rx[u][i].load(static_cast<const E*>(a.x) + at);
                if (form.gate) rt[u][i].load(static_cast<const E*>(a.gate) + at);
            } else {
                rx[u][i].clear();
            }
        }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const I gi = first + u * per;
        const bool live = gi < total;                        // every lane takes part in the shuffles
        const int wbase = column * width;
        column += a.advance;
        if (column >= a.groups) column -= a.groups;
        float x[IT][VEC];
        bool on[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            on[i] = live && (i * L + in) * VEC < width;
            rx[u][i].get(x[i]);
        }
        normalise<VEC, IT>(x, on, L, a.inv, a.eps, form.center);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (!on[i]) continue;
            const int e = (i * L + in) * VEC;
            float out[VEC], t[VEC], w[VEC], b[VEC];
            channel<VEC>(a.weight, wbase + e, wide, 1.f, w);
            channel<VEC>(a.bias, wbase + e, wide, 0.f, b);
            if (form.gate) rt[u][i].get(t);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float z = fmaf(x[i][j], w[j], b[j]);
                const float hot = form.gate ? t[j] : z;
                const float act = form.silu ? hot * sigmoid<E>(hot) : hot;
                out[j] = form.gate ? z * act : act;
            }
            store<E, VEC>(static_cast<E*>(a.y) + static_cast<long long>(gi) * width + e, out);
        }
    }
}

// A group of lanes keeps one group column and walks the rows slot, slot + slots, ..., the next row on
// its way while it works on one; its sums over those rows go to row `slot` of the partial sums.  Lanes
// and rows past the end hold zeros, which add nothing: such rows are normalised with eps = 1, since with
// an eps of 0 their zeros would become 0 / 0.
template <typename E, int VEC, int IT, int FLAGS>
__global__ void __launch_bounds__(kThreads, IT == 1 ? 3 : 1) k_group_norm_grad(const Args a, int lg, int slots, bool wide) {
    const Form<FLAGS> form(a);
    const int width = a.width;
    const int lane = threadIdx.x & 31;
    const int L = 1 << lg, sub = lane >> lg, in = lane & (L - 1);
    const long long sw = (static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * (32 >> lg) + sub;
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
    const float inv = a.inv;
    // every group of lanes of a warp makes the same number of rounds: shuffles need every lane
    const int rounds = static_cast<int>((a.rows + slots - 1) / slots);
    const long long step = static_cast<long long>(slots) * a.C;
    Pack<E, VEC> rx[IT], rd[IT], rt[IT];
    const auto ask = [&](long long row, long long at) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (on[i] && row < a.rows) {
                rx[i].load(static_cast<const E*>(a.x) + at + i * L * VEC);
                rd[i].load(static_cast<const E*>(a.dy) + at + i * L * VEC);
                if (form.gate) rt[i].load(static_cast<const E*>(a.gate) + at + i * L * VEC);
            } else {
                rx[i].clear();
                rd[i].clear();
                rt[i].clear();
            }
        }
    };
    long long row = slot, at = slot * a.C + wbase + in * VEC;
    ask(row, at);
    for (int n = 0; n < rounds; ++n, row += slots, at += step) {
        float x[IT][VEC], t[IT][VEC], dz[IT][VEC];
        const bool live = row < a.rows;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            rx[i].get(x[i]);
            rd[i].get(dz[i]);
            if (form.gate) rt[i].get(t[i]);
        }
        ask(row + slots, at + step);
        const float r = normalise<VEC, IT>(x, on, L, a.inv, live ? a.eps : 1.f, form.center);
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            float dg[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float z = fmaf(x[i][j], w[i][j], bb[i][j]);
                const float hot = form.gate ? t[i][j] : z;
                float act = hot, slope = 1.f;
                if (form.silu) {
                    const float s = sigmoid<E>(hot);
                    act = hot * s;
                    slope = fmaf(act, 1.f - s, s);
                }
                if (form.gate) {
                    dg[j] = dz[i][j] * z * slope;
                    dz[i][j] *= act;
                } else {
                    dz[i][j] *= slope;
                }
                dw[i][j] = fmaf(dz[i][j], x[i][j], dw[i][j]);
                db[i][j] += dz[i][j];
                dz[i][j] *= w[i][j];
                c1 = fmaf(dz[i][j], x[i][j], c1);
                if (form.center) c2 += dz[i][j];
            }
            if (form.gate && live && on[i]) store<E, VEC>(static_cast<E*>(a.dgate) + at + i * L * VEC, dg);
        }
        c1 = lanes_sum(c1, L) * inv;
        if (form.center) c2 = lanes_sum(c2, L) * inv;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (!(live && on[i])) continue;
            float dx[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float d = fmaf(-x[i][j], c1, dz[i][j]);
                dx[j] = r * (form.center ? d - c2 : d);
            }
            store<E, VEC>(static_cast<E*>(a.dx) + at + i * L * VEC, dx);
        }
    }
    if (!a.partial || !mine) return;
    float* pw = a.partial + slot * 2 * a.C + wbase;
    float* pb = pw + a.C;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
        const int e = (i * L + in) * VEC;
        if (!on[i]) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            pw[e + j] = dw[i][j];
            pb[e + j] = db[i][j];
        }
    }
}

// Column sums of the partial rows, in a fixed order: 32 columns a block, a warp to every 32nd row.
__global__ void __launch_bounds__(1024) k_group_norm_columns(const float* partial, int slots, int C, float* dweight,
                                                             float* dbias) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const long long both = 2LL * C, c = static_cast<long long>(blockIdx.x) * 32 + lane;   // over an int from 2^30 channels on
    float sum = 0.f;
    if (c < both) {
#pragma unroll 8
        for (int r = part; r < slots; r += 32) sum += partial[static_cast<long long>(r) * 2 * C + c];
    }
    s[part][lane] = sum;
    __syncthreads();
    sum = s[lane][part];                     // column `part` of the block, its 32 sums over the lanes
    sum = lanes_sum(sum, 32);
    const long long col = static_cast<long long>(blockIdx.x) * 32 + part;
    float* out = col < C ? dweight : dbias;
    if (lane == 0 && col < both && out) out[col < C ? col : col - C] = sum;
}

struct Shape { int vec, it, lg; };

// 16 bytes a lane where the width is a multiple of that, else 8 bytes (bf16), else single elements; the
// fewest lanes that hold the group with IT vectors each.
Shape shape_of(bool is_bf16, int width) {
    const int full = is_bf16 ? 8 : 4;
    Shape s;
    s.vec = width % full == 0 ? full : (is_bf16 && width % 4 == 0 ? 4 : 1);
    const int n = (width + s.vec - 1) / s.vec;
    s.it = n <= 32 && s.vec == full ? 1 : (n <= 128 ? 4 : 16);
    s.lg = 0;
    while (s.lg < 5 && (1 << s.lg) * s.it < n) ++s.lg;
    return s;
}
// weight and bias on 16 bytes (the C ABI asks for 4 only)
bool wide_channels(const Args& a) {
    return ((reinterpret_cast<uintptr_t>(a.weight) | reinterpret_cast<uintptr_t>(a.bias)) & 15u) == 0;
}
int flags_of(const Args& a) { return (a.gate ? GATE : 0) | (a.silu ? SILU : 0) | (a.center ? CENTER : 0); }

// f.go<E, VEC, IT, FLAGS>() for a shape and a call's flags
template <typename E, int VEC, typename F>
void pick_form(int flags, F f) {
    switch (flags) {
    case 0: f.template go<E, VEC, 1, 0>(); break;
    case 1: f.template go<E, VEC, 1, 1>(); break;
    case 2: f.template go<E, VEC, 1, 2>(); break;
    case 3: f.template go<E, VEC, 1, 3>(); break;
    case 4: f.template go<E, VEC, 1, 4>(); break;
    case 5: f.template go<E, VEC, 1, 5>(); break;
    case 6: f.template go<E, VEC, 1, 6>(); break;
    default: f.template go<E, VEC, 1, 7>(); break;
    }
}
template <typename F>
void pick(bool is_bf16, const Shape& s, int flags, F f) {
    if (is_bf16) {
        if (s.vec == 8) { if (s.it == 1) pick_form<bf16, 8>(flags, f); else f.template go<bf16, 8, 4, -1>(); }
        else if (s.vec == 4) f.template go<bf16, 4, 4, -1>();
        else if (s.it == 4) f.template go<bf16, 1, 4, -1>();
        else f.template go<bf16, 1, 16, -1>();
    } else {
        if (s.vec == 4) { if (s.it == 1) pick_form<float, 4>(flags, f); else f.template go<float, 4, 4, -1>(); }
        else if (s.it == 4) f.template go<float, 1, 4, -1>();
        else f.template go<float, 1, 16, -1>();
    }
}

struct Forward {
    const Args& a;
    int lg;
    cudaStream_t st;
    template <typename E, int VEC, int IT, int FLAGS> void go() {
        const long long per = (kThreads / 32) * (32 >> lg) * (IT * VEC <= 8 ? 2 : 1);
        Args b = a;
        b.advance = (32 >> lg) % a.groups;
        const long long total = a.rows * a.groups;
        const unsigned blocks = static_cast<unsigned>((total + per - 1) / per);
        if (total + per < (1LL << 32)) k_group_norm<E, VEC, IT, FLAGS, unsigned><<<blocks, kThreads, 0, st>>>(b, lg, wide_channels(a));
        else k_group_norm<E, VEC, IT, -1, unsigned long long><<<blocks, kThreads, 0, st>>>(b, lg, wide_channels(a));
    }
};
struct Backward {
    const Args& a;
    int lg, slots;
    cudaStream_t st;
    template <typename E, int VEC, int IT, int FLAGS> void go() {
        const long long per = (kThreads / 32) * (32 >> lg);
        const long long blocks = (static_cast<long long>(slots) * a.groups + per - 1) / per;
        k_group_norm_grad<E, VEC, IT, FLAGS><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a, lg, slots, wide_channels(a));
    }
};

}  // namespace

static Args with_width(Args a) {
    a.width = a.C / a.groups;
    a.inv = 1.f / static_cast<float>(a.width);
    return a;
}

cudaError_t forward(const Args& given, bool is_bf16, cudaStream_t st) {
    const Args a = with_width(given);
    const Shape s = shape_of(is_bf16, a.C / a.groups);
    pick(is_bf16, s, flags_of(a), Forward{a, s.lg, st});
    return cudaGetLastError();
}

// About three blocks an SM walk the rows (a partial row costs 8 C bytes twice), never more slots
// than rows.
int partial_rows(bool is_bf16, long long rows, int C, int groups) {
    const Shape s = shape_of(is_bf16, C / groups);
    const long long lanes = 148LL * 3 * kThreads;
    long long slots = lanes / ((1LL << s.lg) * groups);
    if (slots < 1) slots = 1;
    return static_cast<int>(slots < rows ? slots : rows);
}

cudaError_t backward(const Args& given, bool is_bf16, cudaStream_t st) {
    const Args a = with_width(given);
    const Shape s = shape_of(is_bf16, a.C / a.groups);
    const int slots = partial_rows(is_bf16, a.rows, a.C, a.groups);
    pick(is_bf16, s, flags_of(a), Backward{a, s.lg, slots, st});
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.partial) return e;
    k_group_norm_columns<<<static_cast<unsigned>((2LL * a.C + 31) / 32), 1024, 0, st>>>(a.partial, slots, a.C, a.dweight, a.dbias);
    return cudaGetLastError();
}

}  // namespace gnorm
}  // namespace hla
