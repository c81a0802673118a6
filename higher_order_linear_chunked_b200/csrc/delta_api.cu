// C ABI of the gated delta rule: argument checks, workspace sizing, launches.
// Declarations and the contract of every entry point: include/hla_delta.h.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/hla_delta.h"
#include "common.cuh"
#include "delta.h"

namespace {

constexpr int kDeltaAbiVersion = 1;
constexpr int kMaxTokens = 0x7fffffff - 63;   // rounded up to blocks of 64 still an int

bool misaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

bool width_ok(int d) { return d == 32 || d == 64 || d == 128; }

hla_status_t check_shape(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv) {
    if (dtype != HLA_F32 && dtype != HLA_BF16) return HLA_ERR_DTYPE;
    if (B < 1 || Hk < 1 || H < 1 || T < 1 || d < 1 || dv < 1) return HLA_ERR_SHAPE;
    if ((long long)B * H > (1LL << 24) || (long long)B * H * T >= (1LL << 31)) return HLA_ERR_SHAPE;
    if (T > kMaxTokens || H % Hk != 0) return HLA_ERR_SHAPE;
    if (!width_ok(d) || !width_ok(dv)) return HLA_ERR_UNSUPPORTED;
    return HLA_OK;
}

hla_status_t check_norm(hla_dtype_t dtype, long long rows, int C, int groups, int flags) {
    if (dtype != HLA_F32 && dtype != HLA_BF16) return HLA_ERR_DTYPE;
    if (rows < 1 || rows >= (1LL << 31) || C < 1 || groups < 1 || C % groups != 0) return HLA_ERR_SHAPE;
    if (rows * C >= (1LL << 40) || rows * groups >= (1LL << 33)) return HLA_ERR_SHAPE;   // 8 groups a block
    if (C / groups > hla::gnorm::kMaxWidth) return HLA_ERR_UNSUPPORTED;
    if (flags & ~(HLA_NORM_CENTER | HLA_NORM_SILU)) return HLA_ERR_UNSUPPORTED;
    return HLA_OK;
}

hla::delta::Problem sizes(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv) {
    hla::delta::Problem p{};
    p.bf16 = dtype == HLA_BF16;
    p.B = B; p.Hk = Hk; p.H = H; p.T = T; p.d = d; p.dv = dv;
    return p;
}

size_t forward_workspace(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv) {
    return hla::kStatusBytes + hla::delta::forward_bytes(sizes(dtype, B, Hk, H, T, d, dv));
}

}  // namespace

extern "C" {

int hla_delta_abi_version(void) { return kDeltaAbiVersion; }

size_t hla_delta_workspace_bytes(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv) {
    if (check_shape(dtype, B, Hk, H, T, d, dv) != HLA_OK) return 0;
    return forward_workspace(dtype, B, Hk, H, T, d, dv);
}

int hla_delta_kernel_launches(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv) {
    if (check_shape(dtype, B, Hk, H, T, d, dv) != HLA_OK) return 0;
    return hla::delta::forward_launches(sizes(dtype, B, Hk, H, T, d, dv));
}

hla_status_t hla_delta_forward(const void* q, const void* k, const void* v, const float* g, const float* beta,
                               const float* state_in, const int* lengths, void* o, float* state_out, int B,
                               int Hk, int H, int T, int d, int dv, hla_dtype_t dtype, hla_layout_t layout,
                               float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (!q || !k || !v || !g || !beta || !o) return HLA_ERR_NULL;
    const hla_status_t s = check_shape(dtype, B, Hk, H, T, d, dv);
    if (s != HLA_OK) return s;
    if (layout != HLA_BHTD && layout != HLA_BTHD) return HLA_ERR_UNSUPPORTED;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
        misaligned(state_in, 16) || misaligned(state_out, 16) || misaligned(g, 4) || misaligned(beta, 4) ||
        misaligned(lengths, 4))
        return HLA_ERR_ALIGN;
    if (!workspace) return HLA_ERR_WORKSPACE;
    if (misaligned(workspace, 16)) return HLA_ERR_ALIGN;
    if (workspace_bytes < forward_workspace(dtype, B, Hk, H, T, d, dv)) return HLA_ERR_WORKSPACE;
    const hla::delta::Problem p{q, k, v, g, beta, state_in, lengths, o, state_out, B, Hk, H, T, d, dv,
                                dtype == HLA_BF16, layout == HLA_BTHD, scale, static_cast<int*>(workspace)};
    void* body = static_cast<char*>(workspace) + hla::kStatusBytes;
    return hla::delta::forward(p, body, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HLA_OK : HLA_ERR_CUDA;
}

hla_status_t hla_delta_step(float* state, const void* q, const void* k, const void* v, const float* g,
                            const float* beta, void* o, int B, int Hk, int H, int d, int dv, hla_dtype_t dtype,
                            float scale, void* stream) {
    if (!state || !q || !k || !v || !g || !beta || !o) return HLA_ERR_NULL;
    const hla_status_t s = check_shape(dtype, B, Hk, H, 1, d, dv);
    if (s != HLA_OK) return s;
    if (misaligned(state, 16) || misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
        misaligned(g, 4) || misaligned(beta, 4))
        return HLA_ERR_ALIGN;
    const hla::delta::Problem p{q, k, v, g, beta, state, nullptr, o, state, B, Hk, H, 1, d, dv,
                                dtype == HLA_BF16, false, scale, nullptr};
    return hla::delta::step(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HLA_OK : HLA_ERR_CUDA;
}

size_t hla_delta_backward_workspace_bytes(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv) {
    if (check_shape(dtype, B, Hk, H, T, d, dv) != HLA_OK) return 0;
    return hla::kStatusBytes + hla::delta::backward_bytes(sizes(dtype, B, Hk, H, T, d, dv));
}

int hla_delta_backward_kernel_launches(hla_dtype_t dtype, int B, int Hk, int H, int T, int d, int dv) {
    if (check_shape(dtype, B, Hk, H, T, d, dv) != HLA_OK) return 0;
    return hla::delta::backward_launches(sizes(dtype, B, Hk, H, T, d, dv));
}

hla_status_t hla_delta_backward(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                const float* state_in, const int* lengths, const void* dout,
                                const float* dstate_out, void* dq, void* dk, void* dv_out, float* dg, float* dbeta,
                                float* dstate_in, int B, int Hk, int H, int T, int d, int dv, hla_dtype_t dtype,
                                hla_layout_t layout, float scale, void* workspace, size_t workspace_bytes,
                                void* stream) {
    if (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv_out || !dg || !dbeta) return HLA_ERR_NULL;
    const hla_status_t s = check_shape(dtype, B, Hk, H, T, d, dv);
    if (s != HLA_OK) return s;
    if (layout != HLA_BHTD && layout != HLA_BTHD) return HLA_ERR_UNSUPPORTED;
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(dout, 16) ||
        misaligned(state_in, 16) || misaligned(dstate_out, 16) || misaligned(dq, 16) || misaligned(dk, 16) ||
        misaligned(dv_out, 16) || misaligned(dstate_in, 16) || misaligned(g, 4) || misaligned(beta, 4) ||
        misaligned(dg, 4) || misaligned(dbeta, 4) || misaligned(lengths, 4))
        return HLA_ERR_ALIGN;
    if (!workspace) return HLA_ERR_WORKSPACE;
    if (misaligned(workspace, 16)) return HLA_ERR_ALIGN;
    if (workspace_bytes < hla_delta_backward_workspace_bytes(dtype, B, Hk, H, T, d, dv)) return HLA_ERR_WORKSPACE;
    hla::delta::Problem p = sizes(dtype, B, Hk, H, T, d, dv);
    p.q = q; p.k = k; p.v = v; p.g = g; p.beta = beta; p.state_in = state_in; p.lengths = lengths;
    p.bthd = layout == HLA_BTHD;
    p.scale = scale;
    p.status = static_cast<int*>(workspace);
    const hla::delta::Gradients gr{dout, dstate_out, dq, dk, dv_out, dg, dbeta, dstate_in};
    void* body = static_cast<char*>(workspace) + hla::kStatusBytes;
    return hla::delta::backward(p, gr, body, static_cast<cudaStream_t>(stream)) == cudaSuccess ? HLA_OK : HLA_ERR_CUDA;
}

hla_status_t hla_group_norm_forward(const void* x, const void* gate, const float* weight, const float* bias,
                                    void* y, long long rows, int C, int groups, hla_dtype_t dtype, float eps,
                                    int flags, void* stream) {
    if (!x || !y) return HLA_ERR_NULL;
    const hla_status_t s = check_norm(dtype, rows, C, groups, flags);
    if (s != HLA_OK) return s;
    if (misaligned(x, 16) || misaligned(gate, 16) || misaligned(y, 16) || misaligned(weight, 4) ||
        misaligned(bias, 4))
        return HLA_ERR_ALIGN;
    hla::gnorm::Args a{};
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.y = y;
    a.rows = rows; a.C = C; a.groups = groups; a.eps = eps;
    a.center = (flags & HLA_NORM_CENTER) != 0; a.silu = (flags & HLA_NORM_SILU) != 0;
    return hla::gnorm::forward(a, dtype == HLA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? HLA_OK : HLA_ERR_CUDA;
}

size_t hla_group_norm_backward_workspace_bytes(hla_dtype_t dtype, long long rows, int C, int groups) {
    if (check_norm(dtype, rows, C, groups, 0) != HLA_OK) return 0;
    return sizeof(float) * 2 * (size_t)C * hla::gnorm::partial_rows(dtype == HLA_BF16, rows, C, groups);
}

hla_status_t hla_group_norm_backward(const void* x, const void* gate, const float* weight, const float* bias,
                                     const void* dy, void* dx, void* dgate, float* dweight, float* dbias,
                                     long long rows, int C, int groups, hla_dtype_t dtype, float eps, int flags,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    if (!x || !dy || !dx || (gate && !dgate)) return HLA_ERR_NULL;
    const hla_status_t s = check_norm(dtype, rows, C, groups, flags);
    if (s != HLA_OK) return s;
    if (dgate && !gate) return HLA_ERR_UNSUPPORTED;
    if (misaligned(x, 16) || misaligned(gate, 16) || misaligned(dy, 16) || misaligned(dx, 16) ||
        misaligned(dgate, 16) || misaligned(weight, 4) || misaligned(bias, 4) || misaligned(dweight, 4) ||
        misaligned(dbias, 4))
        return HLA_ERR_ALIGN;
    if (dweight || dbias) {
        if (!workspace) return HLA_ERR_WORKSPACE;
        if (misaligned(workspace, 16)) return HLA_ERR_ALIGN;
        if (workspace_bytes < hla_group_norm_backward_workspace_bytes(dtype, rows, C, groups)) return HLA_ERR_WORKSPACE;
    }
    hla::gnorm::Args a{};
    a.x = x; a.gate = gate; a.weight = weight; a.bias = bias; a.dy = dy; a.dx = dx; a.dgate = dgate;
    a.dweight = dweight; a.dbias = dbias;
    a.partial = (dweight || dbias) ? static_cast<float*>(workspace) : nullptr;
    a.rows = rows; a.C = C; a.groups = groups; a.eps = eps;
    a.center = (flags & HLA_NORM_CENTER) != 0; a.silu = (flags & HLA_NORM_SILU) != 0;
    return hla::gnorm::backward(a, dtype == HLA_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? HLA_OK : HLA_ERR_CUDA;
}

}  // extern "C"
