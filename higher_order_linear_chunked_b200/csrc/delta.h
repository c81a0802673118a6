// Gated delta rule and group norm: declarations used by their C ABI layer (delta_api.cu).
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace hla {
namespace delta {

// One call: its tensors, laid out [B][heads][T][..] or, with bthd, [B][T][heads][..], and their sizes.
struct Problem {
    const void *q, *k, *v;
    const float *g, *beta;
    const float* state_in;   // [B*H][d][dv] or null
    const int* lengths;      // [B] or null
    void* o;
    float* state_out;        // [B*H][d][dv] or null
    int B, Hk, H, T, d, dv;
    bool bf16;
    bool bthd;
    float scale;
    int* status;             // the workspace's status word, which prepare() clears; null without a workspace
};

// Chunk by chunk on the tensor cores (delta_forward.cu), with forward_bytes() of workspace.
size_t forward_bytes(const Problem& p);
int forward_launches(const Problem& p);
cudaError_t forward(const Problem& p, void* ws, cudaStream_t st);

// The chunks' records (delta_prepare.cu); gradients: the form that the backward pass reads.  The first
// kernel of every call with a workspace: it clears the status word.
size_t records_bytes(const Problem& p, bool gradients);
cudaError_t prepare(const Problem& p, bool gradients, uint8_t* records, cudaStream_t st);

// How a sequence is cut (delta_fold.cu), in a forward call or for the gradients' two walks: `count`
// segments of `chunks` chunks (1: not at all), and the floats of the segments' summaries and of the
// states before them.
struct Segments {
    int count, chunks;
    size_t sums, starts;
};
Segments segments(const Problem& p, bool gradients);
// Value columns of a block of the gradients' two walks over `walked` heads (times segments).
int gradient_columns(const Problem& p, long long walked);
// Whether those two walks, of `blocks` blocks each, run side by side.
bool gradient_walks_beside(const Problem& p, long long blocks);
// The states between the segments, from the first on: sums [BH][count - 1][d][dv | d] holds (B | A) of
// every segment but the last (the first one's B from the given state), first the given state or null.
// With back: from the last on, S = A^T S' + back [BH][count][d][dv].  out: [BH][count][d][dv].
cudaError_t fold(const Problem& p, const Segments& g, const float* sums, const float* back, const float* first,
                 float* out, cudaStream_t st);

// The forward walk for the gradients, with the records in their form: the segments' summaries (sums for
// fold()); and the state before each block of block_chunks chunks [BH][blocks][d][dv] and each token's
// error R [BH][T][dv], from the states before the segments (or before the first token: one segment).
cudaError_t summarize(const Problem& p, const Segments& g, const uint8_t* records, float* sums, cudaStream_t st);
cudaError_t store_states(const Problem& p, const Segments& g, const uint8_t* records, const float* first, float* states,
                         float* errors, int block_chunks, cudaStream_t st);

// Gradients (delta_backward.cu).  dstate_out: the gradient at the last state, or null; dstate_in: the
// one at the first state, or null when it is not wanted.
struct Gradients {
    const void* dout;
    const float* dstate_out;
    void *dq, *dk, *dv;
    float *dg, *dbeta, *dstate_in;
};
size_t backward_bytes(const Problem& p);
int backward_launches(const Problem& p);
cudaError_t backward(const Problem& p, const Gradients& gr, void* ws, cudaStream_t st);

// Decoding (delta_step.cu): one token, the state at state_out in place; q, k [B][Hk][d], v, o [B][H][dv].
cudaError_t step(const Problem& p, cudaStream_t st);

}  // namespace delta

namespace gnorm {

struct Args {
    const void *x, *gate, *dy;
    const float *weight, *bias;
    void *y, *dx, *dgate;
    float *dweight, *dbias, *partial;
    long long rows;
    int C, groups, center, silu;
    float eps;
    // filled in on the way to the kernels: channels of a group and their reciprocal, and how far a
    // row's groups move on from one of a warp's sets of groups to the next
    int width, advance;
    float inv;
};

constexpr int kMaxWidth = 512;   // channels of a group

cudaError_t forward(const Args& a, bool bf16, cudaStream_t st);
// rows of partial column sums that backward() writes (each 2 C floats)
int partial_rows(bool bf16, long long rows, int C, int groups);
cudaError_t backward(const Args& a, bool bf16, cudaStream_t st);

}  // namespace gnorm
}  // namespace hla
