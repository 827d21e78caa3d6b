// ops_internal.h -- launchers behind include/sparseloco_ops.h.  Arguments are
// already validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sparseloco_ops.h"

namespace sl {

// A strided batch of row-major matrices: element (i, r, c) at
// ptr + i * stride + r * ld + c elements.
struct MatrixView {
    void* ptr;
    int32_t type;  // sl_dtype
    int64_t ld, stride;
};

struct Quintic {
    float a, b, c;
};

// What the orthogonalisation starts from (x, or the momentum's inputs) and
// what its last step writes (out, or theta).
struct UpdateArgs {
    int64_t rows, cols, count;
    MatrixView x;         // sl_orthogonalize: input; sl_muon_step: the gradient
    float* momentum;      // null for sl_orthogonalize
    float grad_scale, decay;
    bool nesterov;
    MatrixView out;       // sl_orthogonalize: output; sl_muon_step: theta
    float keep, move;     // theta <- theta * keep - move * O; unused without momentum
    const Quintic* steps;
    int32_t n_steps;
    float eps;
    bool split;           // products of values held as two fp16 terms
    // The largest product of the first steps' factors |a + b q + c q^2| over the
    // squared singular values q they can meet (1e30 if one factor passes 100).
    float growth;
    float factors[SL_MAX_STEPS];  // each step's own
};

// Bytes of workspace launch_update needs.
// (update: for sl_muon_step.)
size_t update_workspace_bytes(int64_t rows, int64_t cols, int64_t count, bool split, bool update);
hipError_t launch_update(const UpdateArgs& u, void* workspace, hipStream_t stream);

struct LogprobArgs {
    const void* logits;
    int32_t type;  // sl_dtype
    int64_t ld;
    const int64_t* targets;
    int64_t rows, vocab;
    int32_t n_top;
    float *logprob, *entropy, *top_logprob;
    int32_t* top_index;
};

size_t logprob_workspace_bytes(int64_t rows, int64_t vocab, int32_t type, int32_t n_top);
hipError_t launch_logprobs(const LogprobArgs& a, void* workspace, hipStream_t stream);

}  // namespace sl
