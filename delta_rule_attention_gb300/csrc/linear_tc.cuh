// The tensor-core passes of the attention with a decay (decay_attn_tc.cu), and what they
// share with the others (decay_attn.cu).
#pragma once

#include "linear.cuh"

namespace falcon {

int* device_error_word_of_current();  // api.cu

constexpr int kDecayTcChunk = 128;
constexpr int kDecayTcBlocks = 152;  // one for each SM, each taking runs in turn
// One pass, p.runs in chunks of kDecayTcChunk; false where the tensors do not fit it.
bool decay_tc_pass(const DecayPass& p, cudaError_t* status, cudaStream_t stream);
cudaError_t launch_decay_join(const DecayPass& p, cudaStream_t stream);

}  // namespace falcon
