// The tensor-core passes of the attention with a decay (decay_attn_tc.cu), and what they
// share with the others (decay_attn.cu).
#pragma once

#include "linear.cuh"

namespace falcon {

int* device_error_word_of_current();  // api.cu

constexpr int kDecayTcChunk = 128;
// Blocks that one wave of the card holds, by key and value channels.
int64_t decay_tc_blocks(int m, int dv);
// One pass, p.runs in chunks of kDecayTcChunk; false where the tensors do not fit it.
bool decay_tc_pass(const DecayPass& p, cudaError_t* status, cudaStream_t stream);
cudaError_t launch_decay_join(const DecayPass& p, cudaStream_t stream);

}  // namespace falcon
