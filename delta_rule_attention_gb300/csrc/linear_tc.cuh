// The tensor-core passes of the attention with a decay (decay_attn_tc.cu), and what they
// share with the others (decay_attn.cu).
#pragma once

#include "linear.cuh"

namespace falcon {

int* device_error_word_of_current();  // api.cu

constexpr int kDecayTcChunk = 128;
// Chunks of a run at most: the state that the reads carry through a run is added to by the
// tensor cores, which round towards zero, and where nothing decays each chunk leaves it 1.4e-6
// low (160 heads of one sign, runs of 512 chunks: o 7e-4 low, of 1024 1.4e-3; of 64 less
// than 1e-4, where its rounding to bf16 is up to 4e-3).
constexpr int kDecayTcRun = 64;
constexpr int kDecayTcBlocks = 152;  // one for each SM, each taking runs in turn
// One pass, p.runs in chunks of kDecayTcChunk; false where the tensors do not fit it.
bool decay_tc_pass(const DecayPass& p, cudaError_t* status, cudaStream_t stream);
// early: set up while the kernel before it runs.
cudaError_t launch_decay_join(const DecayPass& p, bool early, cudaStream_t stream);

// A ring of `stages` barriers that n uses went through in turn: the phase that the last
// use of barrier s completed (s < n).
__host__ __device__ constexpr int last_phase(int n, int stages, int s) {
  return (n - 1 - s) / stages;
}

// A launch that may be set up while the kernel before it on the stream runs (early): its
// kernel waits for that one (griddepcontrol.wait) before it touches what that one writes
// or reads.
template <typename... P, typename... A>
cudaError_t launch_behind(bool early, void (*kernel)(P...), unsigned grid, unsigned threads,
                          size_t shared, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(grid), c.blockDim = dim3(threads);
  c.dynamicSmemBytes = shared;
  c.stream = stream;
  cudaLaunchAttribute attr[1] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = attr;
  c.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace falcon
