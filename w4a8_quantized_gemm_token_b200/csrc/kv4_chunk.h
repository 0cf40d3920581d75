// kv4_chunk.h -- what kv4_attn.cu calls of kv4_chunk.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace qk {

struct Kv4Args;
size_t kv4_chunk_workspace(int64_t D);
cudaError_t launch_kv4_chunk(const Kv4Args& a, cudaStream_t s);

}  // namespace qk
