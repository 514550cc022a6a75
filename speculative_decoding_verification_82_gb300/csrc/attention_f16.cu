// attention_f16.cu -- spec_attention's kernels for f16 queries.
#include "attention_kernel.cuh"
template cudaError_t specv::attn::launch_attention<__half>(const Params&, int, bool, bool, int, cudaStream_t);
