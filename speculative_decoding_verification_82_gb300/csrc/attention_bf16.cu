// attention_bf16.cu -- spec_attention's kernels for bf16 queries.
#include "attention_kernel.cuh"
template cudaError_t specv::attn::launch_attention<__nv_bfloat16>(const Params&, int, bool, bool, int, cudaStream_t);
