// decode_inst_d64_int4.cu -- decode kernels over INT4 pools for head_dim 64.
#include "decode_int4.cuh"

template cudaError_t pkv::decode::dispatch_int4<64>(const pkv::decode::Plan &, int, bool, int *, cudaStream_t,
                                                      const pkv::decode::LaunchArgs *);
template void pkv::decode::int4_shape<64>(int, int, int *, size_t *);
