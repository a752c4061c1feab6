// decode_inst_d64_int4.cu -- decode kernels over INT4 pools for head_dim 64.
#include "decode_int4.cuh"

template cudaError_t pkv::decode::dispatch_int4<64>(const pkv::decode::Plan &, int, bool, int *, cudaStream_t,
                                                      const pkv::decode::LaunchArgs *);
template size_t pkv::decode::int4_smem<64>(int);
