// LayerNorm's backward pass over bfloat16 rows.
#include "ln_bwd.cuh"

template cudaError_t gbattn::launch_ln_bwd<__nv_bfloat16>(const BwdLnArgs&, bool, int*, int*, unsigned long long,
                                                          cudaStream_t);
