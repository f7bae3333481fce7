// LayerNorm's backward pass over float32 rows.
#include "ln_bwd.cuh"

template cudaError_t gbattn::launch_ln_bwd<float>(const BwdLnArgs&, bool, int*, int*, unsigned long long, cudaStream_t);
