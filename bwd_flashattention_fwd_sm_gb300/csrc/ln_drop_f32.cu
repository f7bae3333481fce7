// Dropout, residual add and LayerNorm over float32 rows.
#include "ln_drop.cuh"

template bool gbattn::launch_ln_drop<float>(const LnDropArgs&, bool, int*, unsigned long long, cudaStream_t,
                                           cudaError_t*);
