// Dropout, residual add and LayerNorm over bfloat16 rows.
#include "ln_drop.cuh"

template bool gbattn::launch_ln_drop<__nv_bfloat16>(const LnDropArgs&, bool, int*, unsigned long long, cudaStream_t,
                                                   cudaError_t*);
