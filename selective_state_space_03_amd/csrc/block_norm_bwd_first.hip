// The block norm's backward with the gate ahead of the norm.
#include "block_norm_bwd_impl.h"

template hipError_t ssm::run_norm_bwd<true>(const NormArgs&, const NormBwdShape&, hipStream_t);
