// ff_pair.h -- large products on pairs of CTAs (ff_pair.cu).
#pragma once
#include "ff_gemm.h"

namespace alx {

// Runs the product; false where the operands cannot be mapped or the
// combination of layouts is none that an operator uses.
bool ff_pair_product(const FfProduct& p, cudaStream_t s, cudaError_t* err);

}  // namespace alx
