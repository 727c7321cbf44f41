// dropout.cuh -- dropout whose mask is computed, not stored (dropout.cu).
#pragma once
#include "common.cuh"

namespace vae {

// y = kept(i) x scale (+ residual); kept(i) where element i's 16 bits are at least
// `threshold`. With state, seed = state[0] and offset counts from state[1].
int dropout(const void *x, int dtype, long long count, uint32_t threshold, uint64_t seed,
            uint64_t offset, const long long *state, const void *residual, void *y,
            cudaStream_t s);

}  // namespace vae
