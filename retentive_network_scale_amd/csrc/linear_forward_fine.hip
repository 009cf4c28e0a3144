// The tiled product (out = gelu(x w^T + bias) in fp32): see linear_mm.hpp.
#include "linear_mm.hpp"

hipError_t ret::mm_forward_fine(MmArgs a, void *ws, hipStream_t st) { return product<true, true, true>(a, ws, st); }
