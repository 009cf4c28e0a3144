// The tiled product (dw = dz^T x): see linear_mm.hpp.
#include "linear_mm.hpp"

hipError_t ret::mm_dw(MmArgs a, void *ws, hipStream_t st) { return product<false, false>(a, ws, st); }
