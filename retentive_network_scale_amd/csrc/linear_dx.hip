// The tiled product (dx = dz w): see linear_mm.hpp.
#include "linear_mm.hpp"

hipError_t ret::mm_dx(MmArgs a, void *ws, hipStream_t st) { return product<true, false>(a, ws, st); }
