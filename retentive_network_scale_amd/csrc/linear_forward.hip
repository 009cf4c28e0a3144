// The tiled product (out = x w^T): see linear_mm.hpp.
#include "linear_mm.hpp"

hipError_t ret::mm_forward(MmArgs a, void *ws, hipStream_t st) {
  return a.f.fine() ? mm_forward_fine(a, ws, st) : product<true, true>(a, ws, st);
}
