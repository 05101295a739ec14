// gdn_wait.cuh -- when a wait inside a kernel is given up.  What a wait waits for may take as long as
// the work in front of it (an item of a key tile's gradients: all query blocks of all query heads of its
// key head); what shows that a CTA is stuck is that nothing has moved.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

// Nothing has moved for `limit`.  `moved`, the time when something last did, may be read after `now`, and
// so be later.
GDN_HD bool stands_still(uint64_t now, uint64_t moved, uint64_t limit) {
  return (int64_t)(now - moved) > (int64_t)limit;
}

}  // namespace gdn
