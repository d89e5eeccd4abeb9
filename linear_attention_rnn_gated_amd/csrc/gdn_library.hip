// The library's one device translation unit: every kernel is compiled together
// with the same flags, and the parts below share the helpers and the kernel
// timing of the first.
#include "gdn_kernels.hip"

#include <new>

#include "gdn_lru.hip"
#include "gdn_qk.hip"
