// The translation unit of the recurrences and the q/k preparation: these kernels
// are compiled together with the same flags, and the parts below share the
// helpers of the first.
#include "gdn_kernels.hip"

#include <new>

#include "gdn_lru.hip"
#include "gdn_qk.hip"
