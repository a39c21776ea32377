// qcache_attend.h for codes of 4 bits and fp16 queries.
#include "qcache_attend.h"

namespace seedlm {
namespace qattend {
int run_4(const Args& p, hipStream_t s) { return run<4, false>(p, s); }
}  // namespace qattend
}  // namespace seedlm
