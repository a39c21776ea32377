// qcache_attend.h for codes of 4 bits and fp32 queries.
#include "qcache_attend.h"

namespace seedlm {
namespace qattend {
int run_4_wide(const Args& p, hipStream_t s) { return run<4, true>(p, s); }
}  // namespace qattend
}  // namespace seedlm
