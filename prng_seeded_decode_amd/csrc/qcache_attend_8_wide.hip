// qcache_attend.h for codes of 8 bits and fp32 queries.
#include "qcache_attend.h"

namespace seedlm {
namespace qattend {
int run_8_wide(const Args& p, hipStream_t s) { return run<8, true>(p, s); }
}  // namespace qattend
}  // namespace seedlm
