// qcache_attend.h for codes of 8 bits and fp16 queries.
#include "qcache_attend.h"

namespace seedlm {
namespace qattend {
int run_8(const Args& p, hipStream_t s) { return run<8, false>(p, s); }
}  // namespace qattend
}  // namespace seedlm
