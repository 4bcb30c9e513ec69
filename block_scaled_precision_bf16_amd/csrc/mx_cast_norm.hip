// mx_cast_norm.hip -- the column-wise MXFP8 casts of a root-mean-square norm's
// output: the cast kernel of mx_cast.h whose elements are (h rstd[row])
// weight[column], rounded to bf16, recomputed from h (2 bytes read instead of
// the 4 that writing and reading y would take).  The row-wise cast leaves with
// the norm itself (norm.hip), which holds whole rows.  The last rows, which the norm
// wrote last, come first: some of them are still in the last cache.  16384 x 7168: 80
// us (0.36 GB, 4.5 TB/s) right behind the norm, whose stores are still draining.
#include "launch_norm.h"
#include "mx_cast.h"

namespace mxk {

template <int FMT>
static hipError_t launch_fmt(const MxArgs &a, const GroupTable *gt, hipStream_t s)
{
    return gt ? launch_one<OP_NORM, FMT, false, true, false, true, true>(a, gt, s)
              : launch_one<OP_NORM, FMT, false, true, false, false, false>(a, nullptr, s);
}

hipError_t launch_mx_cast_norm(unsigned fmt, const MxArgs &a, const GroupTable *gt, hipStream_t s)
{
    switch (fmt) {
    case 0u: return launch_fmt<0>(a, gt, s);
    case kFmtE5M2: return launch_fmt<kFmtE5M2>(a, gt, s);
    case kFmtRoundUp: return launch_fmt<kFmtRoundUp>(a, gt, s);
    case kFmtE5M2 | kFmtRoundUp: return launch_fmt<kFmtE5M2 | kFmtRoundUp>(a, gt, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace mxk
