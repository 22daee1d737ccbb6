// attn_masked.hip -- the kernels of attn_core.h for rows that do not see a
// sequence's first keys: a sliding window with a few first tokens, a tree of drafts.
#include "attn_core.h"

namespace bl {

hipError_t launch_attn_masked(const AttnArgs &a, const AttnPlan &pl, int mask, hipStream_t st)
{
    if (a.dtype == DT_F32)
        return mask == ATTN_TREE ? launch_attn_parts<DT_F32, ATTN_TREE>(a, pl, st)
                                 : launch_attn_parts<DT_F32, ATTN_WINDOW>(a, pl, st);
    return mask == ATTN_TREE ? launch_attn_parts<DT_BF16, ATTN_TREE>(a, pl, st)
                             : launch_attn_parts<DT_BF16, ATTN_WINDOW>(a, pl, st);
}

} // namespace bl
