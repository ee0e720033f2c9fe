// Attention over a paged cache of microscaled blocks.
#include "attention.h"

namespace cqk {

hipError_t launch_attention_mx(const AttentionArgs& a, int form, hipStream_t st) {
    return form == MXFP4 ? launch_kind<MXFP4>(a, st) : launch_kind<MXFP8>(a, st);
}

}  // namespace cqk
