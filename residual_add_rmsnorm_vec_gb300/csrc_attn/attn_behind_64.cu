// Attention behind a shared prefix for head_dim 64 (attn_attend.cuh): the shapes of
// attn_attend_64.cu.
#include "attn_attend.cuh"

namespace rmsattn {

using A = Shape<64, 1, 2, 4, 3>;
using B = Shape<64, 2, 2, 4, 3>;
using C = Shape<64, 4, 1, 4, 2>;

const AttendEntry* attend_behind_64(int* n) {
    static const AttendEntry table[] = {
        attend_entry<A, true>(1), attend_entry<A, true>(2),
        attend_entry<B, true>(1), attend_entry<B, true>(2),
        attend_entry<C, true>(1), attend_entry<C, true>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
