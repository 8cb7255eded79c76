// Attention behind a shared prefix for head_dim 256 (attn_attend.cuh): the shapes of
// attn_attend_256.cu.
#include "attn_attend.cuh"

namespace rmsattn {

using A = Shape<256, 1, 1, 4, 2>;
using B = Shape<256, 2, 1, 8, 1>;

const AttendEntry* attend_behind_256(int* n) {
    static const AttendEntry table[] = {
        attend_entry<A, true>(1), attend_entry<A, true>(2),
        attend_entry<B, true>(1), attend_entry<B, true>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
