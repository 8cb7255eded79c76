// Attention behind a shared prefix for head_dim 128 (attn_attend.cuh): the shapes of
// attn_attend_128.cu.
#include "attn_attend.cuh"

namespace rmsattn {

using Short = Shape<128, 1, 1, 4, 3>;
using A = Shape<128, 1, 2, 4, 2>;
using B = Shape<128, 2, 1, 4, 3>;
using C = Shape<128, 4, 1, 4, 2>;

const AttendEntry* attend_behind_128(int* n) {
    static const AttendEntry table[] = {
        attend_entry<Short, true>(1, 512), attend_entry<Short, true>(2, 512),
        attend_entry<A, true>(1), attend_entry<A, true>(2),
        attend_entry<B, true>(1), attend_entry<B, true>(2),
        attend_entry<C, true>(1), attend_entry<C, true>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
