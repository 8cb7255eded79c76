// Attention over the cache for head_dim 256 (attn_attend.cuh).
#include "attn_attend.cuh"

namespace rmsattn {

using A = Shape<256, 1, 1, 4, 2>;
using B = Shape<256, 2, 1, 8, 1>;

const AttendEntry* attend_kernels_256(int* n) {
    static const AttendEntry table[] = {
        attend_entry<A>(1), attend_entry<A>(2),
        attend_entry<B>(1), attend_entry<B>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
