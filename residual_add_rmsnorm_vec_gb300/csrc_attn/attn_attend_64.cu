// Attention over the cache for head_dim 64 (attn_attend.cuh).
#include "attn_attend.cuh"

namespace rmsattn {

using A = Shape<64, 1, 2, 4, 3>;
using B = Shape<64, 2, 2, 4, 3>;
using C = Shape<64, 4, 1, 4, 2>;

const AttendEntry* attend_kernels_64(int* n) {
    static const AttendEntry table[] = {
        attend_entry<A>(1), attend_entry<A>(2),
        attend_entry<B>(1), attend_entry<B>(2),
        attend_entry<C>(1), attend_entry<C>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
