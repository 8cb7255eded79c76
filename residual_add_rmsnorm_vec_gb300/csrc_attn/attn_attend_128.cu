// Attention over the cache for head_dim 128 (attn_attend.cuh).
#include "attn_attend.cuh"

namespace rmsattn {

// For rows of a few steps, of which steps of 32 tokens would leave warps idle
// (256 x 300 tokens 38 against 49 us), and for the line (64 x 8192 149 either
// way); A where a row's clusters have 32-token steps enough (8 x 2000 10.6
// against 11.2, 16 x 4000 24.7 against 26.8).
using Short = Shape<128, 1, 1, 4, 3>;
using A = Shape<128, 1, 2, 4, 2>;
using B = Shape<128, 2, 1, 4, 3>;
using C = Shape<128, 4, 1, 4, 2>;

const AttendEntry* attend_kernels_128(int* n) {
    static const AttendEntry table[] = {
        attend_entry<Short>(1, 512), attend_entry<Short>(2, 512),
        attend_entry<A>(1), attend_entry<A>(2),
        attend_entry<B>(1), attend_entry<B>(2),
        attend_entry<C>(1), attend_entry<C>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
