// Attention over a shared prefix for head_dim 128 (attn_prefix.cuh).
#include "attn_prefix.cuh"

namespace rmsattn {

const PrefixEntry* prefix_kernels_128(int* n) {
    using namespace prefix;
    static const PrefixEntry table[] = {entry<Shape<128, 1>>(1), entry<Shape<128, 1>>(2),
                                        entry<Shape<128, 2>>(1), entry<Shape<128, 2>>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
