// Attention over a shared prefix for head_dim 64 (attn_prefix.cuh).
#include "attn_prefix.cuh"

namespace rmsattn {

const PrefixEntry* prefix_kernels_64(int* n) {
    using namespace prefix;
    static const PrefixEntry table[] = {entry<Shape<64, 1>>(1), entry<Shape<64, 1>>(2),
                                        entry<Shape<64, 2>>(1), entry<Shape<64, 2>>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
