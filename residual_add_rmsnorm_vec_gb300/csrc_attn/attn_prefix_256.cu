// Attention over a shared prefix for head_dim 256 (attn_prefix.cuh).
#include "attn_prefix.cuh"

namespace rmsattn {

const PrefixEntry* prefix_kernels_256(int* n) {
    using namespace prefix;
    static const PrefixEntry table[] = {entry<Shape<256, 1>>(1), entry<Shape<256, 1>>(2)};
    *n = (int)(sizeof(table) / sizeof(table[0]));
    return table;
}

}  // namespace rmsattn
