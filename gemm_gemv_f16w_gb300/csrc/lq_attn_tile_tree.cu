// lq_attn_tree's instances of the kernels in lq_attn_tile.cu: rows that see, of
// their sequence's new tokens, those that their masks name. A translation unit of
// its own, so that both are compiled side by side and lq_attn_paged's kernels stay
// without the masks' instructions.
#define LQ_ATTN_TREE 1
#include "lq_attn_tile.cu"
