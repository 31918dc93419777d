// Grouped tensor-memory kernel: gradient of the rows.
#define GU_OP G_DX
#define GU_FP8 false
#define GU_ROWM false
#define GU_MT 1
#define GU_CHAIN 0
#define GU_ANY false
#include "gu_inst.inl"
