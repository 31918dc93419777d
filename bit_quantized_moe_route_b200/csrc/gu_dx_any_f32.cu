// Grouped tensor-memory kernel: gradient of the rows, fp32 outputs of any alignment.
#define GU_OP G_DX
#define GU_FP8 false
#define GU_ROWM false
#define GU_MT 1
#define GU_CHAIN kGuChain
#define GU_ANY true
#include "gu_inst.inl"
