// Grouped tensor-memory kernel: 16-bit forward, fp32 outputs of any alignment.
#define GU_OP G_MM
#define GU_FP8 false
#define GU_ROWM false
#define GU_MT 1
#define GU_CHAIN kGuChain
#define GU_ANY true
#include "gu_inst.inl"
