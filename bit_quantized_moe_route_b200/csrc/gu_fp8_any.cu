// Grouped tensor-memory kernel: 8-bit forward, any alignment.
#define GU_OP G_MM
#define GU_FP8 true
#define GU_ROWM false
#define GU_MT 1
#define GU_CHAIN 1
#define GU_ANY true
#include "gu_inst.inl"
