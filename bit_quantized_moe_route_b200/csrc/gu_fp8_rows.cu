// Grouped tensor-memory kernel: 8-bit forward, many rows per expert.
#define GU_OP G_MM
#define GU_FP8 true
#define GU_ROWM true
#define GU_MT 1
#define GU_CHAIN 1
#define GU_ANY false
#include "gu_inst.inl"
