// Grouped tensor-memory kernel: 16-bit forward.
#define GU_OP G_MM
#define GU_FP8 false
#define GU_ROWM false
#define GU_MT 1
#define GU_CHAIN 0
#define GU_ANY false
#include "gu_inst.inl"
