// attn_prompt_kernels.hip -- causal attention of packed rows.
#include <hip/hip_runtime.h>

#include "attn_internal.h"
