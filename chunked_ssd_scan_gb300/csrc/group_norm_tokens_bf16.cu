// Group norm of tokens for bf16 (a translation unit of its own: the two compile side by side).
#define NORM_TOKENS_F32 0
#include "group_norm_tokens.cuh"
