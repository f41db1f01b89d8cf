// Group norm of tokens for f32 (a translation unit of its own: the two compile side by side).
#define NORM_TOKENS_F32 1
#include "group_norm_tokens.cuh"
