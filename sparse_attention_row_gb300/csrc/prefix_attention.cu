// The attention kernel over prefixes that rows share, joined with what they see behind them (paged_attention.cu,
// shared_attention.cu).
#define LTK_ATTENTION_FORM kShared
#define LTK_ATTENTION_CALL attend_shared
#include "paged_attention.cu"
