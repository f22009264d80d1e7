// The attention kernel over what rows see behind a prefix that they share (paged_attention.cu, shared_attention.cu).
#define LTK_ATTENTION_FORM kTail
#define LTK_ATTENTION_CALL attend_tail
#include "paged_attention.cu"
