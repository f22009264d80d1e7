// The attention kernel over rows that begin with a prefix, each by itself (paged_attention.cu, shared_attention.cu).
#define LTK_ATTENTION_FORM kWhole
#define LTK_ATTENTION_CALL attend_whole
#include "paged_attention.cu"
