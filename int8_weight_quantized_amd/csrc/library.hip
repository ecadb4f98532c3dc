// library.hip -- the one translation unit of libck_int8.so: the INT8 linear
// layer, then the decode-step operators, which use its host helpers (status,
// device check, launch) and device helpers (conversions, waits).
#include "ck_int8.hip"

#include "decode_common.hip"
#include "qk_norm_rope.hip"
#include "paged_attention.hip"
#include "int4_linear.hip"
