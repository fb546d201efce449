// gated_scan_bwd_bf16.cu -- the gated scan's backward pass in bf16 storage.
#define LA_SCAN_T __nv_bfloat16
#define LA_SCAN_BWD true
#include "gated_scan_impl.cuh"
