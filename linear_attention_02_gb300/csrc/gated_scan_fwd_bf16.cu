// gated_scan_fwd_bf16.cu -- the gated scan's forward pass in bf16 storage.
#define LA_SCAN_T __nv_bfloat16
#define LA_SCAN_BWD false
#include "gated_scan_impl.cuh"
