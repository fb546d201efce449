// gated_scan_bf16.cu -- the gated scan in bf16 storage.
#define LA_SCAN_T __nv_bfloat16
#define LA_SCAN_SCRATCH gated_scan_scratch_bf16
#include "gated_scan_impl.cuh"
