// gated_scan_bwd_f32.cu -- the gated scan's backward pass in fp32 storage.
#define LA_SCAN_T float
#define LA_SCAN_BWD true
#include "gated_scan_impl.cuh"
