// gated_scan_fwd_f32.cu -- the gated scan's forward pass in fp32 storage.
#define LA_SCAN_T float
#define LA_SCAN_BWD false
#include "gated_scan_impl.cuh"
