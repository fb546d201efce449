// gated_scan_f32.cu -- the gated scan in fp32 storage.
#define LA_SCAN_T float
#define LA_SCAN_SCRATCH gated_scan_scratch_f32
#include "gated_scan_impl.cuh"
