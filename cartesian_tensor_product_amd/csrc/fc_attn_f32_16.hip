// Attention kernels: f32 rows, head dimensions up to 16.
#include "fc_attn_kernels.h"

template void fc::attn_launch<float, 16>(const fc::AttnLaunch&, const fc::AttnArgs&, const fc::AttnPart&, hipStream_t);
