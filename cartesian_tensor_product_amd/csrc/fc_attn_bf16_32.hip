// Attention kernels: bf16 rows, head dimensions up to 32.
#include "fc_attn_kernels.h"

template void fc::attn_launch<fc::bf16, 32>(const fc::AttnLaunch&, const fc::AttnArgs&, const fc::AttnPart&, hipStream_t);
