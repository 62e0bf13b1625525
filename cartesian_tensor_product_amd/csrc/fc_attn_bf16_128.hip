// Attention kernels: bf16 rows, head dimensions up to 128.
#include "fc_attn_kernels.h"

template void fc::attn_launch<fc::bf16, 128>(const fc::AttnLaunch&, const fc::AttnArgs&, const fc::AttnPart&, hipStream_t);
