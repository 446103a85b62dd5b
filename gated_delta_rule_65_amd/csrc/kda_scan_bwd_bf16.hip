// Gated scan, backward, for bf16 x.
#include "kda_scan_bwd.h"

template void kda::scan_bwd_of<false>(const kda::ScanArgs&, hipStream_t);
