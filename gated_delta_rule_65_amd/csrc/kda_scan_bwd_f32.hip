// Gated scan, backward, for fp32 x.
#include "kda_scan_bwd.h"

template void kda::scan_bwd_of<true>(const kda::ScanArgs&, hipStream_t);
