// Gated scan, forward, for fp32 x.
#include "kda_scan_fwd.h"

template void kda::scan_fwd_of<true>(const kda::ScanArgs&, hipStream_t);
