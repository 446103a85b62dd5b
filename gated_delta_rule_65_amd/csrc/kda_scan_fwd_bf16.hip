// Gated scan, forward, for bf16 x.
#include "kda_scan_fwd.h"

template void kda::scan_fwd_of<false>(const kda::ScanArgs&, hipStream_t);
