// dl_scan_gdn.hip -- GDN instantiations of the sequence-scan kernels.
#include "dl_scan_launch.h"

namespace dl {

hipError_t launch_scan_gdn(int dtype, bool backward, const ScanArgs &a, hipStream_t st)
{
    return scan_launch<GDN>(dtype, backward, a, st);
}

} // namespace dl
