// dl_scan_kda.hip -- KDA instantiations of the sequence-scan kernels.
#include "dl_scan_launch.h"

namespace dl {

hipError_t launch_scan_kda(int dtype, bool backward, const ScanArgs &a, hipStream_t st)
{
    return scan_launch<KDA>(dtype, backward, a, st);
}

} // namespace dl
