// dl_scan_rwkv6.hip -- RWKV6 instantiations of the sequence-scan kernels.
#include "dl_scan_launch.h"

namespace dl {

hipError_t launch_scan_rwkv6(int dtype, bool backward, const ScanArgs &a, hipStream_t st)
{
    return scan_launch<RWKV6>(dtype, backward, a, st);
}

} // namespace dl
