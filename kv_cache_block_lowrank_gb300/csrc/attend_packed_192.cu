// attend_packed_192.cu -- the packed cache's attention for heads of 192 elements.
#include "attend_packed_tc.cuh"

namespace hss {
namespace packed {

template <>
hss_status launch_head_dim<192>(const Params& p, const Params* many, int n_tiles, int32_t* flags,
                                cudaStream_t stream) {
    if (many != nullptr) return launch_many<192>(*many, p, flags, stream);
    return n_tiles == 1 ? launch_rows<192, 1>(p, stream) : launch_rows<192, 2>(p, stream);
}

}  // namespace packed
}  // namespace hss
