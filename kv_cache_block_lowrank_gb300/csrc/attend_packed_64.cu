// attend_packed_64.cu -- the packed cache's attention for heads of 64 elements.
#include "attend_packed_tc.cuh"

namespace hss {
namespace packed {

template <>
hss_status launch_head_dim<64>(const Params& p, const Params* many, int n_tiles, int32_t* flags,
                                cudaStream_t stream) {
    if (many != nullptr) return launch_many<64>(*many, p, flags, stream);
    return n_tiles == 1 ? launch_rows<64, 1>(p, stream) : launch_rows<64, 2>(p, stream);
}

}  // namespace packed
}  // namespace hss
