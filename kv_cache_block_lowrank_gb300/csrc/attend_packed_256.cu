// attend_packed_256.cu -- the packed cache's attention for heads of 256 elements.
#include "attend_packed.cuh"

namespace hss {
namespace packed {

template <>
hss_status launch_head_dim<256>(const Params& p, int n_tiles, cudaStream_t stream) {
    return n_tiles == 1 ? launch_rows<256, 1>(p, stream) : launch_rows<256, 2>(p, stream);
}

}  // namespace packed
}  // namespace hss
