// attend_packed_64.cu -- the packed cache's attention for heads of 64 elements.
#include "attend_packed.cuh"

namespace hss {
namespace packed {

template <>
hss_status launch_head_dim<64>(const Params& p, int n_tiles, cudaStream_t stream) {
    return n_tiles == 1 ? launch_rows<64, 1>(p, stream) : launch_rows<64, 2>(p, stream);
}

}  // namespace packed
}  // namespace hss
