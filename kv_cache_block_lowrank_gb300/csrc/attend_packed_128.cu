// attend_packed_128.cu -- the packed cache's attention for heads of 128 elements.
#include "attend_packed.cuh"

namespace hss {
namespace packed {

template <>
hss_status launch_head_dim<128>(const Params& p, int n_tiles, cudaStream_t stream) {
    return n_tiles == 1 ? launch_rows<128, 1>(p, stream) : launch_rows<128, 2>(p, stream);
}

}  // namespace packed
}  // namespace hss
