// The wide-chunk tcgen05 kernel (mq_wide.cuh) over INT8 caches.
#include "mq_wide.cuh"

namespace pkv {

WideLaunch wide_pick_i8(pkv_dtype q_dtype, int D, int G) {
    return q_dtype == PKV_BF16 ? wide_pick_d<I8, BF16>(D, G) : wide_pick_d<I8, F16>(D, G);
}

}  // namespace pkv
