// The wide-chunk tcgen05 kernel (mq_wide.cuh) over fp16 / bf16 caches.
#include "mq_wide.cuh"

namespace pkv {

WideLaunch wide_pick(pkv_dtype kv_dtype, int D, int G) {
    return kv_dtype == PKV_BF16 ? wide_pick_d<BF16, BF16>(D, G) : wide_pick_d<F16, F16>(D, G);
}

}  // namespace pkv
