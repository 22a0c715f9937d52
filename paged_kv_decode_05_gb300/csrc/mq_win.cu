// Multi-query attention with a sliding window over fp16 / bf16 caches (kernels:
// mq_split.cuh; for long runs mq_wide.cuh).
#include "mq_split.cuh"

namespace pkv {

bool mq_pick_win(pkv_dtype kv_dtype, int D, int G, int nw, MqOps* o) {
    return kv_dtype == PKV_BF16 ? mq_pick_d<BF16, BF16, true>(D, G, nw, o)
                                : mq_pick_d<F16, F16, true>(D, G, nw, o);
}

}  // namespace pkv
