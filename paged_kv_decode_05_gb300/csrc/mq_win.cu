// Multi-query attention with a sliding window over fp16 / bf16 caches (kernels:
// mq_split.cuh, mq_tc.cuh).
#include "mq_tc.cuh"

namespace pkv {

bool mq_pick_win(pkv_dtype kv_dtype, int D, int G, int nw, MqOps* o) {
    return kv_dtype == PKV_BF16 ? mq_pick_d<BF16, BF16, true>(D, G, nw, o)
                                : mq_pick_d<F16, F16, true>(D, G, nw, o);
}

TcLaunch tc_pick_win(bool bf16, int D, int G) {
    return bf16 ? tc_pick<BF16, true>(D, G) : tc_pick<F16, true>(D, G);
}

}  // namespace pkv
