// Multi-query attention with a sliding window over INT8 caches (kernel:
// mq_split.cuh).
#include "mq_split.cuh"

namespace pkv {

bool mq_pick_win_i8(pkv_dtype q_dtype, int D, int G, int nw, MqOps* o) {
    return q_dtype == PKV_BF16 ? mq_pick_d<I8, BF16, true>(D, G, nw, o)
                               : mq_pick_d<I8, F16, true>(D, G, nw, o);
}

}  // namespace pkv
