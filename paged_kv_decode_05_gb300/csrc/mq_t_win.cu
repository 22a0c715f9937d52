// The short-run multi-query kernels (mq_t.cuh) with a sliding window.
#include "mq_t.cuh"

namespace pkv {

bool mqt_pick_win(pkv_dtype kv_dtype, pkv_dtype q_dtype, int D, int G, int nt, MqOps* o) {
    if (kv_dtype == PKV_BF16) return mqt_pick_d<BF16, true>(D, G, nt, o);
    if (kv_dtype == PKV_F16) return mqt_pick_d<F16, true>(D, G, nt, o);
    if (D != 128) return false;
    return q_dtype == PKV_BF16 ? mqt_i8_pick_g<BF16, true>(G, nt, o) : mqt_i8_pick_g<F16, true>(G, nt, o);
}

}  // namespace pkv
