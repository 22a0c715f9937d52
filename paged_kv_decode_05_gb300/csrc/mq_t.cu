// The short-run multi-query kernels (mq_t.cuh) without a window.
#include "mq_t.cuh"

namespace pkv {

bool mqt_pick(pkv_dtype kv_dtype, pkv_dtype q_dtype, int D, int G, int nt, MqOps* o) {
    if (kv_dtype == PKV_BF16) return mqt_pick_d<BF16>(D, G, nt, o);
    if (kv_dtype == PKV_F16) return mqt_pick_d<F16>(D, G, nt, o);
    if (kv_dtype == PKV_I8 && D == 128) {
        if (q_dtype == PKV_BF16) return mqt_i8_pick_g<BF16>(G, nt, o);
        if (q_dtype == PKV_F16) return mqt_i8_pick_g<F16>(G, nt, o);
    }
    return false;
}

}  // namespace pkv
