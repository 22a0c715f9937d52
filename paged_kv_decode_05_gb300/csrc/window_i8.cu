// The window mode of ctx_attn.cuh over INT8 caches.
#include "ctx_attn.cuh"

namespace pkv {
namespace ctx {

template <>
bool pick_i8<kWindow>(pkv_dtype q, int D, int G, Ops* o) {
    return q == PKV_BF16 ? pick_d<kWindow, I8, BF16>(D, G, o) : pick_d<kWindow, I8, F16>(D, G, o);
}

}  // namespace ctx
}  // namespace pkv
