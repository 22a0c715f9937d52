// The window mode of ctx_attn.cuh over 4-bit caches.
#include "ctx_attn.cuh"

namespace pkv {
namespace ctx {

bool pick_window_u4(pkv_dtype q, int D, int G, Ops* o) {
    return q == PKV_BF16 ? pick_d<kWindow, U4, BF16>(D, G, o) : pick_d<kWindow, U4, F16>(D, G, o);
}

}  // namespace ctx
}  // namespace pkv
