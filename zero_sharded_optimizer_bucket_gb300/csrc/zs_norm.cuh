// The end of a gradient norm, over a plan's shards or a list of tensors.
#pragma once

#include "zs_device.cuh"
#include "zs_launch.h"

namespace zsk {

// From the sum of squares s: norm = float(sqrt(s)) / S, clip coefficient / S,
// flags; then the loss-scale update when a scaler is given.  S = 1 without
// one, which leaves every result bit-identical to the unscaled formula.
__device__ __forceinline__ void norm_finish(double s, float max_norm, float *d_norm, float *d_coef,
                                            int32_t *d_flags, const ZsScaleArgs &sc) {
    const float S = sc.d_scale ? *sc.d_scale : 1.0f;
    const float norm = __fdiv_rn((float)sqrt(s), S);
    const bool finite = isfinite(norm);
    float coef = 1.0f;
    if (finite) {
        float clip = 1.0f;
        if (max_norm > 0.0f) {
            const float c = __fdiv_rn(max_norm, __fadd_rn(norm, 1e-6f));
            clip = c < 1.0f ? c : 1.0f;
        }
        coef = __fdiv_rn(clip, S);
    }
    *d_norm = norm;
    *d_coef = coef;
    *d_flags = finite ? 0 : ZS_SKIP_NONFINITE;
    if (sc.d_scale && sc.window > 0) {
        if (!finite) {
            const float d = __fdiv_rn(S, sc.factor);
            *sc.d_scale = d > sc.min_scale ? d : sc.min_scale;
            *sc.d_good = 0;
        } else {
            const int32_t g = *sc.d_good + 1;
            if (g >= sc.window) {
                *sc.d_scale = __fmul_rn(S, sc.factor);
                *sc.d_good = 0;
            } else {
                *sc.d_good = g;
            }
        }
    }
}

}  // namespace zsk
