// Host table of rotary frequencies, with the ways of stretching them for
// contexts longer than a model was trained on.
#include <cmath>

#include "pagedkv.h"

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

double clamp01(double x) { return x < 0.0 ? 0.0 : x > 1.0 ? 1.0 : x; }

}  // namespace

extern "C" pkv_status pkv_rotary_frequencies(float* inv_freq, float* attention_scale, int rotary_dim, double base,
                                             pkv_rotary_scaling scaling, double factor, int64_t original_context,
                                             double fast_turns, double slow_turns) {
    if (!inv_freq || !attention_scale || rotary_dim <= 0 || rotary_dim % 2 != 0 || !(base > 1.0) || !std::isfinite(base))
        return PKV_ERR_INVALID_ARG;
    if (scaling < PKV_ROTARY_PLAIN || scaling > PKV_ROTARY_BY_INDEX) return PKV_ERR_UNSUPPORTED;
    if (scaling != PKV_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return PKV_ERR_INVALID_ARG;
    const bool parts = scaling == PKV_ROTARY_BY_TURNS || scaling == PKV_ROTARY_BY_INDEX;
    if (parts && (original_context <= 0 || !(slow_turns > 0.0) || !(fast_turns > slow_turns) || !std::isfinite(fast_turns)))
        return PKV_ERR_INVALID_ARG;
    const double R = rotary_dim;
    // rotary_dim 2 has one frequency, 1, whatever the base
    if (scaling == PKV_ROTARY_BASE && rotary_dim > 2) base *= std::pow(factor, R / (R - 2.0));
    // by index: the pair whose frequency makes `turns` turns over the original
    // context is at R ln(context / (2 pi turns)) / (2 ln base)
    double low = 0.0, high = 0.0;
    if (scaling == PKV_ROTARY_BY_INDEX) {
        auto at = [&](double turns) {
            return R * std::log((double)original_context / (kTwoPi * turns)) / (2.0 * std::log(base));
        };
        low = std::fmax(std::floor(at(fast_turns)), 0.0);
        high = std::fmin(std::ceil(at(slow_turns)), R - 1.0);
        if (high <= low) high = low + 0.001;   // a step instead of a ramp
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / R);
        if (scaling == PKV_ROTARY_LINEAR) {
            f /= factor;
        } else if (parts) {
            // keep: 1 for fast pairs, which keep their frequency, 0 for slow
            // ones, which are divided by the factor
            const double keep =
                scaling == PKV_ROTARY_BY_TURNS
                    ? clamp01(((double)original_context * f / kTwoPi - slow_turns) / (fast_turns - slow_turns))
                    : 1.0 - clamp01((i - low) / (high - low));
            f *= keep + (1.0 - keep) / factor;
        }
        inv_freq[i] = (float)f;
    }
    *attention_scale = scaling == PKV_ROTARY_BY_INDEX ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return PKV_OK;
}
