// Frequencies of the rotary positions (host; tq_rope_plan checks the arguments).
//
// A frequency is kept as a 64-bit fraction of a turn per position, from long double
// arithmetic (64-bit mantissa): its error, 2^-64 relative, is below half a unit of the
// fraction, so position * turns modulo 2^64 is the angle to within position * 2^-64 turns.
#include <algorithm>
#include <cmath>

#include "tq_internal.h"

namespace tq {

void fill_rope_table(int rot_dim, int layout, double base, int scaling, double factor, double original_len, double low,
                     double high, tq_rope_table* out) {
    const long double two_pi = 2.0L * 3.14159265358979323846264338327950288L;
    const long double f = scaling == TQ_ROPE_SCALE_NONE ? 1.0L : factor;
    const long double rot = rot_dim;
    long double b = base;
    if (scaling == TQ_ROPE_SCALE_NTK) b *= std::pow(f, rot / (rot - 2.0L));
    long double first = 0, last = 0;
    if (scaling == TQ_ROPE_SCALE_YARN) {
        auto at = [&](long double beta) { return rot * std::log(original_len / (two_pi * beta)) / (2.0L * std::log(b)); };
        first = std::max(std::floor(at(high)), 0.0L);
        last = std::min(std::ceil(at(low)), rot - 1.0L);
        out->mscale = float(0.1L * std::log(f) + 1.0L);
    } else {
        out->mscale = 1.f;
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        long double th = std::pow(b, -2.0L * i / rot);
        if (scaling == TQ_ROPE_SCALE_LINEAR) {
            th /= f;
        } else if (scaling == TQ_ROPE_SCALE_BANDS) {
            const long double keep = std::clamp((original_len * th / two_pi - low) / ((long double)high - low), 0.0L, 1.0L);
            th *= keep + (1.0L - keep) / f;
        } else if (scaling == TQ_ROPE_SCALE_YARN) {
            const long double ramp = std::clamp((i - first) / std::max(last - first, 0.001L), 0.0L, 1.0L);
            th *= 1.0L - ramp + ramp / f;
        }
        out->turns[i] = (uint64_t)std::floor(std::ldexp(th / two_pi, 64) + 0.5L);  // theta <= 1: below a turn
    }
    out->rot_dim = rot_dim;
    out->layout = layout;
}

}  // namespace tq
