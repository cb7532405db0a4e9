// Host side of the rotary positions: frequencies and their fixed-point table.
#include <cmath>
#include <cstdint>

#include "bsa.h"
#include "bsa_errors.h"

namespace {
constexpr double kTwoPi = 6.283185307179586476925286766559;
}

extern "C" {

bsa_status bsa_rope_frequencies(bsa_rope_params p, double *inv_freq) {
    if (inv_freq == nullptr) return bsa::fail(BSA_ERR_INVALID_ARG, "inv_freq is NULL");
    if (p.rot < 2 || p.rot % 2 != 0)
        return bsa::fail(BSA_ERR_INVALID_ARG, "rot must be even and >= 2 (got %d)", p.rot);
    if (!(p.theta > 0.0) || !std::isfinite(p.theta))
        return bsa::fail(BSA_ERR_INVALID_ARG, "theta must be positive and finite");
    if (p.scaling < BSA_ROPE_NONE || p.scaling > BSA_ROPE_PARTS)
        return bsa::fail(BSA_ERR_INVALID_ARG, "bad scaling %d", p.scaling);
    if (p.scaling != BSA_ROPE_NONE && (!(p.factor > 0.0) || !std::isfinite(p.factor)))
        return bsa::fail(BSA_ERR_INVALID_ARG, "factor must be positive and finite");
    if (p.scaling == BSA_ROPE_PARTS &&
        (!(p.original > 0.0) || !(p.high > p.low) || !std::isfinite(p.original) ||
         !std::isfinite(p.high) || !std::isfinite(p.low)))
        return bsa::fail(BSA_ERR_INVALID_ARG, "parts scaling needs original > 0 and low < high");
    if (p.scaling == BSA_ROPE_BASE && p.rot < 4)
        return bsa::fail(BSA_ERR_INVALID_ARG, "base scaling needs rot >= 4");
    double theta = p.theta;
    if (p.scaling == BSA_ROPE_BASE) theta *= std::pow(p.factor, double(p.rot) / (p.rot - 2));
    for (int32_t i = 0; i < p.rot / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / p.rot);
        if (p.scaling == BSA_ROPE_LINEAR) f /= p.factor;
        if (p.scaling == BSA_ROPE_PARTS) {
            double keep = (p.original * f / kTwoPi - p.low) / (p.high - p.low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = keep * f + (1.0 - keep) * f / p.factor;
        }
        inv_freq[i] = f;
    }
    return bsa::ok();
}

bsa_status bsa_rope_table(const double *inv_freq, int32_t count, uint64_t *table) {
    if (inv_freq == nullptr || table == nullptr)
        return bsa::fail(BSA_ERR_INVALID_ARG, "inv_freq or table is NULL");
    if (count < 1) return bsa::fail(BSA_ERR_INVALID_ARG, "count must be >= 1");
    for (int32_t i = 0; i < count; ++i)
        if (!std::isfinite(inv_freq[i]) || std::fabs(inv_freq[i]) > 1048576.0)
            return bsa::fail(BSA_ERR_INVALID_ARG, "inv_freq[%d] is not finite or above 2^20", i);
    for (int32_t i = 0; i < count; ++i) {
        // turns per position modulo one turn, in units of 2^-64: the fraction
        // is in [0, 1), and both halves of the scaling are exact
        const double turns = inv_freq[i] / kTwoPi;
        const double frac = turns - std::floor(turns);
        const double hi = std::floor(frac * 4294967296.0);
        const double lo = (frac * 4294967296.0 - hi) * 4294967296.0;
        table[i] = (uint64_t(hi) << 32) + uint64_t(lo);
    }
    return bsa::ok();
}

}  // extern "C"
