// Which schedules the block step can run, and where it cuts them (host only).
//
// The chain (blocks_chain.hip) holds A, Q = a + b A + c A^2 and A Q as fp16 pairs
// of fixed scales, so a schedule has to keep them within bounds, from above and from
// below, on every spectrum that a normalised X can have: singular values in [0, 1],
// the largest of them at least 128^-1/2.
#pragma once

#include <algorithm>
#include <cmath>
#include <vector>

#include "../../include/muon_step.h"
#include "blocks.hpp"

namespace muon {

struct BlockSegment {
    int first, steps;
};
struct BlockSchedule {
    bool fits = false;
    std::vector<BlockSegment> segments;  // at least one
};
// The largest gain that a schedule may give a vanishing singular value.  P holds that
// gain, rounded to 24 bits, wherever N has such a direction (a rank below the smaller
// side), and what the rounding adds to O is 2^-24 of it.
constexpr double kMaxGain = 0x1p22;
// What the largest singular value may fall to.  A, which is at least its square on
// the diagonal of an even spectrum, then keeps 22 bits as fp16 pairs of 64 A.
constexpr double kLeastSigma = 0.044;

// Largest |c0 + c1 x + c2 x^2| x^power on [0, top], power 0 or 1.
inline double polynomial_bound(double c0, double c1, double c2, int power, double top) {
    auto value = [&](double x) { return std::fabs((c0 + (c1 + c2 * x) * x) * (power ? x : 1.0)); };
    double best = std::max(value(0.0), value(top));
    auto at = [&](double x) {
        if (x > 0.0 && x < top) best = std::max(best, value(x));
    };
    if (power == 0) {
        if (c2 != 0.0) at(-c1 / (2.0 * c2));
    } else if (c2 == 0.0) {
        if (c1 != 0.0) at(-c0 / (2.0 * c1));
    } else {
        const double d = c1 * c1 - 3.0 * c0 * c2;  // roots of c0 + 2 c1 x + 3 c2 x^2
        if (d >= 0.0) {
            at((-c1 + std::sqrt(d)) / (3.0 * c2));
            at((-c1 - std::sqrt(d)) / (3.0 * c2));
        }
    }
    return best;
}

// Largest |x (a + b x^2 + c x^4)| on [0, top].
inline double map_bound(double a, double b, double c, double top) {
    auto value = [&](double l) { return std::fabs(std::sqrt(l) * (a + (b + c * l) * l)); };
    const double end = top * top;
    double best = value(end);
    auto at = [&](double l) {
        if (l > 0.0 && l < end) best = std::max(best, value(l));
    };
    if (c == 0.0) {  // roots of a + 3 b l + 5 c l^2
        if (b != 0.0) at(-a / (3.0 * b));
    } else {
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (d >= 0.0) {
            at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
            at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
        }
    }
    return best;
}

// Smallest |x (a + b x^2 + c x^4)| on [least, top], least > 0.
inline double map_least(double a, double b, double c, double least, double top) {
    auto value = [&](double l) { return std::sqrt(l) * (a + (b + c * l) * l); };
    const double begin = least * least, end = top * top, first = value(begin);
    double best = std::fabs(first);
    auto at = [&](double l) {
        const double v = l >= begin && l <= end ? value(l) : first;
        best = first * v > 0.0 ? std::min(best, std::fabs(v)) : 0.0;  // a change of sign passes zero
    };
    at(end);
    if (c == 0.0) {  // roots of a + 3 b l + 5 c l^2
        if (b != 0.0) at(-a / (3.0 * b));
    } else {
        const double d = 9.0 * b * b - 20.0 * a * c;
        if (d >= 0.0) {
            at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
            at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
        }
    }
    return best;
}

inline BlockSchedule plan_blocks_schedule(const muon_ns_coeff *c, int n) {
    BlockSchedule out;
    if (n > kMaxChainSteps) return out;
    double x = 1.0, p = 1.0;                                            // bounds of |X| and |P|
    double least = 1.0 / std::sqrt(static_cast<double>(kBlockSide));  // of X's largest singular value
    for (int k = 0; k < n; ++k) {
        const double top = x * x;
        const double q = polynomial_bound(c[k].a, c[k].b, c[k].c, 0, top);
        const double r = polynomial_bound(c[k].a, c[k].b, c[k].c, 1, top);
        const double next = map_bound(c[k].a, c[k].b, c[k].c, x);
        p *= q;
        if (!(q <= 60.0 && r <= 60.0 && next <= 3.9 && p <= kMaxGain)) return out;
        least = map_least(c[k].a, c[k].b, c[k].c, least, x);
        if (!(least >= kLeastSigma)) return out;
        x = next;
    }
    out.fits = true;
    // A step multiplies what noise has put in the directions of vanishing singular
    // values by a^2, relative to what Q makes of them.  A segment goes on while that
    // stays below 2^11 times fp32's rounding (1e-4 of a small direction's gain); the last
    // one, whose noise no later step can grow, up to 2^17.  Both hold where the
    // schedule's last two steps settle what noise does to singular values near 1;
    // otherwise O shows it as it is, and no segment may pass 2^8.
    // Error against 64 bits on spectra over three decades, s of 16 to 128 in long
    // blocks and (in squares), emulated: the hybrid schedule as 4 + 6 steps 1.3e-5
    // (1.9e-4), as 3 + 7 4e-6 to 1.1e-5 (1.2e-3), as 5 + 5 7e-5 (1.7e-4), as 2 + 3 + 5, which
    // is another pass over M and G, 4e-6 to 1e-5 (1.4e-4).  Five quintic steps as one
    // segment 8e-5 to 1.5e-4, as 3 + 2 6e-6; twelve as 4 + 4 + 4 1e-4 to 2e-4, as four times
    // three 1e-5 to 3e-5.  Each segment is another pass: five quintic steps over 1728 heads
    // of 128 x 2048 take 3.28 ms as 3 + 2, 2.52 as one.
    auto gain = [&](int k) { return std::max(1.0, c[k].a * c[k].a); };
    auto settles = [&](int k) { return k >= 0 && std::fabs(c[k].a + 3.0 * c[k].b + 5.0 * c[k].c) < 0.25; };  // |f'(1)|
    const bool settled = settles(n - 1) && settles(n - 2);
    const double most = settled ? 0x1p11 : 0x1p8, most_last = settled ? 0x1p17 : 0x1p8;
    int at = 0;
    while (at < n) {
        double rest = 1.0;
        for (int k = at; k + 1 < n; ++k) rest *= gain(k);
        int steps = n - at;
        if (rest > most_last) {
            double g = 1.0;
            for (steps = 1; at + steps < n && (g *= gain(at + steps - 1)) <= most; ++steps) {
            }
        }
        out.segments.push_back(BlockSegment{at, steps});
        at += steps;
    }
    if (out.segments.empty()) out.segments.push_back(BlockSegment{0, 0});
    return out;
}

}  // namespace muon
