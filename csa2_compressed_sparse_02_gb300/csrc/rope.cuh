// Rotary embedding shared by csa2_rope and csa2_page_write: the frequency table (host)
// and the sine and cosine of one angle (device).
#pragma once

#include <cmath>

#include "common.cuh"

namespace csa2 {

constexpr int kRopeMaxPairs = 256;

// Turns (angle / 2 pi) a position adds to pair i: the YaRN frequency (Peng et al. 2023,
// NTK-by-parts) of base^(-2i/dim), in fp64 as the Compressor's. A kernel argument (2 KB).
struct RopeTable {
    int dim;  // rotated channels; 0: no rotation
    double turns[kRopeMaxPairs];
};

// Built once per thread and setting (a program rarely alternates between two): the powers of
// 32 pairs take about a microsecond, as long as the launch.
inline const RopeTable& rope_table(const csa2_params* p, int dim) {
    struct Built {
        RopeTable t;
        float theta, factor, orig_len, fast, slow;
    };
    static thread_local Built last = {};
    if (last.t.dim == dim && last.theta == p->rope_theta && last.factor == p->rope_factor &&
        last.orig_len == p->rope_orig_len && last.fast == p->rope_beta_fast && last.slow == p->rope_beta_slow)
        return last.t;
    RopeTable* t = &last.t;
    t->dim = dim;
    last.theta = p->rope_theta;
    last.factor = p->rope_factor;
    last.orig_len = p->rope_orig_len;
    last.fast = p->rope_beta_fast;
    last.slow = p->rope_beta_slow;
    for (int i = 0; i < dim / 2; ++i) {
        const double f = std::pow((double)p->rope_theta, -(double)(2 * i) / (double)dim) * 0.15915494309189535;
        const double r = (double)p->rope_orig_len * f;  // turns over the original context
        double keep;
        if (r > p->rope_beta_fast) keep = 1.0;
        else if (r < p->rope_beta_slow) keep = 0.0;
        else keep = (r - p->rope_beta_slow) / ((double)p->rope_beta_fast - (double)p->rope_beta_slow);
        t->turns[i] = f * keep + (f / (double)p->rope_factor) * (1.0 - keep);
    }
    return last.t;
}

inline bool rope_settings_ok(const csa2_params* p) {
    return p->rope_theta > 0.f && p->rope_factor > 0.f && p->rope_orig_len > 0.f &&
           p->rope_beta_fast > p->rope_beta_slow;
}

// Cosine and sine of `pos` positions at `turns` a position. The whole quarter turns are
// taken off in fp64 (a product of about 2^-53 relative error: 2e-11 turns at a million
// positions); what is left, at most an eighth of a turn, keeps 24 bits in fp32.
__device__ __forceinline__ float2 rope_cs(double turns, int pos) {
    const double t = turns * (double)pos;
    const double quarters = rint(4.0 * t);
    float s, c;
    sincospif(2.0f * (float)fma(-0.25, quarters, t), &s, &c);
    switch ((int)(__double2ll_rn(quarters) & 3)) {
        case 0: return make_float2(c, s);
        case 1: return make_float2(-s, c);
        case 2: return make_float2(-c, -s);
        default: return make_float2(s, -c);
    }
}

}  // namespace csa2
