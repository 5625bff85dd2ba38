// Rotary embedding shared by csa2_rope and csa2_page_write: the frequency table (host)
// and the sine and cosine of one angle (device).
#pragma once

#include <cmath>
#include <initializer_list>

#include "common.cuh"

namespace csa2 {

constexpr int kRopeMaxPairs = 256;

// Turns (angle / 2 pi) a position adds to pair i, in units of 2^-64: the YaRN frequency (Peng
// et al. 2023, NTK-by-parts) of base^(-2i/dim), computed in fp64 as the Compressor's. Whole
// turns drop out, as positions are integers. A kernel argument (2 KB).
struct RopeTable {
    int dim;  // rotated channels; 0: no rotation
    uint64_t turns[kRopeMaxPairs];
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
        const double turns = f * keep + (f / (double)p->rope_factor) * (1.0 - keep);
        // the fraction in two halves: fp64 holds 53 bits of it, all of which are kept
        const double hi = (turns - std::floor(turns)) * 4294967296.0, whole = std::floor(hi);
        t->turns[i] = ((uint64_t)whole << 32) + (uint64_t)((hi - whole) * 4294967296.0);
    }
    return last.t;
}

inline bool rope_settings_ok(const csa2_params* p) {
    for (float v : {p->rope_theta, p->rope_factor, p->rope_orig_len, p->rope_beta_fast, p->rope_beta_slow})
        if (!std::isfinite(v)) return false;
    return p->rope_theta > 0.f && p->rope_factor > 0.f && p->rope_orig_len > 0.f &&
           p->rope_beta_fast > p->rope_beta_slow;
}

// Cosine and sine of `pos` positions at `turns` a position. The product is exact modulo whole
// turns in 64-bit integers (GB300's fp64 rate, two lanes a cycle and SM, would bound the
// kernels here: 19 us against 11 for 16,004 rows of csa2_page_write). The quarter turns are
// taken off; the rest, at most an eighth of a turn, keeps 32 bits behind the point (cut off there:
// up to 2^-32 turns low) and 24 bits in fp32.
__device__ __forceinline__ float2 rope_cs(uint64_t turns, int pos) {
    const uint64_t t = turns * (uint64_t)(uint32_t)pos;
    const uint32_t quarters = (uint32_t)((t + (1ull << 61)) >> 62);
    const int rest = (int)((t - ((uint64_t)quarters << 62)) >> 32);
    float s, c;
    sincospif((float)rest * 0x1p-31f, &s, &c);
    const float a = quarters & 1u ? s : c, b = quarters & 1u ? c : s;  // |cos|, |sin| by quarter
    return make_float2(quarters == 1u || quarters == 2u ? -a : a, quarters & 2u ? -b : b);
}

}  // namespace csa2
