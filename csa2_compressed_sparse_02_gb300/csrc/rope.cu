// csa2_rope: rotary embedding of rows x heads, either pair layout, part of the head, both
// directions. A pair (a, b) turns by the angle of its row: (a cos - b sin, a sin + b cos).
//
// Bound by memory: each channel is read once and written once. A row's sines and cosines are
// computed once per CTA into shared memory and serve all its heads; the loads of the CTA's
// first units are issued before that, so their latency covers it.
#include "rope.cuh"

namespace csa2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTable = 2048;  // pairs in shared memory (16 KB)

struct Args {
    const void* x;
    void* out;
    const int32_t* pos;
    int64_t N, x_row, x_head, out_row, out_head;
    int heads, first, half;  // half: CSA2_ROPE_HALF
    int clear;               // padding becomes zeros instead of being left as it is
    int rows_cta, heads_cta;
    int units, rot_units;    // per (row, head): units of work, the rotated ones first
    uint32_t units_magic, heads_magic;
    float sign;              // -1: inverse
};

// n / d for n * d < 2^32, with magic = ceil(2^32 / d) (d > 1; 0 stands for d = 1).
__device__ __forceinline__ uint32_t div_magic(uint32_t n, uint32_t magic) {
    return magic ? __umulhi(n, magic) : n;
}

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

// A vector, read or written once: 16 bytes stream past the caches.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> ld_vec(const T* p) {
    if constexpr (sizeof(T) * V == 16) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
        return *reinterpret_cast<const Vec<T, V>*>(&u);
    } else {
        return *reinterpret_cast<const Vec<T, V>*>(p);
    }
}
template <typename T, int V>
__device__ __forceinline__ void st_vec(T* p, const Vec<T, V>& v) {
    if constexpr (sizeof(T) * V == 16) __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&v));
    else *reinterpret_cast<Vec<T, V>*>(p) = v;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float f, float& o) { o = f; }
__device__ __forceinline__ void from_f(float f, __nv_bfloat16& o) { o = __float2bfloat16_rn(f); }

// A unit is V channels that are copied, or rotated channels: with kTwo the two vectors of
// V channels that hold V pairs' a and b (the half layout, or single channels of adjacent
// pairs where vectors do not fit), without it one vector of V/2 adjacent pairs.
struct Unit {
    int64_t row;  // of the call; -1: past the end
    int head, ch; // first channel
    int second;   // kTwo: distance of the second vector
    int pair;     // first pair's entry in the CTA's table; -1: copied
};
template <int V, bool kTwo>
__device__ __forceinline__ Unit unit_of(const Args& a, int dim, uint32_t n, uint32_t total, int64_t row0,
                                        int head0, int heads) {
    Unit x;
    x.row = -1;
    if (n >= total) return x;
    const uint32_t rh = div_magic(n, a.units_magic), u = n - rh * a.units;
    const uint32_t r = div_magic(rh, a.heads_magic), h = rh - r * heads;
    const int pairs = dim / 2;
    x.row = row0 + r;
    x.head = head0 + h;
    x.second = 0;
    if (u < (uint32_t)a.rot_units) {
        if (!kTwo) {
            x.ch = a.first + u * V;
            x.pair = r * pairs + u * (V / 2);
        } else if (a.half) {
            x.ch = a.first + u * V;
            x.second = pairs;
            x.pair = r * pairs + u * V;
        } else {
            x.ch = a.first + 2 * u;
            x.second = 1;
            x.pair = r * pairs + u;
        }
    } else {
        x.ch = (u - a.rot_units) * V;
        if (x.ch >= a.first) x.ch += dim;
        x.pair = -1;
    }
    return x;
}

template <typename T, int V, bool kTwo>
__global__ void __launch_bounds__(kThreads)
k_rope(const __grid_constant__ Args a, const __grid_constant__ RopeTable tab) {
    using VT = Vec<T, V>;
    constexpr int kBatch = kTwo ? 4 : 8;  // units a thread holds in registers at once
    __shared__ float2 cs[kMaxTable];
    const int tid = threadIdx.x;
    const int64_t row0 = (int64_t)blockIdx.x * a.rows_cta;
    const int rows = (int)min((int64_t)a.rows_cta, a.N - row0);
    const int head0 = blockIdx.y * a.heads_cta;
    const int heads = min(a.heads_cta, a.heads - head0);
    const int pairs = tab.dim / 2;
    const uint32_t total = (uint32_t)rows * heads * a.units;
    const T* x = static_cast<const T*>(a.x);
    T* out = static_cast<T*>(a.out);
    bool ready = false;
    for (uint32_t base = tid; base - tid < total; base += kThreads * kBatch) {
        VT va[kBatch], vb[kTwo ? kBatch : 1];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const Unit u = unit_of<V, kTwo>(a, tab.dim, base + k * kThreads, total, row0, head0, heads);
            if (u.row < 0) continue;
            const T* src = x + u.row * a.x_row + (int64_t)u.head * a.x_head + u.ch;
            va[k] = ld_vec<T, V>(src);
            if (kTwo && u.pair >= 0) vb[kTwo ? k : 0] = ld_vec<T, V>(src + u.second);
        }
        if (!ready) {
            for (int i = tid; i < rows * pairs; i += kThreads) {
                const int r = i / pairs;
                float2 c = rope_cs(tab.turns[i - r * pairs], a.pos[row0 + r]);
                c.y *= a.sign;
                cs[i] = c;
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const Unit u = unit_of<V, kTwo>(a, tab.dim, base + k * kThreads, total, row0, head0, heads);
            if (u.row < 0) continue;
            if (a.pos[u.row] < 0) {  // padding
                if (!a.clear) continue;
                va[k] = VT{};
                if constexpr (kTwo) vb[k] = VT{};
            }
            T* dst = out + u.row * a.out_row + (int64_t)u.head * a.out_head + u.ch;
            if (u.pair >= 0) {
                if constexpr (kTwo) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float2 c = cs[u.pair + i];
                        const float p = to_f(va[k].v[i]), q = to_f(vb[k].v[i]);
                        from_f(p * c.x - q * c.y, va[k].v[i]);
                        from_f(p * c.y + q * c.x, vb[k].v[i]);
                    }
                    st_vec<T, V>(dst + u.second, vb[k]);
                } else {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 c = cs[u.pair + i];
                        const float p = to_f(va[k].v[2 * i]), q = to_f(va[k].v[2 * i + 1]);
                        from_f(p * c.x - q * c.y, va[k].v[2 * i]);
                        from_f(p * c.y + q * c.x, va[k].v[2 * i + 1]);
                    }
                }
            }
            st_vec<T, V>(dst, va[k]);
        }
    }
}

uint32_t magic_of(uint32_t d) { return d > 1 ? (uint32_t)(((uint64_t)1 << 32) / d + (((uint64_t)1 << 32) % d != 0)) : 0; }

template <typename T>
int launch(Args a, const RopeTable& tab, int head_dim, bool pairs_layout, cudaStream_t s) {
    // Vectors of 16 bytes where every address they would use is a multiple of 16 and no
    // vector straddles the rotated channels; else single channels.
    constexpr int V = 16 / (int)sizeof(T);
    const int rot = tab.dim;
    const bool in_place = a.x == a.out;
    bool vec = aligned16(a.x) && aligned16(a.out) && a.x_row % V == 0 && a.out_row % V == 0 &&
               a.x_head % V == 0 && a.out_head % V == 0 && a.first % V == 0 && head_dim % V == 0;
    vec = vec && (pairs_layout ? rot % V == 0 : (rot / 2) % V == 0);
    const int w = vec ? V : 1;
    a.rot_units = pairs_layout && vec ? rot / w : rot / 2 / w;
    a.units = a.rot_units + (in_place ? 0 : (head_dim - rot) / w);
    // Units of a CTA: 2,048 (32 KB of vectors; its table of sines is then a small part),
    // fewer where that would leave less than four CTAs an SM. A head has at most 4,096 units.
    const int64_t all = a.N * a.heads * (int64_t)a.units;
    int64_t target = all / (152 * 4);
    target = target < 256 ? 256 : target > 2048 ? 2048 : target;
    const int64_t per_head = a.units;
    int64_t hc = target / per_head;
    hc = hc < 1 ? 1 : hc > a.heads ? a.heads : hc;
    int64_t rc = 1;
    if (hc == a.heads) {
        rc = target / (per_head * a.heads);
        const int64_t fit = kMaxTable / (rot / 2);
        if (rc > fit) rc = fit;
        if (rc < 1) rc = 1;
    }
    a.heads_cta = (int)hc;
    a.rows_cta = (int)rc;
    a.units_magic = magic_of((uint32_t)a.units);
    // the last CTA of a head split may hold fewer heads, but never more than one row then
    a.heads_magic = magic_of((uint32_t)hc);
    const dim3 grid((unsigned)((a.N + rc - 1) / rc), (unsigned)((a.heads + hc - 1) / hc));
    if (!vec) k_rope<T, 1, true><<<grid, kThreads, 0, s>>>(a, tab);
    else if (pairs_layout) k_rope<T, V, false><<<grid, kThreads, 0, s>>>(a, tab);
    else k_rope<T, V, true><<<grid, kThreads, 0, s>>>(a, tab);
    return check_launch("rope");
}

}  // namespace

cudaError_t preload_rope() {
    cudaError_t (*l[])() = {[] { return preload_kernel(k_rope<float, 4, false>); },
                            [] { return preload_kernel(k_rope<float, 4, true>); },
                            [] { return preload_kernel(k_rope<float, 1, true>); },
                            [] { return preload_kernel(k_rope<__nv_bfloat16, 8, false>); },
                            [] { return preload_kernel(k_rope<__nv_bfloat16, 8, true>); },
                            [] { return preload_kernel(k_rope<__nv_bfloat16, 1, true>); }};
    for (auto f : l)
        if (const cudaError_t e = f()) return e;
    return cudaSuccess;
}

}  // namespace csa2

using namespace csa2;

extern "C" int csa2_rope(const csa2_params* p, int layout, int inverse, int64_t N, int heads,
                         int head_dim, int first, int format, const void* x, int64_t x_row,
                         int64_t x_head, void* out, int64_t out_row, int64_t out_head,
                         const int32_t* pos, void* stream) {
    CSA2_CHECK_PARAMS(p);
    const bool clear = (layout & CSA2_ROPE_CLEAR) != 0;
    layout &= ~CSA2_ROPE_CLEAR;
    if (N < 0 || heads < 0) return fail(CSA2_ERR_INVALID_ARG, "rope: negative size");
    if (layout != CSA2_ROPE_PAIRS && layout != CSA2_ROPE_HALF)
        return fail(CSA2_ERR_UNSUPPORTED, "rope: layout must be PAIRS or HALF");
    if (format != CSA2_BF16 && format != CSA2_F32)
        return fail(CSA2_ERR_UNSUPPORTED, "rope: format must be BF16 or F32");
    const int rot = p->rope_dim;
    if (rot < 2 || rot % 2 || rot > 2 * kRopeMaxPairs || head_dim < rot || head_dim > 4096 || heads > 4096)
        return fail(CSA2_ERR_UNSUPPORTED,
                    "rope: rope_dim must be even, 2 .. 512, at most head_dim; head_dim and heads at most 4096");
    if (first == -1) first = head_dim - rot;
    if (first < 0 || first > head_dim - rot)
        return fail(CSA2_ERR_INVALID_ARG, "rope: the rotated channels must lie within the head");
    if (!rope_settings_ok(p))
        return fail(CSA2_ERR_INVALID_ARG, "rope: needs finite settings, theta, factor, orig_len > 0 and beta_fast > beta_slow");
    if (N > ((int64_t)1 << 31) - 1) return fail(CSA2_ERR_UNSUPPORTED, "rope: more than 2^31 - 1 rows");
    if (N == 0 || heads == 0) return CSA2_OK;
    if (!x || !out || !pos) return fail(CSA2_ERR_INVALID_ARG, "rope: NULL buffer");
    const uintptr_t es = format == CSA2_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(x) % es || reinterpret_cast<uintptr_t>(out) % es)
        return fail(CSA2_ERR_ALIGN, "rope: x and out must be aligned to their element");
    if (N == 1) x_row = out_row = 0;  // strides that nothing is stepped by
    if (heads == 1) x_head = out_head = 0;
    if ((N > 1 && out_row == 0) || (heads > 1 && out_head == 0))
        return fail(CSA2_ERR_INVALID_ARG, "rope: rows or heads of out overlap");
    if (x == out && clear) return fail(CSA2_ERR_INVALID_ARG, "rope: in place, padding stays as it is");
    if (x == out && (x_row != out_row || x_head != out_head))
        return fail(CSA2_ERR_INVALID_ARG, "rope: in place, x and out must have the same strides");
    if (const int rc = ensure_loaded()) return rc;
    const RopeTable& tab = rope_table(p, rot);
    Args a = {};
    a.x = x;
    a.out = out;
    a.pos = pos;
    a.N = N;
    a.x_row = x_row;
    a.x_head = x_head;
    a.out_row = out_row;
    a.out_head = out_head;
    a.heads = heads;
    a.first = first;
    a.half = layout == CSA2_ROPE_HALF;
    a.clear = clear;
    a.sign = inverse ? -1.f : 1.f;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool pl = layout == CSA2_ROPE_PAIRS;
    return format == CSA2_BF16 ? launch<__nv_bfloat16>(a, tab, head_dim, pl, s)
                               : launch<float>(a, tab, head_dim, pl, s);
}
