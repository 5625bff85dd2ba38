// csa2_paged_attn: dense attention of one new token per sequence over a paged cache of
// latents (K = V), with a window, first tokens that stay visible and a sink logit.
//
// Schedule. The positions a sequence sees lie in tiles of 128 (its first tokens' tiles, then
// those from the window's start to its end). The (sequence, tile) items of the whole batch
// are cut into one contiguous range of equal length per CTA, from the lengths on the device.
// A sequence within one range is finished there; one that ranges cut leaves a partial result
// per piece (unnormalised O, running maximum m and sum l of each head), and k_paged_join
// joins them in order: o = sum_i O_i 2^{m_i - M} / (2^{sink - M} + sum_i l_i 2^{m_i - M}).
#include <climits>

#include "pages.cuh"
#include "sm100.cuh"

namespace csa2 {
namespace {
using namespace sm100;

constexpr int kTile = 128;
constexpr int kMaxHeads = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    Pages g;
    const uint8_t* base;  // the layer's first page
    int B, heads, window, n_first;
    int64_t q_seq, q_head;
    const __nv_bfloat16* q;
    const float* sink;
    const int32_t* seq;
    const int32_t* n_tokens;
    __nv_bfloat16* out;
    int64_t* prefix;  // workspace: items before each sequence [B + 1]
    float* part;      // workspace: two partial results per CTA
    int32_t* dev_status;
    float scale_log2;
    int ctas;         // of the attention kernel (the join needs its ranges)
};

__host__ __device__ inline int64_t part_floats(int heads) { return (int64_t)heads * (kD + 2); }

// What sequence b of the call sees: positions [0, nf) and [lo, T), in `tiles` tiles.
struct View {
    int64_t T, lo, nf;
    int row;  // of the table; < 0: padding
    int first_tiles, lo_tile, tiles;
    __device__ __forceinline__ bool sees(int64_t t) const { return t < T && (t >= lo || t < nf); }
    __device__ __forceinline__ int64_t start(int j) const {
        return (int64_t)(j < first_tiles ? j : lo_tile + j - first_tiles) * kTile;
    }
};

__device__ __forceinline__ View view_of(const Args& a, int b, bool report) {
    View v;
    v.row = a.seq ? a.seq[b] : b;
    v.T = v.row < 0 ? 0 : a.n_tokens[b];
    if (v.row >= a.g.max_seqs) {
        if (report) raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
        v.T = 0;
    }
    if (v.T < 0 || v.T > a.g.max_len()) {
        if (report) raise_status(a.dev_status, CSA2_DEV_BAD_LENGTH);
        v.T = v.T < 0 ? 0 : a.g.max_len();
    }
    v.lo = a.window > 0 ? max((int64_t)0, v.T - a.window) : 0;
    v.nf = min((int64_t)max(a.n_first, 0), v.lo);
    v.lo_tile = (int)(v.lo / kTile);
    v.first_tiles = min((int)((v.nf + kTile - 1) / kTile), v.lo_tile);
    v.tiles = v.first_tiles + (int)((v.T + kTile - 1) / kTile) - v.lo_tile;
    return v;
}

// Items [range(c), range(c + 1)) of `total` belong to CTA c of n.
__device__ __forceinline__ int64_t range_of(int64_t total, int c, int n) { return total * c / n; }

// Fewer items than CTAs leave some ranges empty.
__device__ __forceinline__ bool holds(int64_t total, int c, int n) {
    return range_of(total, c, n) < range_of(total, c + 1, n);
}

// The partial result of a piece of CTA c: slot 0 if the piece opens the CTA's range, else 1.
__device__ __forceinline__ float* part_of(const Args& a, int c, int slot) {
    return a.part + (2 * (int64_t)c + slot) * part_floats(a.heads);
}

// This CTA's range of items, and the sequence and tile its first item belongs to; CTA 0
// leaves every sequence's first item in a.prefix for the join. Called by the whole CTA
// (a multiple of 32 threads, at most 1,024).
struct Range {
    int64_t total, at, end;
    int b, j;
};
__device__ void plan(const Args& a, Range* sh) {
    __shared__ int64_t warp_sum[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const bool lead = blockIdx.x == 0;
    int64_t total = 0;
    for (int pass = 0; pass < 2; ++pass) {  // the sum of all items, then the place of this range
        int64_t before = 0;
        for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
            const int b = b0 + tid;
            const int64_t n = b < a.B ? view_of(a, b, lead && pass == 0).tiles : 0;
            int64_t inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
            if (lane == 31) warp_sum[warp] = inc;
            __syncthreads();
            int64_t here = before, all = 0;
            for (int w = 0; w < warps; ++w) {
                if (w < warp) here += warp_sum[w];
                all += warp_sum[w];
            }
            __syncthreads();
            here += inc - n;
            if (pass == 1 && b < a.B) {
                const int64_t at = range_of(total, blockIdx.x, a.ctas);
                if (at >= here && at < here + n) {
                    sh->b = b;
                    sh->j = (int)(at - here);
                }
                if (lead) a.prefix[b] = here;
            }
            before += all;
        }
        total = before;
    }
    if (tid == 0) {
        sh->total = total;
        sh->at = range_of(total, blockIdx.x, a.ctas);
        sh->end = range_of(total, blockIdx.x + 1, a.ctas);
        if (lead) a.prefix[a.B] = total;
    }
    __syncthreads();
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- one CTA's pieces
constexpr int kThreads = 256;
constexpr int kStep = 16;  // positions taken at a time
struct Shared {
    float kv[kStep][kD + 1];
    float z[kMaxHeads][kStep];
    Range range;
};

__device__ __forceinline__ float e4m3_at(const uint8_t* p) { return e4m3_value(*p); }

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) k_paged_attn(Args a) {
    extern __shared__ uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    grid_dep_wait();
    plan(a, &sh.range);
    const int tid = threadIdx.x;
    const int h = tid >> 2, part = tid & 3;  // O of head h, channels part + 4 i
    int64_t at = sh.range.at;
    const int64_t end = sh.range.end;
    int b = sh.range.b, j = sh.range.j;
    bool opens = true;
    while (at < end) {
        const View v = view_of(a, b, false);
        if (j >= v.tiles) {
            ++b;
            j = 0;
            continue;
        }
        const int j1 = (int)min((int64_t)v.tiles, j + (end - at));
        const int32_t* table = a.g.table + (int64_t)v.row * a.g.max_pages;
        float o[kD / 4];
#pragma unroll
        for (int i = 0; i < kD / 4; ++i) o[i] = 0.f;
        float m = -INFINITY, l = 0.f;
        for (int jj = j; jj < j1; ++jj) {
            const int64_t t0 = v.start(jj);
            for (int s = 0; s < kTile; s += kStep) {
                __syncthreads();
                for (int e = tid; e < kStep * kD; e += kThreads) {
                    const int r = e / kD, c = e % kD;
                    const int64_t t = t0 + s + r;
                    float x = 0.f;
                    if (v.sees(t)) {
                        const int page = table[t / a.g.page_size];
                        if (page >= 0 && page < a.g.n_pages) {
                            const uint8_t* row = a.base + page * a.g.page_bytes() + (t % a.g.page_size) * a.g.row_bytes;
                            x = kBf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[c]) : e4m3_at(row + c);
                        } else if (c == 0) {
                            raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
                        }
                    }
                    sh.kv[r][c] = x;
                }
                __syncthreads();
                for (int e = tid; e < a.heads * kStep; e += kThreads) {
                    const int hh = e / kStep, r = e % kStep;
                    const int64_t t = t0 + s + r;
                    bool ok = v.sees(t);
                    if (ok) {
                        const int page = table[t / a.g.page_size];
                        ok = page >= 0 && page < a.g.n_pages;
                    }
                    float z = -INFINITY;
                    if (ok) {
                        const __nv_bfloat16* q = a.q + b * a.q_seq + hh * a.q_head;
                        z = 0.f;
                        for (int c = 0; c < kD; ++c) z = fmaf(__bfloat162float(q[c]), sh.kv[r][c], z);
                        z *= a.scale_log2;
                    }
                    sh.z[hh][r] = z;
                }
                __syncthreads();
                if (h < a.heads) {
                    float mx = m;
                    for (int r = 0; r < kStep; ++r) mx = fmaxf(mx, sh.z[h][r]);
                    if (mx != m) {
                        const float f = m == -INFINITY ? 0.f : ex2(m - mx);
                        l *= f;
#pragma unroll
                        for (int i = 0; i < kD / 4; ++i) o[i] *= f;
                        m = mx;
                    }
                    for (int r = 0; r < kStep; ++r) {
                        const float z = sh.z[h][r];
                        if (z == -INFINITY) continue;
                        const float p = ex2(z - m);
                        l += p;
#pragma unroll
                        for (int i = 0; i < kD / 4; ++i) o[i] = fmaf(p, sh.kv[r][part + 4 * i], o[i]);
                    }
                }
            }
        }
        if (h < a.heads) {
            if (j == 0 && j1 == v.tiles) {
                const float s2 = a.sink ? a.sink[h] * kLog2e : -INFINITY;
                const float M = fmaxf(m, s2);
                const float f = m == -INFINITY ? 0.f : ex2(m - M);
                const float den = l * f + (s2 == -INFINITY ? 0.f : ex2(s2 - M));
                __nv_bfloat16* out = a.out + ((int64_t)b * a.heads + h) * kD;
#pragma unroll
                for (int i = 0; i < kD / 4; ++i)
                    out[part + 4 * i] = __float2bfloat16_rn(den == 0.f ? 0.f : o[i] * f / den);
            } else {
                float* p = part_of(a, blockIdx.x, opens ? 0 : 1);
#pragma unroll
                for (int i = 0; i < kD / 4; ++i) p[(int64_t)h * kD + part + 4 * i] = o[i];
                if (part == 0) {
                    p[(int64_t)a.heads * kD + h] = m;
                    p[(int64_t)a.heads * (kD + 1) + h] = l;
                }
            }
        }
        at += j1 - j;
        j = j1;
        opens = false;
    }
}

// ---------------------------------------------------------------- join
// One warp per (sequence, head), lane = 16 channels in four groups of four. Sequences that
// no range boundary cuts were finished by the attention kernel; those that see nothing get
// their zeros here.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps) k_paged_join(Args a) {
    grid_dep_wait();
    const int lane = threadIdx.x & 31, b = blockIdx.x, h = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
    if (h >= a.heads) return;
    const int64_t total = a.prefix[a.B], s = a.prefix[b], e = a.prefix[b + 1];
    __nv_bfloat16* out = a.out + ((int64_t)b * a.heads + h) * kD + 4 * lane;
    if (s == e) {
        if (!a.seq || a.seq[b] >= 0)
            for (int k = 0; k < 4; ++k) *reinterpret_cast<uint2*>(out + 128 * k) = make_uint2(0u, 0u);
        return;
    }
    int c0 = (int)(s * a.ctas / total);  // the CTA whose range holds item s
    while (range_of(total, c0 + 1, a.ctas) <= s) ++c0;
    int c1 = c0;
    while (range_of(total, c1 + 1, a.ctas) < e) ++c1;
    if (c0 == c1) return;
    const float s2 = a.sink ? a.sink[h] * kLog2e : -INFINITY;
    const int64_t mo = (int64_t)a.heads * kD + h, lo = mo + a.heads;
    const int slot0 = range_of(total, c0, a.ctas) == s ? 0 : 1;
    float M = s2;
    for (int c = c0 + lane; c <= c1; c += 32)
        if (holds(total, c, a.ctas)) M = fmaxf(M, part_of(a, c, c == c0 ? slot0 : 0)[mo]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float den = s2 == -INFINITY ? 0.f : ex2(s2 - M);
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = c0; c <= c1; ++c) {
        if (!holds(total, c, a.ctas)) continue;
        const float* p = part_of(a, c, c == c0 ? slot0 : 0);
        const float m = p[mo];
        const float f = m == -INFINITY ? 0.f : ex2(m - M);
        den = fmaf(p[lo], f, den);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 v = *reinterpret_cast<const float4*>(p + (int64_t)h * kD + 4 * lane + 128 * k);
            acc[k].x = fmaf(v.x, f, acc[k].x);
            acc[k].y = fmaf(v.y, f, acc[k].y);
            acc[k].z = fmaf(v.z, f, acc[k].z);
            acc[k].w = fmaf(v.w, f, acc[k].w);
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv);
        const __nv_bfloat162 y = __floats2bfloat162_rn(acc[k].z * inv, acc[k].w * inv);
        *reinterpret_cast<uint2*>(out + 128 * k) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    }
}

int grid_of(const csa2_params* p) {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return p->max_ctas > 0 && p->max_ctas < n ? p->max_ctas : n;
}

int64_t prefix_bytes(int64_t B) { return (8 * (B + 1) + 255) & ~(int64_t)255; }

int64_t ws_need(int B, int heads, int ctas) { return prefix_bytes(B) + 2 * (int64_t)ctas * part_floats(heads) * 4; }

}  // namespace

cudaError_t preload_paged_attn() {
    cudaError_t (*l[])() = {[] { return preload_kernel(k_paged_attn<true>, (int)sizeof(Shared)); },
                            [] { return preload_kernel(k_paged_attn<false>, (int)sizeof(Shared)); },
                            [] { return preload_kernel(k_paged_join); }};
    for (auto f : l)
        if (const cudaError_t e = f()) return e;
    return cudaSuccess;
}

}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_paged_attn_workspace_size(const csa2_params* p, const csa2_pages* c, int B) {
    if (!p || !c || B <= 0 || p->heads < 1 || p->heads > kMaxHeads) return 0;
    const int ctas = grid_of(p);
    return ctas > 0 ? (size_t)ws_need(B, p->heads, ctas) : 0;
}

extern "C" int csa2_paged_attn(const csa2_params* p, const csa2_pages* c, int layer, int B, const void* q,
                               int64_t q_seq, int64_t q_head, const float* sink, const int32_t* seq,
                               const int32_t* n_tokens, int window, int n_first, void* out, void* workspace,
                               size_t ws_bytes, int32_t* dev_status, void* stream) {
    Args a = {};
    if (const int rc = check_pages("paged_attn", p, c, &a.g)) return rc;
    if (B < 0 || layer < 0 || layer >= a.g.layers)
        return fail(CSA2_ERR_INVALID_ARG, "paged_attn: negative size or layer out of range");
    if (p->heads < 1 || p->heads > kMaxHeads || p->q_format != CSA2_BF16)
        return fail(CSA2_ERR_UNSUPPORTED, "paged_attn: built for 1 .. 64 heads, BF16 queries");
    if (B > 65535) return fail(CSA2_ERR_UNSUPPORTED, "paged_attn: at most 65535 sequences");
    if (B == 0) return CSA2_OK;
    if (!seq && B > a.g.max_seqs) return fail(CSA2_ERR_INVALID_ARG, "paged_attn: B beyond max_seqs needs seq");
    if (!q || !n_tokens || !out || !workspace) return fail(CSA2_ERR_INVALID_ARG, "paged_attn: NULL buffer");
    if (!aligned16(q) || !aligned16(out) || q_seq % 8 || q_head % 8)
        return fail(CSA2_ERR_ALIGN, "paged_attn: q's heads and out must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(CSA2_ERR_ALIGN, "paged_attn: workspace must be 256-byte aligned");
    if (const int rc = ensure_loaded()) return rc;
    const int ctas = grid_of(p);
    if (ctas <= 0) return check_launch("paged_attn: device");
    if ((int64_t)ws_bytes < ws_need(B, p->heads, ctas))
        return fail(CSA2_ERR_SHAPE, "paged_attn: workspace smaller than csa2_paged_attn_workspace_size");
    a.base = a.g.pool + layer * a.g.layer_bytes;
    a.B = B;
    a.heads = p->heads;
    a.window = window;
    a.n_first = n_first;
    a.q_seq = q_seq;
    a.q_head = q_head;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.sink = sink;
    a.seq = seq;
    a.n_tokens = n_tokens;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.prefix = static_cast<int64_t*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + prefix_bytes(B));
    a.dev_status = dev_status;
    a.scale_log2 = p->softmax_scale * kLog2e;
    a.ctas = ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p->kv_format == CSA2_BF16) cudaLaunchKernelEx(&cfg, k_paged_attn<true>, a);
    else cudaLaunchKernelEx(&cfg, k_paged_attn<false>, a);
    if (const int rc = check_launch("paged_attn")) return rc;
    cfg.gridDim = dim3(B, (p->heads + kJoinWarps - 1) / kJoinWarps);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.dynamicSmemBytes = 0;
    cudaLaunchKernelEx(&cfg, k_paged_join, a);
    return check_launch("paged_attn: join");
}
