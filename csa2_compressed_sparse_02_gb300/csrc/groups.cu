// csa2_prefix_groups: which sequences of a batch hold the same leading pages, and how many positions
// they have in common, for csa2_paged_attn_shared.
//
// Pages that are shared are shared from the first on (a fork shares its parent's full pages), so
// sequences with the same page at position least - 1 are candidates; the lowest-numbered one of them
// leads, and the others' rows of the table are compared with its entry by entry. One kernel does
// that with a warp a sequence; in another a warp counts what stands before its sequence, which
// needs no order of arrival; a small batch is done in one. All are chains of round trips; 4 million comparisons for 2,000 sequences
// are nothing to 152 SMs.
#include <climits>

#include "pages.cuh"
#include "sm100.cuh"

namespace csa2 {
namespace {

constexpr int kWarps = 16;     // sequences a CTA takes
constexpr int kKeys = 4096;    // of the batch that it looks at together

// Scratch: of each sequence of the call its leader (INT_MAX: padding) and what they have in common.
struct Scratch {
    int32_t *lead, *common;
};
int64_t scratch_bytes(int64_t B) { return 2 * 4 * B; }
Scratch scratch_of(void* ws, int B) {
    int32_t* p = static_cast<int32_t*>(ws);
    return {p, p + B};
}

struct Args {
    Pages g;
    int B, least;
    const int32_t *seq, *n_tokens;
    int32_t *order, *first, *shared;
    Scratch ws;
    int32_t* dev_status;
};

__device__ __forceinline__ int row_of(const Args& a, int b) { return a.seq ? a.seq[b] : b; }

// Positions that sequence b has (0: it takes no part).
__device__ __forceinline__ int length_of(const Args& a, int b, int row) {
    const int64_t T = a.n_tokens[b];
    return row < 0 || row >= a.g.max_seqs || T < 0 ? 0 : (int)min(T, a.g.max_len());
}

__device__ __forceinline__ bool real(const Args& a, int page) { return page >= 0 && page < a.g.n_pages; }

// The page of position least - 1, or a number that no other sequence has.
__device__ __forceinline__ int key_of(const Args& a, int b) {
    const int row = row_of(a, b), at = (a.least - 1) / a.g.page_size;
    if (length_of(a, b, row) < a.least || at >= a.g.max_pages) return -1 - b;
    const int page = a.g.table[(int64_t)row * a.g.max_pages + at];
    return real(a, page) ? page : -1 - b;
}

__device__ __forceinline__ void check(const Args& a, int b) {
    const int row = row_of(a, b), T = a.n_tokens[b];
    if (row >= a.g.max_seqs) raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
    else if (row >= 0 && (T < 0 || T > a.g.max_len())) raise_status(a.dev_status, CSA2_DEV_BAD_LENGTH);
}

// Keys of n sequences from j0 on, by the whole CTA.
template <int kThreads, int kLoads>  // kLoads: keys a thread, whose three round trips overlap
__device__ __forceinline__ void stage_keys(const Args& a, int32_t* keys, int j0, int n) {
    for (int j = threadIdx.x; j < n; j += kThreads * kLoads) {
        int key[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) key[i] = j + kThreads * i < n ? key_of(a, j0 + j + kThreads * i) : -1;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            if (j + kThreads * i < n) keys[j + kThreads * i] = key[i];
    }
}

// The first of n keys that is `mine`, by a warp; -1: none.
__device__ __forceinline__ int find(const int32_t* keys, int n, int mine, int lane) {
    constexpr int kLook = 4;  // words of 32 keys at a look
    int at = -1;
    for (int j = 0; j < n && at < 0; j += 32 * kLook) {
        uint32_t same[kLook];
#pragma unroll
        for (int i = 0; i < kLook; ++i) {
            const int k = j + 32 * i + lane;
            same[i] = __ballot_sync(0xffffffffu, k < n && keys[min(k, n - 1)] == mine);
        }
#pragma unroll
        for (int i = kLook - 1; i >= 0; --i)
            if (same[i]) at = j + 32 * i + __ffs(same[i]) - 1;
    }
    return at;
}

// Positions that sequences b and `lead` have in common, by a warp.
__device__ __forceinline__ int in_common(const Args& a, int b, int lead, int lane) {
    const int r0 = row_of(a, b), r1 = row_of(a, lead);
    const int n = min(length_of(a, b, r0), length_of(a, lead, r1));
    const int32_t *x = a.g.table + (int64_t)r0 * a.g.max_pages, *y = a.g.table + (int64_t)r1 * a.g.max_pages;
    const int pages = (int)(((int64_t)n + a.g.page_size - 1) / a.g.page_size);
    int same = pages;
    constexpr int kAtOnce = 8;  // entries a lane whose loads are in flight together
    for (int k0 = 0; k0 < pages; k0 += 32 * kAtOnce) {
        int u[kAtOnce], v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int k = k0 + 32 * i + lane;
            u[i] = k < pages ? x[k] : 0;
            v[i] = k < pages ? y[k] : 0;
        }
        bool found = false;
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint32_t other = __ballot_sync(0xffffffffu, u[i] != v[i] || !real(a, u[i]));
            if (other && !found) {
                same = min(same, k0 + 32 * i + __ffs(other) - 1);
                found = true;
            }
        }
        if (found) break;
    }
    return (int)min((int64_t)n, (int64_t)same * a.g.page_size);
}

// Groups in the order of their leaders, members ascending, padding behind them: a sequence's slot is
// the number of those with a lower leader, and of those with the same one before it.
struct Place {
    int lower = 0, before = 0, least = INT_MAX;
    __device__ __forceinline__ void count(const int32_t* leads, const int32_t* commons, int j0, int n, int b, int mine, int lane) {
#pragma unroll 8
        for (int j = lane; j < n; j += 32) {
            const int l = leads[j], c = commons[j];
            lower += l < mine;
            before += l == mine && j0 + j < b;
            least = min(least, l == mine && j0 + j != mine ? c : INT_MAX);
        }
    }
    __device__ __forceinline__ void write(const Args& a, int b, int mine, int lane) {
        lower = __reduce_add_sync(0xffffffffu, lower);
        before = __reduce_add_sync(0xffffffffu, before);
        least = __reduce_min_sync(0xffffffffu, least);
        if (lane) return;
        const int slot = lower + before;
        a.order[slot] = b;
        a.first[slot] = mine == INT_MAX ? slot : lower;
        a.shared[slot] = mine == INT_MAX || least == INT_MAX ? 0 : least;
    }
};

__global__ void __launch_bounds__(32 * kWarps, 1) k_groups_compare(const __grid_constant__ Args a) {
    __shared__ int32_t keys[kKeys];
    __shared__ int left;
    sm100::grid_dep_wait();
    sm100::grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31, b = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int mine = b < a.B ? key_of(a, b) : 0;
    int lead = b < a.B && mine >= 0 ? -1 : b;  // -1: not found yet
    if (b < a.B && lane == 0) check(a, b);
    for (int j0 = 0; j0 < a.B; j0 += kKeys) {
        if (threadIdx.x == 0) left = 0;
        const int n = min(kKeys, a.B - j0);
        __syncthreads();
        stage_keys<32 * kWarps, 4>(a, keys, j0, n);
        if (lead < 0 && lane == 0) left = 1;
        __syncthreads();
        if (!left) break;
        if (lead < 0) {
            const int at = find(keys, n, mine, lane);
            if (at >= 0) lead = j0 + at;
        }
        __syncthreads();
    }
    if (b >= a.B) return;
    int common = 0;
    if (lead != b) {
        common = in_common(a, b, lead, lane);
        if (common < a.least) lead = b;
    }
    if (lane == 0) {
        a.ws.lead[b] = row_of(a, b) < 0 ? INT_MAX : lead;
        a.ws.common[b] = common;
    }
}

__global__ void __launch_bounds__(32 * kWarps, 1) k_groups_order(const __grid_constant__ Args a) {
    __shared__ int32_t leads[kKeys], commons[kKeys];
    sm100::grid_dep_wait();
    const int lane = threadIdx.x & 31, b = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int mine = b < a.B ? a.ws.lead[b] : 0;
    Place place;
    for (int j0 = 0; j0 < a.B; j0 += kKeys) {
        const int n = min(kKeys, a.B - j0);
        __syncthreads();
#pragma unroll 4
        for (int j = threadIdx.x; j < n; j += 32 * kWarps) {
            leads[j] = a.ws.lead[j0 + j];
            commons[j] = a.ws.common[j0 + j];
        }
        __syncthreads();
        place.count(leads, commons, j0, n, b, mine, lane);
    }
    if (b < a.B) place.write(a, b, mine, lane);
}

// A small batch, by one CTA without the second kernel's wait: 32 sequences with rows of 1,000 pages 6.5 us against
// 8.0, 48 with 140 6.8 against 8.6. One SM reads the rows, so 64 with 1,000 pages take 12.3 against 8.0.
constexpr int kSmall = 64, kSmallWarps = 32;
constexpr int64_t kSmallEntries = 1 << 15;

__global__ void __launch_bounds__(32 * kSmallWarps, 1) k_groups_small(const __grid_constant__ Args a) {
    __shared__ int32_t keys[kSmall], leads[kSmall], commons[kSmall];
    sm100::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    stage_keys<32 * kSmallWarps, 1>(a, keys, 0, a.B);
    if ((int)threadIdx.x < a.B) check(a, threadIdx.x);
    __syncthreads();
    for (int b = warp; b < a.B; b += kSmallWarps) {
        int lead = keys[b] >= 0 ? find(keys, a.B, keys[b], lane) : b, common = 0;
        if (lead != b) {
            common = in_common(a, b, lead, lane);
            if (common < a.least) lead = b;
        }
        if (lane == 0) {
            leads[b] = row_of(a, b) < 0 ? INT_MAX : lead;
            commons[b] = common;
        }
    }
    __syncthreads();
    for (int b = warp; b < a.B; b += kSmallWarps) {
        Place place;
        place.count(leads, commons, 0, a.B, b, leads[b], lane);
        place.write(a, b, leads[b], lane);
    }
}

template <typename K>
int launch(K* k, dim3 grid, int threads, void* stream, const Args& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, k, a);
    return check_launch("prefix_groups");
}

}  // namespace

cudaError_t preload_groups() {
    if (const cudaError_t e = preload_kernel(k_groups_small)) return e;
    if (const cudaError_t e = preload_kernel(k_groups_compare)) return e;
    return preload_kernel(k_groups_order);
}

}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_prefix_groups_workspace_size(int B) {
    return B > 0 ? ((size_t)scratch_bytes(B) + 255) & ~(size_t)255 : 0;
}

extern "C" int csa2_prefix_groups(const csa2_params* p, const csa2_pages* c, int B, const int32_t* seq,
                                  const int32_t* n_tokens, int least, int32_t* order, int32_t* first,
                                  int32_t* shared, void* workspace, size_t ws_bytes, int32_t* dev_status,
                                  void* stream) {
    Args a = {};
    if (const int rc = check_pages("prefix_groups", p, c, &a.g)) return rc;
    if (B < 0 || least < 1) return fail(CSA2_ERR_INVALID_ARG, "prefix_groups: negative size, or least below 1");
    if (B > 65535) return fail(CSA2_ERR_UNSUPPORTED, "prefix_groups: at most 65535 sequences");
    if (B == 0) return CSA2_OK;
    if (!seq && B > a.g.max_seqs) return fail(CSA2_ERR_INVALID_ARG, "prefix_groups: B beyond max_seqs needs seq");
    if (!n_tokens || !order || !first || !shared || !workspace)
        return fail(CSA2_ERR_INVALID_ARG, "prefix_groups: NULL buffer");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(CSA2_ERR_ALIGN, "prefix_groups: workspace must be 256-byte aligned");
    if ((int64_t)ws_bytes < scratch_bytes(B))
        return fail(CSA2_ERR_SHAPE, "prefix_groups: workspace smaller than csa2_prefix_groups_workspace_size");
    if (const int rc = ensure_loaded()) return rc;
    a.B = B;
    a.least = least;
    a.seq = seq;
    a.n_tokens = n_tokens;
    a.order = order;
    a.first = first;
    a.shared = shared;
    a.ws = scratch_of(workspace, B);
    a.dev_status = dev_status;
    if (B <= kSmall && B * (int64_t)a.g.max_pages <= kSmallEntries)
        return launch(k_groups_small, dim3(1), 32 * kSmallWarps, stream, a);
    if (const int rc = launch(k_groups_compare, dim3((B + kWarps - 1) / kWarps), 32 * kWarps, stream, a)) return rc;
    return launch(k_groups_order, dim3((B + kWarps - 1) / kWarps), 32 * kWarps, stream, a);
}
