// Pages of a cache: reserving, releasing, forking and compacting them, and writing rows.
//
// A page is free when its count in ref[] is 0, and the lowest-numbered free page is always
// taken first, in the order of the call's list: the state is ref[] and the table alone,
// results do not depend on timing, and no list of free pages has to be kept in step. The
// planning kernels are one CTA (a scan over ref[], a few rows of the table); the copies
// they plan run on every SM.
#include <climits>

#include "pages.cuh"
#include "rope.cuh"
#include "sm100.cuh"

namespace csa2 {

int check_pages(const char* name, const csa2_params* p, const csa2_pages* c, Pages* out) {
    const std::string n(name);
    if (!p) return fail(CSA2_ERR_INVALID_ARG, "params is NULL");
    if (!c) return fail(CSA2_ERR_INVALID_ARG, n + ": pages is NULL");
    if (p->head_dim != kD) return fail(CSA2_ERR_UNSUPPORTED, n + ": built for D=512");
    if (p->kv_format != CSA2_BF16 && p->kv_format != CSA2_E4M3)
        return fail(CSA2_ERR_UNSUPPORTED, n + ": pages hold BF16 or E4M3 rows");
    if (!c->pool || !c->table || !c->ref) return fail(CSA2_ERR_INVALID_ARG, n + ": NULL pool, table or ref");
    if (c->layers < 1 || c->n_pages < 1 || c->max_seqs < 1 || c->max_pages < 1)
        return fail(CSA2_ERR_INVALID_ARG, n + ": layers, n_pages, max_seqs and max_pages must be positive");
    if (c->page_size < 8 || c->page_size > 1024 || c->page_size % 8)
        return fail(CSA2_ERR_UNSUPPORTED, n + ": page_size must be a multiple of 8, 8 .. 1024");
    if ((int64_t)c->n_pages * c->page_size > INT_MAX || (int64_t)c->max_seqs * c->max_pages > INT_MAX)
        return fail(CSA2_ERR_UNSUPPORTED, n + ": more than 2^31 - 1 rows in a pool or entries in the table");
    out->pool = static_cast<uint8_t*>(c->pool);
    out->layer_bytes = c->layer_bytes;
    out->table = c->table;
    out->ref = c->ref;
    out->layers = c->layers;
    out->n_pages = c->n_pages;
    out->page_size = c->page_size;
    out->max_seqs = c->max_seqs;
    out->max_pages = c->max_pages;
    out->row_bytes = p->kv_format == CSA2_BF16 ? 2 * kD : kD;
    if (c->layers > 1 && c->layer_bytes < c->n_pages * out->page_bytes())
        return fail(CSA2_ERR_SHAPE, n + ": layer_bytes smaller than a layer's pages");
    if (!aligned16(c->pool) || !aligned16(c->ref) || c->layer_bytes % 16 ||
        (reinterpret_cast<uintptr_t>(c->table) & 3u))
        return fail(CSA2_ERR_ALIGN, n + ": pool, ref and layer_bytes must be 16-byte aligned, table 4-byte");
    return CSA2_OK;
}

namespace {

constexpr int kPlan = 1024;      // threads of a planning CTA
constexpr int kCopy = 256;       // threads of a copying CTA
constexpr int kSlice = 32768;    // bytes a copying CTA moves at a time
constexpr int kWriteWarps = 8;   // rows a CTA of k_page_write takes
constexpr int kOffsets = 1024;   // list entries whose offsets fit in shared memory
constexpr int kOwners = 4096;    // sequences whose owners do
constexpr int kFresh = 1024;     // free pages that do

// Scratch (256-byte aligned): offsets of reserve [longest list + 1] int64; then int32:
// owner [max_seqs], new pages [longest list], and three lists of n_pages. A list of sequences
// may be as long as there are sequences, or 1,024 with padding.
struct Scratch {
    int64_t* offset;
    int32_t *owner, *fresh, *list, *list2, *map;
    int32_t* count;  // compact: pages to move, pages in use
};

int64_t longest_list(int64_t max_seqs) { return max_seqs > kOffsets ? max_seqs : kOffsets; }

int64_t scratch_bytes(int64_t max_seqs, int64_t n_pages) {
    return 8 * (longest_list(max_seqs) + 1) + 4 * (max_seqs + longest_list(max_seqs) + 3 * n_pages + 2);
}

Scratch scratch_of(void* ws, const Pages& g) {
    Scratch s;
    s.offset = static_cast<int64_t*>(ws);
    s.owner = reinterpret_cast<int32_t*>(s.offset + longest_list(g.max_seqs) + 1);
    s.fresh = s.owner + g.max_seqs;
    s.list = s.fresh + longest_list(g.max_seqs);
    s.list2 = s.list + g.n_pages;
    s.map = s.list2 + g.n_pages;
    s.count = s.map + g.n_pages;
    return s;
}

// Exclusive sum over the CTA's kPlan threads; *total gets the sum. Two CTA barriers.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* total) {
    __shared__ T warp_sum[kPlan / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    T w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T up = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += up;
    }
    const T before = warp ? __shfl_sync(0xffffffffu, w, warp - 1) : T(0);
    *total = __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();  // warp_sum is free for the next call
    return before + inc - v;
}

// Four counts of ref[], from page `at` on; pages past the end read as used.
__device__ __forceinline__ int4 ref4(const Pages& g, int64_t at) {
    if (at + 4 <= g.n_pages) return *reinterpret_cast<const int4*>(g.ref + at);
    int4 v;
    v.x = at < g.n_pages ? g.ref[at] : 1;
    v.y = at + 1 < g.n_pages ? g.ref[at + 1] : 1;
    v.z = at + 2 < g.n_pages ? g.ref[at + 2] : 1;
    v.w = 1;
    return v;
}

// The `want` lowest free pages into list[], by the whole CTA; returns how many there are.
// `first` holds the counts of pages 4 tid .. + 3, requested by the caller ahead of time.
__device__ int lowest_free(const Pages& g, int64_t want, int32_t* list, int4 first) {
    int64_t have = 0;
    int4 v = first;
    for (int64_t base = 0; base < g.n_pages && have < want; base += 4 * kPlan) {
        const int64_t at = base + 4 * (int64_t)threadIdx.x;
        const int4 nx = ref4(g, at + 4 * kPlan);  // the next round's, on its way during this one
        const int f0 = v.x <= 0, f1 = v.y <= 0, f2 = v.z <= 0, f3 = v.w <= 0;
        int total;
        int64_t k = have + block_scan(f0 + f1 + f2 + f3, &total);
        if (f0) { if (k < want) list[k] = (int32_t)at; ++k; }
        if (f1) { if (k < want) list[k] = (int32_t)at + 1; ++k; }
        if (f2) { if (k < want) list[k] = (int32_t)at + 2; ++k; }
        if (f3) { if (k < want) list[k] = (int32_t)at + 3; ++k; }
        have += total;
        v = nx;
    }
    __syncthreads();
    return (int)min(have, want);
}

// ---------------------------------------------------------------- reserve
// The entries of all sequences' ranges form one list, walked kPlan at a time: entry e of
// the list belongs to the sequence whose offsets enclose it, and its rank among the
// entries that lack a page says which free page it takes.
__global__ void __launch_bounds__(kPlan)
k_page_reserve(Pages g, int N, const int32_t* seq, const int32_t* n_from,
               const int32_t* n_to, Scratch ws, int32_t* dev_status) {
    __shared__ int64_t off_s[kOffsets + 1];
    __shared__ int32_t owner_s[kOwners], list_s[kFresh];
    sm100::grid_dep_wait();
    const int tid = threadIdx.x;
    const int4 first_ref = ref4(g, 4 * (int64_t)tid);
    int32_t* owner = g.max_seqs <= kOwners ? owner_s : ws.owner;
    for (int i = tid; i < N; i += kPlan)
        if (seq[i] >= 0 && seq[i] < g.max_seqs) owner[seq[i]] = INT_MAX;
    __syncthreads();
    for (int i = tid; i < N; i += kPlan)
        if (seq[i] >= 0 && seq[i] < g.max_seqs) atomicMin(&owner[seq[i]], i);
    __syncthreads();
    int64_t* off = N <= kOffsets ? off_s : ws.offset;
    int64_t entries = 0;
    for (int i0 = 0; i0 < N; i0 += kPlan) {
        const int i = i0 + tid;
        int64_t n = 0;
        if (i < N && seq[i] >= 0) {
            const int s = seq[i], a = n_from[i], e = n_to[i];
            if (s >= g.max_seqs || owner[s] != i) raise_status(dev_status, CSA2_DEV_BAD_INDEX);
            else if (a < 0 || e > g.max_len()) raise_status(dev_status, CSA2_DEV_BAD_LENGTH);
            else if (e > a) n = ((int64_t)e + g.page_size - 1) / g.page_size - a / g.page_size;
        }
        int64_t total;
        const int64_t before = block_scan(n, &total);
        if (i < N) off[i] = entries + before;
        entries += total;
    }
    if (tid == 0) off[N] = entries;
    int32_t* list = entries <= kFresh ? list_s : ws.list;
    const int free = lowest_free(g, entries, list, first_ref);  // ends with a CTA barrier
    int taken = 0;
    for (int64_t e0 = 0; e0 < entries; e0 += kPlan) {
        const int64_t e = e0 + tid;
        int32_t* entry = nullptr;
        if (e < entries) {
            int lo = 0, hi = N;  // off[lo] <= e < off[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (off[mid] <= e) lo = mid;
                else hi = mid;
            }
            entry = g.table + (int64_t)seq[lo] * g.max_pages + n_from[lo] / g.page_size + (e - off[lo]);
            if (*entry >= 0) entry = nullptr;
        }
        int total;
        const int k = taken + block_scan(entry ? 1 : 0, &total);
        if (entry) {
            if (k < free) {
                const int32_t page = list[k];
                *entry = page;
                g.ref[page] = 1;
            } else {
                raise_status(dev_status, CSA2_DEV_NO_PAGE);
            }
        }
        taken += total;
    }
}

// ---------------------------------------------------------------- release
__global__ void __launch_bounds__(kCopy)
k_page_release(Pages g, const int32_t* seq, const int32_t* n_tokens,
               int window, int n_first, int32_t* dev_status) {
    sm100::grid_dep_wait();
    const int i = blockIdx.x, s = seq[i];
    if (s < 0) return;
    int64_t lo = 0, hi = g.max_pages;  // pages [lo, hi)
    bool bad = s >= g.max_seqs;
    if (!bad && n_tokens) {
        const int64_t T = n_tokens[i];
        if (T < 0 || T > g.max_len()) {
            if (threadIdx.x == 0 && blockIdx.y == 0) raise_status(dev_status, CSA2_DEV_BAD_LENGTH);
            return;
        }
        lo = n_first > 0 ? ((int64_t)n_first + g.page_size - 1) / g.page_size : 0;
        hi = window > 0 && T > window ? (T - window) / g.page_size : 0;
    }
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.y == 0) raise_status(dev_status, CSA2_DEV_BAD_INDEX);
        return;
    }
    int32_t* row = g.table + (int64_t)s * g.max_pages;
    for (int64_t k = lo + (int64_t)blockIdx.y * kCopy + threadIdx.x; k < hi; k += (int64_t)gridDim.y * kCopy) {
        if (row[k] < 0) continue;
        const int32_t page = atomicExch(&row[k], -1);  // a sequence listed twice: only one sees the page
        if (page < 0) continue;
        if (page < g.n_pages) atomicSub(&g.ref[page], 1);
        else raise_status(dev_status, CSA2_DEV_BAD_INDEX);
    }
}

// ---------------------------------------------------------------- fork
// Plan: fresh[i] = the new page that fork i copies rows into, -1: none to copy, -2: skipped.
__global__ void __launch_bounds__(kPlan)
k_fork_plan(Pages g, int N, const int32_t* parent, const int32_t* child,
            const int32_t* n_tokens, Scratch ws, int32_t* dev_status) {
    sm100::grid_dep_wait();
    sm100::grid_dep_launch_dependents();
    __shared__ int32_t owner_s[kOwners], list_s[kFresh];
    const int tid = threadIdx.x;
    const int4 first_ref = ref4(g, 4 * (int64_t)tid);
    int32_t* owner = g.max_seqs <= kOwners ? owner_s : ws.owner;
    for (int i = tid; i < N; i += kPlan) {
        const int c = child[i], p = parent[i];
        if (c >= 0 && c < g.max_seqs) owner[c] = INT_MAX;
        if (p >= 0 && p < g.max_seqs) owner[p] = INT_MAX;
    }
    __syncthreads();
    for (int i = tid; i < N; i += kPlan) {  // a child's owner is its first fork; a parent's is -1
        const int c = child[i], p = parent[i];
        if (c < 0) continue;
        if (c < g.max_seqs) atomicMin(&owner[c], i);
        if (p >= 0 && p < g.max_seqs) atomicMin(&owner[p], -1);
    }
    __syncthreads();
    int copies = 0;
    for (int i0 = 0; i0 < N; i0 += kPlan) {
        const int i = i0 + tid;
        int state = -2;
        if (i < N && child[i] >= 0) {
            const int c = child[i], p = parent[i];
            const int64_t T = n_tokens[i];
            if (c >= g.max_seqs || p < 0 || p >= g.max_seqs || owner[c] != i) {
                raise_status(dev_status, CSA2_DEV_BAD_INDEX);
            } else if (T < 0 || T > g.max_len()) {
                raise_status(dev_status, CSA2_DEV_BAD_LENGTH);
            } else {
                state = -1;
                if (T % g.page_size) {
                    const int page = g.table[(int64_t)p * g.max_pages + T / g.page_size];
                    if (page >= 0 && page < g.n_pages) state = 1;
                    else raise_status(dev_status, CSA2_DEV_BAD_INDEX);
                }
            }
        }
        int total;
        const int k = copies + block_scan(state == 1 ? 1 : 0, &total);
        if (i < N) ws.fresh[i] = state == 1 ? k : state;
        copies += total;
    }
    int32_t* list = copies <= kFresh ? list_s : ws.list;
    const int free = lowest_free(g, copies, list, first_ref);
    for (int i = tid; i < N; i += kPlan) {
        const int k = ws.fresh[i];
        if (k < 0) continue;
        if (k < free) {
            ws.fresh[i] = list[k];
            g.ref[list[k]] = 1;
        } else {
            ws.fresh[i] = -1;
            raise_status(dev_status, CSA2_DEV_NO_PAGE);
        }
    }
}

// Copies bytes [0, n) (a multiple of 16) by one CTA, eight 16-byte loads in flight a thread.
__device__ __forceinline__ void copy_bytes(uint8_t* dst, const uint8_t* src, int64_t n) {
    const uint4* s = reinterpret_cast<const uint4*>(src);
    uint4* d = reinterpret_cast<uint4*>(dst);
    const int64_t units = n / 16;
    for (int64_t u0 = threadIdx.x; u0 < units; u0 += 8 * kCopy) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (u0 + k * kCopy < units) v[k] = __ldcs(s + u0 + k * kCopy);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (u0 + k * kCopy < units) __stcs(d + u0 + k * kCopy, v[k]);
    }
}

// One CTA per (slice of a page's rows, layer) and fork; the CTAs of a fork also share the
// child's row of the table.
__global__ void __launch_bounds__(kCopy)
k_fork_copy(Pages g, int slices, const int32_t* parent, const int32_t* child,
            const int32_t* n_tokens, Scratch ws, int32_t* dev_status) {
    sm100::grid_dep_wait();
    const int i = blockIdx.y, fresh = ws.fresh[i];
    if (fresh == -2) return;
    const int64_t T = n_tokens[i];
    const int64_t full = T / g.page_size;
    const int32_t* prow = g.table + (int64_t)parent[i] * g.max_pages;
    int32_t* crow = g.table + (int64_t)child[i] * g.max_pages;
    if (fresh >= 0) {
        const int layer = blockIdx.x / slices, slice = blockIdx.x % slices;
        const int64_t n = (T % g.page_size) * g.row_bytes, at = (int64_t)slice * kSlice;
        if (at < n) {
            uint8_t* base = g.pool + layer * g.layer_bytes;
            copy_bytes(base + fresh * g.page_bytes() + at, base + prow[full] * g.page_bytes() + at,
                       min((int64_t)kSlice, n - at));
        }
    }
    for (int64_t k = (int64_t)blockIdx.x * kCopy + threadIdx.x; k < g.max_pages; k += (int64_t)gridDim.x * kCopy) {
        const int32_t old = crow[k];
        int32_t page = -1;
        if (k < full) {
            page = prow[k];
            if (page >= 0 && page < g.n_pages) atomicAdd(&g.ref[page], 1);
            else page = -1;
        } else if (k == full) {
            page = fresh;
        }
        crow[k] = page;
        if (old >= 0 && old < g.n_pages) atomicSub(&g.ref[old], 1);
        else if (old >= 0) raise_status(dev_status, CSA2_DEV_BAD_INDEX);
    }
}

// ---------------------------------------------------------------- compact
// Sixteen neighbouring pages a thread: 16,384 a sweep, whose counts stay in registers where
// one sweep holds the pool.
constexpr int kSweep = 16 * kPlan;

// Bits 0..15: which of pages at .. at + 15 are used.
__device__ __forceinline__ uint32_t used16(const Pages& g, int64_t at) {
    int4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = ref4(g, at + 4 * q);
    uint32_t bits = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        bits |= ((v[q].x > 0 ? 1u : 0u) | (v[q].y > 0 ? 2u : 0u) | (v[q].z > 0 ? 4u : 0u) | (v[q].w > 0 ? 8u : 0u)) << (4 * q);
    const int64_t in = g.n_pages - at;  // ref4 reads pages past the end as used
    return in >= 16 ? bits : in <= 0 ? 0u : bits & ((1u << in) - 1u);
}

__global__ void __launch_bounds__(kPlan)
k_compact_plan(Pages g, Scratch ws, int32_t* n_used) {
    sm100::grid_dep_wait();
    sm100::grid_dep_launch_dependents();
    const int tid = threadIdx.x;
    uint32_t bits = 0;
    int mine = 0;
    for (int64_t base = 0; base < g.n_pages; base += kSweep) {
        bits = used16(g, base + 16 * (int64_t)tid);
        mine += __popc(bits);
    }
    int used;
    block_scan(mine, &used);
    int from = 0, to = 0;  // pages to move so far, free pages below `used` so far
    for (int64_t base = 0; base < g.n_pages; base += kSweep) {
        const int64_t at = base + 16 * (int64_t)tid;
        if (g.n_pages > kSweep) bits = used16(g, at);
        const int64_t below = min(max((int64_t)used - at, (int64_t)0), (int64_t)16);  // of the 16, pages < used
        const int64_t in = min(max((int64_t)g.n_pages - at, (int64_t)0), (int64_t)16);
        const uint32_t low = (1u << below) - 1u, all = (1u << in) - 1u;
        uint32_t gaps = ~bits & low & all, moves = bits & ~low & all;
        int total;  // moves in the low half, gaps in the high half (at most 16,384 each)
        const int before = block_scan(__popc(moves) | __popc(gaps) << 16, &total);
        int f = from + (before & 0xffff), t = to + (before >> 16);
        for (; gaps; gaps &= gaps - 1) ws.list2[t++] = (int32_t)at + __ffs(gaps) - 1;
        for (; moves; moves &= moves - 1) ws.list[f++] = (int32_t)at + __ffs(moves) - 1;
        for (uint32_t idle = ~bits & ~low & all; idle; idle &= idle - 1) {  // nothing to follow
            const int32_t page = (int32_t)at + __ffs(idle) - 1;
            ws.map[page] = page;
        }
        from += total & 0xffff;
        to += total >> 16;
    }
    __syncthreads();
    // (map[] is filled from page `used` on: pages below it stay)
    for (int i0 = tid; i0 < from; i0 += 8 * kPlan) {
        int32_t a[8], b[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + k * kPlan < from) a[k] = ws.list[i0 + k * kPlan], b[k] = ws.list2[i0 + k * kPlan];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i0 + k * kPlan < from) ws.map[a[k]] = b[k];
    }
    if (tid == 0) {
        ws.count[0] = from;
        ws.count[1] = used;
        if (n_used) *n_used = used;
    }
}

// Moves the planned pages and their counts (from above the used count to below it: no move
// reads what another writes) and renames the table's entries.
__global__ void __launch_bounds__(kCopy)
k_compact_move(Pages g, Scratch ws, int32_t* dev_status) {
    sm100::grid_dep_wait();
    const int64_t slices = (g.page_bytes() + kSlice - 1) / kSlice;
    const int64_t items = (int64_t)*ws.count * g.layers * slices;
    for (int64_t n = blockIdx.x; n < items; n += gridDim.x) {
        const int64_t page = n / slices, at = (n - page * slices) * kSlice;
        const int layer = (int)(page % g.layers);
        const int64_t i = page / g.layers;
        uint8_t* base = g.pool + layer * g.layer_bytes;
        copy_bytes(base + ws.list2[i] * g.page_bytes() + at, base + ws.list[i] * g.page_bytes() + at,
                   min((int64_t)kSlice, g.page_bytes() - at));
    }
    for (int i = blockIdx.x * kCopy + threadIdx.x; i < ws.count[0]; i += gridDim.x * kCopy) {
        const int32_t a = ws.list[i];
        g.ref[ws.list2[i]] = g.ref[a];
        g.ref[a] = 0;
    }
    const int used = ws.count[1];
    const int64_t entries = (int64_t)g.max_seqs * g.max_pages;
    for (int64_t e = (int64_t)blockIdx.x * kCopy + threadIdx.x; e < entries; e += (int64_t)gridDim.x * kCopy) {
        const int32_t page = g.table[e];
        if (page < used) continue;
        if (page < g.n_pages) g.table[e] = ws.map[page];
        else raise_status(dev_status, CSA2_DEV_BAD_INDEX);
    }
}

// ---------------------------------------------------------------- write
// One warp per row: lane holds channels 4 lane + 128 k (k = 0..3), so a pair stays in a
// thread and every access is contiguous over the warp.
template <typename X, bool kBf16>
__global__ void __launch_bounds__(32 * kWriteWarps)
k_page_write(Pages g, int layer, int64_t N, const X* x, int64_t x_row,
             const int32_t* seq, const int32_t* pos,
             const __grid_constant__ RopeTable tab, int32_t* dev_status) {
    sm100::grid_dep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
    if (i >= N) return;
    const int s = seq[i], p = pos[i];
    float4 v[4];
    const X* row = x + i * x_row + 4 * lane;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(X) == 4) {
            v[k] = __ldcs(reinterpret_cast<const float4*>(row + 128 * k));
        } else {
            const uint2 u = __ldcs(reinterpret_cast<const uint2*>(row + 128 * k));
            v[k] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                               __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
        }
    }
    if (s < 0) return;
    if (s >= g.max_seqs) {
        if (lane == 0) raise_status(dev_status, CSA2_DEV_BAD_INDEX);
        return;
    }
    if (p < 0 || p >= g.max_len()) {
        if (lane == 0) raise_status(dev_status, CSA2_DEV_BAD_LENGTH);
        return;
    }
    const int page = g.table[(int64_t)s * g.max_pages + p / g.page_size];
    if (page < 0 || page >= g.n_pages) {
        if (lane == 0) raise_status(dev_status, CSA2_DEV_BAD_INDEX);
        return;
    }
    uint8_t* dst = g.pool + layer * g.layer_bytes + page * g.page_bytes() + (int64_t)(p % g.page_size) * g.row_bytes;
    const int first = kD - tab.dim;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int ch = 4 * lane + 128 * k;
        if (ch >= first) {
            const float2 a = rope_cs(tab.turns[(ch - first) / 2], p), b = rope_cs(tab.turns[(ch - first) / 2 + 1], p);
            v[k] = make_float4(v[k].x * a.x - v[k].y * a.y, v[k].x * a.y + v[k].y * a.x,
                               v[k].z * b.x - v[k].w * b.y, v[k].z * b.y + v[k].w * b.x);
        }
        if constexpr (kBf16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v[k].x, v[k].y), hi = __floats2bfloat162_rn(v[k].z, v[k].w);
            *reinterpret_cast<uint2*>(dst + 2 * ch) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        } else {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[k].x, v[k].y), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[k].z, v[k].w), __NV_SATFINITE, __NV_E4M3);
            *reinterpret_cast<uint32_t*>(dst + ch) = lo | (hi << 16);
        }
    }
}

// Programmatic launch: the CTAs may be placed while the kernel ahead on the stream still
// runs; every kernel here waits for it (grid_dep_wait) before it reads or writes.
template <typename... P, typename... A>
int launch(const char* name, void (*k)(P...), dim3 grid, int threads, void* stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, k, args...);
    return check_launch(name);
}

int check_scratch(const char* name, const Pages& g, const void* ws, size_t bytes) {
    const std::string n(name);
    if (!ws) return fail(CSA2_ERR_INVALID_ARG, n + ": NULL workspace");
    if ((int64_t)bytes < scratch_bytes(g.max_seqs, g.n_pages))
        return fail(CSA2_ERR_SHAPE, n + ": workspace smaller than csa2_page_workspace_size");
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(CSA2_ERR_ALIGN, n + ": workspace must be 256-byte aligned");
    return CSA2_OK;
}

}  // namespace

cudaError_t preload_pages() {
    cudaError_t (*l[])() = {[] { return preload_kernel(k_page_reserve); },
                            [] { return preload_kernel(k_page_release); },
                            [] { return preload_kernel(k_fork_plan); },
                            [] { return preload_kernel(k_fork_copy); },
                            [] { return preload_kernel(k_compact_plan); },
                            [] { return preload_kernel(k_compact_move); },
                            [] { return preload_kernel(k_page_write<float, true>); },
                            [] { return preload_kernel(k_page_write<float, false>); },
                            [] { return preload_kernel(k_page_write<__nv_bfloat16, true>); },
                            [] { return preload_kernel(k_page_write<__nv_bfloat16, false>); }};
    for (auto f : l)
        if (const cudaError_t e = f()) return e;
    return cudaSuccess;
}

}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_page_workspace_size(const csa2_pages* c) {
    if (!c || c->max_seqs < 1 || c->n_pages < 1) return 0;
    return ((size_t)scratch_bytes(c->max_seqs, c->n_pages) + 255) & ~(size_t)255;
}

extern "C" int csa2_page_reserve(const csa2_params* p, const csa2_pages* c, int N, const int32_t* seq,
                                 const int32_t* n_from, const int32_t* n_to, void* workspace,
                                 size_t ws_bytes, int32_t* dev_status, void* stream) {
    Pages g;
    if (const int rc = check_pages("page_reserve", p, c, &g)) return rc;
    if (N < 0 || N > longest_list(g.max_seqs))
        return fail(CSA2_ERR_INVALID_ARG, "page_reserve: N must be 0 .. max(max_seqs, 1024)");
    if (N == 0) return CSA2_OK;
    if (!seq || !n_from || !n_to) return fail(CSA2_ERR_INVALID_ARG, "page_reserve: NULL buffer");
    if (const int rc = check_scratch("page_reserve", g, workspace, ws_bytes)) return rc;
    if (const int rc = ensure_loaded()) return rc;
    return launch("page_reserve", k_page_reserve, dim3(1), kPlan, stream, g, N, seq, n_from, n_to,
                  scratch_of(workspace, g), dev_status);
}

extern "C" int csa2_page_release(const csa2_params* p, const csa2_pages* c, int N, const int32_t* seq,
                                 const int32_t* n_tokens, int window, int n_first,
                                 int32_t* dev_status, void* stream) {
    Pages g;
    if (const int rc = check_pages("page_release", p, c, &g)) return rc;
    if (N < 0) return fail(CSA2_ERR_INVALID_ARG, "page_release: negative size");
    if (N == 0) return CSA2_OK;
    if (!seq) return fail(CSA2_ERR_INVALID_ARG, "page_release: NULL seq");
    if (const int rc = ensure_loaded()) return rc;
    int gy = (g.max_pages + 4 * kCopy - 1) / (4 * kCopy);
    if (gy > 64) gy = 64;
    return launch("page_release", k_page_release, dim3(N, gy), kCopy, stream, g, seq, n_tokens, window, n_first,
                  dev_status);
}

extern "C" int csa2_page_fork(const csa2_params* p, const csa2_pages* c, int N, const int32_t* parent,
                              const int32_t* child, const int32_t* n_tokens, void* workspace,
                              size_t ws_bytes, int32_t* dev_status, void* stream) {
    Pages g;
    if (const int rc = check_pages("page_fork", p, c, &g)) return rc;
    if (N < 0 || N > longest_list(g.max_seqs) || N > 65535)
        return fail(CSA2_ERR_INVALID_ARG, "page_fork: N must be 0 .. max(max_seqs, 1024), at most 65535");
    if (N == 0) return CSA2_OK;
    if (!parent || !child || !n_tokens) return fail(CSA2_ERR_INVALID_ARG, "page_fork: NULL buffer");
    if (const int rc = check_scratch("page_fork", g, workspace, ws_bytes)) return rc;
    if (const int rc = ensure_loaded()) return rc;
    const int slices = (int)((g.page_bytes() + kSlice - 1) / kSlice);
    if ((int64_t)slices * g.layers > INT_MAX) return fail(CSA2_ERR_UNSUPPORTED, "page_fork: too many layers");
    const Scratch ws = scratch_of(workspace, g);
    if (const int rc = launch("page_fork", k_fork_plan, dim3(1), kPlan, stream, g, N, parent, child, n_tokens, ws,
                              dev_status))
        return rc;
    return launch("page_fork", k_fork_copy, dim3(slices * g.layers, N), kCopy, stream, g, slices, parent, child,
                  n_tokens, ws, dev_status);
}

extern "C" int csa2_page_compact(const csa2_params* p, const csa2_pages* c, int32_t* n_used, void* workspace,
                                 size_t ws_bytes, int32_t* dev_status, void* stream) {
    Pages g;
    if (const int rc = check_pages("page_compact", p, c, &g)) return rc;
    if (const int rc = check_scratch("page_compact", g, workspace, ws_bytes)) return rc;
    if (const int rc = ensure_loaded()) return rc;
    const Scratch ws = scratch_of(workspace, g);
    if (const int rc = launch("page_compact", k_compact_plan, dim3(1), kPlan, stream, g, ws, n_used)) return rc;
    // a CTA moves 32 KB at a time; 6 of them an SM keep its copies in flight
    return launch("page_compact", k_compact_move, dim3(152 * 6), kCopy, stream, g, ws, dev_status);
}

extern "C" int csa2_page_write(const csa2_params* p, const csa2_pages* c, int layer, int64_t N, const void* x,
                               int x_format, int64_t x_row, const int32_t* seq, const int32_t* pos,
                               int32_t* dev_status, void* stream) {
    Pages g;
    if (const int rc = check_pages("page_write", p, c, &g)) return rc;
    if (N < 0 || layer < 0 || layer >= g.layers)
        return fail(CSA2_ERR_INVALID_ARG, "page_write: negative size or layer out of range");
    if (x_format != CSA2_F32 && x_format != CSA2_BF16)
        return fail(CSA2_ERR_UNSUPPORTED, "page_write: x_format must be F32 or BF16");
    if (p->rope_dim < 0 || p->rope_dim > kD || p->rope_dim % 4)
        return fail(CSA2_ERR_UNSUPPORTED, "page_write: rope_dim must be a multiple of 4 in [0, 512]");
    if (p->rope_dim > 0 && !rope_settings_ok(p))
        return fail(CSA2_ERR_INVALID_ARG,
                    "page_write: rope needs finite settings, theta, factor, orig_len > 0 and beta_fast > beta_slow");
    if (N > (int64_t)INT_MAX * kWriteWarps) return fail(CSA2_ERR_UNSUPPORTED, "page_write: too many rows");
    if (N == 0) return CSA2_OK;
    if (!x || !seq || !pos) return fail(CSA2_ERR_INVALID_ARG, "page_write: NULL buffer");
    if (N == 1) x_row = 0;  // not stepped by
    if (!aligned16(x) || x_row % (x_format == CSA2_F32 ? 4 : 8))
        return fail(CSA2_ERR_ALIGN, "page_write: rows of x must be 16-byte aligned");
    if (const int rc = ensure_loaded()) return rc;
    const RopeTable& tab = rope_table(p, p->rope_dim);
    const dim3 grid((unsigned)((N + kWriteWarps - 1) / kWriteWarps));
    const int th = 32 * kWriteWarps;
    const bool bf = p->kv_format == CSA2_BF16;
    if (x_format == CSA2_F32) {
        const float* xf = static_cast<const float*>(x);
        return bf ? launch("page_write", k_page_write<float, true>, grid, th, stream, g, layer, N, xf, x_row, seq, pos, tab, dev_status)
                  : launch("page_write", k_page_write<float, false>, grid, th, stream, g, layer, N, xf, x_row, seq, pos, tab, dev_status);
    }
    const __nv_bfloat16* xb = static_cast<const __nv_bfloat16*>(x);
    return bf ? launch("page_write", k_page_write<__nv_bfloat16, true>, grid, th, stream, g, layer, N, xb, x_row, seq, pos, tab, dev_status)
              : launch("page_write", k_page_write<__nv_bfloat16, false>, grid, th, stream, g, layer, N, xb, x_row, seq, pos, tab, dev_status);
}
