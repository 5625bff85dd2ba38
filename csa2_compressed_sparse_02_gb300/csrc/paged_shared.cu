// csa2_paged_attn_shared: csa2_paged_attn for a batch in which groups of sequences share their
// leading positions. The rows of a group's sequences (a row: a head of a sequence) meet a shared
// position together, so it is read once for up to 128 rows.
//
// A unit is up to 128 rows of one group: floor(128 / heads) sequences. It walks the tiles of 128
// positions of the shared prefix, which all its rows see, then those of each sequence's own
// positions, which only that sequence's rows see (the others' weights are zero there). With the
// rows as the MMA's M, over a pair of CTAs (tcgen05, cta_group::2, fp32 in TMEM):
//   S[128 x 128] = Q . K_tile^T,   P = 2^(S - m),   O[128 x 512] += P . V_tile
// CTA c of the pair has rows 64 c .. 64 c + 63 of Q, S, P and O. The pair shares the other operand:
// for S, CTA c brings positions 64 c .. + 63 with all their channels; for PV all 128 positions with
// channels 256 h + 128 c .. + 127 of both halves h. These are two copies of the tile's bytes (an
// operand's place in shared memory holds the same positions or channels in both CTAs, which differ
// between the two products), so a CTA streams 1,024 bytes a position in bf16, and each place of the
// ring comes free as soon as its own product has read it.
//
// Why a pair: O of 64 rows is 256 of a CTA's 512 TMEM columns, which leaves room for two S, so that the
// products of one tile run beside the softmax of another; 128 rows in one CTA would be all of it. And Q of
// 64 rows (64 KB) leaves shared memory for the rings.
//
// What bounds it. A tile's products take 2,048 cycles of the tensor pipe in bf16; in E4M3, whose S takes two
// products and PV three at twice the rate, 2,560. E4M3: the pipe is busy 90 % of the time (24 sequences of 64 heads
// behind 262,144 positions: 528 us cold, 539 in short bursts). bf16: the copies, 128 KB a tile and CTA, which by
// themselves reach 57 bytes a cycle (2,300 cycles), through rings of half a tile; the pipe is busy 71 % of the time where
// few pairs read the same rows at a time (24 behind 131,072: 252 us cold, 264 in short bursts, 1,560 TFLOP/s), so a tile
// takes 2,770 cycles there, and 2,450 where all do (152 behind 16,384: 186 us). Passes in a queue are 5 to 15 % slower, at
// the power limit. (S of two tiles as one product with N = 256 reads Q half as often, but needs the keys of both at a
// time: 305 us against 295.) Around the tiles: 11,000 cycles until the first S, 6,000 at the end of a unit, and a join of
// 6 to 13 us.
#include <climits>
#include <type_traits>

#include "attn.cuh"
#include "pages.cuh"
#include "sm100.cuh"

namespace csa2 {
namespace {
using namespace sm100;
using namespace attn;

constexpr int kTile = 128;      // positions
constexpr int kRows = 128;      // of a unit
constexpr int kMine = 64;       // of them a CTA's
constexpr int kMaxHeads = 64;
constexpr int kMaxPairs = 128;

struct Args {
    Pages g;
    const uint8_t* base;  // the layer's first page
    int B, heads, members;  // sequences a unit holds: kRows / heads
    int64_t q_seq, q_head;
    const __nv_bfloat16* q;
    const float* sink;
    const int32_t *seq, *n_tokens, *order, *first, *shared;
    __nv_bfloat16* out;
    int32_t* ends;    // workspace: of each pair, how its range ends [pairs]
    float* part;      // workspace: two partial results per pair
    uint8_t* q8;      // workspace, E4M3: the queries as their two parts [B][heads][2][512], and the logits'
    float* q_scale;   // factors [B][heads]
    int32_t* dev_status;
    float scale_log2;
    int pairs;
    int box_rows;     // rows of a copied box, 2^box_shift: divides 64 and the page size
    int box_shift;
};

// How a pair's range ends: its last unit goes on behind it; is its only one; and began before it.
enum { kCut = 1, kSingle = 2, kThrough = 4 };

// A partial result: O as [512 / 4][128 rows] float4, then m [128], l [128] and the rows' places in the
// output [128] (sequence x heads + head, -1: none).
constexpr int kPartFloats = kRows * (kD + 3);

__device__ __forceinline__ float* part_of(const Args& a, int pair, int slot) {
    return a.part + (2 * (int64_t)pair + slot) * kPartFloats;
}

// ---------------------------------------------------------------- the batch
// Slot i of the order: sequence b of the call (-1: padding, whose output is left as it is) with T
// positions in row `row` of the table (T = 0: nothing to see), in the group that begins at slot f and
// shares `sh` positions, which are read through row `prow`.
struct Slot {
    int b, T, row, f, sh, prow;
};

// Sequence b's row of the table: -1 padding, INT_MAX out of range.
__device__ __forceinline__ int row_of(const Args& a, int b, bool report) {
    if (b < 0 || b >= a.B) {
        if (report) raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
        return -1;
    }
    const int row = a.seq ? a.seq[b] : b;
    if (row < a.g.max_seqs) return max(row, -1);
    if (report) raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
    return INT_MAX;
}

__device__ __forceinline__ int length_of(const Args& a, int64_t n, bool report) {
    if (n >= 0 && n <= a.g.max_len()) return (int)n;
    if (report) raise_status(a.dev_status, CSA2_DEV_BAD_LENGTH);
    return n < 0 ? 0 : (int)a.g.max_len();
}

// The slot where the unit of slot i begins.
__device__ __forceinline__ int unit_of(const Args& a, int i, int f) { return i - (i - f) % a.members; }

// The slot where i's group begins. What `first` says of i holds if that slot begins a group and all slots of i's unit
// before i say the same; else i is a group of its own. So a unit's slots stand together, whatever `first` holds.
__device__ __forceinline__ int first_of(const Args& a, int i, bool report) {
    const int f = a.first[i];
    bool holds = f >= 0 && f <= i;
    if (holds && f < i) {
        holds = a.first[f] == f;
        constexpr int kLook = 8;  // a unit of 16 heads in one round trip
        int j = unit_of(a, i, f);
        do {
#pragma unroll
            for (int k = 0; k < kLook; ++k) holds &= a.first[min(j + k, i)] == f;
            j += kLook;
        } while (holds && j < i);
    }
    if (holds) return f;
    if (report) raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
    return i;
}

__device__ __forceinline__ Slot slot_of(const Args& a, int i, bool report) {
    Slot s;
    s.b = a.order[i];
    s.f = first_of(a, i, report);
    s.sh = length_of(a, a.shared[s.f], report && s.f == i);
    s.row = row_of(a, s.b, report);
    if (s.row < 0) s.b = -1;
    if (s.row == INT_MAX) s.row = -1;
    s.T = s.row < 0 ? 0 : length_of(a, a.n_tokens[s.b], report);
    s.prow = row_of(a, a.order[s.f], false);
    if (s.prow < 0 || s.prow == INT_MAX) s.sh = 0;  // no sequence to read them through
    return s;
}

__device__ __forceinline__ int tiles_of(int n) { return n / kTile + (n % kTile != 0); }

// Tiles that slot i brings: the prefix's, if its unit begins with it, and its own positions'.
__device__ __forceinline__ int prefix_tiles(const Args& a, const Slot& s, int i) {
    return unit_of(a, i, s.f) == i ? tiles_of(s.sh) : 0;
}
__device__ __forceinline__ int own_tiles(const Slot& s) { return s.T > s.sh ? tiles_of(s.T) - s.sh / kTile : 0; }

// ---------------------------------------------------------------- schedule
// The batch's tiles, unit after unit, are cut into one contiguous range a pair.
//  - As a rule of equal length: most pairs then have the end of one unit and the beginning of another.
//  - Where there are at most as many units as pairs, a unit may be cut into ceil(tiles / L) equal pieces, one a
//    pair, with the smallest L whose pieces fit the pairs: the longest range is longer, but a pair has one
//    piece. kSecondPiece says what the second one costs.
struct Range {
    int64_t items;
    int i, j;          // it begins with tile j of slot i
    bool cont, cut;    // its first unit began before it; its last one ends behind it
    int wave;          // ranges of equal length: it; else 0
};

// In tiles: its queries, its first tile's way through an empty pipeline and its partial result.
constexpr int kSecondPiece = 4;
constexpr int kTries = kSecondPiece + 1;  // values of L, from ceil(tiles / pairs) on

constexpr int kKept = 40;  // slots from the range's first unit on that stay in shared memory
struct PlanShared {
    Slot slots[kKept];
    int base;  // the first of them
    Range range;
};
struct PlanScratch {  // (where P comes later)
    int64_t warp_sum[32], starts[kMaxPairs];  // starts, tiles: of the units
    uint32_t tiles[kMaxPairs];
    int fits[32];
    long long at, end;        // the range
    int begins, ends;         // whether a unit begins at `at`, and one at `end`
};

// slot_of of all slots, a lane each (32 at most), which look at a group's first slot where its lane has it.
__device__ __forceinline__ Slot slots_of(const Args& a, int lane, bool report) {
    Slot s = {-1, 0, -1, lane, 0, -1};
    int shared = 0;
    if (lane < a.B) {
        s.b = a.order[lane];
        s.f = a.first[lane];
        shared = a.shared[lane];
        s.row = row_of(a, s.b, report);
    }
    // first_of, by votes: no slot of the unit names another than the one before it
    bool holds = s.f >= 0 && s.f <= lane;
    const int u0 = holds ? unit_of(a, lane, s.f) : lane, named = __shfl_sync(0xffffffffu, s.f, holds ? s.f : lane);
    const uint32_t other = __ballot_sync(0xffffffffu, s.f != __shfl_up_sync(0xffffffffu, s.f, 1));
    holds &= named == s.f && !(other & ((2u << lane) - (2u << u0)));
    if (!holds) s.f = lane;
    if (!holds && report) raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
    s.prow = __shfl_sync(0xffffffffu, s.row, s.f);
    shared = __shfl_sync(0xffffffffu, shared, s.f);
    if (lane >= a.B) return s;
    s.sh = length_of(a, shared, report && s.f == lane);
    if (s.row < 0) s.b = -1;
    if (s.row == INT_MAX) s.row = -1;
    s.T = s.row < 0 ? 0 : length_of(a, a.n_tokens[s.b], report);
    if (s.prow < 0 || s.prow == INT_MAX) s.sh = 0;
    return s;
}

// Up to 32 slots: by one warp, a slot a lane.
__device__ void plan_few(const Args& a, PlanShared& sh, int pair) {
    const int lane = threadIdx.x & 31;
    const Slot s = slots_of(a, lane, blockIdx.x == 0);
    const bool head = lane < a.B && unit_of(a, lane, s.f) == lane;
    const uint32_t n = lane < a.B ? (uint32_t)prefix_tiles(a, s, lane) + own_tiles(s) : 0;  // (below 2^26)
    const uint32_t here = warp_scan(n, lane), total = __shfl_sync(0xffffffffu, here + n, 31);
    const uint32_t heads = __ballot_sync(0xffffffffu, head), behind = lane < 31 ? heads & (~0u << (lane + 1)) : 0u;
    const uint32_t next = __shfl_sync(0xffffffffu, here, behind ? __ffs(behind) - 1 : 0);
    const uint32_t t = head ? (behind ? next : total) - here : 0;  // of the unit
    // piece c of k of x tiles, as in Cut: 32 bits hold all of it
    auto piece = [](uint32_t x, uint32_t k, uint32_t c) { return x / k * c + min(c, x % k); };
    uint32_t at = piece(total, a.pairs, pair), end = piece(total, a.pairs, pair + 1);
    int wave = (int)(total / a.pairs);
    if (__popc(heads) <= a.pairs && total > 0) {
        const uint32_t lo = (total + a.pairs - 1) / a.pairs;
        for (int tried = 0; tried < kTries; ++tried) {
            const uint32_t L = lo + tried;
            const uint32_t k = (t + L - 1) / L;
            if (__reduce_add_sync(0xffffffffu, k) > (uint32_t)a.pairs) continue;
            const int i = pair - (int)warp_scan(k, lane);
            const uint32_t mine = __ballot_sync(0xffffffffu, i >= 0 && i < (int)k);
            at = end = total;
            wave = 0;
            if (mine) {
                const int l = __ffs(mine) - 1;
                at = __shfl_sync(0xffffffffu, here + piece(t, max(k, 1u), i), l);
                end = __shfl_sync(0xffffffffu, here + piece(t, max(k, 1u), i + 1), l);
            }
            break;
        }
    }
    // (units of no tiles begin where the next one does)
    const uint32_t first = __reduce_max_sync(0xffffffffu, head && here <= at ? here : 0u);
    const uint32_t last = __reduce_min_sync(0xffffffffu, head && here >= end ? here : total);
    const uint32_t begins = __ballot_sync(0xffffffffu, at >= here && at - here < n);
    const int l = begins ? __ffs(begins) - 1 : 0;
    const int base = __shfl_sync(0xffffffffu, unit_of(a, lane, s.f), l);
    const uint32_t before = __shfl_sync(0xffffffffu, here, l);
    if (lane == 0) {
        sh.base = begins ? base : 0;
        sh.range = {(int64_t)(end - at), l, begins ? (int)(at - before) : 0, first < at, last > end, wave};
    }
    if (lane >= (begins ? base : 0) && lane < a.B) sh.slots[lane - (begins ? base : 0)] = s;
}

// Called by the whole CTA.
__device__ void plan(const Args& a, PlanShared& sh, PlanScratch& x, int pair) {
    static_assert(kKept >= 32, "plan_few keeps its slots");
    if (a.B <= 32) {  // 2.4 us (32 sequences; 80 take 4.1 the other way)
        if (threadIdx.x < 32) plan_few(a, sh, pair);
        __syncthreads();
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    // Exclusive sum over the CTA of n < 2^26, and the sum of all.
    auto scan = [&](uint32_t n, int64_t* all) {
        const uint32_t before = warp_scan(n, lane);
        if (lane == 31) x.warp_sum[warp] = (int64_t)before + n;
        __syncthreads();
        const int64_t w = lane < warps ? x.warp_sum[lane] : 0;
        int64_t warps_before = lane < warp ? w : 0, sum = w;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            warps_before += __shfl_xor_sync(0xffffffffu, warps_before, o);
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        __syncthreads();
        *all = sum;
        return warps_before + before;
    };
    Slot s = {};
    auto items_of = [&](int i, bool report, bool* head) -> uint32_t {
        *head = false;
        if (i >= a.B) return 0;
        s = slot_of(a, i, report);
        *head = unit_of(a, i, s.f) == i;
        return (uint32_t)prefix_tiles(a, s, i) + own_tiles(s);
    };
    const bool once = a.B <= (int)blockDim.x;  // a slot a thread
    int64_t total = 0, all, here = 0;
    uint32_t n = 0;
    bool head = false;
    for (int i0 = 0; i0 < a.B; i0 += blockDim.x) {
        n = items_of(i0 + tid, blockIdx.x == 0, &head);
        here = scan(n, &all);
        total += all;
    }
    const Cut ranges(total, a.pairs);
    if (tid == 0) {
        const int c = min(pair, ranges.n);
        x.at = ranges.at(c);
        x.end = ranges.at(min(c + 1, ranges.n));
        sh.range.i = sh.range.j = 0;
        sh.range.wave = (int)min(ranges.base, (int64_t)INT_MAX);
        sh.base = 0;
        x.begins = x.ends = 0;
    }
    if (once && total > 0) {
        int64_t units;
        const int unit = (int)scan(head ? 1u : 0u, &units) + head - 1;
        if (units <= a.pairs) {
            if (tid < kMaxPairs) x.tiles[tid] = 0;
            __syncthreads();
            if (n) atomicAdd(&x.tiles[max(unit, 0)], n);
            if (head) x.starts[unit] = here;
            __syncthreads();
            const uint32_t lo = (uint32_t)((total + a.pairs - 1) / a.pairs), t = tid < units ? x.tiles[tid] : 0;
            // The smallest L that is tried with sum ceil(tiles / L) <= pairs, a value a warp
            if (warp < kTries) {
                const uint32_t L = lo + warp;
                uint32_t k = 0;
                for (int u = lane; u < (int)units; u += 32) k += (x.tiles[u] + L - 1) / L;
                k = __reduce_add_sync(0xffffffffu, k);
                if (lane == 0) x.fits[warp] = k <= (uint32_t)a.pairs;
            }
            __syncthreads();
            const uint32_t good = __ballot_sync(0xffffffffu, lane < kTries && x.fits[lane]);
            if (good) {
                const uint32_t L = lo + __ffs(good) - 1;
                const uint32_t k = (t + L - 1) / L;
                if (tid == 0) x.at = x.end = total, sh.range.wave = 0;
                const int64_t c = pair - scan(k, &all);
                if (c >= 0 && c < k) {
                    x.at = x.starts[tid] + t * c / k;
                    x.end = x.starts[tid] + t * (c + 1) / k;
                }
            }
        }
    }
    __syncthreads();
    const int64_t at = x.at, end = x.end;
    int64_t before = 0;
    for (int i0 = 0; i0 < a.B; i0 += blockDim.x) {
        const int i = i0 + tid;
        if (!once) {
            n = items_of(i, false, &head);
            here = before + scan(n, &all);
            before += all;
        }
        if (at >= here && at < here + n) {
            sh.range.i = i;
            sh.range.j = (int)(at - here);
            sh.base = unit_of(a, i, s.f);
        }
        if (head && here == at) x.begins = 1;
        if (head && here == end) x.ends = 1;
    }
    __syncthreads();
    if (tid == 0) {
        sh.range.items = end - at;
        sh.range.cont = !x.begins;
        sh.range.cut = end < total && !x.ends;
    }
    if (once) {
        if (tid >= sh.base && tid < min(sh.base + kKept, a.B)) sh.slots[tid - sh.base] = s;
    } else if (tid < kKept && sh.base + tid < a.B) {
        sh.slots[tid] = slot_of(a, sh.base + tid, false);
    }
    __syncthreads();
}

// Slot i, which is not before the range's first unit: a slot's unit begins in it or behind it (first_of).
__device__ __noinline__ Slot slot_far(const Args& a, int i) { return slot_of(a, i, false); }
__device__ __forceinline__ Slot slot_at(const Args& a, const PlanShared& plan, int i) {
    return (uint32_t)(i - plan.base) < (uint32_t)kKept ? plan.slots[i - plan.base] : slot_far(a, i);
}

// A range tile by tile.
struct Tile {
    int t0, lo, hi;  // positions t0 .. t0 + 127, of which [lo, hi) are seen
    int row;         // of the table
    int k;           // the sequence of the unit that sees it, -1: all
    int u0, f;       // first slot of its unit and of its group
};
struct Walk {
    const Args& a;
    const PlanShared& plan;
    int64_t left;
    int i, j;
    Slot s;  // of slot i
    int pre, items, u0;
    int first, len, ahead;  // of the prefix's tiles the range has `len` from `first` on, and begins `ahead` of it
    __device__ __forceinline__ Walk(const Args& a, const PlanShared& plan)
        : a(a), plan(plan), left(plan.range.items), i(plan.range.i), j(plan.range.j) {
        if (left > 0) enter();
    }
    __device__ __forceinline__ void enter() {
        s = slot_at(a, plan, i);
        u0 = unit_of(a, i, s.f);
        pre = u0 == i ? tiles_of(s.sh) : 0;
        items = pre + own_tiles(s);
        // Ranges of equal length begin anywhere in a prefix. Each goes round its part of it so that the tile, modulo
        // that length, is the same for all at a time: pairs that read the same rows then do so together (44 sequences
        // of 64 heads behind 131,072 bf16 positions 452 us against 519, 24 272 against 291; 64 in E4M3 715 against 736).
        first = j;
        len = (int)min((int64_t)max(pre - j, 0), left);
        ahead = 0;
        if (const int wave = plan.range.wave; wave > 1 && len > 1) {
            const int at = (int)((plan.range.items - left + wave - j % wave) % wave);
            if (at < len) ahead = at;
        }
    }
    __device__ __forceinline__ bool next(Tile& t) {
        if (left <= 0) return false;
        while (j >= items) {
            ++i;
            j = 0;
            enter();
        }
        const bool own = j >= pre;
        t.u0 = u0;
        t.f = s.f;
        int tile = j + ahead;
        if (tile >= first + len) tile -= len;
        t.t0 = kTile * (own ? s.sh / kTile + j - pre : tile);
        t.lo = own ? s.sh : 0;
        t.hi = own ? s.T : s.sh;
        t.row = own ? s.row : s.prow;
        t.k = own ? i - u0 : -1;
        ++j;
        --left;
        return true;
    }
};

// What a row of a unit stands for: head `h` of sequence b (-1: nothing), which sees T positions.
struct Row {
    int b, h, k, T;
};
__device__ __noinline__ Row row_info(const Args& a, const PlanShared& plan, int u0, int f, int r) {
    Row x;
    x.k = r / a.heads;
    x.h = r - x.k * a.heads;
    x.b = -1;
    x.T = 0;
    const int i = u0 + x.k;
    if (x.k >= a.members || i >= a.B) return x;
    const Slot s = slot_at(a, plan, i);
    if (s.f != f) return x;
    x.b = s.b;
    x.T = s.T;
    return x;
}

// ---------------------------------------------------------------- shapes
// kBf16: bf16 pages, the products in bf16. Else E4M3 pages, whose bytes are the operand as they
// are; what meets them is split into 8-bit parts that add up to it:
//   q 2^s = hi + lo, both E4M3, with the largest |q| 2^s of a row in [2^7, 2^8): bf16's 8 bits
//   down to 2^-10 of the largest, to 2^-17 of it below; both products into the same S;
//   P in f16 = three parts in E5M2, each the nearest three bits of what is left.
template <bool kBf16>
struct Shape {
    static constexpr int kSoftWarps = 8;
    static constexpr int kScoreWarp = 8, kOutputWarp = 9, kKeyWarp = 10, kValueWarp = 11, kPlanWarp = 12;
    static constexpr int kHelp0 = 13, kHelpWarps = 3;  // (16 warps: 128 registers a thread)
    static constexpr int kThreads = 32 * (kHelp0 + kHelpWarps);
    static constexpr uint32_t kChunk = kMine * 128;            // 64 rows x 128 bytes, 128-byte swizzle
    static constexpr uint32_t kPlace = kBf16 ? 2 * kChunk : kChunk;  // 64 positions x 128 channels
    static constexpr int kKeys = kBf16 ? 4 : 7, kValues = kBf16 ? 4 : 6;  // places; a tile takes four of each
    static_assert(kValues >= 4, "finite_values finds a tile's values all in place");
    static constexpr uint32_t kWeights = (kBf16 ? 2 : 3) * kChunk;  // P: 64 positions a chunk; E4M3: 128, a part each
    static constexpr uint32_t kIdesc = (1u << 4) | ((128u >> 4) << 24);  // D fp32, M = 128 over the pair
    // N = 128 positions, both K-major; N = 256 channels, B MN-major. Types: bf16 1, E4M3 0, E5M2 1
    static constexpr uint32_t kIdescS = kIdesc | ((128u >> 3) << 17) | (kBf16 ? (1u << 7) | (1u << 10) : 0u);
    static constexpr uint32_t kIdescPV = kIdesc | ((256u >> 3) << 17) | (1u << 16) | (1u << 7) | (kBf16 ? 1u << 10 : 0u);
    // P = 2^(x - m + kLift), and m moves only where P would pass 2^(kLazyMax + kLift). E5M2 ends at
    // 1.75 x 2^15 and holds small values as multiples of 2^-16.
    static constexpr float kLazyMax = kBf16 ? 8.f : 6.f;
    static constexpr float kLift = kBf16 ? 0.f : 9.f;
    // A row's maximum as its threads exchange it. In bf16, rounded up, where room is short: what it bounds
    // need not be close, as bf16 weights are as exact at any scale, as long as they are normal numbers. From
    // 2^13 on, where a step is 64 and more, its other bits follow (exact_max).
    using Bound = std::conditional_t<kBf16, __nv_bfloat16, float>;
    // Tiles that add up in TMEM under one maximum (see csa2_paged_attn: of a long tail less than 2^-9
    // of the weight is lost); what came before is added in fp32.
    static constexpr int kRun = kBf16 ? 192 : 128;
};
constexpr uint32_t kColO = 0, kColS = 256;  // TMEM: O 2 x 128 columns, S 2 x 64
constexpr uint32_t kTmemCols = 512;         // one CTA an SM, so it takes them all

constexpr int kInfos = 4;
struct alignas(16) Info {
    enum {
        kFirst = 1, kLast = 2,    // of a run of at most kRun tiles
        kBegins = 4, kEnds = 8,   // the run begins, ends what this pair has of the unit
        kOpens = 16,              // which opens the pair's range
        kWhole = 32,              // and is all of the unit (set with kEnds)
        kStop = 64,               // no tile: the range is done
        kSeen = 128               // every row of the unit sees every position of the tile
    };
    int t0, lo, hi, k, u0, f, flags, pad;
    uint32_t ok[4];  // the positions whose page exists
    int y[16];       // the pool's row where each box of the tile begins
};

template <bool kBf16>
struct Shared {
    using S = Shape<kBf16>;
    uint8_t keys[S::kKeys][S::kPlace], values[S::kValues][S::kPlace];
    uint8_t q[8 * S::kChunk];
    uint8_t p[2][S::kWeights];  // by tile parity
    typename S::Bound red_max[2][4][kMine];
    Info info[kInfos];
    uint64_t key_full[S::kKeys], value_full[S::kValues];  // the even CTA's: the place is full in both
    uint64_t key_empty[S::kKeys], value_empty[S::kValues];
    uint64_t info_full[kInfos], info_empty[kInfos];
    uint64_t s_full[2], s_empty[2], p_full[2], pv_done[2];  // by tile parity; s_empty, p_full: the even CTA's
    uint64_t q_full[2];  // the even CTA's: both CTAs' rows are staged; by run parity
    uint64_t q_empty;
    uint64_t max_bar[2], sum_bar[2];
    uint64_t drain;
    PlanShared plan;
    uint32_t tmem_base;
    int value_asked, value_told;  // the even CTA's: the odd one's softmax waits for V of the tiles before this one; was told
    int value_here;   // the odd CTA's: it has landed (finite_values)
    int abort;
};

// mbar_wait_warp with the loop out of line: the roles' code runs side by side, and together it has to
// fit the instruction cache (see k_paged_shared).
__device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort) {
    for (uint32_t i = 0; i < kSpinLimit; ++i) {
        if (__all_sync(0xffffffffu, mbar_try_wait_at(bar, parity))) return true;
        if ((i & 255u) == 255u && __any_sync(0xffffffffu, *abort != 0)) return false;
    }
    *abort = 1;
    return false;
}
__device__ __forceinline__ bool ready(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait_at(bar, parity));
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return ready(smem_u32(bar), parity) || wait_on(smem_u32(bar), parity, abort);
}

// An arrive on the even CTA's barrier, from either CTA of the pair.
__device__ __forceinline__ void arrive_lead(uint64_t* bar, uint32_t rank) {
    if (rank == 0) mbar_arrive(bar);
    else mbar_arrive_peer(mapa_shared(smem_u32(bar), 0));
}

// What the odd CTA's softmax asks of the even one, on whose barriers both CTAs' copies count (finite_values): that
// V of a tile has landed. The even CTA's plan warp answers while it waits for a barrier of its own, with a release
// at the cluster's scope that covers the odd CTA's copies too. (The value loader, were it to look for requests between
// its tries: 24 sequences of 64 heads behind 131,072 bf16 positions 345 us against 290.)
template <bool kBf16>
__device__ __noinline__ bool wait_answering(Shared<kBf16>& sh, uint64_t* bar, uint32_t parity, int lane, volatile int* abort) {
    using S = Shape<kBf16>;
    for (uint32_t i = 0; i < kSpinLimit; ++i) {
        if (ready(smem_u32(bar), parity)) return true;
        if ((i & 255u) == 255u && __any_sync(0xffffffffu, *abort != 0)) return false;
        if (__shfl_sync(0xffffffffu, ld_relaxed_cluster(smem_u32(&sh.value_asked)), 0) <= sh.value_told) continue;
        const int asked = __shfl_sync(0xffffffffu, ld_acquire_cluster(smem_u32(&sh.value_asked)), 0);
        if (asked <= sh.value_told) continue;
        // Its PV waits for the answer and that of the tile before is done, so the phases that the barriers of its
        // places are in are this tile's.
        const int of = 4 * (asked - 1) + (lane & 3);
        const uint32_t phase = (uint32_t)((of / S::kValues) & 1);
        if (!wait(&sh.value_full[of % S::kValues], phase, abort)) return false;
        if (!__all_sync(0xffffffffu, acquire_phase_cluster(&sh.value_full[of % S::kValues], phase))) return false;
        if (lane == 0) {
            st_release_cluster(mapa_shared(smem_u32(&sh.value_here), 1), asked);
            sh.value_told = asked;
        }
        __syncwarp();
    }
    *abort = 1;
    return false;
}

// ---------------------------------------------------------------- tiles
// One warp walks the range and tells the other roles of each tile. Boxes (rows of one page) that hold
// nothing seen are copied from behind the pool's last row, which reads as zeros: P is zero for them,
// and 0 x whatever the place held before might be NaN.
template <bool kBf16>
__device__ void plan_role(Shared<kBf16>& sh, const Args& a, int lane, int rank, int pair, volatile int* abort) {
    using S = Shape<kBf16>;
    const int br = a.box_rows, shift = a.box_shift, ps = a.g.page_size;
    const int pos = lane << shift;  // of this lane's box in the tile
    const Range range = sh.plan.range;
    Walk walk(a, sh.plan);
    int run = 0, runs = 0, pieces = 0;
    // this lane's box: its page's entry is on its way while the tile before is told
    struct Box {
        int nth, page;  // of the row of the table, and its entry; nth < 0: not seen
    };
    auto look = [&](const Tile& t) {
        Box b = {-1, -1};
        if (pos < kTile && t.t0 + pos < t.hi && t.t0 + pos + (br - 1) >= t.lo) {  // (positions end at 2^31 - 2)
            b.nth = (int)((uint32_t)(t.t0 + pos) / (uint32_t)ps);
            b.page = t.row < 0 ? -1 : a.g.table[(int64_t)t.row * a.g.max_pages + b.nth];
        }
        return b;
    };
    // positions that every sequence of the unit sees, of the shared ones, and whether there is but one
    int reach = 0;
    bool alone = false;
    auto look_at_unit = [&](int u0, int f) {
        int n = INT_MAX, live = 0;
        for (int k = lane; k < a.members && u0 + k < a.B; k += 32) {
            const Slot s = slot_at(a, sh.plan, u0 + k);
            if (s.f != f || s.b < 0) continue;
            n = min(n, s.T);
            ++live;
        }
        reach = __reduce_min_sync(0xffffffffu, n);
        alone = __reduce_add_sync(0xffffffffu, live) == 1;
    };
    Tile cur = {}, nxt = {};
    Box box = {}, box_nx = {};
    bool has = walk.next(cur);
    if (has) box = look(cur);
    int gt = 0;
    for (; has; ++gt) {
        const bool more = walk.next(nxt);
        if (more) box_nx = look(nxt);
        if (runs == 0 && run == 0) look_at_unit(cur.u0, cur.f);
        const bool ends = !more || nxt.u0 != cur.u0 || nxt.f != cur.f;
        const bool last = ends || run == S::kRun - 1;
        if (gt >= kInfos && !(rank == 0 ? wait_answering(sh, &sh.info_empty[gt % kInfos], (uint32_t)((gt / kInfos - 1) & 1), lane, abort)
                                        : wait(&sh.info_empty[gt % kInfos], (uint32_t)((gt / kInfos - 1) & 1), abort)))
            return;
        const bool there = box.nth >= 0 && box.page >= 0 && box.page < a.g.n_pages;
        if (box.nth >= 0 && !there && rank == 0) raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
        const uint32_t held = __ballot_sync(0xffffffffu, there);
        const bool seen = (cur.k < 0 || alone) && cur.lo <= cur.t0 && min(cur.hi, reach) - cur.t0 >= kTile &&
                          __all_sync(0xffffffffu, there || pos >= kTile);
        Info& o = sh.info[gt % kInfos];
        if (pos < kTile) o.y[lane] = there ? box.page * ps + (cur.t0 + pos - box.nth * ps) : a.g.n_pages * ps;
        if (lane < 4) {
            uint32_t ok = 0;
#pragma unroll
            for (int p = 0; p < 32; p += 8)  // (a box has at least eight rows)
                if ((held >> ((32 * lane + p) >> shift)) & 1u) ok |= 0xffu << p;
            o.ok[lane] = ok;
        }
        if (lane == 0) {
            o.t0 = cur.t0;
            o.lo = cur.lo;
            o.hi = cur.hi;
            o.k = cur.k;
            o.u0 = cur.u0;
            o.f = cur.f;
            o.flags = (run == 0 ? Info::kFirst : 0) | (last ? Info::kLast : 0) | (runs == 0 ? Info::kBegins : 0) |
                      (ends ? Info::kEnds : 0) | (pieces == 0 ? Info::kOpens : 0) |
                      (ends && !(pieces == 0 && range.cont) && !(!more && range.cut) ? Info::kWhole : 0) |
                      (seen ? Info::kSeen : 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.info_full[gt % kInfos]);
        ++run;
        if (last) run = 0, ++runs;
        if (ends) runs = 0, ++pieces;
        has = more;
        // for the join
        if (!more && lane == 0 && rank == 0)
            a.ends[pair] = (range.cut ? kCut : 0) | (pieces == 1 ? kSingle : 0) | (pieces == 1 && range.cont ? kThrough : 0);
        cur = nxt;
        box = box_nx;
    }
    if (range.items <= 0 && lane == 0 && rank == 0) a.ends[pair] = 0;
    if (gt >= kInfos && !(rank == 0 ? wait_answering(sh, &sh.info_empty[gt % kInfos], (uint32_t)((gt / kInfos - 1) & 1), lane, abort)
                                    : wait(&sh.info_empty[gt % kInfos], (uint32_t)((gt / kInfos - 1) & 1), abort)))
        return;
    if (lane == 0) {
        sh.info[gt % kInfos].flags = Info::kStop;
        mbar_arrive(&sh.info_full[gt % kInfos]);
    }
    __syncwarp();
    // Up to the last tile's PV there may be questions. (A barrier of one phase: those of pv_done go on while this warp
    // is still busy with the last tiles' entries, and a phase that is two ahead reads as not complete.)
    if (rank == 0) wait_answering(sh, &sh.drain, 0, lane, abort);
}

// The tile's entry, as a warp reads it; false: the wait gave up.
template <bool kBf16>
__device__ __forceinline__ bool info_wait(Shared<kBf16>& sh, int gt, volatile int* abort) {
    return wait(&sh.info_full[gt % kInfos], (uint32_t)((gt / kInfos) & 1), abort);
}
template <bool kBf16>
__device__ __forceinline__ void info_done(Shared<kBf16>& sh, int gt, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.info_empty[gt % kInfos]);
}

// ---------------------------------------------------------------- copies
// One warp copies the keys, one the values, box by box. One elected lane issues, from values of the
// whole warp. Both CTAs' copies count on the even one's barrier, where the MMAs
// wait (a warp of the odd one that passed on that its places were full: 500 cycles later).
template <bool kBf16>
__device__ __noinline__ void load_role(Shared<kBf16>& sh, const Args& a, const CUtensorMap* tmap, bool keys, int lane,
                                       int rank, volatile int* abort) {
    using S = Shape<kBf16>;
    const int places = keys ? S::kKeys : S::kValues;
    uint64_t* const full = keys ? sh.key_full : sh.value_full;
    uint64_t* const empty = keys ? sh.key_empty : sh.value_empty;
    const uint32_t ring = smem_u32(keys ? sh.keys[0] : sh.values[0]);
    const uint32_t lead = mapa_shared(smem_u32(full), 0);
    const int shift = a.box_shift;
    int slot = 0, g = 0;
    uint32_t phase = 1;  // of a place that is free
    for (int gt = 0;; ++gt) {
        if (!info_wait(sh, gt, abort)) break;
        const Info& in = sh.info[gt % kInfos];
        const int flags = in.flags, y = in.y[lane & 15];
        if (flags & Info::kStop) break;
        info_done(sh, gt, lane);
        int i = 0;
#pragma unroll 1
        for (; i < 4; ++i) {
            // (a place that has not been in use: its barrier's phase before the first reads as complete)
            if (!wait(&empty[slot], phase, abort)) break;
            // 64 positions from `first` of the tile, 128 channels from x
            const int first = keys ? kMine * rank : kMine * (i & 1);
            const int x = keys ? 128 * i : 256 * (i >> 1) + 128 * rank;
            const uint32_t at = __shfl_sync(0xffffffffu, slot, 0);
            if (rank == 0 && elect_one()) mbar_arrive_expect_tx(&full[at], 2 * S::kPlace);
#pragma unroll 1
            for (int b = 0; b < kMine; b += a.box_rows) {
                const int yb = __shfl_sync(0xffffffffu, y, (first + b) >> shift);
                if (elect_one()) {
                    const uint32_t dst = ring + at * S::kPlace + b * 128;
                    tma_g2s_2d_pair(dst, tmap, x, yb, lead + 8 * at);
                    if constexpr (kBf16) tma_g2s_2d_pair(dst + S::kChunk, tmap, x + 64, yb, lead + 8 * at);
                }
            }
            __syncwarp();
            ++g;
            if (++slot == places) slot = 0, phase ^= 1u;
        }
        if (i < 4) break;
    }
    // Whatever ended the loop, no copy outlives the pair, which ends together. (Where a wait has given
    // up, the even CTA may have armed less than the odd one has asked for: a copy takes a microsecond.)
    if (rank == 0)
        for (int s = max(0, g - places); s < g; ++s) mbar_wait_drain(&full[s % places], (uint32_t)((s / places) & 1));
    if (*abort) __nanosleep(200000);
}

// ---------------------------------------------------------------- queries
// Three warps stage this CTA's rows of the unit, once a run. For the first one of a range the softmax's
// warps, which have nothing to do yet, take their share of the rows.
template <bool kBf16>
struct Stagers {
    static constexpr int kAll = Shape<kBf16>::kSoftWarps + Shape<kBf16>::kHelpWarps;
};

// A row's operand: 1,024 bytes, in E4M3 hi and lo.
template <bool kBf16>
__device__ __forceinline__ const uint8_t* row_bytes(const Args& a, int b, int h) {
    if constexpr (kBf16) return reinterpret_cast<const uint8_t*>(a.q + b * a.q_seq + h * a.q_head);
    else return a.q8 + ((int64_t)b * a.heads + h) * (2 * kD);
}

// Warp w of n: rows w, w + n and so on, which lane i knows as the warp's row i.
template <bool kBf16>
__device__ __noinline__ void stage_queries(Shared<kBf16>& sh, const Args& a, Row mine, int w, int n, int it, int lane, int rank) {
    using S = Shape<kBf16>;
    const uint8_t* const from = mine.b < 0 ? nullptr : row_bytes<kBf16>(a, mine.b, mine.h);
#pragma unroll 2
    for (int i = 0, r = w; r < kMine; ++i, r += n) {
        const auto* const row = reinterpret_cast<const uint8_t*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(from), i));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int u = lane + 32 * x;
            cp_async_16(smem_u32(sh.q) + (u >> 3) * S::kChunk + sw128(r, u & 7),
                        row ? row + 16 * u : reinterpret_cast<const uint8_t*>(a.q), row != nullptr);
        }
    }
    cp_async_wait_all();
    fence_proxy_async_smem();
    __syncwarp();
    // (of kAll arrivals; warp 0 makes those of the warps that took no part)
    if (lane < (w == 0 ? 1 + Stagers<kBf16>::kAll - n : 1)) arrive_lead(&sh.q_full[it & 1], rank);
}

template <bool kBf16>
__device__ __forceinline__ Row staged_row(const Args& a, const PlanShared& plan, int u0, int f, int w, int n, int lane, int rank) {
    Row mine = row_info(a, plan, u0, f, kMine * rank + min(w + n * lane, kMine - 1));
    if (w + n * lane >= kMine) mine.b = -1;  // (no row)
    return mine;
}

template <bool kBf16>
__device__ void query_role(Shared<kBf16>& sh, const Args& a, int warp, int lane, int rank, volatile int* abort) {
    using S = Shape<kBf16>;
    Walk walk(a, sh.plan);
    Tile t;
    int it = 0, run = 0, u0 = -1, f = -1;
    while (walk.next(t)) {
        if (t.u0 == u0 && t.f == f && run < S::kRun) {
            ++run;
            continue;
        }
        u0 = t.u0;
        f = t.f;
        run = 1;
        const int n = it ? S::kHelpWarps : Stagers<kBf16>::kAll;
        const Row mine = staged_row<kBf16>(a, sh.plan, u0, f, warp, n, lane, rank);
        if (it > 0) {
            // the rows into L2 while the run before still needs its own
            for (int i = 0, r = warp; r < kMine; ++i, r += n) {
                const int b = __shfl_sync(0xffffffffu, mine.b, i), h = __shfl_sync(0xffffffffu, mine.h, i);
                if (lane < 8 && b >= 0) prefetch_l2(row_bytes<kBf16>(a, b, h) + 128 * lane);
            }
            if (!wait(&sh.q_empty, (uint32_t)((it - 1) & 1), abort)) return;
        }
        stage_queries(sh, a, mine, warp, n, it, lane, rank);
        ++it;
    }
}

// ---------------------------------------------------------------- MMAs
// Two warps of the even CTA issue the pair's MMAs, one S, one PV: what a warp does between its MMAs
// (a look at a barrier takes 200 cycles and more) then falls into the other's. The lanes look at a
// product's barriers together, and it is issued in one go. S is up to two tiles ahead of the softmax.
template <int kPlaces>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ int nth(int i) const { return slot + i < kPlaces ? slot + i : slot + i - kPlaces; }
    __device__ __forceinline__ uint32_t parity(int i) const { return slot + i < kPlaces ? phase : phase ^ 1u; }
    __device__ __forceinline__ void step(int n = 1) {
        if ((slot += n) >= kPlaces) slot -= kPlaces, phase ^= 1u;
    }
};

// (the leading offset of V is in a descriptor's low word)
constexpr uint32_t kHigh = (1024u >> 4) | (1u << 14) | (kLayoutSw128 << 29);

template <bool kBf16>
__device__ void score_role(Shared<kBf16>& sh, uint32_t tmem, int lane, volatile int* abort) {
    using S = Shape<kBf16>;
    const uint32_t dQ = (uint32_t)smem_desc(smem_u32(sh.q), 16, 1024, kLayoutSw128);
    const uint32_t dK = (uint32_t)smem_desc(smem_u32(sh.keys[0]), 16, 1024, kLayoutSw128);
    Ring<S::kKeys> keys;
    int it = 0;
    bool last = true;  // the tile before was a run's last
    for (int gt = 0;; ++gt) {
        if (last) {  // a run begins, or the range is done
            if (!info_wait(sh, gt, abort)) return;
            if (*(volatile int*)&sh.info[gt % kInfos].flags & Info::kStop) return;
            if (!wait(&sh.q_full[it & 1], (uint32_t)((it >> 1) & 1), abort)) return;
            ++it;
        }
        const uint32_t at = tmem + kColS + (uint32_t)__shfl_sync(0xffffffffu, gt & 1, 0) * 64u;
#pragma unroll 1
        for (int d = 0; d < 4; ++d) {
            if (!(d & 1)) {  // half of the tile's places at a look: the rest is on its way behind S of the tile before
                uint64_t* bar = &sh.key_full[keys.nth(lane & 1)];
                uint32_t parity = keys.parity(lane & 1);
                if (d == 0 && lane >= 8) {
                    const bool read = lane >= 16 && gt >= 2;  // S of two tiles before
                    bar = read ? &sh.s_empty[gt & 1] : &sh.info_full[gt % kInfos];
                    parity = (uint32_t)(read ? (gt >> 1) - 1 : gt / kInfos) & 1u;
                }
                if (!wait(bar, parity, abort)) return;
                tc_fence_after();
                if (d == 0) {
                    last = *(volatile int*)&sh.info[gt % kInfos].flags & Info::kLast;
                    info_done(sh, gt, lane);
                }
            }
            const uint32_t k = dK + __shfl_sync(0xffffffffu, (uint32_t)keys.slot * (S::kPlace >> 4), 0);
            const uint32_t q = dQ + d * ((kBf16 ? 2 * S::kChunk : S::kChunk) >> 4);
            if (elect_one()) {
                if constexpr (kBf16) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_f16_pair(at, q + ((c * S::kChunk + 32 * i) >> 4), kHigh, k + ((c * S::kChunk + 32 * i) >> 4),
                                         kHigh, S::kIdescS, (c | i) != 0 ? 1u : (uint32_t)(d != 0));
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int part = 0; part < 2; ++part)
                            mma_f8_pair(at, q + ((4 * part * S::kChunk + 32 * i) >> 4), kHigh, k + ((32 * i) >> 4), kHigh,
                                        S::kIdescS, (i | part) != 0 ? 1u : (uint32_t)(d != 0));
                }
                tc_commit_pair(&sh.key_empty[keys.slot]);
                if (d == 3) tc_commit_pair(&sh.s_full[gt & 1]);
                if (d == 3 && last) tc_commit_pair(&sh.q_empty);
            }
            __syncwarp();
            keys.step();
        }
    }
}

template <bool kBf16>
__device__ void output_role(Shared<kBf16>& sh, uint32_t tmem, int lane, volatile int* abort) {
    using S = Shape<kBf16>;
    const uint32_t dP = (uint32_t)smem_desc(smem_u32(sh.p[0]), 16, 1024, kLayoutSw128);
    const uint32_t dV = (uint32_t)smem_desc(smem_u32(sh.values[0]), S::kChunk, 1024, kLayoutSw128);
    Ring<S::kValues> values;
    for (int gt = 0;; ++gt) {
        if (!info_wait(sh, gt, abort)) return;
        const int flags = *(volatile int*)&sh.info[gt % kInfos].flags;
        if (flags & Info::kStop) return;
        info_done(sh, gt, lane);
        const uint32_t weights = dP + __shfl_sync(0xffffffffu, (uint32_t)(gt & 1) * (S::kWeights >> 4), 0);
#pragma unroll 1
        for (int n = 0; n < 4; ++n) {
            if (!(n & 1)) {  // half of the tile's places at a look, as in score_role
                const bool weights_too = n == 0 && lane >= 16;
                if (!wait(weights_too ? &sh.p_full[gt & 1] : &sh.value_full[values.nth(lane & 1)],
                          weights_too ? (uint32_t)((gt >> 1) & 1) : values.parity(lane & 1), abort))
                    return;
                tc_fence_after();
            }
            const uint32_t v = dV + __shfl_sync(0xffffffffu, (uint32_t)values.slot * (S::kPlace >> 4), 0);
            const uint32_t p = weights + (n & 1) * ((kBf16 ? S::kChunk : 64u) >> 4);
            const uint32_t o = tmem + kColO + 128 * (n >> 1), more = (n & 1) || !(flags & Info::kFirst);
            if (elect_one()) {
                if constexpr (kBf16) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_f16_pair(o, p + ((32 * i) >> 4), kHigh, v + ((2048 * i) >> 4), kHigh, S::kIdescPV, i == 0 ? more : 1u);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int part = 0; part < 3; ++part)
                            mma_f8_pair(o, p + ((part * S::kChunk + 32 * i) >> 4), kHigh, v + ((4096 * i) >> 4), kHigh,
                                        S::kIdescPV, (i | part) == 0 ? more : 1u);
                }
                tc_commit_pair(&sh.value_empty[values.slot]);
                if (n == 3) tc_commit_pair(&sh.pv_done[gt & 1]);
            }
            __syncwarp();
            values.step();
        }
    }
}

// ---------------------------------------------------------------- softmax and epilogue
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n"
        " mov.b64 {%0, %1}, z;\n}" : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n"
        " mov.b64 {%0, %1}, z;\n}" : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%6, %7};\n"
        " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}"
        : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
// Zero if all logits are finite, else NaN.
__device__ __forceinline__ float all_finite(const float2 (&x)[16]) {
    float2 t[2] = {};
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i & 1] = fma2(x[i], make_float2(0.f, 0.f), t[i & 1]);
    return (t[0].x + t[0].y) + (t[1].x + t[1].y);
}
// The positions that are not finite in all rows of the warp, as what is not finite in a row of a page makes them (0 x
// infinity is NaN); a query's own NaN does not.
__device__ __forceinline__ uint32_t not_finite(const float2 (&x)[16]) {
    uint32_t which = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        which |= (uint32_t)((__float_as_uint(x[i].x) & 0x7f800000u) == 0x7f800000u) << (2 * i);
        which |= (uint32_t)((__float_as_uint(x[i].y) & 0x7f800000u) == 0x7f800000u) << (2 * i + 1);
    }
    return __reduce_and_sync(0xffffffffu, which);
}

// Makes zeros of what is not finite of positions 32 quarter + (the bits of `which`) in this CTA's
// places of V of tile gt.
template <bool kBf16>
__device__ __noinline__ bool finite_values(Shared<kBf16>& sh, uint32_t which, int gt, int quarter, int lane, int rank,
                                           volatile int* abort) {
    using S = Shape<kBf16>;
    // The tile's V has landed (once PV of the tile before has used what the places held, the phase that
    // their barriers are in is this tile's).
    if (gt > 0 && !wait(&sh.pv_done[(gt - 1) & 1], (uint32_t)((gt - 1) >> 1) & 1u, abort)) return false;
    if (rank) {  // (asked again and again: what another warp has asked for the tile before may come late)
        const uint32_t asked = mapa_shared(smem_u32(&sh.value_asked), 0);
        for (uint32_t i = 0; __any_sync(0xffffffffu, ld_acquire_cluster(smem_u32(&sh.value_here)) <= gt); ++i) {
            if (lane == 0 && i % 64 == 0) st_release_cluster(asked, gt + 1);
            if (i < kSpinLimit && !__any_sync(0xffffffffu, *abort)) continue;
            *abort = 1;
            return false;
        }
    }
    uint8_t* at[2];
    for (int h = 0; h < 2; ++h) {
        const int g = 4 * gt + 2 * h + (quarter >> 1), slot = g % S::kValues;
        if (!rank && !wait(&sh.value_full[slot], (uint32_t)((g / S::kValues) & 1), abort)) return false;
        at[h] = sh.values[slot];
    }
    fence_proxy_async_smem();
    constexpr int kUnits = kBf16 ? 32 : 16;  // of 16 bytes: 128 channels in each half
    if (lane < kUnits) {
        const int h = lane / (kUnits / 2), u = lane % (kUnits / 2);
        uint8_t* const from = (h ? at[1] : at[0]) + (u >> 3) * S::kChunk + (u & 7) * 16 + 32 * (quarter & 1) * 128;
        for (; which; which &= which - 1) {
            uint4* const x = reinterpret_cast<uint4*>(from + (__ffs(which) - 1) * 128);
            uint32_t v[4] = {x->x, x->y, x->z, x->w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (kBf16) {
                    if ((v[i] & 0x7f80u) == 0x7f80u) v[i] &= 0xffff0000u;
                    if ((v[i] & 0x7f800000u) == 0x7f800000u) v[i] &= 0x0000ffffu;
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        if (((v[i] >> k) & 0x7fu) == 0x7fu) v[i] &= ~(0xffu << k);
                }
            }
            *x = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
    return true;
}

// Whether a maximum that was rounded up to bf16 may be 64 or more above the logits that it stands for.
__device__ __forceinline__ bool wide_step(float top) { return fabsf(top) >= 8192.f && top != -INFINITY; }

// The rows' maxima to their last bits, of bf16 pages: of what is left of `mine`, this thread's own, below the rounded one
// `top`, two more words of 8 bits each, which the row's threads exchange as they did the first. (Truncated: what is left
// has one sign; beyond bf16's largest number it counts from that.) Two more phases of max_bar, from `met` on; a wait
// that gives up has set *abort.
__device__ __noinline__ float exact_max(Shared<true>& sh, float top, float mine, int met, int quarter, int grp, int r, int lane,
                                        volatile int* abort) {
    float have = top == INFINITY ? __uint_as_float(0x7f7f0000u) : top;
#pragma unroll 1
    for (int k = met; k < met + 2; ++k) {
        sh.red_max[k & 1][quarter][r] = __float2bfloat16_rz(mine - have);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.max_bar[grp]);
        if (!wait(&sh.max_bar[grp], (uint32_t)(k & 1), abort)) break;
        const auto* four = sh.red_max[k & 1];
        have += fmaxf(fmaxf((float)four[0][r], (float)four[1][r]), fmaxf((float)four[2][r], (float)four[3][r]));
    }
    return wide_step(top) && have == have ? have : top;  // (an infinity stays one)
}

// Warp (qd, ch): rows 32 (qd & 1) + lane of this CTA, positions 64 (qd >> 1) + 32 ch .. + 31 of the
// tile: lane quarter qd of TMEM, whose upper half holds the same rows' other 64 positions. Logits
// are in the log2 domain. A row's four threads agree on its maximum through shared memory; it is
// lazy, and where it moves the row's part of O is rescaled in TMEM.
template <bool kBf16>
__device__ void softmax_role(Shared<kBf16>& sh, const Args& a, uint32_t tmem, int warp, int lane, int rank, int pair,
                             volatile int* abort) {
    using S = Shape<kBf16>;
    const int qd = warp & 3, ch = warp >> 2, grp = qd & 1, quarter = 2 * (qd >> 1) + ch;
    const int r = 32 * grp + lane;                 // of this CTA's rows
    const int p0 = 32 * quarter;                   // first position
    const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
    float m = -INFINITY, l = 0.f, c = a.scale_log2;  // maximum and sum (this thread's share), logit factor
    float m_was = -INFINITY, l_was = 0.f;          // of the piece up to this run
    const float2 c0 = make_float2(0.f, 0.f);
    Row row = {-1, 0, 0, 0};
    int runs = 0;
    int met = 0;       // phases of max_bar so far
    bool last = true;  // the tile before was a run's last
    if (sh.plan.range.items > 0) {
        const int n = Stagers<kBf16>::kAll, w = S::kHelpWarps + warp;
        const int f = slot_at(a, sh.plan, sh.plan.range.i).f;
        stage_queries(sh, a, staged_row<kBf16>(a, sh.plan, sh.plan.base, f, w, n, lane, rank), w, n, 0, lane, rank);
    }
    for (int gt = 0;; ++gt) {
        if (last) {  // a run begins, or the range is done
            if (!info_wait(sh, gt, abort)) return;
            const Info& in = sh.info[gt % kInfos];
            if (in.flags & Info::kStop) return;
            row = row_info(a, sh.plan, in.u0, in.f, kMine * rank + r);
            m = -INFINITY;
            l = 0.f;
            if constexpr (!kBf16) c = row.b < 0 ? 0.f : a.q_scale[(int64_t)row.b * a.heads + row.h];
            ++runs;
        }
        {  // S, the tile's entry, and PV of two tiles before: P may be written again
            uint64_t* bar = lane < 8 ? &sh.s_full[gt & 1] : &sh.info_full[gt % kInfos];
            uint32_t parity = lane < 8 ? gt >> 1 : gt / kInfos;
            if (lane >= 16 && gt > 1) {
                bar = &sh.pv_done[gt & 1];
                parity = (gt >> 1) - 1;
            }
            if (!wait(bar, parity & 1u, abort)) return;
        }
        tc_fence_after();
        uint32_t sv[32];
        tmem_ld_32x32b_x32_nowait(tl + kColS + 64 * (gt & 1) + 32 * ch, sv);
        const Info& in = sh.info[gt % kInfos];
        const int flags = in.flags;
        last = flags & Info::kLast;
        uint32_t seen = ~0u;  // of this thread's positions; rows that stand for nothing see everything
        if (!(flags & Info::kSeen) && row.b >= 0) {
            const int lo = max(0, min(32, in.lo - in.t0 - p0));
            const int hi = in.k >= 0 && in.k != row.k ? 0 : max(0, min(32, min(in.hi, row.T) - in.t0 - p0));
            seen = in.ok[quarter] & (hi == 32 ? ~0u : (1u << hi) - 1u) & (lo == 32 ? 0u : ~0u << lo);
        }
        tmem_wait_ld_regs32(sv);
        tc_fence_before();
        info_done(sh, gt, lane);
        if (lane == 0) arrive_lead(&sh.s_empty[gt & 1], rank);
        float2 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            x[i] = mul2(make_float2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])), make_float2(c, c));
        // Positions whose logits are not finite, where a row may take nothing from them: it does not see them, or (of
        // bf16 pages) its logit is -infinity. (1 to 2 % of a bf16 batch's time: 24 behind 131,072 287 to 290 us, 128 of
        // 16 heads behind 32,768 115 to 117. Such a tile waits for its values first: 24 sequences behind 65,536, of which one's 64
        // queries are NaN, 880 us instead of 145.)
        uint32_t which = 0;
        float off = 0.f;  // not zero: such a position is in a tile that every row sees
        if (!(flags & Info::kSeen)) {
            if (__any_sync(0xffffffffu, all_finite(x) != 0.f)) which = not_finite(x);
            if (!__all_sync(0xffffffffu, seen == ~0u)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i].x = (seen >> (2 * i)) & 1u ? x[i].x : -INFINITY;
                    x[i].y = (seen >> (2 * i + 1)) & 1u ? x[i].y : -INFINITY;
                }
            }
        }
        float top = fmaxf(x[0].x, x[0].y);
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, fmaxf(x[i].x, x[i].y));
        const float mine = top;
        if constexpr (kBf16) sh.red_max[met & 1][quarter][r] = __float2bfloat16_ru(top);
        else sh.red_max[met & 1][quarter][r] = top;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.max_bar[grp]);
        if constexpr (kBf16)
            if (flags & Info::kSeen) off = all_finite(x);
        // P under the maximum so far, while the others' maxima are on their way; again in the few tiles
        // where the maximum moves. Rounded; the sum takes the values that the product multiplies.
        uint32_t w[16], part[kBf16 ? 1 : 3][8];
        float2 sum = c0;
        float alpha = 1.f;
        bool fresh = flags & Info::kFirst, known = false;
        for (;;) {
            if (!fresh) {
                const float sub = m == -INFINITY ? 0.f : S::kLift - m;
                sum = c0;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 e = add2(x[i], make_float2(sub, sub));
                    if constexpr (kBf16) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(ex2(e.x), ex2(e.y));
                        w[i] = *reinterpret_cast<const uint32_t*>(&v);
                        sum = add2(sum, make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)));
                    } else {
                        const __half2 v = __floats2half2_rn(ex2(e.x), ex2(e.y));
                        w[i] = *reinterpret_cast<const uint32_t*>(&v);
                    }
                }
            }
            if (known) break;
            if (!wait(&sh.max_bar[grp], (uint32_t)(met & 1), abort)) return;
            known = true;
            const auto* four = sh.red_max[met & 1];
            ++met;
            top = fmaxf(fmaxf((float)four[0][r], (float)four[1][r]), fmaxf((float)four[2][r], (float)four[3][r]));
            bool move = fresh || top > m + S::kLazyMax;
            if constexpr (kBf16) {  // (all four warps of these rows decide alike)
                if (__any_sync(0xffffffffu, move && wide_step(top))) {
                    top = exact_max(sh, top, mine, met, quarter, grp, r, lane, abort);
                    if (__any_sync(0xffffffffu, *abort)) return;
                    met += 2;
                    move = fresh || top > m + S::kLazyMax;
                }
            }
            if (!__any_sync(0xffffffffu, move)) break;
            if (move) {
                if (m != -INFINITY) alpha = ex2(m - top);
                m = top;
            }
            fresh = false;
        }
        if constexpr (kBf16)
            if (__any_sync(0xffffffffu, off != 0.f)) which = not_finite(x);
        if constexpr (!kBf16) {
            // A NaN loses itself in the first two parts' rounding and stays what is left of them, so the
            // last part holds it. What that one leaves out is at most half its step, and what it leaves of
            // w f16 holds: both differences are exact.
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t x0 = w[2 * k], x1 = w[2 * k + 1];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t q0 = (x0 + 0x00800080u) & 0xff00ff00u, q1 = (x1 + 0x00800080u) & 0xff00ff00u;
                    part[i][k] = __byte_perm(q0, q1, 0x7531);
                    x0 = h2_sub(x0, q0);
                    x1 = h2_sub(x1, q1);
                }
                part[2][k] = h2x2_to_e5m2x4(x0, x1);
                const uint32_t v0 = h2_sub(w[2 * k], h2_sub(x0, __byte_perm(part[2][k], 0u, 0x1404)));
                const uint32_t v1 = h2_sub(w[2 * k + 1], h2_sub(x1, __byte_perm(part[2][k], 0u, 0x3424)));
                sum = add2(sum, __half22float2(*reinterpret_cast<const __half2*>(&v0)));
                sum = add2(sum, __half22float2(*reinterpret_cast<const __half2*>(&v1)));
            }
        }
        l = fmaf(l, alpha, sum.x + sum.y);
        if (__any_sync(0xffffffffu, alpha != 1.f)) {  // (not in a run's first tile)
            if (!wait(&sh.pv_done[(gt - 1) & 1], (uint32_t)((gt - 1) >> 1) & 1u, abort)) return;  // O is that of the tile before
            tc_fence_after();
#pragma unroll 1
            for (int n = 0; n < 128; n += 32) {
                uint32_t ov[32];
                tmem_ld_32x32b_x32(tl + kColO + 128 * ch + n, ov);
#pragma unroll
                for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                tmem_st_32x32b_x32(tl + kColO + 128 * ch + n, ov);
            }
            tmem_wait_st();
        }
        if constexpr (kBf16) {
            uint8_t* dst = sh.p[gt & 1] + (qd >> 1) * S::kChunk;
#pragma unroll
            for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4*>(dst + sw128(r, 4 * ch + u)) = make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    *reinterpret_cast<uint4*>(sh.p[gt & 1] + i * S::kChunk + sw128(r, 2 * quarter + u)) =
                        make_uint4(part[i][4 * u], part[i][4 * u + 1], part[i][4 * u + 2], part[i][4 * u + 3]);
        }
        // A weight of zero takes nothing from a position, unless that is not finite: rows that do not see a position must
        // not notice what it holds, nor rows that a logit of -infinity takes it out of. Its products with the queries
        // tell. What is not finite of it becomes zero for PV; the other rows that see it have NaN weights.
        if (which && !finite_values(sh, which, gt, quarter, lane, rank, abort)) return;
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead(&sh.p_full[gt & 1], rank);
        if (!(flags & Info::kLast)) continue;

        // ---- the run's end: this thread has 128 channels of its row, 256 ch + 128 (qd >> 1) and on
        if (!wait(&sh.pv_done[gt & 1], (uint32_t)(gt >> 1) & 1u, abort)) return;
        tc_fence_after();
        // (in these rows of this tile's P: only the four warps that have them write there, in two tiles'
        // time, when all of them have come past here)
        float* const sums = reinterpret_cast<float*>(sh.p[gt & 1] + 32 * grp * 128);
        sums[32 * quarter + lane] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sum_bar[grp]);
        if (!wait(&sh.sum_bar[grp], (uint32_t)((runs - 1) & 1), abort)) return;
        float total = (sums[lane] + sums[32 + lane]) + (sums[64 + lane] + sums[96 + lane]);
        float top_of = m - S::kLift;  // what P and O are relative to
        float was = 0.f, now = 1.f;
        if (!(flags & Info::kBegins)) {
            const float M = fmaxf(m_was, top_of);
            was = m_was == -INFINITY ? 0.f : ex2(m_was - M);
            now = top_of == -INFINITY ? 0.f : ex2(top_of - M);
            total = fmaf(l_was, was, total * now);
            top_of = M;
        }
        m_was = top_of;
        l_was = total;
        const bool done = (flags & (Info::kEnds | Info::kWhole)) == (Info::kEnds | Info::kWhole);
        float scale = 1.f;
        if (done) {
            const float sink2 = a.sink && row.b >= 0 ? a.sink[row.h] * kLog2e : -INFINITY;
            const float M = fmaxf(top_of, sink2);
            const float f = top_of == -INFINITY ? 0.f : ex2(top_of - M);
            const float den = total * f + (sink2 == -INFINITY ? 0.f : ex2(sink2 - M));
            scale = den == 0.f ? 0.f : f / den;
        }
        const int R = kMine * rank + r, d0 = 256 * ch + 128 * (qd >> 1);
        float* const slot = part_of(a, pair, flags & Info::kOpens ? 0 : 1);
        float4* const kept = reinterpret_cast<float4*>(slot) + (d0 / 4) * kRows + R;
        __nv_bfloat16* const out = a.out + ((int64_t)max(row.b, 0) * a.heads + row.h) * kD + d0;
#pragma unroll 1
        for (int n = 0; n < 128; n += 64) {
            uint32_t ov[2][32];
            tmem_ld_32x32b_x32_nowait(tl + kColO + 128 * ch + n, ov[0]);
            tmem_ld_32x32b_x32_nowait(tl + kColO + 128 * ch + n + 32, ov[1]);
            tmem_wait_ld_regs32(ov[0]);
            tmem_wait_ld_regs32(ov[1]);
            if (row.b < 0) continue;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                float4 o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t* v = &ov[(i + k) >> 3][4 * ((i + k) & 7)];
                    o[k] = make_float4(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]));
                }
                if (!(flags & Info::kBegins)) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 b = kept[(n / 4 + i + k) * kRows];
                        o[k] = make_float4(fmaf(b.x, was, o[k].x * now), fmaf(b.y, was, o[k].y * now),
                                           fmaf(b.z, was, o[k].z * now), fmaf(b.w, was, o[k].w * now));
                    }
                }
                if (done) {
                    const bool none = scale == 0.f;
                    uint32_t v[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(none ? 0.f : o[k].x * scale, none ? 0.f : o[k].y * scale);
                        const __nv_bfloat162 z = __floats2bfloat162_rn(none ? 0.f : o[k].z * scale, none ? 0.f : o[k].w * scale);
                        v[2 * k] = *reinterpret_cast<const uint32_t*>(&y);
                        v[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&z);
                    }
                    if (reinterpret_cast<uintptr_t>(a.out) & 31u) {
                        *reinterpret_cast<uint4*>(out + n + 4 * i) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4*>(out + n + 4 * i + 8) = make_uint4(v[4], v[5], v[6], v[7]);
                    } else {
                        st_global_32(out + n + 4 * i, v);  // a whole sector of the row
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) kept[(n / 4 + i + k) * kRows] = o[k];
                }
            }
        }
        if (!done && quarter == 0) {
            slot[kRows * kD + R] = top_of;
            slot[kRows * (kD + 1) + R] = total;
            slot[kRows * (kD + 2) + R] = __int_as_float(row.b < 0 ? -1 : row.b * a.heads + row.h);
        }
        tc_fence_before();
    }
}

// Sixteen warps in seven roles, whose code runs side by side and competes for the instruction cache: with
// unrolled loops and every wait in line only 54 % of the fetches hit, and a tile took 1.5 times as long. So what a
// role repeats is short, and what is rare stands out of line.
template <bool kBf16>
__global__ void __launch_bounds__(Shape<kBf16>::kThreads, 1)
k_paged_shared(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tmap) {
    using S = Shape<kBf16>;
    extern __shared__ __align__(1024) uint8_t raw[];
    auto& sh = *reinterpret_cast<Shared<kBf16>*>(raw);
    if (smem_u32(raw) & 1023u) {  // (the operands' layout needs it, and there is no room to move up)
        if (threadIdx.x == 0) raise_status(a.dev_status, CSA2_DEV_TIMEOUT);
        return;
    }
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = (int)cluster_ctarank(), pair = blockIdx.x >> 1;
    volatile int* abort = &sh.abort;
    if (tid == 0) {
        for (int i = 0; i < S::kKeys; ++i) {
            mbar_init(&sh.key_full[i], 1);
            mbar_init(&sh.key_empty[i], 1);
        }
        for (int i = 0; i < S::kValues; ++i) {
            mbar_init(&sh.value_full[i], 1);
            mbar_init(&sh.value_empty[i], 1);
        }
        for (int i = 0; i < kInfos; ++i) {
            mbar_init(&sh.info_full[i], 1);
            mbar_init(&sh.info_empty[i], S::kSoftWarps + (rank ? 2 : 4));  // the softmax and MMA warps, the loaders
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 2 * S::kSoftWarps);
            mbar_init(&sh.pv_done[i], 1);
            mbar_init(&sh.s_empty[i], 2 * S::kSoftWarps);
            mbar_init(&sh.q_full[i], 2 * Stagers<kBf16>::kAll);
            mbar_init(&sh.max_bar[i], 4);
            mbar_init(&sh.sum_bar[i], 4);
        }
        mbar_init(&sh.q_empty, 1);
        sh.value_asked = sh.value_told = sh.value_here = 0;
        mbar_init(&sh.drain, 2);
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == S::kScoreWarp) tmem_alloc_pair(&sh.tmem_base, kTmemCols);
    // a programmatic launch: only the setup above may overlap the kernel ahead
    grid_dep_launch_dependents();
    tc_fence_before();
    cluster_arrive();
    if (tid == 0) prefetch_tmap(&tmap);
    grid_dep_wait();
    plan(a, sh.plan, *reinterpret_cast<PlanScratch*>(sh.p), pair);  // ends with a CTA barrier
    if (warp == S::kPlanWarp) plan_role<kBf16>(sh, a, lane, rank, pair, abort);  // (only with this CTA's barriers)
    cluster_wait();  // the other CTA's barriers are there
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0);
    if (warp < S::kSoftWarps) {
        softmax_role<kBf16>(sh, a, tmem, warp, lane, rank, pair, abort);
    } else if (warp == S::kScoreWarp || warp == S::kOutputWarp) {
        if (rank == 0) {
            if (warp == S::kScoreWarp) score_role<kBf16>(sh, tmem, lane, abort);
            else output_role<kBf16>(sh, tmem, lane, abort);
            // every MMA issued must finish before TMEM and shared memory are released
            __syncwarp();
            if (elect_one()) tc_commit_pair(&sh.drain);
            if (!mbar_wait_drain(&sh.drain, 0)) *abort = 1;
        }
    } else if (warp == S::kKeyWarp || warp == S::kValueWarp) {
        load_role<kBf16>(sh, a, &tmap, warp == S::kKeyWarp, lane, rank, abort);
    } else if (warp != S::kPlanWarp) {
        query_role<kBf16>(sh, a, warp - S::kHelp0, lane, rank, abort);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // nothing of the pair is in flight
    if (tid == 0 && sh.abort) raise_status(a.dev_status, CSA2_DEV_TIMEOUT);
    if (warp == S::kScoreWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
    __syncwarp();
    cluster_sync_all();
}

template <bool kBf16>
constexpr int smem_bytes() {
    return (int)sizeof(Shared<kBf16>);
}
static_assert(smem_bytes<true>() <= 227 * 1024 && smem_bytes<false>() <= 227 * 1024, "shared memory of a CTA");

// ---------------------------------------------------------------- queries for E4M3 pages
// A warp a row: hi and lo and the logits' factor, in a kernel of its own, as the staging warps took 10,000 cycles
// for the conversions of 64 rows (four short sequences 19.7 us against 22; 80 drafts 80 against 89; 80 sequences of
// 18 families 135 against 146).
constexpr int kQueryWarps = 8;

__global__ void __launch_bounds__(32 * kQueryWarps) k_shared_queries(const __grid_constant__ Args a) {
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * kQueryWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= (int64_t)a.B * a.heads) return;
    const int b = (int)(row / a.heads), h = (int)(row - (int64_t)b * a.heads);
    const uint4* const src = reinterpret_cast<const uint4*>(row_bytes<true>(a, b, h)) + 2 * lane;
    const uint4 v0 = __ldg(src), v1 = __ldg(src + 1);
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    float mx = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
    mx = warp_max(mx);
    const int s = max(-126, min(126, 7 - ((int)((__float_as_uint(mx) >> 23) & 0xffu) - 127)));
    const float two_s = __uint_as_float((uint32_t)(s + 127) << 23);
    uint32_t hi[4] = {}, lo[4] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        float x = __uint_as_float(w[k] << 16) * two_s, y = __uint_as_float(w[k] & 0xffff0000u) * two_s;
        x = fmaf(x, 0.f, x);  // infinity to NaN: E4M3 has none
        y = fmaf(y, 0.f, y);
        const uint32_t xy = e4m3x2(x, y);
        const float2 got = e4m3x2_to_float2(xy);
        hi[k >> 1] |= xy << (16 * (k & 1));
        lo[k >> 1] |= e4m3x2(x - got.x, y - got.y) << (16 * (k & 1));
    }
    uint4* const to = reinterpret_cast<uint4*>(a.q8 + row * (2 * kD)) + lane;
    to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    to[kD / 16] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (lane == 0) a.q_scale[row] = a.scale_log2 * __uint_as_float((uint32_t)(127 - s) << 23);
}

// ---------------------------------------------------------------- join
// The units that the ranges cut: o = sum_i O_i 2^(m_i - M) / (2^(sink - M) + sum_i l_i 2^(m_i - M)) over the
// pairs' partial results in order. What sees nothing gets its zeros here. A thread has a row and four
// channels and asks for four pieces at once. Many units: the four groups of a CTA have 16 channels of one,
// whose rows are then written 32 bytes at a time. Few units, which are cut into many pieces each: all have
// the same channels, and every group takes every fourth piece.
constexpr int kJoinGroups = 4, kJoinThreads = kRows * kJoinGroups;
constexpr int kBatch = 4;  // pieces

struct JoinShared {
    int first[kMaxPairs], pieces[kMaxPairs], units;  // of the units that are cut
    float4 sums[kJoinGroups][kRows];  // (many units: the result, 48 bytes a row)
    float2 tops[kJoinGroups][kRows];
};

// Where row R of a partial result goes, -1: nowhere. Where a wait of the kernel before gave up, the workspace may hold
// anything there.
__device__ __forceinline__ int place_of(const Args& a, const float* part, int R) {
    const int place = __float_as_int(__ldcg(part + kRows * (kD + 2) + R));
    return (uint32_t)place < (uint32_t)(a.B * a.heads) ? place : -1;
}

__device__ __forceinline__ void join_item(const Args& a, JoinShared& sh, bool few, int unit, int item) {
    const int R = threadIdx.x & (kRows - 1), group = threadIdx.x / kRows;
    const int cg = few ? item : kJoinGroups * item + group, step = few ? kJoinGroups : 1, n = sh.pieces[unit];
    const uint32_t s0 = sh.first[unit];
    // slots of the pieces: the first, and two further on each time from the pair behind it
    const float* const first = part_of(a, 0, 0) + (int64_t)s0 * kPartFloats;
    const float* const rest = part_of(a, 0, 0) + (int64_t)(s0 & ~1u) * kPartFloats;
    const int place = place_of(a, first, R), place_out = place_of(a, first, threadIdx.x >> 1 & (kRows - 1));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f, M = -INFINITY;
    auto add = [&](float4 v, float m, float l) {  // under the maximum M of both
        if (m == -INFINITY && l == 0.f) return;   // (nothing, or nothing seen; a sum of NaN is from logits that are)
        const float w = ex2(m - M);
        den = fmaf(l, w, den);
        acc = make_float4(fmaf(v.x, w, acc.x), fmaf(v.y, w, acc.y), fmaf(v.z, w, acc.z), fmaf(v.w, w, acc.w));
    };
    auto raise = [&](float top) {
        if (top == M) return;
        const float w = M == -INFINITY ? 0.f : ex2(M - top);
        den *= w;
        acc = make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w);
        M = top;
    };
#pragma unroll 1
    for (int i0 = few ? group : 0; i0 < n; i0 += step * kBatch) {
        float4 v[kBatch];
        float m[kBatch], l[kBatch], top = M;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int p = i0 + step * i;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            m[i] = -INFINITY;
            l[i] = 0.f;
            if (p < n) {
                const float* const at = p ? rest + (int64_t)p * (2 * kPartFloats) : first;
                v[i] = __ldcg(reinterpret_cast<const float4*>(at) + cg * kRows + R);
                m[i] = __ldcg(at + kRows * kD + R);
                l[i] = __ldcg(at + kRows * (kD + 1) + R);
            }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) top = fmaxf(top, m[i]);
        raise(top);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) add(v[i], m[i], l[i]);
    }
    if (few) {
        __syncthreads();  // (the item before has read them)
        sh.sums[group][R] = acc;
        sh.tops[group][R] = make_float2(M, den);
        __syncthreads();
        if (group) return;
#pragma unroll 1
        for (int g = 1; g < kJoinGroups; ++g) {
            const float2 o = sh.tops[g][R];
            raise(fmaxf(M, o.x));
            add(sh.sums[g][R], o.x, o.y);
        }
    }
    const float s2 = a.sink && place >= 0 ? a.sink[place % a.heads] * kLog2e : -INFINITY, top = fmaxf(M, s2);
    const float f = M == -INFINITY ? 0.f : ex2(M - top);
    den = den * f + (s2 == -INFINITY ? 0.f : ex2(s2 - top));
    const float inv = den == 0.f ? 0.f : f / den;
    const __nv_bfloat162 x = __floats2bfloat162_rn(inv == 0.f ? 0.f : acc.x * inv, inv == 0.f ? 0.f : acc.y * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(inv == 0.f ? 0.f : acc.z * inv, inv == 0.f ? 0.f : acc.w * inv);
    const uint2 o = make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
    if (few) {
        if (place >= 0) *reinterpret_cast<uint2*>(a.out + (int64_t)place * kD + 4 * cg) = o;
        return;
    }
    uint8_t* const rows = reinterpret_cast<uint8_t*>(sh.sums);
    __syncthreads();
    *reinterpret_cast<uint2*>(rows + 48 * R + 8 * group) = o;
    __syncthreads();
    if (threadIdx.x < 2 * kRows && place_out >= 0)
        *reinterpret_cast<uint4*>(a.out + (int64_t)place_out * kD + 16 * item + 8 * (threadIdx.x & 1)) =
            *reinterpret_cast<const uint4*>(rows + 48 * (threadIdx.x >> 1) + 16 * (threadIdx.x & 1));
}

__global__ void __launch_bounds__(kJoinThreads, 2) k_shared_join(const __grid_constant__ Args a) {
    __shared__ JoinShared sh;
    grid_dep_wait();
    const int tid = threadIdx.x;
    if (tid < 32) {  // 32 pairs at a time: the units that begin in a pair's range and end behind it
        constexpr int kWords = kMaxPairs / 32;
        int units = 0, ends[kWords];
        uint32_t through[kWords];
#pragma unroll
        for (int w = 0; w < kWords; ++w) ends[w] = 32 * w + tid < a.pairs ? __ldcg(a.ends + 32 * w + tid) : 0;
#pragma unroll
        for (int w = 0; w < kWords; ++w) through[w] = __ballot_sync(0xffffffffu, (ends[w] & (kCut | kThrough)) == (kCut | kThrough));
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int c = 32 * w + tid, e = ends[w];
            const bool begins = (e & kCut) && !(e & kThrough);
            const uint32_t all = __ballot_sync(0xffffffffu, begins);
            if (begins) {
                int n = 2;  // the unit's last pair is the first one behind that does not go through
                for (int k = c + 1; k + 1 < a.pairs && ((through[k >> 5] >> (k & 31)) & 1u); ++k) ++n;
                const int at = units + __popc(all & ((1u << tid) - 1u));
                sh.first[at] = 2 * c + (e & kSingle ? 0 : 1);  // its slot, counted over all pairs
                sh.pieces[at] = n;
            }
            units += __popc(all);
        }
        if (tid == 0) sh.units = units;
    } else {  // meanwhile, what sees nothing
        constexpr int kWarps = kJoinThreads / 32 - 1;
        for (int b = blockIdx.x * kWarps + (tid >> 5) - 1; b < a.B; b += gridDim.x * kWarps) {
            const int row = a.seq ? a.seq[b] : b;
            if (row < 0 || (row < a.g.max_seqs && length_of(a, a.n_tokens[b], false) > 0)) continue;
            uint4* out = reinterpret_cast<uint4*>(a.out + (int64_t)b * a.heads * kD);
            for (int u = tid & 31; u < a.heads * (kD / 8); u += 32) out[u] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
    __syncthreads();
    const bool few = sh.units * (kD / 4) <= (int)gridDim.x;
    const int each = few ? kD / 4 : kD / 4 / kJoinGroups;
    for (int item = blockIdx.x; item < sh.units * each; item += gridDim.x)
        join_item(a, sh, few, item / each, item % each);
}

// CTA pairs on the current device: one CTA per SM, at most max_ctas (but one pair). 0: no device.
int pairs_of(const csa2_params* p) {
    int n = sm_count();
    if (n <= 0) return 0;
    if (p->max_ctas > 0 && p->max_ctas < n) n = p->max_ctas;
    return n < 2 ? 1 : n / 2 < kMaxPairs ? n / 2 : kMaxPairs;
}

int64_t ends_bytes(int pairs) { return ((int64_t)pairs * 4 + 255) & ~(int64_t)255; }
int64_t part_bytes(int pairs) { return 2 * (int64_t)pairs * kPartFloats * 4; }
int64_t query_bytes(const csa2_params* p, int B) {
    return p->kv_format == CSA2_BF16 ? 0 : (int64_t)B * p->heads * (2 * kD + 4);
}
int64_t ws_need(const csa2_params* p, int pairs, int B) {
    return ends_bytes(pairs) + part_bytes(pairs) + query_bytes(p, B);
}

}  // namespace

cudaError_t preload_paged_shared() {
    cudaError_t (*l[])() = {[] { return preload_kernel(k_paged_shared<true>, smem_bytes<true>()); },
                            [] { return preload_kernel(k_paged_shared<false>, smem_bytes<false>()); },
                            [] { return preload_kernel(k_shared_queries); }, [] { return preload_kernel(k_shared_join); }};
    for (auto f : l)
        if (const cudaError_t e = f()) return e;
    return cudaSuccess;
}

}  // namespace csa2

using namespace csa2;

extern "C" size_t csa2_paged_attn_shared_workspace_size(const csa2_params* p, const csa2_pages* c, int B) {
    if (!p || !c || B <= 0 || p->heads < 1 || p->heads > kMaxHeads) return 0;
    const int pairs = pairs_of(p);
    return pairs > 0 ? (size_t)ws_need(p, pairs, B) : 0;
}

extern "C" int csa2_paged_attn_shared(const csa2_params* p, const csa2_pages* c, int layer, int B, const void* q,
                                      int64_t q_seq, int64_t q_head, const float* sink, const int32_t* seq,
                                      const int32_t* n_tokens, const int32_t* order, const int32_t* first,
                                      const int32_t* shared, void* out, void* workspace, size_t ws_bytes,
                                      int32_t* dev_status, void* stream) {
    Args a = {};
    if (const int rc = check_pages("paged_attn_shared", p, c, &a.g)) return rc;
    if (B < 0 || layer < 0 || layer >= a.g.layers)
        return fail(CSA2_ERR_INVALID_ARG, "paged_attn_shared: negative size or layer out of range");
    if (p->heads < 1 || p->heads > kMaxHeads || p->q_format != CSA2_BF16)
        return fail(CSA2_ERR_UNSUPPORTED, "paged_attn_shared: built for 1 .. 64 heads, BF16 queries");
    if (B > 65535) return fail(CSA2_ERR_UNSUPPORTED, "paged_attn_shared: at most 65535 sequences");
    if (B == 0) return CSA2_OK;
    if (!seq && B > a.g.max_seqs) return fail(CSA2_ERR_INVALID_ARG, "paged_attn_shared: B beyond max_seqs needs seq");
    if (!q || !n_tokens || !order || !first || !shared || !out || !workspace)
        return fail(CSA2_ERR_INVALID_ARG, "paged_attn_shared: NULL buffer");
    if (B == 1) q_seq = 0;  // strides that nothing is stepped by
    if (p->heads == 1) q_head = 0;
    if (!aligned16(q) || !aligned16(out) || q_seq % 8 || q_head % 8)
        return fail(CSA2_ERR_ALIGN, "paged_attn_shared: q's heads and out must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return fail(CSA2_ERR_ALIGN, "paged_attn_shared: workspace must be 256-byte aligned");
    if (const int rc = ensure_loaded()) return rc;
    const int pairs = pairs_of(p);
    if (pairs <= 0) return check_launch("paged_attn_shared: device");
    if ((int64_t)ws_bytes < ws_need(p, pairs, B))
        return fail(CSA2_ERR_SHAPE, "paged_attn_shared: workspace smaller than csa2_paged_attn_shared_workspace_size");
    a.base = a.g.pool + layer * a.g.layer_bytes;
    a.B = B;
    a.heads = p->heads;
    a.members = kRows / p->heads;
    a.q_seq = q_seq;
    a.q_head = q_head;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.sink = sink;
    a.seq = seq;
    a.n_tokens = n_tokens;
    a.order = order;
    a.first = first;
    a.shared = shared;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.ends = static_cast<int32_t*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ends_bytes(pairs));
    a.q8 = static_cast<uint8_t*>(workspace) + ends_bytes(pairs) + part_bytes(pairs);
    a.q_scale = reinterpret_cast<float*>(a.q8 + (int64_t)B * p->heads * (2 * kD));
    a.dev_status = dev_status;
    a.scale_log2 = p->softmax_scale * kLog2e;
    a.pairs = pairs;
    a.box_rows = a.g.page_size & -a.g.page_size;
    if (a.box_rows > kMine) a.box_rows = kMine;
    while ((1 << a.box_shift) < a.box_rows) ++a.box_shift;
    CUtensorMap rows = {};
    if (const int rc = encode_rows("paged_attn_shared", a.g, a.base, a.box_rows, &rows)) return rc;
    const bool bf16 = p->kv_format == CSA2_BF16;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    if (!bf16) {
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)(((int64_t)B * p->heads + kQueryWarps - 1) / kQueryWarps));
        cfg.blockDim = dim3(32 * kQueryWarps);
        cudaLaunchKernelEx(&cfg, k_shared_queries, a);
        if (const int rc = check_launch("paged_attn_shared: queries")) return rc;
    }
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(2 * pairs);
    cfg.blockDim = dim3(bf16 ? Shape<true>::kThreads : Shape<false>::kThreads);
    cfg.dynamicSmemBytes = bf16 ? smem_bytes<true>() : smem_bytes<false>();
    if (bf16) cudaLaunchKernelEx(&cfg, k_paged_shared<true>, a, rows);
    else cudaLaunchKernelEx(&cfg, k_paged_shared<false>, a, rows);
    if (const int rc = check_launch("paged_attn_shared")) return rc;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(4 * pairs);  // as many as run at once
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    cudaLaunchKernelEx(&cfg, k_shared_join, a);
    return check_launch("paged_attn_shared: join");
}
