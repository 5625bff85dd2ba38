// csa2_paged_attn: dense attention of one new token per sequence over a paged cache of
// latents (K = V), with a window, first tokens that stay visible and a sink logit.
//
// Per tile of 128 positions, with the positions as the MMA's M (tcgen05, fp32 in TMEM):
//   S^T[128 x heads] = K_tile[128 x 512] . Q^T,   P = 2^(S - m),   O^T[512 x heads] += V_tile^T . P^T
// The tile is the A operand of both products, from one copy in shared memory, in the pages' own
// type: bf16 MMAs, or 8-bit ones for E4M3, whose other operands come in 8-bit parts (see Shape).
//
// What bounds it. HBM: a position is 1,024 bytes in bf16 (512 in E4M3), read once (134.68 MB
// of DRAM reads for two sequences of 65,536). Shared memory: a tile of 64 heads moves 530 KB
// through it in bf16 (128 in, 192 for each product, P), 4.1k cycles at 128 bytes a cycle; and
// as one tile and the query fill it (208 KB), a tile's softmax stands between its two products,
// about 1.2k cycles in which nothing else can run. 16 sequences of 131,072 in bf16: 326 us with
// 16 heads (6.6 TB/s, 0.97 of the measured copy rate), 354 with 64 (6.1 TB/s, 0.90; 330 with
// every page in L2, 5.3k cycles a tile). E4M3: 289 us with 64 heads, 209 with up to 32 (3.7 and
// 5.1 TB/s; the rows decoded into f16 operands instead: 419 and 346). The MMAs, 64 a tile, take
// 3.4k of its 5.0k cycles with 64 heads: two tiles fit beside the query's two parts and P's
// three, and a place that PV frees is filled 1.5k to 2k cycles later, so the tensor cores wait
// now for the softmax, now for the copy. The builds with 64 heads use all 128 registers a thread
// and spill a little beside them: 24 bytes in bf16, 52 in E4M3.
//
// Schedule, from the lengths on the device. The positions a sequence sees lie in tiles of 128
// (its first tokens' tiles, then those from the window's start to its end).
//  - At most as many sequences as CTAs: sequence b is cut into ceil(tiles_b / L) pieces of
//    equal length, one CTA each, with the smallest L whose pieces fit the CTAs.
//  - More sequences, or lengths that pieces divide badly: the (sequence, tile) items of the
//    batch are cut into one contiguous range of equal length per CTA.
// A sequence in one piece is finished by its CTA; of a cut one every piece leaves a partial
// result (unnormalised O, running maximum m and sum l of each head), and k_paged_join joins
// them in order: o = sum_i O_i 2^{m_i - M} / (2^{sink - M} + sum_i l_i 2^{m_i - M}). Within a CTA
// the runs of a long piece (see Shape::kRun) are joined by the same rule.
#include <climits>

#include "attn.cuh"
#include "pages.cuh"
#include "sm100.cuh"

namespace csa2 {
namespace {
using namespace sm100;
using namespace attn;

constexpr int kTile = 128;
constexpr int kMaxHeads = 64;

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
    int2* pieces;     // workspace: of each sequence the CTAs of its first and last piece [B]
    float* part;      // workspace: two partial results per CTA
    int32_t* dev_status;
    float scale_log2;
    int ctas;         // of the attention kernel
    int box_rows;     // rows of a copied box, 2^box_shift: divides 128 and the page size
    int box_shift;
};

// O [heads][512], then m [heads] and l [heads]; a multiple of four, as the join reads float4
__host__ __device__ inline int64_t part_floats(int heads) { return ((int64_t)heads * (kD + 2) + 3) & ~(int64_t)3; }

// What sequence b of the call sees: positions [0, nf) and [lo, T), in `tiles` tiles.
struct View {
    uint32_t T, lo, nf;  // below 2^31
    int row;             // of the table; < 0: padding
    int first_tiles, lo_tile, tiles;
    __device__ __forceinline__ bool sees(uint32_t t) const { return t < T && (t >= lo || t < nf); }
    __device__ __forceinline__ uint32_t start(int j) const {
        return (uint32_t)(j < first_tiles ? j : lo_tile + j - first_tiles) * kTile;
    }
};

__device__ __forceinline__ View view_of(const Args& a, int b, bool report) {
    View v;
    int T = a.n_tokens[b];  // (the two loads do not wait for each other)
    v.row = a.seq ? a.seq[b] : b;
    if (v.row < 0) T = 0;
    if (v.row >= a.g.max_seqs) {
        if (report) raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
        T = 0;
    }
    if (T < 0 || T > a.g.max_len()) {
        if (report) raise_status(a.dev_status, CSA2_DEV_BAD_LENGTH);
        T = T < 0 ? 0 : (int)a.g.max_len();
    }
    const int lo = a.window > 0 ? max(0, T - a.window) : 0, nf = min(max(a.n_first, 0), lo);
    v.T = T;
    v.lo = lo;
    v.nf = nf;
    v.lo_tile = lo / kTile;
    v.first_tiles = min(nf / kTile + (nf % kTile != 0), v.lo_tile);
    v.tiles = v.first_tiles + T / kTile + (T % kTile != 0) - v.lo_tile;
    return v;
}

// The partial result of a piece of CTA c: slot 0 if the piece opens the CTA's range, else 1.
__device__ __forceinline__ float* part_of(const Args& a, int c, int slot) {
    return a.part + (2 * (int64_t)c + slot) * part_floats(a.heads);
}

// What a CTA has to do: `items` tiles from tile j of sequence b on.
struct Range {
    int64_t items;
    int b, j;
};

// A sequence's first and last CTA for the join, packed into an int2: y < x where nothing is
// seen; the sign of x says that its first piece does not open its CTA's range.
__device__ __forceinline__ int2 pieces_of(int c0, int c1, bool opens) {
    return make_int2(opens ? c0 : c0 | (int)0x80000000, c1);
}

constexpr int kPlanWarps = 32;  // at most
constexpr int kPlanSeqs = 255;  // sequences the first schedule plans for

// One piece per CTA leaves CTAs idle where the sequences do not divide well; equal ranges do
// not, but give most CTAs a second piece, whose query, first tile and partial result cost about
// a tile. Measured on 152 CTAs, pieces (tiles of the longest) against ranges: 100 sequences of
// 3 tiles 26 us (3) and 33 (2); 20 of 18 on average 28 (3) and 31 (3); 32 of 64 in E4M3 63 (16)
// and 62 (14); 100 of 63 205 (63) and 173 (42).
constexpr uint32_t kSecondPiece = 1;

// At most as many sequences as CTAs (and kPlanSeqs: one a thread). False, with nothing
// planned, where ranges are better.
__device__ bool plan_pieces(const Args& a, Range* sh) {
    __shared__ uint32_t warp_sum[2][kPlanWarps];
    __shared__ uint32_t tiles[kPlanSeqs];
    __shared__ int fits[kPlanWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const bool lead = blockIdx.x == 0;
    const uint32_t t = tid < a.B ? view_of(a, tid, lead).tiles : 0;
    if (tid < a.B) tiles[tid] = t;
    const uint32_t mine = __reduce_add_sync(0xffffffffu, t);
    if (lane == 0) warp_sum[0][warp] = mine;
    if (tid == 0) sh->items = 0;
    __syncthreads();
    // (below 2^32: 255 sequences of at most 2^24 tiles)
    const uint32_t all = __reduce_add_sync(0xffffffffu, lane < warps ? warp_sum[0][lane] : 0u);
    // The smallest L with sum_b ceil(tiles_b / L) <= CTAs: at least all / CTAs, and
    // all / (CTAs - B) is enough, as rounding up adds less than one a sequence. Every warp
    // tries one value a round.
    const uint32_t ctas = a.ctas, spare = ctas - a.B;
    uint32_t lo = max(1u, (uint32_t)(((uint64_t)all + ctas - 1) / ctas));                   // L >= lo
    uint32_t hi = max(lo, spare ? (uint32_t)(((uint64_t)all + spare - 1) / spare) : all);   // L <= hi
    while (lo < hi) {
        const uint32_t step = (hi - lo + warps - 1) / warps;
        const uint64_t cand = lo + (uint64_t)step * warp;
        bool ok = true;  // hi fits
        if (cand < hi) {
            uint32_t n = 0;
            for (int b = lane; b < a.B; b += 32) n += (tiles[b] + (uint32_t)cand - 1) / (uint32_t)cand;
            ok = __reduce_add_sync(0xffffffffu, n) <= ctas;
        }
        if (lane == 0) fits[warp] = ok;
        __syncthreads();
        const uint32_t good = __ballot_sync(0xffffffffu, lane < warps && fits[lane]);
        __syncthreads();
        // the first warp whose value fits: L is at most its value, and above the one before
        const uint32_t w = good ? __ffs(good) - 1 : warps;
        hi = (uint32_t)min((uint64_t)hi, lo + (uint64_t)step * w);
        if (w > 0) lo = (uint32_t)min((uint64_t)hi, lo + (uint64_t)step * (w - 1) + 1);
    }
    if ((uint32_t)(((uint64_t)all + ctas - 1) / ctas) + kSecondPiece < lo) return false;
    const uint32_t k = (t + lo - 1) / lo;
    uint32_t first = warp_scan(k, lane);
    if (lane == 31) warp_sum[1][warp] = first + k;
    __syncthreads();
    first += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[1][lane] : 0u);
    const int64_t i = (int64_t)blockIdx.x - first;
    if (i >= 0 && i < k) {
        sh->b = tid;
        sh->j = (int)(t * i / k);
        sh->items = t * (i + 1) / k - t * i / k;
    }
    if (lead && tid < a.B) a.pieces[tid] = pieces_of((int)first, (int)(first + k) - 1, true);
    __syncthreads();
    return true;
}

// Equal ranges of all items.
__device__ void plan_ranges(const Args& a, Range* sh) {
    __shared__ int64_t warp_sum[kPlanWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const bool lead = blockIdx.x == 0;
    // Exclusive sum over the CTA of n < 2^25, and the sum of all.
    auto scan = [&](uint32_t n, int64_t* all) {
        const uint32_t before = warp_scan(n, lane);
        if (lane == 31) warp_sum[warp] = before + n;
        __syncthreads();
        const int64_t w = lane < warps ? warp_sum[lane] : 0;
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
    if (tid == 0) sh->items = 0;
    int64_t total = 0;
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
        int64_t all;
        scan(b0 + tid < a.B ? view_of(a, b0 + tid, lead).tiles : 0, &all);
        total += all;
    }
    const Cut cut(total, a.ctas);
    const int c = min((int)blockIdx.x, cut.n);
    const int64_t at = cut.at(c), end = cut.at(min(c + 1, cut.n));
    int64_t before = 0;
    for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
        const int b = b0 + tid;
        const uint32_t n = b < a.B ? view_of(a, b, false).tiles : 0;
        int64_t all;
        const int64_t here = before + scan(n, &all);
        before += all;
        if (at >= here && at < here + n) {
            sh->b = b;
            sh->j = (int)(at - here);
            sh->items = end - at;
        }
        if (lead && b < a.B) {
            const int c0 = n ? cut.holder(here) : 0;
            a.pieces[b] = n ? pieces_of(c0, cut.holder(here + n - 1), cut.at(c0) == here) : make_int2(0, -1);
        }
    }
    __syncthreads();
}

// This CTA's range, from the lengths of all sequences; CTA 0 leaves every sequence's pieces in
// a.pieces. Called by the whole CTA (a multiple of 32 threads, 256 to 1,024).
__device__ void plan(const Args& a, Range* sh) {
    if (a.B <= a.ctas && a.B <= kPlanSeqs && plan_pieces(a, sh)) return;
    plan_ranges(a, sh);
}

// ---------------------------------------------------------------- shapes
// kBf16: bf16 pages, the products in bf16. Else E4M3 pages, whose bytes are the operand as they
// are; what meets them is split into 8-bit parts that add up to it:
//   q 2^s = hi + 2^-5 lo, both E4M3, as 2 NH columns of S (they hold bf16's 8 bits);
//   P in f16 = three parts in E5M2, one product each into the same O. Each part takes the
//   nearest three bits of what is left: of a value in [1, 2) that is 2^-3, 2^-7, then nothing.
// NH: the heads, rounded up to the columns of the MMAs (bf16 16, 32 or 64, E4M3 32 or 64).
template <bool kBf16, int NH>
struct Shape {
    static constexpr int kSoftWarps = 8;            // (16 of them: 361 us for the 64-head case above in bf16, 8: 347)
    static constexpr int kGroups = kSoftWarps / 4;  // of heads: one per four lane quarters
    static constexpr int NC = NH / kGroups;         // heads of a softmax warp
    static constexpr int kMmaWarp = kSoftWarps;
    static constexpr int kTmaWarp = kSoftWarps + 1;
    static constexpr int kHelp0 = kSoftWarps + 2;   // first of the warps that stage the query
    static constexpr int kHelpWarps = kBf16 ? 4 : 6;
    static constexpr int kThreads = 32 * (kHelp0 + kHelpWarps);
    // The ring's places hold 128 channels of a tile's positions each, so a tile has 4: what the
    // query and P leave of shared memory. bf16: a tile and the next one's first places. E4M3: two
    // tiles (64 heads) or two and a half.
    static constexpr int kPairs = kBf16 ? (NH == 64 ? 4 : NH == 32 ? 5 : 6) : NH == 64 ? 8 : 10;
    static constexpr int kChunks = kBf16 ? 2 : 1;   // of 128 bytes a row in a place
    static constexpr int kQRows = kBf16 ? NH : 2 * NH;
    static constexpr int kQChunks = kBf16 ? 8 : 4;
    static constexpr int kParts = kBf16 ? 1 : 3;    // of P
    static constexpr uint32_t kColS = 4 * NH;  // TMEM: O^T 4 x NH columns, then S^T (E4M3: two of them)
    // D fp32, N = NH (S of E4M3: its two parts), M = 128; S: both K-major, PV: both MN-major.
    // Types: bf16 1, E4M3 0, E5M2 1 (a kind of MMA each)
    static constexpr uint32_t kIdesc = (1u << 4) | ((128u >> 4) << 24);
    static constexpr uint32_t kIdescS = kIdesc | ((uint32_t)(kQRows >> 3) << 17) | (kBf16 ? (1u << 7) | (1u << 10) : 0u);
    static constexpr uint32_t kIdescPV =
        kIdesc | ((uint32_t)(NH >> 3) << 17) | (kBf16 ? 1u << 7 : 0u) | (1u << 10) | (1u << 15) | (1u << 16);
    // P: a row of NH heads per position, swizzled over its own width (128, 64 or 32 bytes)
    static constexpr uint32_t kPRow = (kBf16 ? 2 : 1) * NH;
    static constexpr uint32_t kPLayout = kPRow == 128 ? kLayoutSw128 : kPRow == 64 ? kLayoutSw64 : kLayoutSw32;
    __device__ static __forceinline__ uint32_t p_unit(int row, int unit) {  // byte of 16-byte unit `unit`
        const int x = kPRow == 128 ? row & 7 : kPRow == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
        return row * kPRow + ((unit ^ x) << 4);
    }
    // P = 2^(x - m + kLift), x - m <= kLazyMax before the maximum has to move. E5M2 ends at
    // 1.75 x 2^15 and holds small values as multiples of 2^-16, half a step off at most: with
    // the largest weight at 2^9 or more, 2^-26 of it (see kRun). (A kLazyMax of 3 would make that
    // 2^-29, but logits of a standard deviation of 3 in log2 then move the maximum in 4 of the first
    // 8 tiles, with 6 in 2.)
    static constexpr float kLazyMax = kBf16 ? 8.0f : 6.0f;
    static constexpr float kLift = kBf16 ? 0.f : 9.f;
    // Tiles that add up in TMEM under one maximum; those that follow start anew, and what came
    // before is added in fp32. The tensor cores align each product to the accumulator and leave out
    // what lies below 2^-25 of it, and E4M3's parts end at 2^-26: with a million positions at
    // 2^-26.1 of one before them in one accumulator, their 1.4 % of the weight were lost. Of
    // 16,384 positions it is below 2^-10 in bf16 (2^-25 a product and 2^-23 a sum of 16 of them) and
    // below 2^-9 in E4M3 (three products, and 2^-26 of the parts), whatever the length. An end costs
    // 12 to 15 us with 64 heads and 6 with up to 32, for the partial result through L2 and a
    // pipeline that starts again: 16 x 131,072, 108 tiles a CTA, in E4M3 293 us with runs of 128,
    // 305 of 64, 318 of 36, in bf16 355 and 370.
    static constexpr int kRun = 128;
};

constexpr uint32_t kChunk = 128 * 128;  // 128 positions x 128 bytes, 128-byte swizzle
constexpr uint32_t kTmemCols = 512;     // one CTA an SM (shared memory), so it takes them all

template <bool kBf16, int NH>
struct Shared {
    using S = Shape<kBf16, NH>;
    uint8_t kv[S::kPairs][S::kChunks][kChunk];        // A operand of both products
    uint8_t q[S::kQChunks][S::kQRows * 128];          // B operand of S: heads x 128 bytes of channels a chunk, K-major
    uint8_t p[S::kParts][kTile * S::kPRow];           // B operand of PV: positions x heads, MN-major
    float col_scale[2][kMaxHeads];     // E4M3: per-head logit factor, by piece parity
    float red_max[4][kMaxHeads];
    float m_sub[4][kMaxHeads];         // per lane quarter: what its logits are reduced by
    alignas(8) int moved[2];           // per head group: the last tile whose maximum had to move
    float red_sum[4][kMaxHeads];
    float2 before[4][NH];              // maximum and sum of the piece up to this run, per lane quarter
    // by tile mod 4: the row holds a position that is seen. (The ring holds less than three
    // tiles, and a place comes free after PV, so tile gt + 4 begins after the softmax of gt.)
    uint8_t row_ok[4][kTile];
    // q_full: two barriers, so that a producer can publish the next piece's query before a
    // softmax warp has waited on this one (a one-tile piece needs no softmax before its S ends)
    uint64_t q_full[2], q_empty, p_full, o_full, drain;
    // bf16 the first; E4M3 by tile parity, as S of tile gt + 1 may end before a warp has waited
    // on that of gt
    uint64_t s_full[2];
    uint64_t pv_done;                  // E4M3: P may be written again, and O rescaled
    uint64_t full[S::kPairs], empty[S::kPairs];
    uint64_t p_again, max_bar[S::kGroups], sum_bar[S::kGroups];
    Range range;
    uint32_t tmem_base;
    int abort;
};

// ---------------------------------------------------------------- a CTA's pieces
// Tiles j0 .. j1 - 1 of sequence b: at most `most` of the CTA's piece of it.
struct Piece {
    // the CTA's range begins with the piece; the piece is the whole sequence; this begins, ends it
    enum { kOpens = 1, kWhole = 2, kBegins = 4, kEnds = 8 };
    View v;
    int b, j0, j1;
    uint32_t is;  // which of these
};
struct Pieces {
    int64_t left;  // items
    int b, from, j, most;
    bool opens;
    __device__ __forceinline__ Pieces(const Range& r, int most)
        : left(r.items), b(r.b), from(r.j), j(r.j), most(most), opens(true) {}
    __device__ __forceinline__ bool next(const Args& a, Piece& p) {
        while (left > 0) {
            p.v = view_of(a, b, false);
            if (j < p.v.tiles) {
                const int to = (int)min((int64_t)p.v.tiles, j + left);
                p.b = b;
                p.j0 = j;
                p.j1 = to - j > most ? j + most : to;
                p.is = (opens ? Piece::kOpens : 0u) | (from == 0 && to == p.v.tiles ? Piece::kWhole : 0u) |
                       (j == from ? Piece::kBegins : 0u) | (p.j1 == to ? Piece::kEnds : 0u);
                left -= p.j1 - j;
                j = p.j1;
                return true;
            }
            ++b;
            from = j = 0;
            opens = false;
        }
        return false;
    }
};

// The same range tile by tile.
struct Tiles {
    Pieces it;
    Piece pc;
    int j;
    __device__ __forceinline__ explicit Tiles(const Range& r) : it(r, INT_MAX), j(0) { pc.j1 = 0; }
    __device__ __forceinline__ bool next(const Args& a) {
        if (++j < pc.j1) return true;
        if (!it.next(a, pc)) return false;
        j = pc.j0;
        return true;
    }
};

// The page that holds position t (which is seen) of table row `table`; -1 and a status bit
// where there is none.
__device__ __forceinline__ int page_of(const Args& a, const int32_t* table, uint32_t t) {
    const int page = table[t / (uint32_t)a.g.page_size];
    if (page >= 0 && page < a.g.n_pages) return page;
    raise_status(a.dev_status, CSA2_DEV_BAD_INDEX);
    return -1;
}

// Every wait is decided by its whole warp: what follows one holds shuffles and TMEM accesses of all
// 32 lanes, for which the others would wait forever if one had given up and left alone.

// ---------------------------------------------------------------- producers
// One warp copies the tile's rows box by box (rows of one page): bf16 straight into the
// swizzled operand. Boxes that hold nothing seen are left out.
struct Boxes {
    uint32_t rows[4];  // the tile's rows that hold a seen position
    bool mine;         // this lane's box is copied: it begins at the pool's row y
    int y;
};
__device__ __forceinline__ Boxes boxes_of(const Args& a, const Tiles& t, int lane) {
    Boxes x;
    const View& v = t.pc.v;
    const uint32_t ps = a.g.page_size, t0 = v.start(t.j), br = a.box_rows;
    // lane i has box i: box_rows divides 128 and the page size, so a box lies in one page
    const uint32_t p = t0 + lane * br;
    const bool any = lane * br < kTile && (p < v.nf || (p < v.T && p + br > v.lo));
    x.mine = false;
    x.y = 0;
    if (any) {
        const int page = page_of(a, a.g.table + (int64_t)v.row * a.g.max_pages, p);
        x.mine = page >= 0;
        x.y = page * (int)ps + (int)(p % ps);
    }
    const uint32_t held = __ballot_sync(0xffffffffu, x.mine);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const uint32_t row = 32 * w + lane;
        x.rows[w] = __ballot_sync(0xffffffffu, v.sees(t0 + row) && ((held >> (row >> a.box_shift)) & 1u));
    }
    return x;
}

template <bool kBf16, int NH>
__device__ void tma_role(Shared<kBf16, NH>& sh, const Args& a, const CUtensorMap* tmap, int lane, volatile int* abort) {
    constexpr int kPairs = Shape<kBf16, NH>::kPairs;
    constexpr int kChunks = Shape<kBf16, NH>::kChunks;  // boxes of 128 bytes a row: 64 channels in bf16
    const uint32_t dst0 = smem_u32(sh.kv[0][0]) + lane * a.box_rows * 128;
    const int box_bytes = a.box_rows * a.g.row_bytes;
    const uint64_t once = l2_policy_evict_first();
    Tiles it(sh.range);
    int g = 0;  // pairs so far
    bool has = it.next(a), gave_up = false;
    Boxes cur, nxt;
    if (has) cur = boxes_of(a, it, lane);
    bool has_nx = false;
    // With few tiles the requests ahead only hold up the other CTAs' first ones: pieces of 11 or
    // 12 tiles (48 windows of 4,096, 16 heads) 45 us without, 49 with them; of 4 (8 sequences of
    // 8,192) 30 and 32; of 14 (32 of 8,192, 64 heads) 75 and 71. E4M3: of 4 tiles 31 and 33, of 9
    // (32 ragged sequences) 46 and 47, of 108 with 32 heads 252 and 213.
    const bool ahead = sh.range.items > 12;
    auto look_ahead = [&](bool request) -> Boxes {
        const Boxes x = boxes_of(a, it, lane);
        if (request && x.mine) bulk_prefetch_l2(a.base + (int64_t)x.y * a.g.row_bytes, box_bytes);
        return x;
    };
    for (int gt = 0; has && !gave_up; ++gt) {
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, cur.mine)) * a.box_rows * 128 * kChunks;
        for (int pr = 0; pr < 4; ++pr, ++g) {
            const int slot = g % kPairs;
            gave_up = g >= kPairs && !mbar_wait_warp(&sh.empty[slot], (uint32_t)((g / kPairs - 1) & 1), abort);
            if (gave_up) break;
            if (pr == 0) {  // four rows a lane: their bits to bytes
                const uint32_t w = lane < 16 ? (lane < 8 ? cur.rows[0] : cur.rows[1]) : lane < 24 ? cur.rows[2] : cur.rows[3];
                *reinterpret_cast<uint32_t*>(&sh.row_ok[gt & 3][4 * lane]) =
                    (((w >> (4 * (lane & 7))) & 15u) * 0x00204081u) & 0x01010101u;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], bytes);
            __syncwarp();
            if (cur.mine) {
                const uint32_t dst = dst0 + kChunks * slot * kChunk;
                tma_g2s_2d_hint(dst, tmap, 128 * pr, cur.y, &sh.full[slot], once);
                if constexpr (kBf16) tma_g2s_2d_hint(dst + kChunk, tmap, 128 * pr + 64, cur.y, &sh.full[slot], once);
            }
        }
        // The ring holds little more than a tile and stands still between a tile's S and its
        // PV. The tile after the next comes into L2 meanwhile (both at the first), so that HBM
        // does not stand still too and the refill is short. What has been copied goes first
        // when L2 makes room, and copies ask for their own lines only, so that it is never what
        // waits there. (16 sequences of 131,072, 64 heads, with 16 softmax warps: 361 us, three
        // tiles ahead 379, none 418; without the hint 393; with it, but copies widened to 256
        // bytes, 414.)
        if (gt == 0) {
            has_nx = it.next(a);
            if (has_nx) nxt = look_ahead(true);
        }
        cur = nxt;
        has = has_nx;
        has_nx = has && it.next(a);
        if (has_nx) nxt = look_ahead(ahead);
    }
    // whatever ended the loop, no copy of this CTA outlives it
    for (int s = max(0, g - kPairs); s < g; ++s) mbar_wait_drain(&sh.full[s % kPairs], (uint32_t)((s / kPairs) & 1));
}

template <int NH>
__device__ void query_role(Shared<true, NH>& sh, const Args& a, int pt, int lane, volatile int* abort) {
    constexpr int kStagers = 32 * Shape<true, NH>::kHelpWarps;
    static_assert(kStagers == 128, "a thread stages unit pt mod 64 of every other head");
    const int u = pt & 63, hb = pt >> 6;
    Pieces pi(sh.range, Shape<true, NH>::kRun);
    Piece pc;
    for (int it = 0; pi.next(a, pc); ++it) {
        if (it > 0 && !mbar_wait_warp(&sh.q_empty, (uint32_t)((it - 1) & 1), abort)) return;
        const __nv_bfloat16* src = a.q + pc.b * a.q_seq + hb * a.q_head + 8 * u;
        const uint32_t dst = smem_u32(sh.q[u >> 3]);
#pragma unroll 4
        for (int h = hb; h < NH; h += 2, src += 2 * a.q_head)
            cp_async_16(dst + sw128(h, u & 7), h < a.heads ? src : a.q, h < a.heads);
        cp_async_wait_all();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full[it & 1]);
    }
}

// E4M3: a warp takes a head, a lane 16 of its channels. The head's values times 2^s, with the
// largest |q| in [2^7, 2^8): hi holds 4 bits, what is left is at most 2^-5 of 2^8 and lo = 2^5
// times it holds the other 4, exactly down to 2^-14 of the largest, to 2^-22 of it below. The
// factor goes into the logit scale. E4M3 has no infinity: one in the query becomes NaN.
template <int NH>
__device__ void query_role(Shared<false, NH>& sh, const Args& a, int pt, int lane, volatile int* abort) {
    constexpr int kWarps = Shape<false, NH>::kHelpWarps, kAtOnce = 4;  // heads whose loads are in flight together
    const int pw = pt >> 5;
    Pieces pi(sh.range, Shape<false, NH>::kRun);
    Piece pc;
    for (int it = 0; pi.next(a, pc); ++it) {
        if (it > 0 && !mbar_wait_warp(&sh.q_empty, (uint32_t)((it - 1) & 1), abort)) return;
#pragma unroll 1
        for (int h1 = pw; h1 < NH; h1 += kWarps * kAtOnce) {
            uint4 w2[kAtOnce][2];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int h = h1 + kWarps * i;
                const uint4* src = reinterpret_cast<const uint4*>(a.q + pc.b * a.q_seq + h * a.q_head) + 2 * lane;
                w2[i][0] = w2[i][1] = make_uint4(0u, 0u, 0u, 0u);
                if (h < a.heads) w2[i][0] = __ldg(src), w2[i][1] = __ldg(src + 1);
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int h = h1 + kWarps * i;
                if (h >= NH) break;
                const uint32_t w[8] = {w2[i][0].x, w2[i][0].y, w2[i][0].z, w2[i][0].w,
                                       w2[i][1].x, w2[i][1].y, w2[i][1].z, w2[i][1].w};
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
                mx = warp_max(mx);
                int s = 7 - ((int)((__float_as_uint(mx) >> 23) & 0xffu) - 127);
                s = max(-126, min(126, s));
                const float two_s = __uint_as_float((uint32_t)(s + 127) << 23);
                uint32_t hi[4] = {}, lo[4] = {};
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float x = __uint_as_float(w[k] << 16) * two_s, y = __uint_as_float(w[k] & 0xffff0000u) * two_s;
                    x = fmaf(x, 0.f, x);  // infinity to NaN
                    y = fmaf(y, 0.f, y);
                    const uint32_t xy = e4m3x2(x, y);
                    const float2 got = e4m3x2_to_float2(xy);
                    hi[k >> 1] |= xy << (16 * (k & 1));
                    lo[k >> 1] |= e4m3x2(32.f * (x - got.x), 32.f * (y - got.y)) << (16 * (k & 1));
                }
                uint8_t* q = sh.q[lane >> 3];
                *reinterpret_cast<uint4*>(q + sw128(h, lane & 7)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(q + sw128(NH + h, lane & 7)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                if (lane == 0) sh.col_scale[it & 1][h] = a.scale_log2 * __uint_as_float((uint32_t)(127 - s) << 23);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full[it & 1]);
    }
}

// Whether a head group's maximum moved at tile gt (read after p_full of that tile).
template <bool kBf16, int NH>
__device__ __forceinline__ bool any_moved(Shared<kBf16, NH>& sh, int gt) {
    static_assert(Shape<kBf16, NH>::kGroups == 2, "a mark each");
    const long long m = *reinterpret_cast<const volatile long long*>(sh.moved);
    return (int)m == gt || (int)(m >> 32) == gt;
}

// ---------------------------------------------------------------- MMA issuer
// The whole warp walks the tiles and one elected lane issues; what the descriptors are made
// from is broadcast from a lane first. Both let them live in the warp's uniform registers,
// where the MMA takes them from: issued by a thread that had left its warp, an MMA followed
// the one before by 75 to 80 cycles, so by 61 to 64. (Alone, M = 128 MMAs from shared memory
// follow by 40 cycles at N = 16 and 49 at N = 64; here the copies of the next rows share
// shared memory with them.)
template <int NH>
__device__ void mma_role(Shared<true, NH>& sh, const Args& a, uint32_t tmem, int, volatile int* abort) {
    using S = Shape<true, NH>;
    const uint64_t dK = smem_desc(smem_u32(sh.kv[0][0]), 16, 1024, kLayoutSw128);
    const uint64_t dQ = smem_desc(smem_u32(sh.q[0]), 16, 1024, kLayoutSw128);
    const uint64_t dV = smem_desc(smem_u32(sh.kv[0][0]), kChunk, 1024, kLayoutSw128);
    const uint64_t dP = smem_desc(smem_u32(sh.p[0]), 1024, 8 * S::kPRow, S::kPLayout);
    Pieces pi(sh.range, S::kRun);
    Piece pc;
    int gt = 0, again = 0;  // tiles so far, those whose P came twice
    int slot0 = 0;          // slot of the tile's first pair, and its phase
    uint32_t phase0 = 0;
    for (int it = 0; pi.next(a, pc); ++it) {
        if (!mbar_wait_warp(&sh.q_full[it & 1], (uint32_t)((it >> 1) & 1), abort)) return;
        tc_fence_after();
        for (int j = pc.j0; j < pc.j1; ++j, ++gt) {
            // S^T = K . Q^T over the 512 channels, pair by pair as they land
            int slot = slot0;
            uint32_t phase = phase0;
#pragma unroll
            for (int pr = 0; pr < 4; ++pr) {
                if (!mbar_wait_warp(&sh.full[slot], phase, abort)) return;
                tc_fence_after();
                const uint64_t dKs = dK + ((2 * (uint32_t)__shfl_sync(0xffffffffu, slot, 0) * kChunk) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f16(tmem + S::kColS, dKs + ((c * kChunk + 32 * k) >> 4),
                                    dQ + (((2 * pr + c) * NH * 128 + 32 * k) >> 4), S::kIdescS, (pr | c | k) != 0);
                }
                __syncwarp();
                if (++slot == S::kPairs) slot = 0, phase ^= 1u;
            }
            if (elect_one()) {
                tc_commit(&sh.s_full[0]);
                if (j == pc.j1 - 1) tc_commit(&sh.q_empty);
            }
            __syncwarp();
            // O^T += V^T . P^T, 128 channels (one pair) at a time
            if (!mbar_wait_warp(&sh.p_full, (uint32_t)(gt & 1), abort)) return;
            if (any_moved(sh, gt) && !mbar_wait_warp(&sh.p_again, (uint32_t)(again++ & 1), abort)) return;
            tc_fence_after();
            slot = slot0;
            const uint32_t more = __shfl_sync(0xffffffffu, j != pc.j0 ? 1u : 0u, 0);
#pragma unroll
            for (int mb = 0; mb < 4; ++mb) {
                const uint64_t dVs = dV + ((2 * (uint32_t)__shfl_sync(0xffffffffu, slot, 0) * kChunk) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_f16(tmem + NH * mb, dVs + ((k * 2048) >> 4),
                                dP + ((k * 16 * S::kPRow) >> 4), S::kIdescPV, k == 0 ? more : 1u);
                    tc_commit(&sh.empty[slot]);
                }
                __syncwarp();
                if (++slot == S::kPairs) slot = 0;
            }
            slot0 = slot;
            phase0 = phase;
        }
        if (elect_one()) tc_commit(&sh.o_full);
        __syncwarp();
    }
}

// E4M3: S of the next tile may come before PV of this one (within a piece: the next one's query
// comes after this one's last S), so that the tensor cores have it to do while the softmax runs.
// S of gt + 1 takes the columns of gt - 1, whose softmax has ended: PV of gt - 1 came after its P.
// Where the ring holds two tiles only, the next one's last rows land when PV of the tile before
// has long ended, and this one's P is often ready first: whichever is, goes first (64 heads, 16 x
// 131,072: 291 us, S always first 314). With half a tile more S always first is better (214, 221).
// The MMAs are short (28 to 65 cycles), so what stands between them counts: a product's are issued
// in one go, after one look at all the barriers it needs (32 heads: 214 us, place by place 245).
// The three MMAs of P's parts share V in the tensor core's collector (114 cycles, 149 without).
template <int NH>
__device__ void mma_role(Shared<false, NH>& sh, const Args& a, uint32_t tmem, int lane, volatile int* abort) {
    using S = Shape<false, NH>;
    const uint64_t dK = smem_desc(smem_u32(sh.kv[0][0]), 16, 1024, kLayoutSw128);
    const uint64_t dQ = smem_desc(smem_u32(sh.q[0]), 16, 1024, kLayoutSw128);
    const uint64_t dV = smem_desc(smem_u32(sh.kv[0][0]), kChunk, 1024, kLayoutSw128);
    const uint64_t dP = smem_desc(smem_u32(sh.p[0]), 1024, 8 * S::kPRow, S::kPLayout);
    Pieces pi(sh.range, S::kRun);
    Piece pc;
    int gt = 0, again = 0;  // tiles whose PV has been issued, those whose P came twice
    int slot = 0, pv_slot = 0;  // first place of the next S and PV
    uint32_t phase = 0;
    // a descriptor's step to place i of a tile that begins at place `from`
    auto place = [&](int from, int i) {
        const int x = from + i < S::kPairs ? from + i : from + i - S::kPairs;
        return (uint64_t)__shfl_sync(0xffffffffu, (uint32_t)x * (kChunk >> 4), 0);
    };
    // the barrier, and its phase, of the next S's place that this lane looks at
    auto landing = [&] { return &sh.full[slot + (lane & 3) < S::kPairs ? slot + (lane & 3) : slot + (lane & 3) - S::kPairs]; };
    auto landing_phase = [&] { return phase ^ (uint32_t)(slot + (lane & 3) >= S::kPairs); };
    auto scores = [&](int tile, bool last) {
        const uint32_t at = tmem + S::kColS + (uint32_t)__shfl_sync(0xffffffffu, tile & 1, 0) * S::kQRows;
        const uint64_t k[4] = {dK + place(slot, 0), dK + place(slot, 1), dK + place(slot, 2), dK + place(slot, 3)};
        if (!mbar_wait_warp(landing(), landing_phase(), abort)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
            for (int pr = 0; pr < 4; ++pr)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mma_f8(at, k[pr] + ((32 * i) >> 4), dQ + ((pr * S::kQRows * 128 + 32 * i) >> 4), S::kIdescS, (pr | i) != 0);
            tc_commit(&sh.s_full[tile & 1]);
            if (last) tc_commit(&sh.q_empty);
        }
        __syncwarp();
        if ((slot += 4) >= S::kPairs) slot -= S::kPairs, phase ^= 1u;
        return true;
    };
    for (int it = 0; pi.next(a, pc); ++it) {
        if (!mbar_wait_warp(&sh.q_full[it & 1], (uint32_t)((it >> 1) & 1), abort)) return;
        tc_fence_after();
        bool ahead = false;  // S of this tile has been issued
        for (int j = pc.j0; j < pc.j1; ++j, ++gt) {
            if (!ahead && !scores(gt, j + 1 == pc.j1)) return;
            ahead = false;
            const uint64_t v[4] = {dV + place(pv_slot, 0), dV + place(pv_slot, 1), dV + place(pv_slot, 2), dV + place(pv_slot, 3)};
            const uint32_t more = __shfl_sync(0xffffffffu, j != pc.j0 ? 1u : 0u, 0);
            if (j + 1 < pc.j1 && S::kPairs > 8) {
                ahead = true;
                if (!scores(gt + 1, j + 2 == pc.j1)) return;
            } else if (j + 1 < pc.j1) {
                const int first = mbar_wait_either_warp(lane < 4 ? landing() : &sh.p_full,
                                                        lane < 4 ? landing_phase() : (uint32_t)(gt & 1), lane, 4, abort);
                if (!first) return;
                ahead = first == 1;
                if (ahead && !scores(gt + 1, j + 2 == pc.j1)) return;
            }
            if ((ahead || j + 1 == pc.j1) && !mbar_wait_warp(&sh.p_full, (uint32_t)(gt & 1), abort)) return;
            if (any_moved(sh, gt) && !mbar_wait_warp(&sh.p_again, (uint32_t)(again++ & 1), abort)) return;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int mb = 0; mb < 4; ++mb) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // 32 positions and the three parts of their P
                        const uint64_t vi = v[mb] + ((i * 32 * 128) >> 4), wi = dP + ((i * 32 * S::kPRow) >> 4);
                        constexpr uint32_t kPart = (kTile * S::kPRow) >> 4;
                        mma_f8<Collector::kFill>(tmem + NH * mb, vi, wi, S::kIdescPV, i == 0 ? more : 1u);
                        mma_f8<Collector::kUse>(tmem + NH * mb, vi, wi + kPart, S::kIdescPV, 1u);
                        mma_f8<Collector::kLast>(tmem + NH * mb, vi, wi + 2 * kPart, S::kIdescPV, 1u);
                    }
                    tc_commit(&sh.empty[pv_slot + mb < S::kPairs ? pv_slot + mb : pv_slot + mb - S::kPairs]);
                }
                tc_commit(&sh.pv_done);
                if (j + 1 == pc.j1) tc_commit(&sh.o_full);
            }
            __syncwarp();
            if ((pv_slot += 4) >= S::kPairs) pv_slot -= S::kPairs;
        }
    }
}

// ---------------------------------------------------------------- softmax and epilogue
template <int NC>
__device__ __forceinline__ void tmem_ld(uint32_t at, uint32_t* r) {
    if constexpr (NC == 32) tmem_ld_32x32b_x32(at, r);
    else if constexpr (NC == 16) tmem_ld_32x32b_x16(at, r);
    else tmem_ld_32x32b_x8(at, r);
}
template <int NC>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t* r) {
    if constexpr (NC == 32) tmem_st_32x32b_x32(at, r);
    else if constexpr (NC == 16) tmem_st_32x32b_x16(at, r);
    else tmem_st_32x32b_x8(at, r);
}

// Sums NC per-head values over the warp's 32 lanes; lane i returns head i mod NC.
template <int NC>
__device__ __forceinline__ float warp_sum(float* v, int lane) {
#pragma unroll
    for (int o = NC / 2; o >= 1; o >>= 1) {
        const bool up = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float s = v[0];
#pragma unroll
    for (int o = NC; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Warp (qd, cg): positions 32 qd + lane of the tile, heads cg NC .. + NC - 1. Logits are in
// the log2 domain.
//
// The running maximum is lazy: it moves only when a tile would push P above 2^kLazyMax. A
// tile therefore needs no maximum of its own as long as its logits stay below that: the warp
// takes P from the maximum it has, and the four warps of a head group only agree that none of
// them saw a larger logit (2,080 -> 850 cycles from S to P against finding each tile's
// maximum). The agreement rides on the barrier that hands P to the MMAs: an issuer that finds
// a group's mark set waits for that group's second P. Where one is set, or at a piece's first
// tile, the maxima are found and exchanged, and the heads' columns of O rescaled in TMEM.
template <bool kBf16, int NH>
__device__ void softmax_role(Shared<kBf16, NH>& sh, const Args& a, uint32_t tmem, int warp, int lane,
                             volatile int* abort) {
    using S = Shape<kBf16, NH>;
    constexpr int NC = S::NC;
    constexpr float kNone = -3.0e38f;  // m_sub before any logit: whatever is finite exceeds it
    const int qd = warp & 3, cg = warp >> 2, h0 = cg * NC, mine = lane & (NC - 1);
    const int r = 32 * qd + lane;
    const uint32_t tl = tmem + ((uint32_t)(32 * qd) << 16);
    const float sink2 = a.sink && h0 + mine < a.heads ? a.sink[h0 + mine] * kLog2e : -INFINITY;
    float* const m_sub = &sh.m_sub[qd][h0];
    // x[i] = logit i of this row (`less`: what m_sub holds), -infinity where nothing is seen
    auto logits = [&](float* x, bool less, int it, int gt, bool ok) {
        uint32_t sv[NC];
        if constexpr (kBf16) {
            tmem_ld<NC>(tl + S::kColS + h0, sv);
        } else {
            const uint32_t at = tl + S::kColS + (gt & 1) * S::kQRows + h0;
            uint32_t lo[NC];
            tmem_ld<NC>(at, sv);
            tmem_ld<NC>(at + NH, lo);
#pragma unroll
            for (int i = 0; i < NC; ++i)
                sv[i] = __float_as_uint(fmaf(__uint_as_float(lo[i]), 0.03125f, __uint_as_float(sv[i])));
        }
#pragma unroll
        for (int i = 0; i < NC; i += 4) {
            float4 c = make_float4(a.scale_log2, a.scale_log2, a.scale_log2, a.scale_log2);
            if constexpr (!kBf16) c = *reinterpret_cast<const float4*>(&sh.col_scale[it & 1][h0 + i]);
            const float4 m = less ? *reinterpret_cast<const float4*>(m_sub + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[i] = ok ? fmaf(__uint_as_float(sv[i]), c.x, -m.x) : -INFINITY;
            x[i + 1] = ok ? fmaf(__uint_as_float(sv[i + 1]), c.y, -m.y) : -INFINITY;
            x[i + 2] = ok ? fmaf(__uint_as_float(sv[i + 2]), c.z, -m.z) : -INFINITY;
            x[i + 3] = ok ? fmaf(__uint_as_float(sv[i + 3]), c.w, -m.w) : -INFINITY;
        }
    };
    // P = 2^x, rounded to bf16 or f16, into the operand. The sums take the values that the product
    // multiplies (E4M3: what the three parts add up to, so without what is left of a weight below
    // the last part's steps), so a row's weights add up to one whatever the rounding does: bf16
    // leaves them in x, E4M3, whose parts need the registers, in pairs in w.
    auto weights = [&](float* x, uint32_t* w, int gt) {
        if constexpr (kBf16) {
#pragma unroll
            for (int u = 0; u < NC / 8; ++u) {
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float& p = x[8 * u + 2 * k];
                    float& q = x[8 * u + 2 * k + 1];
                    const __nv_bfloat162 v = __floats2bfloat162_rn(ex2(p), ex2(q));
                    o[k] = *reinterpret_cast<const uint32_t*>(&v);
                    p = __uint_as_float(o[k] << 16);
                    q = __uint_as_float(o[k] & 0xffff0000u);
                }
                *reinterpret_cast<uint4*>(sh.p[0] + S::p_unit(r, h0 / 8 + u)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) {
                const __half2 v = __floats2half2_rn(ex2(x[2 * i]), ex2(x[2 * i + 1]));
                w[i] = *reinterpret_cast<const uint32_t*>(&v);
            }
            // A NaN loses itself in the first two parts' rounding and stays what is left of them, so
            // the last part holds it. What that one leaves out is at most half its step, and what
            // it leaves of w a multiple of 2^-16 that f16 holds: both differences are exact.
            uint32_t o[3][NC / 4];
#pragma unroll
            for (int k = 0; k < NC / 4; ++k) {
                uint32_t x0 = w[2 * k], x1 = w[2 * k + 1];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t p0 = (x0 + 0x00800080u) & 0xff00ff00u, p1 = (x1 + 0x00800080u) & 0xff00ff00u;
                    o[i][k] = __byte_perm(p0, p1, 0x7531);
                    x0 = h2_sub(x0, p0);
                    x1 = h2_sub(x1, p1);
                }
                o[2][k] = h2x2_to_e5m2x4(x0, x1);
                w[2 * k] = h2_sub(w[2 * k], h2_sub(x0, __byte_perm(o[2][k], 0u, 0x1404)));
                w[2 * k + 1] = h2_sub(w[2 * k + 1], h2_sub(x1, __byte_perm(o[2][k], 0u, 0x3424)));
            }
            if (gt > 0 && !mbar_wait_warp(&sh.pv_done, (uint32_t)((gt - 1) & 1), abort)) return false;
#pragma unroll
            for (int i = 0; i < 3; ++i)
#pragma unroll
                for (int u = 0; u < NC / 16; ++u)
                    *reinterpret_cast<uint4*>(sh.p[i] + S::p_unit(r, h0 / 16 + u)) =
                        make_uint4(o[i][4 * u], o[i][4 * u + 1], o[i][4 * u + 2], o[i][4 * u + 3]);
        }
        return true;
    };
    auto value = [](const float* x, const uint32_t* w, int i) {
        if constexpr (kBf16) return x[i];
        const __half2 v = *reinterpret_cast<const __half2*>(&w[i >> 1]);
        return i & 1 ? __high2float(v) : __low2float(v);
    };
    Pieces pi(sh.range, S::kRun);
    Piece pc;
    int g = 0, gt = 0, moves = 0;
    for (int it = 0; pi.next(a, pc); ++it) {
        if (!mbar_wait_warp(&sh.q_full[it & 1], (uint32_t)((it >> 1) & 1), abort)) return;
        float m_run = -INFINITY;  // running maximum of head h0 + mine
        float lpart[NC];          // this row's share of the sum of P
#pragma unroll
        for (int i = 0; i < NC; ++i) lpart[i] = 0.f;
        for (int j = pc.j0; j < pc.j1; ++j, ++gt, g += 4) {
            if (!mbar_wait_warp(&sh.s_full[kBf16 ? 0 : gt & 1], (uint32_t)((kBf16 ? gt : gt >> 1) & 1), abort)) return;
            // (complete already: orders the read of row_ok after the producer's write)
            if (!mbar_wait_warp(&sh.full[g % S::kPairs], (uint32_t)((g / S::kPairs) & 1), abort)) return;
            tc_fence_after();
            const bool ok = sh.row_ok[gt & 3][r] != 0;
            // Rows that are not seen came with the box or are left from another tile: whatever
            // they hold (NaN among it) must not meet P = 0 in the product. S has read them, PV
            // has not.
            if (!ok) {
                constexpr int kAll = 4 * S::kChunks, kMine = kAll / S::kGroups;
#pragma unroll 1
                for (int c = cg * kMine; c < (cg + 1) * kMine; ++c) {
                    uint4* z = reinterpret_cast<uint4*>(sh.kv[(g + c / S::kChunks) % S::kPairs][c % S::kChunks] + r * 128);
#pragma unroll
                    for (int u = 0; u < 8; ++u) z[(u + lane) & 7] = make_uint4(0u, 0u, 0u, 0u);  // all banks
                }
            }
            const bool opens = j == pc.j0;
            bool move = opens, any = false;
            if (!opens) {
                float x[NC];
                logits(x, true, it, gt, ok);
                bool over = false;
#pragma unroll
                for (int i = 0; i < NC; ++i) over |= x[i] > S::kLazyMax + S::kLift;
                over = __any_sync(0xffffffffu, over) && lane == 0;
                if (kBf16 && over) *(volatile int*)&sh.moved[cg] = gt;
                uint32_t w[NC / 2];
                if (!weights(x, w, gt)) return;
                // (E4M3: after PV of the tile before, whose marks everyone has read by then)
                if (!kBf16 && over) *(volatile int*)&sh.moved[cg] = gt;
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.p_full);
                // the MMA issuer goes on with this P unless a group found a larger logit
                if (!mbar_wait_warp(&sh.p_full, (uint32_t)(gt & 1), abort)) return;
                any = any_moved(sh, gt);
                move = *(volatile int*)&sh.moved[cg] == gt;
                if (!move) {
#pragma unroll
                    for (int i = 0; i < NC; ++i) lpart[i] += value(x, w, i);
                }
            }
            if (move) {
                tc_fence_after();
                float x[NC];
                logits(x, false, it, gt, ok);
#pragma unroll
                for (int i = 0; i < NC; i += 4) {
                    const float4 m4 = make_float4(warp_max(x[i]), warp_max(x[i + 1]), warp_max(x[i + 2]), warp_max(x[i + 3]));
                    if (lane == 0) *reinterpret_cast<float4*>(&sh.red_max[qd][h0 + i]) = m4;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.max_bar[cg]);
                if (!mbar_wait_warp(&sh.max_bar[cg], (uint32_t)(moves++ & 1), abort)) return;
                const float tm = fmaxf(fmaxf(sh.red_max[0][h0 + mine], sh.red_max[1][h0 + mine]),
                                       fmaxf(sh.red_max[2][h0 + mine], sh.red_max[3][h0 + mine]));
                const float m_new = tm > m_run + S::kLazyMax ? tm : m_run;
                const float alpha = (m_new != m_run && m_run != -INFINITY) ? ex2(m_run - m_new) : 1.f;
                const bool rescale = __any_sync(0xffffffffu, alpha != 1.f);
                m_run = m_new;
                __syncwarp();
                if (lane < NC) m_sub[lane] = m_run == -INFINITY ? kNone : m_run - S::kLift;
                __syncwarp();
                // (bf16 reads them again: kept until here they spill, 357 us against 351 for 64 heads
                // and 16 x 131,072; with two reads a logit, E4M3 gains a microsecond by keeping them)
                if constexpr (kBf16) {
                    logits(x, true, it, gt, ok);
                } else {
#pragma unroll
                    for (int i = 0; i < NC; i += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(m_sub + i);
                        x[i] -= m.x;
                        x[i + 1] -= m.y;
                        x[i + 2] -= m.z;
                        x[i + 3] -= m.w;
                    }
                }
                uint32_t w[NC / 2];
                if (!weights(x, w, gt)) return;
#pragma unroll
                for (int i = 0; i < NC; ++i) lpart[i] = fmaf(lpart[i], __shfl_sync(0xffffffffu, alpha, i), value(x, w, i));
                if (rescale) {  // O holds the tiles before this one: their PV has ended
#pragma unroll 1
                    for (int mb = 0; mb < 4; ++mb) {
                        uint32_t ov[NC];
                        tmem_ld<NC>(tl + NH * mb + h0, ov);
#pragma unroll
                        for (int i = 0; i < NC; ++i)
                            ov[i] = __float_as_uint(__uint_as_float(ov[i]) * __shfl_sync(0xffffffffu, alpha, i));
                        tmem_st<NC>(tl + NH * mb + h0, ov);
                    }
                    tmem_wait_st();
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
            }
            if (opens) {
                if (lane == 0) mbar_arrive(&sh.p_full);
            } else if (any) {
                if (lane == 0) mbar_arrive(&sh.p_again);
            }
        }
        if (!mbar_wait_warp(&sh.o_full, (uint32_t)(it & 1), abort)) return;
        tc_fence_after();
        sh.red_sum[qd][h0 + mine] = warp_sum<NC>(lpart, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.sum_bar[cg]);
        if (!mbar_wait_warp(&sh.sum_bar[cg], (uint32_t)(it & 1), abort)) return;
        float l = (sh.red_sum[0][h0 + mine] + sh.red_sum[1][h0 + mine]) +
                  (sh.red_sum[2][h0 + mine] + sh.red_sum[3][h0 + mine]);
        m_run -= S::kLift;  // what P and O are relative to
        float* part = part_of(a, blockIdx.x, pc.is & Piece::kOpens ? 0 : 1);
        if (!(pc.is & Piece::kBegins)) {
            // What came before of the piece is added in TMEM: its O stands in part (written by
            // this thread), its maximum and sum in sh.before.
            const float2 ml = sh.before[qd][h0 + mine];
            const float M = fmaxf(ml.x, m_run);
            const float was = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            const float now = m_run == -INFINITY ? 0.f : ex2(m_run - M);
            l = fmaf(ml.y, was, l * now);
            m_run = M;
            constexpr int kAtOnce = NC < 16 ? NC : 16;  // heads whose loads are in flight together
#pragma unroll 1
            for (int n = 0; n < 4 * NC; n += kAtOnce) {
                const int mb = n / NC, i0 = n % NC;
                const float* src = part + (int64_t)(h0 + i0) * kD + 128 * mb + r;
                float x[kAtOnce];
                uint32_t ov[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) x[i] = h0 + i0 + i < a.heads ? src[i * kD] : 0.f;
                tmem_ld<kAtOnce>(tl + NH * mb + h0 + i0, ov);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    ov[i] = __float_as_uint(fmaf(x[i], __shfl_sync(0xffffffffu, was, i0 + i),
                                                 __uint_as_float(ov[i]) * __shfl_sync(0xffffffffu, now, i0 + i)));
                tmem_st<kAtOnce>(tl + NH * mb + h0 + i0, ov);
            }
            tmem_wait_st();
        }
        __syncwarp();
        if (!(pc.is & Piece::kEnds) && lane < NC) sh.before[qd][h0 + lane] = make_float2(m_run, l);
        __syncwarp();
        // lane = channel 128 mb + 32 qd + lane of NC heads: for each head the warp stores 32
        // neighbouring values
        if ((pc.is & (Piece::kWhole | Piece::kEnds)) == (Piece::kWhole | Piece::kEnds)) {
            const float M = fmaxf(m_run, sink2);
            const float f = m_run == -INFINITY ? 0.f : ex2(m_run - M);
            const float den = l * f + (sink2 == -INFINITY ? 0.f : ex2(sink2 - M));
            const float w = den == 0.f ? 0.f : f / den;
            __nv_bfloat16* out = a.out + ((int64_t)pc.b * a.heads + h0) * kD + r;
#pragma unroll 1
            for (int mb = 0; mb < 4; ++mb) {
                uint32_t ov[NC];
                tmem_ld<NC>(tl + NH * mb + h0, ov);
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const float wi = __shfl_sync(0xffffffffu, w, i);
                    if (h0 + i < a.heads)
                        out[(int64_t)i * kD + 128 * mb] = __float2bfloat16_rn(wi == 0.f ? 0.f : __uint_as_float(ov[i]) * wi);
                }
            }
        } else {
            if (qd == 0 && lane < NC && h0 + lane < a.heads) {
                part[(int64_t)a.heads * kD + h0 + lane] = m_run;
                part[(int64_t)a.heads * (kD + 1) + h0 + lane] = l;
            }
#pragma unroll 1
            for (int mb = 0; mb < 4; ++mb) {
                uint32_t ov[NC];
                tmem_ld<NC>(tl + NH * mb + h0, ov);
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (h0 + i < a.heads) part[(int64_t)(h0 + i) * kD + 128 * mb + r] = __uint_as_float(ov[i]);
            }
        }
        tc_fence_before();
    }
}

template <bool kBf16, int NH>
__global__ void __launch_bounds__(Shape<kBf16, NH>::kThreads, 1)
k_paged_attn(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tmap) {
    using S = Shape<kBf16, NH>;
    extern __shared__ uint8_t raw[];
    auto& sh = *reinterpret_cast<Shared<kBf16, NH>*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &sh.abort;
    if (tid == 0) {
        mbar_init(&sh.q_full[0], S::kHelpWarps);
        mbar_init(&sh.q_full[1], S::kHelpWarps);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.s_full[0], 1);
        mbar_init(&sh.s_full[1], 1);
        mbar_init(&sh.pv_done, 1);
        mbar_init(&sh.p_full, S::kSoftWarps);
        mbar_init(&sh.p_again, S::kSoftWarps);
        mbar_init(&sh.o_full, 1);
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < S::kPairs; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < S::kGroups; ++i) {
            mbar_init(&sh.max_bar[i], 4);
            mbar_init(&sh.sum_bar[i], 4);
        }
        sh.moved[0] = sh.moved[1] = -1;
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == S::kMmaWarp) {
        tmem_alloc(&sh.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    // a programmatic launch: only the setup above may overlap the kernel ahead; the join's
    // CTAs may be placed from now on, and wait for this grid's end
    grid_dep_launch_dependents();
    grid_dep_wait();
    tc_fence_before();
    plan(a, &sh.range);  // ends with a CTA barrier
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sh.tmem_base, 0);
    if (warp < S::kSoftWarps) {
        softmax_role<kBf16, NH>(sh, a, tmem, warp, lane, abort);
    } else if (warp == S::kMmaWarp) {
        mma_role<NH>(sh, a, tmem, lane, abort);
        // every MMA issued must finish before TMEM and shared memory are released
        __syncwarp();
        if (elect_one()) tc_commit(&sh.drain);
        if (!mbar_wait_drain(&sh.drain, 0)) *abort = 1;
    } else if (warp == S::kTmaWarp) {
        tma_role<kBf16, NH>(sh, a, &tmap, lane, abort);
    } else {
        query_role<NH>(sh, a, tid - 32 * S::kHelp0, lane, abort);
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && sh.abort) raise_status(a.dev_status, CSA2_DEV_TIMEOUT);
    if (warp == S::kMmaWarp) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <bool kBf16, int NH>
constexpr int smem_bytes() {
    return (int)sizeof(Shared<kBf16, NH>) + 1024;
}
// (227 KB, of which plan() has 1,664 bytes)
template <bool kBf16, int NH>
constexpr bool kFits = smem_bytes<kBf16, NH>() <= 227 * 1024 - 1664;
static_assert(kFits<true, 64> && kFits<true, 32> && kFits<true, 16> && kFits<false, 64> && kFits<false, 32>,
              "shared memory of a CTA");

// ---------------------------------------------------------------- join
// A thread has four channels of a (sequence, head) and, with G groups of threads, every G-th
// piece; the groups' sums are added in order. Sequences in one piece were finished by the
// attention kernel; those that see nothing get their zeros here. A chain of three round trips
// bounds it (the pieces, their values and maxima, the output): up to eight pieces' values are
// requested together, before the weights they will get are known.
//   narrow: one CTA of 128 threads per (sequence, head), one group;
//   wide: four CTAs, of 32 channels' threads x 16 groups each.
constexpr int kJoinBatch = 8;
constexpr int kMaxCtas = 256;  // of the attention kernel: a sequence has at most as many pieces
template <bool kWide>
struct Join {
    static constexpr int kLanes = kWide ? 32 : 128, kGroups = kWide ? 16 : 1, kThreads = kLanes * kGroups;
};
template <bool kWide>
__global__ void __launch_bounds__(Join<kWide>::kThreads, 1) k_paged_join(Args a) {
    constexpr int kLanes = Join<kWide>::kLanes, G = Join<kWide>::kGroups;
    __shared__ float4 sums[G][kWide ? kLanes : 1];
    __shared__ float dens[G], m_s[kMaxCtas], l_s[kMaxCtas];
    grid_dep_wait();
    const int lane = threadIdx.x & 31, grp = kWide ? threadIdx.x / kLanes : 0;
    const int ch = kWide ? blockIdx.z * kLanes + lane : threadIdx.x;
    const int b = blockIdx.x, h = blockIdx.y;
    const int2 span = a.pieces[b];
    const float s2 = a.sink ? a.sink[h] * kLog2e : -INFINITY;
    __nv_bfloat16* out = a.out + ((int64_t)b * a.heads + h) * kD + 4 * ch;
    const int c0 = span.x & 0x7fffffff, c1 = span.y, slot0 = span.x < 0 ? 1 : 0;
    if (c1 < c0) {
        if (grp == 0 && (!a.seq || a.seq[b] >= 0)) *reinterpret_cast<uint2*>(out) = make_uint2(0u, 0u);
        return;
    }
    if (c0 == c1) return;
    const int64_t mo = (int64_t)a.heads * kD + h, lo = mo + a.heads;
    auto piece = [&](int c) { return part_of(a, c, c == c0 ? slot0 : 0); };
    const int n = c1 - c0 >= grp ? (c1 - c0 - grp) / G + 1 : 0;  // this group's: c0 + grp + G i
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f, M = s2;
    for (int i0 = 0; i0 < n || i0 == 0; i0 += kJoinBatch) {
        float4 v[kJoinBatch];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i)
            if (i0 + i < n)
                v[i] = __ldcg(reinterpret_cast<const float4*>(piece(c0 + grp + G * (i0 + i)) + (int64_t)h * kD) + ch);
        if (i0 == 0) {  // every piece's maximum and sum, once a CTA
            for (int c = threadIdx.x; c <= c1 - c0; c += Join<kWide>::kThreads) {
                const float* p = piece(c0 + c);
                m_s[c] = __ldcg(p + mo);
                l_s[c] = __ldcg(p + lo);
            }
            __syncthreads();
            for (int c = lane; c <= c1 - c0; c += 32) M = fmaxf(M, m_s[c]);
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        }
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i)
            if (i0 + i < n) {
                const int c = grp + G * (i0 + i);
                const float m = m_s[c], w = m == -INFINITY ? 0.f : ex2(m - M);
                den = fmaf(l_s[c], w, den);
                acc.x = fmaf(v[i].x, w, acc.x);
                acc.y = fmaf(v[i].y, w, acc.y);
                acc.z = fmaf(v[i].z, w, acc.z);
                acc.w = fmaf(v[i].w, w, acc.w);
            }
    }
    if constexpr (kWide) {
        sums[grp][lane] = acc;
        if (lane == 0) dens[grp] = den;
        __syncthreads();
        if (grp > 0) return;
#pragma unroll
        for (int i = 1; i < G; ++i) {
            const float4 v = sums[i][lane];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
            den += dens[i];
        }
    }
    den += s2 == -INFINITY ? 0.f : ex2(s2 - M);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    const __nv_bfloat162 y = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(out) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// CTAs of the attention kernel on the current device: one per SM, at most max_ctas. 0: no device.
int grid_of(const csa2_params* p) {
    const int n = min(sm_count(), kMaxCtas);
    return p->max_ctas > 0 && p->max_ctas < n ? p->max_ctas : n;
}

template <bool kBf16, int NH>
int launch_attn(const Args& a, const CUtensorMap& m, cudaLaunchConfig_t* cfg) {
    cfg->gridDim = dim3(a.ctas);
    cfg->blockDim = dim3(Shape<kBf16, NH>::kThreads);
    cfg->dynamicSmemBytes = smem_bytes<kBf16, NH>();
    cudaLaunchKernelEx(cfg, k_paged_attn<kBf16, NH>, a, m);
    return check_launch("paged_attn");
}

int64_t pieces_bytes(int64_t B) { return (8 * B + 255) & ~(int64_t)255; }

int64_t ws_need(int B, int heads, int ctas) { return pieces_bytes(B) + 2 * (int64_t)ctas * part_floats(heads) * 4; }

}  // namespace

cudaError_t preload_paged_attn() {
    cudaError_t (*l[])() = {[] { return preload_kernel(k_paged_attn<true, 64>, smem_bytes<true, 64>()); },
                            [] { return preload_kernel(k_paged_attn<true, 32>, smem_bytes<true, 32>()); },
                            [] { return preload_kernel(k_paged_attn<true, 16>, smem_bytes<true, 16>()); },
                            [] { return preload_kernel(k_paged_attn<false, 64>, smem_bytes<false, 64>()); },
                            [] { return preload_kernel(k_paged_attn<false, 32>, smem_bytes<false, 32>()); },
                            [] { return preload_kernel(k_paged_join<false>); },
                            [] { return preload_kernel(k_paged_join<true>); }};
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
    if (B == 1) q_seq = 0;  // strides that nothing is stepped by
    if (p->heads == 1) q_head = 0;
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
    a.pieces = static_cast<int2*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pieces_bytes(B));
    a.dev_status = dev_status;
    a.scale_log2 = p->softmax_scale * kLog2e;
    a.ctas = ctas;
    a.box_rows = a.g.page_size & -a.g.page_size;
    if (a.box_rows > kTile) a.box_rows = kTile;
    while ((1 << a.box_shift) < a.box_rows) ++a.box_shift;
    CUtensorMap rows = {};
    if (const int rc = encode_rows("paged_attn", a.g, a.base, a.box_rows, &rows)) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // The fewest columns that hold the heads: the query then leaves more of shared memory to
    // the rows, and the softmax and the operand reads shrink with it.
    int rc;
    if (p->kv_format == CSA2_BF16) {
        rc = p->heads > 32 ? launch_attn<true, 64>(a, rows, &cfg)
             : p->heads > 16 ? launch_attn<true, 32>(a, rows, &cfg) : launch_attn<true, 16>(a, rows, &cfg);
    } else {
        rc = p->heads > 32 ? launch_attn<false, 64>(a, rows, &cfg) : launch_attn<false, 32>(a, rows, &cfg);
    }
    if (rc) return rc;
    // A sequence is cut into about ctas / B pieces, at most one a tile, which a narrow thread
    // requests eight at a time. Measured (64 heads, bf16): 1 sequence of 32,768 (128 pieces) 25
    // us wide, 43 narrow; 2 of 131,072 (74 each) 74 and 80; 8 of 8,192 (16 each) 47 and 32; 1 of
    // 200 (2) 14.7 and 13.3.
    int64_t tiles = a.g.max_len() / kTile + 1;
    if (window > 0) {
        const int64_t seen = window / kTile + 2 + (n_first > 0 ? n_first / kTile + 1 : 0);
        if (seen < tiles) tiles = seen;
    }
    const bool wide = ctas / B > 32 && tiles > 32;
    cfg.gridDim = dim3(B, p->heads, wide ? kD / (4 * Join<true>::kLanes) : 1);
    cfg.blockDim = dim3(wide ? Join<true>::kThreads : Join<false>::kThreads);
    cfg.dynamicSmemBytes = 0;
    if (wide) cudaLaunchKernelEx(&cfg, k_paged_join<true>, a);
    else cudaLaunchKernelEx(&cfg, k_paged_join<false>, a);
    return check_launch("paged_attn: join");
}
