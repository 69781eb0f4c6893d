// Attention of a transaction's rows over the paged 8-bit cache (sm_103a).
//
// With R = rows * (h_q / h_kv) query vectors on one kv head a position costs
// 2 d bytes and 4 d R flops: from R of about 8 on only the tensor cores keep
// up with the memory.  Keys and values go to them as they lie in the cache,
// without a conversion: the products are 8-bit with the cache's side exact by
// construction and the other side split into exact 8-bit parts, side by side in
// the N extent, which the few rows leave free:
//   scores   S^T[128 positions][2 RB] = K [q_hi | q_lo]     q = (q_hi + q_lo/32) 2^-k  (bf16's 8 bits)
//   outputs  O^T[d][4 RB] += V^T [p_0 | p_1 | p_2 | p_3]    p = sum p_j 8^-j  (fp16's 11 bits, exactly)
// q in e4m3, exactly but for elements below 2^-14 of their row's largest; where what those
// lose may show, scores are summed by the softmax's threads instead (exact_scores).
// A weight is rounded to fp16, whose upper byte is an e5m2 number, 3 bits of it; a part is
// the upper byte of its predecessor's remainder times 8, so the four hold all 11 bits, of
// subnormals too, and cost neither conversions to 8 bits nor back.
// A position is a tensor-memory lane, so its page's scales are two numbers of
// the thread that owns the lane: K's multiplies the score, V's the weight.
//
// The softmax keeps a reference m per column, not the running maximum: a column's
// weights are 2^(z - m), and what enters the product is a weight times its page's V
// scale, against the largest such scale: 2^(z + e - m).  Only when some z + e passes m
// + kSlack (or a page's V scale the largest so far) is m moved and the sums rescaled;
// usually that is once, at a segment's first tile.  One vote a tile decides.  So a page
// whose large values get next to no weight takes no bits from the others' weights.
//
// Work is measured in tiles of 128 positions: a unit (request, kv head, block of RB
// columns) costs its tiles plus a few for its ends, and the units laid end to end
// are cut into equal ranges, one for each of the persistent CTAs.  A CTA runs the
// units and parts of units of its range as segments.  Its warps:
//   copy     finds the segments, queues them, and moves pages (tiled TMA, K and V
//            tiles through one ring) and their scales, into the next segment while
//            the last one is still being summed
//   product  issues the tensor-core products, and splits the segment's new keys
//   softmax  groups of four warps (thread = position = lane), a share of the
//            columns each: queries in, weights, outputs out
// The transaction's own rows, bf16, come last in a unit: their keys as one more
// tile, each a hi and a lo position (16 + 16 lanes) split like q, their values in
// fp32 in the epilogue.  A unit inside one range is written directly; the parts
// of a cut one leave (m, l, O) in the workspace for kv8_join_kernel.  With a
// given split the cuts are at its multiples instead, whatever the ranges.
//
// Roundings: what the splits of q and of a new key leave out is 2^-14 of a score (in
// powers of two) at most each, an eighth of a weight's rounding.  A weight is rounded to
// fp16, 2^-11 of it at most, an eighth of what an output's rounding to bf16 takes: the four
// 8-bit parts would hold one bit more, and four e4m3 parts 14 bits, but the conversions
// made 16 rows x 32 requests 128 us for 121.  The sum of the weights is of the unrounded
// ones (the log-sum-exp is to be right), so a row that one position makes up keeps that
// position's rounding.  Scores, statistics and outputs are fp32, and an output is rounded
// once, to bf16.
//
// What bounds it (bytes over time, and of the 6.78 TB/s of a copy): HBM and the ends
// of segments in large batches (4 rows x 256 requests, 2 heads of 256: 786 MB in 137
// us, 5.7 TB/s, 84 %) and long requests (256k tokens: 269 MB in 53.5 us, 5.0 TB/s, 74
// %, of which about 5 us are the join and 4 the start; 16 requests of a mixed batch
// 258 MB in 54.5 us, 70 %); from 64 columns on the softmax's chains, about 500
// instructions a warp and tile at 60 % of the issue slots (16 rows x 32 requests, 4
// heads of 128: 123 us, five times what HBM would need); the chain from a segment's
// queries to its outputs, about 4 us, where requests are short, and then also the
// fetching of its instructions: loops there are rolled wherever that costs nothing.
#include "kv8_math.cuh"
#include "tmap.cuh"

namespace {

using namespace kv8;

constexpr int kTile = 128;      // positions a tile
constexpr int kSms = 152;
// Weights (times V scale) are scaled by 2^7 and at most 2^(7 + 8), inside fp16, whose normal
// numbers go down to 2^-14: 2^-21 of a weight at the reference.  More slack moves the reference
// less often (16 rows x 32 requests 145 us with 3, 121 with 6, 119.5 with 8 and with 10).
constexpr float kBase = 128.f, kSlack = 8.f;
constexpr float kUnset = -1e30f;
// How far apart (in powers of two) V scales may lie for a reference to follow them: weights
// before their V scale are then at most 2^(kSlack + 2 kLift), and sums of 2^20 of them finite.
constexpr float kLift = 48.f;
constexpr float kLog2e = 1.4426950408889634f;
// What a score (in powers of two) may be off by for the parts of a query or of a new key;
// where it might be more it is summed from the elements (exact_scores).  One element of a
// normal distribution in 8,000 loses bits, 2^-22 of its row's largest at most: with scores
// of hundreds that is still less, and ordinary requests are never summed that way.
constexpr float kScoreLoss = 0x1p-14f;
constexpr float kUnit = 0x1p30f;  // what rows past 2^67 are divided by there
constexpr int kQueue = 4;       // segments queued
constexpr int kLeast = 2;       // tiles a part of a cut unit has at least

// Tiles that a unit's queries, new rows and outputs cost as much as.  A fit of a CTA's
// cycles to its tiles and segments gives 3 to 7; of those and two tiles more or less,
// these were the fastest (4 rows x 256 requests 140, 136 and 139 us at 4, 6 and 8,
// 16 rows x 32 requests 129, 129 and 136 at 6, 8 and 10, before its weights were fp16).
__host__ __device__ constexpr int unit_cost(int rb) { return rb == 64 ? 8 : rb == 32 ? 6 : 4; }

// Units of at most 2 * kLeast tiles are not cut, nor, where each can have its own CTA,
// of kWhole if they fill half of the CTAs, of half that if a quarter: the join costs
// more (24 windowed requests x 12 heads, 9 tiles: 22.5 us cut, 16.1 whole; 64 requests
// x 2 heads, 8 tiles: 19.6 and 16.5; but 8 heads of one request, 8 tiles: 10.7 and
// 12.3, and 32 units of 16 tiles 16.5 and 22).
constexpr int kWhole = 16;

// Ranges that a total weight is cut into where CTAs do not run out: of four tiles or
// more, or, up to one CTA an SM, of two (two heads of one request of 16 tiles: 17.8 us
// with four, 15.7 with two; 32 units of 16 tiles: 16.7 on 176 CTAs, 18.2 on 304).  No
// fewer than kLeast, or one could lie empty inside a unit.
__host__ __device__ constexpr long long ranges_of(long long total) {
    const long long two = total / kLeast, four = total / 4;
    return four > kSms ? four : two < kSms ? two : kSms;
}

// A part of a unit cut by the ranges: the unit (first row, kv head, block and its
// columns in use) and the CTAs owner .. owner + count - 1 that have its parts
// (count 0: none).
struct alignas(16) Part {
    int owner, count, t0, cols, hk, blk, pad[2];
};

struct AttendArgs {
    CUtensorMap map;
    kv8_cache c;
    int32_t layer, B, row_capacity, table_pages, max_len, max_rows;
    int32_t group, blocks, page_shift;  // page_tokens = 1 << page_shift
    int32_t pinned, piece_tiles, max_pieces;  // given cuts, at multiples of piece_tiles
    int64_t table_stride;
    const int32_t *cu_rows, *cache_len, *table;
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, o_stride;
    uint16_t *o;
    float *lse;
    float *ws_o;       // [part][RB][d]
    float2 *ws_ml;     // [part][RB]
    Part *parts;       // [CTA][2]: of a unit begun before the range, of one that goes on after it
    uint32_t *status;
    uint64_t wait_ns;
    int32_t withhold;  // self-test: a segment's last keys are announced and never copied
};

// What a request asks for; the same test in both kernels.
struct Request {
    int t0, n, len, lo, tiles;  // lo: first position any row sees; tiles from lo / 128 on
    bool bad;
};
__device__ __forceinline__ int3 rows_of(const AttendArgs &a, int r) {
    return make_int3(a.cu_rows[r], a.cu_rows[r + 1], a.cache_len[r]);
}
__device__ __forceinline__ Request request_of(const AttendArgs &a, int3 x) {
    Request q;
    q.t0 = x.x;
    q.n = x.y - x.x;
    q.len = x.z;
    q.bad = q.t0 < 0 || q.n < 0 || q.n > a.max_rows || int64_t(q.t0) + q.n > a.row_capacity || q.len < 0 ||
            q.len > a.max_len || int64_t(q.len) > int64_t(a.table_pages) * a.c.page_tokens;
    const int w = a.c.window;
    q.lo = w ? max(0, q.len + (a.k ? 1 : 0) - w) : 0;
    if (q.lo > q.len) q.lo = q.len;
    const int first = q.lo / kTile;
    q.tiles = q.lo < q.len ? (q.len + kTile - 1) / kTile - first : 0;
    return q;
}

struct Segment {
    int r, t0, len, lo, tile0, nc, out;  // cached tiles tile0 .. + nc; out: part of the workspace, -1: direct
    uint16_t hk, blk;
    uint8_t n, cols, fresh;              // cols 0: no more segments
};

template <int D, int RB>
struct Cfg {
    static constexpr int kRow = D < 128 ? D : 128;       // bytes of an operand tile's row
    static constexpr int kAtoms = D / kRow;              // such tiles side by side
    static constexpr int kNs = 2 * RB;                   // score columns
    static constexpr int kNp = 4 * RB;                   // weight columns
    static constexpr int kPRow = RB == 8 ? 64 : RB == 64 ? 128 : kNp;  // bytes of a weight tile's row (64 or 128)
    static constexpr int kFresh = 32 * D;  // bytes of the fresh keys, and of the values
    static constexpr int kQ = kNs * D;
    static constexpr int kP = kTile * (RB == 8 ? 64 : kNp);
    static constexpr int kSlot = kTile * D;
    // Groups of four softmax warps, each with its share of the columns: a warp waits
    // on its own chain of loads, exponentials and conversions most of the time, so an
    // SM wants eight of them or more (171 requests of 2 rows, 12 columns of 256: 43 us
    // with four, 37 with eight; 64 of 4 rows, 16 columns of 128, two CTAs an SM: 34.7
    // us with eight, 32.2 with sixteen; at d = 64 it is 47.5 and 49), and sixteen where
    // 64 columns leave the products time (16 rows x 32 requests 134 us with eight, 129
    // with sixteen, whose 96 registers spill a little).
    static constexpr int kGroups = RB <= 8 ? 1 : RB == 16 ? (D == 64 ? 1 : 2) : RB == 32 ? 2 : 4;
    static constexpr int kCols = RB / kGroups;           // columns a thread
    static constexpr int kSoft = 128 * kGroups;          // softmax threads
    static constexpr int kThreads = kSoft + 64;
    // CTAs an SM: two, unless 512 tensor-memory columns or two sets of 32 KB slots rule
    // it out (three at d = 64 change nothing: 152 requests of 1 row 45.5 and 45.7 us)
    static constexpr int kCtas = D == 256 || RB == 64 ? 1 : 2;
    static constexpr int kFixed = 2 * kFresh + kQ + 2 * kP + (D == 64 ? kSlot : 0) + 1024;
    static constexpr int kStatic =  // bound on sizeof(Shared)
        RB == 64 ? 5120 : RB == 32 ? 3072 : RB == 16 || D == 64 ? 2560 : 2048;
    static constexpr int kRoom = (kCtas == 1 ? 227 * 1024 : 113 * 1024) - kStatic - kFixed;
    static constexpr int kSlots = kRoom / kSlot > 10 ? 10 : kRoom / kSlot;
    static constexpr int kSmem = kFixed + kSlots * kSlot;
    // Tiles whose scales may wait to be read: the copy of tile i + kScales' keys
    // needs a slot that tile i + 2's keys (or tile i's values) have left, and the
    // scales of tile i are read before either
    static constexpr int kScales = kSlots <= 5 ? 4 : 8;
    static constexpr int kTmemUse = 2 * kNs + kNp * (D == 256 ? 2 : 1);
    static constexpr int kTmem = kTmemUse <= 64 ? 64 : kTmemUse <= 128 ? 128 : kTmemUse <= 256 ? 256 : 512;
    static_assert(kTmemUse <= 512 && kSlots >= 3, "does not fit an SM");
};

template <int D, int RB>
struct Shared {
    using C = Cfg<D, RB>;
    union {  // barriers that one thread or the tensor cores arrive at
        uint64_t ones[C::kSlots * 2 + C::kScales + 4 + kQueue + 3];
        struct {
            uint64_t full[C::kSlots], empty[C::kSlots], sc_full[C::kScales], s_full[2], pv_done[2], seg_full[kQueue],
                fk_ready, fv_full, drain;
        };
    };
    union {  // barriers of the softmax warps
        uint64_t warps[6];
        struct {
            uint64_t s_free[2], p_full[2], q_ready, epi_done;
        };
    };
    uint64_t seg_empty[kQueue];  // of the softmax warps and the product warp
    float2 scales[C::kScales][8];
    alignas(16) float col_nm[RB], col_coef[RB], col_fac[RB];  // -m, score factor, rescaling
    float col_l[RB];  // what a moving reference adds to z; at the end 1 / l
    union {
        float col_max[4][RB];
        long long scan[C::kThreads / 32];
    };
    float v_max[C::kGroups][4];
    // what a new key's and a column's parts are times (negative: always summed from the elements, over kUnit);
    // a new key's loss; the K scale past which a column's loss shows, and the least of a group's (by segments in turn)
    float fresh_k[16], fresh_loss[16], col_down[RB], col_limit[RB], k_limit[2][C::kGroups];
    Segment seg[kQueue];
    int bad[kQueue];
    long long start_at;
    int start_r;
    int3 start_rows;
    uint32_t tmem;
    int fresh_lossy;                    // whether any new key's loss may show
    int col_out[RB];                    // element of o, from the request's first row on
    uint8_t col_row[RB], col_head[RB];  // of the request's rows, of the kv head's queries
};

// Ring positions of a segment's loads, in the order the products use them:
// K0 K1 V0 K2 V1 ... V(n-1).
__device__ __forceinline__ int k_pos(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_pos(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

// What a unit of `tiles` tiles weighs in the ranges: with given cuts its pieces.
__device__ __forceinline__ int cost_of(const AttendArgs &a, int tiles, int rb) {
    return a.pinned ? max(1, (tiles + a.piece_tiles - 1) / a.piece_tiles) : tiles + unit_cost(rb);
}
__device__ __forceinline__ long long weight_of(const AttendArgs &a, const Request &q, int rb) {
    if (q.bad || q.n == 0) return 0;
    return (long long)(a.c.h_kv) * ((q.n * a.group + rb - 1) / rb) * cost_of(a, q.tiles, rb);
}

// a / b for values that usually fit 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)(uint32_t(a) / uint32_t(b)) : a / b;
}

// The tile at which a range's end, x into a unit of `tiles` tiles, cuts it: 0 its
// start, tiles + 1 its end.  Free cuts leave no part of fewer than kLeast tiles.
__device__ __forceinline__ int cut_at(const AttendArgs &a, long long x, int tiles) {
    if (x <= 0) return 0;
    if (x > tiles) return tiles + 1;
    if (!a.pinned) return x < kLeast ? 0 : x > tiles - kLeast ? tiles + 1 : int(x);
    const long long y = x * a.piece_tiles;
    return y >= tiles ? tiles + 1 : int(y);
}

// Of a group's columns those in whose score with this lane's key (a cached one of K scale
// k, or new key j) more than kScoreLoss may be missing.  Every element of a key is below
// 448 times its page's scale, or 256 times what its parts are times; of a query likewise.
template <int D, int RB>
__device__ __noinline__ uint32_t lossy_columns(const Shared<D, RB> &s, int j, float k, int col0, int cols) {
    float loss = 0.f;
    bool all = false;
    if (j >= 0) {
        k = s.fresh_k[j];
        if (k != k) return 0;  // not finite: the parts' scores say so
        all = k < 0.f;
        k = fabsf(k);
        if (s.fresh_lossy) loss = s.fresh_loss[j];
    }
    uint32_t mask = 0;
#pragma unroll 1
    for (int c = 0; c < Cfg<D, RB>::kCols && col0 + c < cols; ++c) {
        const float f = s.col_down[col0 + c], coef = 256.f * fabsf(s.col_coef[col0 + c]);
        if (f < 0.f || (f == f && (all || k > s.col_limit[col0 + c] || loss * coef > kScoreLoss))) mask |= 1u << c;
    }
    return mask;
}
// Such scores, summed in fp32 from the queries and keys in global memory, into this warp's
// lanes of the score tile (the low parts' columns zero).  t: the lane's cached position, -1
// in a tile of new keys; mask: its columns.  Rare: small for the loop's sake, and slow, with
// all of a unit's columns a tile takes some 50 times as long.  (With the keys' codes in
// registers it is 20 times, but then the ordinary tiles suffer: 16 requests 75 us for 53.)
template <int D, int RB>
__device__ __noinline__ void exact_scores(const AttendArgs &a, const Shared<D, RB> &s, const Segment &g, int t,
                                          uint32_t mask, int pos_in, int col0, uint32_t at) {
    const int T = a.c.page_tokens;
    const bool is_fresh = t < 0;
    const uint8_t *codes = a.c.kv;
    const uint16_t *key = a.k + (int64_t(g.t0) + (pos_in & 15)) * a.k_stride + int64_t(g.hk) * D;
    if (!is_fresh && mask) {
        const int page = a.table[int64_t(g.r) * a.table_stride + (t >> a.page_shift)];
        if (page < 0 || page >= a.c.num_pages) mask = 0;
        codes += int64_t(page) * a.c.page_stride + int64_t(a.layer) * a.c.layer_stride +
                 (int64_t(g.hk) * T + (t & (T - 1))) * D;
    }
#pragma unroll 1
    for (int c = 0; c < Cfg<D, RB>::kCols; ++c) {
        const bool mine = mask >> c & 1;
        if (!__any_sync(0xffffffffu, mine)) continue;
        uint32_t hi = tc::ld1(at + c), lo = tc::ld1(at + RB + c);
        if (mine) {
            const uint16_t *q = a.q + (int64_t(g.t0) + s.col_row[col0 + c]) * a.q_stride +
                                int64_t(g.hk * a.group + s.col_head[col0 + c]) * D;
            const float up = 1.f / fabsf(s.col_down[col0 + c]);
            if (!is_fresh)
                hi = __float_as_uint(dot_codes<D>(codes, q, up));
            else  // the low parts of the keys lie 16 lanes on
                hi = pos_in & 16 ? 0u : __float_as_uint(dot_rows<D>(key, 1.f / fabsf(s.fresh_k[pos_in & 15]), q, up));
            lo = 0;
        }
        __syncwarp();
        tc::st1(at + c, hi);
        tc::st1(at + RB + c, lo);
    }
    tc::st_wait();
}

template <int D, int RB>
__global__ void __launch_bounds__(Cfg<D, RB>::kThreads, Cfg<D, RB>::kCtas)
    kv8_attend_kernel(const __grid_constant__ AttendArgs a) {
    using C = Cfg<D, RB>;
    extern __shared__ uint8_t raw[];
    __shared__ Shared<D, RB> s;
    static_assert(sizeof(Shared<D, RB>) <= C::kStatic, "static shared memory");

    gdn::pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kCopyWarp = C::kSoft / 32, kMmaWarp = kCopyWarp + 1;
    // barriers and tensor memory while the launch before may still be running
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&s.tmem, C::kTmem);
    } else if (warp == kCopyWarp) {
        constexpr int kOnes = C::kSlots * 2 + C::kScales + 4 + kQueue + 3, kWarps = C::kSoft / 32;
        for (int i = lane; i < kOnes; i += 32) gdn::mbar_init(s.ones + i, 1);
        if (lane < 6) gdn::mbar_init(s.warps + lane, kWarps);
        if (lane < C::kGroups) s.k_limit[0][lane] = INFINITY;
        if (lane < kQueue) gdn::mbar_init(s.seg_empty + lane, kWarps + 1);
    }
    gdn::pdl_wait();

    // ---- this CTA's range of the units laid end to end
    long long total, begin, end;
    int ctas;
    {
        const int chunk = (a.B + C::kThreads - 1) / C::kThreads, r0 = tid * chunk, r1 = min(a.B, r0 + chunk);
        long long mine = 0;
        for (int r = r0; r < r1; ++r) {
            const Request q = request_of(a, rows_of(a, r));
            mine += weight_of(a, q, RB);
            if (q.bad && blockIdx.x == 0) gdn::set_status(a.status, GDN_DEV_ROWS_BAD);
        }
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        if (lane == 31) s.scan[warp] = incl;
        __syncthreads();
        total = 0;
        long long before = 0;
#pragma unroll
        for (int w = 0; w < C::kThreads / 32; ++w) {
            if (w < warp) before += s.scan[w];
            total += s.scan[w];
        }
        const long long most = a.pinned ? total : ranges_of(total);
        ctas = int(most < 1 ? 1 : most < gridDim.x ? most : gridDim.x);
        const int cta = blockIdx.x;
        if (tid == 0 && a.parts) a.parts[2 * cta].count = a.parts[2 * cta + 1].count = 0;
        if (cta >= ctas || total == 0) {
            if (warp == kMmaWarp) tc::tmem_dealloc(s.tmem, C::kTmem);
            return;
        }
        begin = quotient(total * cta, ctas);
        end = quotient(total * (cta + 1), ctas);
        incl += before;
        if (incl - mine <= begin && begin < incl) {
            long long at = incl - mine;
            for (int r = r0; r < r1; ++r) {
                const int3 x = rows_of(a, r);
                const long long w = weight_of(a, request_of(a, x), RB);
                if (at + w > begin) {
                    s.start_r = r;
                    s.start_rows = x;
                    s.start_at = at;
                    break;
                }
                at += w;
            }
        }
    }

    const int T = a.c.page_tokens, shift = a.page_shift;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *s_fk = sm, *s_fv = s_fk + C::kFresh, *s_q = s_fv + C::kFresh;
    uint8_t *s_p = s_q + ((C::kQ + 1023) & ~1023), *s_ring = s_p + 2 * C::kP;

    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = s.tmem, tm_o = tm + 2 * C::kNs;

    if (warp == kCopyWarp) {
        // ---- copies
        const int per = kTile >> shift;  // pages a tile
        const float *sc0 = a.c.scale + int64_t(a.layer) * a.c.scale_layer_stride;
        const int cta = blockIdx.x;
        bool ok = true;
        int k = 0, ring = 0, issued = 0;       // segments and ring positions so far; copies issued
        int tiles_done = 0, fresh_done = 0;
        auto push = [&](const Segment &g) {
            if (k >= kQueue)
                ok = ok && gdn::mbar_wait_bounded(&s.seg_empty[k % kQueue], (k / kQueue - 1) & 1, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            if (lane == 0) {
                s.seg[k % kQueue] = g;
                s.bad[k % kQueue] = 0;
                arrive(&s.seg_full[k % kQueue]);
            }
            __syncwarp();
        };
        // A segment: queue it, then its tiles.  Page ids and scales come 32 pages at a
        // time, ids two and scales one such batch ahead.
        auto run = [&](const Segment &g) {
            push(g);
            if (!ok) return;
            const int nc = g.nc, page0 = g.tile0 * per, first = g.lo >> shift, last = (g.len + T - 1) >> shift;
            const int32_t *tab = a.table + int64_t(g.r) * a.table_stride;
            auto ids = [&](int batch) {
                const int x = batch * 32 + lane, j = page0 + x;
                return j >= first && j < last && x < nc * per ? tab[j] : -1;
            };
            auto scales = [&](int p) {
                return p >= 0 && p < a.c.num_pages
                           ? *reinterpret_cast<const float2 *>(sc0 + int64_t(p) * a.c.scale_page_stride + 2 * g.hk)
                           : make_float2(0.f, 0.f);
            };
            auto issue = [&](int pos, int page, int is_v) {
                const int slot = pos % C::kSlots;
                if (pos >= C::kSlots)
                    ok = ok && gdn::mbar_wait_bounded(&s.empty[slot], (pos / C::kSlots - 1) & 1, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                const uint32_t have = __ballot_sync(0xffffffffu, lane < per && page >= 0);
                if (lane == 0) gdn::mbar_arrive_expect_tx(&s.full[slot], uint32_t(__popc(have)) * uint32_t(T * D));
                __syncwarp();
                issued = pos + 1;
                if (a.withhold && pos == ring + k_pos(nc - 1)) return;
                if (lane < per && page >= 0) {
#pragma unroll
                    for (int x = 0; x < C::kAtoms; ++x)
                        gdn::tma_load_3d(s_ring + slot * C::kSlot + x * kTile * C::kRow + lane * T * C::kRow, &a.map,
                                         x * C::kRow, (is_v * a.c.h_kv + g.hk) * T, page, &s.full[slot]);
                }
            };
            int cur = ids(0), nxt = ids(1), far = ids(2), batch = 0, prev = -1;
            float2 sc = scales(cur), sc_nxt = scales(nxt);
            for (int i = 0; i <= nc && ok; ++i) {
                int page = -1;
                const int at = i * per, src = (at % 32) + (lane & (per - 1));
                if (i < nc) {
                    if (at / 32 != batch) {
                        batch = at / 32;
                        cur = nxt;
                        sc = sc_nxt;
                        nxt = far;
                        sc_nxt = scales(nxt);
                        far = ids(batch + 2);
                    }
                    page = __shfl_sync(0xffffffffu, cur, src);
                    if (page < 0 || page >= a.c.num_pages) {
                        // a bad id is not loaded, and the segment's outputs are dropped
                        const int j = page0 + at + (lane & (per - 1));
                        if (j >= first && j < last) *reinterpret_cast<volatile int *>(&s.bad[k % kQueue]) = 1;
                        page = -1;
                    }
                    issue(ring + k_pos(i), page, 0);
                }
                if (i > 0 && ok) issue(ring + v_pos(i - 1, nc), prev, 1);
                if (i < nc && ok) {
                    float2 x;
                    x.x = __shfl_sync(0xffffffffu, sc.x, src);
                    x.y = __shfl_sync(0xffffffffu, sc.y, src);
                    const int e = (tiles_done + i) % C::kScales;
                    if (lane < per) s.scales[e][lane] = x;
                    __syncwarp();
                    if (lane == 0) arrive(&s.sc_full[e]);
                }
                prev = page;
            }
            if (ok) {
                ring += 2 * nc;
                tiles_done += nc;
            }
            if (ok && g.fresh) {
                // the new rows' values, once the segment before is done with their place
                if (k > 0)
                    ok = gdn::mbar_wait_bounded(&s.seg_empty[(k - 1) % kQueue], ((k - 1) / kQueue) & 1, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    if (lane == 0) gdn::mbar_arrive_expect_tx(&s.fv_full, uint32_t(g.n) * (2 * D));
                    __syncwarp();
                    if (lane < g.n)
                        gdn::bulk_g2s(s_fv + lane * 2 * D,
                                      a.v + (int64_t(g.t0) + lane) * a.v_stride + int64_t(g.hk) * D, 2 * D, &s.fv_full);
                    ++fresh_done;
                }
            }
            ++k;
        };
        int r = s.start_r;
        long long at = s.start_at;
        Request q = request_of(a, s.start_rows);
        while (at < end && ok) {
            const int3 next = rows_of(a, min(r + 1, a.B - 1));  // looked at when its turn comes
            const long long w = weight_of(a, q, RB);
            if (w > 0) {
                const int cost = cost_of(a, q.tiles, RB), whole = q.tiles + 1;
                const int nb = (q.n * a.group + RB - 1) / RB, units = a.c.h_kv * nb;
                int u = begin > at ? int(quotient(begin - at, cost)) : 0;
                for (; u < units && at + (long long)u * cost < end && ok; ++u) {
                    const long long su = at + (long long)u * cost;
                    const int x0 = cut_at(a, begin - su, q.tiles), x1 = cut_at(a, end - su, q.tiles);
                    Segment g;
                    g.r = r;
                    g.t0 = q.t0;
                    g.n = uint8_t(q.n);
                    g.len = q.len;
                    g.lo = q.lo;
                    g.hk = uint16_t(u / nb);
                    g.blk = uint16_t(u % nb);
                    g.cols = uint8_t(min(RB, q.n * a.group - g.blk * RB));
                    const int y = g.hk * a.blocks + g.blk;
                    // given cuts: a segment for each piece of the range
                    for (int x = x0; x < x1 && ok;) {
                        int to = a.pinned ? min(x + a.piece_tiles, x1) : x1;
                        if (to >= q.tiles) to = whole;  // with the new rows and the end
                        g.tile0 = q.lo / kTile + x;
                        g.nc = min(to, q.tiles) - x;
                        g.fresh = a.k != nullptr && to == whole;
                        g.out = -1;
                        if (a.pinned) {
                            if (q.tiles > a.piece_tiles)
                                g.out = (r * a.max_pieces + x / a.piece_tiles) * (a.c.h_kv * a.blocks) + y;
                        } else if (x0 > 0 || x1 < whole) {
                            // the first CTA whose end lies past the start, the first whose end counts as the unit's
                            const long long lo = su + kLeast, hi = su + q.tiles - kLeast + 1;
                            Part p = {};
                            p.t0 = q.t0;
                            p.cols = g.cols;
                            p.hk = g.hk;
                            p.blk = g.blk;
                            p.owner = int(quotient(lo * ctas + total - 1, total)) - 1;
                            p.count = int(quotient(hi * ctas + total - 1, total)) - p.owner;
                            g.out = 2 * cta + (x0 > 0 ? 0 : 1);
                            if (lane == 0) a.parts[g.out] = p;
                        }
                        run(g);
                        x = to;
                    }
                }
            }
            at += w;
            ++r;
            if (r >= a.B) break;
            q = request_of(a, next);
        }
        if (ok) {
            Segment g = {};
            push(g);
        }
        if (!ok) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
        // every copy has landed before the CTA leaves (on the usual path these waits are over)
        for (int pos = max(0, issued - C::kSlots); pos < issued; ++pos)
            (void)gdn::mbar_wait_bounded(&s.full[pos % C::kSlots], (pos / C::kSlots) & 1, a.wait_ns);
        if (fresh_done) (void)gdn::mbar_wait_bounded(&s.fv_full, (fresh_done - 1) & 1, a.wait_ns);
    } else if (warp == kMmaWarp) {
        // ---- products: the warp runs the loop, one elected lane issues
        constexpr uint32_t id_s = tc::idesc_e4m3(128, C::kNs);
        constexpr uint32_t id_p = tc::idesc_e4m3(128, C::kNp) | tc::kBE5m2 | tc::kAMnMajor | tc::kBMnMajor;
        const uint64_t dq = tc::smem_desc8<C::kRow>(gdn::smem_u32(s_q), 16);
        // weights: rows are positions; RB = 64 has two tiles of 128 columns
        const uint64_t dp = tc::smem_desc8<C::kPRow>(gdn::smem_u32(s_p), kTile * C::kPRow);
        // V has 128 rows of M at d >= 128; at d = 64 rows 64.. read the next slot and are not used
        constexpr uint32_t lbo = C::kRow == 64 ? C::kSlot : 16;
        const uint64_t dk0 = tc::smem_desc8<C::kRow>(gdn::smem_u32(s_ring), 16);
        const uint64_t dv0 = tc::smem_desc8<C::kRow>(gdn::smem_u32(s_ring), lbo);
        const uint64_t dfk = tc::smem_desc8<C::kRow>(gdn::smem_u32(s_fk), 16);
        const bool leader = elect_one();
        bool ok = true;
        int ring = 0, gs = 0, gp = 0;  // ring positions, score tiles and weight tiles before this segment
        int last_fresh = -1;           // the last tile of new keys
        for (int k = 0; ok; ++k) {
            ok = gdn::mbar_wait_bounded(&s.seg_full[k % kQueue], (k / kQueue) & 1, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const Segment &g = s.seg[k % kQueue];
            const int nc = g.nc, n = g.n, fresh = g.fresh, nt = nc + fresh;
            if (g.cols == 0) break;
            const uint16_t *kn = a.k + int64_t(g.t0) * a.k_stride + int64_t(g.hk) * D;
            bool maybe = false;  // some new key may have a loss, and fk_ready is still to come
            if (fresh) {
                // the new keys, while the softmax ends the segment before: their place is free
                // once the scores of the last ones are read
                // (a tile two or more back is waited for before the one that took its buffer)
                const int x = last_fresh;
                if (x >= 0 && x >= gs - 2) ok = gdn::mbar_wait_bounded(&s.s_free[x & 1], (x >> 1) & 1, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint4 w[D / 64], next[D / 64];  // four rows a pass
                load_row<D>(kn + int64_t(lane >> 3) * a.k_stride, lane & 7, (lane >> 3) < n, w);
#pragma unroll 1
                for (int row = lane >> 3; row - (lane >> 3) < n; row += 4) {
                    load_row<D>(kn + int64_t(row + 4) * a.k_stride, lane & 7, row + 4 < n, next);
                    bool here;
                    const float down = split_row<D>(w, lane & 7, s_fk, 32, row, 16 + row, here);
                    maybe |= here;
                    if ((lane & 7) == 0) s.fresh_k[row] = down;
#pragma unroll
                    for (int e = 0; e < D / 64; ++e) w[e] = next[e];
                }
                gdn::fence_proxy_async_smem();
                maybe = __any_sync(0xffffffffu, maybe);
                __syncwarp();
                if (lane == 0 && !maybe) {
                    s.fresh_lossy = 0;
                    arrive(&s.fk_ready);
                }
                last_fresh = gs + nc;
            }
            ok = gdn::mbar_wait_bounded(&s.q_ready, k & 1, a.wait_ns);
            for (int i = 0; i <= nt; ++i) {
                if (i < nt) {
                    const bool cached = i < nc;
                    const int pos = ring + k_pos(i), slot = pos % C::kSlots, x = gs + i;
                    if (ok && cached) ok = gdn::mbar_wait_bounded(&s.full[slot], (pos / C::kSlots) & 1, a.wait_ns);
                    if (ok && x >= 2) ok = gdn::mbar_wait_bounded(&s.s_free[x & 1], ((x >> 1) - 1) & 1, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::fence_after();
                    if (leader) {
                        const uint64_t dk = cached ? tc::desc_at(dk0, slot * C::kSlot) : dfk;
                        const uint32_t atom = cached ? kTile * C::kRow : 32 * C::kRow;
#pragma unroll
                        for (int e = 0; e < D / 32; ++e) {
                            const uint32_t t = e * 32 / C::kRow, in = e * 32 % C::kRow;
                            tc::mma_e4m3(tm + (x & 1) * C::kNs, tc::desc_at(dk, t * atom + in),
                                         tc::desc_at(dq, t * C::kNs * C::kRow + in), id_s, e > 0);
                        }
                        tc::commit(&s.s_full[x & 1]);
                        if (cached) tc::commit(&s.empty[slot]);
                    }
                    __syncwarp();
                    if (maybe) {
                        // the first scores are on their way: time to look at the new keys again
                        float coef = 0.f;  // the columns' largest score factor (a kUnit one counts for itself)
                        for (int c = lane; c < g.cols; c += 32) coef = fmaxf(coef, fabsf(s.col_coef[c]));
                        coef = 256.f * warp_max(coef);
                        bool lossy = false;
#pragma unroll 1
                        for (int row = lane >> 3; row - (lane >> 3) < n; row += 4) {
                            uint4 w[D / 64];
                            load_row<D>(kn + int64_t(row) * a.k_stride, lane & 7, row < n, w);
                            const float loss = row_loss<D>(w);
                            if ((lane & 7) == 0 && row < n) {
                                s.fresh_loss[row] = loss;
                                if (loss < 0.f) s.fresh_k[row] = -kUnit;
                            }
                            lossy |= loss < 0.f || loss * coef > kScoreLoss;
                        }
                        lossy = __any_sync(0xffffffffu, lossy);
                        __syncwarp();
                        if (lane == 0) {
                            s.fresh_lossy = lossy;
                            arrive(&s.fk_ready);
                        }
                        maybe = false;
                    }
                }
                if (i > 0 && i <= nc) {
                    const int j = i - 1, pos = ring + v_pos(j, nc), slot = pos % C::kSlots, x = gp + j;
                    if (ok) ok = gdn::mbar_wait_bounded(&s.full[slot], (pos / C::kSlots) & 1, a.wait_ns);
                    if (ok) ok = gdn::mbar_wait_bounded(&s.p_full[x & 1], (x >> 1) & 1, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::fence_after();
                    if (leader) {
                        const uint64_t dv = tc::desc_at(dv0, slot * C::kSlot), dpx = tc::desc_at(dp, (x & 1) * C::kP);
#pragma unroll
                        for (int t = 0; t < C::kAtoms; ++t)
#pragma unroll
                            for (int e = 0; e < kTile / 32; ++e)
                                tc::mma_e4m3(tm_o + t * C::kNp, tc::desc_at(dv, t * kTile * C::kRow + e * 32 * C::kRow),
                                             tc::desc_at(dpx, e * 32 * C::kPRow), id_p, j > 0 || e > 0);
                        tc::commit(&s.pv_done[x & 1]);
                        tc::commit(&s.empty[slot]);
                    }
                    __syncwarp();
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ring += 2 * nc;
            gs += nt;
            gp += nc;
            if (lane == 0) arrive(&s.seg_empty[k % kQueue]);
        }
        if (!ok) {
            gdn::set_status(a.status, GDN_DEV_TIMEOUT);
            if (leader) tc::commit(&s.drain);  // products in flight read shared and write tensor memory
            (void)gdn::mbar_wait_bounded(&s.drain, 0, a.wait_ns);
        }
        __syncwarp();
    } else {
        // ---- softmax.  This thread's position in a tile and its columns col0 .. col0 + N - 1;
        // eight threads bring a column's queries, of their own group's (columns fill whole warps).
        constexpr int N = C::kCols;
        static_assert(N == 8 || N == 16, "a thread has one column's queries");
        const int grp = warp >> 2, pos_in = tid & 127, col0 = grp * N, cq = col0 + (pos_in >> 3), sub = tid & 7;
        const bool brings = pos_in < 8 * N;
        const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
        bool ok = gdn::mbar_wait_bounded(&s.seg_full[0], 0, a.wait_ns);
        if (group_or(grp, !ok)) ok = false;
        Segment g = s.seg[0];
        if (!ok) g.cols = 0;
        uint4 wq[D / 64];
        auto load_q = [&] {
            const int x = g.blk * RB + cq, row = x / a.group;
            if (brings)
                load_row<D>(a.q + (int64_t(g.t0) + row) * a.q_stride + int64_t(g.hk * a.group + x - row * a.group) * D,
                            sub, cq < g.cols, wq);
        };
        load_q();
        int gs = 0, gp = 0, ring = 0, fresh_seen = 0;  // score and weight tiles, ring positions, fresh tiles so far
        for (int k = 0; g.cols > 0; ++k) {
            bool maybe = false;
            if (brings) {
                const float down = split_row<D>(wq, sub, s_q, C::kNs, cq, RB + cq, maybe);
                if (sub == 0) {
                    const int x = g.blk * RB + cq, row = x / a.group, head = x - row * a.group;
                    s.col_nm[cq] = -kUnset;
                    s.col_coef[cq] = a.c.sm_scale * kLog2e * down;
                    s.col_down[cq] = down;
                    s.col_limit[cq] = INFINITY;
                    s.col_row[cq] = uint8_t(row);
                    s.col_head[cq] = uint8_t(head);
                    s.col_out[cq] = row * int(a.o_stride) + (g.hk * a.group + head) * D;
                }
            }
            gdn::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&s.q_ready);
            // while the first products run: does a column have a loss, and past which K scale does it show?
            if (brings && __any_sync(0xffffffffu, maybe)) {
                const float loss = row_loss<D>(wq), factor = fabsf(a.c.sm_scale * kLog2e);
                if (sub == 0 && loss != 0.f) {
                    // (not negative, so it orders like its bits)
                    const float limit = loss < 0.f ? 0.f : kScoreLoss / (448.f * (loss * factor));
                    s.col_limit[cq] = limit;
                    atomicMin(reinterpret_cast<uint32_t *>(&s.k_limit[k & 1][grp]), __float_as_uint(limit));
                    if (loss < 0.f) {
                        s.col_down[cq] = -kUnit;
                        s.col_coef[cq] = a.c.sm_scale * kLog2e * kUnit;
                    }
                }
            }
            ok = gdn::mbar_wait_bounded(&s.q_ready, k & 1, a.wait_ns);
            group_sync(grp);
            float k_limit = s.k_limit[k & 1][grp];
            if (pos_in == 0) s.k_limit[(k + 1) & 1][grp] = INFINITY;

            const int nc = g.nc, nt = nc + g.fresh;
            // a row sees positions from lo0 + row * lo1 on (g.lo is row 0's, and not negative)
            const int lo0 = a.c.window ? g.len + (a.k ? 1 : 0) - a.c.window : 0, lo1 = a.c.window && a.k ? 1 : 0;
            const int lo_last = lo0 + lo1 * s.col_row[g.cols - 1], lo_request = lo0 + lo1 * (g.n - 1);
            // [16][RB], the new rows' weights, where the next tile's would go
            float *fresh_p = reinterpret_cast<float *>(s_p + ((gp + nc) & 1) * C::kP);
            f2 l[N / 2];
            float z[N];
#pragma unroll
            for (int c = 0; c < N / 2; ++c) l[c] = 0;
            float vref = pow2i(kMinScaleExp), vinv = kBase / vref;  // the largest V scale so far
            float eref = kMinScaleExp, sunk = 0.f;  // its exponent; how far references have followed it down

            // what goes with tile i's scores is there: its pages' scales, or the new keys'
            const auto tile_known = [&](int i) {
                const int y = gp + i;
                return i >= nc ? gdn::mbar_wait_bounded(&s.fk_ready, fresh_seen & 1, a.wait_ns)
                               : gdn::mbar_wait_bounded(&s.sc_full[y % C::kScales], (y / C::kScales) & 1, a.wait_ns);
            };
            // Tile by tile.  From the first tile on where a loss might show, which a vote finds, the loop is left
            // before each, its scores are put right and it goes on.  (In the loop that code, taken or not, called
            // or not, made 16 rows x 32 requests 133 to 136 us, in a second form of the loop 128 to 131, beside it
            // 121.5 to 123.)
            for (int i = 0, stop = nt, fixed = -1;;) {
                for (; i < stop; ++i) {
                    const bool is_fresh = i >= nc;
                    const int x = gs + i, y = gp + i, t = (g.tile0 + i) * kTile + pos_in;
                    if (ok) ok = tile_known(i);
                    if (is_fresh && fixed != i && __any_sync(0xffffffffu, ok && s.fresh_lossy)) break;
                    const float2 sc =
                        is_fresh
                            ? make_float2(fabsf(pos_in < 32 && (pos_in & 15) < g.n ? s.fresh_k[pos_in & 15] : 0.f), 0.f)
                            : s.scales[y % C::kScales][pos_in >> shift];
                    // (the elements of a new key are below 256 times its factor, of a cached one 448 times its scale)
                    const bool look = sc.x > k_limit;
                    // whole: every row sees every position of the tile
                    const int tile = g.tile0 + i;
                    const bool whole = !is_fresh && (tile + 1) * kTile <= g.len && tile * kTile >= lo_last;
                    // While some row of the request may not have seen a position (a segment's first
                    // tile, and those that its window begins in or past) every column's reference
                    // follows its largest weight, and z holds the scores as they are; from then on z is
                    // against the reference.  Both go by the request alone.
                    const bool first = i == 0 || lo_request >= (is_fresh ? g.len : (g.tile0 + i) * kTile);
                    if (ok) ok = gdn::mbar_wait_bounded(&s.s_full[x & 1], (x >> 1) & 1, a.wait_ns);
                    tc::fence_after();
                    {
                        uint32_t hi[N], lo[N];
                        const uint32_t at = tm + lane_base + (x & 1) * C::kNs + col0;
                        if constexpr (N == 16) {
                            tc::ld16_async(at, hi);
                            tc::ld16_async(at + RB, lo);
                        } else {
                            tc::ld8_async(at, hi);
                            tc::ld8_async(at + RB, lo);
                        }
                        tc::ld_wait();
                        tc::ld_fence_regs(hi);
                        tc::ld_fence_regs(lo);
                        f2 v[N / 2];
                        const f2 part = pair(1.f / 32.f, 1.f / 32.f);
#pragma unroll
                        for (int c = 0; c < N / 2; ++c)
                            v[c] = fma2(pair(lo[2 * c], lo[2 * c + 1]), part, pair(hi[2 * c], hi[2 * c + 1]));
                        if (is_fresh) {  // the other part of the position
#pragma unroll
                            for (int c = 0; c < N / 2; ++c) {
                                const float2 b = both(v[c]);
                                const f2 other =
                                    pair(__shfl_xor_sync(0xffffffffu, b.x, 16), __shfl_xor_sync(0xffffffffu, b.y, 16));
                                v[c] = pos_in & 16 ? fma2(v[c], part, other) : fma2(other, part, v[c]);
                            }
                        }
                        const f2 sx = pair(sc.x, sc.x);
#pragma unroll
                        for (int c = 0; c < N; c += 4) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(s.col_coef + col0 + c);
                            ulonglong2 nm = make_ulonglong2(0, 0);
                            if (!first) nm = *reinterpret_cast<const ulonglong2 *>(s.col_nm + col0 + c);
                            const float2 b0 = both(fma2(v[c / 2], mul2(sx, f.x), nm.x)),
                                         b1 = both(fma2(v[c / 2 + 1], mul2(sx, f.y), nm.y));
                            z[c] = b0.x;
                            z[c + 1] = b0.y;
                            z[c + 2] = b1.x;
                            z[c + 3] = b1.y;
                        }
                        if (is_fresh) {
                            const int j = pos_in & 15, w = a.c.window;
#pragma unroll
                            for (int c = 0; c < N; ++c) {
                                const int row = s.col_row[col0 + c];
                                const bool see = pos_in < 32 && j < g.n && j <= row && (!w || j > row - w);
                                z[c] = see ? z[c] : -INFINITY;
                            }
                        } else if (!whole) {
#pragma unroll
                            for (int c = 0; c < N; ++c)
                                z[c] = t < g.len && t >= lo0 + lo1 * s.col_row[col0 + c] ? z[c] : -INFINITY;
                        }
                    }
                    bool move = first;
                    if (!first) {
                        float top[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
                        for (int c = 4; c < N; ++c) top[c & 3] = fmaxf(top[c & 3], z[c]);
                        const float over = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                        move = group_or(grp, over > kSlack || sc.y > vref || look || !ok);
                    }
                    if (__builtin_expect(move, 0)) {
                        // ---- the reference moves (or the scores are to be put right, or a wait ran out)
                        if (group_or(grp, look || !ok)) {
                            k_limit = INFINITY;  // the tiles from here on are looked at one by one
                            if (group_or(grp, !ok)) {
                                ok = false;
                                i = nt;
                            }
                            break;
                        }
                        const uint32_t vm = __reduce_max_sync(0xffffffffu, __float_as_uint(sc.y));
                        if (lane == 0) s.v_max[grp][warp & 3] = __uint_as_float(vm);
                        group_sync(grp);
                        const float vnow = fmaxf(fmaxf(fmaxf(s.v_max[grp][0], s.v_max[grp][1]),
                                                       fmaxf(s.v_max[grp][2], s.v_max[grp][3])), vref);
                        // a reference is to a weight times its V scale (in powers of two, against the largest: 0
                        // or less, so a vote by the weight alone misses none), and follows the largest scale down
                        const float enow = vnow > vref ? exponent_of(vnow) : eref;
                        const float lift = is_fresh ? 0.f : fmaxf(exponent_of(sc.y) - enow, -kLift);
                        const float drop = i > 0 ? fminf(enow - eref, kLift - sunk) : 0.f;
#pragma unroll
                        for (int c = 0; c < N; ++c) {
                            const float top = warp_max(z[c] + lift);
                            if (lane == 0) s.col_max[warp & 3][col0 + c] = top;
                        }
                        group_sync(grp);
                        if (pos_in < N) {
                            const int c = col0 + pos_in;
                            const float was = -s.col_nm[c];
                            const float top = fmaxf(fmaxf(s.col_max[0][c], s.col_max[1][c]),
                                                    fmaxf(s.col_max[2][c], s.col_max[3][c]));
                            // columns within the slack stay, or a column's bits would go by its neighbours
                            const float now = first                  ? fmaxf(top, was - drop)
                                              : top + drop > kSlack ? was + top
                                                                    : was - drop;
                            s.col_nm[c] = -now;
                            s.col_fac[c] = ex2(was - now);
                            s.col_l[c] = first ? -now : was - now;
                        }
                        const float vfac = vref / vnow;
                        vref = vnow;
                        vinv = kBase / vnow;
                        eref = enow;
                        sunk += drop;
                        group_sync(grp);
#pragma unroll
                        for (int c = 0; c < N; c += 2) {
                            l[c / 2] = mul2(l[c / 2], *reinterpret_cast<const f2 *>(s.col_fac + col0 + c));
                            z[c] += s.col_l[col0 + c];
                            z[c + 1] += s.col_l[col0 + c + 1];
                        }
                        if (i > 0) {
                            ok = gdn::mbar_wait_bounded(&s.pv_done[(y - 1) & 1], ((y - 1) >> 1) & 1, a.wait_ns);
                            if (group_or(grp, !ok)) {
                                ok = false;
                                i = nt;
                                break;
                            }
                            tc::fence_after();
#pragma unroll 1
                            for (int e = 0; e < C::kAtoms * 4 * N; e += 8) {  // this group's columns of every part
                                const int at = e / N * RB + col0 + e % N;
                                uint32_t w[8];
                                tc::ld8_async(tm_o + lane_base + at, w);
                                tc::ld_wait();
                                tc::ld_fence_regs(w);
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    w[c] = __float_as_uint(__uint_as_float(w[c]) * (s.col_fac[at % RB + c] * vfac));
                                tc::st8(tm_o + lane_base + at, w);
                            }
                            tc::st_wait();
                        }
                    }
                    // scores are read: their buffer is free
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(&s.s_free[x & 1]);

                    if (is_fresh) {
                        if (ok && y >= 2) ok = gdn::mbar_wait_bounded(&s.pv_done[y & 1], ((y >> 1) - 1) & 1, a.wait_ns);
                        if (pos_in < 16 && ok) {
#pragma unroll
                            for (int c = 0; c < N; c += 2) {
                                const f2 p = pair(ex2(z[c]), ex2(z[c + 1]));
                                l[c / 2] = add2(l[c / 2], p);
                                *reinterpret_cast<f2 *>(fresh_p + pos_in * RB + col0 + c) = p;
                            }
                        }
                        i = nt;  // the last tile
                        break;
                    }
                    const float xw = sc.y * vinv;
                    const f2 xw2 = pair(xw, xw);
                    if (ok && y >= 2) ok = gdn::mbar_wait_bounded(&s.pv_done[y & 1], ((y >> 1) - 1) & 1, a.wait_ns);
                    uint8_t *pb = s_p + (y & 1) * C::kP;
                    uint32_t e[4][N / 2];  // the parts, in the upper bytes
#pragma unroll
                    for (int c = 0; c < N / 2; ++c) {
                        const f2 p = pair(ex2(z[2 * c]), ex2(z[2 * c + 1]));
                        l[c] = add2(l[c], p);
                        const float2 v = both(mul2(p, xw2));
                        e[0][c] = f16x2(v.x, v.y);
                        e[1][c] = rest8(e[0][c]);
                        e[2][c] = rest8(e[1][c]);
                        e[3][c] = rest8(e[2][c]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int b = j * RB + col0;  // byte of the row
                        uint8_t *dst = pb + (b / C::kPRow) * kTile * C::kPRow +
                                       tc::swz8_off<C::kPRow>(pos_in, (b % C::kPRow) >> 4) + (b & 8);
                        const uint32_t w0 = upper4(e[j][0], e[j][1]), w1 = upper4(e[j][2], e[j][3]);
                        if constexpr (N == 16)
                            *reinterpret_cast<uint4 *>(dst) =
                                make_uint4(w0, w1, upper4(e[j][4], e[j][5]), upper4(e[j][6], e[j][7]));
                        else
                            *reinterpret_cast<uint2 *>(dst) = make_uint2(w0, w1);
                    }
                    if (!whole && grp == 0) {
                        // What no row sees may hold anything, NaN codes too, and 0 * NaN is
                        // NaN: its values become zero.  Positions only some rows see keep
                        // their values but for NaN, which the epilogue gives to those rows.
                        const int pos = ring + v_pos(i, nc), slot = pos % C::kSlots;
                        if (ok) ok = gdn::mbar_wait_bounded(&s.full[slot], (pos / C::kSlots) & 1, a.wait_ns);
                        const bool none = t < g.lo || t >= g.len, some = !none && t < lo_last;
                        if (ok && (none || some)) {
#pragma unroll 2
                            for (int e = 0; e < C::kAtoms * C::kRow / 16; ++e) {
                                uint4 *p = reinterpret_cast<uint4 *>(
                                    s_ring + slot * C::kSlot + e / (C::kRow / 16) * kTile * C::kRow +
                                    tc::swz8_off<C::kRow>(pos_in, e % (C::kRow / 16)));
                                uint4 w = make_uint4(0, 0, 0, 0);
                                if (some) {
                                    w = *p;
                                    uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                                    for (int b = 0; b < 4; ++b) u[b] &= ~__vcmpeq4(u[b] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                }
                                *p = w;
                            }
                        }
                    }
                    gdn::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(&s.p_full[y & 1]);
                }
                if (i >= nt) break;
                const int x = gs + i;
                if (ok) ok = tile_known(i);
                if (ok) ok = gdn::mbar_wait_bounded(&s.s_full[x & 1], (x >> 1) & 1, a.wait_ns);
                __syncwarp();
                tc::fence_after();
                const int t = i >= nc ? -1 : (g.tile0 + i) * kTile + pos_in;
                uint32_t mask = 0;
                if (t >= 0 ? t >= g.lo && t < g.len : pos_in < 32 && (pos_in & 15) < g.n)
                    mask = lossy_columns<D, RB>(s, t >= 0 ? -1 : pos_in & 15,
                                                s.scales[(gp + i) % C::kScales][pos_in >> shift].x, col0, g.cols);
                if (__any_sync(0xffffffffu, mask))
                    exact_scores<D, RB>(a, s, s.seg[k % kQueue], t, mask, pos_in, col0,
                                        tm + lane_base + (x & 1) * C::kNs + col0);
                fixed = i;
                stop = i + 1;
            }
            // ---- the segment's end
            if (ok && nc > 0) {
                const int y = gp + nc - 1;
                ok = gdn::mbar_wait_bounded(&s.pv_done[y & 1], (y >> 1) & 1, a.wait_ns);
            }
            if (ok && g.fresh) ok = gdn::mbar_wait_bounded(&s.fv_full, fresh_seen & 1, a.wait_ns);
            if (group_or(grp, !ok)) {
                ok = false;
                break;
            }
            tc::fence_after();
            const bool bad = *reinterpret_cast<volatile int *>(&s.bad[k % kQueue]) != 0;
            if (bad && pos_in == 0) gdn::set_status(a.status, GDN_DEV_PAGE_OOR);
            // the next segment's queries, on their way while this one is written
            ok = gdn::mbar_wait_bounded(&s.seg_full[(k + 1) % kQueue], ((k + 1) / kQueue) & 1, a.wait_ns);
            if (group_or(grp, !ok)) {
                ok = false;
                break;
            }
            const Segment h = g;
            g = s.seg[(k + 1) % kQueue];
            load_q();
            // sums over the 128 positions
            float sums[N];
#pragma unroll
            for (int c = 0; c < N / 2; ++c) {
                sums[2 * c] = both(l[c]).x;
                sums[2 * c + 1] = both(l[c]).y;
            }
            warp_sums<N>(sums, lane);
            if ((lane & (32 / N - 1)) == 0) s.col_max[warp & 3][col0 + lane / (32 / N)] = sums[0];
            group_sync(grp);
            if (pos_in < N) {
                const int c = col0 + pos_in;
                const float sum = (s.col_max[0][c] + s.col_max[1][c]) + (s.col_max[2][c] + s.col_max[3][c]);
                if (h.out >= 0) {
                    a.ws_ml[int64_t(h.out) * RB + c] = make_float2(-s.col_nm[c], bad ? -1.f : sum);
                } else if (a.lse && c < h.cols && !bad) {
                    a.lse[(int64_t(h.t0) + s.col_row[c]) * a.c.h_q + h.hk * a.group + s.col_head[c]] =
                        sum == 0.f ? -INFINITY : (log2f(sum) - s.col_nm[c]) * 0.6931471805599453f;
                }
                s.col_l[c] = sum == 0.f ? 0.f : 1.f / sum;
            }
            group_sync(grp);
            if (!bad) {
                const float back = vref / kBase;
                uint16_t *o_base = a.o + int64_t(h.t0) * a.o_stride;
                float *ws_base = a.ws_o + int64_t(h.out) * RB * D;
                const int edge = min(min(lo_last, h.len), (h.tile0 + nc) * kTile);
#pragma unroll 1
                for (int at = 0; at < C::kAtoms && col0 < h.cols; ++at) {
                    const int e = at * C::kRow + pos_in;  // this thread's element (d = 64: lanes past 63 hold none)
                    f2 acc[N / 2];
#pragma unroll
                    for (int c = 0; c < N / 2; ++c) acc[c] = 0;
                    if (nc > 0) {
                        const f2 part = pair(1.f / 8.f, 1.f / 8.f);
#pragma unroll
                        for (int j = 3; j >= 0; j -= 2) {  // from the last part on
                            uint32_t u[N], v[N];
                            const uint32_t from = tm_o + lane_base + at * C::kNp + col0;
                            if constexpr (N == 16) {
                                tc::ld16_async(from + j * RB, u);
                                tc::ld16_async(from + (j - 1) * RB, v);
                            } else {
                                tc::ld8_async(from + j * RB, u);
                                tc::ld8_async(from + (j - 1) * RB, v);
                            }
                            tc::ld_wait();
                            tc::ld_fence_regs(u);
                            tc::ld_fence_regs(v);
#pragma unroll
                            for (int c = 0; c < N / 2; ++c) {
                                acc[c] = fma2(acc[c], part, pair(u[2 * c], u[2 * c + 1]));
                                acc[c] = fma2(acc[c], part, pair(v[2 * c], v[2 * c + 1]));
                            }
                        }
                        const f2 b2 = pair(back, back);
#pragma unroll
                        for (int c = 0; c < N / 2; ++c) acc[c] = mul2(acc[c], b2);
                    }
                    if (e >= D) continue;
                    uint32_t odd = 0;  // new rows whose value here is not finite
                    if (h.fresh)
#pragma unroll 1
                        for (int j = 0; j < h.n; ++j) {
                            const uint32_t b = uint32_t(reinterpret_cast<const uint16_t *>(s_fv)[j * D + e]) << 16;
                            const bool finite = (b & 0x7f800000u) != 0x7f800000u;
                            if (!finite) odd |= 1u << j;
                            const f2 v = pair(finite ? b : 0u, finite ? b : 0u);
                            const ulonglong2 *p = reinterpret_cast<const ulonglong2 *>(fresh_p + j * RB + col0);
#pragma unroll
                            for (int c = 0; c < N / 4; ++c) {
                                const ulonglong2 w = p[c];
                                acc[2 * c] = fma2(w.x, v, acc[2 * c]);
                                acc[2 * c + 1] = fma2(w.y, v, acc[2 * c + 1]);
                            }
                        }
                    float o[N];
#pragma unroll
                    for (int c = 0; c < N / 2; ++c) {
                        o[2 * c] = both(acc[c]).x;
                        o[2 * c + 1] = both(acc[c]).y;
                    }
                    if (odd) {  // such a value reaches the rows that see it, and no others
                        const int w = a.c.window ? a.c.window : GDN_MAX_ROWS;
#pragma unroll 1
                        for (int j = 0; j < h.n; ++j)
                            if (odd >> j & 1) {
                                const float v = gdn::bf16_to_f32(reinterpret_cast<const uint16_t *>(s_fv)[j * D + e]);
#pragma unroll
                                for (int c = 0; c < N; ++c)
                                    if (uint32_t(s.col_row[col0 + c] - j) < uint32_t(w))
                                        o[c] = fmaf(fresh_p[j * RB + col0 + c], v, o[c]);
                            }
                    }
                    // NaN of positions that only some rows see
#pragma unroll 1
                    for (int t = max(h.lo, h.tile0 * kTile); t < edge; ++t) {
                        const int page = a.table[int64_t(h.r) * a.table_stride + (t >> shift)];
                        const uint8_t code =
                            a.c.kv[int64_t(page) * a.c.page_stride + int64_t(a.layer) * a.c.layer_stride +
                                   (int64_t(a.c.h_kv + h.hk) * T + (t & (T - 1))) * D + e];
                        if ((code & 0x7f) == 0x7f) {
#pragma unroll
                            for (int c = 0; c < N; ++c)
                                if (t >= lo0 + lo1 * s.col_row[col0 + c]) o[c] = __uint_as_float(0x7fc00000u);
                        }
                    }
                    if (h.out < 0) {
#pragma unroll
                        for (int c = 0; c < N; ++c)
                            if (col0 + c < h.cols)
                                o_base[s.col_out[col0 + c] + e] = gdn::f32_to_bf16(o[c] * s.col_l[col0 + c]);
                    } else {
#pragma unroll
                        for (int c = 0; c < N; ++c)
                            if (col0 + c < h.cols) ws_base[(col0 + c) * D + e] = o[c];
                    }
                }
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                arrive(&s.seg_empty[k % kQueue]);
                arrive(&s.epi_done);
            }
            gs += nt;
            gp += nc;
            ring += 2 * nc;
            fresh_seen += h.fresh;
            // the other groups are done with the columns' numbers too
            ok = gdn::mbar_wait_bounded(&s.epi_done, k & 1, a.wait_ns);
            if (group_or(grp, !ok)) {
                ok = false;
                break;
            }
        }
        if (!ok) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
        tc::fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tm, C::kTmem);
    }
}

// Joins a unit's pieces: o = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s, in one pass
// with a running M.  Groups of d/4 threads.  With few pieces a group joins a column
// by itself; with many the groups share one column's pieces, so that their loads are
// in flight together.  Which of the two, and so the order of the sums, goes by the
// pieces alone.  It is latency: 2 to 5 us behind the attention, whose end hides part
// of its launch.  Free cuts: a CTA for each part, the parts of a unit sharing its
// columns.  Given cuts: a CTA for each `per_cta` columns of a unit.  Few are kFew: with 4,
// 8 and 16 one request of 2 heads of 256, 4 rows, 3000 tokens takes 14.6, 14.5 and 16.1 us,
// 4 of 8 heads of 128, 2000..8000 tokens 22.9, 20.1 and 20.7, but one of 16 rows, 4 heads of
// 128, 4000 tokens 25.4, 25.2 and 21.6.
constexpr int kJoin = 512, kFew = 8;

template <int D>
__global__ void __launch_bounds__(kJoin) kv8_join_kernel(const __grid_constant__ AttendArgs a, const int RB,
                                                         const int per_cta) {
    gdn::pdl_enter();
    constexpr int W = D / 4, G = kJoin / W;
    const int tid = threadIdx.x;
    int t0, hk, blk, begin, end, by, count;
    int64_t first, base, step;  // pieces in the workspace: the first, then base + s * step
    // the partial sums of a call in which a wait ran out are not to be trusted
    const uint32_t status = a.status ? *reinterpret_cast<volatile uint32_t *>(a.status) : 0;
    if (a.pinned) {
        const Request rq = request_of(a, rows_of(a, blockIdx.z));
        hk = blockIdx.y / a.blocks;
        blk = blockIdx.y - hk * a.blocks;
        count = rq.bad ? 0 : (rq.tiles + a.piece_tiles - 1) / a.piece_tiles;
        t0 = rq.t0;
        first = base = int64_t(blockIdx.z) * a.max_pieces * gridDim.y + blockIdx.y;
        step = gridDim.y;
        begin = blockIdx.x * per_cta;
        end = min(begin + per_cta, min(RB, rq.n * a.group - blk * RB));
        by = 1;
    } else {
        const Part p = a.parts[2 * blockIdx.y + blockIdx.x];
        hk = p.hk;
        blk = p.blk;
        count = p.count;
        t0 = p.t0;
        first = 2 * p.owner + 1;
        base = 2 * p.owner;
        step = 2;
        begin = int(blockIdx.y) - p.owner;
        end = p.cols;
        by = count;
    }
    if (count <= 1 || (status & GDN_DEV_TIMEOUT)) return;
    __shared__ float2 s_ml[G];
    __shared__ float4 s_o[G][W];
    const int g = tid / W, e = tid % W;
    const bool few = count <= kFew;
    for (int c = begin + (few ? g * by : 0); c < end; c += few ? G * by : by) {
        float m = kUnset, l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        bool skip = false;
        auto add = [&](float2 x, const float4 &o) {
            if (x.y == 0.f) return;  // the row sees nothing of the piece
            const float now = fmaxf(m, x.x), f = ex2(m - now), w = ex2(x.x - now);
            m = now;
            l = fmaf(l, f, x.y * w);
            acc.x = fmaf(acc.x, f, o.x * w);
            acc.y = fmaf(acc.y, f, o.y * w);
            acc.z = fmaf(acc.z, f, o.z * w);
            acc.w = fmaf(acc.w, f, o.w * w);
        };
#pragma unroll 4
        for (int s = few ? 0 : g; s < count; s += few ? 1 : G) {
            const int64_t at = (s == 0 ? first : base + s * step) * RB + c;
            const float2 x = a.ws_ml[at];
            const float4 o = __ldcs(reinterpret_cast<const float4 *>(a.ws_o + at * D) + e);
            skip |= x.y < 0.f;  // the piece was refused
            add(x, o);
        }
        if (!few) {
            __syncthreads();  // the last column's sums are read
            s_o[g][e] = acc;
            if (e == 0) s_ml[g] = make_float2(m, l);
            skip = __syncthreads_or(skip);
            if (skip) return;
            if (g > 0) continue;
            for (int k = 1; k < G; ++k) add(s_ml[k], s_o[k][e]);
        }
        if (skip) return;
        const int x = blk * RB + c, row = x / a.group, h = hk * a.group + x - row * a.group;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint2 w;
        w.x = gdn::f32_to_bf16(acc.x * inv) | (uint32_t(gdn::f32_to_bf16(acc.y * inv)) << 16);
        w.y = gdn::f32_to_bf16(acc.z * inv) | (uint32_t(gdn::f32_to_bf16(acc.w * inv)) << 16);
        *reinterpret_cast<uint2 *>(a.o + (int64_t(t0) + row) * a.o_stride + int64_t(h) * D + e * 4) = w;
        if (e == 0 && a.lse)
            a.lse[(int64_t(t0) + row) * a.c.h_q + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

// A layer's pages as [page][2 h_kv page_tokens rows][d] bytes; boxes of one
// page and head, rows of at most 128 bytes, swizzled to that width.
bool encode_pages(CUtensorMap *m, const kv8_cache *c, int layer) {
    const gdn_host::EncodeTiledFn fn = gdn_host::encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cuuint64_t(c->d), cuuint64_t(2) * c->h_kv * c->page_tokens, cuuint64_t(c->num_pages)};
    const cuuint64_t strides[2] = {cuuint64_t(c->d), cuuint64_t(c->page_stride)};
    const cuuint32_t box[3] = {cuuint32_t(c->d < 128 ? c->d : 128), cuuint32_t(c->page_tokens), 1};
    const cuuint32_t elem[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c->kv + int64_t(layer) * c->layer_stride, dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, c->d < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
    int rb, blocks, pinned, piece_tiles, max_pieces, ctas;
    int64_t parts;  // of the workspace
};

Plan plan_of(const kv8_cache *c, int32_t B, int32_t max_len, int32_t max_rows, int32_t split_tokens) {
    Plan p{};
    const int64_t cols = int64_t(max_rows) * (c->h_q / c->h_kv);
    // positions a request's rows can see, and the tiles they may lie in
    int64_t seen = max_len;
    if (c->window && c->window < seen) seen = int64_t(c->window) + kTile;
    int64_t tiles = (seen + kTile - 1) / kTile;
    if (tiles < 1) tiles = 1;
    const auto slots_of = [&](int rb) { return int64_t(kSms) * (c->d == 256 || rb == 64 ? 1 : 2); };
    const auto units_of = [&](int rb) { return int64_t(B) * c->h_kv * ((cols + rb - 1) / rb); };
    // the narrowest block that holds a request's columns: the work a tile costs goes by its
    // width (1 row x 256 requests, 4 columns: 63 us in 8, 80 in 16, 104 in 32), and a wider
    // one reads the cache less often (16 rows, 128 columns: 131 us by 32, 121 by 64) ...
    const int widest = cols <= 8 ? 8 : cols <= 16 ? 16 : cols <= 32 || c->d == 256 ? 32 : 64;
    // ... or narrower ones, where every one of them can have its CTA and there are few tiles
    // an SM: then they share tiles that are in L2, and a unit's ends are shorter (32 columns of
    // 256, one request of 2 heads: 422 tokens 15.0 us in 32, 11.7 in 8, 8000 tokens 17.5 and
    // 15.9; 512 units of 1 tile 42 in 32, 52 in 16)
    p.rb = 8;
    while (p.rb < widest && (units_of(p.rb) > slots_of(p.rb) || units_of(p.rb) * tiles > 4 * kSms)) p.rb *= 2;
    p.blocks = int((cols + p.rb - 1) / p.rb);
    const int64_t units = units_of(p.rb), slots = slots_of(p.rb);
    int64_t ctas;
    const bool whole = tiles <= 2 * kLeast ||
                       (tiles <= kWhole && units <= slots && tiles * slots <= 2 * kWhole * units);
    if (split_tokens > 0 || whole) {
        const int64_t t = split_tokens > 0 ? (int64_t(split_tokens) + kTile - 1) / kTile : tiles;
        p.pinned = 1;
        p.piece_tiles = int(t < tiles ? t : tiles);
        p.max_pieces = int((tiles + p.piece_tiles - 1) / p.piece_tiles);
        ctas = units * p.max_pieces;
        p.parts = p.max_pieces > 1 ? ctas : 0;
    } else {
        p.piece_tiles = p.max_pieces = 1;
        ctas = ranges_of(units * (tiles + unit_cost(p.rb)));
    }
    p.ctas = int(ctas < slots ? ctas : slots);
    if (!p.pinned) p.parts = p.ctas > 1 ? 2 * int64_t(p.ctas) : 0;
    return p;
}

template <int D, int RB>
int launch(const AttendArgs &a, int ctas, cudaStream_t st) {
    using C = Cfg<D, RB>;
    // for every launch: the limit is the current device's
    if (cudaFuncSetAttribute(kv8_attend_kernel<D, RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
        cudaSuccess)
        return GDN_ERR_CUDA;
    return gdn_host::launch_pdl(kv8_attend_kernel<D, RB>, dim3(unsigned(ctas)), dim3(C::kThreads), C::kSmem, st, a);
}

}  // namespace

static size_t ws_bytes(const kv8_cache *c, const Plan &p) {
    return size_t(p.parts) * p.rb * (size_t(c->d) * 4 + 8) + (p.pinned ? 0 : size_t(p.parts) * sizeof(Part));
}

extern "C" size_t kv8_attend_workspace_bytes(const kv8_cache *cache, int32_t B, int32_t max_len, int32_t max_rows,
                                             int32_t split_tokens) {
    if (gdn_host::kv8_check(cache) != GDN_OK || B <= 0 || max_len < 0 || max_len > gdn_host::kKv8MaxLen ||
        max_rows <= 0 || max_rows > GDN_MAX_ROWS || split_tokens < 0)
        return 0;
    return ws_bytes(cache, plan_of(cache, B, max_len, max_rows, split_tokens));
}

static int attend(const kv8_cache *cache, int32_t layer, int32_t B, int32_t row_capacity, const int32_t *cu_rows,
                  const int32_t *cache_len, const int32_t *table, int32_t table_pages, int64_t table_stride,
                  const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k_new, int64_t k_stride,
                  const gdn_bf16 *v_new, int64_t v_stride, gdn_bf16 *o, int64_t o_stride, float *lse,
                  int32_t max_len, int32_t max_rows, int32_t split_tokens, void *workspace, size_t workspace_bytes,
                  uint32_t *dev_status, uint64_t wait_ns, int32_t withhold, void *stream) {
    const int bad = gdn_host::kv8_check(cache);
    if (bad != GDN_OK) return bad;
    if (layer < 0 || layer >= cache->num_layers || B < 0 || B > 65535 || row_capacity < 0 || table_pages < 0 ||
        table_stride < 0 ||
        max_len < 0 || max_len > gdn_host::kKv8MaxLen || max_rows < 0 || max_rows > GDN_MAX_ROWS || split_tokens < 0)
        return GDN_ERR_ARG;
    if (B == 0 || max_rows == 0) return GDN_OK;
    // (an empty tensor's address is null: with no rows nothing of theirs is read)
    if (!cu_rows || !cache_len || (!table && table_pages > 0) || (row_capacity > 0 && (!q || !o)) || !k_new != !v_new)
        return GDN_ERR_NULL;
    if (!gdn_host::kv8_rows_ok(q, q_stride, cache->h_q, cache->d) ||
        !gdn_host::kv8_rows_ok(o, o_stride, cache->h_q, cache->d))
        return GDN_ERR_ARG;
    if (o_stride > (1 << 26)) return GDN_ERR_ARG;  // a request's outputs are indexed with 32 bits
    if (k_new && (!gdn_host::kv8_rows_ok(k_new, k_stride, cache->h_kv, cache->d) ||
                  !gdn_host::kv8_rows_ok(v_new, v_stride, cache->h_kv, cache->d)))
        return GDN_ERR_ARG;
    const Plan p = plan_of(cache, B, max_len, max_rows, split_tokens);
    const size_t need = ws_bytes(cache, p);
    if (p.parts > (int64_t(1) << 30)) return GDN_ERR_ARG;
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (need && !gdn_host::aligned16(workspace)) return GDN_ERR_ARG;
    if (int64_t(cache->h_kv) * p.blocks > 65535) return GDN_ERR_ARG;
    AttendArgs a{};
    if (!encode_pages(&a.map, cache, layer)) return GDN_ERR_CUDA;
    a.c = *cache;
    a.layer = layer;
    a.B = B;
    a.row_capacity = row_capacity;
    a.table_pages = table_pages;
    a.table_stride = table_stride;
    a.max_len = max_len;
    a.max_rows = max_rows;
    a.group = cache->h_q / cache->h_kv;
    a.blocks = p.blocks;
    a.pinned = p.pinned;
    a.piece_tiles = p.piece_tiles;
    a.max_pieces = p.max_pieces;
    a.page_shift = 31 - __builtin_clz(unsigned(cache->page_tokens));
    a.cu_rows = cu_rows;
    a.cache_len = cache_len;
    a.table = table;
    a.q = q;
    a.k = k_new;
    a.v = v_new;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.o_stride = o_stride;
    a.o = o;
    a.lse = lse;
    if (p.parts) {
        const size_t columns = size_t(p.parts) * p.rb;
        a.ws_o = static_cast<float *>(workspace);
        a.ws_ml = reinterpret_cast<float2 *>(a.ws_o + columns * cache->d);
        if (!p.pinned) a.parts = reinterpret_cast<Part *>(a.ws_ml + columns);
    }
    a.status = dev_status;
    a.wait_ns = wait_ns;
    a.withhold = withhold;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc = GDN_ERR_SHAPE;
    const int key = cache->d * 100 + p.rb;
    switch (key) {
        case 6408: rc = launch<64, 8>(a, p.ctas, st); break;
        case 6416: rc = launch<64, 16>(a, p.ctas, st); break;
        case 6432: rc = launch<64, 32>(a, p.ctas, st); break;
        case 6464: rc = launch<64, 64>(a, p.ctas, st); break;
        case 12808: rc = launch<128, 8>(a, p.ctas, st); break;
        case 12816: rc = launch<128, 16>(a, p.ctas, st); break;
        case 12832: rc = launch<128, 32>(a, p.ctas, st); break;
        case 12864: rc = launch<128, 64>(a, p.ctas, st); break;
        case 25608: rc = launch<256, 8>(a, p.ctas, st); break;
        case 25616: rc = launch<256, 16>(a, p.ctas, st); break;
        case 25632: rc = launch<256, 32>(a, p.ctas, st); break;
        default: break;
    }
    if (rc != GDN_OK || !p.parts) return rc;
    dim3 grid(2, unsigned(p.ctas));
    int per = 1;
    if (p.pinned) {
        // as many columns a CTA as still leave four CTAs for each SM
        const int64_t units = int64_t(B) * cache->h_kv * p.blocks, each = units * p.rb / (4 * kSms);
        per = int(each < 1 ? 1 : each > p.rb ? p.rb : each);
        grid = dim3(unsigned((p.rb + per - 1) / per), unsigned(cache->h_kv * p.blocks), unsigned(B));
    }
    if (cache->d == 64) return gdn_host::launch_pdl(kv8_join_kernel<64>, grid, dim3(kJoin), 0, st, a, p.rb, per);
    if (cache->d == 128) return gdn_host::launch_pdl(kv8_join_kernel<128>, grid, dim3(kJoin), 0, st, a, p.rb, per);
    return gdn_host::launch_pdl(kv8_join_kernel<256>, grid, dim3(kJoin), 0, st, a, p.rb, per);
}

extern "C" int kv8_attend(const kv8_cache *cache, int32_t layer, int32_t B, int32_t row_capacity,
                          const int32_t *cu_rows, const int32_t *cache_len, const int32_t *table,
                          int32_t table_pages, int64_t table_stride, const gdn_bf16 *q, int64_t q_stride,
                          const gdn_bf16 *k_new, int64_t k_stride, const gdn_bf16 *v_new, int64_t v_stride,
                          gdn_bf16 *o, int64_t o_stride, float *lse, int32_t max_len, int32_t max_rows,
                          int32_t split_tokens, void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                          void *stream) {
    return attend(cache, layer, B, row_capacity, cu_rows, cache_len, table, table_pages, table_stride, q, q_stride,
                  k_new, k_stride, v_new, v_stride, o, o_stride, lse, max_len, max_rows, split_tokens, workspace,
                  workspace_bytes, dev_status, gdn::kWaitLimitNs, 0, stream);
}

extern "C" int kv8_selftest_attend_timeout(const kv8_cache *cache, int32_t layer, int32_t B, int32_t row_capacity,
                                           const int32_t *cu_rows, const int32_t *cache_len, const int32_t *table,
                                           int32_t table_pages, int64_t table_stride, const gdn_bf16 *q,
                                           int64_t q_stride, gdn_bf16 *o, int64_t o_stride, int32_t max_len,
                                           int32_t max_rows, int32_t split_tokens, void *workspace,
                                           size_t workspace_bytes, uint32_t *dev_status, uint64_t limit_ns,
                                           void *stream) {
    if (limit_ns == 0 || limit_ns > gdn::kWaitLimitNs) return GDN_ERR_ARG;
    return attend(cache, layer, B, row_capacity, cu_rows, cache_len, table, table_pages, table_stride, q, q_stride,
                  nullptr, 0, nullptr, 0, o, o_stride, nullptr, max_len, max_rows, split_tokens, workspace,
                  workspace_bytes, dev_status, limit_ns, 1, stream);
}
