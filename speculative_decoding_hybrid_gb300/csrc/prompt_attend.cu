// Causal attention of packed rows over dense keys and values (sm_103a): whole
// prompts, and chunks of new rows behind earlier positions of a paged 8-bit cache.
//
// A query tile is 128 rows of the tensor cores: 128 / group positions with all query
// heads of a kv head side by side, so a key is read once for the group.  Per tile of 128
// positions
//   S = Q K^T                 scores, fp32 in tensor memory, a row in a lane
//   p = 2^(c S - m)           a thread a row: its maximum, exponentials and sum in registers
//   O += P V                  P in bf16 from tensor memory
// with m moved (and O rescaled) only when a score passes it by 2^8.  m is a rounded product, which
// c x - m is not: from 2^20 on, where a row's largest weight would not be near 1 for it, the largest
// score is taken off the scores before the scale instead.  At d <= 128 a unit has
// two query tiles that share the keys, so one's softmax runs beside the other's products; at
// d = 256, where one tile's O takes half of tensor memory, the softmax of a tile of positions
// runs beside the products of its neighbours.  P lies where S lay, but for d = 64, which
// leaves it columns of its own: then the next scores need not wait for the products.
//
// Persistent CTAs: one is launched for every unit (request, kv head, rows, part of its
// positions), the first of them on an SM goes on to take over those that have not started
// (try_cancel), when its unit's last tiles are being copied and not before.  Its warps:
//   softmax  a group of four a query tile; at the end the unit's outputs
//   copy     one lane: tiled TMA of queries, and keys and values through one ring
//   product  one lane: waits and issues; the softmax hands it a tile's weights in halves
//   find     takes over units and says what they are, one ahead
//   guard    a zero weight times NaN is NaN: tiles of values that some row does not see
//            all of are looked through, what is not finite is zeroed and, for the rows that
//            do see it, added to the outputs at the end
// A unit's later rows and the longest requests come first.  Long units are cut into parts
// where SMs would idle, whose (m, l, O) prompt_join_kernel joins.  Products with V take the
// steps of 16 positions that some row sees.
//
// A chunk's earlier positions are laid out as bf16 in a workspace first (exactly: 4 bits
// times a power of two): 2 bytes written and read for each stored one, a tenth of the whole
// behind 256K positions.  In the loop the conversion would cost more from about 1,300 query
// vectors a kv head on: shared memory already moves 128 bytes a clock for the products.
//
// Roundings: p to bf16, as V's type wants (both sides of a product have one type), 2^-8 of it at
// most; its sum is of the unrounded ones.  Outputs are 0.0018 to 0.0023 of their size from the
// fp64 form for it, where their own rounding alone, once, to bf16, leaves 0.0016; p in two bf16
// parts would hold 16 bits for half as many products again.  Everything else is fp32.
//
// What bounds it: one prompt of 20,011 tokens, 16/2 heads of 256, 1.98 to 2.0 ms, 1,640 to 1,660
// TFLOP/s, the power limit (a long loop of a library's products reaches 1,736); 8 prompts of 512
// to 12,000 tokens, 32/4 heads of 128, 1.05 ms, 1,390 TFLOP/s: a query tile's chain of scores ->
// tensor-memory load (500 clocks beside products, 60 alone) -> maximum -> exponentials ->
// products, 2,800 clocks a tile for 2,048 of products; short prompts (16 of 100 to 4,000
// tokens, 32/8 heads: 0.45 ms, 1,180 TFLOP/s) the ends of units, 3 us each.  A single short
// prompt is one chain: 37 tokens, 16/2 heads of 256, 9.6 us.
#include "kv8_math.cuh"
#include "prompt.cuh"
#include "tmap.cuh"

namespace {

using namespace kv8;

constexpr int kTile = 128;   // positions a tile, and rows of a query tile
constexpr int kSms = 152;
constexpr float kSlack = 8.f;
constexpr float kFar = 0x1p20f;  // below it c x is off by 2^-5 at most
constexpr int kLeast = 4;    // tiles a part of a cut unit has at least
constexpr int kMostParts = 64;
constexpr double kEnds = 5.0, kPartEnds = 10.0, kJoinCost = 4.0;  // tiles that they cost as much as
constexpr int kAhead = 8;    // tiles of values that the ring holds at most: its slots

struct Info {                // a unit's parts, for the join: parts 0: nothing to join
    int t0, tok0, n, hk, parts, pad[3];
};

struct Args {
    CUtensorMap mq, mk, mv;
    prompt::Requests rq;
    int32_t h_q, h_kv, group, per_tile;  // per_tile: positions a query tile
    int32_t join_rows;       // rows of a CTA of the join
    int32_t window, splits, part_tiles, negate;  // a unit's parts at most, and the tiles that one may have
    float scale_log2;
    int64_t o_stride;
    uint16_t *o;
    float *lse;
    float *ws_o;     // [unit][split][rows][d]
    float2 *ws_ml;
    Info *info;      // [unit]
    const uint16_t *v;  // the values again, for what is not finite in masked places
    int64_t v_head, v_row;
    const int32_t *table;
    int64_t table_stride;
    int32_t page_shift, num_pages;
    uint32_t *status;
    uint64_t wait_ns;
    int32_t withhold;  // self-test: the last values are announced and never copied
};

template <int D>
struct Cfg {
    static constexpr int kStages = D == 256 ? 1 : 2;  // query tiles a CTA
    static constexpr int kPiece = D < 128 ? D : 128;  // channels of a ring slot
    static constexpr int kPieces = D / kPiece;
    static constexpr int kSlot = kTile * kPiece * 2;
    static constexpr int kQTile = kTile * D * 2;
    static constexpr int kRoom = (227 - 3) * 1024 - kStages * kQTile;
    static constexpr int kSlots = kRoom / kSlot > 8 ? 8 : kRoom / kSlot;
    static constexpr int kSmem = kStages * kQTile + kSlots * kSlot + 1024;
    static constexpr int kSoftWarps = 4 * kStages;
    // Columns of outputs at a time: wider loads are fewer (37 tokens, 16/2 heads of 256: 9.6 us with 32, 9.3 with 64), but
    // beside two query tiles' registers they spill (16 prompts 468 -> 545).
    static constexpr int kOut = D == 256 ? 64 : 32;
    // Whether the weights have tensor memory of their own: then the next scores need not wait for the products with them.
    static constexpr bool kApart = D == 64;
    static constexpr int kGuards = kStages == 2 ? 1 : 5;  // warps that look through values
    static constexpr int kThreads = 32 * (kSoftWarps + 3 + kGuards);
    // Registers a thread: of the 168 that 384 threads may have, the softmax's rows take more, the other warps fewer.
    static constexpr int kLaunchRegs = 168, kSoftRegs = kStages == 2 ? 192 : 232, kOtherRegs = kStages == 2 ? 120 : 136;
    static_assert(kThreads == 384 && 32 * kSoftWarps * kSoftRegs + (kThreads - 32 * kSoftWarps) * kOtherRegs <=
                                         kThreads * kLaunchRegs,
                  "more registers than a launch has: the wait for them would not end");
    static_assert(kSlots >= 2 * kPieces + 1 && kSlots <= kAhead, "does not fit an SM");
};

struct Unit {
    int t0, n, len, r, tok0, parts;
    int64_t kv0;  // its first position's row of the keys
};
// What a unit's part sums: tiles tile0 .. of the request's positions, `tiles` of them, of which query tile st uses the
// first ns[st].  Some row of the unit sees positions begin .. end-1, every row sees full .. all-1; tiles before `left` and
// from `right` on are masked: they hold positions that not every row sees.
struct Span {
    int tile0, tiles, ns[2], left, right, begin, end, full, all;
};
struct Work {
    Unit u;
    Span sp;
    int hk, part, x;  // x: the unit's number; -1: no more work
};

constexpr int kQueue = 2;    // units announced: one in work and the next
constexpr int kGroups = 8;   // groups of loads that are freed together, in turn (no more fit the ring)
constexpr int kChunks = 128; // parts of the list of requests whose sums a CTA keeps

template <int D>
struct Shared {
    using C = Cfg<D>;
    uint64_t full[C::kSlots], freed[kGroups], s_full[2], o_done[2], q_full, q_free, drain;  // one arrival
    uint64_t p_ready[4], s_read[2];           // halves of a tile's weights; its scores are read; of four warps
    uint64_t v_sent[kAhead];                  // masked tiles in turn: the copy of the values is under way ...
    uint64_t v_ok[kAhead];                    // ... and looked through
    uint64_t w_full[kQueue], w_free[kQueue];  // a unit is announced; everybody is done with it
    uint64_t pages[kQueue];                   // its pages' numbers are looked through
    uint64_t near, got;                       // a unit's last tiles are being copied; the next one's number is here
    alignas(16) uint4 next;
    Work work[kQueue];
    int fix[kQueue], bad[kQueue];
    int holds[C::kSlots];                     // the group of loads that a slot's is in
    prompt::Scan<C::kThreads> scan;
    alignas(16) int blocks[kChunks], kv[kChunks];  // before each part of the list of requests
    uint8_t order[kChunks];                   // where a part is one request: the one with the longest rows first
    uint32_t tmem;
};

// The ring's slots of a tile's pieces, tile after tile.
template <int D>
struct Slots {
    using C = Cfg<D>;
    int slot[C::kPieces], phase[C::kPieces];
    __device__ __forceinline__ Slots() {
#pragma unroll
        for (int y = 0; y < C::kPieces; ++y) slot[y] = y, phase[y] = 0;
    }
    __device__ __forceinline__ void next() {
#pragma unroll
        for (int y = 0; y < C::kPieces; ++y) {
            slot[y] += C::kPieces;
            if (slot[y] >= C::kSlots) slot[y] -= C::kSlots, phase[y] ^= 1;
        }
    }
};

// Ring positions of the loads of n tiles, in the order the products use them: K0 K1 V0 K2 V1 ... V(n-1).
__device__ __forceinline__ int k_pos(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_pos(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

__device__ __forceinline__ int unit_tiles(const Args &a, const Unit &u, int stages, int &tile0) {
    const int lo = a.window ? max(0, u.len + u.tok0 + 1 - a.window) : 0;
    const int last = min(u.tok0 + stages * a.per_tile, u.n) - 1;
    tile0 = lo / kTile;
    return (u.len + last) / kTile + 1 - tile0;
}
__device__ __forceinline__ Span span_of(const Args &a, const Unit &u, int stages, int part) {
    Span s;
    int tile0;
    const int all = unit_tiles(a, u, stages, tile0);
    const int from = all * part / u.parts, to = all * (part + 1) / u.parts;  // (2^18 tiles, 64 parts)
    s.tile0 = tile0 + from;
    s.tiles = to - from;
#pragma unroll
    for (int st = 0; st < 2; ++st) {
        const int first = u.tok0 + st * a.per_tile, last = min(first + a.per_tile, u.n) - 1;
        s.ns[st] = st < stages && first < u.n ? min(max((u.len + last) / kTile + 1 - s.tile0, 0), s.tiles) : 0;
    }
    const int last = min(u.tok0 + stages * a.per_tile, u.n) - 1;
    s.all = u.len + u.tok0 + 1;
    s.end = u.len + last + 1;
    s.begin = a.window ? max(0, u.len + u.tok0 + 1 - a.window) : 0;
    s.full = a.window ? max(0, u.len + last + 1 - a.window) : 0;
    s.right = s.all / kTile;
    s.left = (s.full + kTile - 1) / kTile;
    return s;
}
__device__ __forceinline__ bool masked(const Span &s, int tile) { return tile >= s.right || tile < s.left; }
// Steps of 16 positions of a tile that some row sees.
__device__ __forceinline__ int2 steps_of(const Span &s, int tile) {
    return make_int2(max(s.begin - tile * kTile, 0) / 16, (min(s.end - tile * kTile, kTile) + 15) / 16);
}

// Adds to a row, as it was written, the values that are not finite at positions of masked tiles that it sees: they were
// taken out of the tiles, where a zero weight would not have kept them from the other rows.
template <int D>
__device__ __noinline__ void add_special(const Args &a, const Work &w, int pos, uint16_t *row, float *part_row) {
    for (int ch = 0; ch < D; ch += 8) {
        float add[8] = {};
        bool any = false;
        for (int j = 0; j < w.sp.tiles; ++j) {
            const int tile = w.sp.tile0 + j;
            if (!masked(w.sp, tile)) continue;
            const int from = max(tile * kTile, a.window ? pos - a.window + 1 : 0),
                      to = min(tile * kTile + kTile - 1, pos);
            const uint16_t *v = a.v + (w.u.kv0 + from) * a.v_row + int64_t(w.hk) * a.v_head + ch;
            for (int t = from; t <= to; ++t, v += a.v_row) {
                const uint4 y = *reinterpret_cast<const uint4 *>(v);
                const uint32_t most = __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu),
                                               __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu));
                if (max(most >> 16, most & 0xffffu) < 0x7f80u) continue;
                const uint32_t x[4] = {y.x, y.y, y.z, y.w};
                any = true;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if ((x[c] & 0x7f80u) == 0x7f80u) add[2 * c] += __uint_as_float(x[c] << 16);
                    if ((x[c] & 0x7f800000u) == 0x7f800000u) add[2 * c + 1] += __uint_as_float(x[c] & 0xffff0000u);
                }
            }
        }
        if (!any) continue;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            if (part_row)
                part_row[ch + c] += add[c];
            else
                row[ch + c] = gdn::f32_to_bf16(gdn::bf16_to_f32(row[ch + c]) + add[c]);
        }
    }
}

// The next launch-grid block that has not started, taken over by this CTA; the answer lands in *to.
__device__ __forceinline__ void ask_next(uint4 *to, uint64_t *bar) {
    gdn::mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
            gdn::smem_u32(to)),
        "r"(gdn::smem_u32(bar))
        : "memory");
}
// Its block numbers; false: there is none left.
__device__ __forceinline__ bool next_of(const uint4 *from, int &x, int &y) {
    uint32_t got, bx, by;
    asm volatile(
        "{\n .reg .b128 r;\n .reg .pred p;\n .reg .b32 z, w;\n ld.shared.b128 r, [%3];\n"
        " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
        " mov.u32 %2, 0;\n @p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, z, w}, r;\n}\n"
        : "=&r"(got), "=&r"(bx), "=&r"(by)
        : "r"(gdn::smem_u32(from))
        : "memory");
    x = int(bx);
    y = int(by);
    return got != 0;
}

// The unit of block (x, part), found by a warp: the later rows of a request, which see most, come first.
template <int D>
__device__ __forceinline__ bool find_unit(const Args &a, const Shared<D> &s, int x, int part, int total, Work &w) {
    constexpr int kStages = Cfg<D>::kStages;
    const int lane = threadIdx.x & 31, per_unit = kStages * a.per_tile;
    const int rank = x / a.h_kv;
    if (rank >= total) return false;
    int i = 0;  // the last part of the list that begins at or before the rank
#pragma unroll
    for (int e = 0; e < kChunks / 32; ++e) i += __popc(__ballot_sync(0xffffffffu, s.blocks[e * 32 + lane] <= rank));
    --i;
    const int chunk = (a.rq.B + kChunks - 1) / kChunks;
    int blocks = s.blocks[i];
    if (chunk == 1) i = s.order[i];
    const int r1 = min(a.rq.B, (i + 1) * chunk);
    int64_t kv = s.kv[i];
    Unit &u = w.u;
    for (int r0 = i * chunk; r0 < r1; r0 += 32) {
        prompt::Request q{};
        if (r0 + lane < r1) q = prompt::request_of(a.rq, r0 + lane);
        const int nb = (q.n + per_unit - 1) / per_unit, rows = int(prompt::kv_rows_of(q));
        int nb_in = nb, rows_in = rows;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, nb_in, o), z = __shfl_up_sync(0xffffffffu, rows_in, o);
            if (lane >= o) nb_in += y, rows_in += z;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, rank < blocks + nb_in);
        if (here) {
            const int l = __ffs(here) - 1;
            const int before = blocks + __shfl_sync(0xffffffffu, nb_in - nb, l);
            const int count = __shfl_sync(0xffffffffu, nb, l);
            kv += __shfl_sync(0xffffffffu, rows_in - rows, l);
            u.t0 = __shfl_sync(0xffffffffu, q.t0, l);
            u.n = __shfl_sync(0xffffffffu, q.n, l);
            u.len = __shfl_sync(0xffffffffu, q.len, l);
            u.r = r0 + l;
            u.tok0 = (count - 1 - (rank - before)) * per_unit;
            u.kv0 = a.rq.kv_capacity ? kv : int64_t(u.t0);
            if (a.rq.kv_capacity && kv + u.len + u.n > a.rq.kv_capacity) return false;
            int tile0;
            const int tiles = unit_tiles(a, u, kStages, tile0);
            u.parts = min(a.splits, (tiles + a.part_tiles - 1) / a.part_tiles);
            if (part >= u.parts) return false;
            w.sp = span_of(a, u, kStages, part);
            w.hk = x - rank * a.h_kv;
            w.part = part;
            w.x = x;
            return true;
        }
        blocks += __shfl_sync(0xffffffffu, nb_in, 31);
        kv += __shfl_sync(0xffffffffu, rows_in, 31);
    }
    return false;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// The loads before a ld_wait are done: no use of them comes earlier.
template <int N>
__device__ __forceinline__ void arrived(uint32_t (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(x[i]));
}
constexpr int kHalf = kTile / 2;
__device__ __forceinline__ void load_half(uint32_t t_s, uint32_t (&x)[kHalf]) {
#pragma unroll
    for (int i = 0; i < kHalf; i += 32) tc::ld32_async(t_s + i, x + i);
}
// Positions past hi and up to lo (from the half's first) are not seen.
__device__ __forceinline__ void hide(uint32_t (&x)[kHalf], int hi, int lo) {
#pragma unroll
    for (int i = 0; i < kHalf / 32; ++i) {
        const int h = hi - 32 * i, b = lo - 32 * i;
        const uint32_t up = h < 0 ? 0u : h >= 31 ? ~0u : (2u << h) - 1u;
        const uint32_t see = b < 0 ? up : b >= 31 ? 0u : up & ~((2u << b) - 1u);
        if (__all_sync(0xffffffffu, see == ~0u)) continue;
#pragma unroll
        for (int c = 0; c < 32; ++c) x[32 * i + c] = see & (1u << c) ? x[32 * i + c] : 0xff800000u;
    }
}
__device__ __forceinline__ float top_of(const uint32_t (&x)[kHalf]) {
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < kHalf / 2; ++i)
        top[i & 3] = max3(top[i & 3], __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
    return max3(fmaxf(top[0], top[1]), top[2], top[3]);
}
// The weights 2^(c x + r) as bf16 pairs; returns their sum before that rounding.
__device__ __forceinline__ float weights(const uint32_t (&x)[kHalf], f2 c2, float r, uint32_t (&p)[kHalf / 2]) {
    const f2 r2 = pair(r, r);
    f2 sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
    for (int c = 0; c < kHalf / 2; ++c) {
        const float2 e = both(fma2(pair(x[2 * c], x[2 * c + 1]), c2, r2));
        const float e0 = ex2(e.x), e1 = ex2(e.y);
        sum[c & 1] = add2(sum[c & 1], pair(e0, e1));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[c]) : "f"(e1), "f"(e0));
    }
    const float2 t = both(add2(sum[0], sum[1]));
    return t.x + t.y;
}
// Four lanes' pieces of four rows, transposed: v[i] becomes lane i's (of the four) piece of this lane's number.
__device__ __forceinline__ void transpose4(uint4 (&v)[4]) {
    const int lane = threadIdx.x;
#pragma unroll
    for (int s = 1; s <= 2; s *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & s) continue;
            const bool up = lane & s;
            uint4 &lo = v[i], &hi = v[i | s];
            uint4 t = up ? lo : hi;
            t.x = __shfl_xor_sync(0xffffffffu, t.x, s);
            t.y = __shfl_xor_sync(0xffffffffu, t.y, s);
            t.z = __shfl_xor_sync(0xffffffffu, t.z, s);
            t.w = __shfl_xor_sync(0xffffffffu, t.w, s);
            lo = up ? t : lo;
            hi = up ? hi : t;
        }
}

// Writes four lanes' pieces of four rows, `c` bytes into the rows.
__device__ __forceinline__ void put(const unsigned long long (&to)[4], uint4 (&v)[4], int c) {
    transpose4(v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (to[i])
            asm volatile("st.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(to[i] + c), "r"(v[i].x), "r"(v[i].y),
                         "r"(v[i].z), "r"(v[i].w)
                         : "memory");
}
__device__ __forceinline__ void rounded(const uint32_t (&x)[32], float inv, uint4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = both(mul2(pair(x[8 * i + 2 * e], x[8 * i + 2 * e + 1]), pair(inv, inv)));
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y[e]) : "f"(f.y), "f"(f.x));
        }
        v[i] = make_uint4(y[0], y[1], y[2], y[3]);
    }
}
template <int D>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1) prompt_attend_kernel(const __grid_constant__ Args a) {
    using C = Cfg<D>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t raw[];
    __shared__ Shared<D> s;
    static_assert(sizeof(Shared<D>) <= 2048, "static shared memory");
    gdn::pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kCopyWarp = C::kSoftWarps, kMmaWarp = kCopyWarp + 1, kFindWarp = kCopyWarp + 2,
                  kGuardWarp = kCopyWarp + 3;
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&s.tmem, 512);
    } else if (warp == kCopyWarp && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.mq) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.mk) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&a.mv) : "memory");
        for (int i = 0; i < C::kSlots; ++i) gdn::mbar_init(s.full + i, 1);
        for (int i = 0; i < kGroups; ++i) gdn::mbar_init(s.freed + i, 1);
        for (int i = 0; i < 2; ++i) {
            gdn::mbar_init(s.s_full + i, 1);
            gdn::mbar_init(s.o_done + i, 1);
            gdn::mbar_init(s.s_read + i, 4);
        }
        for (int i = 0; i < 4; ++i) gdn::mbar_init(s.p_ready + i, 4);
        gdn::mbar_init(&s.q_full, 1);
        gdn::mbar_init(&s.q_free, 1);
        gdn::mbar_init(&s.drain, 1);
        gdn::mbar_init(&s.got, 1);
        gdn::mbar_init(&s.near, 1);
        for (int i = 0; i < kAhead; ++i) {
            gdn::mbar_init(s.v_sent + i, 1);
            gdn::mbar_init(s.v_ok + i, C::kGuards);
        }
        for (int i = 0; i < kQueue; ++i) {
            gdn::mbar_init(s.w_full + i, 1);
            gdn::mbar_init(s.w_free + i, C::kSoftWarps + 2 + C::kGuards);
            gdn::mbar_init(s.pages + i, C::kGuards);
        }
    }
    gdn::pdl_wait();
    // what a CTA left undone that timed out, no other tries again
    const bool late = a.status && (*reinterpret_cast<volatile uint32_t *>(a.status) & GDN_DEV_TIMEOUT);

    // ---- the requests: sums over parts of their list
    const int per_unit = kStages * a.per_tile;
    long long total;
    {
        const int chunk = (a.rq.B + kChunks - 1) / kChunks, r0 = min(a.rq.B, tid * chunk), r1 = min(a.rq.B, r0 + chunk);
        long long blocks = 0, kv = 0, kv_all;
        prompt::Request q{};
        for (int r = r0; r < r1; ++r) {
            q = prompt::request_of(a.rq, r);
            if (q.bad && blockIdx.x == 0 && blockIdx.y == 0) gdn::set_status(a.status, GDN_DEV_ROWS_BAD);
            blocks += (q.n + per_unit - 1) / per_unit;
            kv += prompt::kv_rows_of(q);
        }
        if (chunk == 1 && a.rq.B > 1) {
            // long units started last would run alone (8 prompts of 512..12,000 rows: 1,070 us in the order given)
            if (tid < kChunks) s.kv[tid] = tid >= a.rq.B ? -1 : q.n ? q.len + q.n : 0;
            __syncthreads();
            if (tid < a.rq.B) {
                const int mine = s.kv[tid];
                int at = 0;
                for (int r = 0; r < a.rq.B; r += 4) {
                    const int4 x = *reinterpret_cast<const int4 *>(s.kv + r);
                    at += (x.x > mine || (x.x == mine && r < tid)) + (x.y > mine || (x.y == mine && r + 1 < tid)) +
                          (x.z > mine || (x.z == mine && r + 2 < tid)) + (x.w > mine || (x.w == mine && r + 3 < tid));
                }
                s.order[at] = uint8_t(tid);
                s.blocks[at] = int(blocks);
            }
            __syncthreads();
            blocks = tid < a.rq.B ? s.blocks[tid] : 0;
            __syncthreads();
        } else if (tid < kChunks) {
            s.order[tid] = uint8_t(tid);
        }
        prompt::scan2<C::kThreads>(s.scan, blocks, kv, total, kv_all);
        if (a.rq.kv_capacity && kv_all > a.rq.kv_capacity && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0)
            gdn::set_status(a.status, GDN_DEV_ROWS_BAD);
        if (tid < kChunks) {
            s.blocks[tid] = int(blocks);
            // (past the workspace's rows a request is refused, however far)
            s.kv[tid] = int(min(kv, (long long)gdn_host::kKv8MaxLen));
        }
    }
    tc::fence_before();
    const bool stop = __syncthreads_or(late);
    tc::fence_after();
    const uint32_t tm = s.tmem;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *s_q = sm, *s_ring = sm + kStages * C::kQTile;
    bool ok = !stop;
    // A warp's wait: one lane's.  (Before shared memory is read that it is for: a __syncwarp.  Tensor memory has its fence.)
    auto wait = [&](uint64_t *bar, int phase) {
        if (lane == 0) ok = gdn::mbar_wait_bounded(bar, phase & 1, a.wait_ns);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        return ok;
    };
    // Whether there is a unit k, once that is known, and that this warp is done with it.
    auto take = [&](int k) {
        if (!ok || !wait(&s.w_full[k % kQueue], k / kQueue)) return false;
        __syncwarp();
        return s.work[k % kQueue].x >= 0;
    };
    auto done = [&](int k) {
        __syncwarp();
        if (lane == 0) arrive(&s.w_free[k % kQueue]);
    };

    if (warp < kCopyWarp) {
        // ---- softmax: a thread a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
        const int st = warp >> 2;
        const int row = (warp & 3) * 32 + lane, tok = row / a.group, head = row - tok * a.group;
        const uint32_t lanes = uint32_t(warp & 3) << 21;
        const uint32_t t_o = tm + 256 + (kStages == 2 ? st * D : 0) + lanes;
        const f2 c2 = pair(a.scale_log2, a.scale_log2);
        int g = 0, units = 0;  // tiles so far, and units with any
        for (int k = 0; take(k); ++k) {
            const Work &w = s.work[k % kQueue];
            const int n = w.sp.ns[st];
            // (rows of nobody: weights of 0)
            const auto position = [&] { return w.u.tok0 + st * a.per_tile + tok; };
            const auto valid = [&] { return tok < a.per_tile && position() < w.u.n; };
            // Weights are 2^(c x - m), from kFar on 2^(c (x - base)): then m stays -inf, so that every tile is looked at.
            float m = valid() ? -INFINITY : INFINITY, l = 0.f, base = 0.f;
            for (int j = 0; j < n; ++j, ++g) {
                const int slot = kStages == 2 ? st : g & 1, turn = kStages == 2 ? g : g >> 1;
                if (!wait(&s.s_full[slot], turn)) break;
                tc::fence_after();
                const uint32_t t_s = tm + slot * kTile + lanes, t_p = C::kApart ? tm + 384 + st * kHalf + lanes : t_s;
                uint32_t x[2][kHalf];
                load_half(t_s, x[0]);
                load_half(t_s + kHalf, x[1]);
                tc::ld_wait();
                arrived(x[0]);
                arrived(x[1]);
                if constexpr (C::kApart) {
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(&s.s_read[slot]);
                }
                if (masked(w.sp, w.sp.tile0 + j)) {
                    const int hi = w.u.len + position() - (w.sp.tile0 + j) * kTile, lo = a.window ? hi - a.window : -1;
                    hide(x[0], hi, lo);
                    hide(x[1], hi - kHalf, lo - kHalf);
                }
                const float top = fmaxf(top_of(x[0]), top_of(x[1])), z = top * a.scale_log2;
                if constexpr (C::kApart) {
                    // the last tile's products are done with the sums and the weights
                    if (j > 0 && !wait(&s.o_done[st], g - 1)) break;
                    tc::fence_after();
                }
                if (__any_sync(0xffffffffu, z > m + kSlack)) {
                    float f = 1.f;
                    if (base == 0.f ? z > m : top > base) {
                        const float last_m = base == 0.f ? m : 0.f, last_base = base;
                        const bool far = fabsf(z) >= kFar && fabsf(top) < INFINITY;
                        base = far ? top : 0.f;
                        m = far ? -INFINITY : z;
                        f = ex2(fmaf(a.scale_log2, last_base - base, last_m - (far ? 0.f : z)));
                    }
                    if (j > 0 && __any_sync(0xffffffffu, f != 1.f)) {
                        // (with two query tiles and no room the scores are behind the products before)
                        if (kStages == 1 && !wait(&s.o_done[(g - 1) & 1], (g - 1) >> 1)) break;
                        tc::fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tc::ld16_async(t_o + c, o);
                            tc::ld_wait();
                            arrived(o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tc::st16_async(t_o + c, o);
                        }
                    }
                    l *= f;
                    if (__any_sync(0xffffffffu, base != 0.f)) {
#pragma unroll
                        for (int i = 0; i < kTile; ++i)
                            x[i / kHalf][i % kHalf] = __float_as_uint(__uint_as_float(x[i / kHalf][i % kHalf]) - base);
                    }
                }
                // The products with the first half's weights run beside the second half's exponentials.
                const float r = m == -INFINITY ? 0.f : -m;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[kHalf / 2];
                    l += weights(x[half], c2, r, p);
                    tc::st32_async(t_p + half * (kHalf / 2), p);
                    tc::st_wait();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) arrive(&s.p_ready[2 * slot + half]);
                }
            }
            if (!ok) break;
            if (!wait(&s.pages[k % kQueue], k / kQueue)) break;
            if (n > 0) {
                if (!wait(&s.o_done[kStages == 2 ? st : (g - 1) & 1],
                          C::kApart ? g - 1 : kStages == 2 ? units : (g - 1) >> 1))
                    break;
                ++units;
            }
            tc::fence_after();
            __syncwarp();
            const bool fix = *reinterpret_cast<volatile int *>(&s.fix[k % kQueue]);
            const bool bad = *reinterpret_cast<volatile int *>(&s.bad[k % kQueue]);
            const int at = position();
            const bool write = valid() && !bad, whole = w.u.parts == 1;
            const int64_t wrow = ((int64_t(w.x) * a.splits + w.part) * kStages + st) * kTile + row;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int h = w.hk * a.group + head;
            uint16_t *const row_o = a.o + (int64_t(w.u.t0) + at) * a.o_stride + int64_t(h) * D;
            float *const row_p = whole ? nullptr : a.ws_o + wrow * D;
            // A store of 16 bytes from each of 32 rows is 32 accesses; four lanes trade pieces, so that they write 64 bytes
            // of a row together.  Where this lane's piece of each of four lanes' rows goes (0: nowhere):
            unsigned long long to[4];
            {
                const unsigned long long x = !write  ? 0
                                             : whole ? reinterpret_cast<unsigned long long>(row_o)
                                                     : reinterpret_cast<unsigned long long>(row_p);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    to[i] = __shfl_sync(0xffffffffu, x, (lane & ~3) + i);
                    if (to[i]) to[i] += (lane & 3) * 16;
                }
            }
            // (without a tile there are no rows, or, of a part, sums that the join leaves out)
#pragma unroll 1
            for (int c = 0; n > 0 && c < D; c += C::kOut) {
                uint32_t x[C::kOut / 32][32];
#pragma unroll
                for (int e = 0; e < C::kOut / 32; ++e) tc::ld32_async(t_o + c + 32 * e, x[e]);
                tc::ld_wait();
#pragma unroll
                for (int e = 0; e < C::kOut / 32; ++e) {
                    arrived(x[e]);
                    if (l == 0.f) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[e][i] = 0;
                    }
                    uint4 v[4];
                    if (whole) {
                        rounded(x[e], inv, v);
                        put(to, v, 2 * (c + 32 * e));
                    } else {
#pragma unroll
                        for (int y = 0; y < 32; y += 16) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                v[i] = make_uint4(x[e][y + 4 * i], x[e][y + 4 * i + 1], x[e][y + 4 * i + 2],
                                                  x[e][y + 4 * i + 3]);
                            put(to, v, 4 * (c + 32 * e + y));
                        }
                    }
                }
            }
            if (fix) {
                __syncwarp();
                // (a row of nothing but -inf is zero, whatever the values)
                if (write && n > 0 && l != 0.f) add_special<D>(a, w, w.u.len + at, row_o, row_p);
            }
            if (write && whole) {
                if (a.lse)
                    a.lse[(int64_t(w.u.t0) + at) * a.h_q + h] =
                        l == 0.f ? -INFINITY
                                 : fmaf(a.scale_log2, base, (base == 0.f ? m : 0.f) + log2f(l)) * 0.6931471805599453f;
            } else if (write) {
                a.ws_ml[wrow] = base == 0.f ? make_float2(m, l) : make_float2(base, copysignf(l, -1.f));
            }
            if (tid == 0 && w.part == 0 && a.info) {
                Info f = {};
                f.t0 = w.u.t0;
                f.tok0 = w.u.tok0;
                f.n = w.u.n;
                f.hk = w.hk;
                f.parts = whole || bad ? 0 : w.u.parts;
                a.info[w.x] = f;
            }
            tc::fence_before();
            done(k);
        }
        if (!ok && !stop) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
        if (warp == kCopyWarp) {
            // ---- copies: one lane
            const bool one = elect_one();
            // ring: tiles' places before this unit; group: of loads that the products free together, a tile's keys and the
            // values of the one before, or each by itself where they fill the ring
            int ring = 0, issued = 0, sent = 0, units = 0, group = 0;
            auto load = [&](const CUtensorMap &map, const Work &w, int tile, int place) {
                for (int x = 0; x < C::kPieces; ++x) {
                    const int pos = place * C::kPieces + x, slot = pos % C::kSlots;
                    if (pos >= C::kSlots)
                        ok = ok && gdn::mbar_wait_bounded(&s.freed[s.holds[slot] % kGroups],
                                                          s.holds[slot] / kGroups & 1, a.wait_ns);
                    if (!ok) return;
                    s.holds[slot] = group;
                    gdn::mbar_arrive_expect_tx(&s.full[slot], C::kSlot);
                    for (int c = 0; c < C::kPiece; c += 64)
                        gdn::tma_load_3d(s_ring + slot * C::kSlot + c * kTile * 2, &map, x * C::kPiece + c, w.hk,
                                         int(w.u.kv0) + tile * kTile, &s.full[slot]);
                    issued = pos + 1;
                }
            };
            for (int k = 0; one; ++k) {
                ok = ok && gdn::mbar_wait_bounded(&s.w_full[k % kQueue], k / kQueue & 1, a.wait_ns);
                if (!ok || s.work[k % kQueue].x < 0) break;
                const Work w = s.work[k % kQueue];
                const int nt = w.sp.tiles;
                load(a.mk, w, w.sp.tile0, ring);
                ++group;
                if (ok && k > 0) ok = gdn::mbar_wait_bounded(&s.q_free, (k - 1) & 1, a.wait_ns);
                if (!ok) break;
                int tiles = 0;
                for (int st = 0; st < kStages; ++st) tiles += w.sp.ns[st] > 0;
                gdn::mbar_arrive_expect_tx(&s.q_full, uint32_t(tiles * a.per_tile * a.group) * (D * 2));
                for (int st = 0; st < kStages; ++st)
                    if (w.sp.ns[st] > 0)
                        for (int c = 0; c < D; c += 64)
                            gdn::tma_load_3d(s_q + st * C::kQTile + c * kTile * 2, &a.mq, c, w.hk * a.group,
                                             w.u.t0 + w.u.tok0 + st * a.per_tile, &s.q_full);
                units = k + 1;
                for (int i = 1; i <= nt && ok; ++i) {
                    if (i == max(1, nt - 3)) arrive(&s.near);
                    if (i < nt) {
                        load(a.mk, w, w.sp.tile0 + i, ring + k_pos(i));
                        if (kStages == 1) ++group;
                    }
                    if (!ok || (a.withhold && i == nt)) continue;
                    load(a.mv, w, w.sp.tile0 + i - 1, ring + v_pos(i - 1, nt));
                    ++group;
                    if (ok && masked(w.sp, w.sp.tile0 + i - 1)) {
                        arrive(&s.v_sent[sent % kAhead]);
                        ++sent;
                    }
                }
                if (!ok) break;
                ring += 2 * nt;
                arrive(&s.w_free[k % kQueue]);
            }
            // every copy has landed before the CTA leaves (on the usual path these waits are over)
            if (units) (void)gdn::mbar_wait_bounded(&s.q_full, (units - 1) & 1, a.wait_ns);
            for (int pos = max(0, issued - C::kSlots); pos < issued; ++pos)
                (void)gdn::mbar_wait_bounded(&s.full[pos % C::kSlots], (pos / C::kSlots) & 1, a.wait_ns);
            __syncwarp();
        } else if (warp == kMmaWarp) {
            // ---- products: one lane waits and issues
            if (elect_one()) {
                const uint32_t id_s = tc::idesc_bf16(128, kTile) | (a.negate ? tc::kNegA : 0);
                constexpr uint32_t id_p = tc::idesc_bf16(128, C::kPiece) | tc::kBMnMajor;
                const uint64_t dq = tc::smem_desc(gdn::smem_u32(s_q)), dk = tc::smem_desc(gdn::smem_u32(s_ring));
                const uint64_t dv = tc::smem_desc_mn(gdn::smem_u32(s_ring), kTile * 128);
                int guarded = 0, groups = 0;
                int g0 = 0, g1 = 0;  // tiles of each query tile before this unit
                Slots<D> at;         // of the ring's next tile
                // A tile's pieces have landed.
                auto landed = [&](const Slots<D> &x) {
#pragma unroll
                    for (int y = 0; y < C::kPieces; ++y) ok = ok && gdn::mbar_wait_bounded(&s.full[x.slot[y]], x.phase[y], a.wait_ns);
                    return ok;
                };
                auto scores = [&](int st, int slot, const Slots<D> &x) {
#pragma unroll
                    for (int y = 0; y < C::kPieces; ++y) {
                        const uint64_t d = tc::desc_at(dk, x.slot[y] * C::kSlot), q = tc::desc_at(dq, st * C::kQTile);
#pragma unroll
                        for (int i = 0; i < C::kPiece / 16; ++i) {
                            const int e = y * C::kPiece / 16 + i;
                            tc::mma_bf16(tm + slot * kTile, tc::desc_at(q, (e / 4) * kTile * 128 + (e % 4) * 32),
                                         tc::desc_at(d, (i / 4) * kTile * 128 + (i % 4) * 32), id_s, e > 0);
                        }
                    }
                    tc::commit(&s.s_full[slot]);
                };
                const auto t_p = [&](int slot) { return C::kApart ? tm + 384 + slot * kHalf : tm + slot * kTile; };
                // (the softmax warps give a unit's first weights after they have read the last unit's sums)
                auto outputs = [&](int st, int slot, const Slots<D> &x, bool more, int turn) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = ok && gdn::mbar_wait_bounded(&s.p_ready[2 * slot + half], turn & 1, a.wait_ns);
                        if (!ok) return false;
                        tc::fence_after();
#pragma unroll
                        for (int y = 0; y < C::kPieces; ++y) {
                            const uint64_t d = tc::desc_at(dv, x.slot[y] * C::kSlot);
                            const uint32_t to = tm + 256 + (kStages == 2 ? st * D : 0) + y * C::kPiece;
#pragma unroll
                            for (int i = half * kHalf / 16; i < (half + 1) * kHalf / 16; ++i)
                                tc::mma_bf16_ts(to, t_p(slot) + i * 8, tc::desc_at(d, i * 2048), id_p, more || i > 0);
                        }
                    }
                    return true;
                };
                // The same over the positions that some row sees.
                auto outputs_cut = [&](int st, int slot, const Slots<D> &x, bool more, int2 e) {
#pragma unroll 1
                    for (int i = e.x; i < e.y; ++i)
#pragma unroll
                        for (int y = 0; y < C::kPieces; ++y)
                            tc::mma_bf16_ts(tm + 256 + (kStages == 2 ? st * D : 0) + y * C::kPiece,
                                            t_p(slot) + i * 8, tc::desc_at(dv, x.slot[y] * C::kSlot + i * 2048), id_p,
                                            more || i > e.x);
                };
                auto free_group = [&] {
                    tc::commit(&s.freed[groups % kGroups]);
                    ++groups;
                };
                auto weights_of = [&](int slot, int turn) {
                    for (int half = 0; half < 2; ++half)
                        ok = ok && gdn::mbar_wait_bounded(&s.p_ready[2 * slot + half], turn & 1, a.wait_ns);
                    tc::fence_after();
                    return ok;
                };
                // (each tile's reading is waited for once: by the next tile's scores, or the next unit's first)
                auto read = [&](int st, int turn) {
                    ok = ok && gdn::mbar_wait_bounded(&s.s_read[st], turn & 1, a.wait_ns);
                    tc::fence_after();
                    return ok;
                };
                for (int k = 0;; ++k) {
                    ok = ok && gdn::mbar_wait_bounded(&s.w_full[k % kQueue], k / kQueue & 1, a.wait_ns);
                    if (!ok || s.work[k % kQueue].x < 0) break;
                    const Span sp = s.work[k % kQueue].sp;
                    const int nt = sp.tiles, n0 = sp.ns[0], n1 = sp.ns[1];
                    ok = gdn::mbar_wait_bounded(&s.q_full, k & 1, a.wait_ns);
                    if (!ok) break;
                    if constexpr (kStages == 2) {
                        // a tile's outputs, and the next one's scores where its weights lay
                        Slots<D> kt = at;
                        at.next();
                        if (!landed(kt)) break;
                        if (C::kApart && ((n0 > 0 && g0 > 0 && !read(0, g0 - 1)) || (n1 > 0 && g1 > 0 && !read(1, g1 - 1))))
                            break;
                        tc::fence_after();
                        if (n0 > 0) scores(0, 0, kt);
                        if (n1 > 0) scores(1, 1, kt);
                        free_group();
                        if (nt == 1) tc::commit(&s.q_free);
                        const int whole = min(min(n0, n1) - 1, sp.right - sp.tile0);
#pragma unroll 1
                        for (int j = 0; j < nt; ++j) {
                            kt = at;
                            if (j + 1 < nt) at.next();
                            const Slots<D> vt = at;
                            at.next();
                            if (j > 0 && j < whole && sp.tile0 + j >= sp.left) {
                                // both query tiles, every position
                                if (!landed(kt) || !landed(vt)) break;
                                if constexpr (C::kApart) {
                                    if (!read(0, g0 + j)) break;
                                    scores(0, 0, kt);
                                    if (!read(1, g1 + j)) break;
                                    scores(1, 1, kt);
                                    if (!outputs(0, 0, vt, true, g0 + j)) break;
                                    tc::commit(&s.o_done[0]);
                                    if (!outputs(1, 1, vt, true, g1 + j)) break;
                                    tc::commit(&s.o_done[1]);
                                } else {
                                    if (!outputs(0, 0, vt, true, g0 + j)) break;
                                    scores(0, 0, kt);
                                    if (!outputs(1, 1, vt, true, g1 + j)) break;
                                    scores(1, 1, kt);
                                }
                            } else {
                                const bool cut = masked(sp, sp.tile0 + j);
                                const int2 e = cut ? steps_of(sp, sp.tile0 + j) : make_int2(0, kTile / 16);
                                if (j + 1 < nt) landed(kt);
                                if constexpr (C::kApart) {
#pragma unroll 1
                                    for (int st = 0; st < 2 && ok; ++st)
                                        if (j + 1 < (st ? n1 : n0) && read(st, (st ? g1 : g0) + j)) scores(st, st, kt);
                                }
                                if (!landed(vt)) break;
                                if (cut) {
                                    ok = gdn::mbar_wait_bounded(&s.v_ok[guarded % kAhead], guarded / kAhead & 1, a.wait_ns);
                                    ++guarded;
                                }
#pragma unroll 1
                                for (int st = 0; st < 2; ++st) {
                                    const int n = st ? n1 : n0;
                                    if (j < n) {
                                        if (!weights_of(st, (st ? g1 : g0) + j)) break;
                                        outputs_cut(st, st, vt, j > 0, e);
                                        if (C::kApart || j + 1 == n) tc::commit(&s.o_done[st]);
                                    }
                                    if (!C::kApart && j + 1 < n) scores(st, st, kt);
                                }
                                if (!ok) break;
                            }
                            free_group();
                            if (j + 2 == nt) tc::commit(&s.q_free);
                        }
                        g0 += n0;
                        g1 += n1;
                    } else {
                        // a tile's outputs, and the scores of the next but one where its weights lay
#pragma unroll 1
                        for (int j = -2; j < nt; ++j) {
                            const int y = g0 + j;
                            if (j >= 0) {
                                const Slots<D> vt = at;
                                at.next();
                                const bool cut = masked(sp, sp.tile0 + j);
                                if (!landed(vt)) break;
                                if (cut) {
                                    ok = gdn::mbar_wait_bounded(&s.v_ok[guarded % kAhead], guarded / kAhead & 1,
                                                                a.wait_ns);
                                    ++guarded;
                                }
                                if (!cut) {
                                    if (!outputs(0, y & 1, vt, j > 0, y >> 1)) break;
                                } else {
                                    if (!weights_of(y & 1, y >> 1)) break;
                                    outputs_cut(0, y & 1, vt, j > 0, steps_of(sp, sp.tile0 + j));
                                }
                                tc::commit(&s.o_done[y & 1]);
                                free_group();
                            }
                            if (j + 2 < nt) {
                                const Slots<D> kt = at;
                                at.next();
                                if (!landed(kt)) break;
                                scores(0, y & 1, kt);
                                free_group();
                                if (j + 3 == nt) tc::commit(&s.q_free);
                            }
                        }
                        g0 += nt;
                    }
                    if (!ok) break;
                    arrive(&s.w_free[k % kQueue]);
                }
                if (!ok && !stop) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
                // no product reads shared memory after the CTA has left
                tc::commit(&s.drain);
                (void)gdn::mbar_wait_bounded(&s.drain, 0, a.wait_ns);
            }
            __syncwarp();
        } else if (warp == kFindWarp) {
            // ---- units: this block's own, then those of blocks that have not started
            int x = blockIdx.x, part = blockIdx.y, asked = 0, k = 0;
            bool more = ok;
            while (more) {
                Work w;
                const bool found = find_unit<D>(a, s, x, part, int(total), w);
                if (!found && part == 0 && a.info && lane == 0) a.info[x].parts = 0;
                if (found) {
                    if (k >= kQueue)
                        ok = gdn::mbar_wait_bounded(&s.w_free[k % kQueue], (k / kQueue - 1) & 1, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok && lane == 0) {
                        s.fix[k % kQueue] = s.bad[k % kQueue] = 0;
                        s.work[k % kQueue] = w;
                        arrive(&s.w_full[k % kQueue]);
                    }
                    // the next one is taken over when this one ends, not before: others may be free earlier
                    ok = ok && gdn::mbar_wait_bounded(&s.near, k & 1, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    ++k;
                }
                if (!ok) break;
                if (lane == 0) ask_next(&s.next, &s.got);
                const bool here = gdn::mbar_wait_bounded(&s.got, asked & 1, a.wait_ns);
                ok = __all_sync(0xffffffffu, here);
                ++asked;
                if (!ok) break;
                more = next_of(&s.next, x, part);
                // the answer is read before the next one is written
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
            if (ok) {
                if (k >= kQueue) ok = gdn::mbar_wait_bounded(&s.w_free[k % kQueue], (k / kQueue - 1) & 1, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (ok && lane == 0) {
                    s.work[k % kQueue].x = -1;
                    arrive(&s.w_full[k % kQueue]);
                }
            }
        } else {
            // ---- guards: a zero weight times what is not finite is not zero, so such values go out of masked tiles
            const int me = tid - kGuardWarp * 32;
            int ring = 0, seen = 0;
            for (int k = 0; take(k); ++k) {
                const Work w = s.work[k % kQueue];
                const int nt = w.sp.tiles;
                if (a.table) {
                    const int T = 1 << a.page_shift;
                    const int first = (a.window ? max(0, w.u.len + 1 - a.window) : 0) >> a.page_shift;
                    const int last = w.u.len > 0 ? (w.u.len + T - 1) >> a.page_shift : 0;
                    bool bad = false;
                    for (int i = first + me; i < last; i += 32 * C::kGuards) {
                        const int p = a.table[int64_t(w.u.r) * a.table_stride + i];
                        bad |= p < 0 || p >= a.num_pages;
                    }
                    if (bad) *reinterpret_cast<volatile int *>(&s.bad[k % kQueue]) = 1;
                }
                __syncwarp();
                if (lane == 0) arrive(&s.pages[k % kQueue]);
                for (int j = 0; j < nt && ok; ++j) {
                    if (!masked(w.sp, w.sp.tile0 + j)) continue;
                    // (a copy under way: its barrier is in that copy's phase, not in an earlier one of the same parity)
                    if (!wait(&s.v_sent[seen % kAhead], seen / kAhead)) break;
                    bool any = false;
                    for (int y = 0; y < C::kPieces && ok; ++y) {
                        const int pos = (ring + v_pos(j, nt)) * C::kPieces + y, slot = pos % C::kSlots;
                        if (!wait(&s.full[slot], pos / C::kSlots)) break;
                        __syncwarp();
                        uint4 *p = reinterpret_cast<uint4 *>(s_ring + slot * C::kSlot);
                        // rows of a block of 64 channels: those before `full` and from `all` on, a lane a row
                        const int base = (w.sp.tile0 + j) * kTile;
                        const int2 e = steps_of(w.sp, w.sp.tile0 + j);
                        const int r0 = 16 * e.x, r1 = min(max(w.sp.full - base, r0), 16 * e.y);
                        const int r2 = min(max(w.sp.all - base, r1), 16 * e.y), r3 = 16 * e.y;
                        const int rows = r1 - r0 + r3 - r2;
#pragma unroll 1
                        for (int i = me; i < rows * (C::kPiece / 64); i += 32 * C::kGuards) {
                            const int blk = i >= rows, in = i - blk * rows;
                            const int row = in < r1 - r0 ? r0 + in : r2 - (r1 - r0) + in;
                            uint4 *at = p + (blk * kTile + row) * 8, v[8];
                            uint32_t t = 0;
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                v[c] = at[(c + lane) & 7];  // (lanes on different banks)
                                t = __vmaxu2(t, __vmaxu2(__vmaxu2(v[c].x & 0x7fff7fffu, v[c].y & 0x7fff7fffu),
                                                         __vmaxu2(v[c].z & 0x7fff7fffu, v[c].w & 0x7fff7fffu)));
                            }
                            if (max(t >> 16, t & 0xffffu) < 0x7f80u) continue;
                            any = true;
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint4 x = at[c];
                                x.x &= __vcmpltu2(x.x & 0x7fff7fffu, 0x7f807f80u);
                                x.y &= __vcmpltu2(x.y & 0x7fff7fffu, 0x7f807f80u);
                                x.z &= __vcmpltu2(x.z & 0x7fff7fffu, 0x7f807f80u);
                                x.w &= __vcmpltu2(x.w & 0x7fff7fffu, 0x7f807f80u);
                                at[c] = x;
                            }
                        }
                    }
                    if (any) *reinterpret_cast<volatile int *>(&s.fix[k % kQueue]) = 1;
                    gdn::fence_proxy_async_smem();
                    __syncwarp();
                    if (ok && lane == 0) arrive(&s.v_ok[seen % kAhead]);
                    ++seen;
                }
                if (!ok) break;
                ring += 2 * nt;
                done(k);
            }
        }
        if (!ok && !stop) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
    }
    tc::fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tm, 512);
    }
}

// Joins a unit's parts: o = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p, a warp a row.  Of few parts a lane takes every m
// and l itself (8 chunks of 60 to 2,048 rows in up to 3 parts, 139 MB cold: 56 us -> 45); of many, those of every 32nd
// part, and kFew parts' sums are in flight together (32 rows of 16/2 heads of 256 in 38 parts: 39 us with a part at a
// time, 11 with eight in flight and CTAs of 8 rows).  Latency bounds it, and CTAs to start, many for units that are not.
constexpr int kFew = 8;
// A part's reference, c x + y, of its (m, l) as written: a base has l's sign; and how far one is above another.
__device__ __forceinline__ float2 reference_of(float2 ml) {
    return signbit(ml.y) ? make_float2(ml.x, 0.f) : make_float2(0.f, ml.x);
}
__device__ __forceinline__ float above(float2 a, float2 b, float c) { return fmaf(c, a.x - b.x, a.y - b.y); }
template <int D>
__device__ __forceinline__ void load_part(float (&y)[D / 32], const float *o) {
    constexpr int W = D / 32, V = W < 4 ? W : 4;
#pragma unroll
    for (int e = 0; e < W; e += V) {
        if constexpr (V == 4)
            *reinterpret_cast<float4 *>(&y[e]) = __ldcs(reinterpret_cast<const float4 *>(o + e * 32));
        else
            *reinterpret_cast<float2 *>(&y[e]) = __ldcs(reinterpret_cast<const float2 *>(o + e * 32));
    }
}

template <int D, bool MANY>
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ Args a) {
    gdn::pdl_enter();
    constexpr int kRows = Cfg<D>::kStages * kTile, W = D / 32, V = W < 4 ? W : 4;  // channels of a lane, and of a load
    const Info f = a.info[blockIdx.x];
    const uint32_t status = a.status ? *reinterpret_cast<volatile uint32_t *>(a.status) : 0;
    if (f.parts == 0 || (status & GDN_DEV_TIMEOUT)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned over = 65536u / unsigned(a.group) + 1;  // x / group = x * over >> 16 for x < 128, group <= 64
    for (int i = warp; i < a.join_rows; i += 8) {
        const int row = blockIdx.y * a.join_rows + i, st = row / kTile, in = row % kTile;
        const int tok = in * over >> 16, head = in - tok * a.group, at = f.tok0 + st * a.per_tile + tok;
        if (tok >= a.per_tile || at >= f.n) continue;
        const int64_t base = int64_t(blockIdx.x) * a.splits * kRows + row;
        const float2 *ml = a.ws_ml + base;
        const float *from = a.ws_o + base * D + lane * V;
        float acc[W] = {}, l = 0.f;
        float2 top = make_float2(0.f, -INFINITY);
        // (two references of -inf are a NaN apart, which is not above 0)
        const auto raise = [&](float2 y) {
            if (above(y, top, a.scale_log2) > 0.f) top = y;
        };
        bool based;  // whether some part has one; then x becomes how far it is below the top
        // (of a part without weight its sums say nothing)
        if constexpr (!MANY) {
            float2 x[kFew];
            float y[kFew][W];
#pragma unroll
            for (int p = 0; p < kFew; ++p) {
                if (p >= f.parts) break;
                x[p] = ml[p * kRows];
                load_part<D>(y[p], from + p * kRows * D);
            }
            uint32_t signs = 0;
#pragma unroll
            for (int p = 0; p < kFew; ++p)
                if (p < f.parts) top.y = fmaxf(top.y, x[p].x), signs |= __float_as_uint(x[p].y);
            based = signs >> 31;
            if (__builtin_expect(based, 0)) {
                top.y = -INFINITY;
#pragma unroll
                for (int p = 0; p < kFew; ++p)
                    if (p < f.parts) raise(reference_of(x[p]));
#pragma unroll
                for (int p = 0; p < kFew; ++p)
                    if (p < f.parts) x[p].x = above(reference_of(x[p]), top, a.scale_log2);
            }
            const float from_top = based ? 0.f : top.y;
#pragma unroll
            for (int p = 0; p < kFew; ++p) {
                if (p >= f.parts) break;
                if (x[p].y == 0.f) continue;
                const float w = ex2(x[p].x - from_top);
                l = fmaf(fabsf(x[p].y), w, l);
#pragma unroll
                for (int e = 0; e < W; ++e) acc[e] = fmaf(y[p][e], w, acc[e]);
            }
        } else {
            float2 x[kMostParts / 32];
            uint32_t signs = 0;
#pragma unroll
            for (int e = 0; e < kMostParts / 32; ++e) {
                const int p = lane + 32 * e;
                x[e] = p < f.parts ? ml[int64_t(p) * kRows] : make_float2(-INFINITY, 0.f);
                top.y = fmaxf(top.y, x[e].x);
                signs |= __float_as_uint(x[e].y);
            }
            based = __any_sync(0xffffffffu, signs >> 31);
            if (__builtin_expect(based, 0)) {
                top.y = -INFINITY;
#pragma unroll
                for (int e = 0; e < kMostParts / 32; ++e) raise(reference_of(x[e]));
#pragma unroll
                for (int o = 16; o; o >>= 1)
                    raise(make_float2(__shfl_xor_sync(0xffffffffu, top.x, o), __shfl_xor_sync(0xffffffffu, top.y, o)));
#pragma unroll
                for (int e = 0; e < kMostParts / 32; ++e)
                    x[e].x = above(reference_of(x[e]), top, a.scale_log2);
            } else {
#pragma unroll
                for (int o = 16; o; o >>= 1) top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, o));
            }
            const float from_top = based ? 0.f : top.y;
            float w[kMostParts / 32];
#pragma unroll
            for (int e = 0; e < kMostParts / 32; ++e) {
                w[e] = x[e].y == 0.f ? 0.f : ex2(x[e].x - from_top);
                l += x[e].y == 0.f ? 0.f : fabsf(x[e].y) * w[e];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll 1
            for (int p0 = 0; p0 < f.parts; p0 += kFew) {
                float y[kFew][W];
#pragma unroll
                for (int i = 0; i < kFew; ++i) {
                    if (p0 + i >= f.parts) break;
                    load_part<D>(y[i], from + int64_t(p0 + i) * kRows * D);
                }
#pragma unroll
                for (int i = 0; i < kFew; ++i) {
                    const int p = p0 + i;
                    const float wp = __shfl_sync(0xffffffffu, p < 32 ? w[0] : w[1], p & 31);
                    const float lp = __shfl_sync(0xffffffffu, p < 32 ? x[0].y : x[1].y, p & 31);
                    if (p >= f.parts || lp == 0.f) continue;
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[e] = fmaf(y[i][e], wp, acc[e]);
                }
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int h = f.hk * a.group + head;
        uint16_t *o = a.o + (int64_t(f.t0) + at) * a.o_stride + int64_t(h) * D + lane * V;
#pragma unroll
        for (int e = 0; e < W; e += V) {
            uint32_t r[V / 2];
#pragma unroll
            for (int c = 0; c < V; c += 2)
                r[c / 2] = gdn::f32_to_bf16(acc[e + c] * inv) | uint32_t(gdn::f32_to_bf16(acc[e + c + 1] * inv)) << 16;
            if constexpr (V == 4)
                *reinterpret_cast<uint2 *>(o + e * 32) = make_uint2(r[0], r[1]);
            else
                *reinterpret_cast<uint32_t *>(o + e * 32) = r[0];
        }
        if (lane == 0 && a.lse)
            a.lse[(int64_t(f.t0) + at) * a.h_q + h] =
                l == 0.f ? -INFINITY : fmaf(a.scale_log2, top.x, top.y + log2f(l)) * 0.6931471805599453f;
    }
}

// ---- the workspace's keys and values: cached positions as bf16 (exactly: 4 bits times a power of two), then the new rows

constexpr int kGatherRows = 32, kGatherThreads = 256;  // rows of a CTA at most

struct GatherArgs {
    kv8_cache c;
    int32_t layer, page_shift, rows;  // rows of a CTA, a power of two
    prompt::Requests rq;
    const int32_t *table;
    int64_t table_stride;
    const uint16_t *k, *v;
    int64_t k_stride, v_stride;
    uint16_t *out;  // [2][h_kv][kv_capacity][d]
    uint32_t *status;
};

__device__ __forceinline__ uint32_t bf16x2_scaled(uint16_t codes, float f) {
    const float2 x = f32x2_of(codes);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y * f), "f"(x.x * f));
    return r;
}

__global__ void __launch_bounds__(kGatherThreads) kv8_gather_kernel(const __grid_constant__ GatherArgs a) {
    gdn::pdl_enter();
    __shared__ prompt::Scan<kGatherThreads> scan;
    // of each row: its request and position; then a page (-1: a new row, -2: nothing, -3: zeros) and the place in it or
    // the row
    __shared__ int who[kGatherRows], place[kGatherRows];
    const int tid = threadIdx.x;
    const int64_t w0 = int64_t(blockIdx.x) * a.rows;
    for (int i = tid; i < a.rows; i += kGatherThreads) who[i] = -2;
    {
        const int chunk = (a.rq.B + kGatherThreads - 1) / kGatherThreads, r0 = min(a.rq.B, tid * chunk),
                  r1 = min(a.rq.B, r0 + chunk);
        long long none = 0, kv = 0, none_all, kv_all;
        for (int r = r0; r < r1; ++r) kv += prompt::kv_rows_of(prompt::request_of(a.rq, r));
        const long long mine = kv;
        prompt::scan2<kGatherThreads>(scan, none, kv, none_all, kv_all);
        // what the last tile reads behind the last request is in masked places, but had better not be NaN there
        if (tid < a.rows && w0 + tid >= kv_all && w0 + tid < min(kv_all + kTile, (long long)a.rq.kv_capacity))
            who[tid] = -3;
        if (kv < w0 + a.rows && kv + mine > w0)
            for (int r = r0; r < r1; ++r) {
                const long long n = prompt::kv_rows_of(prompt::request_of(a.rq, r));
                const long long from = max((long long)w0, kv), to = min((long long)w0 + a.rows, kv + n);
                if (kv + n <= a.rq.kv_capacity)  // (the attention refuses those that do not fit)
                    for (long long w = from; w < to; ++w) {
                        who[w - w0] = r;
                        place[w - w0] = int(w - kv);
                    }
                kv += n;
            }
    }
    __syncthreads();
    if (tid < a.rows && who[tid] >= 0) {
        const int r = who[tid], t = place[tid];
        const prompt::Request q = prompt::request_of(a.rq, r);
        if (t >= q.len) {
            who[tid] = -1;
            place[tid] = q.t0 + t - q.len;
        } else if (a.c.window && t <= q.len - a.c.window) {
            // nobody sees it; but a tile reads it, this request's first or the last one of the request before
            who[tid] = t / kTile == (q.len + 1 - a.c.window) / kTile || t < kTile ? -3 : -2;
        } else {
            const int p = a.table[int64_t(r) * a.table_stride + (t >> a.page_shift)];
            const bool bad = p < 0 || p >= a.c.num_pages;
            if (bad) gdn::set_status(a.status, GDN_DEV_PAGE_OOR);
            who[tid] = bad ? -3 : p;
        }
    }
    __syncthreads();
    const int d = a.c.d, h_kv = a.c.h_kv, T = a.c.page_tokens;
    const int per = d / 16, shift = 31 - __clz(per);  // pieces of 16 channels a row
    const int row_shift = 31 - __clz(a.rows), items = 2 * h_kv * a.rows * per;
#pragma unroll 4
    for (int i = tid; i < items; i += kGatherThreads) {
        const int ch = (i & (per - 1)) * 16, w = (i >> shift) & (a.rows - 1), hv = i >> (shift + row_shift);
        const int is_v = hv >= h_kv, h = hv - is_v * h_kv;
        const int p = who[w], at = place[w];
        if (p == -2) continue;
        uint4 lo, hi;
        if (p >= 0) {
            const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(
                a.c.kv + int64_t(p) * a.c.page_stride + int64_t(a.layer) * a.c.layer_stride +
                (int64_t(hv) * T + (at & (T - 1))) * d + ch));
            const float f = a.c.scale[int64_t(p) * a.c.scale_page_stride + int64_t(a.layer) * a.c.scale_layer_stride +
                                      2 * h + is_v];
            lo = make_uint4(bf16x2_scaled(uint16_t(x.x), f), bf16x2_scaled(uint16_t(x.x >> 16), f),
                            bf16x2_scaled(uint16_t(x.y), f), bf16x2_scaled(uint16_t(x.y >> 16), f));
            hi = make_uint4(bf16x2_scaled(uint16_t(x.z), f), bf16x2_scaled(uint16_t(x.z >> 16), f),
                            bf16x2_scaled(uint16_t(x.w), f), bf16x2_scaled(uint16_t(x.w >> 16), f));
        } else if (p == -3) {
            lo = hi = make_uint4(0, 0, 0, 0);
        } else {
            const uint4 *x = reinterpret_cast<const uint4 *>((is_v ? a.v + at * a.v_stride : a.k + at * a.k_stride) +
                                                             int64_t(h) * d + ch);
            lo = x[0];
            hi = x[1];
        }
        uint4 *o = reinterpret_cast<uint4 *>(a.out + (int64_t(hv) * a.rq.kv_capacity + w0 + w) * d + ch);
        o[0] = lo;
        o[1] = hi;
    }
}

// ---- host

// Rows [rows][heads][d] of bf16, boxes of 64 channels, `box_heads` heads and `box_rows` rows, swizzled.
bool encode_rows(CUtensorMap *m, const uint16_t *p, int d, int heads, int64_t rows, int64_t head_stride,
                 int64_t row_stride, int box_heads, int box_rows) {
    const gdn_host::EncodeTiledFn fn = gdn_host::encode_tiled();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(rows)};
    const cuuint64_t strides[2] = {cuuint64_t(head_stride) * 2, cuuint64_t(row_stride) * 2};
    const cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)};
    const cuuint32_t elem[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(p), dims, strides, box, elem,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
    int64_t units;
    int per_tile, splits, part_tiles, rows;
};
Plan plan_of(int h_q, int h_kv, int d, int window, int32_t B, int32_t row_capacity, int32_t max_len, int32_t max_rows,
             int64_t total_len) {
    Plan p{};
    p.per_tile = kTile / (h_q / h_kv);
    p.rows = (d == 256 ? 1 : 2) * kTile;
    const int64_t per_unit = int64_t(d == 256 ? 1 : 2) * p.per_tile;
    const int64_t each = int64_t(B) * ((max_rows + per_unit - 1) / per_unit), all = row_capacity / per_unit + B;
    p.units = h_kv * (each < all ? each : all);
    int64_t seen = int64_t(max_len) + max_rows;
    if (window && window + per_unit < seen) seen = window + per_unit + kTile;
    const int64_t tiles = (seen + kTile - 1) / kTile;
    // Work is cut where SMs would idle, into parts of up to tiles / i tiles.  All units share the SMs; units about as long
    // as one another run in full waves; the longest, which start first, matter where they are not small beside an SM's
    // share.  A unit's ends cost as much as kEnds tiles, those of a part, whose sums are written and read again, kPartEnds.
    // (8 requests of 60..2,048 rows behind 512..32,768 positions, 32/8 heads of 128: 1,270 us whole, 1,144 with 3 for
    // the long ones; 8 prompts of 512..12,000 rows, 32/4 heads: 1,050 whole, 1,490 with 7; one of 2,000 rows, 4/1 heads
    // of 128: 33.6 whole, 21.2 with 4; two of 1,500 and 3,000, 8/1 heads of 256: 48.4 whole, 62.1 with 2.)
    const double rows = double(row_capacity) / B;
    double avg = ((total_len < int64_t(B) * max_len ? double(total_len) / B : double(max_len)) + 0.5 * rows) / kTile + 1.0;
    if (max_len == 0) avg = sqrt(avg * (0.5 * tiles + 1.0));  // of prompts: long ones have more units too
    if (avg > tiles) avg = double(tiles);
    int64_t s = 1;
    double best = 0.0;
    for (int64_t i = 1; p.units && i <= kMostParts && (i == 1 || i <= tiles / kLeast); ++i) {
        const double ends = i > 1 ? kPartEnds : kEnds, longest = double(tiles) / i + kEnds;
        const double parts = avg * i > tiles ? avg * i / tiles : 1.0;
        double cost;
        if (avg > 0.75 * tiles) {
            cost = ceil(double(p.units) * i / kSms) * (avg / i + ends);
        } else {
            cost = p.units * (avg + (parts > 1.0 ? ends : kEnds) * parts) / kSms;
            if (i == 1 && longest < 0.25 * cost) break;
            cost += 0.3 * longest;
        }
        if (cost < longest) cost = longest;
        if (i > 1) cost = 1.05 * (cost + kJoinCost);
        if (i == 1 || cost < best) {
            best = cost;
            s = i;
        }
    }
    p.part_tiles = int((tiles + s - 1) / s);
    p.splits = int(s);
    return p;
}
// (at the end a status word, for calls without one: by it the join knows that units' records were written)
size_t part_bytes(const Plan &p, int d) {
    return p.splits > 1 ? size_t(p.units) * (size_t(p.splits) * p.rows * (size_t(d) * 4 + 8) + sizeof(Info)) + 16 : 0;
}
size_t kv_bytes(const kv8_cache *c, int64_t rows) { return size_t(rows) * c->h_kv * c->d * 4; }

template <int D>
int launch(const Args &a, const Plan &p, cudaStream_t st) {
    using C = Cfg<D>;
    // What its warps take from one another is shared out of this many registers (looked at once: it is the code's).
    static std::atomic<bool> looked{false};
    if (!looked.load(std::memory_order_relaxed)) {
        cudaFuncAttributes have;
        if (cudaFuncGetAttributes(&have, prompt_attend_kernel<D>) != cudaSuccess || have.numRegs != C::kLaunchRegs)
            return GDN_ERR_CUDA;
        looked.store(true, std::memory_order_relaxed);
    }
    // for every launch: the limit is the current device's
    if (cudaFuncSetAttribute(prompt_attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
        cudaSuccess)
        return GDN_ERR_CUDA;
    const int rc = gdn_host::launch_pdl(prompt_attend_kernel<D>, dim3(unsigned(p.units), unsigned(p.splits)),
                                        dim3(C::kThreads), C::kSmem, st, a);
    if (rc != GDN_OK || p.splits == 1) return rc;
    const dim3 grid(unsigned(p.units), unsigned(p.rows / a.join_rows));
    return p.splits > kFew ? gdn_host::launch_pdl(prompt_join_kernel<D, true>, grid, dim3(256), 0, st, a)
                           : gdn_host::launch_pdl(prompt_join_kernel<D, false>, grid, dim3(256), 0, st, a);
}

int run(Args &a, const Plan &p, int d, float sm_scale, uint8_t *parts, cudaStream_t st) {
    a.per_tile = p.per_tile;
    a.splits = p.splits;
    a.part_tiles = p.part_tiles;
    // Rows of a CTA of the join: of few rows it is latency, of many CTAs to start (whole calls: 8 chunks of 60 to 2,048
    // rows 1,174 us with 8, 1,144 with 32, 1,140 with 64; 3 of 100 to 300 74.2 with 32, 75.9 with 64; 32 rows behind
    // 32,000 tokens 55.8 with 8, 80 with 32).
    a.join_rows = p.units * p.rows >= 2 * kSms * 32 ? 32 : 8;
    a.negate = sm_scale < 0.f;
    const float c = fabsf(sm_scale) * 1.4426950408889634f;
    a.scale_log2 = c == 0.f ? 0x1p-149f : c;  // a masked score times zero would be no number; times this, any score is 0
    if (p.splits > 1) {
        const size_t rows = size_t(p.units) * p.splits * p.rows;
        a.ws_o = reinterpret_cast<float *>(parts);
        a.ws_ml = reinterpret_cast<float2 *>(a.ws_o + rows * d);
        a.info = reinterpret_cast<Info *>(a.ws_ml + rows);
        if (!a.status) {
            a.status = reinterpret_cast<uint32_t *>(a.info + p.units);
            if (cudaMemsetAsync(a.status, 0, sizeof(uint32_t), st) != cudaSuccess) return GDN_ERR_CUDA;
        }
    }
    if (d == 64) return launch<64>(a, p, st);
    if (d == 128) return launch<128>(a, p, st);
    return launch<256>(a, p, st);
}

int check_dims(const attn_dims *c) {
    if (!c) return GDN_ERR_NULL;
    if (!(c->d == 64 || c->d == 128 || c->d == 256)) return GDN_ERR_SHAPE;
    if (c->h_kv <= 0 || c->h_q <= 0 || c->h_q % c->h_kv != 0 || c->h_q / c->h_kv > 64 || c->h_kv > 1024)
        return GDN_ERR_SHAPE;
    if (c->window < 0 || !isfinite(c->sm_scale)) return GDN_ERR_ARG;
    return GDN_OK;
}
constexpr int64_t kMostUnits = (int64_t(1) << 31) - 1;
// A unit's longest waits are for all of its tiles, about 2 us each: half a second of the bound's one.
constexpr int64_t kMostPositions = int64_t(1) << 25;

}  // namespace

extern "C" size_t attn_prompts_workspace_bytes(const attn_dims *dims, int32_t B, int32_t row_capacity,
                                               int32_t max_rows) {
    if (check_dims(dims) != GDN_OK || B <= 0 || B > 65535 || row_capacity < 0 || max_rows <= 0 ||
        max_rows > kMostPositions)
        return 0;
    return part_bytes(plan_of(dims->h_q, dims->h_kv, dims->d, dims->window, B, row_capacity, 0, max_rows, 0), dims->d);
}

static int prompts(const attn_dims *dims, int32_t B, int32_t row_capacity, const int32_t *cu_rows, const gdn_bf16 *q,
                   int64_t q_stride, const gdn_bf16 *k, int64_t k_stride, const gdn_bf16 *v, int64_t v_stride,
                   gdn_bf16 *o, int64_t o_stride, float *lse, int32_t max_rows, void *workspace,
                   size_t workspace_bytes, uint32_t *dev_status, uint64_t wait_ns, int32_t withhold, void *stream) {
    const int bad = check_dims(dims);
    if (bad != GDN_OK) return bad;
    if (B < 0 || B > 65535 || row_capacity < 0 || max_rows < 0 || max_rows > kMostPositions) return GDN_ERR_ARG;
    if (B == 0 || max_rows == 0 || row_capacity == 0) return GDN_OK;
    if (!cu_rows || !q || !k || !v || !o) return GDN_ERR_NULL;
    if (!gdn_host::kv8_rows_ok(q, q_stride, dims->h_q, dims->d) ||
        !gdn_host::kv8_rows_ok(k, k_stride, dims->h_kv, dims->d) ||
        !gdn_host::kv8_rows_ok(v, v_stride, dims->h_kv, dims->d) ||
        !gdn_host::kv8_rows_ok(o, o_stride, dims->h_q, dims->d))
        return GDN_ERR_ARG;
    const Plan p = plan_of(dims->h_q, dims->h_kv, dims->d, dims->window, B, row_capacity, 0, max_rows, 0);
    const size_t need = part_bytes(p, dims->d);
    if (p.units > kMostUnits) return GDN_ERR_ARG;
    if (need && (!workspace || workspace_bytes < need)) return GDN_ERR_WORKSPACE;
    if (need && !gdn_host::aligned16(workspace)) return GDN_ERR_ARG;
    Args a{};
    if (!encode_rows(&a.mq, q, dims->d, dims->h_q, row_capacity, dims->d, q_stride, dims->h_q / dims->h_kv,
                     p.per_tile) ||
        !encode_rows(&a.mk, k, dims->d, dims->h_kv, row_capacity, dims->d, k_stride, 1, kTile) ||
        !encode_rows(&a.mv, v, dims->d, dims->h_kv, row_capacity, dims->d, v_stride, 1, kTile))
        return GDN_ERR_CUDA;
    a.rq = {B, row_capacity, max_rows, 0, 0, 0, cu_rows, nullptr};
    a.h_q = dims->h_q;
    a.h_kv = dims->h_kv;
    a.group = dims->h_q / dims->h_kv;
    a.window = dims->window;
    a.o = o;
    a.o_stride = o_stride;
    a.lse = lse;
    a.v = v;
    a.v_head = dims->d;
    a.v_row = v_stride;
    a.status = dev_status;
    a.wait_ns = wait_ns;
    a.withhold = withhold;
    return run(a, p, dims->d, dims->sm_scale, static_cast<uint8_t *>(workspace), static_cast<cudaStream_t>(stream));
}

extern "C" int attn_prompts(const attn_dims *dims, int32_t B, int32_t row_capacity, const int32_t *cu_rows,
                            const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k, int64_t k_stride,
                            const gdn_bf16 *v, int64_t v_stride, gdn_bf16 *o, int64_t o_stride, float *lse,
                            int32_t max_rows, void *workspace, size_t workspace_bytes, uint32_t *dev_status,
                            void *stream) {
    return prompts(dims, B, row_capacity, cu_rows, q, q_stride, k, k_stride, v, v_stride, o, o_stride, lse, max_rows,
                   workspace, workspace_bytes, dev_status, gdn::kWaitLimitNs, 0, stream);
}

extern "C" int attn_selftest_prompts_timeout(const attn_dims *dims, int32_t B, int32_t row_capacity,
                                             const int32_t *cu_rows, const gdn_bf16 *q, int64_t q_stride,
                                             const gdn_bf16 *k, int64_t k_stride, const gdn_bf16 *v, int64_t v_stride,
                                             gdn_bf16 *o, int64_t o_stride, int32_t max_rows, void *workspace,
                                             size_t workspace_bytes, uint32_t *dev_status, uint64_t limit_ns,
                                             void *stream) {
    if (limit_ns == 0 || limit_ns > gdn::kWaitLimitNs) return GDN_ERR_ARG;
    return prompts(dims, B, row_capacity, cu_rows, q, q_stride, k, k_stride, v, v_stride, o, o_stride, nullptr,
                   max_rows, workspace, workspace_bytes, dev_status, limit_ns, 1, stream);
}

// Rows of the workspace's keys: every request's earlier positions and new rows.
static int64_t kv_rows(int32_t B, int32_t row_capacity, int32_t max_len, int64_t total_len) {
    const int64_t most = int64_t(B) * max_len;
    return (total_len < most ? total_len : most) + row_capacity;
}

extern "C" size_t kv8_chunk_workspace_bytes(const kv8_cache *cache, int32_t B, int32_t row_capacity, int32_t max_len,
                                            int32_t max_rows, int64_t total_len) {
    if (gdn_host::kv8_check(cache) != GDN_OK || B <= 0 || B > 65535 || row_capacity < 0 || max_len < 0 ||
        max_rows <= 0 || int64_t(max_len) + max_rows > kMostPositions || total_len < 0)
        return 0;
    const int64_t rows = kv_rows(B, row_capacity, max_len, total_len);
    if (rows >= gdn_host::kKv8MaxLen) return 0;
    return kv_bytes(cache, rows) +
           part_bytes(plan_of(cache->h_q, cache->h_kv, cache->d, cache->window, B, row_capacity, max_len, max_rows,
                              total_len),
                      cache->d);
}

extern "C" int kv8_chunk(const kv8_cache *cache, int32_t layer, int32_t B, int32_t row_capacity,
                         const int32_t *cu_rows, const int32_t *cache_len, const int32_t *table, int32_t table_pages,
                         int64_t table_stride, const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k_new,
                         int64_t k_stride, const gdn_bf16 *v_new, int64_t v_stride, gdn_bf16 *o, int64_t o_stride,
                         float *lse, int32_t max_len, int32_t max_rows, int64_t total_len, void *workspace,
                         size_t workspace_bytes, uint32_t *dev_status, void *stream) {
    const int bad = gdn_host::kv8_check(cache);
    if (bad != GDN_OK) return bad;
    if (layer < 0 || layer >= cache->num_layers || B < 0 || B > 65535 || row_capacity < 0 || table_pages < 0 ||
        table_stride < 0 || max_len < 0 || max_rows < 0 || int64_t(max_len) + max_rows > kMostPositions ||
        total_len < 0)
        return GDN_ERR_ARG;
    if (B == 0 || max_rows == 0 || row_capacity == 0) return GDN_OK;
    if (!cu_rows || !cache_len || (!table && table_pages > 0) || !q || !k_new || !v_new || !o) return GDN_ERR_NULL;
    if (!gdn_host::kv8_rows_ok(q, q_stride, cache->h_q, cache->d) ||
        !gdn_host::kv8_rows_ok(k_new, k_stride, cache->h_kv, cache->d) ||
        !gdn_host::kv8_rows_ok(v_new, v_stride, cache->h_kv, cache->d) ||
        !gdn_host::kv8_rows_ok(o, o_stride, cache->h_q, cache->d))
        return GDN_ERR_ARG;
    const int64_t rows = kv_rows(B, row_capacity, max_len, total_len);
    const Plan p = plan_of(cache->h_q, cache->h_kv, cache->d, cache->window, B, row_capacity, max_len, max_rows,
                           total_len);
    // (row numbers of the workspace are the copy engine's 32-bit coordinates)
    if (rows >= gdn_host::kKv8MaxLen || p.units > kMostUnits) return GDN_ERR_ARG;
    const size_t need = kv_bytes(cache, rows) + part_bytes(p, cache->d);
    if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
    if (!gdn_host::aligned16(workspace)) return GDN_ERR_ARG;
    uint16_t *dense = static_cast<uint16_t *>(workspace);
    const int64_t half = int64_t(cache->h_kv) * rows * cache->d;
    Args a{};
    if (!encode_rows(&a.mq, q, cache->d, cache->h_q, row_capacity, cache->d, q_stride, cache->h_q / cache->h_kv,
                     p.per_tile) ||
        !encode_rows(&a.mk, dense, cache->d, cache->h_kv, rows, rows * cache->d, cache->d, 1, kTile) ||
        !encode_rows(&a.mv, dense + half, cache->d, cache->h_kv, rows, rows * cache->d, cache->d, 1, kTile))
        return GDN_ERR_CUDA;
    GatherArgs g{};
    g.c = *cache;
    g.layer = layer;
    g.page_shift = 31 - __builtin_clz(unsigned(cache->page_tokens));
    g.rq = {B, row_capacity, max_rows, max_len, rows, int64_t(table_pages) * cache->page_tokens, cu_rows, cache_len};
    g.table = table;
    g.table_stride = table_stride;
    g.k = k_new;
    g.v = v_new;
    g.k_stride = k_stride;
    g.v_stride = v_stride;
    g.out = dense;
    g.status = dev_status;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // Rows of a CTA: as many as leave six CTAs for an SM (14,600 positions, 4 heads of 64: 9.9 us with 8, 8.8 with 16,
    // 9.1 with 32, 12.9 with 64; 262,656 positions, 2 heads of 256: 143 with 16, 134 with 32, 142 with 128).
    g.rows = rows >= 6 * kSms * 32 ? 32 : rows >= 6 * kSms * 8 ? 16 : 8;
    const int rc = gdn_host::launch_pdl(kv8_gather_kernel, dim3(unsigned((rows + g.rows - 1) / g.rows)),
                                        dim3(kGatherThreads), 0, st, g);
    if (rc != GDN_OK) return rc;
    a.rq = g.rq;
    a.h_q = cache->h_q;
    a.h_kv = cache->h_kv;
    a.group = cache->h_q / cache->h_kv;
    a.window = cache->window;
    a.o = o;
    a.o_stride = o_stride;
    a.lse = lse;
    a.v = dense + half;
    a.v_head = rows * cache->d;
    a.v_row = cache->d;
    a.table = table;
    a.table_stride = table_stride;
    a.page_shift = g.page_shift;
    a.num_pages = cache->num_pages;
    a.status = dev_status;
    a.wait_ns = gdn::kWaitLimitNs;
    return run(a, p, cache->d, cache->sm_scale, static_cast<uint8_t *>(workspace) + kv_bytes(cache, rows), st);
}
