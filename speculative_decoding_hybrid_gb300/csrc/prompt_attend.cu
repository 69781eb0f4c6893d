// Causal attention of packed rows over dense keys and values (sm_103a): whole
// prompts, and chunks of new rows behind earlier positions of a paged 8-bit cache.
//
// A query tile is 128 rows of the tensor cores: 128 / group positions with all
// query heads of a kv head side by side, so a key is read once for the group.  Per tile of
// 128 positions
//   S = Q K^T                 scores, fp32 in tensor memory, a row in a lane
//   p = 2^(c S - m)           a thread a row: its maximum, exponentials and sum in registers
//   O += P V                  P in bf16 from tensor memory, where S lay
// with m moved (and O rescaled) only when a score passes it by 2^8.  At d <= 128 a CTA has
// two query tiles that share the keys, so one's softmax runs beside the other's products; at
// d = 256, where one tile's O takes half of tensor memory, the softmax of a tile of positions
// runs beside the products of its neighbours.
#include "kv8_math.cuh"
#include "prompt.cuh"
#include "tmap.cuh"

namespace {

using namespace kv8;

constexpr int kTile = 128;   // positions a tile, and rows of a query tile
constexpr int kSms = 152;
constexpr float kSlack = 8.f;
constexpr int kLeast = 4;    // tiles a part of a cut unit has at least
constexpr int kMostParts = 64;
constexpr int kAhead = 4;    // tiles of values that the ring can hold: 8 slots, every other one of values

struct Info {                // a unit's parts, for the join: parts 0: nothing to join
    int t0, tok0, n, hk, parts, pad[3];
};

struct Args {
    CUtensorMap mq, mk, mv;
    prompt::Requests rq;
    int32_t h_q, h_kv, group, per_tile;  // per_tile: positions a query tile
    int32_t window, splits, negate;
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
    static constexpr int kRoom = 227 * 1024 - 3072 - kStages * kQTile;
    static constexpr int kSlots = kRoom / kSlot > 8 ? 8 : kRoom / kSlot;
    static constexpr int kSmem = kStages * kQTile + kSlots * kSlot + 1024;
    static constexpr int kSoft = 128 * kStages;  // softmax threads
    static constexpr int kThreads = kSoft + 128;
    static_assert(kSlots >= 2 * kPieces + 1 && kSlots <= 2 * kAhead * kPieces, "does not fit an SM");
};

struct Unit {
    int t0, n, len, r, tok0, parts;
    int64_t kv0;  // its first position's row of the keys
};

template <int D>
struct Shared {
    using C = Cfg<D>;
    uint64_t full[C::kSlots], empty[C::kSlots], s_full[2], o_done[2], q_full, drain;  // one arrival
    uint64_t p_ready[2];  // of four warps
    uint64_t v_sent[kAhead];        // masked tiles in turn: the copy of the values is under way ...
    uint64_t v_ok[kAhead], pages;   // ... and looked through (of the two guards)
    prompt::Scan<C::kThreads> scan;
    Unit u;
    uint32_t tmem;
    int found, fix, bad;
};

// Ring positions of the loads of n tiles, in the order the products use them: K0 K1 V0 K2 V1 ... V(n-1).
__device__ __forceinline__ int k_pos(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_pos(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

// What a unit's part sums: tiles tile0 .. of the request's positions, `tiles` of them, of which query tile st uses the
// first ns[st].
struct Span {
    int tile0, tiles, ns[2];
};
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
    const int from = int(int64_t(all) * part / u.parts), to = int(int64_t(all) * (part + 1) / u.parts);
    s.tile0 = tile0 + from;
    s.tiles = to - from;
#pragma unroll
    for (int st = 0; st < 2; ++st) {
        const int first = u.tok0 + st * a.per_tile, last = min(first + a.per_tile, u.n) - 1;
        s.ns[st] = st < stages && first < u.n ? min(max((u.len + last) / kTile + 1 - s.tile0, 0), s.tiles) : 0;
    }
    return s;
}
// Whether some row of the unit does not see all of a tile's positions.
__device__ __forceinline__ bool masked(const Args &a, const Unit &u, int stages, int tile) {
    const int last = min(u.tok0 + stages * a.per_tile, u.n) - 1;
    return tile * kTile + kTile - 1 > u.len + u.tok0 || (a.window && tile * kTile <= u.len + last - a.window);
}

// Adds to a row's 32 sums the values that are not finite at positions of masked tiles that it sees: they were taken out
// of the tiles, where a zero weight would not have kept them from the other rows.
template <int D>
__device__ __noinline__ void add_special(const Args &a, const Unit &u, const Span &s, int stages, int hk, int pos,
                                         int ch, float *o) {
    for (int j = 0; j < s.tiles; ++j) {
        const int tile = s.tile0 + j;
        if (!masked(a, u, stages, tile)) continue;
        const int from = max(tile * kTile, a.window ? pos - a.window + 1 : 0), to = min(tile * kTile + kTile - 1, pos);
        for (int t = from; t <= to; ++t) {
            const uint16_t *v = a.v + (u.kv0 + t) * a.v_row + int64_t(hk) * a.v_head + ch;
            for (int c = 0; c < 32; ++c) {
                const float x = gdn::bf16_to_f32(v[c]);
                if (!(fabsf(x) < INFINITY)) o[c] += x;
            }
        }
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
    constexpr int kCopyWarp = C::kSoft / 32, kMmaWarp = kCopyWarp + 1, kGuard = kCopyWarp + 2;
    if (warp == kMmaWarp) {
        tc::tmem_alloc(&s.tmem, 512);
    } else if (warp == kCopyWarp && lane == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            gdn::mbar_init(s.full + i, 1);
            gdn::mbar_init(s.empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            gdn::mbar_init(s.s_full + i, 1);
            gdn::mbar_init(s.o_done + i, 1);
            gdn::mbar_init(s.p_ready + i, 4);
        }
        gdn::mbar_init(&s.q_full, 1);
        gdn::mbar_init(&s.drain, 1);
        for (int i = 0; i < kAhead; ++i) {
            gdn::mbar_init(s.v_sent + i, 1);
            gdn::mbar_init(s.v_ok + i, 2);
        }
        gdn::mbar_init(&s.pages, 2);
        s.found = s.fix = s.bad = 0;
    }
    gdn::pdl_wait();
    __syncthreads();

    // ---- this CTA's unit: the later rows of a request, which see most, come first
    const int hk = blockIdx.x % a.h_kv, rank = blockIdx.x / a.h_kv, part = blockIdx.y;
    const int per_unit = kStages * a.per_tile;
    {
        const int chunk = (a.rq.B + C::kThreads - 1) / C::kThreads, r0 = tid * chunk, r1 = min(a.rq.B, r0 + chunk);
        long long blocks = 0, kv = 0, all, kv_all;
        for (int r = r0; r < r1; ++r) {
            const prompt::Request q = prompt::request_of(a.rq, r);
            if (q.bad && blockIdx.x == 0 && part == 0) gdn::set_status(a.status, GDN_DEV_ROWS_BAD);
            blocks += (q.n + per_unit - 1) / per_unit;
            kv += prompt::kv_rows_of(q);
        }
        const long long mine = blocks;
        prompt::scan2<C::kThreads>(s.scan, blocks, kv, all, kv_all);
        if (blocks <= rank && rank < blocks + mine) {
            for (int r = r0; r < r1; ++r) {
                const prompt::Request q = prompt::request_of(a.rq, r);
                const int nb = (q.n + per_unit - 1) / per_unit;
                if (rank < blocks + nb) {
                    Unit u;
                    u.t0 = q.t0;
                    u.n = q.n;
                    u.len = q.len;
                    u.r = r;
                    u.tok0 = (nb - 1 - int(rank - blocks)) * per_unit;
                    u.kv0 = a.rq.kv_capacity ? kv : int64_t(q.t0);
                    int tile0;
                    const int tiles = unit_tiles(a, u, kStages, tile0);
                    u.parts = min(a.splits, max(1, tiles / kLeast));
                    s.u = u;
                    s.found = !a.rq.kv_capacity || kv + q.len + q.n <= a.rq.kv_capacity;
                    break;
                }
                blocks += nb;
                kv += prompt::kv_rows_of(q);
            }
        }
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tm = s.tmem;
    const Unit u = s.u;
    if (!s.found || part >= u.parts) {
        if (tid == 0 && a.info && part == 0) a.info[blockIdx.x].parts = 0;
        __syncthreads();
        if (warp == kMmaWarp) tc::tmem_dealloc(tm, 512);
        return;
    }
    const Span sp = span_of(a, u, kStages, part);
    const int nt = sp.tiles;
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *s_q = sm, *s_ring = sm + kStages * C::kQTile;

    if (warp < kCopyWarp) {
        // ---- softmax: a thread a row
        const int st = warp >> 2;
        const int row = (warp & 3) * 32 + lane, tok = row / a.group, head = row - tok * a.group;
        const int at = u.tok0 + st * a.per_tile + tok;
        const bool valid = tok < a.per_tile && at < u.n;
        const int pos = u.len + at;
        const uint32_t lanes = uint32_t(warp & 3) << 21;
        const uint32_t t_o = tm + 256 + (kStages == 2 ? st * D : 0) + lanes;
        const int n = sp.ns[st];
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int slot = kStages == 2 ? st : j & 1;
            ok = gdn::mbar_wait_bounded(&s.s_full[slot], (kStages == 2 ? j : j >> 1) & 1, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc::fence_after();
            const uint32_t t_s = tm + slot * kTile + lanes;
            uint32_t x[kTile];
#pragma unroll
            for (int i = 0; i < 4; ++i) tc::ld32_async(t_s + 32 * i, x + 32 * i);
            tc::ld_wait();
#pragma unroll
            for (int i = 0; i < kTile; ++i) asm volatile("" : "+r"(x[i]));
            if (masked(a, u, kStages, sp.tile0 + j)) {
                const int hi = pos - (sp.tile0 + j) * kTile, lo = a.window ? hi - a.window : -1;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int h = hi - 32 * i, b = lo - 32 * i;
                    const uint32_t up = h < 0 ? 0u : h >= 31 ? ~0u : (2u << h) - 1u;
                    const uint32_t see = b < 0 ? up : b >= 31 ? 0u : up & ~((2u << b) - 1u);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!(see >> c & 1)) x[32 * i + c] = 0xff800000u;
                }
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kTile; i += 2)
                top[(i >> 1) & 3] = fmaxf(top[(i >> 1) & 3], fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
            float z = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * a.scale_log2;
            if (!valid) z = -INFINITY;
            if (__any_sync(0xffffffffu, z > m + kSlack)) {
                const float now = fmaxf(m, z), f = ex2(m - (now == -INFINITY ? 0.f : now));
                if (j > 0) {
                    ok = gdn::mbar_wait_bounded(&s.o_done[st], (j - 1) & 1, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::fence_after();
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tc::ld32_async(t_o + c, o);
                        tc::ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            asm volatile("" : "+r"(o[i]));
                            o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        }
                        tc::st32_async(t_o + c, o);
                    }
                }
                l *= f;
                m = now;
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const f2 c2 = pair(a.scale_log2, a.scale_log2), r2 = pair(-ref, -ref);
            f2 sum[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t p[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float2 e = both(fma2(pair(x[64 * i + 2 * c], x[64 * i + 2 * c + 1]), c2, r2));
                    const float e0 = ex2(e.x), e1 = ex2(e.y);
                    sum[c & 1] = add2(sum[c & 1], pair(e0, e1));
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(p[c]) : "f"(e1), "f"(e0));
                }
                tc::st32_async(t_s + 32 * i, p);
            }
            const float2 t = both(add2(sum[0], sum[1]));
            l += t.x + t.y;
            tc::st_wait();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) arrive(&s.p_ready[slot]);
        }
        if (ok) {
            ok = gdn::mbar_wait_bounded(&s.pages, 0, a.wait_ns);
            // (with two tiles of scores ahead, the products of the last tile but one may be running too)
            if (ok && kStages == 1 && n > 1) ok = gdn::mbar_wait_bounded(&s.o_done[st], n & 1, a.wait_ns);
            if (ok && n > 0) ok = gdn::mbar_wait_bounded(&s.o_done[st], (n - 1) & 1, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
        }
        if (ok) {
            tc::fence_after();
            const bool fix = *reinterpret_cast<volatile int *>(&s.fix);
            const bool write = valid && !*reinterpret_cast<volatile int *>(&s.bad);
            const bool whole = u.parts == 1;
            const int64_t wrow = ((int64_t(blockIdx.x) * a.splits + part) * kStages + st) * kTile + row;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int h = hk * a.group + head;
            uint16_t *o_row = a.o + (int64_t(u.t0) + at) * a.o_stride + int64_t(h) * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
                uint32_t x[32];
                float o[32];
                if (n > 0) {
                    tc::ld32_async(t_o + c, x);
                    tc::ld_wait();
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    asm volatile("" : "+r"(x[i]));
                    o[i] = n > 0 && l != 0.f ? __uint_as_float(x[i]) : 0.f;
                }
                if (fix && write && n > 0) add_special<D>(a, u, sp, kStages, hk, pos, c, o);
                if (write && whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint4 w;
                        uint32_t *ww = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                                : "=r"(ww[e])
                                : "f"(o[i + 2 * e + 1] * inv), "f"(o[i + 2 * e] * inv));
                        *reinterpret_cast<uint4 *>(o_row + c + i) = w;
                    }
                } else if (write) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4 *>(a.ws_o + wrow * D + c + i) =
                            make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
            if (write && whole) {
                if (a.lse)
                    a.lse[(int64_t(u.t0) + at) * a.h_q + h] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            } else if (write) {
                a.ws_ml[wrow] = make_float2(m, l);
            }
        }
        if (!ok) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
        tc::fence_before();
    } else if (warp == kCopyWarp) {
        // ---- copies
        const bool leader = elect_one();
        bool ok = true;
        int issued = 0;
        if (leader) {
            int tiles = 0;
            for (int st = 0; st < kStages; ++st) tiles += sp.ns[st] > 0;
            gdn::mbar_arrive_expect_tx(&s.q_full, uint32_t(tiles * a.per_tile * a.group) * (D * 2));
            for (int st = 0; st < kStages; ++st)
                if (sp.ns[st] > 0)
                    for (int c = 0; c < D; c += 64)
                        gdn::tma_load_3d(s_q + st * C::kQTile + c * kTile * 2, &a.mq, c, hk * a.group,
                                         u.t0 + u.tok0 + st * a.per_tile, &s.q_full);
        }
        auto load = [&](const CUtensorMap &map, int tile, int at) {
            for (int x = 0; x < C::kPieces; ++x) {
                const int pos = at * C::kPieces + x, slot = pos % C::kSlots;
                if (pos >= C::kSlots)
                    ok = ok && gdn::mbar_wait_bounded(&s.empty[slot], (pos / C::kSlots - 1) & 1, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                if (leader) {
                    gdn::mbar_arrive_expect_tx(&s.full[slot], C::kSlot);
                    for (int c = 0; c < C::kPiece; c += 64)
                        gdn::tma_load_3d(s_ring + slot * C::kSlot + c * kTile * 2, &map, x * C::kPiece + c, hk,
                                         int(u.kv0) + tile * kTile, &s.full[slot]);
                }
                issued = pos + 1;
            }
        };
        int sent = 0;
        for (int i = 0; i <= nt && ok; ++i) {
            if (i < nt) load(a.mk, sp.tile0 + i, k_pos(i));
            if (i == 0 || !ok || (a.withhold && i == nt)) continue;
            load(a.mv, sp.tile0 + i - 1, v_pos(i - 1, nt));
            if (ok && masked(a, u, kStages, sp.tile0 + i - 1)) {
                if (leader) arrive(&s.v_sent[sent % kAhead]);
                ++sent;
            }
        }
        if (!ok) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
        // every copy has landed before the CTA leaves (on the usual path these waits are over)
        (void)gdn::mbar_wait_bounded(&s.q_full, 0, a.wait_ns);
        for (int pos = max(0, issued - C::kSlots); pos < issued; ++pos)
            (void)gdn::mbar_wait_bounded(&s.full[pos % C::kSlots], (pos / C::kSlots) & 1, a.wait_ns);
    } else if (warp == kMmaWarp) {
        // ---- products: the warp runs the loop, one elected lane issues
        const uint32_t id_s = tc::idesc_bf16(128, kTile) | (a.negate ? tc::kNegA : 0);
        constexpr uint32_t id_p = tc::idesc_bf16(128, C::kPiece) | tc::kBMnMajor;
        const uint64_t dq = tc::smem_desc(gdn::smem_u32(s_q)), dk = tc::smem_desc(gdn::smem_u32(s_ring));
        const uint64_t dv = tc::smem_desc_mn(gdn::smem_u32(s_ring), kTile * 128);
        const bool leader = elect_one();
        bool ok = gdn::mbar_wait_bounded(&s.q_full, 0, a.wait_ns);
        int guarded = 0;
        auto wait_tile = [&](int at) {
            for (int x = 0; x < C::kPieces; ++x) {
                const int pos = at * C::kPieces + x;
                ok = ok && gdn::mbar_wait_bounded(&s.full[pos % C::kSlots], (pos / C::kSlots) & 1, a.wait_ns);
            }
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after();
        };
        auto free_tile = [&](int at) {
            if (leader)
                for (int x = 0; x < C::kPieces; ++x) tc::commit(&s.empty[(at * C::kPieces + x) % C::kSlots]);
        };
        auto scores = [&](int st, int slot, int j) {
            if (!leader) return;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int pos = k_pos(j) * C::kPieces + k * 16 / C::kPiece, in = k * 16 % C::kPiece;
                tc::mma_bf16(tm + slot * kTile,
                             tc::desc_at(dq, st * C::kQTile + (k / 4) * kTile * 128 + (k % 4) * 32),
                             tc::desc_at(dk, (pos % C::kSlots) * C::kSlot + (in / 64) * kTile * 128 + (in % 64) * 2),
                             id_s, k > 0);
            }
            tc::commit(&s.s_full[slot]);
        };
        auto outputs = [&](int st, int slot, int j) {
            if (!leader) return;
#pragma unroll
            for (int x = 0; x < C::kPieces; ++x) {
                const int pos = v_pos(j, nt) * C::kPieces + x;
                const uint64_t d = tc::desc_at(dv, (pos % C::kSlots) * C::kSlot);
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    tc::mma_bf16_ts(tm + 256 + (kStages == 2 ? st * D : 0) + x * C::kPiece, tm + slot * kTile + k * 8,
                                    tc::desc_at(d, k * 2048), id_p, j > 0 || k > 0);
            }
            tc::commit(&s.o_done[st]);
        };
        auto wait_weights = [&](int slot, int phase) {
            ok = ok && gdn::mbar_wait_bounded(&s.p_ready[slot], phase & 1, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after();
        };
        auto wait_values = [&](int j) {
            wait_tile(v_pos(j, nt));
            if (masked(a, u, kStages, sp.tile0 + j)) {
                ok = ok && gdn::mbar_wait_bounded(&s.v_ok[guarded % kAhead], guarded / kAhead & 1, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                ++guarded;
            }
        };
        wait_tile(k_pos(0));
        if constexpr (kStages == 2) {
            if (ok) {
                for (int st = 0; st < 2; ++st)
                    if (sp.ns[st] > 0) scores(st, st, 0);
                free_tile(k_pos(0));
            }
            for (int j = 0; j < nt && ok; ++j) {
                if (j + 1 < nt) wait_tile(k_pos(j + 1));
                if (ok) wait_values(j);
                for (int st = 0; st < 2 && ok; ++st) {
                    if (j < sp.ns[st]) {
                        wait_weights(st, j);
                        if (!ok) break;
                        outputs(st, st, j);
                    }
                    if (st == 1) free_tile(v_pos(j, nt));
                    if (j + 1 < sp.ns[st]) scores(st, st, j + 1);
                }
                if (ok && j + 1 < nt) free_tile(k_pos(j + 1));
            }
        } else {
            if (ok) {
                scores(0, 0, 0);
                free_tile(k_pos(0));
            }
            if (nt > 1 && ok) {
                wait_tile(k_pos(1));
                if (ok) {
                    scores(0, 1, 1);
                    free_tile(k_pos(1));
                }
            }
            for (int j = 0; j < nt && ok; ++j) {
                wait_values(j);
                if (ok) wait_weights(j & 1, j >> 1);
                if (!ok) break;
                outputs(0, j & 1, j);
                free_tile(v_pos(j, nt));
                if (j + 2 < nt) {
                    wait_tile(k_pos(j + 2));
                    if (!ok) break;
                    scores(0, j & 1, j + 2);
                    free_tile(k_pos(j + 2));
                }
            }
        }
        if (!ok) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
        // no product reads shared memory after the CTA has left
        if (leader) tc::commit(&s.drain);
        __syncwarp();
        (void)gdn::mbar_wait_bounded(&s.drain, 0, a.wait_ns);
    } else {
        // ---- guards: a zero weight times what is not finite is not zero, so such values go out of masked tiles
        const int me = tid - kGuard * 32;
        bool ok = true;
        if (a.table) {
            const int T = 1 << a.page_shift;
            const int first = (a.window ? max(0, u.len + 1 - a.window) : 0) >> a.page_shift;
            const int last = u.len > 0 ? (u.len + T - 1) >> a.page_shift : 0;
            bool bad = false;
            for (int i = first + me; i < last; i += 64) {
                const int p = a.table[int64_t(u.r) * a.table_stride + i];
                bad |= p < 0 || p >= a.num_pages;
            }
            if (bad) *reinterpret_cast<volatile int *>(&s.bad) = 1;
        }
        __syncwarp();
        if (lane == 0) arrive(&s.pages);
        int seen = 0;
        for (int j = 0; j < nt && ok; ++j) {
            if (!masked(a, u, kStages, sp.tile0 + j)) continue;
            // (a copy under way: its barrier is in that copy's phase, not in an earlier one of the same parity)
            ok = gdn::mbar_wait_bounded(&s.v_sent[seen % kAhead], seen / kAhead & 1, a.wait_ns);
            bool any = false;
            for (int x = 0; x < C::kPieces && ok; ++x) {
                const int pos = v_pos(j, nt) * C::kPieces + x, slot = pos % C::kSlots;
                ok = gdn::mbar_wait_bounded(&s.full[slot], (pos / C::kSlots) & 1, a.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                uint4 *p = reinterpret_cast<uint4 *>(s_ring + slot * C::kSlot);
#pragma unroll 4
                for (int i = me; i < C::kSlot / 16; i += 64) {
                    uint4 w = p[i];
                    const uint32_t t = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu),
                                                __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
                    if (max(t >> 16, t & 0xffffu) >= 0x7f80u) {
                        w.x &= __vcmpltu2(w.x & 0x7fff7fffu, 0x7f807f80u);
                        w.y &= __vcmpltu2(w.y & 0x7fff7fffu, 0x7f807f80u);
                        w.z &= __vcmpltu2(w.z & 0x7fff7fffu, 0x7f807f80u);
                        w.w &= __vcmpltu2(w.w & 0x7fff7fffu, 0x7f807f80u);
                        p[i] = w;
                        any = true;
                    }
                }
            }
            if (any) *reinterpret_cast<volatile int *>(&s.fix) = 1;
            gdn::fence_proxy_async_smem();
            __syncwarp();
            if (ok && lane == 0) arrive(&s.v_ok[seen % kAhead]);
            ++seen;
        }
        if (!ok) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tm, 512);
    }
    if (tid == 0 && part == 0 && a.info) {
        Info f = {};
        f.t0 = u.t0;
        f.tok0 = u.tok0;
        f.n = u.n;
        f.hk = hk;
        f.parts = u.parts > 1 && !s.bad ? u.parts : 0;
        a.info[blockIdx.x] = f;
    }
}

// Joins a unit's parts: o = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p, a warp a row.
constexpr int kJoinRows = 16;
template <int D>
__global__ void __launch_bounds__(256) prompt_join_kernel(const __grid_constant__ Args a) {
    gdn::pdl_enter();
    constexpr int kRows = Cfg<D>::kStages * kTile, W = D / 32;
    const Info f = a.info[blockIdx.x];
    const uint32_t status = a.status ? *reinterpret_cast<volatile uint32_t *>(a.status) : 0;
    if (f.parts == 0 || (status & GDN_DEV_TIMEOUT)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < kJoinRows; i += 8) {
        const int row = blockIdx.y * kJoinRows + i, st = row / kTile, in = row % kTile;
        const int tok = in / a.group, head = in - tok * a.group, at = f.tok0 + st * a.per_tile + tok;
        if (tok >= a.per_tile || at >= f.n) continue;
        const int64_t base = int64_t(blockIdx.x) * a.splits * kRows + row;
        float2 x[kMostParts / 32];
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < kMostParts / 32; ++e) {
            const int p = lane + 32 * e;
            x[e] = p < f.parts ? a.ws_ml[base + int64_t(p) * kRows] : make_float2(-INFINITY, 0.f);
            top = fmaxf(top, x[e].x);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float w[kMostParts / 32], l = 0.f;
#pragma unroll
        for (int e = 0; e < kMostParts / 32; ++e) {
            w[e] = x[e].y == 0.f ? 0.f : ex2(x[e].x - top);
            l += x[e].y == 0.f ? 0.f : x[e].y * w[e];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        float acc[W] = {};
#pragma unroll 4
        for (int p = 0; p < f.parts; ++p) {
            const float wp = __shfl_sync(0xffffffffu, p < 32 ? w[0] : w[1], p & 31);
            const float lp = __shfl_sync(0xffffffffu, p < 32 ? x[0].y : x[1].y, p & 31);
            if (lp == 0.f) continue;
            const float *o = a.ws_o + (base + int64_t(p) * kRows) * D + lane * 2;
#pragma unroll
            for (int e = 0; e < W / 2; ++e) {
                const float2 y = *reinterpret_cast<const float2 *>(o + e * 64);
                acc[2 * e] = fmaf(y.x, wp, acc[2 * e]);
                acc[2 * e + 1] = fmaf(y.y, wp, acc[2 * e + 1]);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int h = f.hk * a.group + head;
        uint16_t *o = a.o + (int64_t(f.t0) + at) * a.o_stride + int64_t(h) * D + lane * 2;
#pragma unroll
        for (int e = 0; e < W / 2; ++e)
            *reinterpret_cast<uint32_t *>(o + e * 64) =
                gdn::f32_to_bf16(acc[2 * e] * inv) | uint32_t(gdn::f32_to_bf16(acc[2 * e + 1] * inv)) << 16;
        if (lane == 0 && a.lse)
            a.lse[(int64_t(f.t0) + at) * a.h_q + h] = l == 0.f ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
    }
}

// ---- the workspace's keys and values: cached positions as bf16 (exactly: 4 bits times a power of two), then the new rows

constexpr int kGatherRows = 32, kGatherThreads = 256;

struct GatherArgs {
    kv8_cache c;
    int32_t layer, page_shift;
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
    __shared__ int page[kGatherRows], pos[kGatherRows];  // page >= 0: a cached position; -1: new row pos; -2: nothing
    const int tid = threadIdx.x;
    const int64_t w0 = int64_t(blockIdx.x) * kGatherRows;
    if (tid < kGatherRows) page[tid] = -2;
    {
        const int chunk = (a.rq.B + kGatherThreads - 1) / kGatherThreads, r0 = tid * chunk, r1 = min(a.rq.B, r0 + chunk);
        long long rows = 0, kv = 0, all, kv_all;
        for (int r = r0; r < r1; ++r) kv += prompt::kv_rows_of(prompt::request_of(a.rq, r));
        const long long mine = kv;
        prompt::scan2<kGatherThreads>(scan, rows, kv, all, kv_all);
        if (kv < w0 + kGatherRows && kv + mine > w0)
            for (int r = r0; r < r1; ++r) {
                const prompt::Request q = prompt::request_of(a.rq, r);
                const long long n = prompt::kv_rows_of(q);
                const bool fits = kv + n <= a.rq.kv_capacity;
                const int lo = a.c.window ? max(0, q.len + 1 - a.c.window) : 0;
                if (!fits && n && kv < w0 + kGatherRows && kv + n > w0) gdn::set_status(a.status, GDN_DEV_ROWS_BAD);
                for (long long w = max((long long)w0, kv); fits && w < min((long long)w0 + kGatherRows, kv + n); ++w) {
                    const int t = int(w - kv);
                    int p = -1, at = q.t0 + t - q.len;
                    if (t < q.len) {
                        at = t;
                        p = -2;
                        if (t >= lo) {
                            p = a.table[int64_t(r) * a.table_stride + (t >> a.page_shift)];
                            if (p < 0 || p >= a.c.num_pages) {
                                gdn::set_status(a.status, GDN_DEV_PAGE_OOR);
                                p = -2;
                            }
                        }
                    }
                    page[w - w0] = p;
                    pos[w - w0] = at;
                }
                kv += n;
            }
    }
    __syncthreads();
    const int d = a.c.d, h_kv = a.c.h_kv, T = a.c.page_tokens;
    const int per = d / 16, shift = 31 - __clz(per);  // pieces of 16 channels a row
    const int items = 2 * h_kv * kGatherRows * per;
#pragma unroll 4
    for (int i = tid; i < items; i += kGatherThreads) {
        const int ch = (i & (per - 1)) * 16, w = (i >> shift) % kGatherRows, hv = (i >> shift) / kGatherRows;
        const int is_v = hv >= h_kv, h = hv - is_v * h_kv;
        const int p = page[w], at = pos[w];
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
    int per_tile, splits, rows;
};
Plan plan_of(int h_q, int h_kv, int d, int window, int32_t B, int32_t row_capacity, int32_t max_len,
             int32_t max_rows) {
    Plan p{};
    p.per_tile = kTile / (h_q / h_kv);
    p.rows = (d == 256 ? 1 : 2) * kTile;
    const int64_t per_unit = int64_t(d == 256 ? 1 : 2) * p.per_tile;
    const int64_t each = int64_t(B) * ((max_rows + per_unit - 1) / per_unit), all = row_capacity / per_unit + B;
    p.units = h_kv * (each < all ? each : all);
    int64_t seen = int64_t(max_len) + max_rows;
    if (window && window + per_unit < seen) seen = window + per_unit + kTile;
    const int64_t tiles = (seen + kTile - 1) / kTile;
    // work is cut where it leaves SMs idle: every unit into as many parts as make one CTA an SM
    int64_t s = p.units >= kSms || p.units == 0 ? 1 : kSms / p.units;
    if (s > tiles / kLeast) s = tiles / kLeast;
    p.splits = int(s < 1 ? 1 : s > kMostParts ? kMostParts : s);
    return p;
}
size_t part_bytes(const Plan &p, int d) {
    return p.splits > 1 ? size_t(p.units) * (size_t(p.splits) * p.rows * (size_t(d) * 4 + 8) + sizeof(Info)) : 0;
}
size_t kv_bytes(const kv8_cache *c, int64_t rows) { return size_t(rows) * c->h_kv * c->d * 4; }

template <int D>
int launch(const Args &a, const Plan &p, cudaStream_t st) {
    using C = Cfg<D>;
    // for every launch: the limit is the current device's
    if (cudaFuncSetAttribute(prompt_attend_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) !=
        cudaSuccess)
        return GDN_ERR_CUDA;
    const int rc = gdn_host::launch_pdl(prompt_attend_kernel<D>, dim3(unsigned(p.units), unsigned(p.splits)),
                                        dim3(C::kThreads), C::kSmem, st, a);
    if (rc != GDN_OK || p.splits == 1) return rc;
    return gdn_host::launch_pdl(prompt_join_kernel<D>, dim3(unsigned(p.units), unsigned(p.rows / kJoinRows)), dim3(256),
                                0, st, a);
}

int run(Args &a, const Plan &p, int d, float sm_scale, uint8_t *parts, cudaStream_t st) {
    a.per_tile = p.per_tile;
    a.splits = p.splits;
    a.negate = sm_scale < 0.f;
    const float c = fabsf(sm_scale) * 1.4426950408889634f;
    a.scale_log2 = c < 1e-37f ? 1e-37f : c;  // a masked score times zero would be no number
    if (p.splits > 1) {
        const size_t rows = size_t(p.units) * p.splits * p.rows;
        a.ws_o = reinterpret_cast<float *>(parts);
        a.ws_ml = reinterpret_cast<float2 *>(a.ws_o + rows * d);
        a.info = reinterpret_cast<Info *>(a.ws_ml + rows);
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

}  // namespace

extern "C" size_t attn_prompts_workspace_bytes(const attn_dims *dims, int32_t B, int32_t row_capacity,
                                               int32_t max_rows) {
    if (check_dims(dims) != GDN_OK || B <= 0 || B > 65535 || row_capacity < 0 || max_rows <= 0) return 0;
    return part_bytes(plan_of(dims->h_q, dims->h_kv, dims->d, dims->window, B, row_capacity, 0, max_rows), dims->d);
}

static int prompts(const attn_dims *dims, int32_t B, int32_t row_capacity, const int32_t *cu_rows, const gdn_bf16 *q,
                   int64_t q_stride, const gdn_bf16 *k, int64_t k_stride, const gdn_bf16 *v, int64_t v_stride,
                   gdn_bf16 *o, int64_t o_stride, float *lse, int32_t max_rows, void *workspace,
                   size_t workspace_bytes, uint32_t *dev_status, uint64_t wait_ns, int32_t withhold, void *stream) {
    const int bad = check_dims(dims);
    if (bad != GDN_OK) return bad;
    if (B < 0 || B > 65535 || row_capacity < 0 || max_rows < 0) return GDN_ERR_ARG;
    if (B == 0 || max_rows == 0 || row_capacity == 0) return GDN_OK;
    if (!cu_rows || !q || !k || !v || !o) return GDN_ERR_NULL;
    if (!gdn_host::kv8_rows_ok(q, q_stride, dims->h_q, dims->d) ||
        !gdn_host::kv8_rows_ok(k, k_stride, dims->h_kv, dims->d) ||
        !gdn_host::kv8_rows_ok(v, v_stride, dims->h_kv, dims->d) ||
        !gdn_host::kv8_rows_ok(o, o_stride, dims->h_q, dims->d))
        return GDN_ERR_ARG;
    const Plan p = plan_of(dims->h_q, dims->h_kv, dims->d, dims->window, B, row_capacity, 0, max_rows);
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
        max_len > gdn_host::kKv8MaxLen || max_rows <= 0 || total_len < 0)
        return 0;
    const int64_t rows = kv_rows(B, row_capacity, max_len, total_len);
    if (rows >= gdn_host::kKv8MaxLen) return 0;
    return kv_bytes(cache, rows) +
           part_bytes(plan_of(cache->h_q, cache->h_kv, cache->d, cache->window, B, row_capacity, max_len, max_rows),
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
        table_stride < 0 || max_len < 0 || max_len > gdn_host::kKv8MaxLen || max_rows < 0 ||
        max_rows > gdn_host::kKv8MaxLen || total_len < 0)
        return GDN_ERR_ARG;
    if (B == 0 || max_rows == 0 || row_capacity == 0) return GDN_OK;
    if (!cu_rows || !cache_len || (!table && table_pages > 0) || !q || !k_new || !v_new || !o) return GDN_ERR_NULL;
    if (!gdn_host::kv8_rows_ok(q, q_stride, cache->h_q, cache->d) ||
        !gdn_host::kv8_rows_ok(k_new, k_stride, cache->h_kv, cache->d) ||
        !gdn_host::kv8_rows_ok(v_new, v_stride, cache->h_kv, cache->d) ||
        !gdn_host::kv8_rows_ok(o, o_stride, cache->h_q, cache->d))
        return GDN_ERR_ARG;
    const int64_t rows = kv_rows(B, row_capacity, max_len, total_len);
    const Plan p = plan_of(cache->h_q, cache->h_kv, cache->d, cache->window, B, row_capacity, max_len, max_rows);
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
    const int rc = gdn_host::launch_pdl(kv8_gather_kernel, dim3(unsigned((rows + kGatherRows - 1) / kGatherRows)),
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
