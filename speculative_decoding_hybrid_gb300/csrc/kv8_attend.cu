// Attention of a transaction's rows over the paged 8-bit cache (sm_103a).
//
// With R = rows * (h_q / h_kv) query vectors on one kv head a position costs
// 2 d bytes and 4 d R flops: from R of about 8 on only the tensor cores keep
// up with the memory.  Keys and values go to them as they lie in the cache,
// without a conversion: the products are e4m3 x e4m3 with the cache's side
// exact by construction and the other side split into exact or nearly exact
// e4m3 parts, side by side in the N extent, which the few rows leave free:
//   scores   S^T[128 positions][2 RB] = K [q_hi | q_lo]     q = (q_hi + q_lo/32) 2^-k  (bf16's 8 bits, exactly)
//   outputs  O^T[d][4 RB] += V^T [p_0 | p_1 | p_2 | p_3]    p = sum p_j 32^-j
// A part is its predecessor's remainder times 32, so three carry 14 bits of a
// weight; the fourth keeps that precision for weights 2^-12 times smaller.
// A position is a tensor-memory lane, so its page's scales are one register
// of the thread that owns the lane: K's multiplies the score, V's the weight.
//
// The softmax keeps a reference m per column, not the running maximum: a
// column's weights are 2^(z - m), and only when some z passes m + kSlack (or a
// page's V scale the reference one) is m moved and the sums rescaled; usually
// that is once, at a piece's first tile.  One vote a tile decides.
//
// One CTA per (piece of a request's positions, kv head and block of RB
// columns, request): groups of four softmax warps (thread = position = lane,
// a group's share of the columns each), one warp that copies pages (tiled TMA,
// 128- or 64-byte swizzle, K and V tiles through one ring), one that issues
// the products.  The transaction's own rows, bf16, come
// last: their keys as one more tile, each a hi and a lo position (16 + 16
// lanes) split like q, their values in fp32 in the epilogue.
// Pieces leave (m, l, O) in the workspace for kv8_join_kernel; a request with
// one piece is written directly.
#include <cuda.h>

#include "kv8.cuh"
#include "tc.cuh"

namespace {

constexpr int kTile = 128;      // positions a tile
// Weights are scaled by 2^2 and at most 2^(2 + 6) < 448; the last part's rounding
// is 2^-25, so 2^-27 of a weight at the reference.  More slack moves the
// reference less often and costs that many bits at the low end.
constexpr float kBase = 4.f, kSlack = 6.f;
constexpr float kUnset = -1e30f;
constexpr int kScales = 8;      // tiles whose scales may wait to be read; the ring of 10 slots holds back the copies before that

struct AttendArgs {
    CUtensorMap map;
    kv8_cache c;
    int32_t layer, B, row_capacity, table_pages, max_len, max_rows;
    int32_t group, blocks, piece_tiles, max_pieces, page_shift;  // page_tokens = 1 << page_shift
    int64_t table_stride;
    const int32_t *cu_rows, *cache_len, *table;
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, o_stride;
    uint16_t *o;
    float *lse;
    float *ws_o;       // [unit][RB][d]
    float2 *ws_ml;     // [unit][RB]
    uint32_t *status;
    uint64_t wait_ns;
};

// What a request asks for; the same test in both kernels.
struct Request {
    int t0, n, len, lo, tiles, pieces;  // lo: first position any row sees; tiles from lo / 128 on
    bool bad;
};
__device__ __forceinline__ Request request_of(const AttendArgs &a, int r) {
    Request q;
    q.t0 = a.cu_rows[r];
    q.n = a.cu_rows[r + 1] - q.t0;
    q.len = a.cache_len[r];
    q.bad = q.t0 < 0 || q.n < 0 || q.n > a.max_rows || int64_t(q.t0) + q.n > a.row_capacity || q.len < 0 ||
            q.len > a.max_len || int64_t(q.len) > int64_t(a.table_pages) * a.c.page_tokens;
    const int w = a.c.window;
    q.lo = w ? max(0, q.len + (a.k ? 1 : 0) - w) : 0;
    if (q.lo > q.len) q.lo = q.len;
    const int first = q.lo / kTile;
    q.tiles = q.lo < q.len ? (q.len + kTile - 1) / kTile - first : 0;
    q.pieces = max(1, (q.tiles + a.piece_tiles - 1) / a.piece_tiles);
    return q;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// Barrier of a group's four softmax warps with an OR over a predicate.
__device__ __forceinline__ bool group_or(int group, bool p) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, "
        "q;\n}\n"
        : "=r"(r)
        : "r"(uint32_t(p)), "r"(group + 1)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int group) {
    asm volatile("barrier.cta.sync %0, 128;" ::"r"(group + 1) : "memory");
}
template <int THREADS>
__device__ __forceinline__ void soft_sync() {
    asm volatile("barrier.cta.sync 5, %0;" ::"n"(THREADS) : "memory");
}
__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(gdn::smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Pairs of fp32 values: one instruction an operation.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ f2 pair(uint32_t a, uint32_t b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ float2 both(f2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// c - 32 h of two fp32 values c and two fp16 values h.
__device__ __forceinline__ float2 minus32(float2 c, uint32_t h) {
    float2 r;
    asm("{\n .reg .b16 a, b, k;\n mov.b32 {a, b}, %2;\n mov.b16 k, 0xd000;\n fma.rn.f32.f16 %0, a, k, %3;\n"
        " fma.rn.f32.f16 %1, b, k, %4;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ uint32_t join16(uint16_t lo, uint16_t hi) {
    uint32_t r;
    asm("mov.b32 %0, {%1, %2};" : "=r"(r) : "h"(lo), "h"(hi));
    return r;
}

// fp16 pair arithmetic of the splits.
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint16_t e4m3x2_of(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
// (h - back) * 32 of two fp16 values: exact, `back` being h to 4 bits.
__device__ __forceinline__ uint32_t rest32(uint32_t h, uint32_t back) {
    uint32_t t, r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(t) : "r"(h), "r"(0x50005000u));              // 32, 32
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(back), "r"(0xd000d000u), "r"(t));  // -32, -32
    return r;
}

template <int D, int RB>
struct Cfg {
    static constexpr int kRow = D < 128 ? D : 128;       // bytes of an operand tile's row
    static constexpr int kAtoms = D / kRow;              // such tiles side by side
    static constexpr int kNs = 2 * RB;                   // score columns
    static constexpr int kNp = 4 * RB;                   // weight columns
    static constexpr int kPRow = RB == 8 ? 64 : RB == 64 ? 128 : kNp;  // bytes of a weight tile's row (64 or 128)
    static constexpr int kFresh = 32 * D > 64 * RB ? 32 * D : 64 * RB;  // bytes of the fresh keys, and of the values
    static constexpr int kQ = kNs * D;
    static constexpr int kP = kTile * (RB == 8 ? 64 : kNp);
    static constexpr int kSlot = kTile * D;
    // groups of four softmax warps, each with its share of the columns: a warp
    // waits on its own chain of loads, exponentials and conversions most of the
    // time, so an SM wants at least eight of them
    static constexpr int kGroups = RB <= 8 ? 1 : RB == 16 ? (D == 256 ? 2 : 1) : RB / 16;
    static constexpr int kCols = RB / kGroups;           // columns a thread
    static constexpr int kSoft = 128 * kGroups;          // softmax threads
    static constexpr int kThreads = kSoft + 64;
    // CTAs an SM: two, unless 512 tensor-memory columns or two sets of 32 KB slots rule it out
    static constexpr int kCtas = D == 256 || RB == 64 ? 1 : 2;
    static constexpr int kFixed = 2 * kFresh + kQ + 2 * kP + (D == 64 ? kSlot : 0) + 1024;
    static constexpr int kStatic = RB == 64 ? 4096 : 2048;  // at least what __shared__ takes below
    static constexpr int kRoom = (kCtas == 1 ? 227 * 1024 : 113 * 1024) - kStatic - kFixed;
    static constexpr int kSlots = kRoom / kSlot > 10 ? 10 : kRoom / kSlot;
    static constexpr int kSmem = kFixed + kSlots * kSlot;
    static constexpr int kTmemUse = 2 * kNs + kNp * (D == 256 ? 2 : 1);
    static constexpr int kTmem = kTmemUse <= 64 ? 64 : kTmemUse <= 128 ? 128 : kTmemUse <= 256 ? 256 : 512;
    static_assert(kTmemUse <= 512 && kSlots >= 3, "does not fit an SM");
};

// A warp splits four rows of bf16, eight threads (sub) a row: x = (hi + lo/32) 2^-k
// into rows rh and rl of an operand tile of `rows` rows.  -> 2^-k, or NaN for a
// row that is not finite.
template <int D>
__device__ __forceinline__ void load_row(const uint16_t *p, int sub, bool have, uint4 (&w)[D / 64]) {
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
        w[e] = have ? *reinterpret_cast<const uint4 *>(p + sub * (D / 8) + e * 8) : make_uint4(0, 0, 0, 0);
}
template <int D>
__device__ __forceinline__ float split_row(const uint4 (&w)[D / 64], int sub, uint8_t *tile, int rows, int rh, int rl) {
    constexpr int E = D / 8, kRow = D < 128 ? D : 128;
    float m = 0.f, x[E];
    bool finite = true;
#pragma unroll
    for (int e = 0; e < E / 8; ++e) {
        const uint32_t u[4] = {w[e].x, w[e].y, w[e].z, w[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[e * 8 + 2 * i] = __uint_as_float(u[i] << 16);
            x[e * 8 + 2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const bool f = fabsf(x[e]) < INFINITY;
        finite &= f;
        x[e] = f ? x[e] : 0.f;
        m = fmaxf(m, fabsf(x[e]));
    }
    uint32_t top = __float_as_uint(m);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t all = (__ballot_sync(0xffffffffu, finite) >> (threadIdx.x & 24)) & 0xffu;
    const int k = max(-110, min(110, 7 - (int(top >> 23) - 127)));  // largest in [128, 256)
    const float up = kv8::pow2i(k), up32 = up * 32.f, down = kv8::pow2i(-k);
#pragma unroll
    for (int b = 0; b < E / 8; ++b) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t hh[2], ll[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x0 = x[b * 8 + g * 4 + 2 * i], x1 = x[b * 8 + g * 4 + 2 * i + 1];
                hh[i] = kv8::e4m3x2(x0 * up, x1 * up);
                const float2 back = kv8::f32x2_of(uint16_t(hh[i]));
                ll[i] = kv8::e4m3x2(fmaf(back.x, -32.f, x0 * up32), fmaf(back.y, -32.f, x1 * up32));
            }
            h[g] = hh[0] | (hh[1] << 16);
            l[g] = ll[0] | (ll[1] << 16);
        }
        const int e0 = sub * E + b * 8, atom = e0 / kRow, in = e0 % kRow;
        uint8_t *t = tile + atom * rows * kRow + (in & 8);
        *reinterpret_cast<uint2 *>(t + tc::swz8_off<kRow>(rh, in >> 4)) = make_uint2(h[0], h[1]);
        *reinterpret_cast<uint2 *>(t + tc::swz8_off<kRow>(rl, in >> 4)) = make_uint2(l[0], l[1]);
    }
    return all != 0xffu ? __uint_as_float(0x7fc00000u) : down;
}

// Sums of N values over a warp's lanes: value k's sum lands in v[0] of the
// lanes whose top log2(N) bits are k.
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N], int lane) {
    constexpr int kSteps = N == 16 ? 4 : 3;
    static_assert(N == 16 || N == 8, "columns a thread");
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int off = 16 >> s, half = N >> (s + 1);
        const bool up = lane & off;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float give = up ? v[k] : v[k + half], keep = up ? v[k + half] : v[k];
            v[k] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    }
#pragma unroll
    for (int off = 16 >> kSteps; off; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
}

// Ring positions of the tiles' loads, in the order the products use them:
// K0 K1 V0 K2 V1 ... V(n-1).
__device__ __forceinline__ int k_pos(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_pos(int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; }

template <int D, int RB>
__global__ void __launch_bounds__(Cfg<D, RB>::kThreads, Cfg<D, RB>::kCtas)
    kv8_attend_kernel(const __grid_constant__ AttendArgs a) {
    using C = Cfg<D, RB>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[C::kSlots], empty[C::kSlots], s_full[2], s_free[2], p_full[2], pv_done[2], q_ready, drain;
    __shared__ uint64_t sc_full[kScales], fk_ready, fv_full;
    __shared__ float2 sc_ring[kScales][8];
    __shared__ int bad_page;
    __shared__ uint32_t tmem_ptr;
    __shared__ alignas(16) float col_nm[RB], col_coef[RB], col_fac[RB];  // -m
    __shared__ float col_max[4][RB], v_max[C::kGroups][4];
    __shared__ uint8_t col_row[RB], col_head[RB];  // of the request's rows, of the kv head's queries
    __shared__ float fresh_k[16];
    __shared__ float col_l[RB];

    gdn::pdl_enter();
    const int piece = blockIdx.x, hk = blockIdx.y / a.blocks, blk = blockIdx.y % a.blocks, r = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Request rq = request_of(a, r);
    if (rq.bad) {
        if (piece == 0 && blockIdx.y == 0 && tid == 0) gdn::set_status(a.status, GDN_DEV_ROWS_BAD);
        return;
    }
    const int cols = min(RB, rq.n * a.group - blk * RB);  // columns of this block in use
    if (piece >= rq.pieces || cols <= 0) return;

    const int T = a.c.page_tokens, shift = a.page_shift;
    const int tile0 = rq.lo / kTile + piece * a.piece_tiles;
    const int nc = max(0, min(a.piece_tiles, rq.tiles - piece * a.piece_tiles));  // cached tiles
    const bool fresh = a.k != nullptr && piece == rq.pieces - 1;
    const int nt = nc + (fresh ? 1 : 0);

    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *s_fk = sm, *s_fv = s_fk + C::kFresh, *s_q = s_fv + C::kFresh;
    uint8_t *s_p = s_q + ((C::kQ + 1023) & ~1023), *s_ring = s_p + 2 * C::kP;

    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            gdn::mbar_init(&full[i], 1);
            gdn::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            gdn::mbar_init(&s_full[i], 1);
            gdn::mbar_init(&s_free[i], C::kSoft / 32);
            gdn::mbar_init(&p_full[i], C::kSoft / 32);
            gdn::mbar_init(&pv_done[i], 1);
        }
        for (int i = 0; i < kScales; ++i) gdn::mbar_init(&sc_full[i], 1);
        gdn::mbar_init(&q_ready, C::kSoft / 32);
        gdn::mbar_init(&fk_ready, 1);
        gdn::mbar_init(&fv_full, 1);
        gdn::mbar_init(&drain, 1);
        bad_page = 0;
    }
    constexpr int kCopyWarp = C::kSoft / 32, kMmaWarp = kCopyWarp + 1;
    if (warp == kMmaWarp) tc::tmem_alloc(&tmem_ptr, C::kTmem);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    float *fresh_p = reinterpret_cast<float *>(s_fk);  // [16][RB], once the fresh keys' product is done
    static_assert(RB * 16 * 4 <= C::kFresh, "weights of the fresh rows");
    const uint32_t tm = tmem_ptr, tm_o = tm + 2 * C::kNs;

    if (warp == kCopyWarp) {
        // ---- copies.  Page ids and scales come 32 pages at a time, ids two and scales
        // one such batch ahead.
        if (fresh && rq.n > 0) {
            if (lane == 0) gdn::mbar_arrive_expect_tx(&fv_full, uint32_t(rq.n) * (2 * D));
            __syncwarp();
            if (lane < rq.n)
                gdn::bulk_g2s(s_fv + lane * 2 * D, a.v + (int64_t(rq.t0) + lane) * a.v_stride + int64_t(hk) * D, 2 * D,
                              &fv_full);
        }
        const int per = kTile >> shift;  // pages a tile
        const int page0 = tile0 * per, first = rq.lo >> shift, last = (rq.len + T - 1) >> shift;
        const int32_t *tab = a.table + int64_t(r) * a.table_stride;
        const float *sc0 = a.c.scale + int64_t(a.layer) * a.c.scale_layer_stride + 2 * hk;
        constexpr int kNone = -1;  // a page no row sees
        auto wanted = [&](int batch) {
            const int j = page0 + batch * 32 + lane;
            return j >= first && j < last && batch * 32 + lane < nc * per;
        };
        auto ids = [&](int batch) { return wanted(batch) ? tab[page0 + batch * 32 + lane] : kNone; };
        auto scales = [&](int p) {
            return p >= 0 && p < a.c.num_pages
                       ? *reinterpret_cast<const float2 *>(sc0 + int64_t(p) * a.c.scale_page_stride)
                       : make_float2(0.f, 0.f);
        };
        bool ok = true;
        int issued = 0;
        auto issue = [&](int pos, int page, int is_v) {
            const int slot = pos % C::kSlots;
            if (pos >= C::kSlots)
                ok = ok && gdn::mbar_wait_bounded(&empty[slot], ((pos / C::kSlots) - 1) & 1, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) return;
            const uint32_t have = __ballot_sync(0xffffffffu, lane < per && page >= 0);
            if (lane == 0) gdn::mbar_arrive_expect_tx(&full[slot], uint32_t(__popc(have)) * uint32_t(T * D));
            __syncwarp();
            issued = pos + 1;
            if (lane < per && page >= 0) {
#pragma unroll
                for (int x = 0; x < C::kAtoms; ++x)
                    gdn::tma_load_3d(s_ring + slot * C::kSlot + x * kTile * C::kRow + lane * T * C::kRow, &a.map,
                                     x * C::kRow, (is_v * a.c.h_kv + hk) * T, page, &full[slot]);
            }
        };
        int cur = ids(0), nxt = ids(1), far = ids(2), batch = 0, prev = -1;
        float2 sc = scales(cur), sc_nxt = scales(nxt);
        for (int i = 0; i <= nc && ok; ++i) {
            int page = -1;
            float2 s = make_float2(0.f, 0.f);
            if (i < nc) {
                const int at = i * per;
                if (at / 32 != batch) {
                    batch = at / 32;
                    cur = nxt;
                    sc = sc_nxt;
                    nxt = far;
                    sc_nxt = scales(nxt);
                    far = ids(batch + 2);
                }
                // an id out of range is not loaded; the piece's outputs are dropped
                const int src = (at % 32) + (lane & (per - 1));
                page = __shfl_sync(0xffffffffu, cur, src);
                const bool want = page0 + at + (lane & (per - 1)) >= first && page0 + at + (lane & (per - 1)) < last;
                if (page < 0 || page >= a.c.num_pages) {
                    if (want) *reinterpret_cast<volatile int *>(&bad_page) = 1;
                    page = -1;
                }
                issue(k_pos(i), page, 0);
            }
            if (i > 0 && ok) issue(v_pos(i - 1, nc), prev, 1);
            if (i < nc && ok) {
                const int src = (i * per % 32) + (lane & (per - 1));
                s.x = __shfl_sync(0xffffffffu, sc.x, src);
                s.y = __shfl_sync(0xffffffffu, sc.y, src);
                if (lane < per) sc_ring[i % kScales][lane] = s;
                __syncwarp();
                if (lane == 0) arrive(&sc_full[i % kScales]);
            }
            prev = page;
        }
        if (!ok) {
            // wait, again bounded, for the copies in flight into this CTA's shared memory
            gdn::set_status(a.status, GDN_DEV_TIMEOUT);
            for (int pos = max(0, issued - C::kSlots); pos < issued; ++pos)
                (void)gdn::mbar_wait_bounded(&full[pos % C::kSlots], (pos / C::kSlots) & 1, a.wait_ns);
        }
        if (fresh && rq.n > 0) (void)gdn::mbar_wait_bounded(&fv_full, 0, a.wait_ns);
    } else if (warp == kMmaWarp) {
        // ---- products: the warp runs the loop, one elected lane issues
        if (nt > 0) {
            constexpr uint32_t id_s = tc::idesc_e4m3(128, C::kNs);
            constexpr uint32_t id_p = tc::idesc_e4m3(128, C::kNp) | tc::kAMnMajor | tc::kBMnMajor;
            const uint64_t dq = tc::smem_desc8<C::kRow>(gdn::smem_u32(s_q), 16);
            // weights: rows are positions; RB = 64 has two tiles of 128 columns
            const uint64_t dp = tc::smem_desc8<C::kPRow>(gdn::smem_u32(s_p), kTile * C::kPRow);
            // V has 128 rows of M at d >= 128; at d = 64 rows 64.. read the next slot and are not used
            constexpr uint32_t lbo = C::kRow == 64 ? C::kSlot : 16;
            const uint64_t dk0 = tc::smem_desc8<C::kRow>(gdn::smem_u32(s_ring), 16);
            const uint64_t dv0 = tc::smem_desc8<C::kRow>(gdn::smem_u32(s_ring), lbo);
            const uint64_t dfk = tc::smem_desc8<C::kRow>(gdn::smem_u32(s_fk), 16);
            const bool leader = elect_one();
            if (fresh) {
                for (int j0 = 0; j0 < rq.n; j0 += 4) {
                    const int j = j0 + (lane >> 3);
                    uint4 w[D / 64];
                    load_row<D>(a.k + (int64_t(rq.t0) + j) * a.k_stride + int64_t(hk) * D, lane & 7, j < rq.n, w);
                    const float down = split_row<D>(w, lane & 7, s_fk, 32, j, 16 + j);
                    if ((lane & 7) == 0) fresh_k[j] = down;
                }
                gdn::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive(&fk_ready);
            }
            bool ok = gdn::mbar_wait_bounded(&q_ready, 0, a.wait_ns);
            for (int i = 0; i <= nt && ok; ++i) {
                if (i < nt) {
                    const bool cached = i < nc;
                    const int pos = k_pos(i), slot = pos % C::kSlots;
                    if (cached) ok = gdn::mbar_wait_bounded(&full[slot], (pos / C::kSlots) & 1, a.wait_ns);
                    if (ok && i >= 2) ok = gdn::mbar_wait_bounded(&s_free[i & 1], ((i >> 1) - 1) & 1, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::fence_after();
                    if (leader) {
                        const uint64_t dk = cached ? tc::desc_at(dk0, slot * C::kSlot) : dfk;
                        const uint32_t atom = cached ? kTile * C::kRow : 32 * C::kRow;
#pragma unroll
                        for (int s = 0; s < D / 32; ++s) {
                            const uint32_t x = s * 32 / C::kRow, in = s * 32 % C::kRow;
                            tc::mma_e4m3(tm + (i & 1) * C::kNs, tc::desc_at(dk, x * atom + in),
                                         tc::desc_at(dq, x * C::kNs * C::kRow + in), id_s, s > 0);
                        }
                        tc::commit(&s_full[i & 1]);
                        if (cached) tc::commit(&empty[slot]);
                    }
                    __syncwarp();
                }
                if (i > 0 && i <= nc) {
                    const int j = i - 1, pos = v_pos(j, nc), slot = pos % C::kSlots;
                    ok = gdn::mbar_wait_bounded(&full[slot], (pos / C::kSlots) & 1, a.wait_ns);
                    if (ok) ok = gdn::mbar_wait_bounded(&p_full[j & 1], (j >> 1) & 1, a.wait_ns);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc::fence_after();
                    if (leader) {
                        const uint64_t dv = tc::desc_at(dv0, slot * C::kSlot), dpj = tc::desc_at(dp, (j & 1) * C::kP);
#pragma unroll
                        for (int x = 0; x < C::kAtoms; ++x)
#pragma unroll
                            for (int s = 0; s < kTile / 32; ++s)
                                tc::mma_e4m3(tm_o + x * C::kNp,
                                             tc::desc_at(dv, x * kTile * C::kRow + s * 32 * C::kRow),
                                             tc::desc_at(dpj, s * 32 * C::kPRow), id_p, j > 0 || s > 0);
                        tc::commit(&pv_done[j & 1]);
                        tc::commit(&empty[slot]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) {
                gdn::set_status(a.status, GDN_DEV_TIMEOUT);
                if (leader) tc::commit(&drain);  // products in flight read shared and write tensor memory
                (void)gdn::mbar_wait_bounded(&drain, 0, a.wait_ns);
            }
        }
        __syncwarp();
    } else {
        // ---- softmax warps.  First the operands that come as bf16.
        {
            // eight threads a column; the columns fill whole warps, one pass takes them all
            static_assert(RB <= C::kSoft / 8, "a thread has one column");
            const int c = tid >> 3, sub = tid & 7;
            if (c < RB) {
                const int x = blk * RB + c, row = x / a.group, h = hk * a.group + x % a.group;
                uint4 w[D / 64];
                load_row<D>(a.q + (int64_t(rq.t0) + row) * a.q_stride + int64_t(h) * D, sub, c < cols, w);
                const float down = split_row<D>(w, sub, s_q, C::kNs, c, RB + c);
                if (sub == 0) {
                    col_nm[c] = -kUnset;
                    col_coef[c] = a.c.sm_scale * 1.4426950408889634f * down;
                    col_row[c] = uint8_t(row);
                    col_head[c] = uint8_t(x % a.group);
                }
            }
            gdn::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&q_ready);
            soft_sync<C::kSoft>();
        }
        // this thread's position in a tile and its columns col0 .. col0 + N - 1
        constexpr int N = C::kCols;
        const int grp = warp >> 2, pos_in = tid & 127, col0 = grp * N;
        // a row sees positions from lo0 + row * lo1 on (rq.lo is row 0's, and not negative)
        const int lo0 = a.c.window ? rq.len + (a.k ? 1 : 0) - a.c.window : 0, lo1 = a.c.window && a.k ? 1 : 0;
        const int lo_last = lo0 + lo1 * col_row[cols - 1];
        bool ok = true;
        f2 l[N / 2];
        float z[N];
#pragma unroll
        for (int c = 0; c < N / 2; ++c) l[c] = 0;
        float vref = kv8::pow2i(kv8::kMinScaleExp), vinv = kBase / vref;
        const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;

        for (int i = 0; i < nt; ++i) {
            const bool is_fresh = i >= nc;
            const int t = (tile0 + i) * kTile + pos_in;
            if (ok)
                ok = is_fresh ? gdn::mbar_wait_bounded(&fk_ready, 0, a.wait_ns)
                              : gdn::mbar_wait_bounded(&sc_full[i % kScales], (i / kScales) & 1, a.wait_ns);
            const float2 sc = is_fresh ? make_float2(pos_in < 32 && (pos_in & 15) < rq.n ? fresh_k[pos_in & 15] : 0.f, 0.f)
                                       : sc_ring[i % kScales][pos_in >> shift];
            // whole: every row sees every position of the tile
            const bool whole = !is_fresh && (tile0 + i + 1) * kTile <= rq.len && (tile0 + i) * kTile >= lo_last;
            if (ok) ok = gdn::mbar_wait_bounded(&s_full[i & 1], (i >> 1) & 1, a.wait_ns);
            tc::fence_after();

            // z - m of every column (m = 0 where the reference is to move)
            auto load_z = [&](bool plain) {
                uint32_t hi[N], lo[N];
                const uint32_t at = tm + lane_base + (i & 1) * C::kNs + col0;
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
                f2 s[N / 2];
#pragma unroll
                for (int c = 0; c < N / 2; ++c)
                    s[c] = fma2(pair(lo[2 * c], lo[2 * c + 1]), pair(1.f / 32.f, 1.f / 32.f),
                                pair(hi[2 * c], hi[2 * c + 1]));
                if (is_fresh) {  // the other part of the position
#pragma unroll
                    for (int c = 0; c < N / 2; ++c) {
                        const float2 x = both(s[c]);
                        const f2 other = pair(__shfl_xor_sync(0xffffffffu, x.x, 16), __shfl_xor_sync(0xffffffffu, x.y, 16));
                        s[c] = pos_in & 16 ? fma2(s[c], pair(1.f / 32.f, 1.f / 32.f), other)
                                           : fma2(other, pair(1.f / 32.f, 1.f / 32.f), s[c]);
                    }
                }
                const f2 sx = pair(sc.x, sc.x);
#pragma unroll
                for (int c = 0; c < N; c += 4) {
                    const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(col_coef + col0 + c);
                    ulonglong2 nm = make_ulonglong2(0, 0);
                    if (!plain) nm = *reinterpret_cast<const ulonglong2 *>(col_nm + col0 + c);
                    const float2 x = both(fma2(s[c / 2], mul2(sx, k.x), nm.x)),
                                 y = both(fma2(s[c / 2 + 1], mul2(sx, k.y), nm.y));
                    z[c] = x.x;
                    z[c + 1] = x.y;
                    z[c + 2] = y.x;
                    z[c + 3] = y.y;
                }
                if (is_fresh) {
                    const int j = pos_in & 15, w = a.c.window;
#pragma unroll
                    for (int c = 0; c < N; ++c) {
                        const int row = col_row[col0 + c];
                        const bool see = pos_in < 32 && j < rq.n && j <= row && (!w || j > row - w);
                        z[c] = see ? z[c] : -INFINITY;
                    }
                } else if (!whole) {
#pragma unroll
                    for (int c = 0; c < N; ++c) z[c] = t < rq.len && t >= lo0 + lo1 * col_row[col0 + c] ? z[c] : -INFINITY;
                }
            };
            load_z(false);
            float over = -INFINITY;
#pragma unroll
            for (int c = 0; c < N; ++c) over = fmaxf(over, z[c]);
            if (group_or(grp, over > kSlack || sc.y > vref || !ok)) {
                // ---- the reference moves (or a wait ran out)
                if (group_or(grp, !ok)) {
                    ok = false;
                    break;
                }
                load_z(true);
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    const float x = warp_max(z[c]);
                    if (lane == 0) col_max[warp & 3][col0 + c] = x;
                }
                const uint32_t vm = __reduce_max_sync(0xffffffffu, __float_as_uint(sc.y));
                if (lane == 0) v_max[grp][warp & 3] = __uint_as_float(vm);
                group_sync(grp);
                if (pos_in < N) {
                    const int c = col0 + pos_in;
                    const float was = -col_nm[c];
                    const float now =
                        fmaxf(fmaxf(fmaxf(col_max[0][c], col_max[1][c]), fmaxf(col_max[2][c], col_max[3][c])), was);
                    col_fac[c] = ex2(was - now);
                    col_nm[c] = -now;
                }
                const float vnow = fmaxf(fmaxf(fmaxf(v_max[grp][0], v_max[grp][1]), fmaxf(v_max[grp][2], v_max[grp][3])), vref);
                const float vfac = vref / vnow;
                vref = vnow;
                vinv = kBase / vnow;
                group_sync(grp);
#pragma unroll
                for (int c = 0; c < N; c += 2) {
                    l[c / 2] = mul2(l[c / 2], *reinterpret_cast<const f2 *>(col_fac + col0 + c));
                    z[c] += col_nm[col0 + c];
                    z[c + 1] += col_nm[col0 + c + 1];
                }
                if (i > 0) {
                    ok = gdn::mbar_wait_bounded(&pv_done[(i - 1) & 1], ((i - 1) >> 1) & 1, a.wait_ns);
                    if (group_or(grp, !ok)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after();
#pragma unroll 1
                    for (int x = 0; x < C::kAtoms * 4 * N; x += 8) {  // this group's columns of every part
                        const int at = x / N * RB + col0 + x % N;
                        uint32_t w[8];
                        tc::ld8_async(tm_o + lane_base + at, w);
                        tc::ld_wait();
                        tc::ld_fence_regs(w);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            w[c] = __float_as_uint(__uint_as_float(w[c]) * (col_fac[at % RB + c] * vfac));
                        tc::st8(tm_o + lane_base + at, w);
                    }
                    tc::st_wait();
                }
            }
            // scores are read: their buffer is free
            tc::fence_before();
            __syncwarp();
            if (lane == 0) arrive(&s_free[i & 1]);

            if (is_fresh) {
                if (pos_in < 16) {
#pragma unroll
                    for (int c = 0; c < N; c += 2) {
                        const f2 p = pair(ex2(z[c]), ex2(z[c + 1]));
                        l[c / 2] = add2(l[c / 2], p);
                        *reinterpret_cast<f2 *>(fresh_p + pos_in * RB + col0 + c) = p;
                    }
                }
                break;  // the last tile
            }
            const float xw = sc.y * vinv;
            const f2 xw2 = pair(xw, xw), xw32 = pair(32.f * xw, 32.f * xw);
            if (ok && i >= 2) ok = gdn::mbar_wait_bounded(&pv_done[i & 1], ((i >> 1) - 1) & 1, a.wait_ns);
            uint8_t *pb = s_p + (i & 1) * C::kP;
            // sixteen columns (eight if there are no more) at a time: 16 bytes of each part
            constexpr int W = N < 16 ? 8 : 16;
#pragma unroll
            for (int c0 = 0; c0 < N; c0 += W) {
                uint16_t e[4][W / 2];
#pragma unroll
                for (int c = 0; c < W / 2; ++c) {
                    const f2 p = pair(ex2(z[c0 + 2 * c]), ex2(z[c0 + 2 * c + 1]));
                    l[c0 / 2 + c] = add2(l[c0 / 2 + c], p);
                    const float2 x = both(mul2(p, xw2));
                    e[0][c] = uint16_t(kv8::e4m3x2(x.x, x.y));
                    const float2 r = minus32(both(mul2(p, xw32)), kv8::f16x2_of(e[0][c]));  // exact
                    uint32_t rest = f16x2(r.x, r.y);
                    e[1][c] = e4m3x2_of(rest);
                    rest = rest32(rest, kv8::f16x2_of(e[1][c]));
                    e[2][c] = e4m3x2_of(rest);
                    e[3][c] = e4m3x2_of(rest32(rest, kv8::f16x2_of(e[2][c])));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int b = k * RB + col0 + c0;  // byte of the row
                    uint8_t *dst = pb + (b / C::kPRow) * kTile * C::kPRow +
                                   tc::swz8_off<C::kPRow>(pos_in, (b % C::kPRow) >> 4) + (b & 8);
                    if constexpr (W == 16)
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(join16(e[k][0], e[k][1]), join16(e[k][2], e[k][3]),
                                                                     join16(e[k][4], e[k][5]), join16(e[k][6], e[k][7]));
                    else
                        *reinterpret_cast<uint2 *>(dst) = make_uint2(join16(e[k][0], e[k][1]), join16(e[k][2], e[k][3]));
                }
            }
            if (!whole && grp == 0) {
                // What no row sees may hold anything, NaN codes too, and 0 * NaN is
                // NaN: its values become zero.  Positions only some rows see keep
                // their values but for NaN, which the epilogue gives to those rows.
                const int pos = v_pos(i, nc), slot = pos % C::kSlots;
                if (ok) ok = gdn::mbar_wait_bounded(&full[slot], (pos / C::kSlots) & 1, a.wait_ns);
                const bool none = t < rq.lo || t >= rq.len, some = !none && t < lo_last;
                if (ok && (none || some)) {
#pragma unroll
                    for (int x = 0; x < C::kAtoms; ++x)
#pragma unroll
                        for (int k = 0; k < C::kRow / 16; ++k) {
                            uint4 *p = reinterpret_cast<uint4 *>(s_ring + slot * C::kSlot + x * kTile * C::kRow +
                                                                 tc::swz8_off<C::kRow>(pos_in, k));
                            uint4 w = make_uint4(0, 0, 0, 0);
                            if (some) {
                                w = *p;
                                uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                                for (int b = 0; b < 4; ++b)
                                    u[b] &= ~__vcmpeq4(u[b] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            }
                            *p = w;
                        }
                }
            }
            gdn::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&p_full[i & 1]);
        }
        // ---- the piece's end
        if (ok && nc > 0) ok = gdn::mbar_wait_bounded(&pv_done[(nc - 1) & 1], ((nc - 1) >> 1) & 1, a.wait_ns);
        if (ok && fresh && rq.n > 0) ok = gdn::mbar_wait_bounded(&fv_full, 0, a.wait_ns);
        const bool bad = *reinterpret_cast<volatile int *>(&bad_page) != 0;  // set before the last tile's scales
        const bool skip = group_or(grp, !ok || bad);
        if (!ok) gdn::set_status(a.status, GDN_DEV_TIMEOUT);
        if (bad && pos_in == 0) gdn::set_status(a.status, GDN_DEV_PAGE_OOR);
        tc::fence_after();
        // sums over the 128 positions
        float sums[N];
#pragma unroll
        for (int c = 0; c < N / 2; ++c) {
            sums[2 * c] = both(l[c]).x;
            sums[2 * c + 1] = both(l[c]).y;
        }
        warp_sums<N>(sums, lane);
        if ((lane & (32 / N - 1)) == 0) col_max[warp & 3][col0 + lane / (32 / N)] = sums[0];
        group_sync(grp);
        const bool direct = rq.pieces == 1;
        const int64_t unit = (int64_t(r) * a.max_pieces + piece) * gridDim.y + blockIdx.y;
        if (pos_in < N) {
            const int c = col0 + pos_in;
            const float sum = (col_max[0][c] + col_max[1][c]) + (col_max[2][c] + col_max[3][c]);
            if (!direct) {
                a.ws_ml[unit * RB + c] = make_float2(-col_nm[c], skip ? -1.f : sum);
            } else if (a.lse && c < cols && !skip) {
                a.lse[(int64_t(rq.t0) + col_row[c]) * a.c.h_q + hk * a.group + col_head[c]] =
                    sum == 0.f ? -INFINITY : (log2f(sum) - col_nm[c]) * 0.6931471805599453f;
            }
            col_l[c] = sum == 0.f ? 0.f : 1.f / sum;
        }
        group_sync(grp);
        if (!skip) {
            const float back = vref / kBase;
            const int edge = min(min(lo_last, rq.len), (tile0 + nc) * kTile);
#pragma unroll 1
            for (int x = 0; x < C::kAtoms; ++x) {
                const int e = x * C::kRow + pos_in;  // this thread's element (d = 64: lanes past 63 hold none)
                const bool mine = e < D;
#pragma unroll 1
                for (int c0 = col0; c0 < min(cols, col0 + N); c0 += 8) {
                    uint32_t w0[8], w1[8], w2[8], w3[8];
                    float o[8];
                    if (nc > 0) {
                        tc::ld8_async(tm_o + lane_base + x * C::kNp + c0, w0);
                        tc::ld8_async(tm_o + lane_base + x * C::kNp + RB + c0, w1);
                        tc::ld8_async(tm_o + lane_base + x * C::kNp + 2 * RB + c0, w2);
                        tc::ld8_async(tm_o + lane_base + x * C::kNp + 3 * RB + c0, w3);
                        tc::ld_wait();
                        tc::ld_fence_regs(w0);
                        tc::ld_fence_regs(w1);
                        tc::ld_fence_regs(w2);
                        tc::ld_fence_regs(w3);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const float s = fmaf(__uint_as_float(w3[c]), 1.f / 32.f, __uint_as_float(w2[c]));
                            o[c] = back * fmaf(fmaf(s, 1.f / 32.f, __uint_as_float(w1[c])), 1.f / 32.f,
                                               __uint_as_float(w0[c]));
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 8; ++c) o[c] = 0.f;
                    }
                    if (!mine) continue;
                    if (fresh) {
                        int row[8];
#pragma unroll
                        for (int c = 0; c < 8; ++c) row[c] = col_row[c0 + c];
                        const int wdw = a.c.window ? a.c.window : GDN_MAX_ROWS;
                        for (int j = 0; j < rq.n; ++j) {
                            const float v = gdn::bf16_to_f32(reinterpret_cast<const uint16_t *>(s_fv)[j * D + e]);
                            const float4 p0 = *reinterpret_cast<const float4 *>(fresh_p + j * RB + c0),
                                         p1 = *reinterpret_cast<const float4 *>(fresh_p + j * RB + c0 + 4);
                            const float p[8] = {p0.x, p0.y, p0.z, p0.w, p1.x, p1.y, p1.z, p1.w};
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                o[c] = uint32_t(row[c] - j) < uint32_t(wdw) ? fmaf(p[c], v, o[c]) : o[c];
                        }
                    }
                    // NaN of positions that only some rows see
                    for (int t = max(rq.lo, tile0 * kTile); t < edge; ++t) {
                        const int page = a.table[int64_t(r) * a.table_stride + (t >> shift)];
                        const uint8_t code = a.c.kv[int64_t(page) * a.c.page_stride + int64_t(a.layer) * a.c.layer_stride +
                                                    (int64_t(a.c.h_kv + hk) * T + (t & (T - 1))) * D + e];
                        if ((code & 0x7f) == 0x7f) {
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                if (c0 + c < cols && t >= lo0 + lo1 * col_row[c0 + c]) o[c] = __uint_as_float(0x7fc00000u);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        if (c0 + c >= cols) break;
                        if (direct)
                            a.o[(int64_t(rq.t0) + col_row[c0 + c]) * a.o_stride +
                                int64_t(hk * a.group + col_head[c0 + c]) * D + e] = gdn::f32_to_bf16(o[c] * col_l[c0 + c]);
                        else
                            a.ws_o[(unit * RB + c0 + c) * D + e] = o[c];
                    }
                }
            }
        }
        tc::fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after();
        tc::tmem_dealloc(tm, C::kTmem);
    }
}

// Joins a request's pieces: o = sum 2^(m_s - M) O_s / sum 2^(m_s - M) l_s.
// Groups of d/4 threads; a CTA takes `per_cta` columns of a (request, kv head,
// block).  With few pieces a group joins a column by itself; with many the
// groups share one column's pieces, so that their loads are in flight together.
// Which of the two, and so the order of the sums, goes by the pieces alone.
constexpr int kJoin = 512;

template <int D>
__global__ void __launch_bounds__(kJoin) kv8_join_kernel(const __grid_constant__ AttendArgs a, const int RB,
                                                         const int per_cta) {
    gdn::pdl_enter();
    constexpr int W = D / 4, G = kJoin / W;
    const int hk = blockIdx.y / a.blocks, blk = blockIdx.y % a.blocks, r = blockIdx.z, tid = threadIdx.x;
    const Request rq = request_of(a, r);
    if (rq.bad || rq.pieces <= 1) return;
    const int begin = blockIdx.x * per_cta, end = min(min(RB, rq.n * a.group - blk * RB), begin + per_cta);
    const int64_t unit0 = int64_t(r) * a.max_pieces * gridDim.y + blockIdx.y;
    __shared__ float s_l[G];
    __shared__ float4 s_o[G][W];
    const int g = tid / W, e = tid % W;
    const bool few = rq.pieces <= 8;
    const int step = few ? G : 1, ps = few ? 1 : G, p0 = few ? 0 : g;
    for (int c = begin + (few ? g : 0); c < end; c += step) {
        const float2 *ml0 = a.ws_ml + unit0 * RB + c;
        const int64_t ml_step = int64_t(gridDim.y) * RB;
        float m = -INFINITY;
        bool skip = false;
#pragma unroll 8
        for (int s = 0; s < rq.pieces; ++s) {
            const float2 ml = ml0[s * ml_step];
            m = fmaxf(m, ml.x);
            skip |= ml.y < 0.f;
        }
        if (skip) return;  // a piece was refused: so for every thread of the request
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
#pragma unroll 4
        for (int s = p0; s < rq.pieces; s += ps) {
            const float2 ml = ml0[s * ml_step];
            const float4 o =
                __ldcs(reinterpret_cast<const float4 *>(a.ws_o + ((unit0 + int64_t(s) * gridDim.y) * RB + c) * D) + e);
            const float f = ex2(ml.x - m);
            if (ml.y != 0.f) {  // else the row sees nothing of the piece
                l = fmaf(f, ml.y, l);
                acc.x = fmaf(f, o.x, acc.x);
                acc.y = fmaf(f, o.y, acc.y);
                acc.z = fmaf(f, o.z, acc.z);
                acc.w = fmaf(f, o.w, acc.w);
            }
        }
        if (!few) {
            __syncthreads();  // the last column's sums are read
            s_o[g][e] = acc;
            if (e == 0) s_l[g] = l;
            __syncthreads();
            if (g > 0) continue;
            for (int k = 1; k < G; ++k) {
                const float4 o = s_o[k][e];
                acc.x += o.x;
                acc.y += o.y;
                acc.z += o.z;
                acc.w += o.w;
                l += s_l[k];
            }
        }
        const int x = blk * RB + c, row = x / a.group, h = hk * a.group + x % a.group;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint2 w;
        w.x = gdn::f32_to_bf16(acc.x * inv) | (uint32_t(gdn::f32_to_bf16(acc.y * inv)) << 16);
        w.y = gdn::f32_to_bf16(acc.z * inv) | (uint32_t(gdn::f32_to_bf16(acc.w * inv)) << 16);
        *reinterpret_cast<uint2 *>(a.o + (int64_t(rq.t0) + row) * a.o_stride + int64_t(h) * D + e * 4) = w;
        if (e == 0 && a.lse)
            a.lse[(int64_t(rq.t0) + row) * a.c.h_q + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// A layer's pages as [page][2 h_kv page_tokens rows][d] bytes; boxes of one
// page and head, rows of at most 128 bytes, swizzled to that width.
bool encode_pages(CUtensorMap *m, const kv8_cache *c, int layer) {
    const EncodeTiledFn fn = encode_tiled();
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
    int rb, blocks, piece_tiles, max_pieces;
};

Plan plan_of(const kv8_cache *c, int32_t B, int32_t max_len, int32_t max_rows, int32_t split_tokens) {
    Plan p;
    const int64_t cols = int64_t(max_rows) * (c->h_q / c->h_kv);
    const int most = c->d == 256 ? 32 : 64;
    p.rb = cols <= 8 ? 8 : cols <= 16 ? 16 : cols <= 32 || most == 32 ? 32 : 64;
    p.blocks = int((cols + p.rb - 1) / p.rb);
    // positions a request's rows can see, and the tiles they may lie in
    int64_t seen = max_len;
    if (c->window && c->window < seen) seen = int64_t(c->window) + kTile;
    const int64_t tiles = (seen + kTile - 1) / kTile;
    const int64_t units = int64_t(B) * c->h_kv * p.blocks;
    const int64_t slots = 152 * (c->d == 256 || p.rb == 64 ? 1 : 2);
    int64_t t;
    if (split_tokens > 0)
        t = (int64_t(split_tokens) + kTile - 1) / kTile;
    else
        t = (tiles * units + slots - 1) / slots;  // one wave
    if (split_tokens <= 0 && t > 32) t = 32;
    if (t > tiles) t = tiles;
    if (t < 1) t = 1;
    p.piece_tiles = int(t);
    p.max_pieces = int(tiles > 0 ? (tiles + t - 1) / t : 1);
    return p;
}

template <int D, int RB>
int launch(const AttendArgs &a, dim3 grid, cudaStream_t st) {
    using C = Cfg<D, RB>;
    static const cudaError_t set = cudaFuncSetAttribute(kv8_attend_kernel<D, RB>,
                                                        cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (set != cudaSuccess) return GDN_ERR_CUDA;
    return gdn_host::launch_pdl(kv8_attend_kernel<D, RB>, grid, dim3(C::kThreads), C::kSmem, st, a);
}

}  // namespace

static size_t ws_bytes(const kv8_cache *c, int32_t B, const Plan &p) {
    if (p.max_pieces <= 1) return 0;
    const size_t cols = size_t(B) * p.max_pieces * c->h_kv * p.blocks * p.rb;
    return cols * (size_t(c->d) * 4 + 8);
}

extern "C" size_t kv8_attend_workspace_bytes(const kv8_cache *cache, int32_t B, int32_t max_len, int32_t max_rows,
                                             int32_t split_tokens) {
    if (gdn_host::kv8_check(cache) != GDN_OK || B <= 0 || max_len < 0 || max_len > gdn_host::kKv8MaxLen ||
        max_rows <= 0 || max_rows > GDN_MAX_ROWS || split_tokens < 0)
        return 0;
    return ws_bytes(cache, B, plan_of(cache, B, max_len, max_rows, split_tokens));
}

extern "C" int kv8_attend(const kv8_cache *cache, int32_t layer, int32_t B, int32_t row_capacity,
                          const int32_t *cu_rows, const int32_t *cache_len, const int32_t *table,
                          int32_t table_pages, int64_t table_stride, const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k_new,
                          int64_t k_stride, const gdn_bf16 *v_new, int64_t v_stride, gdn_bf16 *o, int64_t o_stride,
                          float *lse, int32_t max_len, int32_t max_rows, int32_t split_tokens, void *workspace,
                          size_t workspace_bytes, uint32_t *dev_status, void *stream) {
    const int bad = gdn_host::kv8_check(cache);
    if (bad != GDN_OK) return bad;
    if (layer < 0 || layer >= cache->num_layers || B < 0 || B > 65535 || row_capacity < 0 || table_pages < 0 ||
        table_stride < 0 ||
        max_len < 0 || max_len > gdn_host::kKv8MaxLen || max_rows < 0 || max_rows > GDN_MAX_ROWS || split_tokens < 0)
        return GDN_ERR_ARG;
    if (B == 0 || max_rows == 0) return GDN_OK;
    if (!cu_rows || !cache_len || (!table && table_pages > 0) || !q || !o || !k_new != !v_new) return GDN_ERR_NULL;
    if (!gdn_host::kv8_rows_ok(q, q_stride, cache->h_q, cache->d) ||
        !gdn_host::kv8_rows_ok(o, o_stride, cache->h_q, cache->d))
        return GDN_ERR_ARG;
    if (k_new && (!gdn_host::kv8_rows_ok(k_new, k_stride, cache->h_kv, cache->d) ||
                  !gdn_host::kv8_rows_ok(v_new, v_stride, cache->h_kv, cache->d)))
        return GDN_ERR_ARG;
    const Plan p = plan_of(cache, B, max_len, max_rows, split_tokens);
    const size_t need = ws_bytes(cache, B, p);
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
    a.ws_o = static_cast<float *>(workspace);
    a.ws_ml = need ? reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) +
                                                need / (size_t(cache->d) * 4 + 8) * (size_t(cache->d) * 4))
                   : nullptr;
    a.status = dev_status;
    a.wait_ns = gdn::kWaitLimitNs;
    const dim3 grid(unsigned(p.max_pieces), unsigned(cache->h_kv * p.blocks), unsigned(B));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int rc = GDN_ERR_SHAPE;
    const int key = cache->d * 100 + p.rb;
    switch (key) {
        case 6408: rc = launch<64, 8>(a, grid, st); break;
        case 6416: rc = launch<64, 16>(a, grid, st); break;
        case 6432: rc = launch<64, 32>(a, grid, st); break;
        case 6464: rc = launch<64, 64>(a, grid, st); break;
        case 12808: rc = launch<128, 8>(a, grid, st); break;
        case 12816: rc = launch<128, 16>(a, grid, st); break;
        case 12832: rc = launch<128, 32>(a, grid, st); break;
        case 12864: rc = launch<128, 64>(a, grid, st); break;
        case 25608: rc = launch<256, 8>(a, grid, st); break;
        case 25616: rc = launch<256, 16>(a, grid, st); break;
        case 25632: rc = launch<256, 32>(a, grid, st); break;
        default: break;
    }
    if (rc != GDN_OK || p.max_pieces <= 1) return rc;
    // as many columns a CTA as still leave four CTAs for each SM
    const int64_t columns = int64_t(B) * grid.y * p.rb;
    const int per = int(columns / (4 * 152) < 1 ? 1 : columns / (4 * 152) > p.rb ? p.rb : columns / (4 * 152));
    const dim3 jgrid{unsigned((p.rb + per - 1) / per), grid.y, unsigned(B)};
    if (cache->d == 64) return gdn_host::launch_pdl(kv8_join_kernel<64>, jgrid, dim3(kJoin), 0, st, a, p.rb, per);
    if (cache->d == 128) return gdn_host::launch_pdl(kv8_join_kernel<128>, jgrid, dim3(kJoin), 0, st, a, p.rb, per);
    return gdn_host::launch_pdl(kv8_join_kernel<256>, jgrid, dim3(kJoin), 0, st, a, p.rb, per);
}
