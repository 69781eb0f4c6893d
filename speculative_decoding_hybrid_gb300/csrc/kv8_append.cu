// Commit of rows into the paged 8-bit key/value cache, and page copies
// (sm_103a).
//
// kv8_append: a unit, a CTA or a warp of one, per (page touched, kv head and K or
// V).  A thread holds its pieces of 16 new elements (32 bytes of bf16) in registers
// between the two things done with them: the page's largest magnitude, which fixes
// the scale 2^e with amax <= 448 * 2^e, and the rounding to codes, so the rows are
// read once.  A power of two makes x / scale exact: a code is x rounded once, to
// e4m3's 4 bits, codes do not depend on the order of appends, and a scale that grows
// moves earlier codes exactly unless they fall into e4m3's subnormals.
// HBM-bound on prompts (2 bytes read and 1 written a value): the new rows are asked
// for before the page they go to is known.  8 prompts of 512..32768 tokens, 8 heads of
// 128, pages of 64: 88 us, 6.45 TB/s, 95 % of a copy's rate.  A decode's commit is
// a launch and one chain of loads: 4 rows x 256 requests, 2 heads of 256: 2.8 us.
#include "kv8_math.cuh"

namespace {

constexpr int kThreads = 256;  // of a page copy
constexpr int kPack = 4;       // units of one warp in a CTA

struct AppendArgs {
    kv8_cache c;
    int32_t layer, B, row_capacity, table_pages, max_rows;
    int32_t pages;  // that there are units for: of every request, or (ragged) of all together
    int64_t table_stride;
    const int32_t *cu_rows, *cache_len, *table, *accept_len;
    const uint16_t *k, *v;
    int64_t k_stride, v_stride;
    uint32_t *status;
};

// Largest magnitudes of pairs of bf16: magnitudes order like their bits.
__device__ __forceinline__ uint32_t max_of(const uint4 &w, uint32_t m) {
    m = __vmaxu2(m, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
    return __vmaxu2(m, __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
}
// The same without infinities and NaN.
__device__ __forceinline__ uint32_t max_finite_of(const uint4 &w, uint32_t m) {
    const uint32_t u[4] = {w.x & 0x7fff7fffu, w.y & 0x7fff7fffu, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, u[i] & __vcmpltu2(u[i], 0x7f807f80u));
    return m;
}

// 16 bf16 values -> 16 codes.
__device__ __forceinline__ uint4 encode16(const uint4 &a, const uint4 &b, float inv) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const kv8::f2 inv2 = kv8::pair(inv, inv);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lo = kv8::both(kv8::mul2(kv8::pair(w[2 * i] << 16, w[2 * i] & 0xffff0000u), inv2)),
                     hi = kv8::both(kv8::mul2(kv8::pair(w[2 * i + 1] << 16, w[2 * i + 1] & 0xffff0000u), inv2));
        o[i] = kv8::join16(uint16_t(kv8::e4m3x2(lo.x, lo.y)), uint16_t(kv8::e4m3x2(hi.x, hi.y)));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

struct Rows {
    int t0, rows, len, n;   // n: the rows to append
    uint32_t bad;
};
__device__ __forceinline__ Rows rows_of(const AppendArgs &a, int r) {
    Rows q;
    q.t0 = a.cu_rows[r];
    q.rows = a.cu_rows[r + 1] - q.t0;
    q.len = a.cache_len[r];
    const int j = a.accept_len ? a.accept_len[r] : 0;
    q.bad = 0;
    if (q.t0 < 0 || q.rows < 0 || q.rows > a.max_rows || int64_t(q.t0) + q.rows > a.row_capacity || q.len < 0 ||
        int64_t(q.len) + q.rows > int64_t(a.table_pages) * a.c.page_tokens)
        q.bad = GDN_DEV_ROWS_BAD;
    else if (a.accept_len && j >= q.rows)
        q.bad = GDN_DEV_ACCEPT_BAD;
    q.n = q.bad ? 0 : !a.accept_len ? q.rows : j < 0 ? 0 : j + 1;
    return q;
}

// One page of request rows `q`, its table's page len / T + step: a unit's THREADS threads,
// a CTA's or a warp's.  PIECES: the most 16-element pieces of a page a thread may hold.
template <int THREADS, int PIECES>
__device__ __forceinline__ void append_page(const AppendArgs &a, int r, const Rows &q, int step, int hv) {
    const int tid = THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int is_v = hv >= a.c.h_kv, h = hv - is_v * a.c.h_kv, T = a.c.page_tokens, d = a.c.d;
    const int page_shift = 31 - __clz(T), per_shift = 31 - __clz(d) - 4;  // 2^per_shift pieces a token
    const int t0 = q.t0, len = q.len;
    const int pj = (len >> page_shift) + step;                 // page of the request's table
    const int p0 = pj << page_shift;                      // its first position
    const int from = max(len, p0), to = min(len + q.n, p0 + T);
    if (from >= to) return;
    const uint16_t *x = is_v ? a.v : a.k;
    const int64_t stride = is_v ? a.v_stride : a.k_stride;
    const int held = from - p0;                    // tokens the page already holds
    const int total = (to - from) << per_shift;
    const uint16_t *src = x + (int64_t(t0) + (from - len)) * stride + int64_t(h) * d;

    uint4 w[PIECES][2];
    uint32_t m = 0;
    const int page = a.table[int64_t(r) * a.table_stride + pj];
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
        const int i = tid + u * THREADS;
        w[u][0] = w[u][1] = make_uint4(0, 0, 0, 0);
        if (i < total) {
            const int in = (i & ((1 << per_shift) - 1)) * 16;
            const uint4 *p = reinterpret_cast<const uint4 *>(src + int64_t(i >> per_shift) * stride + in);
            w[u][0] = __ldcs(p);
            w[u][1] = __ldcs(p + 1);
        }
    }
    if (page < 0 || page >= a.c.num_pages) {
        if (tid == 0) gdn::set_status(a.status, GDN_DEV_PAGE_OOR);
        return;
    }
    uint8_t *codes = a.c.kv + int64_t(page) * a.c.page_stride + int64_t(a.layer) * a.c.layer_stride +
                     (int64_t(is_v) * a.c.h_kv + h) * T * d;
    float *scale = a.c.scale + int64_t(page) * a.c.scale_page_stride + int64_t(a.layer) * a.c.scale_layer_stride +
                   2 * h + is_v;
    const float was = held ? *scale : 0.f;
#pragma unroll
    for (int u = 0; u < PIECES; ++u) m = max_of(w[u][1], max_of(w[u][0], m));
    if (max(m >> 16, m & 0xffffu) >= 0x7f80u) {
        m = 0;
#pragma unroll
        for (int u = 0; u < PIECES; ++u) m = max_finite_of(w[u][1], max_finite_of(w[u][0], m));
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, max(m >> 16, m & 0xffffu));
    if constexpr (THREADS > 32) {
        __shared__ uint32_t red[THREADS / 32];
        if ((tid & 31) == 0) red[tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < THREADS / 32; ++i) top = max(top, red[i]);
    } else {
        __syncwarp();
    }
    const int e = kv8::scale_exp(__uint_as_float(top << 16));
    const float fit = kv8::pow2i(e);
    const float now = fmaxf(was, fit);
    const float inv = 1.f / now;                   // exact: a power of two
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
        const int i = tid + u * THREADS;
        if (i < total) *reinterpret_cast<uint4 *>(codes + (held * d + i * 16)) = encode16(w[u][0], w[u][1], inv);
    }
    if (held && now > was) {
        const float f = was * inv;
#pragma unroll(THREADS <= 64 ? 4 : 1)
        for (int i = tid; i < held << per_shift; i += THREADS) {
            uint4 *p = reinterpret_cast<uint4 *>(codes + int64_t(i) * 16);
            const uint4 old = *p;
            uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 lo = kv8::f32x2_of(uint16_t(o[k])), hi = kv8::f32x2_of(uint16_t(o[k] >> 16));
                o[k] = kv8::e4m3x2(lo.x * f, lo.y * f) | (kv8::e4m3x2(hi.x * f, hi.y * f) << 16);
            }
            *p = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    // every thread has read *scale before the barrier above
    if (tid == 0) *scale = now;
}

constexpr int cta_of(int threads) { return threads == 32 ? 32 * kPack : threads; }
// Registers for a thread's pieces (8 words each) against threads in flight: 8 pieces at
// 512, 768 and 896 threads an SM 55, 50 and 52 us (a prompt of 8 requests, 1000..20000
// tokens, 8 heads of 128, pages of 32), 4 pieces at 1024, 1280 and 1536 (pages of 16) 54, 54 and 60.
// Two pieces at 1024, 1536 and 2048: 256 requests of 1..4 rows, 8 heads of 64, pages of 16
// 4.6, 4.7 and 5.7 us, 8 of 1000..20000 45, 41 and 50, 512 of 1..2 in pages of 32 6.7, 7.2 and 9.0.
constexpr int threads_an_sm(int pieces) { return pieces <= 4 ? 1024 : 768; }

// RAGGED: the units count the pages touched over all requests, each finding its
// request by a scan of the lengths; otherwise the pages one request may touch.
template <int THREADS, int PIECES, bool RAGGED>
__global__ void __launch_bounds__(cta_of(THREADS), threads_an_sm(PIECES) / cta_of(THREADS))
    kv8_append_kernel(const AppendArgs a) {
    gdn::pdl_enter();
    const int lane = threadIdx.x & 31;
    const bool reports = blockIdx.x == 0 && threadIdx.x < 32;
    const int unit = THREADS == 32 ? blockIdx.x * kPack + (threadIdx.x >> 5) : blockIdx.x;
    // the heads of a page side by side: their parts of the rows are neighbours in memory
    const int heads = 2 * a.c.h_kv, first = unit / heads, hv = unit - first * heads;
    if (first >= a.pages) return;
    const int T = a.c.page_tokens, page_shift = 31 - __clz(T);
    if (a.status && (*reinterpret_cast<volatile uint32_t *>(a.status) & GDN_DEV_TIMEOUT)) return;
    if constexpr (!RAGGED) {
        const Rows q = rows_of(a, blockIdx.z);
        if (q.bad && blockIdx.x == 0 && threadIdx.x == 0) gdn::set_status(a.status, q.bad);
        append_page<THREADS, PIECES>(a, blockIdx.z, q, first, hv);
    } else {
        // every warp scans, 32 requests at a time; requests whose rows overlap may make
        // more pages than there are CTAs
        int at = first, total = 0;
        do {
            int r = -1, step = 0;
            total = 0;
            for (int r0 = 0; r0 < a.B; r0 += 32) {
                int pages = 0;
                if (r0 + lane < a.B) {
                    const Rows x = rows_of(a, r0 + lane);
                    if (x.bad && reports) gdn::set_status(a.status, x.bad);
                    if (x.n > 0) pages = ((x.len & (T - 1)) + x.n + T - 1) >> page_shift;
                }
                int incl = pages;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += y;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, total + incl > at);
                if (r < 0 && past) {
                    const int w = __ffs(past) - 1;
                    r = r0 + w;
                    step = at - total - __shfl_sync(0xffffffffu, incl - pages, w);
                }
                total += __shfl_sync(0xffffffffu, incl, 31);
            }
            if (r >= 0) append_page<THREADS, PIECES>(a, r, rows_of(a, r), step, hv);
            at += a.pages;
            if (THREADS > 32) __syncthreads();
        } while (at < total);
    }
}

struct CopyArgs {
    kv8_cache c;
    int32_t n, pieces;  // 16 KB pieces of a page and layer
    const int32_t *src, *dst;
    uint32_t *status;
};

constexpr int kPiece = 16384;

// One CTA per (16 KB piece of a page of a layer, layer, pair): all of its loads before
// its first store.  A copy, bound by HBM: 1.97 GB moved in 280 us, 7.02 TB/s.
__global__ void __launch_bounds__(kThreads) kv8_copy_kernel(const CopyArgs a) {
    gdn::pdl_enter();
    const int64_t id = blockIdx.x;
    const int piece = int(id % a.pieces);
    const int64_t rest = id / a.pieces;
    const int l = int(rest % a.c.num_layers), i = int(rest / a.c.num_layers);
    const int s = a.src[i], t = a.dst[i];
    if (s < 0 || s >= a.c.num_pages || t < 0 || t >= a.c.num_pages) {
        if (piece == 0 && l == 0 && threadIdx.x == 0) gdn::set_status(a.status, GDN_DEV_PAGE_OOR);
        return;
    }
    if (s == t) return;
    const int bytes = 2 * a.c.h_kv * a.c.page_tokens * a.c.d;
    const int at = piece * kPiece, n16 = min(kPiece, bytes - at) / 16;
    const int64_t lo = int64_t(l) * a.c.layer_stride + at;
    const uint4 *from = reinterpret_cast<const uint4 *>(a.c.kv + int64_t(s) * a.c.page_stride + lo);
    uint4 *to = reinterpret_cast<uint4 *>(a.c.kv + int64_t(t) * a.c.page_stride + lo);
    uint4 w[kPiece / 16 / kThreads];
#pragma unroll
    for (int u = 0; u < kPiece / 16 / kThreads; ++u)
        if (threadIdx.x + u * kThreads < n16) w[u] = __ldcs(from + threadIdx.x + u * kThreads);
#pragma unroll
    for (int u = 0; u < kPiece / 16 / kThreads; ++u)
        if (threadIdx.x + u * kThreads < n16) __stcs(to + threadIdx.x + u * kThreads, w[u]);
    if (piece == 0) {
        const int64_t ls = int64_t(l) * a.c.scale_layer_stride;
        for (int k = threadIdx.x; k < 2 * a.c.h_kv; k += kThreads)
            a.c.scale[int64_t(t) * a.c.scale_page_stride + ls + k] =
                a.c.scale[int64_t(s) * a.c.scale_page_stride + ls + k];
    }
}

}  // namespace

extern "C" int kv8_append(const kv8_cache *cache, int32_t layer, int32_t B, int32_t row_capacity,
                          const int32_t *cu_rows, const int32_t *cache_len, const int32_t *table,
                          int32_t table_pages, int64_t table_stride, const gdn_bf16 *k_new, int64_t k_stride,
                          const gdn_bf16 *v_new, int64_t v_stride, const int32_t *accept_len, int32_t max_rows,
                          uint32_t *dev_status, void *stream) {
    const int bad = gdn_host::kv8_check(cache);
    if (bad != GDN_OK) return bad;
    if (layer < 0 || layer >= cache->num_layers || B < 0 || B > 65535 || row_capacity < 0 || table_pages < 0 ||
        (B > 1 && table_stride < table_pages) ||
        max_rows < 0 || max_rows > gdn_host::kKv8MaxLen)
        return GDN_ERR_ARG;
    if (int64_t(table_pages) * cache->page_tokens > gdn_host::kKv8MaxLen) return GDN_ERR_ARG;
    if (B == 0 || max_rows == 0) return GDN_OK;
    // (an empty tensor's address is null: with no rows, or no pages, nothing of theirs is read)
    if (!cu_rows || !cache_len || (!table && table_pages > 0) || (row_capacity > 0 && (!k_new || !v_new)))
        return GDN_ERR_NULL;
    if (!gdn_host::kv8_rows_ok(k_new, k_stride, cache->h_kv, cache->d) ||
        !gdn_host::kv8_rows_ok(v_new, v_stride, cache->h_kv, cache->d))
        return GDN_ERR_ARG;
    AppendArgs a{};
    a.c = *cache;
    a.layer = layer;
    a.B = B;
    a.row_capacity = row_capacity;
    a.table_pages = table_pages;
    a.table_stride = table_stride;
    a.max_rows = max_rows;
    a.cu_rows = cu_rows;
    a.cache_len = cache_len;
    a.table = table;
    a.accept_len = accept_len;
    a.k = k_new;
    a.v = v_new;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.status = dev_status;
    const int T = cache->page_tokens;
    // n rows starting anywhere touch at most (T - 1 + n - 1) / T + 1 pages, and all
    // requests together at most row_capacity / T + 2 B.  Counting those saves units
    // without a page (8 requests of 512..32768 tokens 114 us without, 88 with; of
    // 1000..20000 into pages of 16, heads of 64, 60 and 45) and costs each unit a scan,
    // of 32 requests at a time (95 requests of 1..98 tokens 7.2 us without, 8.5 with; 256
    // of 4 rows 3.0 and 6.8).
    const int64_t each = (max_rows + T - 2) / T + 1, all = row_capacity / T + int64_t(2) * B;
    const bool ragged = all * (2 + B / 16) < each * B * 2;
    const int64_t pages = ragged ? all : each, units = pages * 2 * cache->h_kv;
    if (units > 0x7fffffff - kPack) return GDN_ERR_ARG;
    a.pages = int(pages);
    const int most = max_rows < T ? max_rows : T;
    const auto launch = [&](auto kernel, int threads) {
        const int64_t ctas = threads == 32 ? (units + kPack - 1) / kPack : units;
        return gdn_host::launch_pdl(kernel, dim3(unsigned(ctas), 1, unsigned(ragged ? 1 : B)),
                                    dim3(unsigned(cta_of(threads))), 0, static_cast<cudaStream_t>(stream), a);
    };
    // As few threads a page as hold its new pieces, eight each: units of one warp reduce
    // without a barrier (2 rows x 512 requests 17.2 us with 64 threads a page, 6.8 with
    // 32; the prompts above into pages of 16 tokens 86 and 45), and eight pieces keep more
    // of a prompt in flight than four by twice the threads (8 requests of 1000..20000, 8
    // heads of 128: 66.4 and 64.3 us in pages of 128, but 64.1 and 66.8 in pages of 32).
    // Two pieces, or four, where no page has more.
    const int all_pieces = most * cache->d / 16;
    if (ragged) {
        if (all_pieces <= 64) return launch(kv8_append_kernel<32, 2, true>, 32);
        if (all_pieces <= 128) return launch(kv8_append_kernel<32, 4, true>, 32);
        if (all_pieces <= 256) return launch(kv8_append_kernel<32, 8, true>, 32);
        if (all_pieces <= 512) return launch(kv8_append_kernel<64, 8, true>, 64);
        if (all_pieces <= 1024) return launch(kv8_append_kernel<128, 8, true>, 128);
        return launch(kv8_append_kernel<256, 8, true>, 256);
    }
    if (all_pieces <= 64) return launch(kv8_append_kernel<32, 2, false>, 32);
    if (all_pieces <= 128) return launch(kv8_append_kernel<32, 4, false>, 32);
    if (all_pieces <= 256) return launch(kv8_append_kernel<32, 8, false>, 32);
    if (all_pieces <= 512) return launch(kv8_append_kernel<64, 8, false>, 64);
    if (all_pieces <= 1024) return launch(kv8_append_kernel<128, 8, false>, 128);
    return launch(kv8_append_kernel<256, 8, false>, 256);
}

extern "C" int kv8_copy_pages(const kv8_cache *cache, int32_t n, const int32_t *src, const int32_t *dst,
                              uint32_t *dev_status, void *stream) {
    const int bad = gdn_host::kv8_check(cache);
    if (bad != GDN_OK) return bad;
    if (n < 0) return GDN_ERR_ARG;
    if (n == 0) return GDN_OK;
    if (!src || !dst) return GDN_ERR_NULL;
    CopyArgs a{};
    a.c = *cache;
    a.n = n;
    a.src = src;
    a.dst = dst;
    a.status = dev_status;
    a.pieces = int((int64_t(2) * cache->h_kv * cache->page_tokens * cache->d + kPiece - 1) / kPiece);
    const int64_t grid = int64_t(n) * cache->num_layers * a.pieces;
    if (grid > 0x7fffffffLL) return GDN_ERR_ARG;
    return gdn_host::launch_pdl(kv8_copy_kernel, dim3(unsigned(grid)), dim3(kThreads), 0,
                                static_cast<cudaStream_t>(stream), a);
}
