// Attention of a transaction's rows over the paged 8-bit cache (sm_103a).
//
// One CTA per (row, query head); its warps take every eighth position, each
// keeping a running maximum, sum and weighted value, joined at the end.
#include "kv8.cuh"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct AttendArgs {
    kv8_cache c;
    int32_t layer, B, row_capacity, table_stride, max_len, max_rows;
    const int32_t *cu_rows, *cache_len, *table;
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride, o_stride;
    uint16_t *o;
    float *lse;
    uint32_t *status;
};

template <int D>
__global__ void __launch_bounds__(kThreads) kv8_attend_kernel(const AttendArgs a) {
    gdn::pdl_enter();
    constexpr int E = D / 32;
    const int i = blockIdx.x, h = blockIdx.y, r = blockIdx.z;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int T = a.c.page_tokens;
    const int t0 = a.cu_rows[r], n = a.cu_rows[r + 1] - t0, len = a.cache_len[r];
    if (t0 < 0 || n < 0 || n > a.max_rows || int64_t(t0) + n > a.row_capacity || len < 0 || len > a.max_len ||
        int64_t(len) > int64_t(a.table_stride) * T) {
        if (i == 0 && h == 0 && threadIdx.x == 0) gdn::set_status(a.status, GDN_DEV_ROWS_BAD);
        return;
    }
    if (i >= n) return;
    const int hk = h / (a.c.h_q / a.c.h_kv), w = a.c.window;
    const int lo = w ? max(0, (a.k ? len + i + 1 : len) - w) : 0;
    bool bad = false;
    for (int t = lo / T + threadIdx.x; t * T < len; t += kThreads) {
        const int p = a.table[int64_t(r) * a.table_stride + t];
        bad |= p < 0 || p >= a.c.num_pages;
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) gdn::set_status(a.status, GDN_DEV_PAGE_OOR);
        return;
    }
    float q[E], acc[E], m = -INFINITY, l = 0.f;
    const float c = a.c.sm_scale;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = gdn::bf16_to_f32(a.q[(int64_t(t0) + i) * a.q_stride + int64_t(h) * D + e * 32 + lane]);
        acc[e] = 0.f;
    }
    const int news = a.k ? i + 1 : 0, skip = w ? max(0, i - w + 1) : 0;
    const int total = len - min(lo, len) + max(0, news - skip);
    for (int x = warp; x < total; x += kWarps) {
        float kk[E], vv[E];
        const int t = lo + x;
        if (t < len) {
            const int p = a.table[int64_t(r) * a.table_stride + t / T];
            const uint8_t *base = a.c.kv + int64_t(p) * a.c.page_stride + int64_t(a.layer) * a.c.layer_stride +
                                  (int64_t(hk) * T + t % T) * D;
            const float *s = a.c.scale + int64_t(p) * a.c.scale_page_stride +
                             int64_t(a.layer) * a.c.scale_layer_stride + 2 * hk;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                kk[e] = kv8::f32x2_of(base[e * 32 + lane]).x * s[0];
                vv[e] = kv8::f32x2_of(base[int64_t(a.c.h_kv) * T * D + e * 32 + lane]).x * s[1];
            }
        } else {
            const int64_t j = int64_t(t0) + skip + (x - (len - min(lo, len)));
#pragma unroll
            for (int e = 0; e < E; ++e) {
                kk[e] = gdn::bf16_to_f32(a.k[j * a.k_stride + int64_t(hk) * D + e * 32 + lane]);
                vv[e] = gdn::bf16_to_f32(a.v[j * a.v_stride + int64_t(hk) * D + e * 32 + lane]);
            }
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], kk[e], s);
#pragma unroll
        for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s *= c;
        const float top = fmaxf(m, s), f = m == top ? 1.f : expf(m - top), p = expf(s - top);
        m = top;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + p * vv[e];
    }
    __shared__ float sm[kWarps], sl[kWarps], sa[kWarps][D];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sa[warp][e * 32 + lane] = acc[e];
    __syncthreads();
    float top = -INFINITY;
    for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sm[k]);
    float sum = 0.f, f[kWarps];
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        f[k] = sm[k] == -INFINITY ? 0.f : expf(sm[k] - top);
        sum += f[k] * sl[k];
    }
    for (int e = threadIdx.x; e < D; e += kThreads) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) x += f[k] * sa[k][e];
        a.o[(int64_t(t0) + i) * a.o_stride + int64_t(h) * D + e] = gdn::f32_to_bf16(total ? x / sum : 0.f);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[(int64_t(t0) + i) * a.c.h_q + h] = total ? top + logf(sum) : -INFINITY;
}

}  // namespace

extern "C" size_t kv8_attend_workspace_bytes(const kv8_cache *cache, int32_t B, int32_t max_len, int32_t max_rows,
                                             int32_t split_tokens) {
    return 0;
}

extern "C" int kv8_attend(const kv8_cache *cache, int32_t layer, int32_t B, int32_t row_capacity,
                          const int32_t *cu_rows, const int32_t *cache_len, const int32_t *table,
                          int32_t table_stride, const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k_new,
                          int64_t k_stride, const gdn_bf16 *v_new, int64_t v_stride, gdn_bf16 *o, int64_t o_stride,
                          float *lse, int32_t max_len, int32_t max_rows, int32_t split_tokens, void *workspace,
                          size_t workspace_bytes, uint32_t *dev_status, void *stream) {
    const int bad = gdn_host::kv8_check(cache);
    if (bad != GDN_OK) return bad;
    if (layer < 0 || layer >= cache->num_layers || B < 0 || B > 65535 || row_capacity < 0 || table_stride < 0 ||
        max_len < 0 || max_len > gdn_host::kKv8MaxLen || max_rows < 0 || max_rows > GDN_MAX_ROWS || split_tokens < 0)
        return GDN_ERR_ARG;
    if (B == 0 || max_rows == 0) return GDN_OK;
    if (!cu_rows || !cache_len || (!table && table_stride > 0) || !q || !o || !k_new != !v_new) return GDN_ERR_NULL;
    if (!gdn_host::kv8_rows_ok(q, q_stride, cache->h_q, cache->d) ||
        !gdn_host::kv8_rows_ok(o, o_stride, cache->h_q, cache->d))
        return GDN_ERR_ARG;
    if (k_new && (!gdn_host::kv8_rows_ok(k_new, k_stride, cache->h_kv, cache->d) ||
                  !gdn_host::kv8_rows_ok(v_new, v_stride, cache->h_kv, cache->d)))
        return GDN_ERR_ARG;
    AttendArgs a{};
    a.c = *cache;
    a.layer = layer;
    a.B = B;
    a.row_capacity = row_capacity;
    a.table_stride = table_stride;
    a.max_len = max_len;
    a.max_rows = max_rows;
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
    a.status = dev_status;
    const dim3 grid(unsigned(max_rows), unsigned(cache->h_q), unsigned(B));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache->d == 64) return gdn_host::launch_pdl(kv8_attend_kernel<64>, grid, dim3(kThreads), 0, st, a);
    if (cache->d == 128) return gdn_host::launch_pdl(kv8_attend_kernel<128>, grid, dim3(kThreads), 0, st, a);
    return gdn_host::launch_pdl(kv8_attend_kernel<256>, grid, dim3(kThreads), 0, st, a);
}
