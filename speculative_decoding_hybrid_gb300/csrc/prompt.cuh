// What the attention over prompts and chunks shares between its kernels
// (sm_103a): the packed requests, and where their keys lie.
#pragma once

#include <math.h>

#include "common.cuh"

namespace prompt {

// Requests of packed rows: request r has rows cu_rows[r] .. cu_rows[r+1]-1 behind cache_len[r] earlier positions (NULL:
// none).  Keys and values of a request are consecutive rows of their tensor: the call's own rows (kv_capacity 0), or
// rows of a workspace where the earlier positions and the new rows of all requests lie one behind another.
struct Requests {
    int32_t B, row_capacity, max_rows, max_len;
    int64_t kv_capacity, max_pages_len;  // rows of the workspace; positions a row of the page table holds
    const int32_t *cu_rows, *cache_len;
};

struct Request {
    int t0, n, len;
    bool bad;
};
__device__ __forceinline__ Request request_of(const Requests &a, int r) {
    Request q;
    q.t0 = a.cu_rows[r];
    q.n = a.cu_rows[r + 1] - q.t0;
    q.len = a.cache_len ? a.cache_len[r] : 0;
    q.bad = q.t0 < 0 || q.n < 0 || q.n > a.max_rows || int64_t(q.t0) + q.n > a.row_capacity || q.len < 0 ||
            q.len > a.max_len || int64_t(q.len) > a.max_pages_len;
    if (q.bad) q.n = 0;
    return q;
}
// Rows of the workspace that a request takes.
__device__ __forceinline__ int64_t kv_rows_of(const Request &q) { return q.n ? int64_t(q.len) + q.n : 0; }

// Exclusive sums over a CTA's THREADS threads of two numbers each, and their totals.
template <int THREADS>
struct Scan {
    long long a[THREADS / 32], b[THREADS / 32];
};
template <int THREADS>
__device__ __forceinline__ void scan2(Scan<THREADS> &s, long long &a, long long &b, long long &a_all,
                                      long long &b_all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) a += x, b += y;
    }
    if (lane == 31) s.a[warp] = a, s.b[warp] = b;
    __syncthreads();
    a_all = b_all = 0;
    long long pa = 0, pb = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) pa += s.a[w], pb += s.b[w];
        a_all += s.a[w];
        b_all += s.b[w];
    }
    a += pa - a0;
    b += pb - b0;
}

}  // namespace prompt
