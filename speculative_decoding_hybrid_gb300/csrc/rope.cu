// Rotary positions of packed rows (sm_103a).
//
// Channel pair j of a head turns by position * f_j.  Angles are held in turns, as 64-bit fixed
// point: position * round(2^64 f_j / 2 pi) modulo 2^64 is the fraction of a turn, off by 2^-34 of
// one at the farthest position (a product in fp32 is off by 0.06 rad at position 10^6), and costs
// one integer multiplication.  Its upper 32 bits as an fp32 number of half turns are off by 2^-32
// and 2^-26 of a turn more, 10^-7 rad: a bf16 result wants 2^-9.  A thread makes the cosines and
// sines of its channels once a row and takes them through the row's heads, 16 bytes at a time.
// HBM-bound: 67,237 rows of 40 heads of 128 in 211 us, 6.53 TB/s, 96 % of a copy's rate; 1,024
// rows 6.7 us, one row 3.4 us, a launch and a chain of loads.  Where rot is no multiple of 16 a
// half's pieces do not begin at 16 bytes, and the row goes 2 bytes at a time: the same rows with
// 120 of 128 channels turned 755 us, 1.8 TB/s (rot of 16, 32, 64, 96 and whole heads are wide).
#include "kv8.cuh"
#include "prompt.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kMostRows = 256;  // rows of a CTA

struct RopeArgs {
    rope_spec c;
    prompt::Requests rq;
    int32_t rows, team;  // rows of a CTA; threads of a row
    const uint64_t *turns;
    const uint16_t *q, *k;
    uint16_t *q_out, *k_out;
    int64_t q_stride, k_stride, qo_stride, ko_stride;
    int32_t copy;        // the channels behind the rotated ones go to another place
    uint32_t *status;
};

__device__ __forceinline__ uint32_t turned(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int V>
struct Vec;
template <>
struct Vec<8> {
    typedef uint4 T;
};
template <>
struct Vec<1> {
    typedef uint16_t T;
};

template <int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    gdn::pdl_enter();
    __shared__ int pos[kMostRows];  // -1: nobody's row
    const int tid = threadIdx.x, row0 = blockIdx.x * a.rows, rows = min(a.rows, a.rq.row_capacity - row0);
    for (int i = tid; i < rows; i += kThreads) pos[i] = -1;
    __syncthreads();
    for (int r = tid; r < a.rq.B; r += kThreads) {
        const prompt::Request q = prompt::request_of(a.rq, r);
        if (q.bad || int64_t(q.len) + q.n > INT32_MAX) {
            if (blockIdx.x == 0) gdn::set_status(a.status, GDN_DEV_ROWS_BAD);
            continue;
        }
        for (int i = max(q.t0, row0); i < min(q.t0 + q.n, row0 + rows); ++i) pos[i - row0] = q.len + (i - q.t0);
    }
    __syncthreads();
    const int d = a.c.d, rot = a.c.rot, half = rot / 2, heads = a.c.h_q + a.c.h_kv;
    const int teams = kThreads / a.team, in = tid % a.team;
    const int P = half / V;                    // threads that a head's pairs take
    const int each = max(1, a.team / P);       // heads at a time
    for (int i = tid / a.team; i < rows; i += teams) {
        const int at = pos[i];
        if (at < 0) continue;
        const uint16_t *q = a.q + (int64_t(row0) + i) * a.q_stride, *k = a.k + (int64_t(row0) + i) * a.k_stride;
        uint16_t *qo = a.q_out + (int64_t(row0) + i) * a.qo_stride, *ko = a.k_out + (int64_t(row0) + i) * a.ko_stride;
        auto from = [&](int h) { return h < a.c.h_q ? q + h * d : k + (h - a.c.h_q) * d; };
        auto to = [&](int h) { return h < a.c.h_q ? qo + h * d : ko + (h - a.c.h_q) * d; };
        for (int p0 = in; p0 < P * each; p0 += a.team) {
            const int p = p0 % P, j0 = p * V;
            float c[V], s[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const uint64_t t = a.turns[j0 + e] * uint64_t(uint32_t(at));
                sincospif(float(int32_t(t >> 32)) * 0x1p-31f, &s[e], &c[e]);
                c[e] *= a.c.magnitude;
                s[e] *= a.c.magnitude;
            }
            // halves lie apart, interleaved pairs side by side
            const int x0 = INTER ? 2 * j0 : j0, x1 = INTER ? 2 * j0 + V : half + j0;
#pragma unroll 4
            for (int h = p0 / P; h < heads; h += each) {
                const uint16_t *x = from(h);
                uint16_t *y = to(h);
                if constexpr (V == 8) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(x + x0), w = *reinterpret_cast<const uint4 *>(x + x1);
                    const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
                    uint32_t yu[4], yw[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float a0 = __uint_as_float(uu[e] << 16), a1 = __uint_as_float(uu[e] & 0xffff0000u);
                        const float b0 = __uint_as_float(ww[e] << 16), b1 = __uint_as_float(ww[e] & 0xffff0000u);
                        if constexpr (INTER) {
                            yu[e] = turned(a0 * c[e] - a1 * s[e], a0 * s[e] + a1 * c[e]);
                            yw[e] = turned(b0 * c[e + 4] - b1 * s[e + 4], b0 * s[e + 4] + b1 * c[e + 4]);
                        } else {
                            yu[e] = turned(a0 * c[2 * e] - b0 * s[2 * e], a1 * c[2 * e + 1] - b1 * s[2 * e + 1]);
                            yw[e] = turned(a0 * s[2 * e] + b0 * c[2 * e], a1 * s[2 * e + 1] + b1 * c[2 * e + 1]);
                        }
                    }
                    *reinterpret_cast<uint4 *>(y + x0) = make_uint4(yu[0], yu[1], yu[2], yu[3]);
                    *reinterpret_cast<uint4 *>(y + x1) = make_uint4(yw[0], yw[1], yw[2], yw[3]);
                } else {
                    const float u = gdn::bf16_to_f32(x[x0]), w = gdn::bf16_to_f32(x[x1]);
                    y[x0] = gdn::f32_to_bf16(u * c[0] - w * s[0]);
                    y[x1] = gdn::f32_to_bf16(u * s[0] + w * c[0]);
                }
            }
        }
        if (a.copy) {
            // (d and, for whole vectors, rot are multiples of 8)
            const int n = (d - rot) / V;
#pragma unroll 2
            for (int e = in; e < n * heads; e += a.team) {
                const int h = e / n, ch = rot + (e - h * n) * V;
                *reinterpret_cast<typename Vec<V>::T *>(to(h) + ch) =
                    *reinterpret_cast<const typename Vec<V>::T *>(from(h) + ch);
            }
        }
    }
}

}  // namespace

extern "C" int rope_rows(const rope_spec *spec, int32_t B, int32_t row_capacity, const int32_t *cu_rows,
                         const int32_t *cache_len, const uint64_t *turns, const gdn_bf16 *q, int64_t q_stride,
                         gdn_bf16 *q_out, int64_t q_out_stride, const gdn_bf16 *k, int64_t k_stride, gdn_bf16 *k_out,
                         int64_t k_out_stride, uint32_t *dev_status, void *stream) {
    if (!spec) return GDN_ERR_NULL;
    const int d = spec->d;
    if (d <= 0 || d > 512 || d % 8 || spec->rot <= 0 || spec->rot > d || spec->rot % 2 || spec->h_q < 0 ||
        spec->h_kv < 0 || spec->h_q + int64_t(spec->h_kv) <= 0 || spec->h_q + int64_t(spec->h_kv) > 65535)
        return GDN_ERR_SHAPE;
    if (!isfinite(spec->magnitude) || B < 0 || B > 65535 || row_capacity < 0) return GDN_ERR_ARG;
    if (B == 0 || row_capacity == 0) return GDN_OK;
    if (!cu_rows || !turns || (spec->h_q && (!q || !q_out)) || (spec->h_kv && (!k || !k_out))) return GDN_ERR_NULL;
    if (spec->h_q && (!gdn_host::kv8_rows_ok(q, q_stride, spec->h_q, d) ||
                      !gdn_host::kv8_rows_ok(q_out, q_out_stride, spec->h_q, d) ||
                      (q == q_out && q_stride != q_out_stride)))
        return GDN_ERR_ARG;
    if (spec->h_kv && (!gdn_host::kv8_rows_ok(k, k_stride, spec->h_kv, d) ||
                       !gdn_host::kv8_rows_ok(k_out, k_out_stride, spec->h_kv, d) ||
                       (k == k_out && k_stride != k_out_stride)))
        return GDN_ERR_ARG;
    RopeArgs a{};
    a.c = *spec;
    a.rq = {B, row_capacity, row_capacity, INT32_MAX, 0, INT32_MAX, cu_rows, cache_len};
    a.turns = turns;
    a.q = q;
    a.k = k;
    a.q_out = q_out;
    a.k_out = k_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.qo_stride = q_out_stride;
    a.ko_stride = k_out_stride;
    a.copy = spec->rot < d && ((spec->h_q && q != q_out) || (spec->h_kv && k != k_out));
    a.status = dev_status;
    const bool wide = spec->rot % 16 == 0;
    // A row has a warp; where there are few rows, as much of a CTA as its channels fill.
    a.team = 32;
    const int pieces = (spec->h_q + spec->h_kv) * (d / 8);
    while (a.team < kThreads && row_capacity * int64_t(a.team) < 152 * kThreads * 2 && a.team * 2 <= pieces) a.team *= 2;
    // Eight CTAs an SM, of whole teams.
    const int teams = kThreads / a.team;
    int64_t rows = (int64_t(row_capacity) + 152 * 8 - 1) / (152 * 8);
    rows = (rows + teams - 1) / teams * teams;
    a.rows = int(rows > kMostRows ? kMostRows : rows);
    const dim3 grid(unsigned((int64_t(row_capacity) + a.rows - 1) / a.rows));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (wide)
        return spec->interleaved ? gdn_host::launch_pdl(rope_kernel<8, true>, grid, dim3(kThreads), 0, st, a)
                                 : gdn_host::launch_pdl(rope_kernel<8, false>, grid, dim3(kThreads), 0, st, a);
    return spec->interleaved ? gdn_host::launch_pdl(rope_kernel<1, true>, grid, dim3(kThreads), 0, st, a)
                             : gdn_host::launch_pdl(rope_kernel<1, false>, grid, dim3(kThreads), 0, st, a);
}
