// The quantised KV cache: rows of K and V written as 4- or 8-bit affine codes, and
// read back.
//
// Per (token, kv head, K or V, 64 dims): mn, mx over the 64 fp16 values;
//     s = fp16((mx - mn) / (2^bits - 1)), b = mn,
//     q = clamp(rne((x - mn) / s), 0, 2^bits - 1)    (0 where s = 0),
// and the stored group stands for s q + b.  q is the exact quotient's rounding: the
// kernel rounds the fp32 product (x - mn) * (1 / s), and where that lies next to
// a border it decides by the sign of (x - mn) - (q +- 1/2) s, which fp32 holds
// exactly there.
#include "kvcache.cuh"

namespace edge0 {
namespace {

constexpr int kKvThreads = 256;
constexpr int kMaxRowsPerCta = 16;

// Where the rows of a CTA go: byte offset of each row's page, its token in the page.
struct RowPlace {
    long long page;   // byte offset of the page, or -1: nothing to do
    int token;        // token within the page
};

struct Rows {
    const int* table;
    int B, W;
    const int* start;
    const int* cu;    // [B + 1] or null: row b belongs to sequence b
    int T;
    int* status;
};

// The places of rows r0 .. r0 + n - 1 (n <= kMaxRowsPerCta), by the whole CTA.
__device__ void place_rows(const kv::View& c, const Rows& rows, int r0, int n, int* cu_s, RowPlace* out) {
    if (rows.cu) {
        for (int i = threadIdx.x; i <= rows.B; i += kKvThreads) cu_s[i] = rows.cu[i];
        __syncthreads();
    }
    if (threadIdx.x < n) {
        const int r = r0 + threadIdx.x;
        RowPlace p;
        p.page = -1;
        p.token = 0;
        int b = r;
        long long pos = 0;
        bool in = r < rows.T;
        if (rows.cu) {
            in = in && r >= cu_s[0] && r < cu_s[rows.B];
            int lo = 0, hi = rows.B;        // the last b with cu[b] <= r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu_s[mid] <= r) lo = mid;
                else hi = mid;
            }
            b = lo;
            pos = (long long)r - cu_s[b];
        }
        if (in) {
            const int st = rows.start[b];
            pos += st;
            if (st >= 0) {                  // a negative start: a padding sequence
                const long long pg = pos / c.page_tokens;
                int id = -1;
                if (pos >= 0 && pg < rows.W) id = rows.table[(long long)b * rows.W + pg];
                if (id >= 0 && id < c.n_pages) {
                    p.page = (long long)id * c.page_bytes;
                    p.token = (int)(pos - pg * c.page_tokens);
                } else if (rows.status) {
                    atomicExch(rows.status, EDGE0_EINVAL);
                }
            }
        }
        out[threadIdx.x] = p;
    }
    __syncthreads();
}

// byte address of the strip of (head h, token) in its page
template <int BITS, int D>
__device__ __forceinline__ char* strip_of(const kv::View& c, const RowPlace& p, int h) {
    return c.pages + p.page +
           ((long long)h * (c.page_tokens / kv::kStrip) + p.token / kv::kStrip) * kv::strip_bytes(BITS, D);
}

// Quantises 8 values of a group spread over 8 lanes; codes packed little end first
template <int BITS>
__device__ __forceinline__ void quantise8(const uint4& raw, uint32_t (&word)[2], __half2& sb) {
    constexpr float kTop = (float)((1 << BITS) - 1);
    const __half2* h2 = reinterpret_cast<const __half2*>(&raw);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(h2[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
    float mn = x[0], mx = x[0];
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mn = fminf(mn, x[i]);
        mx = fmaxf(mx, x[i]);
        fine = fine && isfinite(x[i]);
    }
    unsigned bad = fine ? 0u : 1u;
#pragma unroll
    for (int k = 1; k < 8; k <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, k));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        bad |= __shfl_xor_sync(0xffffffffu, bad, k);
    }
    const __half s16 = __float2half_rn(__fdiv_rn(mx - mn, kTop));
    const float s = __half2float(s16);
    uint32_t q[8];
    if (bad || s == 0.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = 0;
    } else {
        const float inv = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = x[i] - mn;
            float r = rintf(d * inv);
            // next to a border: compare x - mn with the border itself.  d + lo is the
            // exact x - mn; the border (r +- 1/2) s and d - border are exact
            const float off = fmaf(-r, s, d);
            if (fabsf(fabsf(off) - 0.5f * s) < 1e-3f * s) {
                const float bb = d - x[i];
                const float lo = (x[i] - (d - bb)) + (-mn - bb);
                const float side = off > 0.f ? 0.5f : -0.5f;
                const float border = (r + side) * s;
                const float e = (d - border) + lo;
                const float up = r + side + 0.5f, down = r + side - 0.5f;
                const bool even_up = ((int)up & 1) == 0;
                r = e > 0.f ? up : e < 0.f ? down : even_up ? up : down;
            }
            q[i] = (uint32_t)fminf(fmaxf(r, 0.f), kTop);
        }
    }
    if (BITS == 4) {
        word[0] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) word[0] |= q[i] << (4 * i);
        word[1] = 0;
    } else {
        word[0] = q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24);
        word[1] = q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24);
    }
    const __half nan16 = __ushort_as_half((unsigned short)0x7fff);
    sb = bad ? __halves2half2(nan16, nan16) : __halves2half2(s16, __float2half_rn(mn));
}

template <int BITS, int D>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(kv::View c, Rows rows, int rows_per_cta,
                                                               const __half* __restrict__ k, long long ldk,
                                                               const __half* __restrict__ v, long long ldv) {
    constexpr int kR = kv::row_bytes(BITS, D);
    __shared__ int cu_s[EDGE0_MAX_BATCHED + 1];
    __shared__ RowPlace place[kMaxRowsPerCta];
    const int r0 = blockIdx.x * rows_per_cta;
    place_rows(c, rows, r0, rows_per_cta, cu_s, place);
    const int per_row = 2 * c.H * (D / 8);          // threads' worth of work per row, a multiple of 8
    const int n = rows_per_cta * per_row;
    for (int i0 = 0; i0 < n; i0 += kKvThreads) {
        const int i = i0 + threadIdx.x;
        const int row = i < n ? i / per_row : 0, j = i < n ? i - row * per_row : 0;
        const RowPlace p = place[row];
        const bool live = i < n && p.page >= 0;     // the same for the 8 lanes of a group
        const int which = j / (c.H * (D / 8)), hj = j - which * c.H * (D / 8);
        const int h = hj / (D / 8), i8 = hj % (D / 8);
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live)
            raw = *reinterpret_cast<const uint4*>((which ? v + (r0 + row) * ldv : k + (r0 + row) * ldk) +
                                                  (long long)h * D + 8 * i8);
        uint32_t word[2];
        __half2 sb;
        quantise8<BITS>(raw, word, sb);
        if (!live) continue;
        char* half = strip_of<BITS, D>(c, p, h) + which * kv::half_bytes(BITS, D);
        const int rr = p.token % kv::kStrip;
        const int off = i8 * BITS;                  // byte of the row
        char* dst = half + rr * kR + (((off >> 4) ^ kv::turn(kR, rr)) << 4) + (off & 15);
        if (BITS == 4) *reinterpret_cast<uint32_t*>(dst) = word[0];
        else *reinterpret_cast<uint2*>(dst) = make_uint2(word[0], word[1]);
        if (i8 % 8 == 0)
            *reinterpret_cast<__half2*>(half + kv::kStrip * kR + rr * kv::sb_bytes(D) + (i8 / 8) * 4) = sb;
    }
}

template <int BITS, int D>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(kv::View c, Rows rows, int rows_per_cta,
                                                             __half* __restrict__ k, __half* __restrict__ v) {
    constexpr int kR = kv::row_bytes(BITS, D);
    __shared__ int cu_s[EDGE0_MAX_BATCHED + 1];
    __shared__ RowPlace place[kMaxRowsPerCta];
    const int r0 = blockIdx.x * rows_per_cta;
    place_rows(c, rows, r0, rows_per_cta, cu_s, place);
    const int per_row = 2 * c.H * (D / 8);
    const int n = rows_per_cta * per_row;
    for (int i = threadIdx.x; i < n; i += kKvThreads) {
        const int row = i / per_row, j = i - row * per_row;
        const RowPlace p = place[row];
        if (p.page < 0) continue;
        const int which = j / (c.H * (D / 8)), hj = j - which * c.H * (D / 8);
        const int h = hj / (D / 8), i8 = hj % (D / 8);
        const char* half = strip_of<BITS, D>(c, p, h) + which * kv::half_bytes(BITS, D);
        const int rr = p.token % kv::kStrip;
        const int off = i8 * BITS;
        const char* src = half + rr * kR + (((off >> 4) ^ kv::turn(kR, rr)) << 4) + (off & 15);
        uint32_t w0, w1 = 0;
        if (BITS == 4) {
            w0 = *reinterpret_cast<const uint32_t*>(src);
        } else {
            const uint2 w = *reinterpret_cast<const uint2*>(src);
            w0 = w.x;
            w1 = w.y;
        }
        const float2 sb = __half22float2(
            *reinterpret_cast<const __half2*>(half + kv::kStrip * kR + rr * kv::sb_bytes(D) + (i8 / 8) * 4));
        __half2 o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t a, b;
            if (BITS == 4) {
                a = (w0 >> (8 * q)) & 15u;
                b = (w0 >> (8 * q + 4)) & 15u;
            } else {
                const uint32_t w = q < 2 ? w0 : w1;
                a = (w >> (16 * (q & 1))) & 255u;
                b = (w >> (16 * (q & 1) + 8)) & 255u;
            }
            o[q] = __floats2half2_rn(fmaf((float)a, sb.x, sb.y), fmaf((float)b, sb.x, sb.y));
        }
        __half* out = (which ? v : k) + ((long long)(r0 + row) * c.H + h) * D + 8 * i8;
        *reinterpret_cast<uint4*>(out) = *reinterpret_cast<uint4*>(o);
    }
}

// rows per CTA: about four CTAs per SM of a full card, at most kMaxRowsPerCta
int rows_per_cta(int T) {
    const int r = ceil_div(T, 152 * 4);
    return r < 1 ? 1 : r > kMaxRowsPerCta ? kMaxRowsPerCta : r;
}

int check_rows(const Rows& r) {
    if (!r.table || !r.start || r.B <= 0 || r.B > EDGE0_MAX_BATCHED || r.W <= 0 || r.T < 0) return EDGE0_EINVAL;
    if (((uintptr_t)r.table | (uintptr_t)r.start | (uintptr_t)r.cu | (uintptr_t)r.status) & 3) return EDGE0_EINVAL;
    if (!r.cu && r.T != r.B) return EDGE0_EINVAL;
    return EDGE0_OK;
}

}  // namespace
}  // namespace edge0

using namespace edge0;

#define EDGE0_KV_DISPATCH(bits, D, CALL)                                  \
    do {                                                                  \
        if ((bits) == 4) {                                                \
            if ((D) == 64) { constexpr int BT = 4, DD = 64; CALL; }       \
            else if ((D) == 128) { constexpr int BT = 4, DD = 128; CALL; } \
            else { constexpr int BT = 4, DD = 256; CALL; }                \
        } else {                                                          \
            if ((D) == 64) { constexpr int BT = 8, DD = 64; CALL; }       \
            else if ((D) == 128) { constexpr int BT = 8, DD = 128; CALL; } \
            else { constexpr int BT = 8, DD = 256; CALL; }                \
        }                                                                 \
    } while (0)

extern "C" size_t edge0_kv_page_bytes(int bits, int n_kv_heads, int head_dim, int page_tokens) {
    if (bits != 4 && bits != 8) return 0;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
    if (n_kv_heads <= 0 || n_kv_heads > EDGE0_MAX_KV_HEADS) return 0;
    if (page_tokens <= 0 || page_tokens % kv::kStrip || page_tokens > EDGE0_MAX_PAGE_TOKENS) return 0;
    return (size_t)n_kv_heads * (page_tokens / kv::kStrip) * kv::strip_bytes(bits, head_dim);
}

extern "C" int edge0_kv_append(const edge0_kv_cache* cache, const uint16_t* k, long long ldk, const uint16_t* v,
                               long long ldv, int T, const int32_t* table, int B, int W, const int32_t* start,
                               const int32_t* cu_rows, int* status, cudaStream_t stream) {
    kv::View c;
    int rc = kv::view_of(cache, &c);
    if (rc) return rc;
    const Rows rows{table, B, W, start, cu_rows, T, status};
    rc = check_rows(rows);
    if (rc) return rc;
    const long long width = (long long)cache->n_kv_heads * cache->head_dim;
    if (!k || !v || (((uintptr_t)k | (uintptr_t)v) & 15) || ldk % 8 || ldv % 8 || ldk < width || ldv < width)
        return EDGE0_EINVAL;
    if (T == 0) return EDGE0_OK;
    const int per = rows_per_cta(T);
    EDGE0_KV_DISPATCH(cache->bits, cache->head_dim,
                      (kv_append_kernel<BT, DD><<<ceil_div(T, per), kKvThreads, 0, stream>>>(
                          c, rows, per, (const __half*)k, ldk, (const __half*)v, ldv)));
    return cudaGetLastError() == cudaSuccess ? EDGE0_OK : EDGE0_ECUDA;
}

extern "C" int edge0_kv_read(const edge0_kv_cache* cache, const int32_t* table, int B, int W, const int32_t* start,
                             const int32_t* cu_rows, int T, uint16_t* k, uint16_t* v, int* status,
                             cudaStream_t stream) {
    kv::View c;
    int rc = kv::view_of(cache, &c);
    if (rc) return rc;
    const Rows rows{table, B, W, start, cu_rows, T, status};
    rc = check_rows(rows);
    if (rc) return rc;
    if (!k || !v || (((uintptr_t)k | (uintptr_t)v) & 15)) return EDGE0_EINVAL;
    if (T == 0) return EDGE0_OK;
    const int per = rows_per_cta(T);
    EDGE0_KV_DISPATCH(cache->bits, cache->head_dim,
                      (kv_read_kernel<BT, DD><<<ceil_div(T, per), kKvThreads, 0, stream>>>(c, rows, per, (__half*)k,
                                                                                         (__half*)v)));
    return cudaGetLastError() == cudaSuccess ? EDGE0_OK : EDGE0_ECUDA;
}
