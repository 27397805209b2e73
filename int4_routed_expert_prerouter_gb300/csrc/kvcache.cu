// The quantised KV cache: rows of K and V written as 4- or 8-bit affine codes, and
// read back.
//
// Per (token, kv head, K or V, 64 dims): mn, mx over the 64 fp16 values;
//     s = fp16((mx - mn) / (2^bits - 1)), b = mn,
//     q = clamp(rne((x - mn) / s), 0, 2^bits - 1)    (0 where s = 0);
// s one fp16 step less where (2^bits - 1) s + b would round to infinity,
// and the stored group stands for s q + b.  q is the exact quotient's rounding: the
// kernel rounds the fp32 products of x - mn with a little less and a little more than
// 1 / s, and where these differ it decides by the sign of (x - mn) - (q +- 1/2) s, which
// fp32 holds exactly there.
//
// Both kernels move rows of fp16 and bytes of codes: the floor is these bytes.  A thread keeps
// its place in the row and goes through its CTA's rows.  Written: 16 dims per thread, 8
// from each half of a group (four threads share its minimum, maximum and reciprocal); the
// next row's values are loaded while one is worked on, the first ones before the rows'
// places are known.  Read: 8 dims per thread, so that a warp's 16-byte stores lie side by
// side, four rows at a time.
// Measured: 8,192 rows of 8 x 128 dims written as 8 bits and read back 21.6 us, 80 MB at 3.7
// TB/s (a copy: 6.8), one third of it start-up of two launches, places and first loads;
// 63,001 such rows of 4 bits read 57 us, 331 MB at 5.8 TB/s; one row for each of 64
// sequences written and read 5.7 us, two launches' latency.
#include "kvcache.cuh"
#include "launch.cuh"

namespace edge0 {
namespace {

constexpr int kKvThreads = 256;
constexpr int kMaxRowsPerCta = 32;
constexpr int kReadRows = 4;         // rows that a reading thread has under way

// Where the rows of a CTA go.
struct RowPlace {
    long long strip;  // byte offset of the row's strip of head 0 in the pool, or -1: nothing to do
    int row;          // row of the strip
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
__device__ void place_rows(const kv::View& c, int strip_bytes, const Rows& rows, int r0, int n, int* cu_s,
                           RowPlace* out) {
    if (rows.cu) {
        for (int i = threadIdx.x; i <= rows.B; i += kKvThreads) cu_s[i] = rows.cu[i];
        __syncthreads();
    }
    if (threadIdx.x < n) {
        const int r = r0 + threadIdx.x;
        RowPlace p;
        p.strip = -1;
        p.row = 0;
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
                    const int token = (int)(pos - pg * c.page_tokens);
                    p.strip = (long long)id * c.page_bytes + (long long)(token / kv::kStrip) * strip_bytes;
                    p.row = token % kv::kStrip;
                } else if (rows.status) {
                    atomicExch(rows.status, EDGE0_EINVAL);
                }
            }
        }
        out[threadIdx.x] = p;
    }
    __syncthreads();
}

// q of one value where the fp32 product may lie next to a border, or above the top code
// where s was rounded down
__device__ __forceinline__ float settle(float x, float mn, float s, float r, float top) {
    const float d = x - mn, off = fmaf(-r, s, d);
    if (fabsf(fabsf(off) - 0.5f * s) < 4e-4f * s) {
        // d + lo is the exact x - mn; the border (r +- 1/2) s and d - border are exact
        const float bb = d - x;
        const float lo = (x - (d - bb)) + (-mn - bb);
        const float side = off > 0.f ? 0.5f : -0.5f;
        const float e = (d - (r + side) * s) + lo;
        const float up = r + side + 0.5f, down = r + side - 0.5f;
        r = e > 0.f ? up : e < 0.f ? down : ((int)up & 1) == 0 ? up : down;
    }
    return fminf(fmaxf(r, 0.f), top);
}

// Quantises 16 values of a group spread over 4 lanes; codes packed little end first
template <int BITS>
__device__ __forceinline__ void quantise16(const uint4 (&raw)[2], uint32_t (&word)[BITS / 2], __half2& sb) {
    constexpr float kTop = (float)((1 << BITS) - 1);
    constexpr float kRound = 12582912.f;                 // 1.5 2^23: an fp32 sum with it is a whole number
    const __half2* h2 = reinterpret_cast<const __half2*>(raw);
    // (minimum, minus maximum) in one register; a NaN stays
    __half2 lo2 = h2[0], hi2 = h2[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo2 = __hmin2_nan(lo2, h2[i]);
        hi2 = __hmax2_nan(hi2, h2[i]);
    }
    __half2 w = __hmin2_nan(__halves2half2(__low2half(lo2), __hneg(__low2half(hi2))),
                            __halves2half2(__high2half(lo2), __hneg(__high2half(hi2))));
    w = __hmin2_nan(w, __shfl_xor_sync(0xffffffffu, w, 1));
    w = __hmin2_nan(w, __shfl_xor_sync(0xffffffffu, w, 2));
    const float mn = __low2float(w), mx = -__high2float(w);
    // (mx - mn) / kTop rounded to nearest: with the rounded reciprocal one residual step is exact
    const float range = mx - mn, s0 = range * (1.f / kTop);
    __half s16 = __float2half_rn(fmaf(fmaf(-s0, kTop, range), 1.f / kTop, s0));
    // a scale rounded up must not carry the top code over fp16's range (65520 rounds to infinity)
    if (fmaf(__half2float(s16), kTop, mn) >= 65520.f) s16 = __ushort_as_half(__half_as_ushort(s16) - 1);
    const float s = __half2float(s16);
    const bool bad = !isfinite(mn) || !isfinite(mx);
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) word[i] = 0;
    if (!bad && s != 0.f) {
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        // Quotients with a reciprocal a little below and a little above: the exact one lies between
        // (its error is at most 2^-23 of the reciprocal and 2^-24 of d), so where both round
        // to the same number it does too.
        const f2 lo = pk(inv * (1.f - 0x1.8p-22f), inv * (1.f - 0x1.8p-22f));
        const f2 hi = pk(inv * (1.f + 0x1.8p-22f), inv * (1.f + 0x1.8p-22f));
        const f2 from = pk(-mn, -mn), round = pk(kRound, kRound);
        float t[16];                                     // kRound + q
        f2 differ = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = __half22float2(h2[i]);
            const f2 d = add2(pk(f.x, f.y), from), below = fma2(d, lo, round);
            differ |= below ^ fma2(d, hi, round);
            unpk(below, t[2 * i], t[2 * i + 1]);
        }
        if (differ != 0 || range * inv > kTop + 0.5f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = __half22float2(h2[i]);
                t[2 * i] = settle(f.x, mn, s, t[2 * i] - kRound, kTop) + kRound;
                t[2 * i + 1] = settle(f.y, mn, s, t[2 * i + 1] - kRound, kTop) + kRound;
            }
        }
        // the low bits of t are q; what its high bits add up to in a word comes off at the end
        constexpr int kPer = 32 / BITS;                  // codes per word
        constexpr uint32_t kHigh = 0x4B400000u * (BITS == 4 ? 0x11111111u : 0x01010101u);
#pragma unroll
        for (int i = 15; i >= 0; --i) word[i / kPer] = word[i / kPer] * (1 << BITS) + __float_as_uint(t[i]);
#pragma unroll
        for (int i = 0; i < BITS / 2; ++i) word[i] -= kHigh;
    }
    const __half nan16 = __ushort_as_half((unsigned short)0x7fff);
    sb = bad ? __halves2half2(nan16, nan16) : __halves2half2(s16, __float2half_rn(mn));
}

// 8 values fp16(s q + b), each rounded once: a code below 1024's exponent adds itself (a nibble
// 4 bits up 16 times itself), so the codes are exact fp16 and s q + b one fused step.
template <int BITS>
__device__ __forceinline__ uint4 values8(const uint32_t (&w)[BITS / 4], uint32_t sb) {
    const uint32_t s = __byte_perm(sb, sb, 0x1010), b = __byte_perm(sb, sb, 0x3232);
    uint4 r;
    if (BITS == 4) {
        const uint32_t h = w[0] >> 8;
        // dims 0, 4 | 1, 5 | 2, 6 | 3, 7
        const uint32_t v0 = hfma2(hadd2((w[0] & 0x000F000Fu) | 0x64006400u, 0xE400E400u), s, b);
        const uint32_t v1 = hfma2(hfma2((w[0] & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u), s, b);
        const uint32_t v2 = hfma2(hadd2((h & 0x000F000Fu) | 0x64006400u, 0xE400E400u), s, b);
        const uint32_t v3 = hfma2(hfma2((h & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u), s, b);
        r = make_uint4(__byte_perm(v0, v1, 0x5410), __byte_perm(v2, v3, 0x5410), __byte_perm(v0, v1, 0x7632),
                       __byte_perm(v2, v3, 0x7632));
    } else {
        const uint32_t w0 = w[0], w1 = w[BITS / 4 - 1];
        r.x = hfma2(hadd2(__byte_perm(w0, 0x64646464u, 0x4140), 0xE400E400u), s, b);
        r.y = hfma2(hadd2(__byte_perm(w0, 0x64646464u, 0x4342), 0xE400E400u), s, b);
        r.z = hfma2(hadd2(__byte_perm(w1, 0x64646464u, 0x4140), 0xE400E400u), s, b);
        r.w = hfma2(hadd2(__byte_perm(w1, 0x64646464u, 0x4342), 0xE400E400u), s, b);
    }
    return r;
}

// A thread's place in K's and V's heads, the same in every row it takes; threads of short
// rows share a CTA's rows.
struct Place {
    int j, sub, step;       // place in the row, first row, rows apart
    __device__ Place(int per_row) {
        const int par = per_row >= kKvThreads ? 1 : kKvThreads / per_row;
        sub = threadIdx.x / per_row;
        j = threadIdx.x - sub * per_row;
        step = par;
        if (per_row >= kKvThreads) {
            sub = 0;
            j = threadIdx.x;
        } else if (sub >= par) {
            sub = 1 << 20;   // a thread left over
        }
    }
};

template <int BITS, int D>
__global__ void __launch_bounds__(kKvThreads, 4) kv_append_kernel(kv::View c, Rows rows, int rows_per_cta,
                                                                  const __half* k, long long ldk,
                                                                  const __half* v, long long ldv) {
    constexpr int kR = kv::row_bytes(BITS, D);
    __shared__ int cu_s[EDGE0_MAX_BATCHED + 1];
    __shared__ RowPlace place[kMaxRowsPerCta];
    const int r0 = blockIdx.x * rows_per_cta;
    const int n = min(rows_per_cta, rows.T - r0);
    const int half_row = c.H * (D / 16), per_row = 2 * half_row;   // threads' worth of work per row
    const Place me(per_row);
    const int last = (per_row + kKvThreads - 1) / kKvThreads * kKvThreads;     // whole warps: the quantiser's shuffles
    wait_predecessor();
    launch_dependents();
    bool placed = false;
    for (int j = me.j; j < last; j += kKvThreads) {
        const int which = j >= half_row, hj = j - which * half_row, h = hj / (D / 16), at = hj % (D / 16);
        const int dim = (at >> 2) * kGroup + (at & 3) * 8;                     // and dim + 32
        const long long ld = which ? ldv : ldk;
        const __half* src = (which ? v : k) + (long long)r0 * ld + h * D + dim;
        char* head = c.pages + (long long)h * (c.page_tokens / kv::kStrip) * kv::strip_bytes(BITS, D) +
                     which * kv::half_bytes(BITS, D);
        const int off0 = dim * BITS / 8, off1 = (dim + 32) * BITS / 8;         // bytes of the row of codes
        auto fetch = [&](int row, uint4 (&raw)[2]) {
            raw[0] = raw[1] = make_uint4(0, 0, 0, 0);
            if (row < n && j < per_row) {
                const uint4* x = reinterpret_cast<const uint4*>(src + row * ld);
                raw[0] = x[0];
                raw[1] = x[4];
            }
        };
        uint4 next[2];
        fetch(me.sub, next);
        if (!placed) place_rows(c, kv::strip_bytes(BITS, D), rows, r0, n, cu_s, place);
        placed = true;
        for (int base = 0; base < n; base += me.step) {
            const int row = base + me.sub;
            const uint4 raw[2] = {next[0], next[1]};
            if (base + me.step < n) fetch(row + me.step, next);
            uint32_t word[BITS / 2];
            __half2 sb;
            quantise16<BITS>(raw, word, sb);
            if (row >= n || j >= per_row) continue;
            const RowPlace p = place[row];
            if (p.strip < 0) continue;
            char* half = head + p.strip;
            char* codes = half + p.row * kR;
            const int turn = kv::turn(kR, p.row) << 4;
            if (BITS == 4) {
                *reinterpret_cast<uint32_t*>(codes + (off0 ^ turn)) = word[0];
                *reinterpret_cast<uint32_t*>(codes + (off1 ^ turn)) = word[1];
            } else {
                *reinterpret_cast<uint2*>(codes + (off0 ^ turn)) = make_uint2(word[0], word[1]);
                *reinterpret_cast<uint2*>(codes + (off1 ^ turn)) = make_uint2(word[BITS / 2 - 2], word[BITS / 2 - 1]);
            }
            if (at % 4 == 0)
                *reinterpret_cast<__half2*>(half + kv::kStrip * kR + p.row * kv::sb_bytes(D) + (at / 4) * 4) = sb;
        }
    }
}

template <int BITS, int D>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(kv::View c, Rows rows, int rows_per_cta,
                                                             __half* k, __half* v) {
    constexpr int kR = kv::row_bytes(BITS, D);
    __shared__ int cu_s[EDGE0_MAX_BATCHED + 1];
    __shared__ RowPlace place[kMaxRowsPerCta];
    const int r0 = blockIdx.x * rows_per_cta;
    wait_predecessor();
    launch_dependents();
    place_rows(c, kv::strip_bytes(BITS, D), rows, r0, rows_per_cta, cu_s, place);
    const int half_row = c.H * (D / 8), per_row = 2 * half_row;
    const Place me(per_row);
    for (int j = me.j; j < per_row; j += kKvThreads) {
        const int which = j >= half_row, hj = j - which * half_row, h = hj / (D / 8), at = hj % (D / 8);
        __half* dst = (which ? v : k) + hj * 8;
        const int off = at * BITS;
        const char* head = c.pages + (long long)h * (c.page_tokens / kv::kStrip) * kv::strip_bytes(BITS, D) +
                           which * kv::half_bytes(BITS, D);
        for (int base = 0; base < rows_per_cta; base += kReadRows * me.step) {
            uint32_t w[kReadRows][BITS / 4], sbw[kReadRows];
            bool live[kReadRows];
#pragma unroll
            for (int u = 0; u < kReadRows; ++u) {
                const int row = base + me.sub + u * me.step;
                RowPlace p;
                p.strip = -1;
                if (row < rows_per_cta) p = place[row];
                live[u] = p.strip >= 0;
                if (live[u]) {
                    const int rr = p.row;
                    const char* half = head + p.strip;
                    const char* src = half + rr * kR + (off ^ (kv::turn(kR, rr) << 4));
                    if (BITS == 4) {
                        w[u][0] = *reinterpret_cast<const uint32_t*>(src);
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2*>(src);
                        w[u][0] = x.x;
                        w[u][BITS / 4 - 1] = x.y;
                    }
                    sbw[u] = *reinterpret_cast<const uint32_t*>(half + kv::kStrip * kR + rr * kv::sb_bytes(D) + (at / 8) * 4);
                }
            }
#pragma unroll
            for (int u = 0; u < kReadRows; ++u) {
                if (!live[u]) continue;
                const uint4 o = values8<BITS>(w[u], sbw[u]);
                const int row = base + me.sub + u * me.step;
                *reinterpret_cast<uint4*>(dst + (long long)(r0 + row) * (c.H * D)) = o;
            }
        }
    }
}

// rows per CTA: so many that `ctas` CTAs per SM, as many as are resident at once, cover T, at most
// `most`.  Measured, us, 8,192 rows of 8 x 128 dims as 8 bits: written with 4 resident CTAs (64
// registers) 12, with 3 and rows for 4 per SM 17; then read with rows for 5 or 8 per SM 22.9
// and 23.3 both together; 63,001 rows read at most 16, 32 or 64 at a time 57, 62 and 69.
int rows_per_cta(int T, int ctas, int most) {
    const int r = ceil_div(T, 152 * ctas);
    return r < 1 ? 1 : r > most ? most : r;
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

#define EDGE0_KV_DISPATCH(bits, D, ...)                                  \
    do {                                                                  \
        if ((bits) == 4) {                                                \
            if ((D) == 64) { constexpr int BT = 4, DD = 64; __VA_ARGS__; }       \
            else if ((D) == 128) { constexpr int BT = 4, DD = 128; __VA_ARGS__; } \
            else { constexpr int BT = 4, DD = 256; __VA_ARGS__; }                \
        } else {                                                          \
            if ((D) == 64) { constexpr int BT = 8, DD = 64; __VA_ARGS__; }       \
            else if ((D) == 128) { constexpr int BT = 8, DD = 128; __VA_ARGS__; } \
            else { constexpr int BT = 8, DD = 256; __VA_ARGS__; }                \
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
    if (T == 0) return EDGE0_OK;
    const long long width = (long long)cache->n_kv_heads * cache->head_dim;
    if (!k || !v || (((uintptr_t)k | (uintptr_t)v) & 15) || ldk % 8 || ldv % 8 || ldk < width || ldv < width)
        return EDGE0_EINVAL;
    const int per = rows_per_cta(T, 4, kMaxRowsPerCta);
    EDGE0_KV_DISPATCH(cache->bits, cache->head_dim,
                      rc = launch_early(kv_append_kernel<BT, DD>, dim3(ceil_div(T, per)), kKvThreads, 0, stream, c, rows, per,
                                        (const __half*)k, ldk, (const __half*)v, ldv));
    return rc;
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
    if (T == 0) return EDGE0_OK;
    if (!k || !v || (((uintptr_t)k | (uintptr_t)v) & 15)) return EDGE0_EINVAL;
    const int per = rows_per_cta(T, 5, 16);
    EDGE0_KV_DISPATCH(cache->bits, cache->head_dim,
                      rc = launch_early(kv_read_kernel<BT, DD>, dim3(ceil_div(T, per)), kKvThreads, 0, stream, c, rows, per,
                                        (__half*)k, (__half*)v));
    return rc;
}
