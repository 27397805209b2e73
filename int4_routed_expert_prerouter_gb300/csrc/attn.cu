// Decode attention over the quantised KV cache: one query token per sequence,
//     o = sum_j softmax_j(scale q . k_j) v_j
// over the shared prefix's tokens and the sequence's own, in fp32 with a running
// maximum and sum.  One CTA per (sequence, query head): its warps take the tokens in
// turn, a lane holds D / 32 dims; the warps' results are joined in shared memory.
#include "kvcache.cuh"

namespace edge0 {
namespace {

constexpr int kAttnWarps = 4;

struct AttnP {
    kv::View c;
    const __half* q;
    long long ldq;
    int B, Hq;
    const int* table;
    int W;
    const int* lens;
    const int* prefix;
    int n_prefix;
    float scale;
    __half* out;
    long long ldo;
    int* status;
};

template <int BITS, int D>
__global__ void __launch_bounds__(32 * kAttnWarps) attn_kernel(AttnP p) {
    constexpr int kN = D / 32;
    constexpr int kR = kv::row_bytes(BITS, D);
    __shared__ float ms[kAttnWarps], ls[kAttnWarps], os[kAttnWarps][D];
    const int b = blockIdx.x, hq = blockIdx.y, h = hq / (p.Hq / p.c.H);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    long long own = p.lens[b];
    if (own < 0) return;                                   // a padding row
    if (own > (long long)p.W * p.c.page_tokens) {
        own = (long long)p.W * p.c.page_tokens;
        if (threadIdx.x == 0 && p.status) atomicExch(p.status, EDGE0_EINVAL);
    }
    float q[kN], o[kN], m = -INFINITY, l = 0.f;
    for (int i = 0; i < kN; ++i) {
        q[i] = __half2float(p.q[b * p.ldq + (long long)hq * D + lane * kN + i]) * p.scale;
        o[i] = 0.f;
    }
    auto value = [&](const char* half, int rr, float (&x)[kN]) {
        const float2 sb = __half22float2(*reinterpret_cast<const __half2*>(
            half + kv::kStrip * kR + rr * kv::sb_bytes(D) + (lane * kN / kGroup) * 4));
        for (int i = 0; i < kN; ++i) {
            const int d = lane * kN + i, off = d * BITS / 8;
            const unsigned char w =
                *reinterpret_cast<const unsigned char*>(half + rr * kR + (((off >> 4) ^ kv::turn(kR, rr)) << 4) + (off & 15));
            const int code = BITS == 8 ? w : (d & 1) ? w >> 4 : w & 15;
            x[i] = fmaf((float)code, sb.x, sb.y);
        }
    };
    const long long n = p.n_prefix + own;
    for (long long j = wid; j < n; j += kAttnWarps) {
        const bool pre = j < p.n_prefix;
        const long long pos = pre ? j : j - p.n_prefix;
        const long long pg = pos / p.c.page_tokens;
        const int tok = (int)(pos - pg * p.c.page_tokens);
        int id = pre ? p.prefix[pg] : p.table[(long long)b * p.W + pg];
        if (id < 0 || id >= p.c.n_pages) {
            id = 0;
            if (lane == 0 && p.status) atomicExch(p.status, EDGE0_EINVAL);
        }
        const char* strip = p.c.pages + id * p.c.page_bytes +
                            ((long long)h * (p.c.page_tokens / kv::kStrip) + tok / kv::kStrip) * kv::strip_bytes(BITS, D);
        float x[kN], s = 0.f;
        value(strip, tok % kv::kStrip, x);
        for (int i = 0; i < kN; ++i) s += q[i] * x[i];
        s = warp_sum(s);
        const float mn = fmaxf(m, s), f = __expf(m - mn), e = __expf(s - mn);
        value(strip + kv::half_bytes(BITS, D), tok % kv::kStrip, x);
        for (int i = 0; i < kN; ++i) o[i] = o[i] * f + e * x[i];
        l = l * f + e;
        m = mn;
    }
    if (lane == 0) {
        ms[wid] = m;
        ls[wid] = l;
    }
    for (int i = 0; i < kN; ++i) os[wid][lane * kN + i] = o[i];
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, ms[w]);
    for (int w = 0; w < kAttnWarps; ++w)
        if (ls[w] != 0.f) sum += ls[w] * __expf(ms[w] - top);
    for (int d = threadIdx.x; d < D; d += 32 * kAttnWarps) {
        float v = 0.f;
        for (int w = 0; w < kAttnWarps; ++w)
            if (ls[w] != 0.f) v += os[w][d] * __expf(ms[w] - top);
        p.out[b * p.ldo + (long long)hq * D + d] = __float2half_rn(n > 0 ? v / sum : 0.f);
    }
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" size_t edge0_attn_workspace_bytes(const edge0_kv_cache* cache, int B, int n_q_heads) {
    kv::View c;
    if (kv::view_of(cache, &c) || B <= 0 || B > EDGE0_MAX_BATCHED) return 0;
    if (n_q_heads <= 0 || n_q_heads % c.H || n_q_heads / c.H > EDGE0_MAX_Q_PER_KV) return 0;
    return 256;
}

extern "C" int edge0_attn_decode(const edge0_kv_cache* cache, const uint16_t* q, long long ldq, int B, int n_q_heads,
                                 const int32_t* table, int W, const int32_t* lens, const int32_t* prefix,
                                 int n_prefix, float scale, uint16_t* out, long long ldo, int* status,
                                 void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    AttnP p;
    int rc = kv::view_of(cache, &p.c);
    if (rc) return rc;
    if (!q || !table || !lens || !out || !workspace || B <= 0 || B > EDGE0_MAX_BATCHED || W <= 0) return EDGE0_EINVAL;
    if (n_q_heads <= 0 || n_q_heads % p.c.H) return EDGE0_EINVAL;
    if (n_q_heads / p.c.H > EDGE0_MAX_Q_PER_KV) return EDGE0_EUNSUPPORTED;
    if (n_prefix < 0 || (n_prefix > 0 && !prefix)) return EDGE0_EINVAL;
    if (!(scale > 0.f) || !(scale <= 1e6f)) return EDGE0_EINVAL;
    const long long width = (long long)n_q_heads * cache->head_dim;
    if (ldq < width || ldq % 8 || ldo < width || ldo % 8) return EDGE0_EINVAL;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15) return EDGE0_EINVAL;
    if (((uintptr_t)table | (uintptr_t)lens | (uintptr_t)prefix | (uintptr_t)status) & 3) return EDGE0_EINVAL;
    if (workspace_bytes < edge0_attn_workspace_bytes(cache, B, n_q_heads)) return EDGE0_EINVAL;
    p.q = (const __half*)q;
    p.ldq = ldq;
    p.B = B;
    p.Hq = n_q_heads;
    p.table = table;
    p.W = W;
    p.lens = lens;
    p.prefix = prefix;
    p.n_prefix = n_prefix;
    p.scale = scale;
    p.out = (__half*)out;
    p.ldo = ldo;
    p.status = status;
    const dim3 grid(B, n_q_heads);
    const int D = cache->head_dim;
    if (cache->bits == 4) {
        if (D == 64) attn_kernel<4, 64><<<grid, 32 * kAttnWarps, 0, stream>>>(p);
        else if (D == 128) attn_kernel<4, 128><<<grid, 32 * kAttnWarps, 0, stream>>>(p);
        else attn_kernel<4, 256><<<grid, 32 * kAttnWarps, 0, stream>>>(p);
    } else {
        if (D == 64) attn_kernel<8, 64><<<grid, 32 * kAttnWarps, 0, stream>>>(p);
        else if (D == 128) attn_kernel<8, 128><<<grid, 32 * kAttnWarps, 0, stream>>>(p);
        else attn_kernel<8, 256><<<grid, 32 * kAttnWarps, 0, stream>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? EDGE0_OK : EDGE0_ECUDA;
}
