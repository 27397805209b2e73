// Rotary positions: pairs of a head's dims turned by the angle position x frequency.
//
// Angles.  Far positions lose what matters in 32 bits (position 131,071 times a frequency
// rounded to fp32 is off by up to 4e-3 rad), and a table of cosines has to be read.  A
// frequency is kept as the 64-bit fraction of a turn per position instead; position x
// fraction modulo 2^64 is then the angle's own fraction of a turn in one integer product,
// whatever the position, off by at most position x 2^-65 turns plus the rounding of the frequency
// to fp64 (position x 2^-53 of it).  Signed it is an angle in [-1/2, 1/2) turns, and sincospi
// of twice that takes no reduction.
//
// A CTA forms its tokens' cosines and sines once, in shared memory; every head then takes them
// from there (a pair costs 4 multiplications beside 8 bytes of traffic).  A thread keeps its place
// in the row, 2 x 8 dims (half layout) or 8 dims (interleaved), and goes through its CTA's tokens,
// kRopeRows of them under way.
//
// 8,192 tokens of prompts, 32 + 8 heads of 128 of which 64 dims turn: 31.5 us for 158 MB, 0.74 of a copy.  What bounds it is
// latency: one wave of CTAs, all of which form sines first and load afterwards (DRAM 44 %, issue slots 47 %, warps 40 %).
// (First values under way while the sines are formed: 36.7; places and tokens as one row of units, so that no thread
// is left over: 32.4; at most 8 tokens a CTA: 33.4.)  A step of 64 tokens: 4.6 us, launch and two dependent reads.
#include "kvcache.cuh"
#include "launch.cuh"

#include <math.h>

namespace edge0 {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxRows = 16;         // tokens per CTA
constexpr int kRopeRows = 4;             // tokens that a thread has under way
constexpr int kRopeMaxDim = 512;

struct RopeSide {
    const __half* x;
    __half* y;
    long long ldx, ldy;
    int heads;
};

struct RopeP {
    const unsigned long long* turns;     // [rot / 2]
    RopeSide side[2];                    // queries, keys
    int D, rot;
    float magnitude, sign;
    int T, B;
    const int* start;
    const int* cu;                       // [B + 1] or null: row b belongs to sequence b
    int rows_per_cta;
};

// V: values of each half of a pair that a thread takes, 8 (a 16-byte access each) or 1.
template <bool HALF, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeP p) {
    extern __shared__ __align__(16) float2 table[];       // [rows_per_cta][rot / 2] (cos, sin), read in pairs
    __shared__ int cu_s[EDGE0_MAX_BATCHED + 1];
    __shared__ long long pos_s[kRopeMaxRows];            // -1: nothing to do
    const int r0 = blockIdx.x * p.rows_per_cta, n = min(p.rows_per_cta, p.T - r0);
    const int pairs = p.rot >> 1, tid = threadIdx.x;
    wait_predecessor();
    launch_dependents();
    if (p.cu) {
        for (int i = tid; i <= p.B; i += kRopeThreads) cu_s[i] = p.cu[i];
        __syncthreads();
    }
    if (tid < n) {
        const int r = r0 + tid;
        long long pos = -1;
        if (!p.cu) {
            pos = p.start[r];
        } else if (r >= cu_s[0] && r < cu_s[p.B]) {
            int lo = 0, hi = p.B;                        // the last b with cu[b] <= r
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu_s[mid] <= r) lo = mid;
                else hi = mid;
            }
            const int st = p.start[lo];
            if (st >= 0) pos = (long long)st + r - cu_s[lo];
        }
        pos_s[tid] = pos < 0 ? -1 : pos;
    }
    __syncthreads();
    for (int i = tid; i < n * pairs; i += kRopeThreads) {
        const int row = i / pairs, f = i - row * pairs;
        const unsigned long long turn = (unsigned long long)pos_s[row] * p.turns[f];
        float s, c;
        sincospif((float)(long long)turn * 0x1p-63f, &s, &c);
        table[i] = make_float2(c * p.magnitude, s * p.magnitude * p.sign);
    }
    __syncthreads();
    // a head's places: its pairs, then what is left as it is
    constexpr int kW = V == 8 ? 8 : 1;
    const int turned = HALF ? pairs / kW : p.rot / (V == 8 ? 8 : 2);
    const int kept = (p.D - p.rot) / kW, per_head = turned + kept;
    const int per_row = per_head * (p.side[0].heads + p.side[1].heads);
    const int par = per_row >= kRopeThreads ? 1 : kRopeThreads / per_row;
    const int sub = per_row >= kRopeThreads ? 0 : tid / per_row;
    if (sub >= par) return;                              // a thread left over
    for (int j = per_row >= kRopeThreads ? tid : tid - sub * per_row; j < per_row; j += kRopeThreads) {
        const int head = j / per_head, at = j - head * per_head;
        const bool key = head >= p.side[0].heads;
        const RopeSide& sd = p.side[key];
        const long long h0 = (long long)(key ? head - p.side[0].heads : head) * p.D;
        const bool turn = at < turned;
        // first and (half layout) second place of the thread's values
        const int d0 = !turn ? p.rot + (at - turned) * kW : HALF ? at * kW : at * (V == 8 ? 8 : 2), d1 = d0 + pairs;
        const __half* x = sd.x + (long long)r0 * sd.ldx + h0;
        __half* y = sd.y + (long long)r0 * sd.ldy + h0;
        if (!turn && sd.x == sd.y) continue;
        for (int base = sub; base < n; base += kRopeRows * par) {
            if constexpr (V == 8) {
                uint4 a[kRopeRows], b[kRopeRows];
#pragma unroll
                for (int u = 0; u < kRopeRows; ++u) {
                    const int row = base + u * par;
                    if (row < n && pos_s[row] >= 0) {
                        a[u] = *reinterpret_cast<const uint4*>(x + row * sd.ldx + d0);
                        if (HALF && turn) b[u] = *reinterpret_cast<const uint4*>(x + row * sd.ldx + d1);
                    }
                }
#pragma unroll
                for (int u = 0; u < kRopeRows; ++u) {
                    const int row = base + u * par;
                    if (row >= n || pos_s[row] < 0) continue;
                    if (turn) {
                        __half2* av = reinterpret_cast<__half2*>(&a[u]);
                        const float2* cs = table + row * pairs + (HALF ? d0 : d0 / 2);
                        if (HALF) {
                            __half2* bv = reinterpret_cast<__half2*>(&b[u]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 fa = __half22float2(av[i]), fb = __half22float2(bv[i]);
                                const float4 t = *reinterpret_cast<const float4*>(cs + 2 * i);       // (cos, sin) twice
                                av[i] = __floats2half2_rn(fa.x * t.x - fb.x * t.y, fa.y * t.z - fb.y * t.w);
                                bv[i] = __floats2half2_rn(fa.x * t.y + fb.x * t.x, fa.y * t.w + fb.y * t.z);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 f = __half22float2(av[i]), t = cs[i];
                                av[i] = __floats2half2_rn(f.x * t.x - f.y * t.y, f.x * t.y + f.y * t.x);
                            }
                        }
                    }
                    *reinterpret_cast<uint4*>(y + row * sd.ldy + d0) = a[u];
                    if (HALF && turn) *reinterpret_cast<uint4*>(y + row * sd.ldy + d1) = b[u];
                }
            } else {
                for (int u = 0; u < kRopeRows; ++u) {
                    const int row = base + u * par;
                    if (row >= n || pos_s[row] < 0) continue;
                    const __half* xr = x + row * sd.ldx;
                    __half* yr = y + row * sd.ldy;
                    if (!turn) {
                        yr[d0] = xr[d0];
                        continue;
                    }
                    const int other = HALF ? d1 : d0 + 1;
                    const float fa = __half2float(xr[d0]), fb = __half2float(xr[other]);
                    const float2 t = table[row * pairs + (HALF ? d0 : d0 / 2)];
                    yr[d0] = __float2half_rn(fa * t.x - fb * t.y);
                    yr[other] = __float2half_rn(fa * t.y + fb * t.x);
                }
            }
        }
    }
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" int edge0_rope_turns(const edge0_rope_spec* s, unsigned long long* turns, double* radians, float* magnitude) {
    if (!s || !turns || !magnitude) return EDGE0_EINVAL;
    const int r = s->rot_dim;
    if (r < 2 || r % 2) return EDGE0_EINVAL;
    if (r > kRopeMaxDim) return EDGE0_EUNSUPPORTED;
    if (!(s->base > 1.0) || !isfinite(s->base)) return EDGE0_EINVAL;
    const bool stretched = s->scaling != EDGE0_ROPE_PLAIN;
    if (s->scaling < EDGE0_ROPE_PLAIN || s->scaling > EDGE0_ROPE_BANDS) return EDGE0_EINVAL;
    if (stretched && (!(s->factor >= 1.0) || !isfinite(s->factor))) return EDGE0_EINVAL;
    const bool ranged = s->scaling == EDGE0_ROPE_RAMP || s->scaling == EDGE0_ROPE_BANDS;
    if (ranged && (!(s->trained_len > 0.0) || !isfinite(s->trained_len) || !(s->low > 0.0) || !(s->high > s->low) ||
                   !isfinite(s->high)))
        return EDGE0_EINVAL;
    if (s->scaling == EDGE0_ROPE_BASE && r == 2) return EDGE0_EINVAL;      // (its one pair does not depend on the base)
    constexpr double kTurn = 6.283185307179586476925;
    const double base = s->scaling == EDGE0_ROPE_BASE ? s->base * pow(s->factor, (double)r / (r - 2)) : s->base;
    if (!isfinite(base)) return EDGE0_EINVAL;
    double from = 0, to = 0;                             // the ramp's first and last pair
    if (s->scaling == EDGE0_ROPE_RAMP) {
        from = floor(r * log(s->trained_len / (s->high * kTurn)) / (2 * log(s->base)));
        to = ceil(r * log(s->trained_len / (s->low * kTurn)) / (2 * log(s->base)));
        from = from < 0 ? 0 : from;
        to = to > r - 1 ? r - 1 : to;
    }
    for (int i = 0; i < r / 2; ++i) {
        double f = pow(base, -2.0 * i / r), keep = 1;
        if (s->scaling == EDGE0_ROPE_LINEAR) keep = 0;
        if (s->scaling == EDGE0_ROPE_RAMP) keep = 1 - (i - from) / (to - from > 0.001 ? to - from : 0.001);
        if (s->scaling == EDGE0_ROPE_BANDS) keep = (s->trained_len * f / kTurn - s->low) / (s->high - s->low);
        keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
        if (stretched && s->scaling != EDGE0_ROPE_BASE) f = f * keep + f / s->factor * (1 - keep);
        if (radians) radians[i] = f;
        // f <= 1: less than a sixth of a turn, so that its 2^64-fold fits
        turns[i] = (unsigned long long)rint(f / kTurn * 0x1p64);
    }
    *magnitude = s->scaling == EDGE0_ROPE_RAMP ? (float)(0.1 * log(s->factor) + 1) : 1.f;
    return EDGE0_OK;
}

extern "C" int edge0_rope(const unsigned long long* turns, int head_dim, int rot_dim, int layout, float magnitude, int backward,
                          const uint16_t* q, long long ldq, int n_q_heads, uint16_t* q_out, long long ldqo, const uint16_t* k,
                          long long ldk, int n_k_heads, uint16_t* k_out, long long ldko, int T, const int32_t* start,
                          const int32_t* cu_rows, int B, cudaStream_t stream) {
    if (!turns || ((uintptr_t)turns & 7) || !start || !q || !q_out || T < 0 || B <= 0) return EDGE0_EINVAL;
    if (((uintptr_t)start | (uintptr_t)cu_rows) & 3) return EDGE0_EINVAL;
    if (cu_rows ? B > EDGE0_MAX_BATCHED : T != B) return EDGE0_EINVAL;
    if (layout != EDGE0_ROPE_HALF && layout != EDGE0_ROPE_INTERLEAVED) return EDGE0_EINVAL;
    if (head_dim <= 0 || rot_dim < 2 || rot_dim % 2 || rot_dim > head_dim) return EDGE0_EINVAL;
    if (head_dim % 8 || head_dim > kRopeMaxDim) return EDGE0_EUNSUPPORTED;
    if (n_q_heads <= 0 || n_k_heads < 0 || !(magnitude > 0.f) || !isfinite(magnitude)) return EDGE0_EINVAL;
    constexpr int kMaxHeads = EDGE0_MAX_KV_HEADS * EDGE0_MAX_Q_PER_KV;
    if (n_q_heads > kMaxHeads || n_k_heads > kMaxHeads) return EDGE0_EUNSUPPORTED;
    if (n_k_heads && (!k || !k_out)) return EDGE0_EINVAL;
    RopeP p;
    p.turns = turns;
    p.side[0] = RopeSide{(const __half*)q, (__half*)q_out, ldq, ldqo, n_q_heads};
    p.side[1] = RopeSide{(const __half*)k, (__half*)k_out, ldk, ldko, n_k_heads};
    for (int i = 0; i < (n_k_heads ? 2 : 1); ++i) {
        const RopeSide& s = p.side[i];
        const long long width = (long long)s.heads * head_dim;
        if ((((uintptr_t)s.x | (uintptr_t)s.y) & 15) || s.ldx < width || s.ldy < width || s.ldx % 8 || s.ldy % 8)
            return EDGE0_EINVAL;
        if (s.x == s.y && s.ldx != s.ldy) return EDGE0_EINVAL;
    }
    if (T == 0) return EDGE0_OK;
    p.D = head_dim;
    p.rot = rot_dim;
    p.magnitude = magnitude;
    p.sign = backward ? -1.f : 1.f;
    p.T = T;
    p.B = B;
    p.start = start;
    p.cu = cu_rows;
    // tokens per CTA: so many that four CTAs per SM cover T
    const int want = (T - 1) / (152 * 4) + 1;                // (T up to the largest int)
    p.rows_per_cta = want > kRopeMaxRows ? kRopeMaxRows : want;
    const int grid = (T - 1) / p.rows_per_cta + 1, smem = p.rows_per_cta * (rot_dim / 2) * (int)sizeof(float2);
    // 16-byte places need every run of turned dims to begin and end on one
    if (layout == EDGE0_ROPE_HALF)
        return rot_dim % 16 == 0 ? launch_early(rope_kernel<true, 8>, dim3(grid), kRopeThreads, smem, stream, p)
                                 : launch_early(rope_kernel<true, 1>, dim3(grid), kRopeThreads, smem, stream, p);
    return rot_dim % 8 == 0 ? launch_early(rope_kernel<false, 8>, dim3(grid), kRopeThreads, smem, stream, p)
                            : launch_early(rope_kernel<false, 1>, dim3(grid), kRopeThreads, smem, stream, p);
}
