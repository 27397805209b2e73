// Dense int4 projection y = W x, W int4 affine group-64 in the row-tile layout of
// edge0_pack_q4_rows: per 16-row tile and group of 64 inputs one 576-byte unit.
//
//     y[b][o] = sum_g ( s[o,g] sum_{i in g} q[o,i] x[b,i]  +  b[o,g] sum_{i in g} x[b,i] )
//
// Nibbles enter m16n8k16 steps as fp16 subnormals (exact products, fp32 sums); the
// group's scale and bias are applied to the fp32 sums.
//
// Few tokens (q4_few_kernel): bound by the weights' bytes.  A CTA takes row tiles in
// turn, its eight warps a slice of the groups each, through rings of bulk copies (a
// slice is one run of bytes); x and its group sums stay in shared memory.
// More tokens (q4_many_kernel): bound by the matrix steps.  64 rows x up to 64 tokens per
// CTA, four warps for the even groups and four for the odd ones; x comes through a
// ring of asynchronous copies, the weights straight into registers two groups ahead,
// and the group sums of x are one more matrix step against ones.
#include "common.cuh"
#include "mma.cuh"

namespace edge0 {
namespace {

constexpr int kFewTokens = 16;          // most tokens of q4_few_kernel
constexpr int kWarps = 8;
constexpr int kThreadsQ = 32 * kWarps;
constexpr int kChunk = 4;               // groups per bulk copy
constexpr int kChunkBytes = kChunk * kQ4Unit;
constexpr int kPartLd = 20;             // floats per token of a warp's part: its stores then miss each other's banks

__device__ __forceinline__ void copy_bulk(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
// Waits for a copy, at most kDefaultWaitNs; the whole warp agrees on the answer.
__device__ __forceinline__ bool wait_copy(uint64_t* bar, uint32_t parity) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        unsigned long long t0, now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        do {
            ok = mbar_try_wait(bar, parity);
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        } while (!ok && now - t0 < kDefaultWaitNs);
    }
    return __all_sync(0xffffffffu, ok);
}

// Shared memory of q4_few_kernel: rings, x in fragment order, group sums, partial sums.
// RT: row tiles taken together (2 where there are enough of them: x's fragments, the
// joins and the barrier then serve both).
__host__ __device__ constexpr int few_stages(int RT) { return RT == 2 ? 2 : 4; }
struct FewLayout {
    int ld, x, xsum, part, bars, total;     // bytes; ld: of one token of x
};
__host__ __device__ inline FewLayout few_layout(int in, int tokens, int NT, int RT) {
    FewLayout l;
    const int n_g = in / kGroup;
    l.ld = in * 2 + 16;                     // 16 bytes on: two tokens' 16-byte pieces never share a bank
    l.x = kWarps * few_stages(RT) * RT * kChunkBytes;
    l.xsum = l.x + tokens * l.ld;
    l.part = l.xsum + n_g * 8 * NT * 4;
    l.bars = l.part + 2 * kWarps * RT * 8 * NT * kPartLd * 4;
    l.total = l.bars + kWarps * few_stages(RT) * 8;
    return l;
}

template <int NT, int RT>
__global__ void __launch_bounds__(kThreadsQ) q4_few_kernel(const char* __restrict__ w, int out, int in,
                                                           const __half* __restrict__ x, long long ldx, int B, int tokens,
                                                           __half* __restrict__ y, long long ldy) {
    constexpr int kStages = few_stages(RT);
    extern __shared__ __align__(128) char smem[];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t = lane & 3;
    const int n_g = in / kGroup, n_rt = ceil_div(out, kRowTile);
    const FewLayout L = few_layout(in, tokens, NT, RT);
    const int b0 = blockIdx.y * tokens, nb = min(tokens, B - b0);
    float* xsum = reinterpret_cast<float*>(smem + L.xsum);
    float* part = reinterpret_cast<float*>(smem + L.part);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L.bars) + wid * kStages;
    char* ring = smem + wid * kStages * RT * kChunkBytes;

    if (lane < kStages) mbar_init(&bar[lane], 1);
    fence_mbar_init();
    __syncwarp();
    // this warp's groups of every row tile, in chunks
    const int c0 = n_g * wid / kWarps, c1 = n_g * (wid + 1) / kWarps;
    const int chunks = (c1 - c0 + kChunk - 1) / kChunk;
    const int n_t = ceil_div(n_rt, RT);                      // steps over the row tiles
    int next_t = blockIdx.x, next_chunk = 0, issued = 0;
    auto issue = [&]() {
        if (next_t < n_t && chunks) {
            if (lane == 0) {
                const int a = c0 + next_chunk * kChunk, bytes = min(kChunk, c1 - a) * kQ4Unit;
                const int st = issued % kStages, n = min(RT, n_rt - next_t * RT);
                mbar_arrive_expect_tx(&bar[st], n * bytes);
                const char* src = w + ((long long)next_t * RT * n_g + a) * kQ4Unit;
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    if (i < n)
                        copy_bulk(ring + (st * RT + i) * kChunkBytes, src + (long long)i * n_g * kQ4Unit, bytes, &bar[st]);
            }
            ++issued;
            if (++next_chunk == chunks) {
                next_chunk = 0;
                next_t += gridDim.x;
            }
        }
    };
    for (int s = 0; s < kStages - 1; ++s) issue();

    // x: lane t's 16 inputs of a group (2t, 2t + 1, 2t + 8, 2t + 9 of each 16) side by side
    for (int i = tid; i < nb * n_g * 4; i += kThreadsQ) {
        const int tt = i & 3, c = (i >> 2) % n_g, b = (i >> 2) / n_g;
        const __half* src = x + (long long)(b0 + b) * ldx + c * kGroup + 2 * tt;
        uint32_t v[8];
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = *reinterpret_cast<const uint32_t*>(src + 8 * j);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
            s += f.x + f.y;
        }
        uint4* dst = reinterpret_cast<uint4*>(smem + L.x + b * L.ld + c * 128 + tt * 32);
        dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
        dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
        // (a group's four threads are four lanes of one warp, all in the loop)
        const unsigned quad = 0xfu << (lane & ~3);
        s += __shfl_xor_sync(quad, s, 1);
        s += __shfl_xor_sync(quad, s, 2);
        if (tt == 0) xsum[c * 8 * NT + b] = s;
    }
    __syncthreads();

    // tokens that are not there repeat the last one; their sums are not written
    const char* xrow[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xrow[nt] = smem + L.x + min(nt * 8 + g, nb - 1) * L.ld + t * 32;
    int it = 0, buf = 0;
    bool dead = false;
    for (int rt = blockIdx.x; rt < n_t; rt += gridDim.x, buf ^= 1) {
        float y4[RT][NT][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) y4[r][nt][i] = 0.f;
        for (int ch = 0; ch < chunks && !dead; ++ch, ++it) {
            issue();
            const int st = it % kStages;
            if (!wait_copy(&bar[st], (uint32_t)(it / kStages) & 1)) {
                dead = true;                     // a copy that never came: NaN marks the rows from here on
                break;
            }
            const char* u = ring + st * RT * kChunkBytes;
            const int a = c0 + ch * kChunk, n = min(kChunk, c1 - a);
            auto group = [&](int q) {
                uint4 xa[NT], xb[NT];
                float2 xs[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    xa[nt] = *reinterpret_cast<const uint4*>(xrow[nt] + (a + q) * 128);
                    xb[nt] = *reinterpret_cast<const uint4*>(xrow[nt] + (a + q) * 128 + 16);
                    xs[nt] = *reinterpret_cast<const float2*>(xsum + (a + q) * 8 * NT + nt * 8 + 2 * t);
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {   // (a tile behind the last holds an older tile's codes; not written)
                    const char* unit = u + r * kChunkBytes + q * kQ4Unit;
                    const uint4 qw = *reinterpret_cast<const uint4*>(unit + 16 * lane);
                    const uint2 sbw = *reinterpret_cast<const uint2*>(unit + 512 + 8 * g);
                    const uint32_t words[4] = {qw.x, qw.y, qw.z, qw.w};
                    uint32_t A[4][4];
#pragma unroll
                    for (int s = 0; s < 4; ++s) q4_masks(words[s], A[s]);
                    const float2 sb0 = __half22float2(*reinterpret_cast<const __half2*>(&sbw.x));
                    const float2 sb1 = __half22float2(*reinterpret_cast<const __half2*>(&sbw.y));
                    const float s0 = sb0.x * kTwo24, s1 = sb1.x * (kTwo24 / 16.f);     // nibbles of rows g + 8: x16
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float acc[4];
                        mma_16816_first(acc, A[0], xa[nt].x, xa[nt].y);
                        mma_16816_v(acc, A[1], xa[nt].z, xa[nt].w);
                        mma_16816_v(acc, A[2], xb[nt].x, xb[nt].y);
                        mma_16816_v(acc, A[3], xb[nt].z, xb[nt].w);
                        float(&o)[4] = y4[r][nt];
                        o[0] = fmaf(s0, acc[0], fmaf(sb0.y, xs[nt].x, o[0]));
                        o[1] = fmaf(s0, acc[1], fmaf(sb0.y, xs[nt].y, o[1]));
                        o[2] = fmaf(s1, acc[2], fmaf(sb1.y, xs[nt].x, o[2]));
                        o[3] = fmaf(s1, acc[3], fmaf(sb1.y, xs[nt].y, o[3]));
                    }
                }
            };
            if (n == kChunk) {                   // without branches between them the groups overlap
#pragma unroll
                for (int q = 0; q < kChunk; ++q) group(q);
            } else {
                for (int q = 0; q < n; ++q) group(q);
            }
            __syncwarp();                        // the stage is free again
        }
        // the warps' parts, [row tile][token][row]: two buffers, so that one barrier per step is enough
        float* mine = part + (buf * kWarps + wid) * RT * 8 * NT * kPartLd;
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int b = nt * 8 + 2 * t + (i & 1);
                    if (b < nb) mine[(r * 8 * NT + b) * kPartLd + g + 8 * (i >> 1)] = dead ? __int_as_float(0x7fffffff) : y4[r][nt][i];
                }
        __syncthreads();
        for (int i = tid; i < RT * nb * 16; i += kThreadsQ) {
            const int r = i & 15, rb = i >> 4, b = rb % nb, tile = rt * RT + rb / nb;
            const float* src = part + buf * kWarps * RT * 8 * NT * kPartLd + (rb / nb * 8 * NT + b) * kPartLd + r;
            float s = 0.f;
#pragma unroll
            for (int q = 0; q < kWarps; ++q) s += src[q * RT * 8 * NT * kPartLd];
            const int row = tile * kRowTile + r;
            if (row < out) y[(long long)(b0 + b) * ldy + row] = __float2half_rn(s);
        }
    }
}

// 16 bytes, or zeros where there is nothing to copy
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

constexpr int kManyStages = 3;

// NT: 8-token blocks per CTA (4 or 8)
template <int NT>
__global__ void __launch_bounds__(256, 2) q4_many_kernel(const char* __restrict__ w, int out, int in,
                                                      const __half* __restrict__ x, long long ldx, int B,
                                                      __half* __restrict__ y, long long ldy) {
    constexpr int kTok = 8 * NT, kTile = kTok * 128;          // tokens; bytes of one group of them
    extern __shared__ __align__(128) char smem[];
    char* ring = smem;
    __shared__ float xs[2][2][kTok];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t = lane & 3;
    const int half = wid >> 2, rw = wid & 3;                  // parity of this warp's groups, its 16 rows
    const int n_g = in / kGroup, n_rt = ceil_div(out, kRowTile);
    const int rt = blockIdx.x * 4 + rw, b0 = blockIdx.y * kTok, nb = min(kTok, B - b0);
    const bool rows = rt < n_rt;
    const int steps = (n_g + 1) / 2;                          // a step is two groups

    // this thread's 16-byte pieces of a step: piece c of tokens b, b + 32.. of either group
    const int pc = tid & 7, pb = tid >> 3;
    const __half* px = x + (long long)(b0 + pb) * ldx + pc * 8;
    const uint32_t pdst = smem_u32(ring) + pb * 128 + ((pc ^ (pb & 7)) << 4);
    auto fetch = [&](int step) {
        if (step < steps) {
            const uint32_t dst = pdst + (step % kManyStages) * 2 * kTile;
            const __half* src = px + step * 2 * kGroup;
#pragma unroll
            for (int j = 0; j < kTok / 32; ++j) {
                const bool there = pb + 32 * j < nb;
                const __half* row = src + (there ? (long long)(32 * j) * ldx : -(long long)pb * ldx);
                cp_async16(dst + j * 32 * 128, row, there);
                if (2 * step + 1 < n_g) cp_async16(dst + j * 32 * 128 + kTile, row + kGroup, there);
            }
        }
        cp_commit();
    };
    const char* tile = w + (long long)(rows ? rt : 0) * n_g * kQ4Unit;
    uint4 qn[2];
    uint2 sn[2];
    auto weights = [&](int step, int slot) {
        const int c = 2 * step + half;
        if (c < n_g) {
            qn[slot] = __ldg(reinterpret_cast<const uint4*>(tile + (long long)c * kQ4Unit + 16 * lane));
            sn[slot] = __ldg(reinterpret_cast<const uint2*>(tile + (long long)c * kQ4Unit + 512 + 8 * g));
        }
    };
    weights(0, 0);
    weights(1, 1);
    for (int s = 0; s < kManyStages - 1; ++s) fetch(s);

    float y4[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) y4[nt][i] = 0.f;
    float bias0 = 0.f, bias1 = 0.f;                           // of the group before: its sums come a step later
    const uint32_t ones[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
    auto add_bias = [&](int step) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 v = *reinterpret_cast<const float2*>(&xs[step & 1][half][nt * 8 + 2 * t]);
            y4[nt][0] = fmaf(bias0, v.x, y4[nt][0]);
            y4[nt][1] = fmaf(bias0, v.y, y4[nt][1]);
            y4[nt][2] = fmaf(bias1, v.x, y4[nt][2]);
            y4[nt][3] = fmaf(bias1, v.y, y4[nt][3]);
        }
    };
    // ldmatrix rows of this lane: token (lane & 7) + 8 (lane >> 4), 16-byte half (lane >> 3) & 1 of a k step
    const int lt = (lane & 7) + 8 * (lane >> 4), lh = (lane >> 3) & 1;
    for (int step = 0; step < steps; ++step) {
        cp_wait<kManyStages - 2>();
        __syncthreads();
        fetch(step + kManyStages - 1);
        if (step > 0) add_bias(step - 1);
        const bool mine = 2 * step + half < n_g;
        if (mine) {
            const uint4 q = step & 1 ? qn[1] : qn[0];
            const uint2 sbw = step & 1 ? sn[1] : sn[0];
            if (step & 1) weights(step + 2, 1);
            else weights(step + 2, 0);
            const uint32_t words[4] = {q.x, q.y, q.z, q.w};
            const float2 sb0 = __half22float2(*reinterpret_cast<const __half2*>(&sbw.x));
            const float2 sb1 = __half22float2(*reinterpret_cast<const __half2*>(&sbw.y));
            const float s0 = sb0.x * kTwo24, s1 = sb1.x * (kTwo24 / 16.f);
            bias0 = sb0.y;
            bias1 = sb1.y;
            uint32_t A[4][4];
#pragma unroll
            for (int s = 0; s < 4; ++s) q4_masks(words[s], A[s]);
            const uint32_t base = smem_u32(ring) + ((step % kManyStages) * 2 + half) * kTile;
            // two 8-token blocks at a time, the next blocks' fragments under way meanwhile
            uint32_t bf[2][4][4];
            auto frags = [&](int np, uint32_t (&b)[4][4]) {
                const uint32_t at = base + (np * 16 + lt) * 128;
#pragma unroll
                for (int s = 0; s < 4; ++s)
                    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                                 : "=r"(b[s][0]), "=r"(b[s][1]), "=r"(b[s][2]), "=r"(b[s][3])
                                 : "r"(at + (((2 * s + lh) ^ (lt & 7)) << 4))
                                 : "memory");
            };
            frags(0, bf[0]);
#pragma unroll
            for (int np = 0; np < NT / 2; ++np) {
                if (np + 1 < NT / 2) frags(np + 1, bf[(np + 1) & 1]);
                const uint32_t(&b)[4][4] = bf[np & 1];
                float acc[2][4];
#pragma unroll
                for (int j = 0; j < 2; ++j) mma_16816_first(acc[j], A[0], b[0][2 * j], b[0][2 * j + 1]);
#pragma unroll
                for (int s = 1; s < 4; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) mma_16816_v(acc[j], A[s], b[s][2 * j], b[s][2 * j + 1]);
                if ((np & 3) == rw) {                         // each row-warp adds up its share of the tokens
                    float sum[2][4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        mma_16816_first(sum[j], ones, b[0][2 * j], b[0][2 * j + 1]);
#pragma unroll
                        for (int s = 1; s < 4; ++s) mma_16816_v(sum[j], ones, b[s][2 * j], b[s][2 * j + 1]);
                        if (g == 0)
                            *reinterpret_cast<float2*>(&xs[step & 1][half][(2 * np + j) * 8 + 2 * t]) =
                                make_float2(sum[j][0], sum[j][1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float(&o)[4] = y4[2 * np + j];
                    o[0] = fmaf(s0, acc[j][0], o[0]);
                    o[1] = fmaf(s0, acc[j][1], o[1]);
                    o[2] = fmaf(s1, acc[j][2], o[2]);
                    o[3] = fmaf(s1, acc[j][3], o[3]);
                }
            }
        }
    }
    __syncthreads();
    if (2 * (steps - 1) + half < n_g) add_bias(steps - 1);
    // the odd groups' sums through shared memory
    cp_wait<0>();
    __syncthreads();
    float* other = reinterpret_cast<float*>(ring);            // [4][kTok / 2 pairs ..][lane] as written
    if (half == 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            *reinterpret_cast<float4*>(other + ((rw * NT + nt) * 32 + lane) * 4) =
                make_float4(y4[nt][0], y4[nt][1], y4[nt][2], y4[nt][3]);
    __syncthreads();
    if (half == 0 && rows) {
        const int r0 = rt * kRowTile + g;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float4 o = *reinterpret_cast<const float4*>(other + ((rw * NT + nt) * 32 + lane) * 4);
            const float v[4] = {y4[nt][0] + o.x, y4[nt][1] + o.y, y4[nt][2] + o.z, y4[nt][3] + o.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int b = nt * 8 + 2 * t + (i & 1), row = r0 + 8 * (i >> 1);
                if (b < nb && row < out) y[(long long)(b0 + b) * ldy + row] = __float2half_rn(v[i]);
            }
        }
    }
}

constexpr int kFewSmem = 220 * 1024;
constexpr int many_smem(int NT) { return kManyStages * 2 * 8 * NT * 128; }

// what a device needs before its first launch
int setup(int dev, int* sms) {
    constexpr int kDevices = 64;
    static int known[kDevices];
    if (dev < 0 || dev >= kDevices) return EDGE0_ECUDA;
    int n = __atomic_load_n(&known[dev], __ATOMIC_ACQUIRE);
    if (n == 0) {
        const void* few[4] = {(const void*)q4_few_kernel<1, 1>, (const void*)q4_few_kernel<1, 2>,
                              (const void*)q4_few_kernel<2, 1>, (const void*)q4_few_kernel<2, 2>};
        for (const void* f : few)
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem) != cudaSuccess)
                return EDGE0_ECUDA;
        if (cudaFuncSetAttribute(q4_many_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, many_smem(8)) !=
                cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return EDGE0_ECUDA;
        __atomic_store_n(&known[dev], n, __ATOMIC_RELEASE);
    }
    *sms = n;
    return EDGE0_OK;
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" int edge0_q4_linear(const void* packed, int out, int in, const uint16_t* x, long long ldx, int B,
                               uint16_t* y, long long ldy, cudaStream_t stream) {
    if (!packed || !x || !y || out <= 0 || in <= 0 || in % kGroup) return EDGE0_EINVAL;
    if (B <= 0 || B > EDGE0_MAX_BATCHED || ldx < in || ldx % 8 || ldy < out) return EDGE0_EINVAL;
    if (out > EDGE0_MAX_LINEAR || in > EDGE0_MAX_LINEAR) return EDGE0_EUNSUPPORTED;    // row and byte counts are ints
    if ((((uintptr_t)packed | (uintptr_t)x) & 15) || ((uintptr_t)y & 1)) return EDGE0_EINVAL;
    const char* w = (const char*)packed;
    const __half* xh = (const __half*)x;
    __half* yh = (__half*)y;
    const int n_rt = ceil_div(out, kRowTile);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return EDGE0_ECUDA;
    const int rc = setup(dev, &sms);
    if (rc) return rc;
    // few tokens at once: as many as shared memory holds beside the rings; two row tiles
    // together once that still leaves every SM two CTAs' worth of them
    const int RT = n_rt >= 4 * sms ? 2 : 1;
    int tokens = B <= kFewTokens && in <= kFewSmem / 2 ? B : 0;
    while (tokens && few_layout(in, tokens, tokens > 8 ? 2 : 1, RT).total > kFewSmem)
        tokens = tokens > 8 ? 8 : tokens / 2;
    if (tokens) {
        const int NT = tokens > 8 ? 2 : 1, smem = few_layout(in, tokens, NT, RT).total, n_t = ceil_div(n_rt, RT);
        const int most = sms * (smem <= 113 * 1024 ? 2 : 1);
        const dim3 grid(n_t < most ? n_t : most, ceil_div(B, tokens));
        auto* f = NT == 1 ? (RT == 1 ? q4_few_kernel<1, 1> : q4_few_kernel<1, 2>)
                          : (RT == 1 ? q4_few_kernel<2, 1> : q4_few_kernel<2, 2>);
        f<<<grid, kThreadsQ, smem, stream>>>(w, out, in, xh, ldx, B, tokens, yh, ldy);
    } else {
        // 64 tokens per CTA where that fills the card, else 32
        const int rows = ceil_div(n_rt, 4);
        if (B > 32 && rows * ceil_div(B, 64) >= sms)
            q4_many_kernel<8><<<dim3(rows, ceil_div(B, 64)), 256, many_smem(8), stream>>>(w, out, in, xh, ldx, B, yh, ldy);
        else
            q4_many_kernel<4><<<dim3(rows, ceil_div(B, 32)), 256, many_smem(4), stream>>>(w, out, in, xh, ldx, B, yh, ldy);
    }
    return cudaGetLastError() == cudaSuccess ? EDGE0_OK : EDGE0_ECUDA;
}
