// Dense int4 projection y = W x, W int4 affine group-64 in the row-tile layout of
// edge0_pack_q4_rows: per 16-row tile and group of 64 inputs one 576-byte unit.
//
//     y[b][o] = sum_g ( s[o,g] sum_{i in g} q[o,i] x[b,i]  +  b[o,g] sum_{i in g} x[b,i] )
//
// Nibbles enter m16n8k16 steps as fp16 subnormals (exact products, fp32 sums); the
// group's scale and bias are applied to the fp32 sums.
//
// Few tokens (q4_few_kernel).  Its floor is the weights' bytes.  A CTA takes row tiles in
// turn, its eight warps a slice of the groups each, through rings of bulk copies (a
// slice is one run of bytes); x and its group sums stay in shared memory, laid down
// once.  A warp has its 16 rows for all tokens, so a nibble is unpacked once.  Measured:
// 65,537 x 2048 at one token 16.5 us, 4.6 TB/s of weights, 0.68 of what a copy reaches:
// the unpacking's instructions (issue slots 54 % taken) and the step's join across
// warps, not the memory, are the limit; 5120 x 2048 at 7 tokens 6.0 us and
// 2048 x 2048 at one token 2.5 us are launch, one latency of x, one of the weights and
// the join.
// More tokens (q4_many_kernel).  64 rows x 32 tokens per CTA, four warps for the even
// groups and four for the odd ones, x and weights through one ring, four groups
// between two barriers; the group sums of x are one more matrix step against ones.
// A CTA alone on its SM is bound by latency (0.8 us per step of four groups, with two 1.3 us:
// the matrix pipe is half taken then).  6144 x 1536 at 64 tokens 10.5 us, 115
// TFLOP/s; 20,000 x 2048 at 256 tokens 103 us, 205 TFLOP/s.  Against it: 64 tokens per
// CTA 13.9 and 105 us (against 11.1 and 103, all in plain launch order); 32 rows 13.6 us in the first; weights straight into registers,
// two groups between barriers, 12.5 us in the first.
#include "common.cuh"
#include "launch.cuh"
#include "mma.cuh"
#include "wait.cuh"

namespace edge0 {
namespace {

// Most tokens of q4_few_kernel.  Against q4_many_kernel, us: 1,000 x 2048 at 16 and 17 tokens 6.6 and
// 9.1, 5120 x 2048 10.6 and 9.7, 20,000 x 2048 16 and 21.
constexpr int kFewTokens = 16;
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
__global__ void __launch_bounds__(kThreadsQ) q4_few_kernel(const char* w, int out, int in,
                                                           const __half* x, long long ldx, int B, int tokens,
                                                           __half* y, long long ldy, unsigned long long wait_ns) {
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
    const int chunks = wait_ns ? (c1 - c0 + kChunk - 1) / kChunk : 0;      // (limit 0: given up from the start)
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
    wait_predecessor();
    launch_dependents();
    for (int s = 0; s < kStages - 1; ++s) issue();

    // x: lane t's 16 inputs of a group (2t, 2t + 1, 2t + 8, 2t + 9 of each 16) side by side.  A
    // thread takes 16-byte pieces (piece p of a group: word p of each t), four under way at a time;
    // the four groups of a warp start with a different t each, so that they miss each other's banks.
    const int pieces = n_g * 8, all_pieces = nb * pieces;
    for (int i0 = tid; i0 < all_pieces; i0 += 4 * kThreadsQ) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kThreadsQ, b = i / pieces;
            if (i < all_pieces) v[j] = *reinterpret_cast<const uint4*>(x + (long long)(b0 + b) * ldx + (i - b * pieces) * 8);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kThreadsQ, b = i / pieces, at = i - b * pieces, c = at >> 3, q = at & 7;
            if (i >= all_pieces) break;
            const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&v[j].x));
            const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&v[j].y));
            const float2 f2 = __half22float2(*reinterpret_cast<const __half2*>(&v[j].z));
            const float2 f3 = __half22float2(*reinterpret_cast<const __half2*>(&v[j].w));
            float sum = ((f0.x + f0.y) + (f1.x + f1.y)) + ((f2.x + f2.y) + (f3.x + f3.y));
            // (a group's eight threads are eight lanes of one warp, all here)
            const unsigned octet = 0xffu << (lane & ~7);
            sum += __shfl_xor_sync(octet, sum, 1);
            sum += __shfl_xor_sync(octet, sum, 2);
            sum += __shfl_xor_sync(octet, sum, 4);
            if (q == 0) xsum[c * 8 * NT + b] = sum;
            uint32_t w0 = v[j].x, w1 = v[j].y, w2 = v[j].z, w3 = v[j].w;
            const int turn = (lane >> 3) & 3;
            if (turn & 1) {
                const uint32_t o = w0;
                w0 = w1, w1 = w2, w2 = w3, w3 = o;
            }
            if (turn & 2) {
                const uint32_t o0 = w0, o1 = w1;
                w0 = w2, w1 = w3, w2 = o0, w3 = o1;
            }
            char* dst = smem + L.x + b * L.ld + c * 128 + q * 4;
            *reinterpret_cast<uint32_t*>(dst + turn * 32) = w0;
            *reinterpret_cast<uint32_t*>(dst + ((turn + 1) & 3) * 32) = w1;
            *reinterpret_cast<uint32_t*>(dst + ((turn + 2) & 3) * 32) = w2;
            *reinterpret_cast<uint32_t*>(dst + ((turn + 3) & 3) * 32) = w3;
        }
    }
    __syncthreads();

    // tokens that are not there repeat the last one; their sums are not written
    const char* xrow[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xrow[nt] = smem + L.x + min(nt * 8 + g, nb - 1) * L.ld + t * 32;
    int it = 0, buf = 0;
    bool dead = wait_ns == 0;
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
            if (!wait_copy(&bar[st], (uint32_t)(it / kStages) & 1, wait_ns)) {
                // (inline or called as leaves the other ways their registers: each 2 % faster in its place)
                if (RT == 2) drain_copies(bar, it, issued, kStages);
                else drain_copies_call(bar, it, issued, kStages);
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

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
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

constexpr int kManyTok = 32;            // tokens of a CTA
constexpr int kStep = 4;                // groups between two barriers
constexpr int kManyStages = 4;          // steps under way: x of the tokens, the four row tiles' units
constexpr int kManyStage = kStep * (kManyTok * 128 + 4 * kQ4Unit);
constexpr int kManySmem = kManyStages * kManyStage;

__global__ void __launch_bounds__(256, 2) q4_many_kernel(const char* w, int out, int in,
                                                      const __half* x, long long ldx, int B,
                                                      __half* y, long long ldy, unsigned long long wait_ns) {
    constexpr int kTok = kManyTok, NT = kTok / 8, kTile = kTok * 128;     // kTile: bytes of one group of them
    constexpr int kStages = kManyStages, kStage = kManyStage, kJ = kStep / 2;
    extern __shared__ __align__(128) char smem[];
    char* ring = smem;
    __shared__ float xs[2][kStep][kTok];
    __shared__ uint64_t full[kStages];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t = lane & 3;
    const int half = wid >> 2, rw = wid & 3;                  // parity of this warp's groups, its 16 rows
    const int n_g = in / kGroup, n_rt = ceil_div(out, kRowTile);
    const int rt = blockIdx.x * 4 + rw, b0 = blockIdx.y * kTok, nb = min(kTok, B - b0);
    const bool rows = rt < n_rt;
    const int steps = ceil_div(n_g, kStep);

    // this thread's 16-byte pieces of a step: piece pc of token pb, of each group
    const int pc = tid & 7, pb = tid >> 3;
    const __half* px = x + (long long)(b0 + min(pb, nb - 1)) * ldx + pc * 8;
    const uint32_t pdst = smem_u32(ring) + pb * 128 + ((pc ^ (pb & 7)) << 4);
    const int tiles = min(4, n_rt - (int)blockIdx.x * 4);
    const char* wsrc = w + (long long)blockIdx.x * 4 * n_g * kQ4Unit;
    int good = wait_ns ? steps : 0;                           // steps whose weights this warp has seen arrive
    auto fetch = [&](int step) {
        if (step < steps) {
            const int at = (step % kStages) * kStage;
            if (tid == 0 && step < good + kStages - 1) {
                const uint32_t bytes = min(kStep, n_g - kStep * step) * kQ4Unit;
                uint64_t* bar = &full[step % kStages];
                mbar_arrive_expect_tx(bar, tiles * bytes);
                for (int i = 0; i < tiles; ++i)
                    copy_bulk(ring + at + kStep * kTile + i * kStep * kQ4Unit, wsrc + ((long long)i * n_g + kStep * step) * kQ4Unit,
                              bytes, bar);
            }
            const __half* src = px + step * kStep * kGroup;
            const int have = n_g - kStep * step;
#pragma unroll
            for (int q = 0; q < kStep; ++q)
                if (q < have) cp_async16(pdst + at + q * kTile, src + q * kGroup, pb < nb);
        }
        cp_commit();
    };
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncthreads();
    wait_predecessor();
    launch_dependents();
    for (int s = 0; s < kStages - 1; ++s) fetch(s);

    float y4[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) y4[nt][i] = 0.f;
    float2 bias[kJ];                                          // of the step before: x's sums come a step later
    const uint32_t ones[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
    auto add_bias = [&](int step, int j) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 v = *reinterpret_cast<const float2*>(&xs[step & 1][2 * j + half][nt * 8 + 2 * t]);
            y4[nt][0] = fmaf(bias[j].x, v.x, y4[nt][0]);
            y4[nt][1] = fmaf(bias[j].x, v.y, y4[nt][1]);
            y4[nt][2] = fmaf(bias[j].y, v.x, y4[nt][2]);
            y4[nt][3] = fmaf(bias[j].y, v.y, y4[nt][3]);
        }
    };
    // ldmatrix rows of this lane: token (lane & 7) + 8 (lane >> 4), 16-byte half (lane >> 3) & 1 of a k step
    const int lt = (lane & 7) + 8 * (lane >> 4), lh = (lane >> 3) & 1;
    auto group = [&](int step, int j, const char* stage) {    // group 2 j + half of the step
        const int c = 2 * j + half;
        // (a row tile behind the last: whatever is there, its rows are not written)
        const char* unit = stage + kStep * kTile + (rw * kStep + c) * kQ4Unit;
        const uint4 q = *reinterpret_cast<const uint4*>(unit + 16 * lane);
        const uint2 sbw = *reinterpret_cast<const uint2*>(unit + 512 + 8 * g);
        const uint32_t words[4] = {q.x, q.y, q.z, q.w};
        const float2 sb0 = __half22float2(*reinterpret_cast<const __half2*>(&sbw.x));
        const float2 sb1 = __half22float2(*reinterpret_cast<const __half2*>(&sbw.y));
        const float s0 = sb0.x * kTwo24, s1 = sb1.x * (kTwo24 / 16.f);
        bias[j] = make_float2(sb0.y, sb1.y);
        uint32_t A[4][4];
#pragma unroll
        for (int s = 0; s < 4; ++s) q4_masks(words[s], A[s]);
        const uint32_t base = smem_u32(stage) + c * kTile;
        uint32_t b[4][2][4];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int np = 0; np < 2; ++np) ldsm4(b[s][np], base + (np * 16 + lt) * 128 + (((2 * s + lh) ^ (lt & 7)) << 4));
        float acc[NT][4], sum[4];
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < NT; ++i) {                    // blocks next to each other: none waits for the one before
                const uint32_t x0 = b[s][i >> 1][2 * (i & 1)], x1 = b[s][i >> 1][2 * (i & 1) + 1];
                if (s == 0) mma_16816_first(acc[i], A[0], x0, x1);
                else mma_16816_v(acc[i], A[s], x0, x1);
            }
        // each row-warp adds up x of one of the four blocks
        uint32_t xb[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) ldsm4(xb[h], base + (rw * 8 + (lane & 7)) * 128 + (((4 * h + (lane >> 3)) ^ (lane & 7)) << 4));
        mma_16816_first(sum, ones, xb[0][0], xb[0][1]);
        mma_16816_v(sum, ones, xb[0][2], xb[0][3]);
        mma_16816_v(sum, ones, xb[1][0], xb[1][1]);
        mma_16816_v(sum, ones, xb[1][2], xb[1][3]);
        if (g == 0) *reinterpret_cast<float2*>(&xs[step & 1][c][rw * 8 + 2 * t]) = make_float2(sum[0], sum[1]);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            y4[i][0] = fmaf(s0, acc[i][0], y4[i][0]);
            y4[i][1] = fmaf(s0, acc[i][1], y4[i][1]);
            y4[i][2] = fmaf(s1, acc[i][2], y4[i][2]);
            y4[i][3] = fmaf(s1, acc[i][3], y4[i][3]);
        }
    };
    for (int step = 0; step < steps; ++step) {
        const char* stage = ring + (step % kStages) * kStage;
        cp_wait<kStages - 2>();
        if (step < good && !wait_copy(&full[step % kStages], (uint32_t)(step / kStages) & 1, wait_ns)) good = step;
        __syncthreads();                                      // the stage of the step before is free, too
        fetch(step + kStages - 1);
        if (step > 0)
#pragma unroll
            for (int j = 0; j < kJ; ++j) add_bias(step - 1, j);
        const int have = n_g - kStep * step;
        if (have >= kStep) {
#pragma unroll
            for (int j = 0; j < kJ; ++j) group(step, j, stage);
        } else {
#pragma unroll
            for (int j = 0; j < kJ; ++j)
                if (2 * j + half < have) group(step, j, stage);
        }
    }
    __syncthreads();
    const int have = n_g - kStep * (steps - 1);
#pragma unroll
    for (int j = 0; j < kJ; ++j)
        if (2 * j + half < have) add_bias(steps - 1, j);
    if (good < steps) {                                       // a copy that never came: NaN marks the rows
        if (wid == 0) drain_copies(full, good, min(good + kStages - 1, steps), kStages);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) y4[nt][i] = __int_as_float(0x7fffffff);
    }
    // the odd groups' sums through shared memory
    cp_wait<0>();
    __syncthreads();
    float4* other = reinterpret_cast<float4*>(ring);          // [row tile][8-token block][lane]
    if (half == 1)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            other[(rw * NT + nt) * 32 + lane] = make_float4(y4[nt][0], y4[nt][1], y4[nt][2], y4[nt][3]);
    __syncthreads();
    if (half == 0 && rows) {
        const int r0 = rt * kRowTile + g;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float4 o = other[(rw * NT + nt) * 32 + lane];
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

unsigned long long wait_limit = kDefaultWaitNs;

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
        if (cudaFuncSetAttribute(q4_many_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kManySmem) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return EDGE0_ECUDA;
        __atomic_store_n(&known[dev], n, __ATOMIC_RELEASE);
    }
    *sms = n;
    return EDGE0_OK;
}

}  // namespace

unsigned long long block_wait_limit() { return __atomic_load_n(&wait_limit, __ATOMIC_RELAXED); }

}  // namespace edge0

using namespace edge0;

extern "C" void edge0_block_set_wait_limit(unsigned long long wait_ns) {
    __atomic_store_n(&wait_limit, wait_ns, __ATOMIC_RELAXED);
}

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
        return launch_early(f, grid, kThreadsQ, smem, stream, w, out, in, xh, ldx, B, tokens, yh, ldy,
                            block_wait_limit());
    }
    return launch_early(q4_many_kernel, dim3(ceil_div(n_rt, 4), ceil_div(B, kManyTok)), 256, kManySmem, stream, w, out, in, xh, ldx,
                        B, yh, ldy, block_wait_limit());
}
