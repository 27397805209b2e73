// Attention of all sequences' queries over the prefix they share, on the
// fifth-generation tensor cores.
//
// One CTA: 128 query rows (sequence, head of one K/V head's group) x a share of the
// prefix, 64 tokens a step.  Per step
//   warps 8-11  turn a strip of codes each into fp16 (code - z, z half the code range: exact)
//               in shared memory, K as K-major, V as MN-major operand tiles, and its scales
//               into fp32 tables; the next step's codes are loaded into registers meanwhile;
//   warp 0      issues the scores' products, and once the weights are there O_g += P'_g V_g for
//               each 64 dims g; accumulators and P' (over the scores that the same warp has
//               read) in TMEM;
//   warps 0-7   32 rows x 32 tokens each: S, running maximum and sum, weights p,
//               P'_g = fp16(p s_g), and sum_j P'_g r_g in fp32.
// Scores: with K = s (code - z + r), r = b / s + z, a group's product is
// Q_g (code - z) + mean(Q_g) 64 r; the second term is one more step of 16 of the same
// product, its factors split into two fp16 each (the mean's second one 2^11 times as large,
// which a subnormal mean needs), so that S = sum_g s_g S_g carries no rounding of K or Q beyond
// 2^-22.  Each weight is rounded once (to fp16, 2^-11 of itself):
// with V = s (code - z + r) likewise, o = (O_g + sum P'_g r_g) / sum p.  Scores have the running
// maximum, scales a power of two above the largest so far as reference (kUp, kRise, kLowS:
// attn.cuh); a reference moves only when exceeded by 2^4, and the accumulators are
// then rescaled in TMEM.  A tile with a scale below 2^-9 of the reference gets a second product,
// of what the rounding took from its subnormal weights.
// The accumulators are read and P' written as 8-column fragments (a lane: 2 tokens of
// 4 rows): a token's scales, read from shared memory, serve 4 rows; with a row per
// thread reading them alone took 2000 cycles a step.
// Two CTAs per SM (D <= 128): one's tensor steps run under the other's softmax.
// The floor is the products: 2 x 2 x 128 x 8191 x 4096 of them for 256 sequences of 16 heads
// behind 8,191 tokens, 17 GFLOP, 9 us.  Measured: 46 us of that call's 68.  Neither pipe is full:
// issue slots 56 %, shared memory about half (operands written, read by the matrix steps,
// tables), matrix pipe 16 %; a tile's steps (scores, weights, product) wait for one another,
// and two CTAs are what shared memory, tensor memory (2 x 256 columns) and registers hold.
#include "attn.cuh"
#include "tc05.cuh"
#include "wait.cuh"

namespace edge0 {
namespace {

constexpr int kSoftmax = 256;             // threads of the softmax warps
constexpr int kThreads = kSoftmax + 128;  // and the operand warps
constexpr int kRowsQ = kPrefixRows;
constexpr int kTile = kPrefixTile;
constexpr int kAgain = 1, kLeave = 2;     // after a tile's product: another one for it; a wait ran out

template <int BITS, int D>
struct Cfg {
    static constexpr int R = kv::row_bytes(BITS, D);
    static constexpr int CH = R / 16;
    static constexpr int GR = D / kGroup;
    static constexpr int STRIP = kv::strip_bytes(BITS, D);
    static constexpr int HALF = kv::half_bytes(BITS, D);
    static constexpr int NP = CH / 2;                       // 16-byte pieces of K (and of V) per thread and step
    static constexpr int kQ = kRowsQ * D * 2;
    static constexpr int kMean = GR * kRowsQ * 32;          // means of Q_g, a step of 16 each
    static constexpr int kOp = kTile * D * 2;               // one operand tile
    static constexpr int kOffs = kTile * 32;                // r of the tile's tokens, a step of 16
    static constexpr int kTab = 3 * GR * kTile * 4;         // K s; V (s, r)
    static constexpr int kStage = 2 * kOp + kOffs + kTab;
    static constexpr int kSmem = kQ + kMean + 2 * kStage;
    static constexpr int kCols = GR * kTile + D <= 128 ? 128 : GR * kTile + D <= 256 ? 256 : 512;
    static constexpr int kCtas = D <= 128 ? 2 : 1;
};

// 16 rows x 32 columns of fp32: lane (g, t) = (lane / 4, lane % 4) holds of each 8-column block
// columns 2t, 2t + 1 of row g (r[4j], r[4j + 1]) and of row g + 8 (r[4j + 2], r[4j + 3])
__device__ __forceinline__ void tmem_ld_frag(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_st_frag(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 16 rows x 32 columns of fp16 in pairs: of each 8-column block row g (r[2j]) and row g + 8 (r[2j + 1])
__device__ __forceinline__ void tmem_st_pairs(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Matrix steps and their commit, issued by the lane with `lead` set: the whole warp comes
// here together, so that the descriptors are warp-uniform values (from a branch that one
// thread takes alone a step and its commit took twice as long).
// D[tmem] (+)= A[smem] B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]; B MN-major
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void commit(uint64_t* bar, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}
__device__ __forceinline__ uint32_t elect() {
    uint32_t r;
    asm volatile("{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n selp.u32 %0, 1, 0, q;\n}\n" : "=r"(r));
    return r;
}

// Operand descriptors: the low word advances with the address, the high word is fixed.
// MN-major tile without swizzle: blocks of 8 tokens x 16 bytes (8 dims); the blocks of
// consecutive tokens lie 128 bytes apart (leading offset), of consecutive dims kTile * 16 (stride).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading) { return (saddr >> 4) | ((leading >> 4) << 16); }
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t stride) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((stride >> 4) | (1u << 14)));
    return d;
}
// whether any of the threads that meet at a barrier wants it
template <int THREADS>
__device__ __forceinline__ bool any_of(int barrier, bool want) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n"
        " selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)want), "r"(barrier), "n"(THREADS)
        : "memory");
    return r != 0;
}
// ... the two warps that share 32 rows
__device__ __forceinline__ bool any_of_rows(int quad, bool want) { return any_of<64>(4 + quad, want); }

// codes of 8 dims less z as fp16 (of K times 2^-10); 4 bits: one word, dims in the order
// 0 4 1 5 2 6 3 7; 8 bits: two words, in order.  0x6400 is 1024: a code below it adds itself,
// a nibble 4 bits up 16 times itself.
template <int BITS, bool K>
__device__ __forceinline__ uint4 codes8(uint32_t w0, uint32_t w1) {
    uint4 r;
    if (BITS == 4) {
        constexpr uint32_t m0 = K ? 0x14001400u : 0x3C003C00u, a0 = K ? 0xBC08BC08u : 0xE408E408u;   // 2^-10 | 1
        constexpr uint32_t m1 = K ? 0x04000400u : 0x2C002C00u, a1 = K ? 0xAC80AC80u : 0xD480D480u;   // 2^-14 | 2^-4
        const uint32_t h = w0 >> 8;
        r.x = hfma2((w0 & 0x000F000Fu) | 0x64006400u, m0, a0);
        r.y = hfma2((w0 & 0x00F000F0u) | 0x64006400u, m1, a1);
        r.z = hfma2((h & 0x000F000Fu) | 0x64006400u, m0, a0);
        r.w = hfma2((h & 0x00F000F0u) | 0x64006400u, m1, a1);
    } else {
        constexpr uint32_t m = K ? 0x14001400u : 0x3C003C00u, a = K ? 0xBC80BC80u : 0xE480E480u;
        r.x = hfma2(__byte_perm(w0, 0x64646464u, 0x4140), m, a);
        r.y = hfma2(__byte_perm(w0, 0x64646464u, 0x4342), m, a);
        r.z = hfma2(__byte_perm(w1, 0x64646464u, 0x4140), m, a);
        r.w = hfma2(__byte_perm(w1, 0x64646464u, 0x4342), m, a);
    }
    return r;
}
// v = hi + lo 2^-k: two fp16 in one word, lo of 2^k times what hi leaves
template <int K>
__device__ __forceinline__ uint32_t split(float v) {
    const __half hi = __float2half_rn(v);
    const __half2 r = __halves2half2(hi, __float2half_rn((v - __half2float(hi)) * (float)(1 << K)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Waits for a phase of a barrier; gives up after `limit` ns or when another thread did.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead, unsigned long long limit) {
    if (mbar_try_wait(bar, parity)) return true;
    unsigned long long t0, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (*dead || now - t0 > limit) {
            *dead = 1;
            return false;
        }
    }
}

template <int BITS, int D>
__global__ void __launch_bounds__(kThreads, Cfg<BITS, D>::kCtas) attn_prefix_kernel(const PrefixP p) {
    using X = Cfg<BITS, D>;
    constexpr int GR = X::GR;
    constexpr float kZ = BITS == 4 ? 8.f : 128.f;
    extern __shared__ __align__(128) char smem[];
    __shared__ uint64_t full[2], freed[2], s_ready, again, drained;
    __shared__ uint32_t taddr_s;
    __shared__ int dead, n_again, next_s[2];
    __shared__ float part_max[2][kRowsQ];
    char *sQ = smem, *sM = smem + X::kQ, *stages = sM + X::kMean;
    const int tid = threadIdx.x, wid = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int h = blockIdx.z, rb = blockIdx.y;
    const int t0 = blockIdx.x * p.tiles_per_split;
    const int all = (p.n_tok - 1) / kTile + 1;
    const int n = min(p.tiles_per_split, all - t0);
    const int r0 = rb * kRowsQ;

    if (wid == 0) {
        tc::tmem_alloc(&taddr_s, X::kCols);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 4);
            mbar_init(&freed[i], 1);
        }
        mbar_init(&s_ready, 1);
        mbar_init(&again, 1);
        mbar_init(&drained, 1);
        fence_mbar_init();
        n_again = 0;
        dead = p.wait_ns == 0;                                 // (limit 0: given up from the start)
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = taddr_s;
    launch_dependents();     // the sequences' own parts do not need this kernel's results

    if (wid < 8) {
        // queries, K-major, 8 dims in the order of the codes; a thread's pieces 16 rows (of D = 128) apart
        constexpr int kC8 = D / 8, kApart = kSoftmax / kC8, kPer = kRowsQ / kApart;
        const int c8 = (tid >> 3) % kC8, rq = (tid & 7) + 8 * (tid / (8 * kC8));
        uint4 v[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int row = r0 + rq + kApart * j;
            v[j] = make_uint4(0, 0, 0, 0);
            if (row < p.rows)
                v[j] = *reinterpret_cast<const uint4*>(p.q + (long long)(row / p.G) * p.ldq +
                                                       (long long)(h * p.G + row % p.G) * D + 8 * c8);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int r = rq + kApart * j;
            const uint4 x = v[j];
            *reinterpret_cast<uint4*>(sQ + (c8 >> 1) * (kRowsQ * 32) + tc::kstep_off(r, (c8 & 1) * 8)) =
                BITS == 4 ? make_uint4(__byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632),
                                       __byte_perm(x.y, x.w, 0x5410), __byte_perm(x.y, x.w, 0x7632))
                          : x;
        }
        // the means' tiles: zero where nothing is written below
        for (int i = tid; i < X::kMean / 16; i += kSoftmax) reinterpret_cast<uint4*>(sM)[i] = make_uint4(0, 0, 0, 0);
        named_bar_sync(2, kSoftmax);
        for (int i = tid; i < kRowsQ * GR; i += kSoftmax) {
            const int r = i % kRowsQ, gr = i / kRowsQ;
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int c8 = gr * 8 + c;
                const uint4 v = *reinterpret_cast<const uint4*>(sQ + (c8 >> 1) * (kRowsQ * 32) + tc::kstep_off(r, (c8 & 1) * 8));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                    s += f.x + f.y;
                }
            }
            // A mean is a multiple of 2^-30 (the queries' step is 2^-24 at least), 2^11 times what its first
            // fp16 leaves one of 2^-19: exact, or within 2^-24 of the mean, however small the queries.
            const uint32_t hl = split<11>(s * (1.f / kGroup));
            *reinterpret_cast<uint2*>(sM + gr * (kRowsQ * 32) + tc::kstep_off(r, 4 * gr)) = make_uint2(hl, hl);
        }
        tc::fence_async_smem();
        named_bar_sync(2, kSoftmax);
    }
    if (wid >= 8) {
        // ---------------------------------------------------------- operands
        if (X::kCtas == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
        const int w = wid - 8;                                 // strip of the tile
        const int spp = p.c.page_tokens / kv::kStrip;
        const int last_strip = (p.n_tok - 1) / kv::kStrip;
        int strip = t0 * (kTile / 16) + w, pg = strip / spp, in_page = strip - pg * spp;
        // the strip's place in the pool; behind the last token, that strip again
        auto page_of = [&]() -> int {
            if (strip > last_strip) {
                strip = last_strip;
                pg = strip / spp;
                in_page = strip - pg * spp;
            }
            return p.pages[pg];
        };
        int id = page_of();
        uint4 rk[X::NP], rv[X::NP];
        uint32_t rs[GR];                                       // (s, b) words: K's, then V's
        auto load = [&]() {
            if (id < 0 || id >= p.c.n_pages) {
                id = 0;
                if (p.status) atomicExch(p.status, EDGE0_EINVAL);
            }
            const char* base = p.c.pages + id * p.c.page_bytes + ((long long)h * spp + in_page) * X::STRIP;
#pragma unroll
            for (int j = 0; j < X::NP; ++j) {
                const int i = j * 32 + lane, c = (i >> 3) % X::CH, tok = (i & 7) + 8 * ((i >> 3) / X::CH);
                const char* src = base + tok * X::R + ((c ^ kv::turn(X::R, tok)) << 4);
                rk[j] = *reinterpret_cast<const uint4*>(src);
                rv[j] = *reinterpret_cast<const uint4*>(src + X::HALF);
            }
#pragma unroll
            for (int j = 0; j < GR; ++j) {
                const int i = j * 32 + lane;                   // word of the strip's 2 x 16 GR
                const bool v = i >= 16 * GR;
                rs[j] = *reinterpret_cast<const uint32_t*>(base + (v ? X::HALF : 0) + 16 * X::R + (i - (v ? 16 * GR : 0)) * 4);
            }
            // the next tile's strip, its page's number under way by then
            strip += kTile / 16;
            in_page += kTile / 16;
            while (in_page >= spp) {
                in_page -= spp;
                ++pg;
            }
            id = page_of();
        };
        auto put = [&](int i) {
            char* stage = stages + (i & 1) * X::kStage;
            char *sK = stage, *sV = stage + X::kOp, *sR = stage + 2 * X::kOp;
            float* tab_k = reinterpret_cast<float*>(sR + X::kOffs);
            float* tab_v = tab_k + GR * kTile;
#pragma unroll
            for (int j = 0; j < X::NP; ++j) {
                const int q = j * 32 + lane, c = (q >> 3) % X::CH, tok = 16 * w + (q & 7) + 8 * ((q >> 3) / X::CH);
                const uint32_t k4[4] = {rk[j].x, rk[j].y, rk[j].z, rk[j].w}, v4[4] = {rv[j].x, rv[j].y, rv[j].z, rv[j].w};
                constexpr int kW = BITS == 4 ? 1 : 2;          // words per 8 dims
#pragma unroll
                for (int x = 0; x < 4 / kW; ++x) {
                    const int c8 = c * (4 / kW) + x;           // 8 dims
                    *reinterpret_cast<uint4*>(sK + (c8 >> 1) * (kTile * 32) + tc::kstep_off(tok, (c8 & 1) * 8)) =
                        codes8<BITS, true>(k4[x * kW], k4[x * kW + kW - 1]);
                    *reinterpret_cast<uint4*>(sV + c8 * (kTile * 16) + tok * 16) =
                        codes8<BITS, false>(v4[x * kW], v4[x * kW + kW - 1]);
                }
            }
            const int left = p.n_tok - (t0 + i) * kTile;
#pragma unroll
            for (int j = 0; j < GR; ++j) {
                const int q = j * 32 + lane, v = q >= 16 * GR ? 1 : 0, e = q - v * 16 * GR;
                const int tok = 16 * w + e / GR, gr = e % GR;
                float2 sb = __half22float2(*reinterpret_cast<const __half2*>(&rs[j]));
                const bool none = tok >= left;
                const bool flat = sb.x == 0.f;                 // a constant group: codes 0
                if (v) {
                    // b = |b| (0 - z + z +- 1)
                    float* at = tab_v + ((tok >> 1) * GR + gr) * 4 + (tok & 1);
                    const float s = flat ? fabsf(sb.y) : sb.x;     // (zeros: no weight, as where there is no token)
                    at[0] = none ? 0.f : s;
                    at[2] = none || s == 0.f ? 0.f : __fdividef(sb.y, s) + kZ;
                } else {
                    // b = 1 (0 - z + b + z)
                    const float off = flat ? sb.y + kZ : __fdividef(sb.y, sb.x) + kZ;
                    tab_k[(tok >> 1) * 2 * GR + 2 * gr + (tok & 1)] = none ? 0.f : (flat ? 1.f : sb.x) * p.k * 1024.f;
                    // (hi, 2^11 lo) of the mean against (off, off / 2^11), then against what these leave
                    const uint32_t a = split<0>(none ? 0.f : off * (kGroup / 1024.f));
                    const uint32_t b = split<0>(none ? 0.f : off * (kGroup / 1024.f / 2048.f));
                    *reinterpret_cast<uint2*>(sR + tc::kstep_off(tok, 4 * gr)) =
                        make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
                }
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[i & 1]);
        };
        load();
        // the offsets' tiles of this warp's tokens in both stages: zero where put() writes nothing
        {
            char* sR = stages + (lane >> 4) * X::kStage + 2 * X::kOp;
            *reinterpret_cast<uint4*>(sR + tc::kstep_off(16 * w + (lane & 15), 0)) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(sR + tc::kstep_off(16 * w + (lane & 15), 8)) = make_uint4(0, 0, 0, 0);
            __syncwarp();
        }
        for (int i = 0; i < n; ++i) {
            if (i >= 2 && !__all_sync(0xffffffffu, wait_bar(&freed[i & 1], ((i >> 1) - 1) & 1, &dead, p.wait_ns))) break;
            put(i);
            if (i + 1 < n) load();
        }
    } else {
        // ----------------------------------------------------------- softmax
        // 128 x 64 + 256 x 88 registers: what the CTA was launched with (384 x 80)
        if (X::kCtas == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 88;\n");
        const int hf = wid >> 2, quad = wid & 3, g = lane >> 2, t = lane & 3;      // 32 tokens, 32 rows
        const uint32_t my = tm + ((uint32_t)(32 * quad) << 16);
        // rows 32 quad + 16 rh + g + 8 k, index 2 rh + k; weight of a score: 2^(S - mu), S in
        // exponent units, mu the running maximum; of a code beside it s / es kUp times that
        float mu[4], l[4], beta[4][GR], es = 0x1p-40f;          // (below any scale: the first one moves it)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            mu[r] = l[r] = 0.f;
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) beta[r][gr] = 0.f;
        }
        const uint32_t a0 = desc_lo(smem_u32(sQ), tc::kLbo), m0 = desc_lo(smem_u32(sM), tc::kLbo);
        const uint32_t st0 = smem_u32(stages);
        auto issue_scores = [&](int i, uint32_t lead) {        // warp 0: the products of tile i
            const uint32_t k0 = st0 + (i & 1) * X::kStage;
            const uint32_t sK = desc_lo(k0, tc::kLbo), sR = desc_lo(k0 + 2 * X::kOp, tc::kLbo);
            if (!__all_sync(0xffffffffu, wait_bar(&full[i & 1], (i >> 1) & 1, &dead, p.wait_ns))) return;
            tc::fence_after_sync();
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
#pragma unroll
                for (int ks = 4 * gr; ks < 4 * gr + 4; ++ks)
                    mma_ss(tm + gr * kTile, desc(a0 + ks * (kRowsQ * 32 / 16), tc::kSbo),
                           desc(sK + ks * (kTile * 32 / 16), tc::kSbo), tc::idesc_f16(kRowsQ, kTile), ks % 4 != 0, lead);
                mma_ss(tm + gr * kTile, desc(m0 + gr * (kRowsQ * 32 / 16), tc::kSbo), desc(sR, tc::kSbo),
                       tc::idesc_f16(kRowsQ, kTile), true, lead);
            }
            commit(&s_ready, lead);
        };
        auto issue_values = [&](int i, bool accumulate, uint32_t lead) {   // warp 0: O_g (+)= P'_g V_g of tile i
            const uint32_t sV = desc_lo(st0 + (i & 1) * X::kStage + X::kOp, 128);
            tc::fence_after_sync();
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    mma_ts(tm + GR * kTile + gr * kGroup, tm + gr * kTile + (kk >> 1) * 32 + (kk & 1) * 8,
                           desc(sV + (gr * (kGroup / 8) * (kTile * 16) + kk * 256) / 16, kTile * 16),
                           tc::idesc_f16(kRowsQ, kGroup) | (1u << 16), accumulate || kk > 0, lead);
        };
        if (wid == 0) issue_scores(0, elect());
        for (int i = 0; i < n; ++i) {
            const char* stage = stages + (i & 1) * X::kStage;
            const float* tab_k = reinterpret_cast<const float*>(stage + 2 * X::kOp + X::kOffs);
            const float* tab_v = tab_k + GR * kTile;
            const float* mk = tab_k + (hf * 16 + t) * 2 * GR;      // this lane's pairs of tokens, 4 apart
            const float* mv = tab_v + (hf * 16 + t) * 4 * GR;
            // (after a wait that gave up the warps go on to where all meet, and leave together)
            (void)(wait_bar(&full[i & 1], (i >> 1) & 1, &dead, p.wait_ns) && wait_bar(&s_ready, i & 1, &dead, p.wait_ns));
            __syncwarp();
            tc::fence_after_sync();
            float most_s = 0.f, least_s = INFINITY;            // (0: no token)
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                const float2 v = *reinterpret_cast<const float2*>(tab_v + (lane * GR + gr) * 4);
                most_s = fmaxf(most_s, fmaxf(v.x, v.y));
                least_s = fminf(least_s, fminf(v.x == 0.f ? INFINITY : v.x, v.y == 0.f ? INFINITY : v.y));
            }
            bool tiny = false;
            f2 S[2][4][2];                                     // [rh][8 tokens][k]: tokens 2t, 2t + 1
            const int left = p.n_tok - (t0 + i) * kTile - hf * 32 - 2 * t;     // of this lane's tokens
            float mx[4];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                f2 s2[4];                                      // a token's scale serves the lane's four rows
#pragma unroll
                for (int j = 0; j < 4; ++j) s2[j] = *reinterpret_cast<const f2*>(mk + j * 8 * GR + 2 * gr);
                uint32_t raw[2][16];
#pragma unroll
                for (int rh = 0; rh < 2; ++rh)
                    tmem_ld_frag(my + ((uint32_t)(16 * rh) << 16) + gr * kTile + hf * 32, raw[rh]);
                tc::tmem_wait_ld();
#pragma unroll
                for (int rh = 0; rh < 2; ++rh)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const f2 v = pk(__uint_as_float(raw[rh][4 * j + 2 * k]), __uint_as_float(raw[rh][4 * j + 2 * k + 1]));
                            S[rh][j][k] = fma2(v, s2[j], gr ? S[rh][j][k] : pk(-mu[2 * rh + k], -mu[2 * rh + k]));
                        }
            }
#pragma unroll
            for (int rh = 0; rh < 2; ++rh) {
                if (left < 26) {                               // tokens behind the last
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float a, b;
                            unpk(S[rh][j][k], a, b);
                            S[rh][j][k] = pk(8 * j < left ? a : -INFINITY, 8 * j + 1 < left ? b : -INFINITY);
                        }
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float a[4], b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) unpk(S[rh][j][k], a[j], b[j]);
                    mx[2 * rh + k] = fmaxf(fmaxf(fmaxf(a[0], b[0]), fmaxf(a[1], b[1])), fmaxf(fmaxf(a[2], b[2]), fmaxf(a[3], b[3])));
                }
            }
            const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (any_of_rows(quad, i == 0 || most > kRise || most_s > es * kHighS || least_s < es * kLowS)) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                    mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
                    if (t == 0) part_max[hf][32 * quad + 16 * (r >> 1) + g + 8 * (r & 1)] = mx[r];
                }
#pragma unroll
                for (int s = 16; s; s >>= 1) most_s = fmaxf(most_s, __shfl_xor_sync(0xffffffffu, most_s, s));
                named_bar_sync(8 + quad, 64);
                float f_s = 1.f;
                if (most_s > es * kHighS) {
                    const uint32_t be = __float_as_uint(most_s) >> 23;        // most_s < 2^(be - 126)
                    const float to = __uint_as_float(((be < 240 ? be : 240) + 1) << 23);
                    f_s = es * reciprocal2(to);
                    es = to;
                }
                tiny = __any_sync(0xffffffffu, least_s < es * kLowS);
                float f[4];
                bool move = f_s != 1.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float both = fmaxf(mx[r], part_max[hf ^ 1][32 * quad + 16 * (r >> 1) + g + 8 * (r & 1)]);
                    const float by = (i == 0 || both > kRise) && both != -INFINITY ? both : 0.f;
                    mu[r] += by;
                    f[r] = i ? ex2(-by) : 0.f;
                    move = move || by != 0.f;
                    l[r] *= f[r];
                    f[r] *= f_s;
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) beta[r][gr] *= f[r];
#pragma unroll
                    for (int j = 0; j < 4; ++j) S[r >> 1][j][r & 1] = add2(S[r >> 1][j][r & 1], pk(-by, -by));
                }
                // (the first tile overwrites the accumulators)
                if (i > 0 && __any_sync(0xffffffffu, move)) {
#pragma unroll 1
                    for (int c = 0; c < D / 64 * 2; ++c) {
                        const int rh = c & 1;
                        uint32_t a[16];
                        const uint32_t at = my + ((uint32_t)(16 * rh) << 16) + GR * kTile + hf * (D / 2) + (c >> 1) * 32;
                        tmem_ld_frag(at, a);
                        tc::tmem_wait_ld();
                        const float f0 = rh ? f[2] : f[0], f1 = rh ? f[3] : f[1];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            a[j] = __float_as_uint(__uint_as_float(a[j]) * (j & 2 ? f1 : f0));
                        tmem_st_frag(at, a);
                    }
                }
            }
#pragma unroll
            for (int rh = 0; rh < 2; ++rh)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    f2 sum = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float a, b;
                        unpk(S[rh][j][k], a, b);
                        S[rh][j][k] = pk(ex2(a), ex2(b));
                        sum = j ? add2(sum, S[rh][j][k]) : S[rh][j][k];
                    }
                    float a, b;
                    unpk(sum, a, b);
                    l[2 * rh + k] += a + b;
                }
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                const float up = kUp * reciprocal2(es);
                ulonglong2 sc[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sc[j] = *reinterpret_cast<const ulonglong2*>(mv + j * 16 * GR + gr * 4);
                    sc[j].x = mul2(sc[j].x, pk(up, up));
                }
#pragma unroll
                for (int rh = 0; rh < 2; ++rh) {
                    uint32_t w[8];
                    f2 acc[2] = {0, 0};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float a, b;
                            unpk(mul2(S[rh][j][k], sc[j].x), a, b);
                            w[2 * j + k] = pack2(a, b);
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[2 * j + k]));
                            acc[k] = j ? fma2(pk(f.x, f.y), sc[j].y, acc[k]) : mul2(pk(f.x, f.y), sc[j].y);
                        }
                    tmem_st_pairs(my + ((uint32_t)(16 * rh) << 16) + gr * kTile + hf * 32, w);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float a, b;
                        unpk(acc[k], a, b);
                        beta[2 * rh + k][gr] += a + b;
                    }
                }
            }
            tmem_wait_st();
            tc::fence_before_sync();
            if (wid == 0) *(volatile int*)&next_s[i & 1] = *(volatile int*)&dead ? kLeave : tiny ? kAgain : 0;
            named_bar_sync(3, kSoftmax);
            // what all warps do, whatever each has seen (a barrier that reduces a flag took 1 us of 68)
            const int next = *(volatile int*)&next_s[i & 1];
            if (next == kLeave) break;
            if (wid == 0) {
                const uint32_t lead = elect();
                issue_values(i, i > 0, lead);
                commit(next ? &again : &freed[i & 1], lead);
                if (!next && i + 1 < n) issue_scores(i + 1, lead);
            }
            __syncwarp();
            if (__builtin_expect(next, 0)) {
                // Weights below fp16's normal range: what the rounding took from them, 2^24 times, on V's codes
                // 2^-24 times (exact as subnormals), in another product; from all weights, in the offsets' sum.
                (void)wait_bar(&again, n_again & 1, &dead, p.wait_ns);     // the weights and codes have been used
                __syncwarp();
                tc::fence_after_sync();
                const float up = kUp * reciprocal2(es);
                auto taken = [](float w) { return w - __half2float(__float2half_rn(w)); };
                auto rest = [&](float w) { return fabsf(w) < 0x1p-14f ? taken(w) * kTwo24 : 0.f; };
#pragma unroll
                for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                    for (int rh = 0; rh < 2; ++rh) {
                        uint32_t w[8];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 v = *reinterpret_cast<const float4*>(mv + j * 16 * GR + gr * 4);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float a, b;
                                unpk(S[rh][j][k], a, b);
                                a *= v.x * up;
                                b *= v.y * up;
                                w[2 * j + k] = pack2(rest(a), rest(b));
                                float& sum = beta[2 * rh + k][gr];
                                sum = fmaf(taken(a), v.z, fmaf(taken(b), v.w, sum));
                            }
                        }
                        tmem_st_pairs(my + ((uint32_t)(16 * rh) << 16) + gr * kTile + hf * 32, w);
                    }
                uint4* codes = reinterpret_cast<uint4*>(stages + (i & 1) * X::kStage + X::kOp);
#pragma unroll 1
                for (int c = tid; c < X::kOp / 16; c += kSoftmax) {
                    uint4 v = codes[c];
                    v.x = hfma2(v.x, 0x00010001u, 0x80008000u);
                    v.y = hfma2(v.y, 0x00010001u, 0x80008000u);
                    v.z = hfma2(v.z, 0x00010001u, 0x80008000u);
                    v.w = hfma2(v.w, 0x00010001u, 0x80008000u);
                    codes[c] = v;
                }
                tc::fence_async_smem();
                tmem_wait_st();
                tc::fence_before_sync();
                if (any_of<kSoftmax>(3, *(volatile int*)&dead)) break;
                if (tid == 0) ++n_again;
                if (wid == 0) {
                    const uint32_t lead = elect();
                    issue_values(i, true, lead);
                    commit(&freed[i & 1], lead);
                    if (i + 1 < n) issue_scores(i + 1, lead);
                }
                __syncwarp();
            }
        }
        const bool ok = !*(volatile int*)&dead && wait_bar(&freed[(n - 1) & 1], ((n - 1) >> 1) & 1, &dead, p.wait_ns);
        // a row's sums: its 4 lanes, then both halves of the tokens (all operands are done with by now)
        float* sums = reinterpret_cast<float*>(smem);          // [hf][1 + GR][row]
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 32 * quad + 16 * (r >> 1) + g + 8 * (r & 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (t == 0) sums[hf * (1 + GR) * kRowsQ + row] = l[r];
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                beta[r][gr] += __shfl_xor_sync(0xffffffffu, beta[r][gr], 1);
                beta[r][gr] += __shfl_xor_sync(0xffffffffu, beta[r][gr], 2);
                if (t == 0) sums[(hf * (1 + GR) + 1 + gr) * kRowsQ + row] = beta[r][gr];
            }
        }
        const long long slot = ((long long)h * p.RB + rb) * p.splits + blockIdx.x;
        if (any_of<kSoftmax>(2, !ok)) {
            // tokens are lacking: a sum of NaN marks the rows, whatever was in the slot before
            if (tid < kRowsQ && r0 + tid < p.rows)
                p.part_ml[slot * kRowsQ + tid] = make_float2(0.f, __int_as_float(0x7fffffff));
        } else {
            tc::fence_after_sync();
            // rows of o in shared memory, 16 bytes apart so that eight of them do not share banks, and
            // from there in one copy each
            constexpr int kLd = D + 4;
            const float down = es * (1.f / kUp);
            float* rows = reinterpret_cast<float*>(smem + 2 * (1 + GR) * kRowsQ * 4);
#pragma unroll
            for (int c = 0; c < D / 64 * 2; ++c) {
                const int rh = c & 1, d0 = hf * (D / 2) + (c >> 1) * 32, gr = d0 / kGroup;
                uint32_t a[16];
                tmem_ld_frag(my + ((uint32_t)(16 * rh) << 16) + GR * kTile + d0, a);
                tc::tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int row = 32 * quad + 16 * rh + g + 8 * k;
                    const float add = sums[(1 + gr) * kRowsQ + row] + sums[(1 + GR + 1 + gr) * kRowsQ + row];
                    float* dst = rows + row * kLd + d0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = (__uint_as_float(a[4 * j + 2 * k]) + add) * down;
                        const float y = (__uint_as_float(a[4 * j + 2 * k + 1]) + add) * down;
                        if (BITS == 4) {                       // columns 2t, 2t + 1 hold dims t, t + 4
                            dst[8 * j + t] = x;
                            dst[8 * j + t + 4] = y;
                        } else {
                            *reinterpret_cast<float2*>(dst + 8 * j + 2 * t) = make_float2(x, y);
                        }
                    }
                }
            }
            tc::fence_async_smem();
            named_bar_sync(8 + quad, 64);                      // both halves of these 32 rows
            if (hf == 0) {
                const int row = 32 * quad + lane;
                if (r0 + row < p.rows)
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(
                                     p.part_o + (slot * kRowsQ + row) * D),
                                 "r"(smem_u32(rows + row * kLd)), "r"(D * 4)
                                 : "memory");
                asm volatile("cp.async.bulk.commit_group;\n" ::: "memory");
            }
            if (hf == 0 && t == 0)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 32 * quad + 16 * (r >> 1) + g + 8 * (r & 1);
                    if (r0 + row < p.rows)
                        p.part_ml[slot * kRowsQ + row] = make_float2(mu[r], sums[row] + sums[(1 + GR) * kRowsQ + row]);
                }
            if (hf == 0) asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (wid == 0) {
        if (dead) {              // matrix steps under way still read shared memory and write the accumulators
            commit(&drained, elect());
            wait_copy(&drained, 0, kDefaultWaitNs);
            if (lane == 0 && p.status) atomicExch(p.status, EDGE0_ETIMEOUT);
        }
        tc::tmem_dealloc(tm, X::kCols);
    }
}

template <int BITS, int D>
int launch(const PrefixP& p, cudaStream_t stream) {
    constexpr int kDevices = 64;
    static int set[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return EDGE0_ECUDA;
    if (!__atomic_load_n(&set[dev], __ATOMIC_ACQUIRE)) {
        if (cudaFuncSetAttribute(attn_prefix_kernel<BITS, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<BITS, D>::kSmem) != cudaSuccess)
            return EDGE0_ECUDA;
        __atomic_store_n(&set[dev], 1, __ATOMIC_RELEASE);
    }
    // (Not launch_early: CTAs that are placed while the kernel before still holds its SMs share SMs
    // that others leave empty; 64 sequences behind 3,100 tokens 39.5 us, so 36.1.)
    attn_prefix_kernel<BITS, D><<<dim3(p.splits, p.RB, p.H), kThreads, Cfg<BITS, D>::kSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? EDGE0_OK : EDGE0_ECUDA;
}

}  // namespace

// Two CTAs per SM overlap tensor steps and softmax, but a share costs a start and a partial
// result: at least kShareTiles steps each while every SM has one.  (17 shares of 3 steps
// against 9 of 6, 64 x 4 query rows per head: 21.3 and 21.2 us, and 2.8 us less to join;
// 9 shares of 15 against 4 of 32, 256 x 8 rows: 44.3 and 55.1 us.)
void prefix_shares(int n_tok, int segs, int D, int sms, int* splits, int* tiles_per_split) {
    constexpr int kShareTiles = 6;
    const int tiles = (n_tok - 1) / kTile + 1;
    int s = tiles / kShareTiles;
    const int most = sms * (D <= 128 ? 2 : 1) / segs, least = sms / segs;
    s = s > most ? most : s < least ? least : s;
    s = s < 1 ? 1 : s > tiles ? tiles : s;
    *tiles_per_split = ceil_div(tiles, s);
    *splits = ceil_div(tiles, *tiles_per_split);
}

int prefix_launch(const PrefixP& p, int bits, int D, cudaStream_t stream) {
    if (bits == 4) {
        if (D == 64) return launch<4, 64>(p, stream);
        if (D == 128) return launch<4, 128>(p, stream);
        return launch<4, 256>(p, stream);
    }
    if (D == 64) return launch<8, 64>(p, stream);
    if (D == 128) return launch<8, 128>(p, stream);
    return launch<8, 256>(p, stream);
}

}  // namespace edge0
