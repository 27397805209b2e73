// Attention of all sequences' queries over the prefix they share, on the
// fifth-generation tensor cores.
//
// One CTA: 128 query rows (sequence, head of one K/V head's group) x a share of the
// prefix, 64 tokens a step.  Per step
//   warps 8-11  turn a strip of codes each into fp16 (code - z, z half the code range: exact)
//               in shared memory, K as K-major, V as MN-major operand tiles, and its scales
//               into fp32 tables; the next step's codes are loaded into registers meanwhile;
//   thread 0    issues S_g = Q_g K_g^T per 64 dims g, and once the weights are there
//               O_g += P'_g V_g; accumulators and P' (over S, which is read by then) in TMEM;
//   warps 0-7   two threads per row, 32 tokens each: S = sum_g s_g S_g + (b_g + z s_g) sum Q_g,
//               running maximum and sum, weights p, P'_g = fp16(p s_g), and
//               sum_j p (b_g + z s_g) in fp32.
// So the scores carry no rounding of K, and each weight is rounded once (to fp16, 2^-11 of
// itself).  o = (O_g + sum p (b_g + z s_g)) / sum p.  The exponents' reference is the
// running maximum plus the exponent of the largest scale so far, so that p s stays within
// fp16's normal range whatever the scales; it moves only when a score exceeds it by
// 2^8 or a scale by 2^6, and the accumulators are then rescaled in TMEM.
// Two CTAs per SM (D <= 128): one's tensor steps run under the other's softmax.
#include "attn.cuh"
#include "tc05.cuh"

namespace edge0 {
namespace {

constexpr int kSoftmax = 256;             // threads of the softmax warps
constexpr int kThreads = kSoftmax + 128;  // and the operand warps
constexpr int kRowsQ = kPrefixRows;
constexpr int kTile = kPrefixTile;

template <int BITS, int D>
struct Cfg {
    static constexpr int R = kv::row_bytes(BITS, D);
    static constexpr int CH = R / 16;
    static constexpr int GR = D / kGroup;
    static constexpr int STRIP = kv::strip_bytes(BITS, D);
    static constexpr int HALF = kv::half_bytes(BITS, D);
    static constexpr int NP = CH / 2;                       // 16-byte pieces of K (and of V) per thread and step
    static constexpr int kQ = kRowsQ * D * 2;
    static constexpr int kOp = kTile * D * 2;               // one operand tile
    static constexpr int kTab = 4 * GR * kTile * 4;         // K s, K c, V s, V c
    static constexpr int kStage = 2 * kOp + kTab;
    static constexpr int kSmem = kQ + 2 * kStage;
    static constexpr int kCols = GR * kTile + D <= 128 ? 128 : GR * kTile + D <= 256 ? 256 : 512;
    static constexpr int kCtas = D <= 128 ? 2 : 1;
};

typedef unsigned long long f2;      // two packed fp32

__device__ __forceinline__ f2 pk(float a, float b) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpk(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// D[tmem] (+)= A[tmem] B[smem]; B MN-major
__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
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
// whether any of the softmax threads wants it
__device__ __forceinline__ bool any_softmax(bool want) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 256, p;\n"
        " selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)want)
        : "memory");
    return r != 0;
}

// codes of 8 dims less z as fp16; 4 bits: one word, dims in the order 0 4 1 5 2 6 3 7;
// 8 bits: two words, in order
template <int BITS>
__device__ __forceinline__ uint4 codes8(uint32_t w0, uint32_t w1) {
    uint4 r;
    if (BITS == 4) {
        const uint32_t h = w0 >> 8;
        r.x = hadd2((w0 & 0x000F000Fu) | 0x64006400u, 0xE408E408u);                  // 1024 + n - 1032
        r.y = hfma2((w0 & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);     // (1024 + 16 n) / 16 - 72
        r.z = hadd2((h & 0x000F000Fu) | 0x64006400u, 0xE408E408u);
        r.w = hfma2((h & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
    } else {
        r.x = hadd2(__byte_perm(w0, 0x64646464u, 0x4140), 0xE480E480u);              // 1024 + n - 1152
        r.y = hadd2(__byte_perm(w0, 0x64646464u, 0x4342), 0xE480E480u);
        r.z = hadd2(__byte_perm(w1, 0x64646464u, 0x4140), 0xE480E480u);
        r.w = hadd2(__byte_perm(w1, 0x64646464u, 0x4342), 0xE480E480u);
    }
    return r;
}

// Waits for a phase of a barrier; gives up after kDefaultWaitNs or when another thread did.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* dead) {
    if (mbar_try_wait(bar, parity)) return true;
    unsigned long long t0, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (;;) {
        if (mbar_try_wait(bar, parity)) return true;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (*dead || now - t0 > kDefaultWaitNs) {
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
    extern __shared__ __align__(1024) char smem[];
    __shared__ uint64_t full[2], freed[2], s_ready;
    __shared__ uint32_t taddr_s;
    __shared__ int dead;
    __shared__ float part_max[2][kRowsQ], part_sum[2][1 + GR][kRowsQ];
    char* sQ = smem;
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31;
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
        fence_mbar_init();
        dead = 0;
    }
    if (wid < 8) {
        // queries, K-major, 8 dims in the order of the codes
        for (int i = tid; i < kRowsQ * (D / 8); i += kSoftmax) {
            const int r = (i & 7) + 8 * (i / (8 * (D / 8))), c8 = (i >> 3) % (D / 8);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r0 + r < p.rows) {
                const int row = r0 + r;
                v = *reinterpret_cast<const uint4*>(p.q + (long long)(row / p.G) * p.ldq +
                                                    (long long)(h * p.G + row % p.G) * D + 8 * c8);
                if (BITS == 4)
                    v = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                   __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
            }
            *reinterpret_cast<uint4*>(sQ + (c8 >> 1) * (kRowsQ * 32) + tc::kstep_off(r, (c8 & 1) * 8)) = v;
        }
        tc::fence_async_smem();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = taddr_s;

    if (wid >= 8) {
        // ---------------------------------------------------------- operands
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
            char* stage = smem + X::kQ + (i & 1) * X::kStage;
            char *sK = stage, *sV = stage + X::kOp;
            float* tab = reinterpret_cast<float*>(stage + 2 * X::kOp);
#pragma unroll
            for (int j = 0; j < X::NP; ++j) {
                const int q = j * 32 + lane, c = (q >> 3) % X::CH, tok = 16 * w + (q & 7) + 8 * ((q >> 3) / X::CH);
                const uint32_t k4[4] = {rk[j].x, rk[j].y, rk[j].z, rk[j].w}, v4[4] = {rv[j].x, rv[j].y, rv[j].z, rv[j].w};
                constexpr int kW = BITS == 4 ? 1 : 2;          // words per 8 dims
#pragma unroll
                for (int x = 0; x < 4 / kW; ++x) {
                    const int c8 = c * (4 / kW) + x;           // 8 dims
                    *reinterpret_cast<uint4*>(sK + (c8 >> 1) * (kTile * 32) + tc::kstep_off(tok, (c8 & 1) * 8)) =
                        codes8<BITS>(k4[x * kW], k4[x * kW + kW - 1]);
                    *reinterpret_cast<uint4*>(sV + c8 * (kTile * 16) + tok * 16) =
                        codes8<BITS>(v4[x * kW], v4[x * kW + kW - 1]);
                }
            }
            const int left = p.n_tok - (t0 + i) * kTile;
#pragma unroll
            for (int j = 0; j < GR; ++j) {
                const int q = j * 32 + lane, v = q >= 16 * GR ? 1 : 0, e = q - v * 16 * GR;
                const int tok = 16 * w + e / GR, gr = e % GR;
                float2 sb = __half22float2(*reinterpret_cast<const __half2*>(&rs[j]));
                if (tok >= left) sb = make_float2(0.f, 0.f);
                tab[(2 * v * GR + gr) * kTile + tok] = sb.x;
                tab[((2 * v + 1) * GR + gr) * kTile + tok] = fmaf(sb.x, kZ, sb.y);
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[i & 1]);
        };
        load();
        for (int i = 0; i < n; ++i) {
            if (i >= 2 && !__all_sync(0xffffffffu, wait_bar(&freed[i & 1], ((i >> 1) - 1) & 1, &dead))) break;
            put(i);
            if (i + 1 < n) load();
        }
    } else {
        // ----------------------------------------------------------- softmax
        const int hf = wid >> 2, quad = wid & 3;               // 32 tokens, 32 rows
        const uint32_t my = tm + ((uint32_t)(32 * quad) << 16);
        const int row = 32 * quad + lane;
        f2 qs[GR];
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int c8 = gr * 8 + c;
                const uint4 v = *reinterpret_cast<const uint4*>(sQ + (c8 >> 1) * (kRowsQ * 32) +
                                                                tc::kstep_off(row, (c8 & 1) * 8));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
                    s += f.x + f.y;
                }
            }
            qs[gr] = pk(s, s);
        }
        // exponent of a score: k S - mu, mu = k m + e; m the running maximum, 2^e the scales'
        float m = -INFINITY, thr = -INFINITY, e = 0.f, thr_s = 0.f, mu = 0.f;
        f2 l2 = 0, beta[GR];
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) beta[gr] = 0;
        const f2 k2 = pk(p.k, p.k);
        auto issue_scores = [&](int i) {                       // thread 0: S = Q K^T of tile i
            const uint32_t sK = desc_lo(smem_u32(smem + X::kQ + (i & 1) * X::kStage), tc::kLbo);
            const uint32_t a0 = desc_lo(smem_u32(sQ), tc::kLbo);
            if (!wait_bar(&full[i & 1], (i >> 1) & 1, &dead)) return;
            tc::fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                tc::mma_f16(tm + (ks / 4) * kTile, desc(a0 + ks * (kRowsQ * 32 / 16), tc::kSbo),
                            desc(sK + ks * (kTile * 32 / 16), tc::kSbo), tc::idesc_f16(kRowsQ, kTile), ks % 4 != 0);
            tc::mma_commit(&s_ready);
        };
        if (tid == 0) issue_scores(0);
        __syncwarp();
        bool ok = true;
        for (int i = 0; i < n; ++i) {
            const char* stage = smem + X::kQ + (i & 1) * X::kStage;
            const float* tab = reinterpret_cast<const float*>(stage + 2 * X::kOp);
            const float* mine = tab + hf * 32;
            // (after a wait that gave up the rest runs through without waiting: the warps
            // meet at barriers in every step)
            ok = wait_bar(&full[i & 1], (i >> 1) & 1, &dead) && wait_bar(&s_ready, i & 1, &dead);
            __syncwarp();
            tc::fence_after_sync();
            // 16 tokens of one group at a time, the next ones under way meanwhile
            f2 S[16];
            uint32_t raw[2][16];
            tmem_ld16(my + hf * 32, raw[0]);
            float top_s = fmaxf(tab[2 * GR * kTile + lane], tab[2 * GR * kTile + lane + 32]);
#pragma unroll
            for (int gr = 1; gr < GR; ++gr)
                top_s = fmaxf(top_s, fmaxf(tab[(2 * GR + gr) * kTile + lane], tab[(2 * GR + gr) * kTile + lane + 32]));
            tc::tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < GR * 2; ++q) {
                const int c = q / GR, gr = q % GR;
                if (q + 1 < GR * 2) tmem_ld16(my + ((q + 1) % GR) * kTile + hf * 32 + ((q + 1) / GR) * 16, raw[(q + 1) & 1]);
                const uint32_t(&a)[16] = raw[q & 1];
                const ulonglong2* ks = reinterpret_cast<const ulonglong2*>(mine + gr * kTile + c * 16);
                const ulonglong2* kc = reinterpret_cast<const ulonglong2*>(mine + (GR + gr) * kTile + c * 16);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const ulonglong2 s4 = ks[j], c4 = kc[j];
                    const f2 x0 = pk(__uint_as_float(a[4 * j]), __uint_as_float(a[4 * j + 1]));
                    const f2 x1 = pk(__uint_as_float(a[4 * j + 2]), __uint_as_float(a[4 * j + 3]));
                    f2& d0 = S[c * 8 + 2 * j];
                    f2& d1 = S[c * 8 + 2 * j + 1];
                    d0 = fma2(x0, s4.x, gr ? fma2(c4.x, qs[gr], d0) : mul2(c4.x, qs[gr]));
                    d1 = fma2(x1, s4.y, gr ? fma2(c4.y, qs[gr], d1) : mul2(c4.y, qs[gr]));
                }
                if (q + 1 < GR * 2) tc::tmem_wait_ld();
            }
            const int left = p.n_tok - (t0 + i) * kTile - hf * 32;
            if (left < 32) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float a, b;
                    unpk(S[j], a, b);
                    S[j] = pk(2 * j < left ? a : -INFINITY, 2 * j + 1 < left ? b : -INFINITY);
                }
            }
            float mx4[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) mx4[j] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                float a, b;
                unpk(S[j], a, b);
                mx4[j & 3] = fmaxf(mx4[j & 3], fmaxf(a, b));
            }
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            // (this barrier also ends every read of S before P' goes over it)
            if (any_softmax(mx > thr || top_s > thr_s)) {
                part_max[hf][row] = mx;
#pragma unroll
                for (int s = 16; s; s >>= 1) top_s = fmaxf(top_s, __shfl_xor_sync(0xffffffffu, top_s, s));
                named_bar_sync(2, kSoftmax);
                const float both = fmaxf(mx, part_max[hf ^ 1][row]);
                if (top_s > thr_s) {
                    const int be = (int)(__float_as_uint(top_s) >> 23);      // top_s < 2^(be - 126)
                    e = (float)((be < 240 ? be : 240) - 126);
                    thr_s = __uint_as_float((unsigned)((int)e + 6 + 127) << 23);
                }
                const bool first = m == -INFINITY;
                if (both > thr) {
                    m = both;
                    thr = m + 8.f / p.k;
                }
                const float to = m == -INFINITY ? 0.f : fmaf(m, p.k, e);
                const float f = first ? 0.f : ex2(mu - to);
                mu = to;
                const f2 ff = pk(f, f);
                l2 = mul2(l2, ff);
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) beta[gr] = mul2(beta[gr], ff);
                // (the first tile overwrites the accumulators)
                if (i > 0 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t a[16];
                        const uint32_t at = my + GR * kTile + hf * (D / 2) + c * 16;
                        tmem_ld16(at, a);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) a[j] = __float_as_uint(__uint_as_float(a[j]) * f);
                        tmem_st16(at, a);
                    }
                }
            }
            const f2 mu2 = pk(-mu, -mu);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                f2 pr[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float a, b;
                    unpk(fma2(S[c * 8 + j], k2, mu2), a, b);
                    pr[j] = pk(ex2(a), ex2(b));
                }
                l2 = add2(l2, add2(add2(add2(pr[0], pr[1]), add2(pr[2], pr[3])), add2(add2(pr[4], pr[5]), add2(pr[6], pr[7]))));
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    const ulonglong2* vs = reinterpret_cast<const ulonglong2*>(mine + (2 * GR + gr) * kTile + c * 16);
                    const ulonglong2* vc = reinterpret_cast<const ulonglong2*>(mine + (3 * GR + gr) * kTile + c * 16);
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const ulonglong2 s4 = vs[j], c4 = vc[j];
                        float a, b;
                        unpk(mul2(pr[2 * j], s4.x), a, b);
                        w[2 * j] = pack2(a, b);
                        unpk(mul2(pr[2 * j + 1], s4.y), a, b);
                        w[2 * j + 1] = pack2(a, b);
                        beta[gr] = fma2(pr[2 * j], c4.x, fma2(pr[2 * j + 1], c4.y, beta[gr]));
                    }
                    tmem_st8(my + gr * kTile + hf * 16 + c * 8, w);
                }
            }
            tmem_wait_st();
            tc::fence_before_sync();
            named_bar_sync(3, kSoftmax);
            if (tid == 0) {
                const uint32_t sV = desc_lo(smem_u32(stage) + X::kOp, 128);
                tc::fence_after_sync();
#pragma unroll
                for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_f16_ta(tm + GR * kTile + gr * kGroup, tm + gr * kTile + kk * 8,
                                   desc(sV + (gr * (kGroup / 8) * (kTile * 16) + kk * 256) / 16, kTile * 16),
                                   tc::idesc_f16(kRowsQ, kGroup) | (1u << 16), i > 0 || kk > 0);
                tc::mma_commit(&freed[i & 1]);
                if (i + 1 < n) issue_scores(i + 1);
            }
            __syncwarp();
        }
        // the two threads of a row add up their sums, each writes half of the dims
        float a, b;
        unpk(l2, a, b);
        part_sum[hf][0][row] = a + b;
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
            unpk(beta[gr], a, b);
            part_sum[hf][1 + gr][row] = a + b;
        }
        ok = wait_bar(&freed[(n - 1) & 1], ((n - 1) >> 1) & 1, &dead) && ok;
        named_bar_sync(2, kSoftmax);
        if (__all_sync(0xffffffffu, ok)) {
            tc::fence_after_sync();
            const long long slot = ((long long)h * p.RB + rb) * p.splits + blockIdx.x;
            float* dst = p.part_o + (slot * kRowsQ + row) * D + hf * (D / 2);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t r[16];
                tmem_ld16(my + GR * kTile + hf * (D / 2) + c * 16, r);
                const int gr = (hf * (D / 2) + c * 16) / kGroup;
                const float add = part_sum[0][1 + gr][row] + part_sum[1][1 + gr][row];
                tc::tmem_wait_ld();
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    // column j of 8 dims holds dim 0 4 1 5 2 6 3 7 (4 bits)
                    const int d = BITS == 4 ? (j & 8) + ((j & 1) << 2) + ((j & 7) >> 1) : j;
                    v[d] = __uint_as_float(r[j]) + add;
                }
                if (r0 + row < p.rows)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        reinterpret_cast<float4*>(dst + c * 16)[j] =
                            make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
            if (hf == 0 && r0 + row < p.rows)
                p.part_ml[slot * kRowsQ + row] =
                    make_float2(m == -INFINITY ? m : mu, part_sum[0][0][row] + part_sum[1][0][row]);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid == 0 && dead && p.status) atomicExch(p.status, EDGE0_ETIMEOUT);
    if (wid == 0) tc::tmem_dealloc(tm, X::kCols);
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
    attn_prefix_kernel<BITS, D><<<dim3(p.splits, p.RB, p.H), kThreads, Cfg<BITS, D>::kSmem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? EDGE0_OK : EDGE0_ECUDA;
}

}  // namespace

void prefix_shares(int n_tok, int segs, int D, int sms, int* splits, int* tiles_per_split) {
    const int tiles = (n_tok - 1) / kTile + 1;
    int s = sms * (D <= 128 ? 2 : 1) / segs;
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
