// Decode attention over the quantised KV cache, one query token per sequence:
//     o = sum_j softmax_j(scale q . k_j) v_j
// over a prefix that all sequences share and over the sequence's own tokens.
//
// Work.  A "segment" is one K/V head of one list of pages with up to 8 NT query rows
// that read it: for a sequence's own pages the head's query group, for the shared
// prefix the groups of all sequences (so its pages are read once per 8 NT rows, not
// once per sequence).  The units (16 US tokens) of all segments in a row are cut
// into equal shares, one per CTA; a segment that falls into several shares leaves
// partial results (running maximum, sum, unnormalised o) that attn_join_kernel adds up
// in the order of the units.  Lengths are read on the device, so the launch does
// not depend on them.
//
// Kernel.  The warps of a CTA take the units of its share in turn, each through its
// own ring of bulk copies (a strip of 16 tokens of one head is one run of bytes).
// Tokens are the M side of m16n8k16 steps and query rows the N side, so a group of
// up to 8 query heads wastes nothing:
//   S^T = K Q^T   codes enter as fp16 subnormals q 2^-24 (exact products, fp32 sums); nibbles
//                 4 bits up come in 16 times as large, into sums of their own that are
//                 taken down in fp32 (Q / 16 in fp16 loses bits below 2^-10; nibbles shifted down
//                 cost 7 % on long contexts); per 64 dims S += s acc + b sum(Q), in fp32:
//                 scores carry no rounding of K or Q;
//   O^T = V'^T P' V = s (q - z + r), z half the code range, r = b / s + z: q - z is
//                 exact in fp16, the weight p s is rounded to fp16 (its only rounding),
//                 and sum p s r, of the rounded weights, is kept in fp32 beside it: the
//                 error is that of a rounded weight on the exact V.  (With sum p (b + s z)
//                 of the unrounded weights it was a sixth larger.)
// Both factors of p s have a reference: the running maximum of the row's scores, and the
// power of two 2^e above the largest V scale so far.  p s / 2^e times 2^7 uses fp16's range
// to its top, so that it is normal down to 2^-21 of the largest.  Where a scale is below 2^-9
// of the reference (a token of large V may have raised it, whatever its own weight; r = b / s
// + z can be large there), sum p s r takes the unrounded weights, and what the rounding took
// from subnormal ones enters in a second product, 2^24 times on codes 2^-24 times: weights
// are then good to 2^-48 of the range.  Scores are formed less their reference from the first
// term on, and e stays out of that sum, so that neither is lost to the other's magnitude.
//
// The floor is the pages' bytes.  Measured: four sequences of 100,003 to 131,072 tokens, 8 K/V
// heads of 128 dims at 4 bits, 112.5 us, 549 MB at 4.9 TB/s, 0.72 of what a copy reaches: what
// bounds it are the instructions that unpack the codes and take care of scales (64 % of the issue
// slots, 61 % of the integer and half-precision pipe); the matrix pipe is a quarter taken.
// Four CTAs of four warps per SM (128 registers each); with three, and query fragments read
// from shared memory, 133 us.  One sequence of 777 tokens 10.5 us: two launches and
// the reads that wait for one another (length, page, codes; shares, sums, parts).
//
// ldmatrix delivers K codes as A fragments and, transposed, V codes with the
// token pairs that the A fragments of V^T want; P^T goes from accumulator to
// B fragment with movmatrix.  A reference moves only when exceeded by 2^4, so most units
// rescale nothing.
#include "attn.cuh"
#include "mma.cuh"
#include "wait.cuh"

namespace edge0 {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxGrid = 152 * 8;
constexpr int kMinShare = kWarps;       // units a CTA takes at least
constexpr int kSegCost = 8;             // what starting and joining a segment costs, in units

struct AttnP {
    kv::View c;
    const __half* q;
    long long ldq;
    int G, H;                // query heads per K/V head, K/V heads
    // segments: n_seq lists of pages; rows of list i of head h: r -> query
    // row (i * q_step + r / G, h G + r % G)
    int n_seq, rows, RB, q_step;
    const int* pages;        // [n_seq][W]
    int W;
    const int* lens;         // [n_seq], or null: every list has n_tok tokens
    int n_tok;
    float k;                 // 2^24 scale log2(e): raw scores to the exponent
    float* part_o;           // [slots][8 NT][D]
    float2* part_ml;         // [slots][8 NT] (reference in exponent units, sum)
    int2* seg;               // [segments] (first slot, slots)
    __half* out;             // set: segments that one CTA has whole are written here
    long long ldo;
    int* status;
    unsigned long long wait_ns;   // limit of a wait for a copy
    bool after_prefix;       // begins while the prefix's kernel runs, which has waited for what came before
};

template <int BITS, int D, int NT>
struct Cfg {
    static constexpr int R = kv::row_bytes(BITS, D);
    static constexpr int CH = R / 16;                 // 16-byte pieces of a row
    static constexpr int GR = D / kGroup;
    static constexpr int CPG = CH / GR;               // pieces of a group
    static constexpr int QW = BITS == 4 ? 4 : 2;      // words of a query fragment per piece
    static constexpr int STRIP = kv::strip_bytes(BITS, D);
    static constexpr int HALF = kv::half_bytes(BITS, D);
    static constexpr int SB = kv::sb_bytes(D);
    static constexpr int US = STRIP <= 2304 ? 2 : 1;  // strips per unit
    static constexpr int STAGES = STRIP * US >= 8000 ? 2 : STRIP * US >= 4300 ? (US == 2 ? 2 : 3) : 4;
    static constexpr int MT = D / 16;
    // shared memory
    static constexpr int kRingBytes = kWarps * STAGES * US * STRIP;
    static constexpr bool kQRegs = NT == 1;           // query fragments stay in registers
    static constexpr int kQ = kQRegs ? 0 : NT * CH * 32 * QW * 4;
    static constexpr int kQsum = kQRegs ? 0 : NT * 8 * GR * 4;
    static constexpr int kRedLd = D + 4;
    static constexpr int kRed = kWarps * 8 * kRedLd * 4;   // the ring's memory, once a segment's copies are used up
    static constexpr int kMl = kWarps * NT * 8 * 8;
    static constexpr int kRing = kRingBytes > kRed ? kRingBytes : kRed;
    static constexpr int kSmem = kRing + kQ + kQsum + kMl + kWarps * STAGES * 8 + 257 * 8 + 256 * 4;
    static constexpr int kMinCtas = NT == 1 && D <= 128 ? 4 : NT == 4 || (D == 256 && NT == 2) ? 2 : 3;
};

__device__ __forceinline__ void copy_strip(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float max_over_rows(float v) {   // the 8 lanes of one t
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float sum_over_rows(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 4);
    v += __shfl_xor_sync(0xffffffffu, v, 8);
    return v + __shfl_xor_sync(0xffffffffu, v, 16);
}

// A fragments of V^T, one 16-dim tile, from two transposed words (tokens 0-7 and 8-15):
// the codes less z as fp16.  4 bits: tile `j` of the piece holds its nibbles 2j, 2j + 1.
template <int BITS>
__device__ __forceinline__ void v_frag(uint32_t x0, uint32_t x1, int j, uint32_t (&A)[4]) {
    if (BITS == 4) {
        if (j) {
            x0 >>= 8;
            x1 >>= 8;
        }
        // 0x6400 is 1024: the nibble adds itself (low) or 16 times itself (high)
        A[0] = hadd2((x0 & 0x000F000Fu) | 0x64006400u, 0xE408E408u);                  // - 1032
        A[1] = hfma2((x0 & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);     // / 16 - 72
        A[2] = hadd2((x1 & 0x000F000Fu) | 0x64006400u, 0xE408E408u);
        A[3] = hfma2((x1 & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);
    } else {
        A[0] = hadd2(__byte_perm(x0, 0x64646464u, 0x4240), 0xE480E480u);              // - 1152
        A[1] = hadd2(__byte_perm(x0, 0x64646464u, 0x4341), 0xE480E480u);
        A[2] = hadd2(__byte_perm(x1, 0x64646464u, 0x4240), 0xE480E480u);
        A[3] = hadd2(__byte_perm(x1, 0x64646464u, 0x4341), 0xE480E480u);
    }
}

// first dim of the pair that a lane holds in rows g and g + 8 of tile mt
template <int BITS>
__device__ __forceinline__ int dim_of(int mt, int g) {
    return BITS == 4 ? 32 * (mt >> 1) + 4 * g + 2 * (mt & 1) : 16 * mt + 2 * g;
}

// (s, b) words of a token, one per group
template <int GR>
__device__ __forceinline__ void load_sb(const char* p, uint32_t (&w)[GR]) {
    if (GR == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if (GR == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x;
        w[GR - 1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x;
        w[1 % GR] = v.y;
        w[2 % GR] = v.z;
        w[3 % GR] = v.w;
    }
}
// two fp16 of a word
__device__ __forceinline__ float2 sb_of(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// B fragment words of one piece of one query row (lane t's dims; zeros where there is no row)
template <int BITS>
__device__ __forceinline__ void q_frag(const __half* src, bool there, uint32_t* w) {
    if (BITS == 4) {
        // even nibbles 0,4 | 2,6, odd ones 1,5 | 3,7
        const uint4 v = there ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
        w[0] = __byte_perm(v.x, v.z, 0x5410);
        w[1] = __byte_perm(v.y, v.w, 0x5410);
        w[2] = __byte_perm(v.x, v.z, 0x7632);
        w[3] = __byte_perm(v.y, v.w, 0x7632);
    } else {
        const uint2 v = there ? *reinterpret_cast<const uint2*>(src) : make_uint2(0, 0);
        w[0] = __byte_perm(v.x, v.y, 0x5410);    // dims 0, 2
        w[1] = __byte_perm(v.x, v.y, 0x7632);    // dims 1, 3
    }
}

template <int BITS, int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, Cfg<BITS, D, NT>::kMinCtas) attn_kernel(const AttnP p) {
    using X = Cfg<BITS, D, NT>;
    constexpr int GR = X::GR, QW = X::QW;
    extern __shared__ __align__(128) char smem[];
    char* ring = smem;
    uint32_t* sq = reinterpret_cast<uint32_t*>(ring + X::kRing);
    float* sqsum = reinterpret_cast<float*>(reinterpret_cast<char*>(sq) + X::kQ);
    float* red = reinterpret_cast<float*>(ring);
    float2* sml = reinterpret_cast<float2*>(reinterpret_cast<char*>(sqsum) + X::kQsum);
    uint64_t* bars = reinterpret_cast<uint64_t*>(reinterpret_cast<char*>(sml) + X::kMl);
    long long* cum = reinterpret_cast<long long*>(bars + kWarps * X::STAGES);
    int* tokens = reinterpret_cast<int*>(cum + 257);
    __shared__ int first_seq;
    __shared__ long long share_s;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, t = lane & 3;
    constexpr int kUnit = 16 * X::US;
    constexpr float kZ = BITS == 4 ? 8.f : 128.f;

    if (!p.after_prefix) wait_predecessor();
    launch_dependents();     // attn_join_kernel, which waits for this kernel's end
    // lengths, and the cost before each list: a scan over at most 256 of them
    const int per_list = p.H * p.RB;
    {
        const long long cap = (long long)p.W * p.c.page_tokens;
        for (int i = tid; i < p.n_seq; i += 32 * kWarps) {
            int n = p.lens ? p.lens[i] : p.n_tok;
            if (n > cap) {
                n = (int)cap;
                if (blockIdx.x == 0 && p.status) atomicExch(p.status, EDGE0_EINVAL);
            }
            tokens[i] = n < 0 ? 0 : n;
        }
        if (tid < kWarps * X::STAGES) mbar_init(&bars[tid], 1);
        fence_mbar_init();
        __syncthreads();
        if (wid == 0) {
            long long part[9], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int n = lane * 8 + j < p.n_seq ? tokens[lane * 8 + j] : 0;
                part[j] = sum;
                sum += n ? (long long)((n - 1) / kUnit + 1 + kSegCost) * per_list : 0;
            }
            part[8] = sum;
            long long upto = sum;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const long long o = __shfl_up_sync(0xffffffffu, upto, s);
                if (lane >= s) upto += o;
            }
            const long long total = __shfl_sync(0xffffffffu, upto, 31), before = upto - sum;
            long long share = total < 0x7fffffff ? ((unsigned)total + gridDim.x - 1) / gridDim.x : (total + gridDim.x - 1) / gridDim.x;
            if (share < kMinShare + kSegCost) share = kMinShare + kSegCost;
            const long long at = share * blockIdx.x - before;    // this CTA's first position, from this lane's lists on
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (lane * 8 + j < p.n_seq) {
                    cum[lane * 8 + j] = before + part[j];
                    if (at >= part[j] && at < part[j + 1]) first_seq = lane * 8 + j;
                }
            if (lane == 31) {
                cum[p.n_seq] = total;
                share_s = share;
            }
        }
        __syncthreads();
    }
    const long long total = cum[p.n_seq], share = share_s;
    long long pos = share * blockIdx.x;
    const long long end = pos + share < total ? pos + share : total;

    char* my_ring = ring + wid * X::STAGES * X::US * X::STRIP;
    uint64_t* my_bar = bars + wid * X::STAGES;
    int it = 0;              // units this warp has taken so far: stage and parity
    bool dead = p.wait_ns == 0;   // a copy did not arrive in time
    if (dead && tid == 0 && p.status) atomicExch(p.status, EDGE0_ETIMEOUT);
    // the lane's row and piece in the 8x8 matrix loads
    const int lr = (lane & 7) + 8 * ((lane >> 3) & 1);
    const uint32_t row_off = lr * X::R;
    const uint32_t piece = ((lane >> 4) ^ kv::turn(X::R, lr)) << 4;
    const int spp = p.c.page_tokens / kv::kStrip;
    // copies per unit: one where a unit's strips always lie in one page
    const int cpu = X::US == 1 || spp % X::US == 0 ? 1 : X::US;

    int seq = pos < total ? first_seq : 0;
    while (pos < end) {
        while (cum[seq + 1] <= pos) ++seq;                       // (lists without tokens take no room)
        const int n_tok = tokens[seq];
        const int units = (n_tok - 1) / kUnit + 1, cost = units + kSegCost;
        const long long in_list = pos - cum[seq];
        const int hr = in_list < 0x7fffffff ? (int)in_list / cost : (int)(in_list / cost);
        const long long seg_at = cum[seq] + (long long)hr * cost;
        const long long first_unit = seg_at + kSegCost;          // where its unit 0 lies
        const int u0 = pos > first_unit ? (int)(pos - first_unit) : 0;
        const int u1 = end - first_unit < units ? (int)(end - first_unit) : units;
        pos = seg_at + cost;
        if (u1 <= u0) continue;                                  // the share ends before its first unit
        const int h = hr / p.RB, rb = hr - h * p.RB;
        const int sidx = (seq * p.H + h) * p.RB + rb;
        const int* pages = p.pages + (long long)seq * p.W;
        const int n_strips = (n_tok - 1) / kv::kStrip + 1;

        // Copies: lane i prepares the address of the warp's i-th copy from here on (32 / cpu
        // units), and the page number of the one 32 copies later.
        const int per_batch = 32 / cpu;
        int batch = dead ? u1 : u0 + wid, in_batch = 0;          // first unit of the batch; units of it issued
        auto strip_at = [&](int unit0) {                         // this lane's strip, behind the last: any valid one
            const int s = (unit0 + kWarps * (lane / cpu)) * X::US + (cpu == 1 ? 0 : lane % cpu);
            return s < n_strips ? s : n_strips - 1;
        };
        auto address = [&](int unit0, int id) -> const char* {
            const int s = strip_at(unit0);
            if (id < 0 || id >= p.c.n_pages) {
                id = 0;
                if (p.status) atomicExch(p.status, EDGE0_EINVAL);
            }
            return p.c.pages + id * p.c.page_bytes + ((long long)h * spp + s % spp) * X::STRIP;
        };
        const char* src = address(batch, pages[strip_at(batch) / spp]);
        int id_later = pages[strip_at(batch + kWarps * per_batch) / spp];
        int issued = it;
        auto issue = [&]() {                                     // the whole warp: the next unit, if there is one
            const int u = batch + kWarps * in_batch;
            if (u >= u1) return;
            const int stage = issued % X::STAGES;
            const int n = min(X::US, n_strips - u * X::US);
            if (lane == in_batch * cpu) mbar_arrive_expect_tx(&my_bar[stage], n * X::STRIP);
            if (cpu == 1) {
                if (lane == in_batch) copy_strip(my_ring + stage * X::US * X::STRIP, src, n * X::STRIP, &my_bar[stage]);
            } else {
                __syncwarp();
                const int s = lane - in_batch * cpu;
                if (s >= 0 && s < n) copy_strip(my_ring + (stage * X::US + s) * X::STRIP, src, X::STRIP, &my_bar[stage]);
            }
            ++issued;
            if (++in_batch == per_batch) {
                in_batch = 0;
                batch += kWarps * per_batch;
                src = address(batch, id_later);
                id_later = pages[strip_at(batch + kWarps * per_batch) / spp];
            }
        };
#pragma unroll 1
        for (int s = 0; s < X::STAGES - 1; ++s) issue();

        // query rows of the block as B fragments; their sums over each 64 dims are
        // matrix steps against ones
        const int r0 = rb * 8 * NT;
        uint32_t qf[X::kQRegs ? X::CH : 1][QW];
        float qs[X::kQRegs ? GR : 1][2];
        const uint32_t ones[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
        auto q_at = [&](int r, int c) {
            return p.q + (long long)(seq * p.q_step + r / p.G) * p.ldq + (long long)(h * p.G + r % p.G) * D +
                   (BITS == 4 ? 32 * c + 8 * t : 16 * c + 4 * t);
        };
        auto sums_of = [&](const uint32_t* f, int gr, float (&sum)[4]) {     // f: fragments of a row block
#pragma unroll
            for (int c = gr * X::CPG; c < (gr + 1) * X::CPG; ++c) {
                const uint32_t* w = f + c * QW;
                if (c == gr * X::CPG) mma_16816_first(sum, ones, w[0], w[1]);
                else mma_16816_v(sum, ones, w[0], w[1]);
                if (BITS == 4) mma_16816_v(sum, ones, w[QW - 2], w[QW - 1]);
            }
        };
        if constexpr (X::kQRegs) {
            const int r = r0 + g;
#pragma unroll
            for (int c = 0; c < X::CH; ++c) q_frag<BITS>(q_at(r < p.rows ? r : 0, c), r < p.rows, qf[c]);
#pragma unroll
            for (int gr = 0; gr < GR; ++gr) {
                float sum[4];
                sums_of(&qf[0][0], gr, sum);
                qs[gr][0] = sum[0] * (1.f / kTwo24);
                qs[gr][1] = sum[1] * (1.f / kTwo24);
            }
        } else {
            for (int nt = wid; nt < NT; nt += kWarps) {
                const int r = r0 + nt * 8 + g;
                uint32_t f[X::CH][QW];
#pragma unroll
                for (int c = 0; c < X::CH; ++c) {
                    q_frag<BITS>(q_at(r < p.rows ? r : 0, c), r < p.rows, f[c]);
#pragma unroll
                    for (int j = 0; j < QW; ++j) sq[((nt * X::CH + c) * 32 + lane) * QW + j] = f[c][j];
                }
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    float sum[4];
                    sums_of(&f[0][0], gr, sum);
                    if (g == 0) {
                        sqsum[(nt * 8 + 2 * t) * GR + gr] = sum[0] * (1.f / kTwo24);
                        sqsum[(nt * 8 + 2 * t + 1) * GR + gr] = sum[1] * (1.f / kTwo24);
                    }
                }
            }
            __syncthreads();
        }

        // Weight of a score S: 2^(k (S - m)), m the row's reference; of a code beside it, s / es 2^kUp
        // times that, es = 2^e the scales' reference.
        float O[X::MT][NT][4], beta[NT][GR][2], m[NT][2], l[NT][2];
        float es = 0x1p-40f, high = -INFINITY;                   // (below any scale: the first one moves it)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < X::MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) O[mt][nt][i] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[nt][i] = l[nt][i] = 0.f;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) beta[nt][gr][i] = 0.f;
            }
        }

#pragma unroll 1
        for (int u = dead ? u1 : u0 + wid; u < u1; u += kWarps, ++it) {
            issue();
            const int stage = it % X::STAGES;
            if (!wait_copy(&my_bar[stage], (it / X::STAGES) & 1, p.wait_ns)) {
                drain_copies_call(my_bar, it, issued, X::STAGES);     // give up: nothing more is issued or read
                if (lane == 0 && p.status) atomicExch(p.status, EDGE0_ETIMEOUT);
                dead = true;
                break;
            }
            const char* buf = my_ring + stage * X::US * X::STRIP;
            const int left = n_tok - u * kUnit < kUnit ? n_tok - u * kUnit : kUnit;   // valid tokens

            // scores of the unit less their references, in raw units
            float S[X::US][NT][4];
#pragma unroll
            for (int st = 0; st < X::US; ++st) {
                const char* kb = buf + st * X::STRIP;
                const uint32_t ka = smem_u32(kb) + row_off;
                uint32_t wa[GR], wb[GR];
                load_sb<GR>(kb + 16 * X::R + g * X::SB, wa);
                load_sb<GR>(kb + 16 * X::R + (g + 8) * X::SB, wb);
                // (a strip behind the last token holds what was there before; it is masked below)
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    float acc[NT][4], odd[NT][4];              // odd: of the nibbles 4 bits up
#pragma unroll
                    for (int cp = 0; cp < X::CPG; cp += 2) {
                        const int c0 = gr * X::CPG + cp;
                        uint32_t w[4];
                        ldsm4(w, ka + (piece ^ (c0 << 4)));
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t x = w[2 * j], y = w[2 * j + 1];
                            constexpr uint32_t kLow = BITS == 4 ? 0x000F000Fu : 0x00FF00FFu;
                            const uint32_t A0[4] = {x & kLow, y & kLow, (x >> 8) & kLow, (y >> 8) & kLow};
                            const uint32_t A1[4] = {x & 0x00F000F0u, y & 0x00F000F0u, (x >> 8) & 0x00F000F0u,
                                                    (y >> 8) & 0x00F000F0u};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                uint32_t f[QW];
                                if constexpr (X::kQRegs) {
#pragma unroll
                                    for (int i = 0; i < QW; ++i) f[i] = qf[c0 + j][i];
                                } else if constexpr (QW == 4) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(sq + ((nt * X::CH + c0 + j) * 32 + lane) * 4);
                                    f[0] = v.x, f[1] = v.y, f[QW - 2] = v.z, f[QW - 1] = v.w;
                                } else {
                                    const uint2 v = *reinterpret_cast<const uint2*>(sq + ((nt * X::CH + c0 + j) * 32 + lane) * 2);
                                    f[0] = v.x, f[1] = v.y;
                                }
                                if (cp + j == 0) mma_16816_first(acc[nt], A0, f[0], f[1]);
                                else mma_16816_v(acc[nt], A0, f[0], f[1]);
                                if (BITS == 4 && cp + j == 0) mma_16816_first(odd[nt], A1, f[QW - 2], f[QW - 1]);
                                else if (BITS == 4) mma_16816_v(odd[nt], A1, f[QW - 2], f[QW - 1]);
                            }
                        }
                    }
                    const float2 sa = sb_of(wa[gr]), sb = sb_of(wb[gr]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (BITS == 4)
#pragma unroll
                            for (int i = 0; i < 4; i += 2)
                                unpk(fma2(pk(odd[nt][i], odd[nt][i + 1]), pk(1.f / 16, 1.f / 16), pk(acc[nt][i], acc[nt][i + 1])),
                                     acc[nt][i], acc[nt][i + 1]);
                        float q0, q1;
                        if constexpr (X::kQRegs) {
                            q0 = qs[gr][0];
                            q1 = qs[gr][1];
                        } else {
                            q0 = sqsum[(nt * 8 + 2 * t) * GR + gr];
                            q1 = sqsum[(nt * 8 + 2 * t + 1) * GR + gr];
                        }
                        float(&s)[4] = S[st][nt];
                        const f2 qq = pk(q0, q1), mm = pk(-m[nt][0], -m[nt][1]);
                        unpk(fma2(pk(sa.x, sa.x), pk(acc[nt][0], acc[nt][1]), fma2(pk(sa.y, sa.y), qq, gr ? pk(s[0], s[1]) : mm)), s[0], s[1]);
                        unpk(fma2(pk(sb.x, sb.x), pk(acc[nt][2], acc[nt][3]), fma2(pk(sb.y, sb.y), qq, gr ? pk(s[2], s[3]) : mm)), s[2], s[3]);
                    }
                }
            }

            // V's scales of the unit's tokens g and g + 8: (s, r).  A token that is not there gets no
            // weight, whatever its bytes.
            float2 vs[X::US][GR][2];
#pragma unroll
            for (int st = 0; st < X::US; ++st)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t w[GR];
                    load_sb<GR>(buf + st * X::STRIP + X::HALF + 16 * X::R + (g + 8 * i) * X::SB, w);
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) {
                        const float2 sb = sb_of(w[gr]);
                        float inv;
                        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(sb.x));
                        vs[st][gr][i] = make_float2(sb.x, fmaf(sb.y, inv, kZ));
                    }
                }
            if (left < kUnit)
#pragma unroll
                for (int st = 0; st < X::US; ++st)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (st * 16 + g + 8 * i >= left) {
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) S[st][nt][2 * i] = S[st][nt][2 * i + 1] = -INFINITY;
#pragma unroll
                            for (int gr = 0; gr < GR; ++gr) vs[st][gr][i] = make_float2(es, kZ);
                        }

            // a score more than 2^kRise above its reference, a scale outside [es kLowS, es kHighS]?
            float most_s = 0.f, least_s = INFINITY;
            bool look = false, tiny = false;
#pragma unroll
            for (int st = 0; st < X::US; ++st)
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    most_s = fmaxf(most_s, fmaxf(vs[st][gr][0].x, vs[st][gr][1].x));
                    least_s = fminf(least_s, fminf(vs[st][gr][0].x, vs[st][gr][1].x));
                }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = fmaxf(S[0][nt][i], S[0][nt][i + 2]);
#pragma unroll
                    for (int st = 1; st < X::US; ++st) v = fmaxf(v, fmaxf(S[st][nt][i], S[st][nt][i + 2]));
                    look = look || v > high;
                }
            if (__any_sync(0xffffffffu, look || most_s > es * kHighS || least_s < es * kLowS)) {
                most_s = 0.f;
                least_s = INFINITY;
#pragma unroll
                for (int st = 0; st < X::US; ++st)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (st * 16 + g + 8 * i < left)
#pragma unroll
                            for (int gr = 0; gr < GR; ++gr) {
                                if (vs[st][gr][i].x == 0.f) {    // a constant group, codes 0: b = |b| (0 - z + z +- 1)
                                    const float b = __half2float(*reinterpret_cast<const __half*>(
                                        buf + st * X::STRIP + X::HALF + 16 * X::R + (g + 8 * i) * X::SB + gr * 4 + 2));
                                    vs[st][gr][i] = make_float2(fabsf(b), b == 0.f ? kZ : kZ + copysignf(1.f, b));
                                }
                                most_s = fmaxf(most_s, vs[st][gr][i].x);
                                if (vs[st][gr][i].x != 0.f) least_s = fminf(least_s, vs[st][gr][i].x);   // (zeros: no weight)
                            }
                most_s = max_over_rows(most_s);
                float f_s = 1.f;
                if (most_s > es * kHighS) {
                    const uint32_t be = __float_as_uint(most_s) >> 23;        // most_s < 2^(be - 126)
                    const float to = __uint_as_float(((be < 240 ? be : 240) + 1) << 23);
                    f_s = es * reciprocal2(to);
                    es = to;
                }
                tiny = __any_sync(0xffffffffu, least_s < es * kLowS);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v = fmaxf(S[0][nt][i], S[0][nt][i + 2]);
#pragma unroll
                        for (int st = 1; st < X::US; ++st) v = fmaxf(v, fmaxf(S[st][nt][i], S[st][nt][i + 2]));
                        v = max_over_rows(v);
                        if (!(v > high)) v = 0.f;      // each row by its own scores alone
                        const float f = high == -INFINITY ? 0.f : ex2(-v * p.k);      // (nothing to move at first)
                        m[nt][i] += v;
#pragma unroll
                        for (int st = 0; st < X::US; ++st) {
                            S[st][nt][i] -= v;
                            S[st][nt][i + 2] -= v;
                        }
                        l[nt][i] *= f;
#pragma unroll
                        for (int gr = 0; gr < GR; ++gr) beta[nt][gr][i] *= f * f_s;
#pragma unroll
                        for (int mt = 0; mt < X::MT; ++mt) {
                            O[mt][nt][i] *= f * f_s;
                            O[mt][nt][i + 2] *= f * f_s;
                        }
                    }
                high = kRise / p.k;
            }
#pragma unroll
            for (int st = 0; st < X::US; ++st)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) S[st][nt][i] = ex2(S[st][nt][i] * p.k);
#pragma unroll
                    for (int i = 0; i < 2; ++i) l[nt][i] += S[st][nt][i] + S[st][nt][i + 2];
                }
            if (__builtin_expect(tiny, 0)) {
                // Weights below fp16's normal range: what the rounding took from them, 2^24 times, on the codes
                // 2^-24 times (exact as subnormals); from all weights, in the offsets' sum.
                const float up = kUp * reciprocal2(es);
                auto taken = [](float w) { return w - __half2float(__float2half_rn(w)); };
                auto rest = [&](float w) { return fabsf(w) < 0x1p-14f ? taken(w) * kTwo24 : 0.f; };
#pragma unroll
                for (int st = 0; st < X::US; ++st) {
                    const uint32_t va = smem_u32(buf + st * X::STRIP + X::HALF) + row_off;
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) {
                        uint32_t b0[NT], b1[NT];
                        const float2 v0 = vs[st][gr][0], v1 = vs[st][gr][1];
                        const float u0 = v0.x * up, u1 = v1.x * up;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const float(&P)[4] = S[st][nt];
                            b0[nt] = transpose8(pack2(rest(P[0] * u0), rest(P[1] * u0)));
                            b1[nt] = transpose8(pack2(rest(P[2] * u1), rest(P[3] * u1)));
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                beta[nt][gr][i] = fmaf(taken(P[i] * u0), v0.y, fmaf(taken(P[i + 2] * u1), v1.y, beta[nt][gr][i]));
                        }
#pragma unroll
                        for (int cp = 0; cp < X::CPG; cp += 2) {
                            const int c0 = gr * X::CPG + cp;
                            uint32_t w[4];
                            ldsm4t(w, va + (piece ^ (c0 << 4)));
#pragma unroll
                            for (int j = 0; j < 2; ++j)
#pragma unroll
                                for (int q = 0; q < (BITS == 4 ? 2 : 1); ++q) {
                                    uint32_t A[4];
                                    v_frag<BITS>(w[2 * j], w[2 * j + 1], q, A);
#pragma unroll
                                    for (int i = 0; i < 4; ++i) A[i] = hfma2(A[i], 0x00010001u, 0x80008000u);
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        mma_16816_v(O[(BITS == 4 ? 2 : 1) * (c0 + j) + q][nt], A, b0[nt], b1[nt]);
                                }
                        }
                    }
                }
            }
#pragma unroll
            for (int st = 0; st < X::US; ++st) {
                const uint32_t va = smem_u32(buf + st * X::STRIP + X::HALF) + row_off;
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) {
                    uint32_t b0[NT], b1[NT];
                    const float2 v0 = vs[st][gr][0], v1 = vs[st][gr][1];
                    const float up = kUp * reciprocal2(es);
                    const float u0 = v0.x * up, u1 = v1.x * up;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float(&P)[4] = S[st][nt];
                        const uint32_t h0 = pack2(P[0] * u0, P[1] * u0), h1 = pack2(P[2] * u1, P[3] * u1);
                        const float2 f0 = sb_of(h0), f1 = sb_of(h1);         // the rounded weights
                        b0[nt] = transpose8(h0);
                        b1[nt] = transpose8(h1);
                        beta[nt][gr][0] = fmaf(f0.x, v0.y, fmaf(f1.x, v1.y, beta[nt][gr][0]));
                        beta[nt][gr][1] = fmaf(f0.y, v0.y, fmaf(f1.y, v1.y, beta[nt][gr][1]));
                    }
#pragma unroll
                    for (int cp = 0; cp < X::CPG; cp += 2) {
                        const int c0 = gr * X::CPG + cp;
                        uint32_t w[4];
                        ldsm4t(w, va + (piece ^ (c0 << 4)));
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int q = 0; q < (BITS == 4 ? 2 : 1); ++q) {
                                uint32_t A[4];
                                v_frag<BITS>(w[2 * j], w[2 * j + 1], q, A);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma_16816_v(O[(BITS == 4 ? 2 : 1) * (c0 + j) + q][nt], A, b0[nt], b1[nt]);
                            }
                    }
                }
            }
            __syncwarp();    // every lane has read the stage before it is copied into again
        }

        // join the warps: maximum, then 8 query rows at a time through the ring's memory
        const bool any = high != -INFINITY;                      // this warp had a unit
        const float down = es * (1.f / kUp);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[nt][i] = sum_over_rows(l[nt][i]);
#pragma unroll
                for (int gr = 0; gr < GR; ++gr) beta[nt][gr][i] = sum_over_rows(beta[nt][gr][i]);
                // (a warp that gave up lacks tokens: NaN marks its rows)
                if (g == 0) sml[(wid * NT + nt) * 8 + 2 * t + i] =
                                dead ? make_float2(0.f, __int_as_float(0x7fffffff))
                                     : make_float2(any ? __fmul_rn(m[nt][i], p.k) : -INFINITY, l[nt][i]);
            }
        __syncthreads();
        const bool whole = u0 == 0 && u1 == units;
        const bool direct = whole && p.out;
        const int slot = blockIdx.x + sidx;
        if (u0 == 0 && tid == 0) {
            const long long last = (first_unit + units - 1) / share;
            p.seg[sidx] = make_int2(slot, (int)(last - blockIdx.x) + 1);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // this warp's share of columns 2t, 2t + 1
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int col = 2 * t + i;
                float top = -INFINITY;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[(w * NT + nt) * 8 + col].x);
                const float f = any ? ex2(__fmul_rn(m[nt][i], p.k) - top) * down : 0.f;   // (not one fused step: `top` is rounded)
                float* dst = red + (wid * 8 + col) * X::kRedLd;
#pragma unroll
                for (int mt = 0; mt < X::MT; ++mt) {
                    const float add = beta[nt][mt / (X::MT / GR)][i];
                    const float2 v = make_float2((O[mt][nt][i] + add) * f, (O[mt][nt][i + 2] + add) * f);
                    *reinterpret_cast<float2*>(dst + dim_of<BITS>(mt, g)) = v;
                }
            }
            __syncthreads();
            for (int i = tid; i < 8 * D / 4; i += 32 * kWarps) {
                const int col = i / (D / 4), d = (i % (D / 4)) * 4;
                const int r = r0 + nt * 8 + col;
                if (r >= p.rows) continue;
                float top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[(w * NT + nt) * 8 + col].x);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 ml = sml[(w * NT + nt) * 8 + col];
                    sum += ml.x == -INFINITY ? 0.f : ml.y * ex2(ml.x - top);
                }
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 a = *reinterpret_cast<const float4*>(red + (w * 8 + col) * X::kRedLd + d);
                    v.x += a.x;
                    v.y += a.y;
                    v.z += a.z;
                    v.w += a.w;
                }
                if (direct) {
                    const float inv = 1.f / sum;
                    const uint2 o = make_uint2(pack2(v.x * inv, v.y * inv), pack2(v.z * inv, v.w * inv));
                    *reinterpret_cast<uint2*>(p.out + (long long)(seq * p.q_step + r / p.G) * p.ldo +
                                              (long long)(h * p.G + r % p.G) * D + d) = o;
                } else {
                    const long long row = (long long)slot * (8 * NT) + nt * 8 + col;
                    *reinterpret_cast<float4*>(p.part_o + row * D + d) = v;
                    if (d == 0) p.part_ml[row] = make_float2(top, sum);
                }
            }
            fence_proxy_async_smem();    // copies of the next segment go where these values are
            __syncthreads();
        }
    }
    // The prefix's kernel may still be running, which this one does not need: its end comes
    // before this kernel's, so that the join finds both parts.
    wait_predecessor();
}

struct JoinP {
    int B, G, H, D;
    const int* lens;
    int n_prefix;
    // own parts and the prefix's parts
    int RB[2], rows[2];      // row blocks per head, rows per block
    const float* part_o[2];
    const float2* part_ml[2];
    const int2* seg[2];
    int splits;              // > 0: the prefix's parts come from attn_prefix_kernel, so many per block
    __half* out;
    long long ldo;
    int n_rows;
};

// A row's parts, (sequence, query head): the prefix's [0, n0), then its own [n0, n).
struct RowParts {
    int n0, n, b, hq;
    const float* o[2];       // prefix's, own; parts step[] rows apart
    const float2* ml[2];
    long long step[2];
    bool done;               // nothing to join: a padding row, or written by the CTA that had it whole

    __device__ RowParts(const JoinP& p, int row, int len, int D) {
        b = row / (p.G * p.H);
        hq = row - b * p.G * p.H;
        const int h = hq / p.G, j = hq - h * p.G;
        int count[2] = {0, 0};
        o[0] = o[1] = nullptr;
        ml[0] = ml[1] = nullptr;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (len < 0 || (w ? p.n_prefix == 0 : len == 0)) continue;
            const int r = w ? b * p.G + j : j;
            const int block = ((w ? 0 : b) * p.H + h) * p.RB[w] + r / p.rows[w];
            const int2 sg = w && p.splits ? make_int2(block * p.splits, p.splits) : p.seg[w][block];
            const long long at = (long long)sg.x * p.rows[w] + r % p.rows[w];
            count[w] = sg.y;
            o[1 - w] = p.part_o[w] + at * D;
            ml[1 - w] = p.part_ml[w] + at;
        }
        n0 = count[1];
        n = n0 + count[0];
        step[0] = p.rows[1];
        step[1] = p.rows[0];
        done = len < 0 || (p.n_prefix == 0 && n == 1);
    }
    __device__ const float* o_of(int s, int D) const { return s < n0 ? o[0] + s * step[0] * D : o[1] + (s - n0) * step[1] * D; }
    __device__ float2 ml_of(int s) const { return s < n0 ? ml[0][s * step[0]] : ml[1][(s - n0) * step[1]]; }
};

// By a warp: the weighted sum of the parts first, first + STRIDE .. (a lane: D / 32 dims), and the
// sum of all parts.  The first parts are on their way before the weights are known.
template <int D, int STRIDE, int BATCH>
__device__ __forceinline__ float join_parts(const RowParts& x, int first, int lane, float (&v)[D / 32]) {
    constexpr int kN = D / 32;
    float part[BATCH][kN];
    auto fetch = [&](int s0) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int s = s0 + STRIDE * u;
            if (s < x.n) {
                const float* src = x.o_of(s, D) + lane * kN;
                if constexpr (kN == 2) {
                    const float2 a = *reinterpret_cast<const float2*>(src);
                    part[u][0] = a.x, part[u][1] = a.y;
                } else {
#pragma unroll
                    for (int e = 0; e < kN; e += 4) {
                        const float4 a = *reinterpret_cast<const float4*>(src + e);
                        part[u][e] = a.x, part[u][e + 1] = a.y, part[u][e + 2] = a.z, part[u][e + 3] = a.w;
                    }
                }
            }
        }
    };
    fetch(first);
    float top = -INFINITY, sum = 0.f;
    for (int s = lane; s < x.n; s += 32) top = fmaxf(top, x.ml_of(s).x);
#pragma unroll
    for (int s = 16; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
    auto weight = [&](float m) { return m == -INFINITY ? 1.f : ex2(m - top); };     // (a part of NaN keeps its NaN)
    for (int s = lane; s < x.n; s += 32) {
        const float2 a = x.ml_of(s);
        sum = fmaf(a.y, weight(a.x), sum);
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int e = 0; e < kN; ++e) v[e] = 0.f;
    for (int s0 = first; s0 < x.n; s0 += STRIDE * BATCH) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int s = s0 + STRIDE * u;
            if (s < x.n) {
                const float f = weight(x.ml_of(s).x);
#pragma unroll
                for (int e = 0; e < kN; ++e) v[e] = fmaf(part[u][e], f, v[e]);
            }
        }
        fetch(s0 + STRIDE * BATCH);
    }
    return sum;
}

// By a CTA of four warps: a row's parts dealt to them in turn.
template <int D>
__device__ __forceinline__ void join_by_cta(const JoinP& p, const RowParts& x, float (&acc)[4][D]) {
    constexpr int kN = D / 32;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    float v[kN];
    const float sum = join_parts<D, 4, 4>(x, wid, lane, v);
#pragma unroll
    for (int e = 0; e < kN; ++e) acc[wid][lane * kN + e] = v[e];
    __syncthreads();
    const float inv = x.n ? 1.f / sum : 0.f;        // no token at all: zeros
    __half* out = p.out + (long long)x.b * p.ldo + (long long)x.hq * D;
    for (int d = 2 * threadIdx.x; d < D; d += 256)
        *reinterpret_cast<uint32_t*>(out + d) =
            pack2(((acc[0][d] + acc[1][d]) + (acc[2][d] + acc[3][d])) * inv,
                  ((acc[0][d + 1] + acc[1][d + 1]) + (acc[2][d + 1] + acc[3][d + 1])) * inv);
}

// Few rows: a CTA each, bound by the latency of a few dependent reads.
template <int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const JoinP p) {
    __shared__ float acc[4][D];
    const int len = p.lens[blockIdx.x / (p.G * p.H)];      // before the wait: see launch.cuh
    wait_predecessor();
    launch_dependents();
    const RowParts x(p, blockIdx.x, len, D);
    if (!x.done) join_by_cta<D>(p, x, acc);
}

// Many rows: a warp each, unless a row has many parts, which its CTA then joins together.
// Against a CTA each, the whole call with about ten parts per row: 4,096 rows 67.6 and 69.5 us,
// 2,048 rows 36.1 and 36.2.
constexpr int kAlone = 24, kManyRows = 1024;
template <int D>
__global__ void __launch_bounds__(128) attn_join_rows_kernel(const JoinP p) {
    constexpr int kN = D / 32;
    __shared__ float acc[4][D];
    __shared__ int many[4];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, row = blockIdx.x * 4 + wid;
    const int len = row < p.n_rows ? p.lens[row / (p.G * p.H)] : -1;      // before the wait: see launch.cuh
    wait_predecessor();
    launch_dependents();
    bool alone = false;
    if (row < p.n_rows) {
        const RowParts x(p, row, len, D);
        alone = x.done || x.n <= kAlone;
        if (!x.done && alone) {
            float v[kN];
            const float sum = join_parts<D, 1, D == 256 ? 4 : 8>(x, 0, lane, v), inv = x.n ? 1.f / sum : 0.f;
            __half* out = p.out + (long long)x.b * p.ldo + (long long)x.hq * D + lane * kN;
            uint32_t h[kN / 2];
#pragma unroll
            for (int e = 0; e < kN / 2; ++e) h[e] = pack2(v[2 * e] * inv, v[2 * e + 1] * inv);
            if constexpr (kN == 2) *reinterpret_cast<uint32_t*>(out) = h[0];
            else if constexpr (kN == 4) *reinterpret_cast<uint2*>(out) = make_uint2(h[0], h[kN / 2 - 1]);
            else *reinterpret_cast<uint4*>(out) = make_uint4(h[0], h[1 % (kN / 2)], h[2 % (kN / 2)], h[3 % (kN / 2)]);
        }
    }
    if (lane == 0) many[wid] = row < p.n_rows && !alone;
    __syncthreads();
    for (int r = 0; r < 4; ++r) {
        if (!many[r]) continue;
        const int row_r = blockIdx.x * 4 + r;
        const RowParts x(p, row_r, p.lens[row_r / (p.G * p.H)], D);
        join_by_cta<D>(p, x, acc);
        __syncthreads();
    }
}

// Query rows that a CTA of one segment takes, 8 NT: the whole group of one sequence
// where it fits 16; of the prefix's rows up to 32 of 64-wide heads (of wider ones the
// accumulators of 32 rows do not fit the registers).
int nt_of(int rows, int D, bool prefix) {
    if (rows <= 8) return 1;
    return rows <= 16 || D != 64 || !prefix ? 2 : 4;
}

// The prefix's rows per K/V head from which the fifth-generation tensor cores take it (a step
// of theirs costs the same for any number of rows up to 128).  Measured on prefixes of 700
// to 16,000 tokens, this file's kernel against theirs, us: D = 128, 16 rows 12-21 and 12-34,
// 32 rows 17-35 and 11-34; D = 64, 32 rows 11-23 and 10-29, 64 rows 12-26 and 10-30, from
// there on theirs hold while this one's grow; D = 256, 32 rows 15-44 and 14-54, 64 rows
// 15-65 and 15-55.
int prefix_from(int D) { return D == 64 ? 65 : D == 128 ? 17 : 33; }
constexpr int kSmsAssumed = 152;      // for the workspace's size; a card with fewer needs less

struct Part {
    int NT, RB, segs, splits, tiles;  // NT == 0: attn_prefix_kernel
    int rows;                         // rows per block
    long long slots, o, ml, seg;      // workspace offsets
};

// workspace: own parts then the prefix's; returns its size
long long layout(int B, int G, int H, int D, int n_prefix, Part (&part)[2]) {
    long long at = 0;
    for (int w = 0; w < 2; ++w) {
        Part& x = part[w];
        const int rows = w ? B * G : G;
        x.NT = w && rows >= prefix_from(D) ? 0 : nt_of(rows, D, w == 1);
        x.rows = x.NT ? 8 * x.NT : kPrefixRows;
        x.RB = ceil_div(rows, x.rows);
        x.segs = (w ? 1 : B) * H * x.RB;
        x.splits = x.tiles = 0;
        if (x.NT == 0) {
            prefix_shares(n_prefix > 0 ? n_prefix : 1, x.segs, D, kSmsAssumed, &x.splits, &x.tiles);
            x.slots = 2 * kSmsAssumed + x.segs;
        } else {
            x.slots = (long long)kMaxGrid + x.segs;
        }
        x.o = at;
        at += x.slots * x.rows * D * 4;
        x.ml = at;
        at += x.slots * x.rows * 8;
        x.seg = at;
        at += ((long long)x.segs * 8 + 15) / 16 * 16;
    }
    return at;
}

template <int BITS, int D, int NT>
int launch(const AttnP& p, long long most_units, cudaStream_t stream) {
    using X = Cfg<BITS, D, NT>;
    constexpr int kDevices = 64;
    static int ctas[kDevices];           // per device: CTAs that fill it, set on the first call
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return EDGE0_ECUDA;
    int n = __atomic_load_n(&ctas[dev], __ATOMIC_ACQUIRE);
    if (n == 0) {
        int sms = 0, occ = 0;
        if (cudaFuncSetAttribute(attn_kernel<BITS, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, X::kSmem) !=
                cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, attn_kernel<BITS, D, NT>, 32 * kWarps, X::kSmem) !=
                cudaSuccess ||
            occ < 1)
            return EDGE0_ECUDA;
        n = sms * occ < kMaxGrid ? sms * occ : kMaxGrid;
        __atomic_store_n(&ctas[dev], n, __ATOMIC_RELEASE);
    }
    const long long want = (most_units + kMinShare + kSegCost - 1) / (kMinShare + kSegCost);
    const int grid = want < n ? (int)(want < 1 ? 1 : want) : n;
    return launch_early(attn_kernel<BITS, D, NT>, dim3(grid), 32 * kWarps, X::kSmem, stream, p);
}

template <int BITS, int D>
int launch_nt(const AttnP& p, int NT, cudaStream_t stream) {
    constexpr int kUnit = 16 * Cfg<BITS, D, 1>::US;
    const long long cap = p.lens ? (long long)p.W * p.c.page_tokens : p.n_tok;
    const long long most = ((cap + kUnit - 1) / kUnit + kSegCost) * p.n_seq * p.H * p.RB;
    if (NT == 1) return launch<BITS, D, 1>(p, most, stream);
    if (NT == 2) return launch<BITS, D, 2>(p, most, stream);
    if constexpr (D == 64) return launch<BITS, D, 4>(p, most, stream);
    return EDGE0_EUNSUPPORTED;
}

int launch_any(const AttnP& p, int bits, int D, int NT, cudaStream_t stream) {
    if (bits == 4) {
        if (D == 64) return launch_nt<4, 64>(p, NT, stream);
        if (D == 128) return launch_nt<4, 128>(p, NT, stream);
        return launch_nt<4, 256>(p, NT, stream);
    }
    if (D == 64) return launch_nt<8, 64>(p, NT, stream);
    if (D == 128) return launch_nt<8, 128>(p, NT, stream);
    return launch_nt<8, 256>(p, NT, stream);
}

template <int D>
int launch_join(const JoinP& j, int rows, cudaStream_t stream) {
    if (rows < kManyRows) return launch_early(attn_join_kernel<D>, dim3(rows), 128, 0, stream, j);
    JoinP many = j;
    many.n_rows = rows;
    return launch_early(attn_join_rows_kernel<D>, dim3(ceil_div(rows, 4)), 128, 0, stream, many);
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" size_t edge0_attn_workspace_bytes(const edge0_kv_cache* cache, int B, int n_q_heads) {
    kv::View c;
    if (kv::view_of(cache, &c) || B <= 0 || B > EDGE0_MAX_BATCHED) return 0;
    if (n_q_heads <= 0 || n_q_heads % c.H || n_q_heads / c.H > EDGE0_MAX_Q_PER_KV) return 0;
    Part part[2];
    return (size_t)layout(B, n_q_heads / c.H, c.H, cache->head_dim, 0, part);
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
    if (n_prefix > EDGE0_MAX_PREFIX) return EDGE0_EUNSUPPORTED;
    if (!(scale > 0.f) || !(scale <= 1e6f)) return EDGE0_EINVAL;
    const int D = cache->head_dim;
    const long long width = (long long)n_q_heads * D;
    if (ldq < width || ldq % 8 || ldo < width || ldo % 8) return EDGE0_EINVAL;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15) return EDGE0_EINVAL;
    if (((uintptr_t)table | (uintptr_t)lens | (uintptr_t)prefix | (uintptr_t)status) & 3) return EDGE0_EINVAL;
    Part part[2];
    p.H = p.c.H;
    p.G = n_q_heads / p.H;
    if ((long long)workspace_bytes < layout(B, p.G, p.H, D, n_prefix, part)) return EDGE0_EINVAL;
    char* ws = (char*)workspace;
    p.q = (const __half*)q;
    p.ldq = ldq;
    p.k = kTwo24 * scale * 1.4426950408889634f;
    p.ldo = ldo;
    p.status = status;
    p.wait_ns = block_wait_limit();
    for (int w = 1; w >= 0; --w) {
        if (w && !n_prefix) continue;
        if (part[w].NT == 0) {
            const PrefixP x{p.c, p.q, ldq, p.G, p.H, B * p.G, part[w].RB, part[w].splits, part[w].tiles, prefix, n_prefix,
                            scale * 1.4426950408889634f, (float*)(ws + part[w].o), (float2*)(ws + part[w].ml), status, p.wait_ns};
            rc = prefix_launch(x, cache->bits, D, stream);
            if (rc) return rc;
            continue;
        }
        p.n_seq = w ? 1 : B;
        p.rows = w ? B * p.G : p.G;
        p.RB = part[w].RB;
        p.q_step = w ? 0 : 1;
        p.pages = w ? prefix : table;
        p.W = w ? ceil_div(n_prefix, p.c.page_tokens) : W;
        p.lens = w ? nullptr : lens;
        p.n_tok = n_prefix;
        p.part_o = (float*)(ws + part[w].o);
        p.part_ml = (float2*)(ws + part[w].ml);
        p.seg = (int2*)(ws + part[w].seg);
        p.out = !w && !n_prefix ? (__half*)out : nullptr;
        p.after_prefix = !w && n_prefix;
        rc = launch_any(p, cache->bits, D, part[w].NT, stream);
        if (rc) return rc;
    }
    JoinP j;
    j.B = B;
    j.G = p.G;
    j.H = p.H;
    j.D = D;
    j.lens = lens;
    j.n_prefix = n_prefix;
    for (int w = 0; w < 2; ++w) {
        j.RB[w] = part[w].RB;
        j.rows[w] = part[w].rows;
        j.part_o[w] = (const float*)(ws + part[w].o);
        j.part_ml[w] = (const float2*)(ws + part[w].ml);
        j.seg[w] = (const int2*)(ws + part[w].seg);
    }
    j.splits = part[1].NT ? 0 : part[1].splits;
    j.out = (__half*)out;
    j.ldo = ldo;
    j.n_rows = 0;
    const int rows = B * n_q_heads;
    if (D == 64) return launch_join<64>(j, rows, stream);
    if (D == 128) return launch_join<128>(j, rows, stream);
    return launch_join<256>(j, rows, stream);
}
