// Attention of drafted tokens over the quantised KV cache: each sequence's rows see its context and,
// of the tokens drafted behind it, those that a mask names (a tree's ancestors) or those up to
// themselves.  Blocks of 128 rows (token, head of the group) and their shares: flash.cuh.
//
// K and V enter the tensor core as exact fp16 operands, code - z (z half the code range), so that the weights' rounding
// to fp16 is the only one beside the result's; an earlier form with the values s q + b themselves as operands
// was off by 4.3e-4 of the outputs' size against 64 bits, this one by 2.9e-4 (plain form: 2.1e-4).  Per group g of 64 dims
//   S = sum_g s_g S_g,       S_g = Q_g (code - z) + 64 mean(Q_g) r_g,   r = (b + z s) / s;
//   o = sum_g P'_g V'_g,     P'_g = fp16(p m_g 2^10),  V' = (code - z) 2^e and r'_g = (b + z s) / m beside it,
// s = m 2^e with m in [1, 2): a weight's place in fp16's range does not depend on V's scales.  The mean's and the offsets'
// products are part of the same matrix steps (one more step of 16 for S, two more columns for o), each factor as
// two fp16 (2^-22).
//
// A step: 64 tokens (32 of 256-wide heads).  Tensor memory holds two buffers of scores (one for 256; weights lie
// over the scores they come from), the accumulators and, up to 128 dims, the queries; with those in shared
// memory a step's products would read them from there each time.
// Warps: 0-7 softmax, fragments of 16 rows, two a lane, so that a token's scales, read from shared memory, serve
// two rows; a block's rows are dealt 16 to a quarter of tensor memory and half of it.  Of more than 64 rows each of two sets
// of four warps has half (both halves a set, steps in turn: four contexts of 131,072 tokens 1,020 us instead of 915); up
// to 64 the sets take the steps in turn, so that one's latencies lie under the other's work, and hand the rows' references on
// from step to step.  Loops over pieces stay rolled: with all of it unrolled a third of the
// stalls were for instructions to arrive.  8 the matrix steps; 9 copies strips' halves (16 tokens of K or of V, one run of
// bytes) into a ring of raw ones; the rest turn those into operands and tables.
//
// What bounds it: neither bytes (15 % of DRAM's cycles) nor the tensor cores (28 % of theirs) but the latencies between
// the roles and their instructions, half of them spent on turning codes into operands: about 2,300 cycles a step of 64
// tokens.  64 sequences of up to 4,000 tokens with up to 16 drafted ones: 157 us; four of up to 131,072 with up to 48: 925
// us, 393 TFLOP/s; one of 777 tokens: 25.6 us.  A block costs nearly the same whatever its rows: chains of 2 and of 8 tokens
// over those four contexts take 386 and 390 us, where a single token's attention takes 112.
// Weights in columns of their own, so that the next scores need not wait for their product, leave no room for the queries, which the
// steps then read from shared memory: 171 and 990 us.
#include "flash.cuh"

namespace edge0 {
namespace {

using namespace flash;

constexpr int kMaxRaw = 40;              // raw entries
constexpr int kExt = 16;                 // columns of V' beside a group's 64 dims
constexpr float kUpV = 1024.f;           // weights are that many times as large: p <= 2^4, m < 2.2

template <int BITS_, int D>
struct Tile {
    // what the shares go by
    static constexpr int kD = D, kBlock = kRowsQ, kTile = D == 256 ? 32 : 64, kEntries = 1, kEntry = kTile, kMinSplit = 8, kMinWhole = 8,
                         kMinShare = 4, kOwn = 4;
    static constexpr int kBufs = D == 256 ? 1 : 2;                   // of scores
    __host__ __device__ static constexpr int lead(int) { return kBufs; }

    static constexpr int BITS = BITS_, GR = D / kGroup, kR = kv::row_bytes(BITS, D), kHalf = kv::half_bytes(BITS, D);
    static constexpr int kUnits = kTile / kv::kStrip;                // raw entries of a tile's K or V
    static constexpr int kCols = kGroup + kExt;
    static constexpr bool kQTmem = D <= 128;
    // Warps that turn codes into operands: six, and ten for twice the bytes of 128 dims in 8 bits (30 sequences of 3,000 tokens
    // 98 us -> 92; 64 dims 76 -> 78, 128 in 4 bits, 64 sequences of up to 4,000, 157 -> 163).  Of 256 dims a warp may not
    // be more than three entries ahead of its own last, or a stage could be two phases behind what the warp waits for.
    static constexpr int kMakers = BITS_ == 8 && D == 128 ? 10 : 6;
    static constexpr int kThreads = kSoftmax + 64 + 32 * kMakers;
    // TMEM columns
    static constexpr int kScores = GR * kTile, kO = kBufs * kScores, kQ = kO + GR * kCols, kAll = kQ + (kQTmem ? D / 2 + 8 * GR : 0);
    static_assert(kAll <= 512, "tensor memory");
    // shared memory: queries and their means (wide heads), K stages [operand | offsets | table], V stages
    // [operand with the extra columns | table], raw entries
    static constexpr int kStages = D == 256 ? 2 : 4;
    static constexpr int kQBytes = kQTmem ? 0 : kRowsQ * D * 2, kMean = kQTmem ? 0 : GR * kRowsQ * 32;
    static constexpr int kTable = GR * kTile * 4;
    static constexpr int kKOffs = kTile * D * 2, kKTab = kKOffs + kTile * 32, kKStage = kKTab + kTable;
    static constexpr int kVTab = GR * kCols * kTile * 2, kVStage = kVTab + kTable;
    static constexpr int kK = kQBytes + kMean, kV = kK + kStages * kKStage, kRaw = kV + kStages * kVStage;
    static constexpr int kControlBytes = 4096;
    static constexpr int kRoom = 232448 - 128 - kControlBytes - kRaw;
    static constexpr int kRaws = kRoom / kHalf < kMaxRaw ? kRoom / kHalf : kMaxRaw;
    static constexpr int kControl = kRaw + kRaws * kHalf, kSmem = kControl + kControlBytes + 128;
    static_assert(kKStage % 128 == 0 && kVStage % 128 == 0 && kHalf % 16 == 0 && kRaws >= 2 * kUnits && kRaws >= kMakers * kUnits / 2, "layout");
};

struct TreeControl {
    uint64_t k_full[4], k_freed[4], v_full[4], v_freed[4];           // stages
    uint64_t raw_full[kMaxRaw], raw_freed[kMaxRaw];
    uint64_t q_full, s_full[2], p_full[2], o_step[2], o_last, drained;      // (pairs: of even and of odd steps)
    uint64_t ref_full[4];                                            // a quarter's references after a step
    Place cut[2];
    uint32_t tmem;
    int dead;
    int issued;           // copies into the raw ring in all, when the warp that issues them has ended
    int special[16];      // numbers of the share's blocks with NaN of V that some rows do not see, by their last bits
    float ref[kRowsQ], sums[2][kRowsQ];
};

struct TreeP {
    Out o;
    kv::View c;
    const __half* q;
    long long ldq;
    int B, H, G, T, W, cap;              // cap: tokens that a row of the table holds
    const int* cu;
    const int* lens;
    const int* table;
    const unsigned* mask;                // [T][words] or null: each row sees the drafted tokens up to itself
    int words;
    int* status;
};

template <class X>
struct Tree : TreeP {
    static constexpr int D = X::kD, BITS = X::BITS;

    __device__ Seq seq(int b) const {
        Seq s;
        s.q0 = min(max(cu[b], 0), T);
        s.n_q = min(max(cu[b + 1], s.q0), T) - s.q0;
        s.k0 = 0;
        const int len = lens[b];
        if (len < 0) s.n_q = 0;                                      // padding
        s.ctx = min(max(len, 0), cap);
        s.n_k = (int)min((long long)s.ctx + s.n_q, (long long)cap);
        s.off = mask ? s.n_k : s.ctx;                                // (with a mask any row may see the last token)
        return s;
    }
    // what the caller is told of: more tokens than the table holds, more drafted ones than the mask names
    __device__ bool over(int b) const {
        const Seq s = seq(b);
        return s.n_q > 0 && ((long long)lens[b] + s.n_q > cap || (mask && s.n_q > 32 * words));
    }
    __device__ int seen(const Seq& s, int token) const { return mask ? s.n_k : min(token + 1 + s.off, s.n_k); }
    __device__ int seen_by_all(const Seq& s, int token) const { return mask ? min(s.ctx, s.n_k) : seen(s, token); }
    // which of the tokens from .. from + 31 a row sees, as bits
    __device__ uint32_t seen_word(const Item& x, int token, int from) const {
        const int k = seen(x.s, token) - from, d = from - x.s.ctx;
        uint32_t v = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1;
        if (mask && d > -32) {
            const unsigned* bits = mask + (long long)(x.s.q0 + token) * words;
            auto word = [&](int i) -> uint32_t { return i < words ? bits[i] : 0u; };
            // drafted tokens d .. d + 31; those below 0 are the context's
            v &= d < 0 ? (word(0) << -d) | ((1u << -d) - 1) : __funnelshift_r(word(d >> 5), word((d >> 5) + 1), d & 31);
        }
        return v;
    }
    // the half strip that a token lies in
    __device__ const char* place(int b, int h, int token, bool value) const {
        const int pg = token / c.page_tokens, in = token - pg * c.page_tokens;
        int id = table[(long long)b * W + pg];
        if (id < 0 || id >= c.n_pages) {
            id = 0;
            if (status) atomicExch(status, EDGE0_EINVAL);
        }
        return c.pages + id * c.page_bytes + ((long long)h * (c.page_tokens / kv::kStrip) + in / kv::kStrip) * kv::strip_bytes(BITS, D) +
               (value ? kv::half_bytes(BITS, D) : 0);
    }
    // groups of V with a NaN among the drafted tokens that a row sees, as bits (they enter the product as zeros)
    __device__ uint32_t nan_groups(const Item& x, int token) const {
        uint32_t v = 0;
        for (int j = max(x.s.ctx, x.lo * X::kTile); j < min(x.s.n_k, x.hi * X::kTile); ++j) {
            if (!(seen_word(x, token, j) & 1)) continue;
            const char* sb = place(x.b, x.h, j, true) + 16 * X::kR + (j % 16) * kv::sb_bytes(D);
            for (int g = 0; g < X::GR; ++g) {
                const __half2 h = reinterpret_cast<const __half2*>(sb)[g];
                if (__hisnan(__low2half(h)) || __hisnan(__high2half(h))) v |= 1u << g;
            }
        }
        return v;
    }
};

// ------------------------------------------------ fragments, matrix steps ----
// 16 rows x 8 N columns of fp32: lane (g, t) = (lane / 4, lane % 4) holds of each 8-column block columns 2t, 2t + 1 of
// row g (r[4j], r[4j + 1]) and of row g + 8 (r[4j + 2], r[4j + 3])
template <int N>
__device__ __forceinline__ void ld_frag(uint32_t a, uint32_t (&r)[4 * N]) {
    static_assert(N == 1 || N == 2 || N == 4, "");
    if constexpr (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                     : EDGE0_R4(r, 0), EDGE0_R4(r, 4), EDGE0_R4(r, 8), EDGE0_R4(r, 12)
                     : "r"(a)
                     : "memory");
    else if constexpr (N == 2)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                     : EDGE0_R4(r, 0), EDGE0_R4(r, 4)
                     : "r"(a)
                     : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];\n" : EDGE0_R4(r, 0) : "r"(a) : "memory");
}
__device__ __forceinline__ void st_frag2(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), EDGE0_I4(r, 0), EDGE0_I4(r, 4)
                 : "memory");
}
// 16 rows x 8 N columns of fp16 in pairs: of each 8-column block row g (r[2j]) and row g + 8 (r[2j + 1])
template <int N>
__device__ __forceinline__ void st_pairs(uint32_t a, const uint32_t (&r)[2 * N]) {
    if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), EDGE0_I4(r, 0), EDGE0_I4(r, 4)
                     : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(a), EDGE0_I4(r, 0) : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(a), EDGE0_I4(r, 0), EDGE0_I4(r, 4)
                 : "memory");
}
// an operand's descriptor without swizzle: 8 x 16-byte blocks, `leading` in the low word and `stride` apart
__device__ __forceinline__ uint64_t desc_plain(uint32_t lo, uint32_t stride) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((stride >> 4) | (1u << 14)));
    return d;
}
// v = hi + lo 2^-k: two fp16 in one word, lo of 2^k times what hi leaves
template <int K>
__device__ __forceinline__ uint32_t split(float v) {
    const __half hi = __float2half_rn(v);
    const __half2 r = __halves2half2(hi, __float2half_rn((v - __half2float(hi)) * (float)(1 << K)));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// ----------------------------------------------------------------- makers ----
// (code - z) 2^e of 8 dims; 4 bits: one word, dims in the order 0 4 1 5 2 6 3 7; 8 bits: two words, in order.  0x6400 is 1024:
// a code below it adds itself, a nibble 4 bits up 16 times itself; m and a: 2^e and -(1024 + z) 2^e, 2^(e-4) and
// -(64 + z) 2^e for such nibbles.
template <int BITS>
__device__ __forceinline__ uint4 codes8(uint32_t w0, uint32_t w1, const uint32_t (&m)[2], const uint32_t (&a)[2]) {
    uint4 r;
    if (BITS == 4) {
        const uint32_t h = w0 >> 8;
        r.x = hfma2((w0 & 0x000F000Fu) | 0x64006400u, m[0], a[0]);
        r.y = hfma2((w0 & 0x00F000F0u) | 0x64006400u, m[1], a[1]);
        r.z = hfma2((h & 0x000F000Fu) | 0x64006400u, m[0], a[0]);
        r.w = hfma2((h & 0x00F000F0u) | 0x64006400u, m[1], a[1]);
    } else {
        r.x = hfma2(__byte_perm(w0, 0x64646464u, 0x4140), m[0], a[0]);
        r.y = hfma2(__byte_perm(w0, 0x64646464u, 0x4342), m[0], a[0]);
        r.z = hfma2(__byte_perm(w1, 0x64646464u, 0x4140), m[0], a[0]);
        r.w = hfma2(__byte_perm(w1, 0x64646464u, 0x4342), m[0], a[0]);
    }
    return r;
}

constexpr int kFastE = 5;                // up to there the one step of codes8 stays within fp16
constexpr uint32_t kZeros = 1u << 31;

// A raw entry (16 tokens, the tile's from row0 on) into operands and tables, by a warp.  Tokens from `left` on come out as
// zeros, and so do V's groups of NaN from `drafted` on, which some rows may not see (true: there were any).
template <class X, bool VALUE>
__device__ __forceinline__ bool make_rows(const char* raw, char* stage, int row0, float c, int left, int drafted) {
    constexpr int BITS = X::BITS, GR = X::GR, CH = X::kR / 16, CPG = CH / GR, T = X::kTile;
    constexpr int kPer = BITS == 4 ? 4 : 2, kW = BITS == 4 ? 1 : 2;  // 8-dim words per piece, 32-bit words of one
    constexpr float kZ = BITS == 4 ? 8.f : 128.f;
    constexpr int kMostE = BITS == 4 ? 12 : 8, kPass = (16 * GR + 31) / 32;
    const int lane = threadIdx.x & 31;
    bool found = false;
    // tables and offsets, a (token, group) per lane; what V's codes need of them stays there: e, or kZeros
    uint32_t kept[kPass];
#pragma unroll
    for (int q = 0; q < kPass; ++q) {
        const int i = q * 32 + lane, tok = i / GR & 15, g = i % GR, row = row0 + tok;
        const float2 sb = __half22float2(*reinterpret_cast<const __half2*>(raw + 16 * X::kR + (tok * GR + g) * 4));
        const bool none = tok >= left, flat = sb.x == 0.f;
        float* table = reinterpret_cast<float*>(stage + (VALUE ? X::kVTab : X::kKTab)) + (row >> 1) * 2 * GR + 2 * g + (row & 1);
        if (!VALUE) {
            // b = 1 (0 - z + b + z) of a constant group; else (b + z s) / s, the sum first: it may be far smaller than b
            const float off = none ? 0.f : flat ? sb.y + kZ : __fdividef(fmaf(kZ, sb.x, sb.y), sb.x);
            // (hi, 2^11 lo) of the mean against (off, off / 2^11), then against what these leave
            const uint32_t a = split<0>(off * (kGroup / 1024.f)), b = split<0>(off * (kGroup / 1024.f / 2048.f));
            if (i < 16 * GR) {
                *table = none ? 0.f : (flat ? 1.f : sb.x) * c * 1024.f;
                *reinterpret_cast<uint2*>(stage + X::kKOffs + tc::kstep_off(row, 4 * g)) =
                    make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
            }
        } else {
            const bool nan = sb.x != sb.x || sb.y != sb.y, out = none || (nan && tok >= drafted);
            found = found || (nan && !none && tok >= drafted && i < 16 * GR);
            // z is 1 less in every other token: codes lie around half a step below half their range, and sums that grow with the
            // context, of codes and offsets apart, would lose to the rounding of the matrix steps' accumulators, which
            // is towards one side (after 25,000 tokens 1e-5 of V's size)
            const float z = kZ - (float)(row & 1);
            const int e = max(-10, min(kMostE, (int)(__float_as_uint(sb.x) >> 23 & 255) - 127));
            const float m = out ? 0.f : nan ? __int_as_float(0x7fffffff) : flat ? 1.f : sb.x * __uint_as_float((uint32_t)(127 - e) << 23);
            const float r = out || nan ? 0.f : flat ? sb.y : __fdividef(fmaf(z, sb.x, sb.y), m);
            kept[q] = out || nan || flat ? kZeros : (uint32_t)(e + 16);
            if (i < 16 * GR) {
                *table = m * kUpV;
                *reinterpret_cast<uint4*>(stage + (g * (X::kCols / 8) + 8) * (T * 16) + row * 16) = make_uint4(split<0>(r), 0, 0, 0);
            }
        }
    }
#pragma unroll 1
    for (int j = 0; j < CH / 2; ++j) {
        const int i = j * 32 + lane, p = (i >> 3) % CH, tok = (i & 7) + 8 * ((i >> 3) / CH), g = p / CPG, row = row0 + tok;
        const uint4 codes = *reinterpret_cast<const uint4*>(raw + tok * X::kR + ((p ^ kv::turn(X::kR, tok)) << 4));
        const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
        uint32_t m[2] = {0x14001400u, 0x04000400u}, a[2] = {BITS == 4 ? 0xBC08BC08u : 0xBC80BC80u, 0xAC80AC80u};     // K: e = -10
        int e = -10;
        if (VALUE) {
            const int from = tok * GR + g;
            uint32_t k = __shfl_sync(0xffffffffu, kept[0], from & 31);
            if (kPass == 2) {
                const uint32_t k1 = __shfl_sync(0xffffffffu, kept[kPass - 1], from & 31);
                k = from >= 32 ? k1 : k;
            }
            e = (int)(k & 31) - 16;
            const uint32_t up = (uint32_t)(min(e, kFastE) << 10) * 0x10001u, less = row & 1;
            m[0] = 0x3C003C00u + up;
            a[0] = (BITS == 4 ? 0xE408E408u : 0xE480E480u) - less * 0x10001u + up;
            m[1] = 0x2C002C00u + up;
            a[1] = 0xD480D480u - less * 0x100010u + up;
            if (k & kZeros) m[0] = m[1] = a[0] = a[1] = 0u;
        }
        // 8-dim words: K's in steps of 16 dims, V's in columns of 8
        const int c8 = p * kPer;
        char* to = stage + (VALUE ? (g * (X::kCols / 8) + (c8 & 7)) * (T * 16) + row * 16 : (c8 >> 1) * (T * 32) + tc::kstep_off(row, 0));
        uint4 v[kPer];
#pragma unroll
        for (int x = 0; x < kPer; ++x) v[x] = codes8<BITS>(w[x * kW], w[x * kW + kW - 1], m, a);
        if (VALUE && __any_sync(0xffffffffu, e > kFastE)) {
            const uint32_t up = (uint32_t)(0x3C00 + (max(e - kFastE, 0) << 10)) * 0x10001u;
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                v[x].x = hfma2(v[x].x, up, 0x80008000u);
                v[x].y = hfma2(v[x].y, up, 0x80008000u);
                v[x].z = hfma2(v[x].z, up, 0x80008000u);
                v[x].w = hfma2(v[x].w, up, 0x80008000u);
            }
        }
#pragma unroll
        for (int x = 0; x < kPer; ++x) *reinterpret_cast<uint4*>(to + (VALUE ? x * (T * 16) : (x & 1) * 128 + (x >> 1) * (T * 32))) = v[x];
    }
    return found;
}

// A block's entries: K of its tiles, X::kBufs of them ahead of V's, then V's that are left.
template <class X>
__device__ __forceinline__ int tile_of_entry(int entry, int n, bool& v) {
    const int lead = min(X::kBufs, n), r = entry - lead, turns = 2 * (n - lead);
    v = r >= 0 && (r >= turns || !(r & 1));
    return r < 0 ? entry : r < turns ? (r >> 1) + (v ? 0 : lead) : r - (n - lead);
}

// ------------------------------------------------- the softmax warps ----
template <class X>
__device__ __forceinline__ void tree_softmax(const Tree<X>& p, TreeControl& c, char* smem) {
    constexpr int D = X::kD, GR = X::GR, T = X::kTile, NB = T / 16;             // 8-token blocks of half a tile
    const int wid = threadIdx.x >> 5, set = wid >> 2, quad = wid & 3, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t tm = c.tmem + ((uint32_t)(32 * quad) << 16);
    const unsigned long long limit = p.o.wait_ns;
    // row 2 rh + k of a lane: fragment row g + 8 k of the quarter's half rh
    auto local_of = [&](int r) { return 64 * (r >> 1) + 16 * quad + g + 8 * (r & 1); };
    Walk<X, Tree<X>> walk(p, c.cut, blockIdx.x);
    Item x;
    int base = 0, blocks = 0, number = 0, links = 0;                 // (links: steps that passed references on)
    // No wait of the warp's has given up so far.  From the first on it does not arrive any more where an arrival counts
    // twice: phases stand still then, and it could be more than the one under way lacks, which is a fault.
    bool alive = true;
    while (walk.next(x)) {
        const int n = x.hi - x.lo;
        const bool both = x.rows > 64;                               // else no row lies in the second half
        bool ok = true;
        if (n > 0) {
            ++number;
            // queries: a thread has a row's dims of some groups
            const int local = 64 * (lane >> 4) + 16 * quad + (lane & 15);
            const bool live = local < x.rows;
            const int at = x.row0 + (live ? local : 0), token = at / p.G, head = x.h * p.G + at - token * p.G;
            const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(x.s.q0 + token) * p.ldq + (long long)head * D);
#pragma unroll 1
            for (int gr = set; gr < GR; gr += 2) {
                uint4 v[8];
                uint32_t w[32];
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = live ? src[8 * gr + i] : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t q4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q4[k]));
                        sum += f.x + f.y;
                    }
                    w[4 * i] = X::BITS == 4 ? __byte_perm(v[i].x, v[i].z, 0x5410) : v[i].x;
                    w[4 * i + 1] = X::BITS == 4 ? __byte_perm(v[i].x, v[i].z, 0x7632) : v[i].y;
                    w[4 * i + 2] = X::BITS == 4 ? __byte_perm(v[i].y, v[i].w, 0x5410) : v[i].z;
                    w[4 * i + 3] = X::BITS == 4 ? __byte_perm(v[i].y, v[i].w, 0x7632) : v[i].w;
                }
                // A mean is a multiple of 2^-30 (the queries' step is 2^-24 at least), 2^11 times what its first fp16 leaves one
                // of 2^-19: exact, or within 2^-24 of the mean, however small the queries.
                const uint32_t hl = split<11>(sum * (1.f / kGroup));
                if constexpr (X::kQTmem) {
                    uint32_t ext[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) ext[i] = i >> 1 == gr ? hl : 0u;
                    tmem_st32(tm + X::kQ + gr * 32, w);
                    tmem_st8(tm + X::kQ + GR * 32 + gr * 8, ext);
                } else {
                    const int row = 32 * quad + lane;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(smem + (4 * gr + (i >> 1)) * (kRowsQ * 32) + tc::kstep_off(row, (i & 1) * 8)) =
                            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                    *reinterpret_cast<uint2*>(smem + X::kQBytes + gr * (kRowsQ * 32) + tc::kstep_off(row, 4 * gr)) = make_uint2(hl, hl);
                }
            }
            if (X::kQTmem) tmem_wait_st();
            else tc::fence_async_smem();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.q_full);
        }
        // of each of its two rows: the reference that the warp has its sum at (exponent units; -infinity while the row has seen
        // nothing, and then 0 in its place), and the sum of its steps
        float ref[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        // Up to 64 rows the sets take the steps in turn, and a warp's arrival counts twice where both sets' are counted; else a
        // set has half the rows.
        const int rh = both ? set : 0, arrivals = both ? 1 : 2;
        auto off = [](float ref) { return ref == -INFINITY ? 0.f : -ref; };
        // takes a sum to the reference that the row has by now
        auto take = [](float& ref, float& l, float now) {
            if (now != ref) {
                l *= ref == -INFINITY ? 0.f : ex2(ref - now);
                ref = now;
            }
        };
        for (int j = both ? 0 : (base + set) & 1; j < n; j += both ? 1 : 2) {
            const int tile = base + j, stage = tile % X::kStages, buf = tile % X::kBufs, tile_at = x.lo + j;
            const uint32_t parity = (tile / X::kStages) & 1;
            const float* mk = reinterpret_cast<const float*>(smem + X::kK + stage * X::kKStage + X::kKTab) + t * 2 * GR;
            const float* mv = reinterpret_cast<const float*>(smem + X::kV + stage * X::kVStage + X::kVTab) + t * 2 * GR;
            // (after a wait that gave up the warp goes on with what is there; the rows are marked in the end)
            ok = wait_alone(&c.k_full[stage], parity, c.dead, limit) && ok;
            ok = wait_alone(&c.s_full[tile & 1], (tile >> 1) & 1, c.dead, limit) && ok;
            __syncwarp();
            tc::fence_after_sync();
            const uint32_t s_at = tm + ((uint32_t)(16 * rh) << 16) + buf * X::kScores;
            // what the sums begin with: less the reference, but where that is far (flash.cuh), when it comes off the rounded sum
            const float start[2] = {is_far(ref[0]) ? 0.f : off(ref[0]), is_far(ref[1]) ? 0.f : off(ref[1])};
            f2 S[2 * NB][2];                                     // [8 tokens][k]: tokens 2t, 2t + 1
            {
                uint32_t raw[GR][2][4 * NB];
#pragma unroll
                for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                    for (int h = 0; h < 2; ++h) ld_frag<NB>(s_at + gr * T + h * (T / 2), raw[gr][h]);
                tc::tmem_wait_ld();
                const f2 from[2] = {pk(start[0], start[0]), pk(start[1], start[1])};
#pragma unroll
                for (int b = 0; b < 2 * NB; ++b)
#pragma unroll
                    for (int gr = 0; gr < GR; ++gr) {
                        const f2 s2 = *reinterpret_cast<const f2*>(mk + b * 8 * GR + 2 * gr);
                        const uint32_t* v = &raw[gr][b / NB][4 * (b % NB)];
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            S[b][k] = fma2(pk(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), s2, gr ? S[b][k] : from[k]);
                    }
            }
            __syncwarp();
            alive = alive && ok;
            if (lane == 0 && alive) mbar_arrive_n(&c.k_freed[stage], arrivals);
            if (tile_at >= x.clear) {
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    const int local = 64 * rh + 16 * quad + g + 8 * k;
                    uint32_t seen[2] = {0, 0};
                    if (local < x.rows) {
                        const int token = (x.row0 + local) / p.G;
                        seen[0] = p.seen_word(x, token, tile_at * T) >> (2 * t);
                        seen[1] = p.seen_word(x, token, tile_at * T + T / 2) >> (2 * t);
                    }
#pragma unroll
                    for (int b = 0; b < 2 * NB; ++b) {
                        float u, v;
                        const uint32_t bits = seen[b / NB] >> (8 * (b % NB));
                        unpk(k ? S[b][1] : S[b][0], u, v);
                        const f2 to = pk(bits & 1 ? u : -INFINITY, bits & 2 ? v : -INFINITY);
                        S[b][0] = k ? S[b][0] : to;
                        S[b][1] = k ? to : S[b][1];
                    }
                }
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int b = 0; b < 2 * NB; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float u, v;
                    unpk(S[b][k], u, v);
                    mx[k] = fmaxf(mx[k], fmaxf(u, v));
                }
            // the references after the step before: its own, or the other set's (a block's first step starts afresh)
            if (!both) {
                ok = wait_alone(&c.ref_full[quad], (links + j + 1) & 1, c.dead, limit) && ok;
                __syncwarp();
            }
            float* at = c.ref + 16 * quad + g;
            float now[2], by[2];
            bool want = false;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                now[k] = both ? ref[k] : j ? at[8 * k] : -INFINITY;
                by[k] = off(now[k]) - start[k];                  // what these scores lack
                want = want || mx[k] + by[k] > (now[k] == -INFINITY ? -INFINITY : kRise);
            }
            float f[2] = {1.f, 1.f};
            bool move = false;
            if (__any_sync(0xffffffffu, want)) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 1));
                    mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], 2));
                    const bool fresh = now[k] == -INFINITY;
                    const float rise = mx[k] + by[k];
                    if (rise > (fresh ? -INFINITY : kRise)) {
                        f[k] = fresh ? 0.f : ex2(-rise);
                        now[k] = mx[k] - start[k];
                        by[k] = is_far(now[k]) ? -mx[k] : off(now[k]) - start[k];      // (the largest score becomes zero)
                        move = true;
                    }
                }
            }
            if (!both) {
                if ((move || j == 0) && t == 0) {
                    at[0] = now[0];
                    at[8] = now[1];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.ref_full[quad]);
            }
            if (__any_sync(0xffffffffu, by[0] != 0.f || by[1] != 0.f || now[0] != ref[0] || now[1] != ref[1])) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    take(ref[k], l[k], now[k]);
#pragma unroll
                    for (int b = 0; b < 2 * NB; ++b) S[b][k] = add2(S[b][k], pk(by[k], by[k]));
                }
                // (the block's first tile overwrites the accumulators)
                if (j > 0 && __any_sync(0xffffffffu, move)) {
                    if (X::kBufs == 2) {    // (one buffer: the product was over before these scores were formed)
                        ok = wait_alone(&c.o_step[(tile - 1) & 1], ((tile - 1) >> 1) & 1, c.dead, limit) && ok;
                        __syncwarp();
                        tc::fence_after_sync();
                    }
#pragma unroll 1
                    for (int q = 0; q < GR * (X::kCols / 16); ++q) {
                        uint32_t a[8];
                        const uint32_t o_at = tm + ((uint32_t)(16 * rh) << 16) + X::kO + 16 * q;
                        ld_frag<2>(o_at, a);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) a[i] = __float_as_uint(__uint_as_float(a[i]) * (i & 2 ? f[1] : f[0]));
                        st_frag2(o_at, a);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f2 sum = 0;
#pragma unroll
                for (int b = 0; b < 2 * NB; ++b) {
                    float u, v;
                    unpk(S[b][k], u, v);
                    S[b][k] = pk(ex2(u), ex2(v));
                    sum = b ? add2(sum, S[b][k]) : S[b][k];
                }
                float u, v;
                unpk(sum, u, v);
                l[k] += u + v;
            }
            ok = wait_alone(&c.v_full[stage], parity, c.dead, limit) && ok;
            __syncwarp();
#pragma unroll
            for (int gr = 0; gr < GR; ++gr)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[2 * NB];
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        const f2 m2 = *reinterpret_cast<const f2*>(mv + (h * NB + b) * 8 * GR + 2 * gr);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float u, v;
                            unpk(mul2(S[h * NB + b][k], m2), u, v);
                            w[2 * b + k] = pack2(u, v);
                        }
                    }
                    st_pairs<NB>(s_at + gr * T + h * (T / 2), w);
                }
            tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            alive = alive && ok;
            if (lane == 0 && alive) mbar_arrive_n(&c.p_full[tile & 1], arrivals);
        }
        base += n;
        float refs[4], sums[4];                                      // of the lane's rows of both halves
        uint32_t nans[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            refs[r] = -INFINITY;
            sums[r] = 0.f;
        }
        if (n > 0) {
            if (!both) {
                links += n;
                ok = wait_alone(&c.ref_full[quad], (links + 1) & 1, c.dead, limit) && ok;
            }
            ok = wait_alone(&c.o_last, blocks++ & 1, c.dead, limit) && ok;
            __syncwarp();
            tc::fence_after_sync();
            const bool special = *(volatile int*)&c.special[number & 15] == number;
            // (once a wait has run out phases stand still, and a later one may look like one gone by)
            ok = ok && !*(volatile int*)&c.dead;
            // a row's sum at its last reference: its 4 lanes, then both sets' steps
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int local = local_of(2 * rh + k);
                if (!both) take(ref[k], l[k], c.ref[local]);
                l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
                l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
                if (!ok) l[k] = __int_as_float(0x7fffffff);
                if (t == 0) {
                    c.sums[both ? 0 : set][local] = l[k];
                    if (both) c.ref[local] = ref[k];
                }
            }
            named_bar_sync(8 + quad, 64);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int local = local_of(r);
                if (r >= 2 && !both) continue;
                refs[r] = c.ref[local];
                sums[r] = both ? c.sums[0][local] : c.sums[0][local] + c.sums[1][local];
                if (special && local < x.rows) nans[r] = p.nan_groups(x, (x.row0 + local) / p.G);
            }
        }
        const bool whole = x.part < 0;
        // a row's place and factor
        __half* out[4];
        float* part[4];
        float by[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int local = local_of(r), at = x.row0 + min(local, x.rows - 1), token = at / p.G, head = x.h * p.G + at - token * p.G;
            out[r] = local < x.rows && whole ? p.o.out + (long long)(x.s.q0 + token) * p.o.ldo + (long long)head * D : nullptr;
            part[r] = local < x.rows && !whole ? p.o.part_o + ((long long)x.part * X::kBlock + local) * D : nullptr;
            by[r] = whole ? (sums[r] == 0.f ? 0.f : 1.f / (sums[r] * kUpV)) : 1.f / kUpV;
            if (sums[r] != sums[r]) by[r] = sums[r];
            if (part[r] && set == 0 && t == 0) p.o.part_ml[(long long)x.part * X::kBlock + local] = make_float2(refs[r], sums[r]);
        }
#pragma unroll 1
        for (int q = set; q < D / 32; q += 2) {
            const int gr = q >> 1;
#pragma unroll
            for (int rh = 0; rh < 2; ++rh) {
                if (rh && !both) continue;
                uint32_t a[16], ext[4];
                float add[2] = {0.f, 0.f};
                if (n > 0) {
                    const uint32_t o_at = tm + ((uint32_t)(16 * rh) << 16) + X::kO + gr * X::kCols;
                    ld_frag<4>(o_at + (q & 1) * 32, a);
                    ld_frag<1>(o_at + kGroup, ext);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        add[k] = __shfl_sync(0xffffffffu, __uint_as_float(ext[2 * k]) + __uint_as_float(ext[2 * k + 1]), lane & 28);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) a[i] = 0u;
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = 2 * rh + k;
                    const float f = (nans[r] >> gr) & 1 ? __int_as_float(0x7fffffff) : by[r];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const float u = (__uint_as_float(a[4 * b + 2 * k]) + add[k]) * f, v = (__uint_as_float(a[4 * b + 2 * k + 1]) + add[k]) * f;
                        if (X::BITS == 4) {                          // columns 2t, 2t + 1 hold dims t, t + 4
                            if (out[r]) {
                                out[r][32 * q + 8 * b + t] = __float2half_rn(u);
                                out[r][32 * q + 8 * b + t + 4] = __float2half_rn(v);
                            } else if (part[r]) {
                                part[r][32 * q + 8 * b + t] = u;
                                part[r][32 * q + 8 * b + t + 4] = v;
                            }
                        } else if (out[r]) {
                            *reinterpret_cast<uint32_t*>(out[r] + 32 * q + 8 * b + 2 * t) = pack2(u, v);
                        } else if (part[r]) {
                            *reinterpret_cast<float2*>(part[r] + 32 * q + 8 * b + 2 * t) = make_float2(u, v);
                        }
                    }
                }
            }
        }
        tc::fence_before_sync();
    }
}

// -------------------------------------------------------- the matrix warp ----
template <class X>
__device__ __forceinline__ void tree_matrix(const Tree<X>& p, TreeControl& c, char* smem) {
    constexpr int GR = X::GR, T = X::kTile;
    const uint32_t tm = c.tmem, lead_lane = elect();
    const uint32_t k0 = smem_u32(smem + X::kK), v0 = smem_u32(smem + X::kV), q0 = smem_u32(smem);
    const unsigned long long limit = p.o.wait_ns;
    Walk<X, Tree<X>> walk(p, c.cut, blockIdx.x);
    Item x;
    int base = 0, blocks = 0;
    auto scores = [&](int tile) {
        const int stage = tile % X::kStages, buf = tile % X::kBufs;
        if (!wait_phase(&c.k_full[stage], (tile / X::kStages) & 1, c.dead, limit)) return;
        tc::fence_after_sync();
        const uint32_t b = desc_lo(k0 + stage * X::kKStage, tc::kLbo), offs = desc_lo(k0 + stage * X::kKStage + X::kKOffs, tc::kLbo);
#pragma unroll
        for (int gr = 0; gr < GR; ++gr) {
            const uint32_t d = tm + buf * X::kScores + gr * T;
#pragma unroll
            for (int ks = 0; ks < 5; ++ks) {                         // four of the dims, one of the mean
                const uint64_t bd = desc_plain(ks < 4 ? b + (4 * gr + ks) * (T * 32 / 16) : offs, tc::kSbo);
                if constexpr (X::kQTmem)
                    mma_ts(d, tm + X::kQ + (ks < 4 ? gr * 32 + 8 * ks : GR * 32 + gr * 8), bd, tc::idesc_f16(kRowsQ, T), ks > 0, lead_lane);
                else
                    mma_ss(d, tc::smem_desc(q0 + (ks < 4 ? (4 * gr + ks) * (kRowsQ * 32) : X::kQBytes + gr * (kRowsQ * 32))), bd,
                           tc::idesc_f16(kRowsQ, T), ks > 0, lead_lane);
            }
        }
        commit(&c.k_freed[stage], lead_lane);
        commit(&c.s_full[tile & 1], lead_lane);
    };
    auto values = [&](int tile, bool first, bool last) {
        const int stage = tile % X::kStages, buf = tile % X::kBufs;
        if (!wait_phase(&c.p_full[tile & 1], (tile >> 1) & 1, c.dead, limit)) return;
        if (!wait_phase(&c.v_full[stage], (tile / X::kStages) & 1, c.dead, limit)) return;
        tc::fence_after_sync();
        const uint32_t b = desc_lo(v0 + stage * X::kVStage, 128);
#pragma unroll
        for (int gr = 0; gr < GR; ++gr)
#pragma unroll
            for (int kk = 0; kk < T / 16; ++kk)
                mma_ts(tm + X::kO + gr * X::kCols, tm + buf * X::kScores + gr * T + (kk / (T / 32)) * (T / 2) + (kk % (T / 32)) * 8,
                       desc_plain(b + (gr * X::kCols * T * 2 + kk * 256) / 16, T * 16), tc::idesc_f16(kRowsQ, X::kCols) | (1u << 16),
                       !first || kk > 0, lead_lane);
        commit(&c.v_freed[stage], lead_lane);
        commit(&c.o_step[tile & 1], lead_lane);
        if (last) commit(&c.o_last, lead_lane);
    };
    while (walk.next(x)) {
        const int n = x.hi - x.lo;
        if (n == 0) continue;
        wait_phase(&c.q_full, blocks++ & 1, c.dead, limit);
        tc::fence_after_sync();
        scores(base);
        for (int j = 0; j < n; ++j) {
            if (X::kBufs == 2 && j + 1 < n) scores(base + j + 1);
            values(base + j, j == 0, j + 1 == n);
            if (X::kBufs == 1 && j + 1 < n) scores(base + j + 1);
        }
        base += n;
    }
}

template <class X>
__global__ void __launch_bounds__(X::kThreads, 1) attn_tree_kernel(const __grid_constant__ Tree<X> p, bool joins) {
    extern __shared__ char start[];
    char* smem = start + ((128 - (smem_u32(start) & 127)) & 127);
    static_assert(sizeof(TreeControl) <= X::kControlBytes, "control");
    TreeControl& c = *reinterpret_cast<TreeControl*>(smem + X::kControl);
    const int wid = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const unsigned long long limit = p.o.wait_ns;
    if (wid == 8) {
        tc::tmem_alloc(&c.tmem, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < X::kStages; ++i) {
            mbar_init(&c.k_full[i], 2);                              // halves of the tile
            mbar_init(&c.k_freed[i], 1 + 8);                         // the matrix steps, and the warps that read the table
            mbar_init(&c.v_full[i], 2);
            mbar_init(&c.v_freed[i], 1);
        }
        for (int i = 0; i < X::kRaws; ++i) {
            mbar_init(&c.raw_full[i], 1);
            mbar_init(&c.raw_freed[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.s_full[i], 1);
            mbar_init(&c.p_full[i], 8);
            mbar_init(&c.o_step[i], 1);
        }
        mbar_init(&c.q_full, kSoftmax / 32);
        for (int i = 0; i < 4; ++i) mbar_init(&c.ref_full[i], 1);
        mbar_init(&c.o_last, 1);
        mbar_init(&c.drained, 1);
        fence_mbar_init();
        for (int i = 0; i < 16; ++i) c.special[i] = 0;
        c.issued = 0;
        c.dead = limit == 0;                                         // (limit 0: given up from the start)
    }
    // means, offsets and V's extra columns: zero where nothing is written later
    for (int i = X::kQBytes / 16 + threadIdx.x; i < X::kRaw / 16; i += X::kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_async_smem();
    tc::fence_before_sync();
    wait_predecessor();
    launch_dependents();
    find_share<X>(static_cast<const Tree<X>&>(p), blockIdx.x, gridDim.x, reinterpret_cast<long long*>(smem + X::kRaw), c.cut);
    tc::fence_after_sync();
    if (joins && threadIdx.x == 0) p.o.places[blockIdx.x] = c.cut[0];
    if (blockIdx.x == 0 && threadIdx.x < p.B && p.status && p.over(threadIdx.x)) atomicExch(p.status, EDGE0_EINVAL);

    // registers, as many as the CTA was launched with: 256 x 160 + 256 x 96 of 512 x 128, or 256 x 144 + 384 x 64 of 640 x 96
    static_assert(X::kMakers == 6 || X::kMakers == 10, "the register split");
    if constexpr (X::kMakers == 6) {
        if (wid < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;\n");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 96;\n");
    } else {
        if (wid < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 144;\n");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;\n");
    }
    if (wid < 8) {
        tree_softmax<X>(p, c, smem);
    } else if (wid == 8) {
        tree_matrix<X>(p, c, smem);
    } else if (wid == 9) {
        // a round: the ring's next two entries, a strip of one of them a lane; behind the last token, that token's.  Pages'
        // numbers are asked for kAhead rounds ahead.  (One entry a round: this warp held up all others, 185 us for drafts
        // of 64 sequences.)
        constexpr int kAhead = 2, kLanes = 2 * X::kUnits;
        const int place = lane % kLanes, strip = place % X::kUnits, strips = p.c.page_tokens / kv::kStrip;
        Walk<X, Tree<X>> walk(p, c.cut, blockIdx.x);
        Item x;
        int n = 0, round = 0, unit = 0, slot = place, id[kAhead], at[kAhead];
        uint32_t parity = 0;
        bool ok = limit != 0, more = true, of_v[kAhead];
        // asks for the page of the next round's strip; false: none is left
        auto ask = [&](int& id, int& at, bool& of_v) {
            if (more && ++round >= n) {
                do more = walk.next(x);
                while (more && x.hi == x.lo);
                n = x.hi - x.lo;
                round = 0;
            }
            id = -1;
            if (!more) return;
            const int i = tile_of_entry<X>(2 * round + place / X::kUnits, n, of_v);
            const int from = min((x.lo + i) * X::kTile / kv::kStrip + strip, (x.s.n_k - 1) / kv::kStrip), pg = from / strips;
            id = p.table[(long long)x.b * p.W + pg];
            at = x.h * strips + from - pg * strips;
        };
        int asked = 0, had = 0;
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            ask(id[q], at[q], of_v[q]);
            asked += more;
        }
        while (ok && had < asked) {
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                if (!ok || had >= asked) break;
                ++had;
                int page = id[q];
                if (page < 0 || page >= p.c.n_pages) {
                    page = 0;
                    if (p.status) atomicExch(p.status, EDGE0_EINVAL);
                }
                const char* from = p.c.pages + page * p.c.page_bytes + (long long)at[q] * kv::strip_bytes(X::BITS, X::kD) + (of_v[q] ? X::kHalf : 0);
                ask(id[q], at[q], of_v[q]);
                asked += more;
                // (the phase before a barrier's first counts as over)
                ok = __all_sync(0xffffffffu, wait_alone(&c.raw_freed[slot], parity ^ 1, c.dead, limit));
                if (!ok) break;
                if (lane < kLanes) {
                    mbar_arrive_expect_tx(&c.raw_full[slot], X::kHalf);
                    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                                     smem_u32(smem + X::kRaw + slot * X::kHalf)),
                                 "l"(from), "r"((uint32_t)X::kHalf), "r"(smem_u32(&c.raw_full[slot]))
                                 : "memory");
                }
                __syncwarp();
                unit += kLanes;
                if ((slot += kLanes) >= X::kRaws) {
                    slot -= X::kRaws;
                    parity ^= 1;
                }
            }
        }
        if (lane == 0) c.issued = unit;
    } else {
        // a maker: every kMakers-th half of a tile's K or V, in the ring's order
        constexpr int kHalves = 2, kEach = X::kUnits / kHalves;
        Walk<X, Tree<X>> walk(p, c.cut, blockIdx.x);
        Item x;
        int base = 0, number = 0, at = wid - 10;                     // tiles before the block; the next half, from the block's first on
        while (walk.next(x)) {
            const int n = x.hi - x.lo;
            if (n > 0) ++number;
            for (; at < 2 * n * kHalves; at += X::kMakers) {
                bool v;
                const int entry = at / kHalves, i = tile_of_entry<X>(entry, n, v);
                const int tile = base + i, stage = tile % X::kStages;
                const uint32_t parity = (tile / X::kStages) & 1;
                char* to = v ? smem + X::kV + stage * X::kVStage : smem + X::kK + stage * X::kKStage;
                if (!__all_sync(0xffffffffu, wait_alone(v ? &c.v_freed[stage] : &c.k_freed[stage], parity ^ 1, c.dead, limit))) break;
                bool found = false, ok = true;
#pragma unroll 1
                for (int k = 0; k < kEach; ++k) {
                    const int strip = at % kHalves * kEach + k, u = (2 * base + entry) * X::kUnits + strip, slot = u % X::kRaws;
                    const int token = (x.lo + i) * X::kTile + 16 * strip;
                    const char* raw = smem + X::kRaw + slot * X::kHalf;
                    // (first that the slot's entry before is done with: a maker skips slots' phases, and one that had fallen two
                    // behind would look like the one it waits for.  The one before that is over: copies are issued in order,
                    // and this warp has had a later one)
                    ok = wait_alone(&c.raw_freed[slot], (u / X::kRaws + 1) & 1, c.dead, limit) && ok;
                    ok = wait_alone(&c.raw_full[slot], (u / X::kRaws) & 1, c.dead, limit) && ok;
                    __syncwarp();
                    if (v) found = make_rows<X, true>(raw, to, 16 * strip, p.o.c, x.s.n_k - token, x.s.ctx - token) || found;
                    else make_rows<X, false>(raw, to, 16 * strip, p.o.c, x.s.n_k - token, 0);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c.raw_freed[slot]);
                }
                if (found) *(volatile int*)&c.special[number & 15] = number;
                tc::fence_async_smem();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(v ? &c.v_full[stage] : &c.k_full[stage]);
            }
            if (*(volatile int*)&c.dead) break;
            at -= 2 * n * kHalves;
            base += n;
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (wid == 8) {
        if (c.dead) {                // matrix steps under way still read shared memory and write the accumulators
            commit(&c.drained, elect());
            wait_copy(&c.drained, 0, kDefaultWaitNs);
            // ... and copies under way, whoever gave up, must not land in what has become another CTA's memory
            drain_copies_call(c.raw_full, c.issued > X::kRaws ? c.issued - X::kRaws : 0, c.issued, X::kRaws);
            if (lane == 0 && p.status) atomicExch(p.status, EDGE0_ETIMEOUT);
        }
        tc::tmem_dealloc(c.tmem, 512);
    }
}

template <int BITS, int D>
int launch(const TreeP& base, char* ws, cudaStream_t stream) {
    using X = Tile<BITS, D>;
    constexpr int kDevices = 64;
    static int set[kDevices];            // per device: multiprocessors, set on the first call
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return EDGE0_ECUDA;
    int sms = __atomic_load_n(&set[dev], __ATOMIC_ACQUIRE);
    if (sms == 0) {
        if (cudaFuncSetAttribute(attn_tree_kernel<X>, cudaFuncAttributeMaxDynamicSharedMemorySize, X::kSmem) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return EDGE0_ECUDA;
        sms = sms < kMaxCtas ? sms : kMaxCtas;
        __atomic_store_n(&set[dev], sms, __ATOMIC_RELEASE);
    }
    Tree<X> p;
    static_cast<TreeP&>(p) = base;
    lay_out<X>(ws, &p.o);
    // blocks at most: no more CTAs than that
    const long long blocks = ((long long)p.T * p.G / X::kBlock + p.B) * p.H;
    const bool joins = (p.cap + X::kTile - 1) / X::kTile >= X::kMinSplit;
    const int grid = joins || blocks > sms ? sms : (int)blocks;
    const int rc = launch_early(attn_tree_kernel<X>, dim3(grid), X::kThreads, X::kSmem, stream, p, joins);
    if (rc || !joins || grid < 2) return rc;
    return launch_early(flash_join<X, Tree<X>>, dim3(grid - 1, X::kBlock / 32), 32 * kJoinWarps, 0, stream, p);
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" size_t edge0_attn_tree_workspace_bytes(const edge0_kv_cache* cache) {
    kv::View c;
    if (kv::view_of(cache, &c)) return 0;
    return cache->head_dim == 64    ? flash::workspace_bytes<Tile<4, 64>>()
           : cache->head_dim == 128 ? flash::workspace_bytes<Tile<4, 128>>()
                                    : flash::workspace_bytes<Tile<4, 256>>();
}

extern "C" int edge0_attn_tree(const edge0_kv_cache* cache, const uint16_t* q, long long ldq, int T, int n_q_heads,
                               const int32_t* table, int B, int W, const int32_t* lens, const int32_t* cu_rows, const uint32_t* mask,
                               int mask_words, float scale, uint16_t* out, long long ldo, int* status, void* workspace,
                               size_t workspace_bytes, cudaStream_t stream) {
    TreeP p;
    const int rc = kv::view_of(cache, &p.c);
    if (rc) return rc;
    if (!table || !lens || !cu_rows || B <= 0 || B > EDGE0_MAX_BATCHED || W <= 0 || T < 0) return EDGE0_EINVAL;
    if (n_q_heads <= 0 || n_q_heads % p.c.H) return EDGE0_EINVAL;
    const int G = n_q_heads / p.c.H, D = cache->head_dim;
    if (G > EDGE0_MAX_Q_PER_KV || (long long)T * G > (1ll << 31) - 512) return EDGE0_EUNSUPPORTED;
    if (!(scale > 0.f) || !(scale <= 1e6f)) return EDGE0_EINVAL;
    if (mask ? mask_words <= 0 : mask_words != 0) return EDGE0_EINVAL;
    if (mask_words > (1 << 20)) return EDGE0_EUNSUPPORTED;
    if (((uintptr_t)table | (uintptr_t)lens | (uintptr_t)cu_rows | (uintptr_t)mask | (uintptr_t)status) & 3) return EDGE0_EINVAL;
    if (T == 0) return EDGE0_OK;
    if (!q || !out || !workspace) return EDGE0_EINVAL;
    const long long width = (long long)n_q_heads * D;
    if (ldq < width || ldq % 8 || ldo < width || ldo % 8) return EDGE0_EINVAL;
    if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15) return EDGE0_EINVAL;
    if (workspace_bytes < edge0_attn_tree_workspace_bytes(cache)) return EDGE0_EINVAL;
    p.o.out = (__half*)out;
    p.o.ldo = ldo;
    p.o.c = scale * 1.4426950408889634f;
    p.o.wait_ns = block_wait_limit();
    p.q = (const __half*)q;
    p.ldq = ldq;
    p.B = B;
    p.H = p.c.H;
    p.G = G;
    p.T = T;
    p.W = W;
    const long long cap = (long long)W * p.c.page_tokens;
    p.cap = (int)(cap < (1ll << 30) ? cap : 1ll << 30);
    p.cu = cu_rows;
    p.lens = lens;
    p.table = table;
    p.mask = mask;
    p.words = mask_words;
    p.status = status;
    char* ws = (char*)workspace;
    if (cache->bits == 4)
        return D == 64 ? launch<4, 64>(p, ws, stream) : D == 128 ? launch<4, 128>(p, ws, stream) : launch<4, 256>(p, ws, stream);
    return D == 64 ? launch<8, 64>(p, ws, stream) : D == 128 ? launch<8, 128>(p, ws, stream) : launch<8, 256>(p, ws, stream);
}
