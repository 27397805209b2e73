// Attention of drafted tokens over the quantised KV cache: each sequence's rows see its context and,
// of the tokens drafted behind it, those that a mask names (a tree's ancestors) or those up to
// themselves.  The mathematics, the blocks and their shares: flash.cuh.
//
// K and V enter the tensor core as fp16 operands made from the codes in shared memory.
//   V = fp16(s q + b), the value that edge0_kv_read returns: its rounding weighs as much as that of the weight it meets.
//   K = fp16(s q + m) + o, m = 1024 s + fp16(-(1024 + z) s) a number near -z s (z half the code range), o = b - m exact in
//   fp32: what is rounded is the distance from the group's middle, so that an offset shared by the group's
//   64 dims, whatever its size, takes nothing from it.  1024 s and -(1024 + z) s are what one fused step on codes with
//   1024 in front of them needs.  o . sum(Q of the group) is one more step of 16 of the scores' product, both
//   factors split into two fp16 (to 2^-22); a query row is scaled by a power of two before, so that its sums
//   stay in range whatever its size.  Groups with s above kWide (that step would leave fp16) take code - z + 1/2 and
//   s apart.
//
// Warps: 0-7 softmax, 8 the matrix steps, 9 copies strips' halves (16 tokens of K or of V, one run of bytes)
// into a ring of raw ones, 10-15 turn those into operand entries.  16 tokens of 4-bit codes and 128 dims are
// 1,152 bytes; raw entries keep about 40 KB under way per SM, which the latency of memory asks for.
#include "flash.cuh"

namespace edge0 {
namespace {

using namespace flash;

constexpr int kThreadsF = kSoftmax + 256;
constexpr int kMakers = 6;               // warps that turn codes into operands
constexpr int kMaxRaw = 40;              // raw entries
constexpr float kWide = 48.f;

template <int BITS, int D>
struct Shapes {
    using X = Shape<D>;
    static constexpr int kStages = D == 64 ? 5 : 3;
    static constexpr int kR = kv::row_bytes(BITS, D), kHalf = kv::half_bytes(BITS, D);
    static constexpr int kGroups = D / kGroup;
    static constexpr int kUnits = X::kEntry / kv::kStrip;            // raw entries of an operand entry
    static constexpr int kXk = X::kEntry * 32;                       // a K entry's offsets
    // shared memory
    static constexpr int kXq = X::kStreams * X::kQBytes;
    static constexpr int kRing = kXq + X::kStreams * kRowsQ * 32;
    static constexpr int kXkAt = kRing + kStages * X::kEntryBytes;
    static constexpr int kRaw = kXkAt + kStages * kXk;
    static constexpr int kRoom = 232448 - 1024 - (int)sizeof(Control) - 2 * kMaxRaw * 8 - kRaw;
    static constexpr int kRaws = kRoom / kHalf < kMaxRaw ? kRoom / kHalf : kMaxRaw;
    static constexpr int kControl = kRaw + kRaws * kHalf;
    static constexpr int kBars = kControl + (int)sizeof(Control);
    static constexpr int kSmem = kBars + 2 * kMaxRaw * 8 + 1024;
    static_assert(kRing % 1024 == 0 && kRaw % 16 == 0 && kControl % 16 == 0 && kRaws >= 2 * kUnits && sizeof(Control) % 8 == 0, "layout");
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

template <int BITS, int D>
struct Tree : TreeP {
    static constexpr bool kExtra = true, kLooked = false;
    static constexpr int kHeld = 64;
    // columns of 4-bit V: the codes of a word in the order that masking gives them
    __host__ __device__ static constexpr int dim_of(int column) { return BITS == 4 ? (column >> 1) + 4 * (column & 1) : column; }

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

    struct Row {
        int n;                           // tokens that the row sees, or with a mask those it may see
        const unsigned* bits;
        __device__ Row(const Tree& p, const Item& x, int token)
            : n(p.seen(x.s, token)), bits(p.mask ? p.mask + (long long)(x.s.q0 + token) * p.words : nullptr) {}
        __device__ uint32_t seen(const Tree& p, const Item& x, int from) const {
            const int k = n - from, d = from - x.s.ctx;
            uint32_t v = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1;
            if (bits && d > -32) {
                auto word = [&](int i) -> uint32_t { return i < p.words ? bits[i] : 0u; };
                // drafted tokens d .. d + 31; those below 0 are the context's
                v &= d < 0 ? (word(0) << -d) | ((1u << -d) - 1)
                           : __funnelshift_r(word(d >> 5), word((d >> 5) + 1), d & 31);
            }
            return v;
        }
    };

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

    __device__ void load_queries(const Item& x, bool live, int token, int head, char* dst, char* sums, int row, float& cc) const {
        const uint4* src = reinterpret_cast<const uint4*>(q + (long long)(x.s.q0 + token) * ldq + (long long)head * D);
        uint32_t top = 0;                                            // largest magnitude's bits, two at a time
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i) {
            const uint4 v = live ? src[i] : make_uint4(0, 0, 0, 0);
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
        top = max(top & 0xffffu, top >> 16);
        // the row times 2^e: its largest value in [8, 16) where a normal fp16 factor does that
        int e = top == 0 ? 0 : 18 - (int)(top >> 10);
        e = max(-14, min(15, e));
        const uint32_t f = (uint32_t)(15 + e) << 10, f2x = f | f << 16;
        cc *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 1
        for (int g = 0; g < D / kGroup; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint4 v = live ? src[8 * g + i] : make_uint4(0, 0, 0, 0);
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    w[k] = hfma2(w[k], f2x, 0x80008000u);            // (a product by a power of two; -0 changes nothing)
                    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
                    sum += t.x + t.y;
                }
                if (BITS == 4)
                    v = make_uint4(__byte_perm(w[0], w[2], 0x5410), __byte_perm(w[0], w[2], 0x7632), __byte_perm(w[1], w[3], 0x5410),
                                   __byte_perm(w[1], w[3], 0x7632));
                else
                    v = make_uint4(w[0], w[1], w[2], w[3]);
                *reinterpret_cast<uint4*>(dst + g * (kRowsQ * 128) + swizzled(row, i)) = v;
            }
            // (hi, hi / 2^11, what hi leaves) against (offset's hi, 2^11 times what that leaves, hi)
            const __half hi = __float2half_rn(sum), small = __float2half_rn(__half2float(hi) * 0x1p-11f),
                         lo = __float2half_rn(sum - __half2float(hi));
            const __half2 a = __halves2half2(hi, small), b = __halves2half2(lo, __ushort_as_half(0));
            *reinterpret_cast<uint2*>(sums + tc::kstep_off(row, 4 * g)) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
    }
    // NaN of V's groups among the drafted tokens that the row sees (they enter the product as zeros)
    __device__ void add_special(const Item& x, const Row& r, int, int k, float (&o)[32]) const {
        for (int j = max(x.s.ctx, x.lo * kTile); j < min(x.s.n_k, x.hi * kTile); ++j) {
            if (!(r.seen(*this, x, j) & 1)) continue;
            const __half2 sb = *reinterpret_cast<const __half2*>(place(x.b, x.h, j, true) + 16 * kv::row_bytes(BITS, D) +
                                                                 (j % 16) * kv::sb_bytes(D) + k / kGroup * 4);
            if (__hisnan(__low2half(sb)) || __hisnan(__high2half(sb)))
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __int_as_float(0x7fffffff);
        }
    }
};

// 1024 + code, two dims a word: 4 bits: dims (0, 4), (1, 5), (2, 6), (3, 7) of the word; 8 bits: in order
template <int BITS>
__device__ __forceinline__ void raised(uint32_t w0, uint32_t w1, uint32_t (&r)[4]) {
    if (BITS == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = ((w0 >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
    } else {
        r[0] = __byte_perm(w0, 0x64646464u, 0x4140);
        r[1] = __byte_perm(w0, 0x64646464u, 0x4342);
        r[2] = __byte_perm(w1, 0x64646464u, 0x4140);
        r[3] = __byte_perm(w1, 0x64646464u, 0x4342);
    }
}
__device__ __forceinline__ uint32_t twice(__half h) {
    const __half2 v = __halves2half2(h, h);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// A raw entry (16 tokens) into rows row0 .. row0 + 15 of an operand entry, by a warp.  V's tokens from `left` on are zeros,
// and so are groups of NaN from `drafted` on, which some rows may not see: true where there are any.
template <int BITS, int D>
__device__ __forceinline__ bool make_rows(const char* raw, char* entry, char* offsets, int row0, bool value, int left, int drafted) {
    using Z = Shapes<BITS, D>;
    constexpr int CH = Z::kR / 16, kPer = BITS == 4 ? 4 : 2;         // pieces of a row, 8-dim words per piece
    constexpr float kZ = BITS == 4 ? 8.f : 128.f;
    const int lane = threadIdx.x & 31;
    bool found = false;
#pragma unroll
    for (int j = 0; j < CH / 2; ++j) {
        const int i = j * 32 + lane, c = (i >> 3) % CH, tok = (i & 7) + 8 * ((i >> 3) / CH), g = c / (CH / Z::kGroups);
        const uint4 codes = *reinterpret_cast<const uint4*>(raw + tok * Z::kR + ((c ^ kv::turn(Z::kR, tok)) << 4));
        const __half2 sb = *reinterpret_cast<const __half2*>(raw + 16 * Z::kR + tok * kv::sb_bytes(D) + g * 4);
        const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
        const __half s = __low2half(sb), b = __high2half(sb);
        const float sf = __half2float(s), bf = __half2float(b);
        const int row = row0 + tok;
        uint4 out[kPer];
        const uint32_t s2 = twice(s);
        if (value) {
            const bool hidden = tok >= left, bad = tok >= drafted && (sf != sf || bf != bf);
            found = found || (bad && !hidden);
            const uint32_t b2 = twice(b), keep = hidden || bad ? 0u : 0xffffffffu;
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                uint32_t r[4];
                raised<BITS>(w[BITS == 4 ? x : 2 * x], w[BITS == 4 ? x : 2 * x + 1], r);
#pragma unroll
                for (int k = 0; k < 4; ++k) r[k] = hfma2(hadd2(r[k], 0xE400E400u), s2, b2) & keep;
                out[x] = make_uint4(r[0], r[1], r[2], r[3]);
            }
        } else {
            const bool wide = sf > kWide;
            const __half e16 = __float2half_rn(-(1024.f + kZ) * sf);
            const uint32_t e2 = twice(e16);
#pragma unroll
            for (int x = 0; x < kPer; ++x) {
                uint32_t r[4];
                raised<BITS>(w[BITS == 4 ? x : 2 * x], w[BITS == 4 ? x : 2 * x + 1], r);
                if (!wide) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) r[k] = hfma2(r[k], s2, e2);
                } else {
                    const uint32_t z2 = twice(__float2half_rn(0.5f - kZ));
#pragma unroll
                    for (int k = 0; k < 4; ++k) r[k] = hfma2(hadd2(hadd2(r[k], 0xE400E400u), z2), s2, 0x80008000u);
                }
                out[x] = make_uint4(r[0], r[1], r[2], r[3]);
            }
            if (c % (CH / Z::kGroups) == 0) {
                const float off = wide ? fmaf(kZ - 0.5f, sf, bf) : bf - fmaf(1024.f, sf, __half2float(e16));
                const __half hi = __float2half_rn(off), lo = __float2half_rn((off - __half2float(hi)) * 2048.f);
                const __half2 p = __halves2half2(hi, lo), q = __halves2half2(hi, __ushort_as_half(0));
                *reinterpret_cast<uint2*>(offsets + tc::kstep_off(row, 4 * g)) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
            }
        }
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
            const int c8 = c * kPer + x;                             // 8 dims
            *reinterpret_cast<uint4*>(entry + (c8 >> 3) * (Shape<D>::kEntry * 128) + swizzled(row, c8 & 7)) = out[x];
        }
    }
    return found;
}

template <int BITS, int D>
__global__ void __launch_bounds__(kThreadsF, 1) attn_tree_kernel(const __grid_constant__ Tree<BITS, D> p, bool joins) {
    using X = Shape<D>;
    using Z = Shapes<BITS, D>;
    using Src = Tree<BITS, D>;
    extern __shared__ char start[];
    char* smem = start + ((1024 - (smem_u32(start) & 1023)) & 1023);
    Control& c = *reinterpret_cast<Control*>(smem + Z::kControl);
    uint64_t *raw_full = reinterpret_cast<uint64_t*>(smem + Z::kBars), *raw_freed = raw_full + kMaxRaw;
    const int wid = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (wid == 8) {
        tc::tmem_alloc(&c.tmem, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < Z::kRaws; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_freed[i], 1);
        }
        control_init(c, Z::kUnits, 1, 1, p.o.wait_ns == 0);
    }
    // the steps of 16 for the offsets: zero where nothing is written later
    for (int i = threadIdx.x; i < (Z::kRing - Z::kXq) / 16; i += kThreadsF) reinterpret_cast<uint4*>(smem + Z::kXq)[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < (Z::kRaw - Z::kXkAt) / 16; i += kThreadsF) reinterpret_cast<uint4*>(smem + Z::kXkAt)[i] = make_uint4(0, 0, 0, 0);
    tc::fence_async_smem();
    tc::fence_before_sync();
    wait_predecessor();
    launch_dependents();
    find_share<D>(static_cast<const Src&>(p), blockIdx.x, gridDim.x, reinterpret_cast<long long*>(smem), c.cut);
    tc::fence_after_sync();
    if (joins && threadIdx.x == 0) p.o.places[blockIdx.x] = c.cut[0];
    if (blockIdx.x == 0 && threadIdx.x < p.B && p.status && p.over(threadIdx.x)) atomicExch(p.status, EDGE0_EINVAL);

    // registers: 256 x 168 + 256 x 88, what the CTA was launched with (512 x 128)
    if (wid < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;\n");
        softmax_warps<D, Src>(p, c, smem, smem + Z::kXq);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
        if (wid == 8) {
            matrix_warp<D, Z::kStages, Src>(p, c, smem_u32(smem), smem_u32(smem + Z::kRing), smem_u32(smem + Z::kXq), smem_u32(smem + Z::kXkAt));
        } else if (wid == 9) {
            Feed<D, Src> feed(p, c.cut, blockIdx.x);
            int unit = 0;
            bool ok = p.o.wait_ns != 0, more = feed.next();
            // a lane: one of the entry's strips; behind the last token, that token's
            auto source = [&]() { return p.place(feed.x.b, feed.x.h, min(feed.token() + 16 * (lane % Z::kUnits), feed.x.s.n_k - 1), feed.value); };
            const char* src = more ? source() : nullptr;
            while (ok && more) {
                const int u = unit + lane % Z::kUnits, slot = u % Z::kRaws;
                const char* from = src;
                more = feed.next();
                if (more) src = source();                            // on its way during the wait
                // (the phase before a barrier's first counts as over)
                ok = wait_phase(&raw_freed[slot], (u / Z::kRaws + 1) & 1, c, p.o.wait_ns);
                if (!ok) break;
                if (lane < Z::kUnits) {
                    mbar_arrive_expect_tx(&raw_full[slot], Z::kHalf);
                    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                                     smem_u32(smem + Z::kRaw + slot * Z::kHalf)),
                                 "l"(from), "r"((uint32_t)Z::kHalf), "r"(smem_u32(&raw_full[slot]))
                                 : "memory");
                }
                __syncwarp();
                unit += Z::kUnits;
            }
            // nothing may land in this memory when it has become another CTA's
            if (!ok) drain_copies_call(raw_full, unit > Z::kRaws ? unit - Z::kRaws : 0, unit, Z::kRaws);
        } else {
            Feed<D, Src> feed(p, c.cut, blockIdx.x);
            int unit = 0;
            for (int at = 0; feed.next(); ++at, unit += Z::kUnits) {
                const int stage = at % Z::kStages;
                const Item& x = feed.x;
                bool ready = at < Z::kStages;
                for (int i = (wid - 10 + kMakers - unit % kMakers) % kMakers; i < Z::kUnits; i += kMakers) {
                    const int u = unit + i, slot = u % Z::kRaws;
                    ready = ready || wait_phase(&c.freed[stage], (at / Z::kStages - 1) & 1, c, p.o.wait_ns);
                    if (!ready || !wait_phase(&raw_full[slot], (u / Z::kRaws) & 1, c, p.o.wait_ns)) break;
                    const int token = feed.token() + 16 * i;
                    if (make_rows<BITS, D>(smem + Z::kRaw + slot * Z::kHalf, smem + Z::kRing + stage * X::kEntryBytes,
                                           smem + Z::kXkAt + stage * Z::kXk, 16 * i, feed.value, x.s.n_k - token, x.s.ctx - token))
                        special_of(c, feed.number) = feed.number;
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&c.full[stage]);
                        mbar_arrive(&raw_freed[slot]);
                    }
                }
            }
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (wid == 8) {
        if (c.dead) {                // matrix steps under way still read shared memory and write the accumulators
            commit(&c.drained, elect());
            wait_copy(&c.drained, 0, kDefaultWaitNs);
            if (lane == 0 && p.status) atomicExch(p.status, EDGE0_ETIMEOUT);
        }
        tc::tmem_dealloc(c.tmem, 512);
    }
}

template <int BITS, int D>
int launch(const TreeP& base, char* ws, cudaStream_t stream) {
    using Z = Shapes<BITS, D>;
    constexpr int kDevices = 64;
    static int set[kDevices];            // per device: multiprocessors, set on the first call
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return EDGE0_ECUDA;
    int sms = __atomic_load_n(&set[dev], __ATOMIC_ACQUIRE);
    if (sms == 0) {
        if (cudaFuncSetAttribute(attn_tree_kernel<BITS, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::kSmem) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return EDGE0_ECUDA;
        sms = sms < kMaxCtas ? sms : kMaxCtas;
        __atomic_store_n(&set[dev], sms, __ATOMIC_RELEASE);
    }
    Tree<BITS, D> p;
    static_cast<TreeP&>(p) = base;
    lay_out<D>(ws, &p.o);
    // blocks at most: no more CTAs than that
    const long long blocks = ((long long)p.T * p.G / Shape<D>::kBlock + p.B) * p.H;
    const bool joins = (p.cap + kTile - 1) / kTile >= kMinSplit;
    const int grid = joins || blocks > sms ? sms : (int)blocks;
    const int rc = launch_early(attn_tree_kernel<BITS, D>, dim3(grid), kThreadsF, Z::kSmem, stream, p, joins);
    if (rc || !joins || grid < 2) return rc;
    return launch_early(flash_join<D, Tree<BITS, D>>, dim3(grid - 1, Shape<D>::kBlock / 32), 128, 0, stream, p);
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" size_t edge0_attn_tree_workspace_bytes(const edge0_kv_cache* cache) {
    kv::View c;
    return kv::view_of(cache, &c) ? 0 : edge0_attn_prompt_workspace_bytes(cache->head_dim);
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
