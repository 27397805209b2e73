// Attention of many query rows per K/V head on the fifth-generation tensor cores: what attention of
// packed prompts (attn_prompt.cu) and of drafted tokens over the quantised cache (attn_tree.cu) share.
//
//     o_i = sum_j p_ij v_j / sum_j p_ij,   p_ij = exp(scale q_i . k_j) over the tokens j that row i sees.
//
// Rows.  A K/V head's query rows of a sequence in the order (token, head of the group): a block
// of them shares every K and V tile that it reads, whatever the number of query heads per K/V head, and
// ragged sequences leave at most one block partly empty per K/V head.
//
// Streams.  With up to 128 dims a block has two streams, each a softmax warpgroup with a score tile
// and an accumulator of 128 rows in TMEM (512 columns in all): two row tiles on the same K/V tiles, or, of a
// block of at most 128 rows, one row tile on alternate K/V tiles, added up at the end.  While one stream's
// scores become weights the tensor core works for the other.  256 dims: one stream, whose next scores
// are formed (in a second buffer) while the present ones become weights.
//
// Step of a stream.  S = Q K^T (128 x 128) into TMEM; a thread reads its row, takes the maximum, forms the
// weights 2^(S c - ref + 11) and writes them as fp16 over the scores; O += P V with P from TMEM.  The
// reference moves only when exceeded by 2^4 (the accumulator is then rescaled in TMEM), so that
// weights lie within 2^15 and stay normal in fp16 down to 2^-25 of the largest; their rounding, 2^-11 of each,
// is the only one beside the result's.  Statistics and sums are fp32.
//
// Shares.  All blocks of all sequences and heads in a row, each at the cost of the tokens it sees and of
// its start and end, are cut into equal shares, one per CTA, from lengths read on the device; a cut that falls
// into a block too small to be worth it moves to the block's edge.  Blocks cut leave parts (reference, sum, fp32 o),
// which flash_join adds up in the order of the tokens: the same bits on every run.
#pragma once
#include "kvcache.cuh"
#include "launch.cuh"
#include "tc05.cuh"
#include "wait.cuh"

namespace edge0 {
namespace flash {

constexpr int kTile = 128;            // tokens per step
constexpr int kRowsQ = 128;           // rows of an accumulator
constexpr int kMaxCtas = 160;         // shares at most (an SM each)
constexpr float kRise = 4.f;          // how far scores may exceed the reference, as a power of two
constexpr float kUp = 11.f;           // weights are 2^kUp times as large: kRise + kUp = 15
constexpr int kSoftmax = 256;         // threads of the two softmax warpgroups

// What the shares go by: a block's rows (kBlock), tokens per step (kTile), head width, and in tiles
//   kOwn        what a block costs beside its tiles (its queries, the first scores, the last product, its outputs).  1 instead
//               of 4: 64 prompts of up to 1,024 tokens 279 us instead of 263, one short prompt 18 instead of 10, drafts of 64
//               sequences of 500 to 4,000 tokens 179 instead of 159; 8: 278, 10 and 150;
//   kMinSplit   from which on a block may be cut (a cut costs a start and an end more, parts of fp32 and their join).  4
//               instead of 8: drafts behind 300 tokens 17.7 us instead of 14.5, prompts the same;
//   kMinWhole   likewise, where a block is not as much as two shares: there it is only the shares' evenness that a cut
//               serves.  8 instead of 32: a prompt of 1,000 tokens 31.6 us instead of 25, of 2,000 63 instead of 54, of 4,000
//               129 instead of 120; drafted tokens' blocks cost less to cut (8 and 32: drafts of 64 sequences 159.6 and 160.5 us);
//   kMinShare   that a share has at least.  2, 4, 8, 12: one short prompt 10.0, 10.0, 14.0 and 18.3 us, drafts behind 2,000
//               tokens 20.9, 20.1, 24.0 and 25.0.
template <int D>
struct Shape {
    static constexpr int kD = D, kTile = flash::kTile, kMinSplit = 8, kMinWhole = 32, kMinShare = 4, kOwn = 4;
    static constexpr int kStreams = D <= 128 ? 2 : 1;
    static constexpr int kBlock = kStreams * kRowsQ;          // rows of a block
    static constexpr int kEntry = D == 256 ? 64 : kTile;      // tokens of a ring entry
    static constexpr int kEntries = kTile / kEntry;           // entries of a K (or V) tile
    static constexpr int kEntryBytes = kEntry * D * 2;
    static constexpr int kChunks = D / 64;                    // 128-byte swizzled columns of an operand
    static constexpr int kQBytes = kRowsQ * D * 2;
    // how many tiles K runs ahead of V for a block of so many rows
    __host__ __device__ static constexpr int lead(int rows) { return kStreams == 2 && rows > kRowsQ ? 1 : 2; }
    // TMEM columns: scores (or weights) of a stream or buffer, accumulators behind both
    static constexpr int kO = 2 * kTile;
};

// A block, or the place of a cut in it; tile > 0: inside.
struct Place {
    int b, h, t, tile;
};
__device__ __forceinline__ bool same_block(const Place& x, const Place& y) { return x.b == y.b && x.h == y.h && x.t == y.t; }

// Rows and keys of a sequence: its n_q rows begin at row q0, its n_k keys at k0; its row i sees at most the keys
// before i + 1 + off; all see those before ctx.
struct Seq {
    int q0, n_q, k0, n_k, off, ctx;
};

struct Item {
    int b, h;
    Seq s;
    int row0, rows;       // (token, head) rows of the block
    int lo, hi, tiles;    // the share's tiles, all of them
    int clear;            // tiles that every row sees in whole
    int part;             // slot of the share's part, -1: the share has the block whole

    template <int D>
    __device__ __forceinline__ bool pair() const { return Shape<D>::kStreams == 2 && rows > kRowsQ; }
    // tiles of a stream: all of them, or every other one
    template <int D>
    __device__ __forceinline__ int of_stream(int s) const {
        const int n = hi - lo;
        return Shape<D>::kStreams == 1 || pair<D>() ? n : (n + 1 - s) >> 1;
    }
    template <int D>
    __device__ __forceinline__ int tile_of(int s, int j) const {
        return lo + (Shape<D>::kStreams == 1 || pair<D>() ? j : 2 * j + s);
    }
};

// ----------------------------------------------------------------- shares ----
// Costs count a (row of a token's group, token) pair as 1 / block rows of it: a block costs the tokens its last row
// sees times G, and kOwn tiles.
template <class Sh>
struct Costs {
    static constexpr int R = Sh::kBlock;
    long long per, own;   // cost of a tile: kTile G; of a block beside its tiles
    long long off, all;   // off G, n_k G
    int blocks;
    long long some, whole;   // the first blocks that see a token, that see all (R: a power of two)

    __host__ __device__ Costs(const Seq& s, int G) {
        per = (long long)Sh::kTile * G;
        own = Sh::kOwn * per;
        off = (long long)s.off * G;
        all = (long long)s.n_k * G;
        blocks = (int)(((long long)s.n_q * G + R - 1) / R);
        some = off >= 0 ? 0 : -off / R;
        whole = all <= off ? 0 : (all - off + R - 1) / R - 1;
    }
    __host__ __device__ long long tokens(int t) const {        // times G
        if (t == blocks - 1) return all;
        const long long v = off + (long long)R * (t + 1);
        return v < 0 ? 0 : v < all ? v : all;
    }
    __host__ __device__ long long before(int t) const {        // cost of the blocks 0 .. t - 1, t < blocks
        // blocks some .. whole - 1 see off + R (their number + 1), those from there on all (drafted tokens with a mask, or cut off)
        const long long from = some < t ? some : t, to = whole < from ? from : whole < t ? whole : t;
        return t * own + (to - from) * off + R * (to * (to + 1) - from * (from + 1)) / 2 + (t - to) * all;
    }
    __host__ __device__ long long total() const { return blocks ? before(blocks - 1) + own + all : 0; }
};

// a / b, both not negative; 64-bit divisions take a microsecond together where 32 bits do
__device__ __forceinline__ long long divide(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The places of the cuts `first` and first + 1 of the CTAs' shares, by the whole CTA of at least 256 threads;
// prefix: [EDGE0_MAX_BATCHED + 1] of scratch.
template <class Sh, class Src>
__device__ void find_share(const Src& p, int cta, int ctas, long long* prefix, Place* out) {
    const int tid = threadIdx.x;
    long long mine = 0;
    if (tid < p.B) mine = Costs<Sh>(p.seq(tid), p.G).total() * p.H;
    if (tid < EDGE0_MAX_BATCHED) prefix[tid + 1] = mine;
    __syncthreads();
    if (tid < 32) {                                   // 8 sequences a lane
        long long v[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = sum += prefix[1 + 8 * tid + i];
        long long scan = sum;
#pragma unroll
        for (int s = 1; s < 32; s *= 2) {
            const long long o = __shfl_up_sync(0xffffffffu, scan, s);
            if (tid >= s) scan += o;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) prefix[1 + 8 * tid + i] = v[i] + scan - sum;
        if (tid == 0) prefix[0] = 0;
    }
    __syncthreads();
    if (tid == 0 || tid == 32) {
        const long long all = prefix[p.B], least = (long long)Sh::kMinShare * Sh::kTile * p.G;
        long long share = divide(all + ctas - 1, ctas);
        if (share < least) share = least;             // (so that two cuts never fall on one tile of a block)
        const int i = cta + (tid == 32);
        const long long x = share * i;
        Place at{p.B, 0, 0, 0};
        if (x < all) {
            int lo = 0, hi = p.B;                     // the last b with prefix[b] <= x
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (prefix[mid] <= x) lo = mid;
                else hi = mid;
            }
            const Costs<Sh> c(p.seq(lo), p.G);
            const long long head = c.total();
            long long in = x - prefix[lo];
            at.b = lo;
            at.h = (int)divide(in, head);
            in -= at.h * head;
            int t0 = 0, t1 = c.blocks;
            while (t1 - t0 > 1) {
                const int mid = (t0 + t1) >> 1;
                if (c.before(mid) <= in) t0 = mid;
                else t1 = mid;
            }
            at.t = t0;
            in -= c.before(t0);
            const long long seen = c.tokens(t0), cost = seen + c.own;
            const int tiles = (int)divide(seen + c.per - 1, c.per);
            // the nearest, less the block's own cost
            int tile = in < c.own ? 0 : (int)divide(in - c.own + c.per / 2, c.per);
            if (tiles < (cost >= 2 * share ? Sh::kMinSplit : Sh::kMinWhole) || cost * 8 <= share) tile = 2 * in > cost ? tiles : 0;
            if (tile >= tiles && tile > 0) {          // the next block's start
                tile = 0;
                if (++at.t == c.blocks) {
                    at.t = 0;
                    if (++at.h == p.H) {
                        at.h = 0;
                        do ++at.b;
                        while (at.b < p.B && prefix[at.b + 1] == prefix[at.b]);
                    }
                }
            }
            at.tile = tile;
        }
        out[tid == 32] = at;
    }
    tc::fence_async_smem();                           // (copies come where the scratch was)
    __syncthreads();
}

// Goes through a share's blocks.
template <class Sh, class Src>
struct Walk {
    const Src& p;
    Place at, end;
    Seq s;
    int blocks, cta;
    bool inside;          // the share begins inside a block

    __device__ Walk(const Src& p, const Place* cut, int cta) : p(p), at(cut[0]), end(cut[1]), cta(cta), inside(cut[0].tile > 0) { enter(); }
    __device__ void enter() {
        while (at.b < p.B) {
            s = p.seq(at.b);
            blocks = (int)(((long long)s.n_q * p.G + Sh::kBlock - 1) / Sh::kBlock);
            if (blocks) break;
            ++at.b;
        }
    }
    // the next piece of work; false: none is left
    __device__ bool next(Item& x) {
        for (;;) {
            const bool last = same_block(at, end);
            if (at.b >= p.B || (last && end.tile <= at.tile)) return false;
            if (at.b > end.b || (at.b == end.b && (at.h > end.h || (at.h == end.h && at.t > end.t)))) return false;
            constexpr int R = Sh::kBlock, kTile = Sh::kTile;
            const int all = s.n_q * p.G;
            x.b = at.b;
            x.h = at.h;
            x.s = s;
            x.row0 = at.t * R;
            x.rows = min(R, all - x.row0);
            const int seen = p.seen(s, (x.row0 + x.rows - 1) / p.G);
            x.tiles = (seen + kTile - 1) / kTile;
            x.clear = p.seen_by_all(s, x.row0 / p.G) / kTile;
            x.lo = min(at.tile, x.tiles);
            x.hi = last ? min(end.tile, x.tiles) : x.tiles;
            const bool from = at.tile > 0;
            x.part = x.lo == 0 && !last ? -1 : 2 * cta + (from ? 0 : 1);
            if (last) {
                at.tile = end.tile;
            } else {
                at.tile = 0;
                if (++at.t == blocks) {
                    at.t = 0;
                    if (++at.h == p.H) {
                        at.h = 0;
                        ++at.b;
                        enter();
                    }
                }
            }
            return true;
        }
    }
};

// ----------------------------------------------------- matrix steps, TMEM ----
// A 128-byte-swizzled operand: columns of 64 values (128 bytes) of all rows, one after the other; the 16-byte
// piece c of row r of a column lies at piece c ^ (r & 7).
__device__ __forceinline__ uint32_t swizzled(int row, int piece) { return (uint32_t)(row * 128 + ((piece ^ (row & 7)) << 4)); }

// Descriptors of such operands; the low word advances with the address.  K-major: 8-row blocks 1024
// bytes apart.  MN-major (rows are the product's inner dimension): 8-row blocks 1024 bytes
// apart likewise, columns `apart` bytes.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t apart) { return (saddr >> 4) | ((apart >> 4) << 16); }
__device__ __forceinline__ uint64_t desc128(uint32_t lo) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"((1024u >> 4) | (1u << 14) | (2u << 29)));
    return d;
}
// Matrix steps and their commit, issued by the lane with `lead` set of a warp that comes here together.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate, uint32_t lead) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(lead)
        : "memory");
}
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
#define EDGE0_R4(r, i) "=r"((r)[i]), "=r"((r)[i + 1]), "=r"((r)[i + 2]), "=r"((r)[i + 3])
#define EDGE0_I4(r, i) "r"((r)[i]), "r"((r)[i + 1]), "r"((r)[i + 2]), "r"((r)[i + 3])
// 32 columns of the thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t a, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : EDGE0_R4(r, 0), EDGE0_R4(r, 4), EDGE0_R4(r, 8), EDGE0_R4(r, 12), EDGE0_R4(r, 16), EDGE0_R4(r, 20), EDGE0_R4(r, 24),
          EDGE0_R4(r, 28)
        : "r"(a)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t a, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(a),
        EDGE0_I4(r, 0), EDGE0_I4(r, 4), EDGE0_I4(r, 8), EDGE0_I4(r, 12), EDGE0_I4(r, 16), EDGE0_I4(r, 20), EDGE0_I4(r, 24),
        EDGE0_I4(r, 28)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// -------------------------------------------------------------------- CTA ----
constexpr int kMaxStages = 8;
constexpr int kStageBytes = kRowsQ * 128;       // staging of a stream's outputs: 64 dims
struct Control {
    uint64_t full[kMaxStages];      // a ring entry has arrived
    uint64_t clean[kMaxStages];     // ... and been looked through
    uint64_t freed[kMaxStages];     // ... and is done with
    uint64_t q_full[2], q_freed[2]; // a stream's queries are in place, are done with
    uint64_t s_full[2];             // scores of a stream (two streams) or a buffer (one)
    uint64_t p_full[2];             // ... have become weights
    uint64_t o_step[2];             // one stream: the product with V of a tile of this buffer is done
    uint64_t o_last[2];             // a stream's last product of a block is done
    uint64_t drained;
    Place cut[2];
    uint32_t tmem;
    int q_loads[2];                 // copies of a stream's queries so far
    int issued;                     // copies of ring entries in all, when the warp that issues them has ended
    int dead;                       // a wait ran out: nothing more is issued, what is not done becomes NaN
    int special[kMaxStages * 2];    // numbers of the share's blocks with non-finite V that some rows do not see, by their last bits
    float2 ml[kRowsQ];              // the second stream's (reference, sum)
};

// One look at a phase.  What it orders is this CTA's alone: the scope of a cluster invalidates L1 with every look (one long
// prompt 1,495 -> 1,418 us, drafts of 64 sequences 211 -> 200 when it came in).  Looks that do not suspend cost more (1,535 and 207), and
// so do those that name the time to suspend for (1,493 and 218) and sixteen looks in a row between two readings of the clock
// (1,417 and 223).
__device__ __forceinline__ bool look(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// Waits for a phase of a barrier, each thread by itself; gives up after `limit` ns or when another warp did
__device__ __forceinline__ bool wait_alone(uint64_t* bar, uint32_t parity, int& dead, unsigned long long limit) {
    if (look(bar, parity)) return true;
    unsigned long long t0, now;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (;;) {
        if (look(bar, parity)) return true;
        if (*(volatile int*)&dead) return false;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        if (now - t0 > limit) *(volatile int*)&dead = 1;
    }
}
// ... by a whole warp, which agrees on the answer
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int& dead, unsigned long long limit) {
    bool ok = !*(volatile int*)&dead && look(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        unsigned long long t0, now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        while (!ok) {
            if (*(volatile int*)&dead) break;
            ok = look(bar, parity);
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
            if (!ok && now - t0 > limit) *(volatile int*)&dead = 1;
        }
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

// Where a block of the share (numbers from 1, of those with tiles) is marked: whoever looks V through runs no more than the
// ring's entries ahead.
__device__ __forceinline__ volatile int& special_of(Control& c, int number) {
    return *(volatile int*)&c.special[number & (kMaxStages * 2 - 1)];
}

// Place of a tile's first entry in the ring, counted from the block's first: K tiles run `lead` ahead of V's.
__device__ __forceinline__ int k_entry(int i, int lead) { return i < lead ? i : 2 * i - lead + 1; }
__device__ __forceinline__ int v_entry(int i, int lead, int n) { return i + min(n, lead + i); }

struct Out {
    __half* out;
    long long ldo;
    float* part_o;        // [2 kMaxCtas][block rows][D]
    float2* part_ml;      // [2 kMaxCtas][block rows]
    Place* places;        // [CTAs + 1]: where the shares begin
    float c;              // scale log2(e)
    unsigned long long wait_ns;
};

// -------------------------------------------------------- the matrix warp ----
// A ring's entries in their order: K tiles run ahead of V's, by one where two streams share the tiles, else by two.
template <class Sh, class Src>
struct Feed {
    Walk<Sh, Src> walk;
    Item x;
    int n = 0, lead = 0, k = 0, v = 0, e = Sh::kEntries, number = 0;
    bool value = false;   // the entry is of V
    int tile = 0;         // of the share's part of the block

    __device__ Feed(const Src& p, const Place* cut, int cta) : walk(p, cut, cta) {}
    __device__ bool next() {
        if (++e < Sh::kEntries) return true;
        e = 0;
        while (v == n) {
            if (!walk.next(x)) return false;
            n = x.hi - x.lo;
            lead = Sh::lead(x.rows);
            k = v = 0;
            if (n > 0) ++number;
        }
        value = k == min(n, v + lead);
        tile = value ? v++ : k++;
        return true;
    }
    // first token of the entry
    __device__ int token() const { return (x.lo + tile) * Sh::kTile + e * Sh::kEntry; }
};

// Ring entries: STAGES of Shape<D>::kEntryBytes at `ring`; queries of a stream at q + stream * kQBytes.
template <int D, int STAGES, class Src>
__device__ __forceinline__ void matrix_warp(const Src& p, Control& c, uint32_t q, uint32_t ring) {
    using X = Shape<D>;
    constexpr int E = X::kEntries;
    constexpr uint32_t kIdS = (1u << 4) | ((uint32_t)(X::kEntry >> 3) << 17) | ((uint32_t)(kRowsQ >> 4) << 24);
    constexpr uint32_t kIdO = (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kRowsQ >> 4) << 24);
    const uint32_t tm = c.tmem;
    Walk<Shape<D>, Src> walk(p, c.cut, blockIdx.x);
    Item x;
    int base = 0;                               // ring entries before the block's, in tiles
    uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0};
    const uint32_t lead_lane = elect();
    while (walk.next(x)) {
        const int n = x.hi - x.lo;
        if (n == 0) continue;
        const bool pair = x.pair<D>();
        const int lead = pair ? 1 : 2;
        auto scores = [&](int s, int i, int buf, bool release, bool last) {        // of the share's tile i
            bool ok = true;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int at = (base + k_entry(i, lead)) * E + e, stage = at % STAGES;
                ok = wait_phase(&c.full[stage], (at / STAGES) & 1, c.dead, p.o.wait_ns);
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t a = desc_lo(q + s * X::kQBytes, 16), b = desc_lo(ring + stage * X::kEntryBytes, 16);
                const uint32_t d = tm + buf * kTile + e * X::kEntry;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_ss(d, desc128(a + (ks >> 2) * (kRowsQ * 128 / 16) + (ks & 3) * 2),
                           desc128(b + (ks >> 2) * (X::kEntry * 128 / 16) + (ks & 3) * 2), kIdS, ks > 0, lead_lane);
                if (release) commit(&c.freed[stage], lead_lane);
            }
            if (ok) commit(&c.s_full[buf], lead_lane);
            if (ok && last) commit(&c.q_freed[s], lead_lane);
        };
        auto values = [&](int s, int i, int j, int buf, bool release, bool last) {
            bool ok = wait_phase(&c.p_full[buf], n_p[buf] & 1, c.dead, p.o.wait_ns);
            ++n_p[buf];
            const uint32_t d = tm + X::kO + s * D;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int at = (base + v_entry(i, lead, n)) * E + e, stage = at % STAGES;
                ok = ok && wait_phase(&c.clean[stage], (at / STAGES) & 1, c.dead, p.o.wait_ns);
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t b = desc_lo(ring + stage * X::kEntryBytes, X::kEntry * 128);
#pragma unroll
                for (int kk = 0; kk < X::kEntry / 16; ++kk)
                    mma_ts(d, tm + buf * kTile + (e * (X::kEntry / 16) + kk) * 8, desc128(b + kk * (2048 / 16)), kIdO,
                           j > 0 || e > 0 || kk > 0, lead_lane);
                if (release) commit(&c.freed[stage], lead_lane);
            }
            if (ok && X::kStreams == 1) commit(&c.o_step[buf], lead_lane);
            if (ok && last) commit(&c.o_last[s], lead_lane);
        };
        if constexpr (X::kStreams == 2) {
            const int n1 = x.of_stream<D>(1), n0 = x.of_stream<D>(0);
            auto tile = [&](int s, int j) { return x.tile_of<D>(s, j) - x.lo; };
            wait_phase(&c.q_full[0], n_q[0]++ & 1, c.dead, p.o.wait_ns);
            scores(0, 0, 0, !pair, n0 == 1);
            if (n1) {
                wait_phase(&c.q_full[1], n_q[1]++ & 1, c.dead, p.o.wait_ns);
                scores(1, tile(1, 0), 1, true, n1 == 1);
            }
            for (int j = 0; j < n0; ++j) {
                values(0, tile(0, j), j, 0, !pair, j + 1 == n0);
                if (j + 1 < n0) scores(0, tile(0, j + 1), 0, !pair, j + 2 == n0);
                if (j < n1) {
                    values(1, tile(1, j), j, 1, true, j + 1 == n1);
                    if (j + 1 < n1) scores(1, tile(1, j + 1), 1, true, j + 2 == n1);
                }
            }
        } else {
            wait_phase(&c.q_full[0], n_q[0]++ & 1, c.dead, p.o.wait_ns);
            // (a block's tile i has the score buffer (base + i) % 2: base counts two tiles, K's and V's, for each)
            const int g = base / 2;
            scores(0, 0, g & 1, true, n == 1);
            for (int j = 0; j < n; ++j) {
                if (j + 1 < n) scores(0, j + 1, (g + j + 1) & 1, true, j + 2 == n);
                values(0, j, j, (g + j) & 1, true, j + 1 == n);
            }
        }
        base += 2 * n;
    }
}

// ------------------------------------------------- the softmax warpgroups ----
// References whose fp32 step is 1/2 or more.  The product S c in full, less a reference that is one rounded, may be half a step above
// zero for the largest score itself, and a weight beyond fp16; rounded before the reference comes off, as the
// reference was, it is not.  (Such scores are good to a few steps, whichever way they are formed.)
__device__ __forceinline__ bool is_far(float ref) { return fabsf(ref) >= 0x1p22f && ref != -INFINITY; }

// Thread: one row of stream s.
template <int D, class Src>
__device__ __forceinline__ void softmax_warps(const Src& p, Control& c, char* q_smem, char* stage_smem) {
    using X = Shape<D>;
    const int s = threadIdx.x >> 7, quad = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, row = threadIdx.x & 127;
    if (s >= X::kStreams) return;
    const uint32_t tm = c.tmem + ((uint32_t)(32 * quad) << 16), o_at = tm + X::kO + s * D;
    char* my_q = q_smem + s * X::kQBytes;
    Walk<Shape<D>, Src> walk(p, c.cut, blockIdx.x);
    Item x;
    uint32_t n_s[2] = {0, 0}, n_last = 0;
    int base = 0, number = 0;
    while (walk.next(x)) {
        if (x.hi > x.lo) ++number;
        const bool pair = x.pair<D>();
        const int n = x.of_stream<D>(s);
        // (of a block of one row tile the second stream turns its rows by 64, so that few rows fall to other
        // quarters of the multiprocessor than the first's)
        const int local = pair ? s * kRowsQ + row : row ^ (64 * s);
        const bool live = local < x.rows, idle = (local & ~31) >= x.rows;
        const int at = x.row0 + (live ? local : 0), token = at / p.G, head = x.h * p.G + at - token * p.G;
        const float cc = p.o.c;                  // from a score to the exponent
        if (n > 0 && !p.q_copied) {
            p.load_queries(x, live, token, head, my_q, row);
            tc::fence_async_smem();
            mbar_arrive(&c.q_full[s]);
        }
        float ref = -INFINITY, l = 0.f;
        bool ok = true, far = false;
        for (int j = 0; j < n; ++j) {
            const int buf = X::kStreams == 2 ? s : (base + j) & 1;
            const uint32_t s_at = tm + buf * kTile;
            ok = wait_phase(&c.s_full[buf], n_s[buf] & 1, c.dead, p.o.wait_ns);
            ++n_s[buf];
            if (!ok) continue;
            if (idle) {                              // no row of this warp's: whatever lies there
                if (lane == 0) mbar_arrive(&c.p_full[buf]);
                continue;
            }
            tc::fence_after_sync();
            uint32_t v[kTile];
#pragma unroll
            for (int k = 0; k < kTile; k += 32) tmem_ld32(s_at + k, v + k);
            tc::tmem_wait_ld();
            const int tile = x.tile_of<D>(s, j);
            if (tile >= x.clear) {
#pragma unroll
                for (int k = 0; k < kTile; k += 32) {
                    const uint32_t seen = p.seen_word(x, token, tile * kTile + k);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((seen >> i) & 1)) v[k + i] = 0xff800000u;      // -infinity
                }
            }
            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < kTile; k += 8)
#pragma unroll
                for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], fmaxf(__uint_as_float(v[k + 2 * i]), __uint_as_float(v[k + 2 * i + 1])));
            const float most = __fmul_rn(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), cc);
            const bool move = most - ref > kRise;
            if (__any_sync(0xffffffffu, move || far)) {
                const float to = move ? most : ref, f = to == ref ? 1.f : ex2(ref - to);
                l *= f;
                ref = to;
                far = is_far(ref);
                if (__any_sync(0xffffffffu, move)) {
                    if (X::kStreams == 1 && j > 0) {
                        // the product of the tile before, the other buffer's latest (with two streams it was issued
                        // before these scores)
                        const int g = base + j - 1;
                        ok = wait_phase(&c.o_step[g & 1], (g >> 1) & 1, c.dead, p.o.wait_ns);
                        tc::fence_after_sync();
                    }
                    if (j > 0) {
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            uint32_t o[32];
                            tmem_ld32(o_at + k, o);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(o_at + k, o);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, far)) {
                    // rounded exponents less the reference in the scores' place, 32 at a time (all in registers, next to the
                    // scores, cost calls without such rows 2 to 4 %); intrinsics: never one fused step
#pragma unroll 1
                    for (int k = 0; k < kTile; k += 32) {
                        uint32_t o[32];
                        tmem_ld32(s_at + k, o);
                        tc::tmem_wait_ld();
                        const uint32_t seen = tile >= x.clear ? p.seen_word(x, token, tile * kTile + k) : 0xffffffffu;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float e = (seen >> i) & 1 ? __uint_as_float(o[i]) : -INFINITY;
                            o[i] = __float_as_uint(far ? __fsub_rn(__fmul_rn(e, cc), ref) : e);
                        }
                        tmem_st32(s_at + k, o);
                    }
                    tmem_wait_st();
#pragma unroll
                    for (int k = 0; k < kTile; k += 32) tmem_ld32(s_at + k, v + k);
                    tc::tmem_wait_ld();
                }
            }
            const float by = far ? 1.f : cc, sub = far ? kUp : ref == -INFINITY ? 0.f : kUp - ref;
            const f2 c2 = pk(by, by), sub2 = pk(sub, sub);
            f2 sum[2] = {0, 0};
#pragma unroll
            for (int k = 0; k < kTile; k += 2) {
                float a, b;
                unpk(fma2(pk(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2, sub2), a, b);
                a = ex2(a);
                b = ex2(b);
                sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pk(a, b));
                v[k >> 1] = pack2(a, b);
                if ((k & 63) == 62) tmem_st32(s_at + (k >> 6) * 32, v + (k >> 6) * 32);
            }
            float a, b;
            unpk(add2(sum[0], sum[1]), a, b);
            l += a + b;
            tmem_wait_st();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c.p_full[buf]);
        }
        if (X::kStreams == 1) base += n;
        if (n > 0) {
            ok = wait_phase(&c.o_last[s], n_last++ & 1, c.dead, p.o.wait_ns) && ok;
            tc::fence_after_sync();
        }
        if (!ok) l = __int_as_float(0x7fffffff);

        // a block of one row tile: the second stream's sums and accumulator come through its staging memory
        float f0 = 1.f, f1 = 0.f;
        const bool merge = X::kStreams == 2 && !pair && x.of_stream<D>(1) > 0;
        if (merge) {
            if (s == 1) c.ml[local] = make_float2(ref, l);
            named_bar_sync(1, kSoftmax);
            if (s == 0) {
                const float2 other = c.ml[local];
                const float top = fmaxf(ref, other.x);
                if (top != -INFINITY) {
                    f0 = ex2(ref - top);
                    f1 = ex2(other.x - top);
                }
                l = l * f0 + other.y * f1;      // (a sum of NaN stays one)
                ref = top;
            }
        }
        // (read only here: the first stream adds what the rows see of both streams' V tiles, and the second one's last has
        // been looked through for certain when that stream's last product is done)
        const bool fix = n > 0 && special_of(c, number) == number;
        const bool whole = x.part < 0;
        // (a row without weights: of finite values, those of V that it does not see among them; an l of NaN stays one)
        const float inv = l == 0.f ? 0.f : 1.f / l;
        __half* out = p.o.out + (long long)(x.s.q0 + token) * p.o.ldo + (long long)head * D;
        float* part = p.o.part_o + ((long long)x.part * X::kBlock + local) * D;
        const bool writes = live && (s == 0 || pair);
        float* swap = reinterpret_cast<float*>(stage_smem + kStageBytes);               // [32][kRowsQ], the second stream's
        char* stage = stage_smem + s * kStageBytes + 4096 * quad;                       // the warp's [32 rows][64 dims], swizzled
        // rows that the lane writes 8 dims of at a time: eight lanes a row (a row per lane would take a line per lane and access)
        __half* row_out[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            row_out[i] = reinterpret_cast<__half*>(
                __shfl_sync(0xffffffffu, writes && whole ? (unsigned long long)out : 0ull, 4 * i + (lane >> 3)));
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
            if (merge) {
                if (s == 1) {
                    uint32_t o[32];
                    tmem_ld32(o_at + k, o);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) swap[e * kRowsQ + local] = __uint_as_float(o[e]);
                }
                named_bar_sync(3, kSoftmax);
            }
            if (X::kStreams == 1 || pair || s == 0) {
                float o[32];                            // dims k .. k + 31
                if (n > 0) {
                    uint32_t raw[32];
                    tmem_ld32(o_at + k, raw);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(raw[i]);
                    if (merge) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = o[i] * f0 + swap[i * kRowsQ + local] * f1;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0.f;
                }
                if (fix && live) p.add_special(x, token, k, o);
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float u, v;
                            unpk(mul2(pk(o[i + 2 * e], o[i + 2 * e + 1]), pk(inv, inv)), u, v);
                            w[e] = pack2(u, v);
                        }
                        *reinterpret_cast<uint4*>(stage + swizzled(lane, ((k & 32) + i) >> 3)) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    if (k & 32) {                       // 64 dims of the warp's rows are there
                        __syncwarp();
                        uint4 w[8];                     // (all under way together)
#pragma unroll
                        for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint4*>(stage + swizzled(4 * i + (lane >> 3), lane & 7));
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (row_out[i]) *reinterpret_cast<uint4*>(row_out[i] + (k & ~32) + 8 * (lane & 7)) = w[i];
                        __syncwarp();
                    }
                } else if (writes) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<float4*>(part + k + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
            }
            if (merge) named_bar_sync(2, kSoftmax);                 // the second stream's dims have been read
        }
        if (writes && !whole) p.o.part_ml[(long long)x.part * X::kBlock + local] = make_float2(ref, l);
        tc::fence_before_sync();
    }
}

// Start of a CTA.  Barriers' counts: arrivals of a ring entry's copy, of those that have looked it through, of those that
// are done with it, of a stream's queries.
__device__ __forceinline__ void control_init(Control& c, int full_count, int clean_count, int free_count, int q_count, bool dead) {
    for (int i = 0; i < kMaxStages; ++i) {
        mbar_init(&c.full[i], full_count);
        mbar_init(&c.clean[i], clean_count);
        mbar_init(&c.freed[i], free_count);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(&c.q_full[i], q_count);
        mbar_init(&c.q_freed[i], 1);
        mbar_init(&c.s_full[i], 1);
        mbar_init(&c.p_full[i], 4);
        mbar_init(&c.o_last[i], 1);
        mbar_init(&c.o_step[i], 1);
    }
    mbar_init(&c.drained, 1);
    fence_mbar_init();
    c.dead = dead;
    c.q_loads[0] = c.q_loads[1] = c.issued = 0;
    for (int i = 0; i < kMaxStages * 2; ++i) c.special[i] = 0;
}

// ------------------------------------------------------------------- join ----
// A CTA of 16 warps: 32 rows of the block that the cut in front of share blockIdx.x + 1 is the first to fall into, a warp
// each, a few parts under way at a time (it is the latency of reads that wait for one another that counts).
constexpr int kJoinWarps = 16;
template <class Sh, class Src>
__global__ void __launch_bounds__(32 * kJoinWarps) flash_join(const Src p) {
    constexpr int D = Sh::kD, kN = D / 32, R = Sh::kBlock, kBatch = D == 256 ? 4 : 8;
    wait_predecessor();
    launch_dependents();
    const int i = blockIdx.x + 1, ctas = gridDim.x + 1, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const Place before = p.o.places[i - 1], at = p.o.places[i];
    if (at.tile == 0 || (before.tile > 0 && same_block(before, at))) return;
    int last = i;                                   // the last share that begins in the block
    for (int from = i + 1; from < ctas; from += 32) {
        bool in = false;
        if (from + lane < ctas) {
            const Place z = p.o.places[from + lane];
            in = z.tile > 0 && same_block(z, at);
        }
        const unsigned ins = __ballot_sync(0xffffffffu, in);
        last += ins == 0xffffffffu ? 32 : __ffs(~ins) - 1;
        if (ins != 0xffffffffu) break;
    }
    const Seq s = p.seq(at.b);
    const int row0 = at.t * R, rows = min(R, s.n_q * p.G - row0), parts = last - i + 2;
    for (int local = blockIdx.y * 32 + wid; local < min(rows, blockIdx.y * 32 + 32); local += kJoinWarps) {
        auto slot = [&](int k) { return (long long)(2 * (i - 1 + k) + (k == 0 ? 1 : 0)) * R + local; };
        float top = -INFINITY;
        for (int k = lane; k < parts; k += 32) top = fmaxf(top, p.o.part_ml[slot(k)].x);
#pragma unroll
        for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        float v[kN], l = 0.f;
#pragma unroll
        for (int e = 0; e < kN; ++e) v[e] = 0.f;
        for (int k0 = 0; k0 < parts; k0 += kBatch) {
            float part[kBatch][kN];
            float2 ml[kBatch];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (k0 + u >= parts) break;
                ml[u] = p.o.part_ml[slot(k0 + u)];
                const float* o = p.o.part_o + slot(k0 + u) * D;
#pragma unroll
                for (int e = 0; e < kN; ++e) part[u][e] = o[e * 32 + lane];
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                if (k0 + u >= parts) break;
                const float f = ml[u].x == -INFINITY ? 0.f : ex2(ml[u].x - top);
                l += ml[u].y != ml[u].y ? ml[u].y : ml[u].y * f;
#pragma unroll
                for (int e = 0; e < kN; ++e) v[e] = fmaf(part[u][e], f, v[e]);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int r = row0 + local, token = r / p.G, head = at.h * p.G + r - token * p.G;
        __half* out = p.o.out + (long long)(s.q0 + token) * p.o.ldo + (long long)head * D;
#pragma unroll
        for (int e = 0; e < kN; ++e) out[e * 32 + lane] = __float2half_rn(v[e] * inv);
    }
}

// workspace: places, parts' statistics, parts
template <class Sh>
inline long long workspace_bytes() {
    return (long long)(kMaxCtas + 1) * sizeof(Place) + 15 + 2ll * kMaxCtas * Sh::kBlock * (Sh::kD * 4 + 8) + 16;
}
template <class Sh>
inline void lay_out(char* ws, Out* o) {
    o->places = (Place*)ws;
    char* at = ws + ((kMaxCtas + 1) * sizeof(Place) + 15) / 16 * 16;
    o->part_ml = (float2*)at;
    o->part_o = (float*)(at + 2ll * kMaxCtas * Sh::kBlock * 8);
}

}  // namespace flash
}  // namespace edge0
