// Moves inside the quantised KV cache: kept rows drawn together (accepted drafts, evicted
// contexts), whole pages copied (forks).  Codes and (s, b) pairs move as they are.
//
// Copies of pages are bound by the bytes; rows by reads that depend on one another (row number, page numbers, the
// row), a chunk of rows after the other.  Accepted ones of 64 sequences' 16 drafted tokens, 8 heads of
// 128 dims in 4 bits: 4.5 us, hardly more than an empty kernel's.  A quarter of 7 contexts of 8,191 tokens in 8 bits: 19.5 us
// for 31 MB: the longest sequence's CTAs go through ten chunks while the others have ended.  1,000 pages copied eight times over:
// 131 to 140 us for 664 MB, 70 to 74 % of what a plain copy moves.
#include "kvcache.cuh"
#include "launch.cuh"

namespace edge0 {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 2;             // rows that a thread has under way

struct CompactP {
    kv::View c;
    const int* table;
    int W;
    const int* start;
    const int* src;                      // [T]
    const int* cu;                       // [B + 1] or null: row b belongs to sequence b
    int T;
    int* status;
};

// One CTA: a (sequence, head, K or V).  A row goes to a place at or before its own, so no row's source is the
// destination of one before it: it is enough that the CTA has read a chunk of rows before it writes them,
// and chunks follow in order.  A chunk is read while the one before is still to be written, its rows' places are
// looked up before that.
template <int BITS, int D, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_compact_kernel(const CompactP p) {
    constexpr int kR = kv::row_bytes(BITS, D), kSb = kv::sb_bytes(D), kPieces = kR / 16 + 1;
    constexpr int kPar = THREADS / kPieces, kChunk = kPar * kMoveRows;
    constexpr int kStripBytes = kv::strip_bytes(BITS, D), kHalf = kv::half_bytes(BITS, D);
    __shared__ long long from_s[2][kChunk], to_s[2][kChunk];         // strip's offset | row of the strip, or -1: nothing to do
    wait_predecessor();
    launch_dependents();
    const int h = blockIdx.x >> 1, half = blockIdx.x & 1, b = blockIdx.y;
    const int begin = p.cu ? p.cu[b] : b, start = p.start[b];
    const int first = max(begin, 0), last = p.cu ? min(p.cu[b + 1], p.T) : b + 1;
    if (start < 0 || last <= first) return;
    const unsigned lo = first, hi = last;            // (a few chunks behind 2^31 - 1 rows still count up)
    const int sub = threadIdx.x / kPieces, piece = threadIdx.x - sub * kPieces;
    const bool idle = sub >= kPar, pairs = piece == kPieces - 1;     // the row's (s, b) pairs come last
    char* base = p.c.pages + (long long)h * (p.c.page_tokens / kv::kStrip) * kStripBytes + half * kHalf;
    auto strip_of = [&](unsigned pos) -> long long {
        const unsigned pg = pos / (unsigned)p.c.page_tokens;
        if (pg >= (unsigned)p.W) return -1;
        const int id = p.table[(long long)b * p.W + pg];
        if (id < 0 || id >= p.c.n_pages) return -1;
        const unsigned token = pos - pg * p.c.page_tokens;
        return id * p.c.page_bytes + (long long)(token / kv::kStrip) * kStripBytes + token % kv::kStrip;
    };
    auto look = [&](unsigned r0, int buf) {
        for (int i = threadIdx.x; i < kChunk; i += THREADS) {
            const unsigned r = r0 + i;
            long long from = -1, to = -1;
            if (r < hi) {
                const long long dst = (long long)start + r - begin;
                const int src = p.src[r];
                if (src != dst) {
                    if (src > dst) {
                        to = strip_of((unsigned)dst);
                        from = strip_of((unsigned)src);
                    }
                    if (to < 0 || from < 0) {
                        to = -1;
                        if (p.status && h == 0 && half == 0) atomicExch(p.status, EDGE0_EINVAL);
                    }
                }
            }
            from_s[buf][i] = from;
            to_s[buf][i] = to;
        }
    };
    auto place = [&](long long strip) -> char* {
        const int row = (int)(strip & 15);
        return base + (strip - row) + (pairs ? kv::kStrip * kR + row * kSb : row * kR + ((piece ^ kv::turn(kR, row)) << 4));
    };
    uint4 v[2][kMoveRows];
    char* to[2][kMoveRows];
    auto load = [&](int buf, uint4 (&v)[kMoveRows], char* (&to)[kMoveRows]) {
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            to[u] = nullptr;
            if (idle || to_s[buf][sub + u * kPar] < 0) continue;
            to[u] = place(to_s[buf][sub + u * kPar]);
            const char* s = place(from_s[buf][sub + u * kPar]);
            if (!pairs) v[u] = *reinterpret_cast<const uint4*>(s);
            else if (kSb == 4) v[u].x = *reinterpret_cast<const uint32_t*>(s);
            else if (kSb == 8) *reinterpret_cast<uint2*>(&v[u]) = *reinterpret_cast<const uint2*>(s);
            else v[u] = *reinterpret_cast<const uint4*>(s);
        }
    };
    auto store = [&](const uint4 (&v)[kMoveRows], char* const (&to)[kMoveRows]) {
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            if (!to[u]) continue;
            if (!pairs) *reinterpret_cast<uint4*>(to[u]) = v[u];
            else if (kSb == 4) *reinterpret_cast<uint32_t*>(to[u]) = v[u].x;
            else if (kSb == 8) *reinterpret_cast<uint2*>(to[u]) = make_uint2(v[u].x, v[u].y);
            else *reinterpret_cast<uint4*>(to[u]) = v[u];
        }
    };
    look(lo, 0);
    __syncthreads();
    load(0, v[0], to[0]);
    if (lo + kChunk < hi) look(lo + kChunk, 1);
    for (unsigned r0 = lo;; r0 += 2 * kChunk) {
        __syncthreads();                         // chunk r0 has been read by all, the next one's places are there
        if (r0 + kChunk < hi) {
            load(1, v[1], to[1]);
            look(r0 + 2 * kChunk, 0);
        }
        store(v[0], to[0]);
        if (r0 + kChunk >= hi) break;
        __syncthreads();
        if (r0 + 2 * kChunk < hi) {
            load(0, v[0], to[0]);
            look(r0 + 3 * kChunk, 1);
        }
        store(v[1], to[1]);
        if (r0 + 2 * kChunk >= hi) break;
    }
}

struct CopyP {
    kv::View c;
    const int* src;
    const int* dst;
    int n, parts;                        // pages, parts of a page
    int* status;
};

constexpr int kCopyVec = 8;              // 16-byte loads that a thread has under way
constexpr int kCopyPart = kMoveThreads * kCopyVec;      // pieces of 16 bytes of a part, at most

__global__ void __launch_bounds__(kMoveThreads) kv_copy_pages_kernel(const CopyP p) {
    wait_predecessor();
    launch_dependents();
    const long long units = (long long)p.n * p.parts;
    for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
        // (all pages' first parts, then their second ones: a page that several copies read is asked for again after a part of
        // all pages instead of after all of them, when it is still in the L2: 348 MB of reads -> 193, 144 us -> 131)
        const int part = (int)(unit / p.n), e = (int)(unit - (long long)part * p.n);
        const int s = p.src[e], d = p.dst[e];
        if (s < 0 || d < 0 || s == d) continue;          // (-1: an entry that asks for nothing)
        if (s >= p.c.n_pages || d >= p.c.n_pages) {
            if (p.status && part == 0 && threadIdx.x == 0) atomicExch(p.status, EDGE0_EINVAL);
            continue;
        }
        // parts of one length, so that none is nearly empty
        const int pieces = (int)(p.c.page_bytes / 16), each = (pieces + p.parts - 1) / p.parts, first = part * each;
        const int n = min(each, pieces - first);
        const uint4* from = reinterpret_cast<const uint4*>(p.c.pages + s * p.c.page_bytes) + first;
        uint4* to = reinterpret_cast<uint4*>(p.c.pages + d * p.c.page_bytes) + first;
        uint4 v[kCopyVec];
#pragma unroll
        for (int u = 0; u < kCopyVec; ++u)
            if (u * kMoveThreads + (int)threadIdx.x < n) v[u] = from[u * kMoveThreads + threadIdx.x];
#pragma unroll
        for (int u = 0; u < kCopyVec; ++u)
            if (u * kMoveThreads + (int)threadIdx.x < n) __stcs(&to[u * kMoveThreads + threadIdx.x], v[u]);      // (sources stay in the L2)
    }
}

template <int BITS, int D>
int launch_compact(const CompactP& p, int B, cudaStream_t stream) {
    // few rows per sequence: small CTAs, so that many fit; many: as many threads as there are, for chunks follow one another
    // (7 contexts of 8,191 tokens of which up to 2,047 are kept, 256 and 1,024 threads: 27 and 19.6 us)
    if (p.T / B <= 64) return launch_early(kv_compact_kernel<BITS, D, 256>, dim3(2 * p.c.H, B), 256, 0, stream, p);
    return launch_early(kv_compact_kernel<BITS, D, 1024>, dim3(2 * p.c.H, B), 1024, 0, stream, p);
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" int edge0_kv_compact(const edge0_kv_cache* cache, const int32_t* table, int B, int W, const int32_t* start,
                                const int32_t* src, const int32_t* cu_rows, int T, int* status, cudaStream_t stream) {
    CompactP p;
    const int rc = kv::view_of(cache, &p.c);
    if (rc) return rc;
    if (!table || !start || B <= 0 || B > EDGE0_MAX_BATCHED || W <= 0 || T < 0 || (!cu_rows && T != B)) return EDGE0_EINVAL;
    if (T == 0) return EDGE0_OK;
    if (!src) return EDGE0_EINVAL;
    if (((uintptr_t)table | (uintptr_t)start | (uintptr_t)src | (uintptr_t)cu_rows | (uintptr_t)status) & 3) return EDGE0_EINVAL;
    p.table = table;
    p.W = W;
    p.start = start;
    p.src = src;
    p.cu = cu_rows;
    p.T = T;
    p.status = status;
    const int D = cache->head_dim;
    if (cache->bits == 4)
        return D == 64    ? launch_compact<4, 64>(p, B, stream)
               : D == 128 ? launch_compact<4, 128>(p, B, stream)
                          : launch_compact<4, 256>(p, B, stream);
    return D == 64    ? launch_compact<8, 64>(p, B, stream)
           : D == 128 ? launch_compact<8, 128>(p, B, stream)
                      : launch_compact<8, 256>(p, B, stream);
}

extern "C" int edge0_kv_copy_pages(const edge0_kv_cache* cache, const int32_t* src, const int32_t* dst, int n, int* status,
                                   cudaStream_t stream) {
    CopyP p;
    const int rc = kv::view_of(cache, &p.c);
    if (rc) return rc;
    if (n < 0) return EDGE0_EINVAL;
    if (n == 0) return EDGE0_OK;
    if (!src || !dst || (((uintptr_t)src | (uintptr_t)dst | (uintptr_t)status) & 3)) return EDGE0_EINVAL;
    p.src = src;
    p.dst = dst;
    p.n = n;
    p.parts = (int)((p.c.page_bytes / 16 + kCopyPart - 1) / kCopyPart);
    p.status = status;
    const long long units = (long long)n * p.parts, most = 152 * 8;
    return launch_early(kv_copy_pages_kernel, dim3((unsigned)(units < most ? units : most)), kMoveThreads, 0, stream, p);
}
