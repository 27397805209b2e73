// Moves inside the quantised KV cache: kept rows drawn together (accepted drafts, evicted
// contexts), whole pages copied (forks).  Codes and (s, b) pairs move as they are.
//
// Both are bound by the bytes read and written, or by a few dependent reads where there is
// little to move (row number, page numbers, the row).
#include "kvcache.cuh"
#include "launch.cuh"

namespace edge0 {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;             // rows that a thread has under way

struct CompactP {
    kv::View c;
    const int* table;
    int W;
    const int* start;
    const int* src;                      // [T]
    const int* cu;                       // [B + 1] or null: row b belongs to sequence b
    int T;
    int splits;                          // CTAs that share the pieces of a (sequence, head, half)
    int* status;
};

// One CTA: some of the 16-byte pieces of one (sequence, head, K or V).  A row goes to a place
// at or before its own, so no row's source is the destination of one before it: it is enough that
// the CTA has read a chunk of rows before it writes them, and chunks follow in order.
template <int BITS, int D>
__global__ void __launch_bounds__(kMoveThreads) kv_compact_kernel(const CompactP p) {
    constexpr int kR = kv::row_bytes(BITS, D), kCh = kR / 16, kSb = kv::sb_bytes(D), kPieces = kCh + 1;
    constexpr int kStripBytes = kv::strip_bytes(BITS, D), kHalf = kv::half_bytes(BITS, D);
    wait_predecessor();
    launch_dependents();
    const int split = blockIdx.x % p.splits, half = (blockIdx.x / p.splits) & 1;
    const int h = blockIdx.y, b = blockIdx.z;
    const int lo = p.cu ? max(p.cu[b], 0) : b, hi = p.cu ? min(p.cu[b + 1], p.T) : b + 1;
    const int begin = p.cu ? p.cu[b] : b, start = p.start[b];
    if (start < 0 || hi <= lo) return;
    const int p0 = split * kPieces / p.splits, mine = (split + 1) * kPieces / p.splits - p0;
    const int par = kMoveThreads / mine, sub = threadIdx.x / mine, piece = p0 + threadIdx.x - sub * mine;
    const bool idle = sub >= par;
    const bool pairs = piece == kCh;     // the row's (s, b) pairs
    const bool tells = p.status && split == 0 && half == 0 && h == 0 && threadIdx.x == sub * mine;
    // where the thread's piece of a position lies, or null
    auto place = [&](long long pos) -> char* {
        const long long pg = pos / p.c.page_tokens;
        if (pos < 0 || pg >= p.W) return nullptr;
        const int id = p.table[(long long)b * p.W + pg];
        if (id < 0 || id >= p.c.n_pages) return nullptr;
        const int token = (int)(pos - pg * p.c.page_tokens), row = token % kv::kStrip;
        char* at = p.c.pages + id * p.c.page_bytes +
                   ((long long)h * (p.c.page_tokens / kv::kStrip) + token / kv::kStrip) * kStripBytes + half * kHalf;
        return at + (pairs ? kv::kStrip * kR + row * kSb : row * kR + ((piece ^ kv::turn(kR, row)) << 4));
    };
    uint4 v[2][kMoveRows];
    char* to[2][kMoveRows];
    auto load = [&](int r0, uint4 (&v)[kMoveRows], char* (&to)[kMoveRows]) {
#pragma unroll
        for (int u = 0; u < kMoveRows; ++u) {
            const int r = r0 + sub + u * par;
            to[u] = nullptr;
            if (idle || r >= hi) continue;
            const long long dst = (long long)start + r - begin, src = p.src[r];
            if (src == dst) continue;
            char* t = src > dst ? place(dst) : nullptr;
            const char* s = src > dst ? place(src) : nullptr;
            if (!t || !s) {
                if (tells) atomicExch(p.status, EDGE0_EINVAL);
                continue;
            }
            to[u] = t;
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
    // a chunk is read while the one before is still to be written: what that one writes lies in front of its sources
    const int chunk = par * kMoveRows;
    load(lo, v[0], to[0]);
    for (int r0 = lo; r0 < hi; r0 += 2 * chunk) {
        load(r0 + chunk, v[1], to[1]);
        __syncthreads();
        store(v[0], to[0]);
        if (r0 + chunk >= hi) break;
        load(r0 + 2 * chunk, v[0], to[0]);
        __syncthreads();
        store(v[1], to[1]);
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
        const int e = (int)(unit / p.parts), part = (int)(unit - (long long)e * p.parts);
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
            if (u * kMoveThreads + (int)threadIdx.x < n) to[u * kMoveThreads + threadIdx.x] = v[u];
    }
}

template <int BITS, int D>
int launch_compact(CompactP p, int B, cudaStream_t stream) {
    constexpr int kPieces = kv::row_bytes(BITS, D) / 16 + 1;
    // CTAs that share a (sequence, head, half): until four per SM are there; each a piece at least
    const long long ctas = (long long)B * p.c.H * 2;
    const long long want = (608 + ctas - 1) / ctas;
    p.splits = want > kPieces ? kPieces : (int)want;
    return launch_early(kv_compact_kernel<BITS, D>, dim3(2 * p.splits, p.c.H, B), kMoveThreads, 0, stream, p);
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
