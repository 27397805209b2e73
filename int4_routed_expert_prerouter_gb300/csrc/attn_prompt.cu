// Causal attention of packed prompts: the rows of each sequence are the queries of its last n_q of n_k
// tokens, and row i sees the keys up to i + n_k - n_q.  The mathematics, the blocks and their shares: flash.cuh.
//
// Warps: 0-7 softmax, 8 the matrix steps, 9 K and V by TMA (tiles of 128 tokens, 64 of 256-wide heads, through a ring of
// 4 entries of 32 KB, of 8 of 16 KB for 64-wide heads), 10 and 11 look the V tiles through that some
// row does not see in whole: a weight of zero times an infinity or NaN would be NaN.  They put zeros
// in place of such values and of other sequences' rows behind the last key; what the rows see of them is added
// to the sums at the end.
//
// What bounds it.  Long prompts: a stream's chain of scores, weights and product (about 2,900 cycles a tile, of which
// the tensor core works 2,048 for both streams) and the power it takes; 16,384 tokens, 32 heads of 128: 1,420 to 1,580 us with
// the clocks, 1,390 to 1,550 TFLOP/s.  Short ones: a block's start and end; 64 prompts of up to 1,024 tokens 263 us, of
// which each CTA spends a fifth on outputs (their reads from staging one by one instead of together, and a look at
// empty rows apart: 279 instead of 269).  One prompt of 131 tokens, heads of 256: 10 us.  Weights formed before the maximum is
// known, and the maximum looked for only of too large a sum, gained nothing (273 instead of 269 at that time).
#include "flash.cuh"

#include <cuda.h>

namespace edge0 {
namespace {

using namespace flash;

constexpr int kThreadsF = kSoftmax + 128;

// What does not depend on the head's width.
struct PromptP {
    Out o;
    const __half* q;
    const __half* v;
    long long ldq, ldv;
    int B, H, G, T, Tk;
    const int* cu_q;
    const int* cu_k;
    bool q_copied;                     // queries come by TMA: 64 rows are whole tokens' groups
};

template <int D>
struct Prompt : PromptP {
    // (numbers outside [0, T] are cut, so that nothing beside the rows is touched whatever they say)
    __device__ Seq seq(int b) const {
        Seq s;
        s.q0 = min(max(cu_q[b], 0), T);
        s.n_q = min(max(cu_q[b + 1], s.q0), T) - s.q0;
        s.k0 = min(max(cu_k[b], 0), Tk);
        s.n_k = min(max(cu_k[b + 1], s.k0), Tk) - s.k0;
        s.off = s.n_k - s.n_q;
        s.ctx = 0;
        return s;
    }
    __device__ static int seen(const Seq& s, int token) { return min(max(token + 1 + s.off, 0), s.n_k); }
    __device__ static int seen_by_all(const Seq& s, int token) { return seen(s, token); }

    // which of the tokens from .. from + 31 a row sees, as bits
    __device__ static uint32_t seen_word(const Item& x, int token, int from) {
        const int k = seen(x.s, token) - from;
        return k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1;
    }

    __device__ void load_queries(const Item& x, bool live, int token, int head, char* dst, int row) const {
        const __half* src = q + (long long)(x.s.q0 + token) * ldq + (long long)head * D;
#pragma unroll
        for (int c0 = 0; c0 < D / 8; c0 += 8) {
            uint4 r[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) r[c] = live ? reinterpret_cast<const uint4*>(src)[c0 + c] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(dst + (c0 / 8) * (kRowsQ * 128) + swizzled(row, c)) = r[c];
        }
    }
    // adds the infinities and NaN that the row sees of the tiles looked through (dims k .. k + 31)
    __device__ void add_special(const Item& x, int token, int k, float (&o)[32]) const {
        const __half* at = v + (long long)x.h * D + k;
        for (int j = max(x.clear, x.lo) * kTile; j < min(seen(x.s, token), x.hi * kTile); ++j)
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float f = __half2float(at[(long long)(x.s.k0 + j) * ldv + i]);
                if (!isfinite(f)) o[i] += f;
            }
    }
};

template <int D>
struct Ring {
    static constexpr int kStages = D == 64 ? 8 : 4;
    static constexpr int kQ = Shape<D>::kStreams * Shape<D>::kQBytes;
    static constexpr int kOut = kQ + kStages * Shape<D>::kEntryBytes;        // staging of the outputs
    static constexpr int kBytes = kOut + Shape<D>::kStreams * kStageBytes;
    static constexpr int kSmem = kBytes + (int)sizeof(Control) + 1024;       // (1024: to begin on such a boundary)
};
static_assert(Ring<128>::kSmem <= 232448 && Ring<256>::kSmem <= 232448 && Ring<64>::kStages <= kMaxStages, "shared memory");

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreadsF, 1) attn_prompt_kernel(const __grid_constant__ Prompt<D> p,
                                                                   const __grid_constant__ CUtensorMap map_q,
                                                                   const __grid_constant__ CUtensorMap map_k,
                                                                   const __grid_constant__ CUtensorMap map_v, bool joins) {
    using X = Shape<D>;
    using R = Ring<D>;
    using Src = Prompt<D>;
    extern __shared__ char raw[];
    char* smem = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    char* ring = smem + R::kQ;
    Control& c = *reinterpret_cast<Control*>(smem + R::kBytes);
    const int wid = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (wid == 8) {
        tc::tmem_alloc(&c.tmem, 512);
        tc::tmem_relinquish();
    }
    if (threadIdx.x == 0) control_init(c, 1, 2, 3, p.q_copied ? 1 : kRowsQ, p.o.wait_ns == 0);
    tc::fence_before_sync();
    wait_predecessor();
    launch_dependents();
    find_share<X>(static_cast<const Src&>(p), blockIdx.x, gridDim.x, reinterpret_cast<long long*>(smem), c.cut);
    tc::fence_after_sync();
    if (joins && threadIdx.x == 0) p.o.places[blockIdx.x] = c.cut[0];

    // registers: 256 x 216 + 128 x 72, what the CTA was launched with (384 x 168)
    if (wid < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;\n");
        softmax_warps<D, Src>(p, c, smem, smem + R::kOut);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;\n");
        if (wid == 8) {
            matrix_warp<D, R::kStages, Src>(p, c, smem_u32(smem), smem_u32(ring));
        } else if (wid == 9) {
            Feed<X, Src> feed(p, c.cut, blockIdx.x);
            int at = 0, block = 0;
            bool ok = p.o.wait_ns != 0;
            const uint32_t lead_lane = elect();
            // a block's queries, 64 rows at a time, as soon as the one's before are done with; one row tile for both streams
            // lies in the second's turned by 64 rows
            auto queries = [&](const Item& x) {
                const bool pair = x.pair<D>();
#pragma unroll 1
                for (int s = 0; s < X::kStreams; ++s) {
                    if (x.of_stream<D>(s) == 0) continue;
                    ok = ok && wait_phase(&c.q_freed[s], (c.q_loads[s] + 1) & 1, c.dead, p.o.wait_ns);
                    if (!ok) return;
                    if (lead_lane) {
                        ++c.q_loads[s];
                        mbar_arrive_expect_tx(&c.q_full[s], X::kQBytes);
#pragma unroll 1
                        for (int half = 0; half < 2; ++half) {
                            const int from = pair ? s * kRowsQ + 64 * half : 64 * (half ^ s);
#pragma unroll 1
                            for (int k = 0; k < X::kChunks; ++k)
                                tma_load(smem_u32(smem) + s * X::kQBytes + k * (kRowsQ * 128) + half * (64 * 128), &map_q, 64 * k, x.h * p.G,
                                         x.s.q0 + (x.row0 + from) / p.G, &c.q_full[s]);
                        }
                    }
                    __syncwarp();
                }
            };
            for (; ok && feed.next(); ++at) {
                if (p.q_copied && feed.number != block) {
                    block = feed.number;
                    queries(feed.x);
                    if (!ok) break;
                }
                const int stage = at % R::kStages;
                if (at >= R::kStages) ok = wait_phase(&c.freed[stage], (at / R::kStages - 1) & 1, c.dead, p.o.wait_ns);
                if (!ok) break;
                if (lead_lane) {
                    mbar_arrive_expect_tx(&c.full[stage], X::kEntryBytes);
#pragma unroll
                    for (int k = 0; k < X::kChunks; ++k)
                        tma_load(smem_u32(ring) + stage * X::kEntryBytes + k * (X::kEntry * 128), feed.value ? &map_v : &map_k, 64 * k,
                                 feed.x.h, feed.x.s.k0 + feed.token(), &c.full[stage]);
                }
                __syncwarp();
            }
            if (lead_lane) c.issued = at;
        } else {
            Feed<X, Src> feed(p, c.cut, blockIdx.x);
            for (int at = 0; feed.next(); ++at) {
                const int stage = at % R::kStages;
                if (!wait_phase(&c.full[stage], (at / R::kStages) & 1, c.dead, p.o.wait_ns)) continue;
                const Item& x = feed.x;
                if (feed.value && x.lo + feed.tile >= x.clear) {
                    uint4* entry = reinterpret_cast<uint4*>(ring + stage * X::kEntryBytes) + (wid - 10) * 32 + lane;
                    constexpr int kPieces = X::kEntryBytes / 16 / 64;
                    const int left = x.s.n_k - feed.token();
                    // the largest magnitude; a NaN stays
                    __half2 most = __halves2half2(__ushort_as_half(0), __ushort_as_half(0));
#pragma unroll 8
                    for (int k = 0; k < kPieces; ++k) {
                        uint4 w = entry[k * 64];
                        if (((((wid - 10) * 32 + lane + k * 64) >> 3) & (X::kEntry - 1)) >= left)      // behind the last key
                            entry[k * 64] = w = make_uint4(0, 0, 0, 0);
                        const __half2* h = reinterpret_cast<const __half2*>(&w);
                        const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])), __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
                        most = __hmax2_nan(most, m);
                    }
                    const bool bad = !(__hlt(__low2half(most), __ushort_as_half(0x7C00)) && __hlt(__high2half(most), __ushort_as_half(0x7C00)));
                    if (__any_sync(0xffffffffu, bad)) {
                        if (bad) special_of(c, feed.number) = feed.number;
#pragma unroll 1
                        for (int k = 0; k < kPieces; ++k) {
                            const uint4 w = entry[k * 64];
                            const uint32_t bx = __vcmpeq2(w.x & 0x7C007C00u, 0x7C007C00u), by = __vcmpeq2(w.y & 0x7C007C00u, 0x7C007C00u),
                                           bz = __vcmpeq2(w.z & 0x7C007C00u, 0x7C007C00u), bw = __vcmpeq2(w.w & 0x7C007C00u, 0x7C007C00u);
                            if ((bx | by | bz | bw) != 0) entry[k * 64] = make_uint4(w.x & ~bx, w.y & ~by, w.z & ~bz, w.w & ~bw);
                        }
                    }
                    tc::fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&c.clean[stage]);
                    mbar_arrive(&c.freed[stage]);
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
            // ... and copies under way, whoever gave up, must not land in what has become another CTA's memory
            drain_copies_call(c.full, c.issued > R::kStages ? c.issued - R::kStages : 0, c.issued, R::kStages);
            for (int s = 0; s < 2; ++s)
                if (c.q_loads[s]) wait_copy(&c.q_full[s], (c.q_loads[s] - 1) & 1, kDefaultWaitNs);
        }
        tc::tmem_dealloc(c.tmem, 512);
    }
}

// cuTensorMapEncodeTiled, looked up once (the library does not link the driver)
typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                           const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                           CUtensorMapFloatOOBfill);
Encode encoder() {
    static Encode f = nullptr;
    Encode g = __atomic_load_n(&f, __ATOMIC_ACQUIRE);
    if (!g) {
        void* at = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return nullptr;
        g = (Encode)at;
        __atomic_store_n(&f, g, __ATOMIC_RELEASE);
    }
    return g;
}

// rows of `heads` x D fp16, ld apart: boxes of 64 dims of `group` heads of `rows` rows, 128-byte swizzled
int make_map(CUtensorMap* map, const void* base, int T, int heads, int D, long long ld, int group, int rows) {
    const Encode f = encoder();
    if (!f) return EDGE0_ECUDA;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)rows}, step[3] = {1, 1, 1};
    const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? EDGE0_OK : EDGE0_EINVAL;
}

template <int D>
int launch(const PromptP& base, const uint16_t* k, long long ldk, char* ws, cudaStream_t stream) {
    using R = Ring<D>;
    constexpr int kDevices = 64;
    static int set[kDevices];            // per device: multiprocessors, set on the first call
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return EDGE0_ECUDA;
    int sms = __atomic_load_n(&set[dev], __ATOMIC_ACQUIRE);
    if (sms == 0) {
        if (cudaFuncSetAttribute(attn_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, R::kSmem) != cudaSuccess ||
            cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return EDGE0_ECUDA;
        sms = sms < kMaxCtas ? sms : kMaxCtas;
        __atomic_store_n(&set[dev], sms, __ATOMIC_RELEASE);
    }
    Prompt<D> p;
    static_cast<PromptP&>(p) = base;
    lay_out<Shape<D>>(ws, &p.o);
    CUtensorMap mq, mk, mv;
    p.q_copied = 64 % p.G == 0;
    int rc = make_map(&mq, p.q, p.T, p.H * p.G, D, p.ldq, p.q_copied ? p.G : 1, p.q_copied ? 64 / p.G : 1);
    if (rc) return rc;
    // without any key nothing is loaded, but a map has to describe something: the queries
    const bool none = p.Tk == 0;
    rc = make_map(&mk, none ? (const void*)p.q : k, none ? p.T : p.Tk, none ? p.H * p.G : p.H, D, none ? p.ldq : ldk, 1, Shape<D>::kEntry);
    if (rc) return rc;
    rc = make_map(&mv, none ? p.q : p.v, none ? p.T : p.Tk, none ? p.H * p.G : p.H, D, none ? p.ldq : p.ldv, 1, Shape<D>::kEntry);
    if (rc) return rc;
    // blocks at most: no more CTAs than that
    const long long blocks = ((long long)p.T * p.G / Shape<D>::kBlock + p.B) * p.H;
    const bool joins = (p.Tk + kTile - 1) / kTile >= Shape<D>::kMinSplit;
    const int grid = joins || blocks > sms ? sms : (int)blocks;
    rc = launch_early(attn_prompt_kernel<D>, dim3(grid), kThreadsF, R::kSmem, stream, p, mq, mk, mv, joins);
    if (rc || !joins || grid < 2) return rc;
    return launch_early(flash_join<Shape<D>, Prompt<D>>, dim3(grid - 1, Shape<D>::kBlock / 32), 32 * kJoinWarps, 0, stream, p);
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" size_t edge0_attn_prompt_workspace_bytes(int head_dim) {
    return head_dim == 64    ? flash::workspace_bytes<flash::Shape<64>>()
           : head_dim == 128 ? flash::workspace_bytes<flash::Shape<128>>()
           : head_dim == 256 ? flash::workspace_bytes<flash::Shape<256>>()
                             : 0;
}

extern "C" int edge0_attn_prompt(const uint16_t* q, long long ldq, int T, int n_q_heads, const uint16_t* k, long long ldk,
                                 const uint16_t* v, long long ldv, int Tk, int n_kv_heads, int head_dim, const int32_t* cu_rows,
                                 const int32_t* cu_keys, int B, float scale, uint16_t* out, long long ldo, void* workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
    if (!cu_rows || B <= 0 || B > EDGE0_MAX_BATCHED || T < 0 || Tk < 0) return EDGE0_EINVAL;
    if (n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads || head_dim <= 0) return EDGE0_EINVAL;
    if (!(scale > 0.f) || !(scale <= 1e6f)) return EDGE0_EINVAL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return EDGE0_EUNSUPPORTED;
    const int G = n_q_heads / n_kv_heads;
    if (n_kv_heads > EDGE0_MAX_KV_HEADS || G > EDGE0_MAX_Q_PER_KV) return EDGE0_EUNSUPPORTED;
    if ((long long)T * G > (1ll << 31) - 512 || Tk > (1 << 30)) return EDGE0_EUNSUPPORTED;
    if (!cu_keys && T != Tk) return EDGE0_EINVAL;
    if ((((uintptr_t)cu_rows | (uintptr_t)cu_keys) & 3) != 0) return EDGE0_EINVAL;
    if (T == 0) return EDGE0_OK;
    if (!q || !out || !workspace || (Tk > 0 && (!k || !v))) return EDGE0_EINVAL;
    const long long wq = (long long)n_q_heads * head_dim, wk = (long long)n_kv_heads * head_dim, most = 1ll << 38;
    if (ldq < wq || ldo < wq || ldq % 8 || ldo % 8 || ldq > most) return EDGE0_EINVAL;
    if (Tk > 0 && (ldk < wk || ldv < wk || ldk % 8 || ldv % 8 || ldk > most || ldv > most)) return EDGE0_EINVAL;
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)out | (uintptr_t)workspace) & 15) return EDGE0_EINVAL;
    if (workspace_bytes < edge0_attn_prompt_workspace_bytes(head_dim)) return EDGE0_EINVAL;
    PromptP p;
    p.o.out = (__half*)out;
    p.o.ldo = ldo;
    p.o.c = scale * 1.4426950408889634f;
    p.o.wait_ns = block_wait_limit();
    p.q = (const __half*)q;
    p.v = (const __half*)v;
    p.ldq = ldq;
    p.ldv = ldv;
    p.B = B;
    p.H = n_kv_heads;
    p.G = G;
    p.T = T;
    p.Tk = Tk;
    p.cu_q = cu_rows;
    p.cu_k = cu_keys ? cu_keys : cu_rows;
    if (head_dim == 64) return launch<64>(p, k, ldk, (char*)workspace, stream);
    if (head_dim == 128) return launch<128>(p, k, ldk, (char*)workspace, stream);
    return launch<256>(p, k, ldk, (char*)workspace, stream);
}
