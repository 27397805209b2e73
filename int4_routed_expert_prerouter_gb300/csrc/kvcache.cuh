// Layout of the quantised KV cache's pages (see edge0_kv_cache in edge0.h) and the
// kernels' view of a cache.
//
// A page is [kv head][strip of 16 tokens]; a strip holds the 16 tokens' K codes, K
// (s, b) pairs, V codes, V (s, b) pairs, so that whatever the page size, 16 tokens of
// one head are one contiguous run of bytes that a single bulk copy brings in.
// Rows of codes are cut into 16-byte pieces; piece c of row r is stored at piece
// c ^ turn(r): eight consecutive rows' piece c then lie in eight different 16-byte
// banks, which is what the 8x8 matrix loads of the attention kernel want.
#pragma once
#include "internal.cuh"

namespace edge0 {
namespace kv {

constexpr int kStrip = 16;   // tokens per strip

// bytes of one token's codes
__host__ __device__ constexpr int row_bytes(int bits, int D) { return D * bits / 8; }
// bytes of one token's (s, b) pairs
__host__ __device__ constexpr int sb_bytes(int D) { return D / kGroup * 4; }
// bytes of the K (or V) half of a strip, and of a strip
__host__ __device__ constexpr int half_bytes(int bits, int D) {
    return kStrip * (row_bytes(bits, D) + sb_bytes(D));
}
__host__ __device__ constexpr int strip_bytes(int bits, int D) { return 2 * half_bytes(bits, D); }
// the number that row r's piece indices are exclusive-ored with (R = row_bytes)
__host__ __device__ constexpr int turn(int R, int r) {
    return R >= 128 ? (r & 7) : ((r * R / 128) & (R / 16 - 1));
}

struct View {
    char* pages;
    long long page_bytes;
    int n_pages, page_tokens, H;
};

// Checks a cache descriptor and derives the kernels' view of it.
inline int view_of(const edge0_kv_cache* c, View* v) {
    if (!c || !c->pages || ((uintptr_t)c->pages & 15)) return EDGE0_EINVAL;
    if (c->n_pages <= 0 || c->n_kv_heads <= 0 || c->page_tokens <= 0) return EDGE0_EINVAL;
    if (edge0_kv_page_bytes(c->bits, c->n_kv_heads, c->head_dim, c->page_tokens) == 0) return EDGE0_EUNSUPPORTED;
    v->pages = (char*)c->pages;
    v->page_bytes = (long long)edge0_kv_page_bytes(c->bits, c->n_kv_heads, c->head_dim, c->page_tokens);
    v->n_pages = c->n_pages;
    v->page_tokens = c->page_tokens;
    v->H = c->n_kv_heads;
    return EDGE0_OK;
}

}  // namespace kv

// two fp16 in a word
__device__ __forceinline__ uint32_t hadd2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

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

}  // namespace edge0
