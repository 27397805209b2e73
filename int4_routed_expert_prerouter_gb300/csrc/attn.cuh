// What the attention kernels share: the description of a prefix's work on the
// fifth-generation tensor cores (attn_prefix.cu), launched by attn.cu.
#pragma once
#include "kvcache.cuh"
#include "launch.cuh"

namespace edge0 {

constexpr int kPrefixRows = 128;     // query rows of a CTA: the rows of one accumulator
constexpr int kPrefixTile = 64;      // tokens per step

// Both factors of a weight p s have a reference, es = 2^e the scales': p <= 2^kRise and s <=
// es kHighS, so that p s / es kUp < 2^15 stays within fp16.  Below es kLowS p s may leave
// fp16's normal range while it still counts: such scales get a second product of what the rounding
// took.  With one in every tile, us so: four contexts of 131,072 tokens at 4 bits 119 and 218,
// of 65,536 at 8 bits 97 and 118, 256 sequences of 32 heads behind 8,191 tokens 91 and 176.
constexpr float kRise = 4.f, kHighS = 16.f, kUp = 128.f, kLowS = 1.f / 512;

struct PrefixP {
    kv::View c;
    const __half* q;
    long long ldq;
    int G, H, rows;                  // query heads per K/V head, K/V heads, query rows per K/V head
    int RB, splits, tiles_per_split; // row blocks; shares of the prefix, each of so many tiles
    const int* pages;
    int n_tok;
    float k;                         // scale log2(e)
    float* part_o;                   // [(h RB + rb) splits + share][kPrefixRows][D]
    float2* part_ml;                 // [..][kPrefixRows] (maximum in exponent units, sum)
    int* status;
    unsigned long long wait_ns;      // limit of a wait
};

// shares of the prefix that fill the card for `segs` (K/V head, row block) pairs
void prefix_shares(int n_tok, int segs, int D, int sms, int* splits, int* tiles_per_split);
int prefix_launch(const PrefixP& p, int bits, int D, cudaStream_t stream);

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / x of a power of two
__device__ __forceinline__ float reciprocal2(float x) { return __uint_as_float((254u << 23) - __float_as_uint(x)); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace edge0
