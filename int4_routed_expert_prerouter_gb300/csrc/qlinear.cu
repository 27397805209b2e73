// Dense int4 projection y = W x, W int4 affine group-64 in the row-tile layout of
// edge0_pack_q4_rows: per 16-row tile and group of 64 inputs one 576-byte unit.
//
//     y[b][o] = sum_g ( s[o,g] sum_{i in g} q[o,i] x[b,i]  +  b[o,g] sum_{i in g} x[b,i] )
//
// One CTA per (row tile, 8 tokens); its warps take the groups in turn, feed the
// nibbles to m16n8k16 steps as fp16 subnormals (exact products, fp32 sums), apply
// the group's scale and bias to the fp32 sums, and are added up in shared memory.
#include "common.cuh"

namespace edge0 {
namespace {

constexpr int kQlWarps = 8;

__global__ void __launch_bounds__(32 * kQlWarps) q4_linear_kernel(const char* __restrict__ w, int out, int in,
                                                                  const __half* __restrict__ x, long long ldx, int B,
                                                                  __half* __restrict__ y, long long ldy) {
    __shared__ float part[kQlWarps][16][8];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int n_g = in / kGroup;
    const int tok = blockIdx.y * 8 + g;
    const char* tile = w + (long long)blockIdx.x * n_g * kQ4Unit;
    const __half* xr = x + (long long)(tok < B ? tok : 0) * ldx;
    float y4[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = wid; c < n_g; c += kQlWarps) {
        const char* u = tile + (long long)c * kQ4Unit;
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(u + 16 * lane));
        const uint2 sbw = __ldg(reinterpret_cast<const uint2*>(u + 512 + 8 * g));
        const uint32_t words[4] = {q.x, q.y, q.z, q.w};
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
        float xs = 0.f;
#pragma unroll
        for (int st = 0; st < 4; ++st) {
            uint32_t A[4];
            q4_masks(words[st], A);
            uint32_t b0 = 0, b1 = 0;
            if (tok < B) {
                b0 = *reinterpret_cast<const uint32_t*>(xr + c * kGroup + 16 * st + 2 * t);
                b1 = *reinterpret_cast<const uint32_t*>(xr + c * kGroup + 16 * st + 2 * t + 8);
            }
            const float2 f0 = __half22float2(*reinterpret_cast<__half2*>(&b0));
            const float2 f1 = __half22float2(*reinterpret_cast<__half2*>(&b1));
            xs += (f0.x + f0.y) + (f1.x + f1.y);
            mma_16816(acc, A, b0, b1);
        }
        xs += __shfl_xor_sync(0xffffffffu, xs, 1);
        xs += __shfl_xor_sync(0xffffffffu, xs, 2);
        const float xs0 = __shfl_sync(0xffffffffu, xs, 8 * t), xs1 = __shfl_sync(0xffffffffu, xs, 8 * t + 4);
        const float2 sb0 = __half22float2(*reinterpret_cast<const __half2*>(&sbw.x));
        const float2 sb1 = __half22float2(*reinterpret_cast<const __half2*>(&sbw.y));
        y4[0] += sb0.x * kTwo24 * acc[0] + sb0.y * xs0;
        y4[1] += sb0.x * kTwo24 * acc[1] + sb0.y * xs1;
        y4[2] += sb1.x * (kTwo24 / 16.f) * acc[2] + sb1.y * xs0;   // nibbles of rows g + 8 enter x16
        y4[3] += sb1.x * (kTwo24 / 16.f) * acc[3] + sb1.y * xs1;
    }
    part[wid][g][2 * t] = y4[0];
    part[wid][g][2 * t + 1] = y4[1];
    part[wid][g + 8][2 * t] = y4[2];
    part[wid][g + 8][2 * t + 1] = y4[3];
    __syncthreads();
    if (threadIdx.x < 128) {
        const int r = threadIdx.x & 15, n = threadIdx.x >> 4;
        const int row = blockIdx.x * kRowTile + r, b = blockIdx.y * 8 + n;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kQlWarps; ++i) s += part[i][r][n];
        if (row < out && b < B) y[b * ldy + row] = __float2half_rn(s);
    }
}

}  // namespace
}  // namespace edge0

using namespace edge0;

extern "C" int edge0_q4_linear(const void* packed, int out, int in, const uint16_t* x, long long ldx, int B,
                               uint16_t* y, long long ldy, cudaStream_t stream) {
    if (!packed || !x || !y || out <= 0 || in <= 0 || in % kGroup) return EDGE0_EINVAL;
    if (B <= 0 || B > EDGE0_MAX_BATCHED || ldx < in || ldx % 8 || ldy < out) return EDGE0_EINVAL;
    if ((((uintptr_t)packed | (uintptr_t)x) & 15) || ((uintptr_t)y & 1)) return EDGE0_EINVAL;
    dim3 grid(ceil_div(out, kRowTile), ceil_div(B, 8));
    q4_linear_kernel<<<grid, 32 * kQlWarps, 0, stream>>>((const char*)packed, out, in, (const __half*)x, ldx, B,
                                                         (__half*)y, ldy);
    return cudaGetLastError() == cudaSuccess ? EDGE0_OK : EDGE0_ECUDA;
}
