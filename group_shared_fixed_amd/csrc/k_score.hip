// Logits from 8-bit features and 8-bit label weights:
// Z[b, l] = hs[b] ws[l] sum_j hq[b, j] Wq[l, j], both operands E4M3.
//
// The codes are widened to bf16, which holds every E4M3 value, and multiplied
// by the bf16 matrix product: exact products, fp32 sums (measured error
// against fp64 at H = 768: 3e-8 of the result's norm).  The 8-bit matrix
// products keep fewer bits of the terms they add (1.5e-5 there), past what
// an fp32 output stands for.
//
// One wave per 16 x 16 tile of (labels, rows), operands straight from memory.
#include "elem.hpp"
#include "kernels.hpp"

namespace haste {
namespace {

// Sixteen codes as two matrix operands of eight bf16.
__device__ __forceinline__ void widen16(u32x4_t c, u32x4_t& lo, u32x4_t& hi)
{
    lo = widen_w8(u32x2_t{c[0], c[1]}, 1.0f);
    hi = widen_w8(u32x2_t{c[2], c[3]}, 1.0f);
}

__global__ __launch_bounds__(256) void k_score(ScoreArgs a)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, r16 = lane & 15, q = lane >> 4;
    const int64_t l0 = ((int64_t)blockIdx.x * 4 + w) * 16, b0 = (int64_t)blockIdx.y * 16;
    if (l0 >= a.L) return;
    const int64_t l = l0 + r16 < a.L ? l0 + r16 : a.L - 1, b = b0 + r16 < a.B ? b0 + r16 : a.B - 1;
    const uint8_t* pw = a.Wq + l * a.H;
    const uint8_t* ph = a.hq + b * a.H;
    const u32x4_t zero = {0u, 0u, 0u, 0u};
    f32x4_t acc = zero4();
    for (int64_t k = 16 * q; k < a.H + 16 * q; k += 64) {
        u32x4_t w0, w1, h0, h1;
        widen16(k < a.H ? ldg16(pw + k) : zero, w0, w1);
        widen16(k < a.H ? ldg16(ph + k) : zero, h0, h1);
        acc = mfma16(w0, h0, acc);
        acc = mfma16(w1, h1, acc);
    }
    // lane: row b0 + r16, labels l0 + 4 q + i
    if (b0 + r16 < a.B) {
        const float s = a.hs[b0 + r16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t o = l0 + 4 * q + i;
            if (o < a.L) a.Z[(b0 + r16) * a.L + o] = acc[i] * s * a.ws[o];
        }
    }
}

}  // namespace

void launch_score(const ScoreArgs& a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.L + 63) / 64), (unsigned)((a.B + 15) / 16));
    k_score<<<grid, 256, 0, s>>>(a);
}

}  // namespace haste
