// Sliding-window attention with sinks over packed sequences.
//
// One warp per (query, query head): 32 visible keys at a time, one per lane, with
// a running maximum and sum.
#include "kda_common.cuh"

#include <math.h>

namespace kda {
namespace win {

template <int D>
__global__ void __launch_bounds__(256)
window_prefill_kernel(kda_window_prefill_args a) {
    __shared__ float s_q[8][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long unit = (long)blockIdx.x * 8 + warp;
    if (unit >= (long)a.T_total * a.Hq) return;
    const int t = (int)(unit / a.Hq), h = (int)(unit % a.Hq), hk = h / (a.Hq / a.Hkv);
    int lo = 0, hi = a.num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_seqlens[mid] <= t) lo = mid; else hi = mid;
    }
    const int k0 = a.cu_seqlens_k[lo], k1 = a.cu_seqlens_k[lo + 1];
    const int pos = (k1 - k0) - (a.cu_seqlens[lo + 1] - t);
    const int first = max(a.sinks, pos - a.window + 1), ns = min(a.sinks, pos + 1);
    const int total = ns + max(0, pos - first + 1);
    for (int c = lane; c < D; c += 32)
        s_q[warp][c] = bf16_to_f(reinterpret_cast<const uint16_t*>(a.q)[(size_t)t * a.q_stride + (size_t)h * D + c]);
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[D / 32] = {};
    for (int u0 = 0; u0 < total; u0 += 32) {
        const int u = u0 + lane, j = u < ns ? u : first + (u - ns);
        float s = -INFINITY;
        if (u < total) {
            s = 0.f;
            const uint16_t* kr = reinterpret_cast<const uint16_t*>(a.k) + (size_t)(k0 + j) * a.k_stride + (size_t)hk * D;
            for (int c = 0; c < D; c += 8) {
                float x[8];
                load8_bf16(kr + c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) s += x[i] * s_q[warp][c + i];
            }
            s *= a.scale * 1.4426950408889634f;
        }
        float x = s;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, i));
        const float mn = fmaxf(m, x), b = mn == -INFINITY ? 0.f : mn;
        const float c = exp2f(m - b), p = exp2f(s - b);
        l = l * c + p;
        m = mn;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] *= c;
        const int cnt = min(32, total - u0);
        for (int y = 0; y < cnt; ++y) {
            const float w = __shfl_sync(~0u, p, y);
            const int jj = __shfl_sync(~0u, j, y);
            const uint16_t* vr = reinterpret_cast<const uint16_t*>(a.v) + (size_t)(k0 + jj) * a.v_stride + (size_t)hk * D;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) o[i] += w * bf16_to_f(vr[lane + 32 * i]);
        }
    }
    l = warp_sum(l);
    const size_t row = (size_t)t * a.Hq + h;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        reinterpret_cast<uint16_t*>(a.o)[row * D + lane + 32 * i] = f_to_bf16(o[i] / l);
    if (a.lse && lane == 0) a.lse[row] = 0.6931471805599453f * m + logf(l);
}

cudaError_t launch_prefill(const kda_window_prefill_args& a, cudaStream_t s) {
    const long blocks = ((long)a.T_total * a.Hq + 7) / 8;
    if (blocks == 0) return cudaSuccess;
    if (a.d == 64) window_prefill_kernel<64><<<(unsigned)blocks, 256, 0, s>>>(a);
    else window_prefill_kernel<128><<<(unsigned)blocks, 256, 0, s>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace win
}  // namespace kda
