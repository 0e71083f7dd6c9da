// RMSNorm of each query and key head with the position rotation in the same pass.
//
// Streaming, HBM-bound: every value is read once and written once.  A head row of
// d channels is held by LANES lanes, 8 channels each (one 16-byte bf16 access, two
// for float32); the mean square is a shuffle reduction over those lanes, and the
// partner channel of a rotated pair is another register of the same lane
// (neighbouring pairs) or the same register of the lane rot/16 away (halves: rot
// is a multiple of 16, so a pair never straddles an 8-channel group unevenly).
// A lane group takes HPG heads of one token, so that the token's cosines and
// sines are read once for all of them.
#include "kda_common.cuh"

namespace kda {
namespace qknr {

constexpr int NT = 256;

template <bool BF16>
struct Raw;
template <>
struct Raw<true> {
    uint4 u;
    KDA_DEV void load(const void* p, size_t i) { u = __ldcs(reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p) + i)); }
    KDA_DEV void get(float* x) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[2 * i] = __uint_as_float(w[i] << 16); x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u); }
    }
};
template <>
struct Raw<false> {
    float4 a, b;
    KDA_DEV void load(const void* p, size_t i) {
        const float4* f = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + i);
        a = __ldcs(f);
        b = __ldcs(f + 1);
    }
    KDA_DEV void get(float* x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

template <bool BF16>
KDA_DEV void put(void* p, size_t i, const float* x) {
    if (BF16) {
        store8_bf16(reinterpret_cast<uint16_t*>(p) + i, x);
    } else {
        float4* f = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

KDA_DEV void load8f(const float* p, float* x) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

template <bool BF16, bool PAIRS, int LANES, int HPG>
__global__ void __launch_bounds__(NT)
qk_norm_rope_kernel(kda_qk_norm_rope_args a, int groups) {
    const int H = a.Hq + a.Hkv;
    const long g = ((long)blockIdx.x * NT + threadIdx.x) / LANES;     // lane group = (token, HPG heads)
    const int l = threadIdx.x % LANES, c = 8 * l;
    const int t = (int)(g / groups), h0 = (int)(g % groups) * HPG;
    bool live = t < a.T;                  // every lane stays for the shuffles
    const int pos = live ? a.positions[t] : -1;
    live = live && pos >= 0 && pos < a.num_pos;
    const bool ch = live && c < a.d;
    Raw<BF16> raw[HPG];
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        const int h = h0 + j;
        if (ch && h < H) {
            if (h < a.Hq) raw[j].load(a.q, (size_t)t * a.q_stride + (size_t)h * a.d + c);
            else raw[j].load(a.k, (size_t)t * a.k_stride + (size_t)(h - a.Hq) * a.d + c);
        }
    }
    const int half = a.rot >> 1;
    const bool turned = ch && c < a.rot;
    // halves: this lane's channels are pairs c % half .. + 7, first members below half;
    // neighbouring pairs: channels c .. c + 7 are pairs c/2 .. c/2 + 3
    float cs[8], sn[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { cs[i] = 1.f; sn[i] = 0.f; w[i] = 1.f; }
    if (turned) {
        const size_t row = (size_t)pos * half;
        if (PAIRS) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(a.cos + row + (c >> 1)));
            const float4 y = __ldg(reinterpret_cast<const float4*>(a.sin + row + (c >> 1)));
            cs[0] = cs[1] = x.x; cs[2] = cs[3] = x.y; cs[4] = cs[5] = x.z; cs[6] = cs[7] = x.w;
            sn[0] = -y.x; sn[1] = y.x; sn[2] = -y.y; sn[3] = y.y; sn[4] = -y.z; sn[5] = y.z; sn[6] = -y.w; sn[7] = y.w;
        } else {
            const bool first = c < half;
            load8f(a.cos + row + (first ? c : c - half), cs);
            load8f(a.sin + row + (first ? c : c - half), sn);
#pragma unroll
            for (int i = 0; i < 8; ++i) sn[i] = first ? -sn[i] : sn[i];
        }
    }
    const float* held = nullptr;          // the weight vector in w (null: ones)
    const int step = half >> 3;           // lanes between the members of a pair (halves)
    const int src = PAIRS ? 0 : (l < step ? l + step : l - step);
    const float inv_d = 1.0f / (float)a.d;
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        const int h = h0 + j;
        const bool on = ch && h < H;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (on) raw[j].get(x);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float r = rsqrtf(ss * inv_d + a.eps);
        const float* weight = h < a.Hq ? a.q_weight : a.k_weight;
        if (on && weight != held) {
            if (weight) {
                load8f(weight + c, w);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = 1.f;
            }
            held = weight;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float other = PAIRS ? x[i ^ 1] : __shfl_sync(~0u, x[i], src, LANES);
            y[i] = turned ? x[i] * cs[i] + other * sn[i] : x[i];
        }
        if (on) {
            if (h < a.Hq) put<BF16>(a.q_out, ((size_t)t * a.Hq + h) * a.d + c, y);
            else put<BF16>(a.k_out, ((size_t)t * a.Hkv + (h - a.Hq)) * a.d + c, y);
        }
    }
}

template <bool BF16, bool PAIRS, int LANES, int HPG>
static cudaError_t go(const kda_qk_norm_rope_args& a, cudaStream_t s) {
    const int groups = (a.Hq + a.Hkv + HPG - 1) / HPG;
    const long threads = (long)a.T * groups * LANES;
    qk_norm_rope_kernel<BF16, PAIRS, LANES, HPG><<<(unsigned)((threads + NT - 1) / NT), NT, 0, s>>>(a, groups);
    count_launches(1);
    return cudaGetLastError();
}
template <bool BF16, bool PAIRS, int LANES>
static cudaError_t by_heads(const kda_qk_norm_rope_args& a, cudaStream_t s) {
    // Several heads per lane group share the token's cosines and sines; where that
    // would leave threads idle (fewer than two full waves of them), one head each.
    const long rows = (long)a.T * (a.Hq + a.Hkv);
    return rows * LANES >= 4L * 2 * 152 * 2048 ? go<BF16, PAIRS, LANES, 4>(a, s) : go<BF16, PAIRS, LANES, 1>(a, s);
}
template <bool BF16, bool PAIRS>
static cudaError_t by_width(const kda_qk_norm_rope_args& a, cudaStream_t s) {
    if (a.d <= 64) return by_heads<BF16, PAIRS, 8>(a, s);
    if (a.d <= 128) return by_heads<BF16, PAIRS, 16>(a, s);
    return by_heads<BF16, PAIRS, 32>(a, s);
}

cudaError_t launch(const kda_qk_norm_rope_args& a, cudaStream_t s) {
    if (a.T == 0) return cudaSuccess;
    if (a.dtype == KDA_BF16) return a.interleaved ? by_width<true, true>(a, s) : by_width<true, false>(a, s);
    return a.interleaved ? by_width<false, true>(a, s) : by_width<false, false>(a, s);
}

}  // namespace qknr
}  // namespace kda
