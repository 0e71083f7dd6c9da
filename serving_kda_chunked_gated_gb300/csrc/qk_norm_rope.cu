// RMSNorm of each query and key head with the position rotation in the same pass.
//
// Streaming, HBM-bound: every value is read once and written once.  A head row of
// d channels is held by LANES lanes, 8 channels each, as 4 pairs (a, b): a lane of
// the rotated part takes channels 4 l .. 4 l + 3 and rot/2 + 4 l .. rot/2 + 4 l + 3
// (halves) or 8 l .. 8 l + 7 (neighbouring pairs), one of the rest 8 l .. 8 l + 7 with
// an angle of 0.  Both members of a pair so sit in one lane: the only exchange between
// lanes is the mean square's reduction (with whole 16-byte pieces of a row per lane and
// a shuffle for the partner, half style ran at 0.64 of HBM).  A lane group takes HPG heads
// of one token: the loads of all of them are in flight together, and the token's
// cosines and sines are read once.
#include "kda_common.cuh"

namespace kda {
namespace qknr {

constexpr int NT = 128;     // small blocks and streaming stores: 146 -> 126 us for 32768 tokens x 40 heads of 128

// 4 + 4 channels, as the type holds them
template <bool BF16>
struct Raw;
template <>
struct Raw<true> {
    uint2 a, b;
    KDA_DEV void load(const void* p, size_t i, size_t j, bool joined) {
        const uint16_t* x = reinterpret_cast<const uint16_t*>(p);
        if (joined) {
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(x + i));
            a = make_uint2(u.x, u.y);
            b = make_uint2(u.z, u.w);
        } else {
            a = __ldcs(reinterpret_cast<const uint2*>(x + i));
            b = __ldcs(reinterpret_cast<const uint2*>(x + j));
        }
    }
    KDA_DEV void get(float* x) const {
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) { x[2 * i] = __uint_as_float(w[i] << 16); x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u); }
    }
};
template <>
struct Raw<false> {
    float4 a, b;
    KDA_DEV void load(const void* p, size_t i, size_t j, bool) {
        const float* x = reinterpret_cast<const float*>(p);
        a = __ldcs(reinterpret_cast<const float4*>(x + i));
        b = __ldcs(reinterpret_cast<const float4*>(x + j));
    }
    KDA_DEV void get(float* x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

KDA_DEV uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool BF16>
KDA_DEV void put(void* p, size_t i, size_t j, bool joined, const float* x) {
    if (BF16) {
        uint16_t* y = reinterpret_cast<uint16_t*>(p);
        const uint2 u = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3])), v = make_uint2(pack2(x[4], x[5]), pack2(x[6], x[7]));
        if (joined) {
            __stcs(reinterpret_cast<uint4*>(y + i), make_uint4(u.x, u.y, v.x, v.y));
        } else {
            __stcs(reinterpret_cast<uint2*>(y + i), u);
            __stcs(reinterpret_cast<uint2*>(y + j), v);
        }
    } else {
        float* y = reinterpret_cast<float*>(p);
        __stcs(reinterpret_cast<float4*>(y + i), make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4*>(y + j), make_float4(x[4], x[5], x[6], x[7]));
    }
}

KDA_DEV void load4f(const float* p, float* x) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}

template <bool BF16, bool PAIRS, int LANES, int HPG>
__global__ void __launch_bounds__(NT)
qk_norm_rope_kernel(kda_qk_norm_rope_args a, int groups) {
    const int H = a.Hq + a.Hkv;
    const long g = ((long)blockIdx.x * NT + threadIdx.x) / LANES;     // lane group = (token, HPG heads)
    const int l = threadIdx.x % LANES;
    const long t = g / groups;
    const int h0 = (int)(g % groups) * HPG;
    const bool have = t < a.T;            // every lane stays for the shuffles
    const int pos = have ? __ldg(a.positions + t) : -1;
    const int half = a.rot >> 1;
    const bool turned = 8 * l < a.rot, mine = have && 8 * l < a.d;
    const bool joined = PAIRS || !turned;                             // 8 neighbouring channels
    const int i0 = joined ? 8 * l : 4 * l, j0 = joined ? 8 * l + 4 : half + 4 * l;
    Raw<BF16> raw[HPG];
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        const int h = h0 + j;
        if (mine && h < H) {                 // in flight while the position arrives
            const bool q = h < a.Hq;
            const size_t row = q ? (size_t)t * a.q_stride + (size_t)h * a.d : (size_t)t * a.k_stride + (size_t)(h - a.Hq) * a.d;
            raw[j].load(q ? a.q : a.k, row + i0, row + j0, joined);
        }
    }
    const bool on = mine && pos >= 0 && pos < a.num_pos;
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f}, w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (on && turned) {
        const size_t row = (size_t)pos * half + 4 * l;
        load4f(a.cos + row, cs);
        load4f(a.sin + row, sn);
    }
    const float* held = nullptr;          // the weight vector in w (null: ones)
    const float inv_d = 1.0f / (float)a.d;
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        const int h = h0 + j;
        const bool here = on && h < H;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
        if (here) raw[j].get(x);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const float r = rsqrtf(ss * inv_d + a.eps);
        if (here) {
            const float* weight = h < a.Hq ? a.q_weight : a.k_weight;
            if (weight != held) {
                if (weight) {
                    load4f(weight + i0, w);
                    load4f(weight + j0, w + 4);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = 1.f;
                }
                held = weight;
            }
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int p = PAIRS ? 2 * i : i, q = PAIRS ? 2 * i + 1 : i + 4;
                const float u = x[p] * r * w[p], v = x[q] * r * w[q];
                y[p] = u * cs[i] - v * sn[i];
                y[q] = v * cs[i] + u * sn[i];
            }
            if (h < a.Hq) put<BF16>(a.q_out, ((size_t)t * a.Hq + h) * a.d + i0, ((size_t)t * a.Hq + h) * a.d + j0, joined, y);
            else put<BF16>(a.k_out, ((size_t)t * a.Hkv + (h - a.Hq)) * a.d + i0, ((size_t)t * a.Hkv + (h - a.Hq)) * a.d + j0, joined, y);
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
    // Several heads per lane group share the token's cosines and sines; where that would
    // leave SMs short of threads (less than one full wave of them with a head each), one
    // head each.  40 heads of 128, bf16: 64 tokens 2.0 us by ones, 3.1 by fives; 512
    // tokens 3.8 both; 1024 tokens 5.9, 5.1; 16384 tokens 82.6, 60.2.
    const int H = a.Hq + a.Hkv;
    if ((long)a.T * H * LANES < 152L * 2048) return go<BF16, PAIRS, LANES, 1>(a, s);
    // 4, 5 or 6, whichever leaves the fewest of a token's lane groups' places empty (8 need
    // more registers than they save time)
    const int idle4 = (4 - H % 4) % 4, idle5 = (5 - H % 5) % 5, idle6 = (6 - H % 6) % 6;
    if (idle6 <= idle5 && idle6 <= idle4) return go<BF16, PAIRS, LANES, 6>(a, s);
    return idle5 <= idle4 ? go<BF16, PAIRS, LANES, 5>(a, s) : go<BF16, PAIRS, LANES, 4>(a, s);
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
