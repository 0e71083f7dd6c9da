// RMSNorm of each query and key head with the position rotation in the same pass.
//
// Streaming, HBM-bound: every value is read once and written once.  A head row of
// d channels is held by LANES lanes, 8 channels each, as 4 pairs (a, b): a lane of
// the rotated part takes channels 4 l .. 4 l + 3 and rot/2 + 4 l .. rot/2 + 4 l + 3
// (halves) or 8 l .. 8 l + 7 (neighbouring pairs), one of the rest 8 l .. 8 l + 7 with
// an angle of 0.  Both members of a pair so sit in one lane: the only exchange between
// lanes is the mean square's reduction (with whole 16-byte pieces of a row per lane and
// a shuffle for the partner, half style ran at 0.64 of HBM).  A lane group takes HPG
// query or key heads of one token: the loads of all of them are in flight together, and
// the products of the weights with the token's cosines and sines are formed once.
//
// Issue slots come next after HBM (0.73 of them busy before the products were shared and
// the pairs' arithmetic ran two operations at a time): 32768 tokens x 40 heads of 128,
// bf16, 0.69 GB: 127 -> 108 us, 6.4 TB/s, 0.94 of a copy's rate.
#include "kda_common.cuh"

namespace kda {
namespace qknr {

constexpr int NT = 128;     // 64 and 256 threads: 1 to 2 % slower

KDA_DEV void load4f(const float* p, float* x) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}

// 4 pairs of channels, as the type holds them: first and second members apart (halves), or in turn
template <bool BF16>
struct Raw;
template <>
struct Raw<true> {
    uint2 a = {0, 0}, b = {0, 0};
    KDA_DEV void load(const void* p, int i, int j, bool joined) {
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
    template <bool PAIRS>
    KDA_DEV void get(float* x, float* y) const {
        const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
            if (PAIRS) { x[i] = lo; y[i] = hi; }
            else { float* z = i < 2 ? x + 2 * i : y + 2 * i - 4; z[0] = lo; z[1] = hi; }
        }
    }
};
template <>
struct Raw<false> {
    float4 a = {0.f, 0.f, 0.f, 0.f}, b = {0.f, 0.f, 0.f, 0.f};
    KDA_DEV void load(const void* p, int i, int j, bool) {
        const float* x = reinterpret_cast<const float*>(p);
        a = __ldcs(reinterpret_cast<const float4*>(x + i));
        b = __ldcs(reinterpret_cast<const float4*>(x + j));
    }
    template <bool PAIRS>
    KDA_DEV void get(float* x, float* y) const {
        if (PAIRS) {
            x[0] = a.x; y[0] = a.y; x[1] = a.z; y[1] = a.w; x[2] = b.x; y[2] = b.y; x[3] = b.z; y[3] = b.w;
        } else {
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; y[0] = b.x; y[1] = b.y; y[2] = b.z; y[3] = b.w;
        }
    }
};

KDA_DEV uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool BF16, bool PAIRS>
KDA_DEV void put(void* p, int i, int j, bool joined, const float* x, const float* y) {
    if (BF16) {
        uint16_t* o = reinterpret_cast<uint16_t*>(p);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = PAIRS ? pack2(x[e], y[e]) : e < 2 ? pack2(x[2 * e], x[2 * e + 1]) : pack2(y[2 * e - 4], y[2 * e - 3]);
        if (joined) {
            __stcs(reinterpret_cast<uint4*>(o + i), make_uint4(w[0], w[1], w[2], w[3]));
        } else {
            __stcs(reinterpret_cast<uint2*>(o + i), make_uint2(w[0], w[1]));
            __stcs(reinterpret_cast<uint2*>(o + j), make_uint2(w[2], w[3]));
        }
    } else {
        float* o = reinterpret_cast<float*>(p);
        __stcs(reinterpret_cast<float4*>(o + i), PAIRS ? make_float4(x[0], y[0], x[1], y[1]) : make_float4(x[0], x[1], x[2], x[3]));
        __stcs(reinterpret_cast<float4*>(o + j), PAIRS ? make_float4(x[2], y[2], x[3], y[3]) : make_float4(y[0], y[1], y[2], y[3]));
    }
}

// two float32 operations in one instruction
KDA_DEV void mul2(float* d, const float* a, const float* b) {
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.ftz.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d[0]), "=f"(d[1]) : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}
KDA_DEV void fma2(float* d, const float* a, const float* b, const float* c) {
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.ftz.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d[0]), "=f"(d[1]) : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}

template <bool BF16, bool PAIRS, int LANES, int HPG>
__global__ void __launch_bounds__(NT)
qk_norm_rope_kernel(const __grid_constant__ kda_qk_norm_rope_args a, unsigned qgroups, unsigned groups) {
    const unsigned g = blockIdx.x * (NT / LANES) + threadIdx.x / LANES;    // lane group = (token, HPG heads of q or of k)
    const int l = threadIdx.x % LANES;
    const unsigned t = g / groups, gi = g % groups;
    const bool have = t < (unsigned)a.T;  // every lane stays for the shuffles
    const bool q = gi < qgroups;
    const int H = q ? a.Hq : a.Hkv, h0 = (int)(q ? gi : gi - qgroups) * HPG;
    const int half = a.rot >> 1;
    const bool turned = 8 * l < a.rot, mine = have && 8 * l < a.d;
    const bool joined = PAIRS || !turned;                                  // 8 neighbouring channels
    const int i0 = joined ? 8 * l : 4 * l, j0 = joined ? 8 * l + 4 : half + 4 * l;
    constexpr int SIZE = BF16 ? 2 : 4;
    const int step = a.d * SIZE;
    const char* src = reinterpret_cast<const char*>(q ? a.q : a.k) + ((size_t)t * (q ? a.q_stride : a.k_stride) + (size_t)h0 * a.d) * SIZE;
    char* dst = reinterpret_cast<char*>(q ? a.q_out : a.k_out) + ((size_t)t * H + h0) * (size_t)step;
    const int pos = have ? __ldg(a.positions + t) : -1;
    Raw<BF16> raw[HPG];
#pragma unroll
    for (int j = 0; j < HPG; ++j)            // in flight while the position arrives
        if (mine && h0 + j < H) raw[j].load(src + j * step, i0, j0, joined);
    const bool on = mine && pos >= 0 && pos < a.num_pos;
    // y_a = r (x_a w_a cos - x_b w_b sin), y_b = r (x_b w_b cos + x_a w_a sin): the products
    // without r are the same for every head of the group
    float ac[4], bs[4], bc[4], as[4];
    {
        float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f}, w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 1.f;
        const float* weight = q ? a.q_weight : a.k_weight;
        if (mine && weight) {
            load4f(weight + i0, w);
            load4f(weight + j0, w + 4);
        }
        if (on && turned) {
            const size_t row = (size_t)pos * half + 4 * l;
            load4f(a.cos + row, cs);
            load4f(a.sin + row, sn);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float wa = w[PAIRS ? 2 * i : i], wb = w[PAIRS ? 2 * i + 1 : i + 4];
            ac[i] = wa * cs[i]; bs[i] = -wb * sn[i]; bc[i] = wb * cs[i]; as[i] = wa * sn[i];
        }
    }
    const float inv_d = 1.0f / (float)a.d;
#pragma unroll
    for (int j = 0; j < HPG; ++j) {
        float x[4], y[4], u[4], v[4], ss[2];
        raw[j].template get<PAIRS>(x, y);
        mul2(ss, x, x);
        fma2(ss, x + 2, x + 2, ss);
        fma2(ss, y, y, ss);
        fma2(ss, y + 2, y + 2, ss);
        float sum = ss[0] + ss[1];
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        const float r = rsqrtf(sum * inv_d + a.eps), rr[2] = {r, r};
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            mul2(u + i, x + i, ac + i);
            fma2(u + i, y + i, bs + i, u + i);
            mul2(v + i, y + i, bc + i);
            fma2(v + i, x + i, as + i, v + i);
            mul2(u + i, u + i, rr);
            mul2(v + i, v + i, rr);
        }
        if (on && h0 + j < H) put<BF16, PAIRS>(dst + j * step, i0, j0, joined, u, v);
    }
}

template <bool BF16, bool PAIRS, int LANES, int HPG>
static cudaError_t go(const kda_qk_norm_rope_args& a, cudaStream_t s) {
    const long qgroups = ((long)a.Hq + HPG - 1) / HPG, groups = qgroups + ((long)a.Hkv + HPG - 1) / HPG;
    const long blocks = ((long)a.T * groups * LANES + NT - 1) / NT;
    qk_norm_rope_kernel<BF16, PAIRS, LANES, HPG><<<(unsigned)blocks, NT, 0, s>>>(a, (unsigned)qgroups, (unsigned)groups);
    count_launches(1);
    return cudaGetLastError();
}
template <bool BF16, bool PAIRS, int LANES>
static cudaError_t by_heads(const kda_qk_norm_rope_args& a, cudaStream_t s) {
    // Several heads per lane group share the token's cosines, sines and weights; where that would
    // leave SMs short of threads (less than half a wave of them with a head each), one head
    // each.  32 + 8 heads of 128, bf16: 64 tokens 1.9 us by ones, 2.2 by fours; 512 tokens 3.6,
    // 3.0; 16384 tokens 75, 52.
    if ((long)a.T * (a.Hq + a.Hkv) * LANES < 152L * 1024) return go<BF16, PAIRS, LANES, 1>(a, s);
    // Eight where they leave no more places empty than fours: 32768 tokens 109 us against 114 (for 12 + 2
    // heads 54, 47).  Float32 and heads of 64 gain nothing: 105, 105 and 61, 59.
    const int places4 = (a.Hq + 3) / 4 * 4 + (a.Hkv + 3) / 4 * 4, places8 = (a.Hq + 7) / 8 * 8 + (a.Hkv + 7) / 8 * 8;
    if constexpr (BF16 && LANES > 8)
        if (places8 <= places4) return go<BF16, PAIRS, LANES, 8>(a, s);
    return go<BF16, PAIRS, LANES, 4>(a, s);
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
