// Tokens into the pages of the key/value cache and back out of them.
//
// One warp per token: it finds the token's place once (a search of the sequence bounds, one page table entry), then its
// lanes move the key and value rows in pieces of 8 channels, 16 bytes of bf16, AHEAD of them in flight.  8-bit rows: d / 8
// lanes hold a row, its largest magnitude goes round them by shuffles.
// Both are copies.  Device time, 8 heads of 128: 32768 tokens out of bf16 pages 42 us (6.4 TB/s), out of 8-bit ones 34 (6.0), 16384 into
// bf16 pages 23 (5.8): HBM.  16384 into 8-bit pages 20 us (5.0 TB/s), DRAM at 41 % of its peak: a warp's start, the search of the
// bounds, the length and the table entry one behind the other before its first row.
#include <type_traits>

#include "paged.cuh"

namespace kda {
namespace paged {

constexpr int WARPS = 4;       // tokens of a CTA
// Pieces that a lane has in flight, of keys and of values each.  16384 tokens of 8 heads of 128, bf16 to 8-bit pages, us with 1,
// 2, 4: 19.3, 17.8, 17.5 (the same inputs in every call, partly in the L2; other ones each time 20.2 with 2); 32768 the other way
// with 2, 4, 8: 33.6, 33.7, 33.2 (one piece at a time: 24.6 and 43).
constexpr int READ_AHEAD = 4, WRITE_AHEAD = 2;

// 8 channels as they lie in memory, in float32, and from there
template <typename T>
struct Raw {
    using type = uint4;                    // bf16
};
template <>
struct Raw<float> {
    struct type {
        float4 a, b;
    };
};
KDA_DEV void load_raw(const uint16_t* p, uint4* r) { *r = __ldg(reinterpret_cast<const uint4*>(p)); }
KDA_DEV void load_raw(const float* p, Raw<float>::type* r) {
    r->a = __ldg(reinterpret_cast<const float4*>(p));
    r->b = __ldg(reinterpret_cast<const float4*>(p) + 1);
}
KDA_DEV void floats(const uint4& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
KDA_DEV void floats(const Raw<float>::type& r, float* x) {
    x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
    x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}
KDA_DEV void store8(uint16_t* p, const float* x) { store8_bf16(p, x); }
KDA_DEV void store8(float* p, const float* x) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// T: type of the tokens (uint16_t: bf16, or float); D8: lanes of a row, d / 8
template <typename T, int D8, bool E4M3>
__global__ void __launch_bounds__(WARPS * 32)
write_kernel(const __grid_constant__ kda_paged_write_args a) {
    const int t = blockIdx.x * WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    Token at;
    if (t >= a.T || !token_at(a.cache, a.cu_seqlens, a.T, t, &at) || at.pos < 0) return;
    const int row = row_of(a.cache, at.n, at.pos);
    if (row < 0) return;
    const int pieces = a.cache.Hkv * D8;
    const T* src[2] = {reinterpret_cast<const T*>(a.k) + (size_t)t * a.k_stride, reinterpret_cast<const T*>(a.v) + (size_t)t * a.v_stride};
    // whole turns of the warp, so that the lanes of a row stay together
#pragma unroll 1
    for (int first = lane; first < pieces + lane; first += 32 * WRITE_AHEAD) {
        typename Raw<T>::type r[WRITE_AHEAD][2];
#pragma unroll
        for (int u = 0; u < WRITE_AHEAD; ++u) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                r[u][kv] = {};
                if (first + 32 * u < pieces) load_raw(src[kv] + (first + 32 * u) * 8, &r[u][kv]);
            }
        }
#pragma unroll
        for (int u = 0; u < WRITE_AHEAD; ++u) {
            const int p = first + 32 * u;
            const bool on = p < pieces;
            const size_t dst = (size_t)row * pieces + p;                 // in pieces
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                if constexpr (!E4M3 && sizeof(T) == 2) {
                    if (on) reinterpret_cast<uint4*>(kv ? a.cache.v : a.cache.k)[dst] = r[u][kv];
                } else {
                    float x[8];
                    floats(r[u][kv], x);
                    if constexpr (!E4M3) {
                        if (on) store8(reinterpret_cast<uint16_t*>(kv ? a.cache.v : a.cache.k) + dst * 8, x);
                    } else {
                        uint32_t m = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
                        for (int o = D8 / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
                        const bool fine = m < 0x7f800000u;
                        const int e = row_exponent(m);
                        const float s = power(-e);
                        uint32_t w[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            w[i] = fine ? codes2(x[4 * i] * s, x[4 * i + 1] * s) | (uint32_t)codes2(x[4 * i + 2] * s, x[4 * i + 3] * s) << 16 : 0u;
                        if (on) {
                            reinterpret_cast<uint2*>(kv ? a.cache.v : a.cache.k)[dst] = make_uint2(w[0], w[1]);
                            if (p % D8 == 0)
                                (kv ? a.cache.v_scale : a.cache.k_scale)[(size_t)row * a.cache.Hkv + p / D8] = (uint8_t)(fine ? e + 127 : 255);
                        }
                    }
                }
            }
        }
    }
}

template <typename T, int D8, bool E4M3>
__global__ void __launch_bounds__(WARPS * 32)
read_kernel(const __grid_constant__ kda_paged_read_args a) {
    using Piece = std::conditional_t<E4M3, uint2, uint4>;
    const int t = blockIdx.x * WARPS + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    Token at;
    if (t >= a.T || !token_at(a.cache, a.cu_seqlens, a.T, t, &at)) return;
    const int row = at.pos < 0 ? -1 : row_of(a.cache, at.n, at.pos);         // -1: zeros
    const int pieces = a.cache.Hkv * D8;
#pragma unroll 1
    for (int first = lane; first < pieces; first += 32 * READ_AHEAD) {
        Piece w[READ_AHEAD][2];
        uint32_t byte[READ_AHEAD][2];
#pragma unroll
        for (int u = 0; u < READ_AHEAD; ++u) {
            const int p = first + 32 * u;
            const bool on = row >= 0 && p < pieces;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                w[u][kv] = Piece{};
                byte[u][kv] = 0;
                if (on) w[u][kv] = __ldg(reinterpret_cast<const Piece*>(kv ? a.cache.v : a.cache.k) + (size_t)row * pieces + p);
                if (E4M3 && on) byte[u][kv] = (kv ? a.cache.v_scale : a.cache.k_scale)[(size_t)row * a.cache.Hkv + p / D8];
            }
        }
#pragma unroll
        for (int u = 0; u < READ_AHEAD; ++u) {
            const int p = first + 32 * u;
            if (p >= pieces) break;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                T* dst = reinterpret_cast<T*>(kv ? a.v : a.k) + ((size_t)t * pieces + p) * 8;
                if constexpr (!E4M3 && sizeof(T) == 2) {
                    *reinterpret_cast<uint4*>(dst) = w[u][kv];
                } else {
                    float x[8];
                    if constexpr (!E4M3) {
                        floats(w[u][kv], x);
                    } else {
                        const uint32_t c[2] = {w[u][kv].x, w[u][kv].y};
                        const float s = scale_of(byte[u][kv]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 v = values2((uint16_t)(c[i / 2] >> (16 * (i & 1))));
                            x[2 * i] = v.x * s;
                            x[2 * i + 1] = v.y * s;
                        }
                    }
                    store8(dst, x);
                }
            }
        }
    }
}

template <typename A, typename K>
static cudaError_t go(K kernel, const A& a, cudaStream_t s) {
    kernel<<<(a.T + WARPS - 1) / WARPS, WARPS * 32, 0, s>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

// instance of the kernel template K for the call's types and row width
#define KDA_PAGED_PICK(K, a, s)                                                                             \
    do {                                                                                                    \
        const bool f32 = (a).dtype == KDA_F32, q8 = (a).cache.dtype == KDA_E4M3, wide = (a).cache.d == 128; \
        if (f32) {                                                                                          \
            if (q8) return wide ? go(K<float, 16, true>, a, s) : go(K<float, 8, true>, a, s);               \
            return wide ? go(K<float, 16, false>, a, s) : go(K<float, 8, false>, a, s);                     \
        }                                                                                                   \
        if (q8) return wide ? go(K<uint16_t, 16, true>, a, s) : go(K<uint16_t, 8, true>, a, s);             \
        return wide ? go(K<uint16_t, 16, false>, a, s) : go(K<uint16_t, 8, false>, a, s);                   \
    } while (0)

cudaError_t launch_write(const kda_paged_write_args& a, cudaStream_t s) { KDA_PAGED_PICK(write_kernel, a, s); }
cudaError_t launch_read(const kda_paged_read_args& a, cudaStream_t s) { KDA_PAGED_PICK(read_kernel, a, s); }

}  // namespace paged
}  // namespace kda
