// Chunked prefill of the gated delta rule with one decay per value head, bf16, on tcgen05.
//
// With g_i the log-decay summed over a chunk's tokens up to i, rk_i and rq_i the inverse
// key and query norms (1 without qk_l2norm) and S the state before the chunk:
//   A_ij  = beta_i rk_i rk_j e^{g_i - g_j} (k_i . k_j)        (j < i)
//   T     = (I + A)^-1
//   R_i   = beta_i (v_i - e^{g_i} rk_i (K S)_i)
//   V'    = T R
//   o_i   = scale rq_i (e^{g_i} (Q S)_i + sum_{j <= i} e^{g_i - g_j} rk_j (q_i . k_j) V'_j)
//   S    <- e^{g_C} S + K^T V'',   V''_j = e^{g_C - g_j} rk_j V'_j
// The decay is a scalar per token, so every factor sits outside the matrix products and K
// and Q are MMA operands as they come from memory, bf16 without a rounding: only S, T, R
// and V'' are float32, and each is fed as two bf16 parts (x = hi + lo, 2^-17 left): states
// come out within 4e-6 of exact ones, relative (a third part would need more shared memory than
// there is); its float32 update adds up to 2^-24 a chunk, which shows where thousands of chunks
// decay slowly.  Exponents are differences of exact sums (64-bit fixed point) of steps rounded to
// 2^-41: a decay of e^-600 over the chunk costs the short ones nothing.  The product behind o alone,
// masked Q K^T times V', has both operands rounded to fp16, which keeps 11 bits where each is scaled by
// a power of two into its range: rows of the masked Q K^T by their largest possible entry, V' of a chunk
// and its 32 columns by the largest there is.  (In bf16 o was within 2.8e-3, where its own rounding is
// 1.7e-3, and where keys are alike and little decays V' cancels from token to token: 1.1e-2 for a token
// repeated; fp16 leaves 1.7e-3 and 1.8e-3 for 4.20 -> 4.23 ms.  Forming (masked Q K^T) T in prep and
// feeding R instead measures 2.2e-3 and 2.1e-3, and 4.63 ms.)
//
// prep: one CTA per (chunk, key head) forms K K^T and Q K^T once for all value heads of
// the key head, then per value head A, its inverse (16 x 16 blocks by substitution, merged
// by [[X, 0], [B, Z]]^-1 = [[X^-1, 0], [-Z^-1 B X^-1, Z^-1]]), and writes a record: T as two
// bf16 parts, the masked and scaled Q K^T in fp16, the tokens' factors.
// scan: one CTA per (sequence, value head, 32 value columns) walks the chunks.  Tokens (or
// key channels) are TMEM lanes, the 32 columns of an operand's hi and lo parts one
// 128-byte row of 64 MN-major elements: one N = 64 MMA forms both products.
//
// Neither is near HBM: prep is bound by the issue and latency of the inverse (some 19000 cycles
// of an SM per chunk and value head), the scan by its chain K S -> R -> T R -> V'' -> K^T V'' -> S,
// some 4450 cycles a chunk of which 1450 are MMAs, 1600 the rows' arithmetic and 1300 the
// hand-overs between them; 32 columns rather than 64 or 128 because 32 heads then fill 128 SMs.
// Measured: 131072 tokens, 16 key and 32 value heads, S0: 4.23 ms (31.0 M tokens/s); 8192
// tokens, 32 / 32 heads: 0.30 ms, one half prep and one half scan.
#include <math.h>

#include <algorithm>

#include "gdn.cuh"
#include "kda_common.cuh"
#include "tcgen05.cuh"
#include "tma_host.cuh"

namespace kda {
namespace gdn {

constexpr int C = 128;                        // chunk length
constexpr int DH = 128;                       // key and value width
constexpr int TILE = C * DH * 2;              // a K or Q tile: two slabs of 64 channels

// One record per (chunk, value head).  A 128 x 128 lower-triangular operand is stored as its
// slab of columns 0 .. 63 and the lower half of its slab of columns 64 .. 127 (the upper
// half is zero), rows of 128 bytes in the 128-byte swizzle.
constexpr int TRI = 16384 + 8192;
constexpr int REC_THI = 0, REC_TLO = TRI, REC_A = 2 * TRI, REC_F = 3 * TRI;
constexpr int REC_O = REC_F + C * 16 + 128;   // behind four factors per token, e^{g_C} and the record's ERR_ bits
constexpr int REC = REC_O + C * 4;            // + a factor of the masked product per token
constexpr int WS_HEAD = 256;                  // the error word's line

// For up to MAX_LISTED sequences the host lays the work out.  Scans of the longest start first: one of
// 4097 tokens among eight shorter ones otherwise starts when these are done.  Beyond, every CTA
// adds up cu_seqlens itself, and every sequence goes in chunks: the lists are kernel arguments.
//
// A chunk takes its two kernels 33 us however full it is, and where the GPU is full 240 ns for each value
// head; the recurrence 1 us a token, and where the GPU is full 20 ns for each state and 11 for each of its
// tokens.  So batches of at most SHORT tokens a sequence take the recurrence.  Chunks and recurrence, 32
// heads, us: 1 sequence of 4 tokens 33, 7, of 24 33, 26; 256 of 4 1812, 402, of 20 1822, 1670, of 24
// 1818, 1985; 1000 of 24 7065, 7655; 4 heads, 1000 of 24 910, 975: from 22 tokens on the recurrence of a full GPU
// is up to 9 % behind, that of an idle one ahead.  Such sequences in a listed batch with longer ones take it
// where the estimates say so, in a launch of their own beside the scan's last CTAs: 200 sequences of one
// token and one of 2000, 32 heads: 1490 us all in chunks, 239 so; one of 9 and one of 6433: 244, 261; 1023
// of one token and one of 2000: 7234, 841.  The list's end is a step: 1024 of one token and one
// of 2000, not listed any more, take 8451.
constexpr int SHORT = 24;

struct Params {
    kda_gdn_prefill_args a;
    uint32_t wait_limit;
    int tail;                                 // a launch for the short sequences follows the scan
    int listed;                               // whether what follows is filled in
    uint32_t first[MAX_LISTED + 1];           // chunks before sequence n (a short one has none)
    uint16_t order[MAX_LISTED];               // the sequences with chunks, longest first
};

// byte offset of 16-byte piece c (0 .. 7) of row r in a slab of 128-byte rows
KDA_DEV uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// Sequence and position of chunk `idx`, counted over the sequences; by whole warps.
KDA_DEV void chunk_at(const Params& p, long idx, int* seq, int* chunk) {
    const kda_gdn_prefill_args& a = p.a;
    if (p.listed) {
        int lo = 0, hi = a.num_seqs;          // the last sequence with first <= idx (empty ones come before it)
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.first[mid] <= (uint32_t)idx) lo = mid;
            else hi = mid;
        }
        *seq = lo;
        *chunk = (int)(idx - p.first[lo]);
        return;
    }
    const int lane = threadIdx.x & 31;
    for (int base = 0; base < a.num_seqs; base += 32) {
        const int m = base + lane;
        const int len = m < a.num_seqs ? a.cu_seqlens[m + 1] - a.cu_seqlens[m] : 0;
        int pre = (len + C - 1) / C;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, pre, o);
            if (lane >= o) pre += x;
        }
        const unsigned hit = __ballot_sync(~0u, idx < pre);
        if (hit) {
            const int f = __ffs(hit) - 1;
            const int before = __shfl_sync(~0u, pre, f > 0 ? f - 1 : 0);
            *seq = base + f;
            *chunk = (int)(idx - (f > 0 ? before : 0));
            return;
        }
        idx -= __shfl_sync(~0u, pre, 31);
    }
    *seq = 0;
    *chunk = 0;
}

// chunks of the sequences before n; by whole warps
KDA_DEV long chunks_before(const Params& p, int n) {
    if (p.listed) return p.first[n];
    const kda_gdn_prefill_args& a = p.a;
    long s = 0;
    for (int m = threadIdx.x & 31; m < n; m += 32) s += (a.cu_seqlens[m + 1] - a.cu_seqlens[m] + C - 1) / C;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    return s;
}

// x = hi + lo, both bf16: pairs packed with the lower index in the low half
KDA_DEV void split2(float x0, float x1, uint32_t* hi, uint32_t* lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&h);
    const __nv_bfloat162 l =
        __floats2bfloat162_rn(x0 - __uint_as_float(u << 16), x1 - __uint_as_float(u & 0xffff0000u));
    *hi = u;
    *lo = *reinterpret_cast<const uint32_t*>(&l);
}

KDA_DEV uint32_t pack_f16(float x0, float x1) {
    const __half2 h = __floats2half2_rn(x0, x1);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------------------
// prep
// ---------------------------------------------------------------------------
constexpr int PT = 512;                       // threads
constexpr int XS = 140;                       // row stride of the inverse's float matrix
constexpr int YS = 68;                        // and of the merges' intermediate one
constexpr int P_X = 0, P_Y = P_X + C * XS * 4, P_W = P_Y + TRI, P_END = P_W + 8 * C * 4;
constexpr int P_SMEM = P_END + 1024;
static_assert(64 * YS * 4 <= TRI && 2 * TILE <= P_Y, "the intermediate matrix shares the record part's place, the tiles the inverse's");

// x = hi + lo with hi a tf32 value; what the tensor core drops of lo is below 2^-21 of x
KDA_DEV void split_tf32(float x, float* hi, float* lo) {
    *hi = __uint_as_float(__float_as_uint(x) & 0xffffe000u);
    *lo = x - *hi;
}

// out (16 x 16, row-major with stride os) = sign L[16 x 8 nk] R[8 nk x 16], row-major float
// matrices in shared memory, by one warp: float32 operands as two tf32 parts each, the product
// of the low parts left out.  (Two bf16 parts would leave 2^-17, which the inverse of strongly
// correlated keys amplifies to 2e-5 of the state; as float32 FMAs the tiles are bound by
// shared-memory reads, 3700 cycles for the 64 x 64 products against some 2800 here.)  Within each
// step of 8, k is taken in the order 0, 2, 4, 6, 1, 3, 5, 7, so that a lane's two values of L
// are neighbours.  Six independent accumulators: the steps wait for nothing but their loads.
KDA_DEV void tile_product(float* out, int os, float sign, const float* Lm, int ls, const float* Rm, int rs, int nk, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float acc[2][3][4] = {};
    const float* l0 = Lm + g * ls + 2 * t;
    const float* r0 = Rm + 2 * t * rs + g;
#pragma unroll 2
    for (int k = 0; k < nk; ++k) {
        float ah[4], al[4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float2 x = *reinterpret_cast<const float2*>(l0 + q * 8 * ls + k * 8);
            split_tf32(x.x, &ah[q], &al[q]);
            split_tf32(x.y, &ah[q + 2], &al[q + 2]);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float bh[2], bl[2];
            const float* r = r0 + k * 8 * rs + n * 8;
            split_tf32(r[0], &bh[0], &bl[0]);
            split_tf32(r[rs], &bh[1], &bl[1]);
            tc::mma_m16n8k8_tf32(acc[n][0], ah, bh);
            tc::mma_m16n8k8_tf32(acc[n][1], al, bh);
            tc::mma_m16n8k8_tf32(acc[n][2], ah, bl);
        }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = sign * (acc[n][0][i] + (acc[n][1][i] + acc[n][2][i]));
        *reinterpret_cast<float2*>(out + g * os + n * 8 + 2 * t) = make_float2(v[0], v[1]);
        *reinterpret_cast<float2*>(out + (g + 8) * os + n * 8 + 2 * t) = make_float2(v[2], v[3]);
    }
}

__global__ void __launch_bounds__(PT, 2)
gdn_prep_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk) {
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t loaded, done;
    __shared__ uint32_t s_tmem;
    __shared__ int s_err;
    __shared__ float s_rk[C], s_rq[C], s_beta[C], s_part[4][C], s_down[C], s_wmax[4];
    __shared__ long long s_g[C], s_wsum[4];
    const kda_gdn_prefill_args& a = p.a;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = tid & 127, quarter = tid >> 7;          // TMEM lane of this thread, its share of the columns
    const int hk = blockIdx.x % a.Hk, rep = a.Hv / a.Hk;
    const long idx = blockIdx.x / a.Hk;
    int n, ch;
    chunk_at(p, idx, &n, &ch);
    const int t0 = a.cu_seqlens[n] + ch * C, len = min(C, a.cu_seqlens[n + 1] - t0);
    const bool live = row < len;

    if (tid == 0) {
        // This grid's own errors go into its records, the scan adds them to the word.
        if (blockIdx.x == 0) *reinterpret_cast<int*>(a.workspace) = 0;
        tc::mbar_init(&loaded, 1);
        tc::mbar_init(&done, 1);
        tc::mbar_fence_init();
        s_err = 0;
        tc::mbar_arrive_expect_tx(&loaded, 2 * TILE);
        for (int s = 0; s < 2; ++s) {
            tc::tma_load_3d(sm + s * 16384, &mk, s * 64, hk, t0, &loaded);
            tc::tma_load_3d(sm + TILE + s * 16384, &mq, s * 64, hk, t0, &loaded);
        }
    }
    // a head's decay logit and write strength are fetched a head ahead
    float zn = 0.f, bn = 0.f;
    auto fetch = [&](int e) {
        if (quarter == 0 && live) {
            const size_t at = (size_t)(t0 + row) * a.Hv + hk * rep + e;
            zn = __ldg(a.z + at);
            bn = __ldg(a.beta + at);
        }
    };
    fetch(0);
    if (warp == 1) {
        tc::tmem_alloc(&s_tmem, 256);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = s_tmem;
    // One thread waits and the others stop at the barrier: sixteen polling warps would take
    // issue slots from the SM's other CTA.
    auto wait_for = [&](uint64_t* bar) {
        if (tid == 0 && !tc::mbar_wait_bounded(bar, 0, p.wait_limit)) {
            const bool d = tc::mbar_wait_bounded(bar, 0, tc::WAIT_POLLS);    // give up, but not before what was issued
            s_err = d ? tc::ERR_WAIT : tc::ERR_WAIT | tc::ERR_DRAIN;
        }
        __syncthreads();
        return s_err == 0;
    };
    bool ok = wait_for(&loaded);
    if (ok) {
        // rows behind the sequence belong to its neighbour: zero them
        if (len < C) {
            for (int e = tid; e < (C - len) * 32; e += PT) {
                const int r = len + (e >> 5), q = e & 31;       // 16 pieces of K, 16 of Q
                *reinterpret_cast<uint4*>(sm + (q >> 4) * TILE + ((q >> 3) & 1) * 16384 + r * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            tc::fence_proxy_async();
            __syncthreads();
        }
        if (warp == 0) {
            const uint32_t kb = tc::smem_u32(sm), id = tc::idesc_bf16(128, 128);
            const uint64_t dk = tc::sw128_desc(kb), dq = tc::sw128_desc(kb + TILE);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
                tc::mma_f16_ss_elect(tm, dk + off, dk + off, id, k > 0);
                tc::mma_f16_ss_elect(tm + 128, dq + off, dk + off, id, k > 0);
            }
            tc::mma_commit_elect(&done);
        }
        {
            // squares of this row: two threads the key's, two the query's, 64 channels each
            const uint8_t* base = sm + quarter * 16384;
            float ss = 0.f;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint4 u = *reinterpret_cast<const uint4*>(base + swz(row, c));
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
                    ss += lo * lo + hi * hi;
                }
            }
            s_part[quarter][row] = ss;
        }
        ok = wait_for(&done);
        tc::fence_after_sync();
        if (quarter < 2) {
            const float ss = s_part[2 * quarter][row] + s_part[2 * quarter + 1][row];
            (quarter ? s_rq : s_rk)[row] = a.qk_l2norm ? rsqrtf(ss + 1e-6f) : 1.0f;
        }
    }
    uint8_t* recs = reinterpret_cast<uint8_t*>(a.workspace) + WS_HEAD + (idx * a.Hv + hk * rep) * (size_t)REC;
    for (int e = tid; !ok && e < rep; e += PT) *reinterpret_cast<int*>(recs + e * (size_t)REC + REC_F + C * 16 + 4) = s_err;
    float* X = reinterpret_cast<float*>(sm + P_X);        // the tiles have been consumed
    uint8_t* img = sm + P_Y;                              // the masked Q K^T on its way out, then Y
    float* W = reinterpret_cast<float*>(sm + P_W);        // W[b][j] = rk_j e^{g_(16 b - 1) - g_j}, j < 16 b
    constexpr float FIX = 1099511627776.f, UNFIX = 1.f / 1099511627776.f;      // 2^40
    for (int e = 0; ok && e < rep; ++e) {
        const int h = hk * rep + e;
        uint8_t* rec = recs + e * (size_t)REC;
        // sums of the log-decays (base 2) in fixed point: a step is rounded to 2^-41 (to nearest: a
        // cut would make every state last longer), the sums are exact, below 2^59.  A step below
        // -4096 is an exponential of 0 in any sum; a NaN travels with beta.
        if (quarter == 0) {
            long long g = 0;
            float beta = 0.f;
            if (live) {
                const float x = log_decay_mode(zn, __expf(__ldg(a.A + h)), a.g_min, a.gate_mode) * 1.4426950408889634f;
                beta = x == x ? bn : x;
                g = __float2ll_rn(fminf(fmaxf(x, -4096.f), 4096.f) * FIX);
            }
            if (e + 1 < rep) fetch(e + 1);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(~0u, g, o);
                if (lane >= o) g += y;
            }
            if (lane == 31) s_wsum[warp] = g;
            asm volatile("bar.sync 1, 128;" ::: "memory");
            for (int w = 0; w < warp; ++w) g += s_wsum[w];
            s_g[row] = g;
            s_beta[row] = beta;
            // The largest entry that the masked Q K^T can have in this row, as a power of two: 1 between unit
            // vectors, else |q_i| max_j e^{g_i - g_j} |k_j|.
            float up = 1.f;
            if (!a.qk_l2norm) {
                const float gi = (float)g * UNFIX;
                float m = __log2f(s_part[0][row] + s_part[1][row]) * 0.5f - gi;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float y = __shfl_up_sync(~0u, m, o);
                    if (lane >= o) m = fmaxf(m, y);
                }
                if (lane == 31) s_wmax[warp] = m;
                asm volatile("bar.sync 1, 128;" ::: "memory");
                for (int w = 0; w < warp; ++w) m = fmaxf(m, s_wmax[w]);
                m += gi + __log2f(s_part[2][row] + s_part[3][row]) * 0.5f;
                up = exp2f(fminf(fmaxf(ceilf(m), -100.f), 100.f));
            }
            s_down[row] = 1.f / up;
            *reinterpret_cast<float*>(rec + REC_O + row * 4) = up * a.scale;
        }
        __syncthreads();
        const long long gi = s_g[row], gC = s_g[C - 1];
        for (int j = tid; j < 8 * C; j += PT) {
            const int b = j / C, c = j % C;
            W[j] = c < 16 * b ? s_rk[c] * exp2f((float)(s_g[16 * b - 1] - s_g[c]) * UNFIX) : 0.f;
        }
        if (quarter == 1) {
            const float eg = exp2f((float)gi * UNFIX), beta = s_beta[row];
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live)
                f = make_float4(beta, beta * eg * s_rk[row], exp2f((float)(gC - gi) * UNFIX) * s_rk[row],
                                eg * s_rq[row] * a.scale);
            *reinterpret_cast<float4*>(rec + REC_F + row * 16) = f;
            if (row == 0) {
                // The state is multiplied by e^{g_C} once a chunk.  exp2f is low by 0.5 to 2e-8 on average
                // just below 0, which a state that hardly decays would add up; 1 + expm1 rounds without a bias.
                const float x = (float)gC * UNFIX, t = x * 0.6931471805599453f;
                *reinterpret_cast<float2*>(rec + REC_F + C * 16) = make_float2(t > -0.25f ? 1.0f + expm1f(t) : exp2f(x), 0.f);
            }
        }
        if (tid == 0) tc::bulk_wait_read();       // the last head's image has left
        __syncthreads();
        // A into X and the masked Q K^T into its image: 16 x 16 blocks on and below the diagonal,
        // column block quarter or quarter + 4 of the row
        {
            const int b = row >> 4;
            const float u = b ? exp2f((float)(gi - s_g[16 * b - 1]) * UNFIX) : 0.f;     // e^{g_i - g_(16 b - 1)}
            const float ka = live ? s_beta[row] * s_rk[row] : 0.f, qa = live ? s_rq[row] * s_down[row] : 0.f;
            const float kau = ka * u, qau = qa * u;
            const uint32_t lane0 = tm + ((uint32_t)(warp & 3) << 21);
#pragma unroll 1
            for (int cb = quarter; cb < 8; cb += 4) {
                if (cb >= 4 && (warp & 3) < 2) break;        // rows 0 .. 63 have no columns behind 63
                uint8_t* dst = img + (cb < 4 ? 0 : 16384 - 64 * 128);
                const int piece = (cb & 3) * 2;
                float G[16], P[16];
                tc::tmem_ld16(lane0 + cb * 16, G);
                tc::tmem_ld16(lane0 + 128 + cb * 16, P);
                tc::tmem_ld_wait();
                uint32_t q[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (cb < b) {
                    // below the diagonal nothing is masked, and rows behind the sequence have ka = qa = 0
                    // over zeroed (finite) products
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const float4 w = *reinterpret_cast<const float4*>(W + b * C + cb * 16 + c);
                        *reinterpret_cast<float4*>(X + row * XS + cb * 16 + c) =
                            make_float4(kau * (w.x * G[c]), kau * (w.y * G[c + 1]), kau * (w.z * G[c + 2]), kau * (w.w * G[c + 3]));
                        q[c >> 1] = pack_f16(qau * (w.x * P[c]), qau * (w.y * P[c + 1]));
                        q[(c >> 1) + 1] = pack_f16(qau * (w.z * P[c + 2]), qau * (w.w * P[c + 3]));
                    }
                } else if (cb == b) {
                    // masked places by selection, not by a product with 0
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        float x[4], y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int j = cb * 16 + c + i;
                            const float w = s_rk[j] * exp2f((float)(gi - s_g[j]) * UNFIX);      // rk_j e^{g_i - g_j}
                            x[i] = j < row && live ? ka * w * G[c + i] : 0.f;
                            y[i] = j <= row && live ? qa * w * P[c + i] : 0.f;
                        }
                        *reinterpret_cast<float4*>(X + row * XS + cb * 16 + c) = make_float4(x[0], x[1], x[2], x[3]);
                        q[c >> 1] = pack_f16(y[0], y[1]);
                        q[(c >> 1) + 1] = pack_f16(y[2], y[3]);
                    }
                }
                *reinterpret_cast<uint4*>(dst + swz(row, piece)) = make_uint4(q[0], q[1], q[2], q[3]);
                *reinterpret_cast<uint4*>(dst + swz(row, piece + 1)) = make_uint4(q[4], q[5], q[6], q[7]);
                __syncwarp();
            }
            tc::fence_proxy_async();
        }
        __syncthreads();
        if (tid == 0) {
            tc::bulk_store(rec + REC_A, img, TRI);
            tc::bulk_commit();
        }
        // inverses of the diagonal blocks: lane c < 16 of warp b solves for column c of block b
        if (warp >= 8) {
            float* B = X + (warp - 8) * 16 * XS + (warp - 8) * 16;
            float x[16];
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float s = i == lane ? 1.f : 0.f, s2 = 0.f;
#pragma unroll
                    for (int j = 0; j < i; j += 4) {           // B's row in fours: its upper part is zero
                        const float4 r = *reinterpret_cast<const float4*>(B + i * XS + j);
                        s -= r.x * x[j];
                        if (j + 1 < i) s2 -= r.y * x[j + 1];
                        if (j + 2 < i) s -= r.z * x[j + 2];
                        if (j + 3 < i) s2 -= r.w * x[j + 3];
                    }
                    x[i] = s + s2;
                }
            }
            __syncwarp();
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < 16; ++i) B[i * XS + lane] = x[i];
            }
        }
        if (tid == 0) tc::bulk_wait_read();       // the image becomes Y
        __syncthreads();
        // Merges to blocks of 32, 64, 128 in 16 x 16 tiles, a warp each: Y = B X, then - Z Y with Z the
        // lower block's inverse.  X and Z are lower triangular: k from the tile's column on, and up
        // to the tile's row; the tiles are dealt so that every scheduler gets long and short ones.
        float* Y = reinterpret_cast<float*>(img);
#pragma unroll 1
        for (int s = 16; s < C; s *= 2) {
            const int nb = s / 16, per = nb * nb, m = warp / per, i = (warp % per) / nb, j = (i + warp) % nb, o = m * 2 * s;
            const bool on = m < C / (2 * s);
            if (on)         // tile (i, j)
                tile_product(Y + (m * s + 16 * i) * YS + 16 * j, YS, 1.f, X + (o + s + 16 * i) * XS + o + 16 * j, XS,
                             X + (o + 16 * j) * XS + o + 16 * j, XS, 2 * (nb - j), lane);
            __syncthreads();
            if (on)         // tile (j, i): the result takes B's place
                tile_product(X + (o + s + 16 * j) * XS + o + 16 * i, XS, -1.f, X + (o + s + 16 * j) * XS + o + s, XS,
                             Y + m * s * YS + 16 * i, YS, 2 * (j + 1), lane);
            __syncthreads();
        }
        // T = hi + lo, 16 bytes of each per thread and step; blocks above the diagonal are zero
        for (int i = tid; i < (C + 64) * 8; i += PT) {
            const int c = i & 7, rr = i >> 3;
            const int r = rr < C ? rr : rr - 64, col = (rr < C ? 0 : 64) + c * 8;
            uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
            if (col / 16 <= r / 16) {
                const float4 x = *reinterpret_cast<const float4*>(X + r * XS + col), y = *reinterpret_cast<const float4*>(X + r * XS + col + 4);
                split2(x.x, x.y, &hi[0], &lo[0]);
                split2(x.z, x.w, &hi[1], &lo[1]);
                split2(y.x, y.y, &hi[2], &lo[2]);
                split2(y.z, y.w, &hi[3], &lo[3]);
            }
            const uint32_t at = (rr < C ? 0 : 16384 - 64 * 128) + swz(r, c);
            *reinterpret_cast<uint4*>(rec + REC_THI + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(rec + REC_TLO + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        __syncthreads();
    }
    if (tid == 0) tc::bulk_wait_all();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) tc::tmem_dealloc(tm, 256);
}

// ---------------------------------------------------------------------------
// scan
// ---------------------------------------------------------------------------
constexpr int COLS = 32;                      // value columns per CTA
constexpr int ST = 448;                       // warps 0-7 state rows, 8-11 output rows, 12 loads, 13 MMAs
constexpr int S_K = 0, S_Q = 2 * TILE, S_THI = 3 * TILE, S_TLO = S_THI + 32768, S_A = S_TLO + 32768,
              S_S = S_A + 32768, S_R = S_S + 16384, S_END = S_R + 16384;
constexpr int S_SMEM = S_END + 1024;
// The zero half-slabs of the triangular operands are lent out while no MMA reads them and
// zeroed again by their readers (all are 128 rows of 64 bytes, 64-byte swizzle): T's high part
// takes the chunk's values v until R is formed, its low part V' in fp16 (the masked product's
// operand) from T R on, the masked Q K^T the output rows on their way out.
constexpr int S_VIN = S_THI + 16384, S_V = S_TLO + 16384, S_O = S_A + 16384;
// TMEM columns (Q S twice: the outputs of a chunk are read while the next one's are formed)
constexpr int D_KS = 0, D_TR = 64, D_KV = 128, D_AV = 192, D_QS = 256, D_COLS = 512;

// descriptor of the 128 x 32 MN-major operand with 64-byte rows (64-byte swizzle)
KDA_DEV uint64_t sw64_desc_mn(uint32_t addr) {
    uint64_t d = 0;
    d |= (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)1 << 16;                            // one 32-element block: unused
    d |= (uint64_t)((512u >> 4) & 0x3FFFu) << 32;      // 8-row K groups
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)4 << 61;                            // 64-byte swizzle
    return d;
}

// byte offset of 16-byte piece c (0 .. 3) of row r in rows of 64 bytes
KDA_DEV uint32_t swz64(int r, int c) { return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

// A wait that gives up by raising *abort and going on: everything behind it stays within
// the CTA's own buffers and rows, later waits return soon, and the roles look at *abort
// every eighth chunk (a vote in every wait would cost the serial chain some 50 cycles each).
KDA_DEV void wait_go(uint64_t* bar, uint32_t parity, uint32_t limit, volatile int* abort) {
    if (limit && tc::mbar_try_wait(bar, parity)) return;
    tc::mbar_wait_role(bar, parity, limit, abort);
}

// whether any of the 128 output threads says so
KDA_DEV bool any_of_128(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((uint32_t)x) : "memory");
    return r != 0;
}
// and of the 256 state threads
KDA_DEV bool any_of_256(bool x) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"((uint32_t)x) : "memory");
    return r != 0;
}

// this thread's 16 columns of a row, hi and lo parts, into the 128-byte row [hi 32 | lo 32]
KDA_DEV void store_split(uint8_t* base, int row, int w, const float* x) {
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split2(x[2 * i], x[2 * i + 1], &hi[i], &lo[i]);
    *reinterpret_cast<uint4*>(base + swz(row, 2 * w)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(base + swz(row, 2 * w + 1)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
    *reinterpret_cast<uint4*>(base + swz(row, 4 + 2 * w)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(base + swz(row, 5 + 2 * w)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
}

__global__ void __launch_bounds__(ST, 1)
gdn_scan_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t k_full[2], k_empty[2], q_full, t_full, a_full, v_full, edge, s_ready, r_ready, v_ready, av_ready,
        ks_done, qs_done, tr_done, kv_done, av_done, drained;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ __align__(16) float s_vmax[8];
    __shared__ float s_vup[2];
    const kda_gdn_prefill_args& a = p.a;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slice = blockIdx.x % (DH / COLS);
    const int h = blockIdx.x / (DH / COLS) % a.Hv;
    const int place = blockIdx.x / (DH / COLS) / a.Hv, n = p.listed ? p.order[place] : place;
    const int hk = h / (a.Hv / a.Hk);
    const int t0 = a.cu_seqlens[n], T = a.cu_seqlens[n + 1] - t0;
    const int nc = (T + C - 1) / C;
    const uint32_t limit = p.wait_limit;
    volatile int* abort = &s_abort;

    if (tid == 0) {
        uint64_t* ones[] = {&k_full[0], &k_full[1], &k_empty[0], &k_empty[1], &q_full, &t_full, &a_full, &v_full, &edge, &ks_done,
                            &qs_done, &tr_done, &kv_done, &av_done, &drained};
        for (uint64_t* b : ones) tc::mbar_init(b, 1);
        tc::mbar_init(&s_ready, 8);         // warps
        tc::mbar_init(&r_ready, 8 + 4);
        tc::mbar_init(&v_ready, 8);
        tc::mbar_init(&av_ready, 8 + 4);
        tc::mbar_fence_init();
        s_abort = 0;
    }
    // the halves above the diagonal of the three triangular operands
    for (int i = tid; i < 3 * 512; i += ST)
        *reinterpret_cast<uint4*>(sm + S_THI + (i >> 9) * 32768 + 16384 + (i & 511) * 16) = make_uint4(0, 0, 0, 0);
    tc::fence_proxy_async();
    if (warp == 13) {
        tc::tmem_alloc(&s_tmem, D_COLS);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = s_tmem;
    if (p.tail) tc::launch_dependents();
    tc::wait_prerequisites();                 // prep's records
    const long base = chunks_before(p, n);
    const uint8_t* recs = reinterpret_cast<const uint8_t*>(a.workspace) + WS_HEAD + (base * a.Hv + h) * (size_t)REC;
    const size_t rec_step = (size_t)a.Hv * REC;

    if (warp == 12) {
        // ---------------- loads ----------------
        // Stops at a wait that gave up: arming a barrier whose last phase is open is not defined.
        auto wait_all = [&](uint64_t* bar, uint32_t parity) {
            wait_go(bar, parity, limit, abort);
            return !__any_sync(~0u, *abort);
        };
        uint32_t nk0 = 0, nk1 = 0, nq = 0, nt = 0, na = 0, ne = 0;    // phases begun per barrier
        for (int c = 0; c < nc; ++c) {
            if (__any_sync(~0u, *abort)) break;
            const uint8_t* rec = recs + c * rec_step;
            const int b = c & 1, left = T - c * C;
            uint8_t* kt = sm + S_K + b * TILE;
            if (c >= 2 && !wait_all(&k_empty[b], (c / 2 - 1) & 1)) break;
            const bool zero = left < C;                  // rows of the next sequence: 0 x NaN
            uint64_t* bar = zero ? &edge : &k_full[b];
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(bar, TILE);
                for (int s = 0; s < 2; ++s) tc::tma_load_3d(kt + s * 16384, &mk, s * 64, hk, t0 + c * C, bar);
            }
            if (zero) ++ne;
            else if (b) ++nk1;
            else ++nk0;
            if (c >= 1 && !wait_all(&qs_done, (c - 1) & 1)) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&q_full, TILE);
                for (int s = 0; s < 2; ++s) tc::tma_load_3d(sm + S_Q + s * 16384, &mq, s * 64, hk, t0 + c * C, &q_full);
            }
            ++nq;
            if (zero) {
                if (!wait_all(&edge, 0)) break;
                for (int e = lane; e < (C - left) * 16; e += 32) {
                    const int r = left + (e >> 4), q = e & 15;
                    *reinterpret_cast<uint4*>(kt + (q >> 3) * 16384 + r * 128 + (q & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&k_full[b]);
                if (b) ++nk1;
                else ++nk0;
            }
            if (c >= 1 && !wait_all(&tr_done, (c - 1) & 1)) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&v_full, C * COLS * 2);
                tc::tma_load_3d(sm + S_VIN, &mv, slice * COLS, h, t0 + c * C, &v_full);
                tc::mbar_arrive_expect_tx(&t_full, 2 * TRI);
                tc::bulk_load(sm + S_THI, rec + REC_THI, 16384, &t_full);
                tc::bulk_load(sm + S_THI + 16384 + 8192, rec + REC_THI + 16384, 8192, &t_full);
                tc::bulk_load(sm + S_TLO, rec + REC_TLO, 16384, &t_full);
                tc::bulk_load(sm + S_TLO + 16384 + 8192, rec + REC_TLO + 16384, 8192, &t_full);
            }
            ++nt;
            if (c >= 1 && !wait_all(&av_done, (c - 1) & 1)) break;
            if (lane == 0) {
                tc::mbar_arrive_expect_tx(&a_full, TRI);
                tc::bulk_load(sm + S_A, rec + REC_A, 16384, &a_full);
                tc::bulk_load(sm + S_A + 16384 + 8192, rec + REC_A + 16384, 8192, &a_full);
                // two chunks ahead into L2: this slice's values, and its share of what all slices read
                if (c + 2 < nc) {
                    const uint8_t* far = rec + 2 * rec_step;
                    const int t2 = t0 + (c + 2) * C;
                    tc::tma_prefetch_3d(&mv, slice * COLS, h, t2);
                    if (slice < 2) tc::tma_prefetch_3d(&mk, slice * 64, hk, t2);
                    else tc::tma_prefetch_3d(&mq, (slice - 2) * 64, hk, t2);
                    if (slice < 3) tc::bulk_prefetch(far + slice * TRI, TRI);
                    else tc::bulk_prefetch(far + REC_F, REC - REC_F);
                }
            }
            ++na;
        }
        // the last phase of every load has landed before the CTA leaves
        if (lane == 0) {
            const bool d = tc::drain_phase(&edge, ne) && tc::drain_phase(&k_full[0], nk0) && tc::drain_phase(&k_full[1], nk1) &&
                           tc::drain_phase(&q_full, nq) && tc::drain_phase(&t_full, nt) && tc::drain_phase(&v_full, nt) &&
                           tc::drain_phase(&a_full, na);
            if (*abort || !d)
                atomicOr(reinterpret_cast<int*>(a.workspace), d ? tc::ERR_WAIT : tc::ERR_WAIT | tc::ERR_DRAIN);
        }
    } else if (warp == 13) {
        // ---------------- MMAs: the warp computes together, one lane issues ----------------
        // Per chunk 48 MMAs of 41 (N = 32) or 47 (N = 64) cycles: K S, T R and K^T V'' on the chain from
        // state to state, Q S and (masked Q K^T) V' in the gaps that the rows' arithmetic leaves.
        const uint32_t tmu = __shfl_sync(~0u, tm, 0), sb = __shfl_sync(~0u, tc::smem_u32(sm), 0);
        const uint32_t id64 = tc::idesc_bf16(128, 64, false, true), id32 = tc::idesc_bf16(128, 32, false, true),
                       idt = tc::idesc_bf16(128, 64, true, true), idh = tc::idesc_f16(128, 32, false, true);
        const uint64_t dS = tc::sw128_desc_mn(sb + S_S, 16384), dR = tc::sw128_desc_mn(sb + S_R, 16384);
        // D[., cols] = A (K-major tile of two slabs) times B (MN-major, 16 K rows per step)
        auto rows = [&](uint32_t d, uint64_t ad, uint64_t bd, uint32_t step, uint32_t id, bool acc) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                tc::mma_f16_ss_elect(d, ad + (((k >> 2) * 16384 + (k & 3) * 32) >> 4), bd + k * (step >> 4), id, acc || k > 0);
        };
        // Turn i: K^T V'' and (masked Q K^T) V' of chunk i - 1, then K S, Q S and T R of chunk i.  The
        // way back to the loop's top (some 500 cycles of instruction fetch) so falls into the
        // wait for V'', not between a state and the next K S.
#pragma unroll 1
        for (int i = 0; i <= nc; ++i) {
            if ((i & 7) == 7 && __any_sync(~0u, *abort)) break;
            if (i > 0) {
                const uint32_t ph = (i - 1) & 1;
                const uint64_t dKt = tc::sw128_desc_mn(sb + S_K + ph * TILE, 16384);
                wait_go(&v_ready, ph, limit, abort);
                __syncwarp();
                tc::fence_after_sync();
#pragma unroll
                for (int k = 0; k < 8; ++k)                                        // K^T: tokens are the K rows
                    tc::mma_f16_ss_elect(tmu + D_KV, dKt + k * (2048 >> 4), dR + k * (2048 >> 4), idt, k > 0);
                tc::mma_commit_elect(&kv_done);
                tc::mma_commit_elect(&k_empty[ph]);
                wait_go(&a_full, ph, limit, abort);
                wait_go(&av_ready, ph, limit, abort);
                __syncwarp();
                tc::fence_after_sync();
                rows(tmu + D_AV, tc::sw128_desc(sb + S_A), sw64_desc_mn(sb + S_V), 1024, idh, false);
                tc::mma_commit_elect(&av_done);
            }
            if (i < nc) {
                const uint32_t ph = i & 1;
                const uint64_t dK = tc::sw128_desc(sb + S_K + ph * TILE);
                wait_go(&k_full[ph], (i / 2) & 1, limit, abort);
                wait_go(&s_ready, ph, limit, abort);
                __syncwarp();
                tc::fence_after_sync();
                rows(tmu + D_KS, dK, dS, 2048, id64, false);
                tc::mma_commit_elect(&ks_done);
                wait_go(&q_full, ph, limit, abort);
                __syncwarp();
                rows(tmu + D_QS + 64 * ph, tc::sw128_desc(sb + S_Q), dS, 2048, id64, false);
                tc::mma_commit_elect(&qs_done);
                wait_go(&t_full, ph, limit, abort);
                wait_go(&r_ready, ph, limit, abort);
                __syncwarp();
                tc::fence_after_sync();
                rows(tmu + D_TR, tc::sw128_desc(sb + S_THI), dR, 2048, id64, false);
                rows(tmu + D_TR, tc::sw128_desc(sb + S_TLO), dR, 2048, id32, true);
                tc::mma_commit_elect(&tr_done);
            }
        }
        __syncwarp();
        tc::mma_commit_elect(&drained);
        if (lane == 0) {
            if (!tc::mbar_wait_bounded(&drained, 0, tc::WAIT_POLLS))
                atomicOr(reinterpret_cast<int*>(a.workspace), tc::ERR_WAIT | tc::ERR_DRAIN);
        }
        __syncwarp();
    } else if (warp >= 8) {
        // ---------------- output rows: one token per thread, 32 columns ----------------
        const int row = tid & 127;
        const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21);
        if (nc > 0) {
            tc::mbar_arrive_warp(&r_ready);
            tc::mbar_arrive_warp(&av_ready);
        }
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            if ((c & 7) == 7 && any_of_128(*abort != 0)) break;    // all four warps or none: they share barriers
            const uint32_t ph = c & 1;
            const float fw = __ldcg(reinterpret_cast<const float*>(recs + c * rec_step + REC_F + row * 16 + 12));
            const float fo = __ldcg(reinterpret_cast<const float*>(recs + c * rec_step + REC_O + row * 4));
            float o[32], x[32];
            // A V' is the chunk's last product, and the next one waits for these rows: a barrier that
            // could run two phases ahead of its reader (that of Q S) is not waited on here
            wait_go(&av_done, ph, limit, abort);
            __syncwarp();
            tc::fence_after_sync();
            tc::tmem_ld32(tl + D_QS + 64 * ph, o);
            tc::tmem_ld32(tl + D_QS + 64 * ph + 32, x);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = fw * (o[i] + x[i]);                // scale rq e^g (Q S)
            tc::tmem_ld32(tl + D_AV, x);
            const float fv = fo * s_vup[ph];                                       // undoes both operands' scaling
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(sm + S_V + row * 64 + 16 * i) = zero;   // T's zeros again
            tc::tmem_ld_wait();
            tc::fence_proxy_async();
            tc::fence_before_sync();
            if (c + 1 < nc) tc::mbar_arrive_warp(&r_ready);
            const bool whole = (c + 1) * C <= T;
            if (a.o) {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] += fv * x[i];
                if (whole) {
                    // through shared memory and one TMA store; the last chunk's rows one by one
#pragma unroll
                    for (int i = 0; i < 4; ++i) store8_bf16(reinterpret_cast<uint16_t*>(sm + S_O + swz64(row, i)), o + 8 * i);
                    tc::fence_proxy_async();
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    if (tid == 256) {
                        tc::tma_store_3d(&mo, slice * COLS, h, t0 + c * C, sm + S_O);
                        tc::bulk_commit();
                        tc::bulk_wait_read();
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
                    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(sm + S_O + row * 64 + 16 * i) = zero;
                    tc::fence_proxy_async();
                } else if (c * C + row < T) {
                    uint16_t* out = reinterpret_cast<uint16_t*>(a.o) + ((size_t)(t0 + c * C + row) * a.Hv + h) * DH + slice * COLS;
#pragma unroll
                    for (int i = 0; i < 4; ++i) store8_bf16(out + 8 * i, o + 8 * i);
                }
            }
            if (c + 1 < nc) tc::mbar_arrive_warp(&av_ready);
            __syncwarp();
        }
        if (tid == 256) tc::bulk_wait_all();
    } else {
        // ---------------- state rows: thread (row, w) owns columns 16 w .. 16 w + 15 of its row ----------------
        const int row = tid & 127, w = tid >> 7;
        const int col = slice * COLS + 16 * w;
        const uint32_t tl = tm + ((uint32_t)(warp & 3) << 21) + 16 * w;
        const size_t sbase = ((size_t)n * a.Hv + h) * (size_t)DH * DH + (size_t)row * DH + col;   // row = key channel
        float S[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 x = a.S0 ? *reinterpret_cast<const float4*>(a.S0 + sbase + i) : make_float4(0.f, 0.f, 0.f, 0.f);
            S[i] = x.x; S[i + 1] = x.y; S[i + 2] = x.z; S[i + 3] = x.w;
        }
        // A chunk's factors are fetched while T R of the chunk before runs: the next proxy fence, which
        // waits for loads in flight, is then as far as their latency.
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f), fn = f;
        float gamma = 0.f, gn = 0.f;
        int err = 0;                         // of the records
        auto fetch = [&](int c) {
            const uint8_t* rec = recs + c * rec_step;
            // (not the read-only path: the grid before may still be writing when this one starts)
            fn = __ldcg(reinterpret_cast<const float4*>(rec + REC_F + row * 16));
            const float2 ge = __ldcg(reinterpret_cast<const float2*>(rec + REC_F + C * 16));
            gn = ge.x;
            err |= __float_as_int(ge.y);
        };
        if (nc > 0) fetch(0);
        // R = beta (v - e^g rk K S) of chunk c; the values' place is zero again afterwards
        float x[16], y[16];
        auto form_r = [&](int c) {
            const uint32_t ph = c & 1;
            const bool live = c * C + row < T;                // row = token
            wait_go(&v_full, ph, limit, abort);
            __syncwarp();
            uint4* vp = reinterpret_cast<uint4*>(sm + S_VIN + swz64(row, 2 * w));
            uint4* vq = reinterpret_cast<uint4*>(sm + S_VIN + swz64(row, 2 * w + 1));
            const uint4 va = *vp, vc = *vq;
            *vp = *vq = make_uint4(0, 0, 0, 0);
            wait_go(&ks_done, ph, limit, abort);
            __syncwarp();
            tc::fence_after_sync();
            tc::tmem_ld16(tl + D_KS, x);
            tc::tmem_ld16(tl + D_KS + 32, y);
            tc::tmem_ld_wait();
            const uint32_t vr[8] = {va.x, va.y, va.z, va.w, vc.x, vc.y, vc.z, vc.w};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float v = __uint_as_float(i & 1 ? vr[i >> 1] & 0xffff0000u : vr[i >> 1] << 16);
                x[i] = live ? f.x * v - f.y * (x[i] + y[i]) : 0.f;
            }
            store_split(sm + S_R, row, w, x);
            tc::fence_proxy_async();
            tc::fence_before_sync();
            tc::mbar_arrive_warp(&r_ready);
        };
        auto give_s = [&] {
            store_split(sm + S_S, row, w, S);
            tc::fence_proxy_async();
            tc::fence_before_sync();
            tc::mbar_arrive_warp(&s_ready);
        };
        // The loop turns over while T R runs: from R of one chunk to R of the next.
#pragma unroll 1
        for (int i = 0; i <= nc; ++i) {
            if ((i & 7) == 7 && any_of_256(*abort != 0)) break;    // all eight warps or none: they share a barrier
            if (i > 0) {
                const int c = i - 1;
                const uint32_t ph = c & 1;
                const bool live = c * C + row < T;
                // V' = T R, and V'' = e^{g_C - g} rk V' over R (T R is done with it)
                wait_go(&tr_done, ph, limit, abort);
                __syncwarp();
                tc::fence_after_sync();
                tc::tmem_ld16(tl + D_TR, x);
                tc::tmem_ld16(tl + D_TR + 32, y);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    x[e] = live ? x[e] + y[e] : 0.f;
                    y[e] = x[e] * f.z;
                }
                store_split(sm + S_R, row, w, y);
                tc::fence_proxy_async();
                tc::fence_before_sync();
                tc::mbar_arrive_warp(&v_ready);
                // V' for o, while K^T V'' runs: fp16, the largest of the chunk's 128 x 32 below 2^15.  (Where
                // that is infinite nothing is scaled, so that no finite value becomes 0 beside it.)
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
                m = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(m)));
                if (lane == 0) s_vmax[warp] = m;
                asm volatile("bar.sync 2, 256;" ::: "memory");
                const float4 m0 = *reinterpret_cast<const float4*>(s_vmax), m1 = *reinterpret_cast<const float4*>(s_vmax + 4);
                m = fmaxf(fmaxf(fmaxf(m0.x, m0.y), fmaxf(m0.z, m0.w)), fmaxf(fmaxf(m1.x, m1.y), fmaxf(m1.z, m1.w)));
                int ex = (int)(__float_as_uint(m) >> 23);              // biased exponent: m < 2^(ex - 126)
                ex = ex == 255 ? 141 : max(ex, 16);
                const float down = __uint_as_float((uint32_t)(268 - ex) << 23);              // 2^(141 - ex)
                if (tid == 0) s_vup[ph] = __uint_as_float((uint32_t)(ex - 14) << 23);        // 2^(ex - 141)
                uint32_t vh[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) vh[e] = pack_f16(x[2 * e] * down, x[2 * e + 1] * down);
                *reinterpret_cast<uint4*>(sm + S_V + swz64(row, 2 * w)) = make_uint4(vh[0], vh[1], vh[2], vh[3]);
                *reinterpret_cast<uint4*>(sm + S_V + swz64(row, 2 * w + 1)) = make_uint4(vh[4], vh[5], vh[6], vh[7]);
                tc::fence_proxy_async();
                tc::mbar_arrive_warp(&av_ready);
                // S <- e^{g_C} S + K^T V''
                wait_go(&kv_done, ph, limit, abort);
                __syncwarp();
                tc::fence_after_sync();
                tc::tmem_ld16(tl + D_KV, x);
                tc::tmem_ld16(tl + D_KV + 32, y);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) S[e] = gamma * S[e] + (x[e] + y[e]);
            }
            if (i < nc) {
                give_s();
                f = fn;
                gamma = gn;
                form_r(i);
                if (i + 1 < nc) fetch(i + 1);
            }
        }
        if (tid == 0 && err) atomicOr(reinterpret_cast<int*>(a.workspace), err);
        if (a.S_T) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(a.S_T + sbase + i) = make_float4(S[i], S[i + 1], S[i + 2], S[i + 3]);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 13) tc::tmem_dealloc(tm, D_COLS);
}

// ---------------------------------------------------------------------------

static long count_chunks(const kda_gdn_prefill_args& a) {
    long s = 0;
    for (int n = 0; n < a.num_seqs; ++n) s += (a.cu_seqlens_host[n + 1] - a.cu_seqlens_host[n] + C - 1) / C;
    return s;
}

size_t chunked_workspace_size(const kda_gdn_prefill_args& a) {
    return WS_HEAD + (size_t)count_chunks(a) * a.Hv * REC;
}

cudaError_t launch_chunked(const kda_gdn_prefill_args& a, cudaStream_t s) {
    const int32_t* cu = a.cu_seqlens_host;
    const auto len = [cu](int n) { return cu[n + 1] - cu[n]; };
    Params p;
    Sequences few;                            // the short ones
    p.a = a;
    p.wait_limit = wait_limit();
    p.listed = a.num_seqs <= MAX_LISTED;
    few.count = 0;
    long chunks = count_chunks(a);
    int scans = a.num_seqs, longest = 0;
    for (int n = 0; n < a.num_seqs; ++n) longest = std::max(longest, len(n));
    if (longest <= SHORT) return launch_recurrent(a, few, s);       // all of them; clears the error word
    if (p.listed) {
        long shorts = 0, tokens = 0;
        int most = 0;                         // tokens of a short one
        for (int n = 0; n < a.num_seqs; ++n)
            if (len(n) <= SHORT) { ++shorts; tokens += len(n); most = std::max(most, len(n)); }
        const double chunked = 0.24 * shorts * a.Hv, apart = 4 + std::max((double)most, (0.02 * shorts + 0.011 * tokens) * a.Hv);   // us
        const int least = apart < chunked ? SHORT + 1 : 0;
        p.first[0] = 0;
        scans = 0;
        for (int n = 0; n < a.num_seqs; ++n) {
            const bool in_chunks = len(n) >= least;
            p.first[n + 1] = p.first[n] + (in_chunks ? (uint32_t)((len(n) + C - 1) / C) : 0);
            if (in_chunks) p.order[scans++] = (uint16_t)n;
            else few.seq[few.count++] = (uint16_t)n;
        }
        std::stable_sort(p.order, p.order + scans, [len](uint16_t x, uint16_t y) { return len(x) > len(y); });
        chunks = p.first[a.num_seqs];
    }
    p.tail = few.count > 0;
    CUtensorMap mq = {}, mk = {}, mv = {}, mo = {};
    cudaError_t e = make_map_heads(&mq, a.q, DH, a.Hk, a.T_total, (uint64_t)a.Hk * DH, 1, C);
    if (e == cudaSuccess) e = make_map_heads(&mk, a.k, DH, a.Hk, a.T_total, (uint64_t)a.Hk * DH, 1, C);
    if (e == cudaSuccess) e = make_map_heads(&mv, a.v, DH, a.Hv, a.T_total, (uint64_t)a.Hv * DH, 1, C, COLS);
    if (e == cudaSuccess && a.o) e = make_map_heads(&mo, a.o, DH, a.Hv, a.T_total, (uint64_t)a.Hv * DH, 1, C, COLS);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P_SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(gdn_scan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S_SMEM);
    if (e != cudaSuccess) return e;
    gdn_prep_kernel<<<(unsigned)(chunks * a.Hk), PT, P_SMEM, s>>>(p, mq, mk);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    count_launches(1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long)scans * a.Hv * (DH / COLS)));
    cfg.blockDim = dim3(ST);
    cfg.dynamicSmemBytes = S_SMEM;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    // The scan's start beside prep's end: 33 tokens 43.1 -> 40.2 us, 8192 306 -> 303.  (Started as soon as
    // all of prep has, its CTAs are in the way of prep's last ones: 308.)
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, gdn_scan_kernel, p, mq, mk, mv, mo);
    if (e != cudaSuccess) return e;
    count_launches(1);
    if (!few.count) return cudaSuccess;
    kda_gdn_prefill_args rest = a;
    rest.workspace = nullptr;                 // the error word is the others'
    return launch_recurrent(rest, few, s);
}

}  // namespace gdn
}  // namespace kda
