// Gated delta rule with one decay per value head: the per-token recurrence and
// the batched decode step.
//
//   S_bar = e^g S,  u = beta (v - S_bar^T k),  S <- S_bar + k u^T,
//   o = scale (S_bar^T q + (k.q) u)
//
// The columns of S (value channels) are independent of one another, so a state
// can be cut into column slices of COLS channels, one CTA each: nothing is
// exchanged between the slices, only k, q (2 x 128 values) are read again.
#include "gdn.cuh"
#include "kda_common.cuh"
#include "tcgen05.cuh"

namespace kda {
namespace gdn {

constexpr int D = 128;
constexpr int NT = 256;
constexpr int NW = NT / 32;

// Thread layout of a 128 x COLS column slice: thread t owns columns 4 (t % CG) ..
// + 3 of rows rg, rg + RG, ... with rg = t / CG.
template <int COLS>
struct Slice {
    static constexpr int CG = COLS / 4;
    static constexpr int RG = NT / CG;
    static constexpr int RPT = D / RG;        // rows per thread
    static constexpr int GPW = 32 / CG;       // row groups in one warp (1 for COLS = 128)
};

// Column sums of k_i S_i and q_i S_i over all rows: in the warp by shuffles
// between its row groups, then across the warps through shared memory.
template <int COLS>
KDA_DEV void slice_products(const float4* st, const float* s_k, const float* s_q, int rg, int cg, int warp, int lane,
                            float (*part)[NW][COLS]) {
    using L = Slice<COLS>;
    float4 wk = make_float4(0.f, 0.f, 0.f, 0.f), wq = wk;
#pragma unroll
    for (int r = 0; r < L::RPT; ++r) {
        const float ki = s_k[rg + r * L::RG], qi = s_q[rg + r * L::RG];
        wk.x += ki * st[r].x; wk.y += ki * st[r].y; wk.z += ki * st[r].z; wk.w += ki * st[r].w;
        wq.x += qi * st[r].x; wq.y += qi * st[r].y; wq.z += qi * st[r].z; wq.w += qi * st[r].w;
    }
#pragma unroll
    for (int o = L::CG; o < 32; o <<= 1) {
        wk.x += __shfl_xor_sync(~0u, wk.x, o); wk.y += __shfl_xor_sync(~0u, wk.y, o);
        wk.z += __shfl_xor_sync(~0u, wk.z, o); wk.w += __shfl_xor_sync(~0u, wk.w, o);
        wq.x += __shfl_xor_sync(~0u, wq.x, o); wq.y += __shfl_xor_sync(~0u, wq.y, o);
        wq.z += __shfl_xor_sync(~0u, wq.z, o); wq.w += __shfl_xor_sync(~0u, wq.w, o);
    }
    if (lane < L::CG) {
        *reinterpret_cast<float4*>(&part[0][warp][4 * cg]) = wk;
        *reinterpret_cast<float4*>(&part[1][warp][4 * cg]) = wq;
    }
}

// ---------------------------------------------------------------------------
// decode: one CTA per (sequence, value head, column slice).  Bound by HBM: the
// state is read once (all of a thread's loads are issued before anything else)
// and written once, both as 128-bit streaming accesses.  256 sequences x 32 heads:
// 1.09 GB in 167 us, 6.5 TB/s, 0.95 of a copy's rate.
// ---------------------------------------------------------------------------
template <int COLS>
__global__ void __launch_bounds__(NT)
gdn_decode_kernel(kda_gdn_decode_args a) {
    using L = Slice<COLS>;
    constexpr int NS = D / COLS;
    const int slice = blockIdx.x % NS;
    const int h = (blockIdx.x / NS) % a.Hv;
    const int n = blockIdx.x / NS / a.Hv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cg = tid % L::CG, rg = tid / L::CG;
    const int slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots) return;   // out-of-range slot: skipped

    __shared__ float s_k[D], s_q[D], s_u[COLS], s_red[3][4];
    __shared__ __align__(16) float s_part[2][NW][COLS];

    float* S = a.state + ((size_t)slot * a.Hv + h) * (size_t)D * D + slice * COLS + 4 * cg;
    float4 st[L::RPT];
#pragma unroll
    for (int r = 0; r < L::RPT; ++r) st[r] = ld_stream_f4(S + (size_t)(rg + r * L::RG) * D);

    const size_t row = (size_t)n * a.Hv + h;
    const size_t krow = (size_t)n * a.Hk + h / (a.Hv / a.Hk);
    float qi = 0.f, ki = 0.f;
    if (tid < D) {
        qi = bf16_to_f(reinterpret_cast<const uint16_t*>(a.q)[krow * D + tid]);
        ki = bf16_to_f(reinterpret_cast<const uint16_t*>(a.k)[krow * D + tid]);
        const float qq = warp_sum(qi * qi), kk = warp_sum(ki * ki), kq = warp_sum(ki * qi);
        if (lane == 0) { s_red[0][warp] = qq; s_red[1][warp] = kk; s_red[2][warp] = kq; }
    }
    const float decay = __expf(log_decay_mode(a.z[row], __expf(a.A[h]), a.g_min, a.gate_mode));
    __syncthreads();
    float rq = 1.0f, rk = 1.0f;
    if (a.qk_l2norm) {
        rq = rsqrtf(s_red[0][0] + s_red[0][1] + s_red[0][2] + s_red[0][3] + 1e-6f);
        rk = rsqrtf(s_red[1][0] + s_red[1][1] + s_red[1][2] + s_red[1][3] + 1e-6f);
    }
    const float kq = (s_red[2][0] + s_red[2][1] + s_red[2][2] + s_red[2][3]) * rq * rk;
    if (tid < D) { s_k[tid] = ki * rk; s_q[tid] = qi * rq; }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < L::RPT; ++r) { st[r].x *= decay; st[r].y *= decay; st[r].z *= decay; st[r].w *= decay; }
    slice_products<COLS>(st, s_k, s_q, rg, cg, warp, lane, s_part);
    __syncthreads();
    if (tid < COLS) {
        float w = 0.f, qs = 0.f;
#pragma unroll
        for (int j = 0; j < NW; ++j) { w += s_part[0][j][tid]; qs += s_part[1][j][tid]; }
        const size_t e = row * D + slice * COLS + tid;
        const float u = a.beta[row] * (bf16_to_f(reinterpret_cast<const uint16_t*>(a.v)[e]) - w);
        s_u[tid] = u;
        reinterpret_cast<uint16_t*>(a.o)[e] = f_to_bf16(a.scale * (qs + kq * u));
    }
    __syncthreads();
    const float4 u4 = make_float4(s_u[4 * cg], s_u[4 * cg + 1], s_u[4 * cg + 2], s_u[4 * cg + 3]);
#pragma unroll
    for (int r = 0; r < L::RPT; ++r) {
        const float k1 = s_k[rg + r * L::RG];
        float4 s = st[r];
        s.x += k1 * u4.x; s.y += k1 * u4.y; s.z += k1 * u4.z; s.w += k1 * u4.w;
        st_stream_f4(S + (size_t)(rg + r * L::RG) * D, s);
    }
}

cudaError_t launch_decode(const kda_gdn_decode_args& a, cudaStream_t stream) {
    const long heads = (long)a.N * a.Hv;
    if (heads == 0) return cudaSuccess;
    // Few heads leave SMs idle and each state waits on one SM's loads: four column
    // slices of 32 channels then (a row of a slice is still one 128-byte line), while at
    // most two share an SM.  8 heads 2.6 us sliced, 3.5 whole; 64 heads 3.2, 3.6; 128
    // heads 4.3, 3.7; 512 heads 10.4, 9.8.
    if (heads * 4 <= 2 * 152)
        gdn_decode_kernel<32><<<(unsigned)(heads * 4), NT, 0, stream>>>(a);
    else
        gdn_decode_kernel<128><<<(unsigned)heads, NT, 0, stream>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// per-token recurrence: one CTA per (sequence, value head, slice of 32 columns),
// the slice in registers for the whole sequence.  Sequential in the tokens: bound by
// the latency of one step (two reductions, four barriers), 1 us with 32 heads.
// ---------------------------------------------------------------------------
template <bool BF16>
KDA_DEV float load1(const void* p, size_t i) {
    return BF16 ? bf16_to_f(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

template <bool BF16>
KDA_DEV void recurrence(const kda_gdn_prefill_args& a, const Sequences& which) {
    constexpr int COLS = 32, NS = D / COLS;
    using L = Slice<COLS>;
    const int slice = blockIdx.x % NS;
    const int h = (blockIdx.x / NS) % a.Hv;
    const int place = blockIdx.x / NS / a.Hv, n = which.count ? which.seq[place] : place;
    const int hk = h / (a.Hv / a.Hk);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cg = tid % L::CG, rg = tid / L::CG;
    const int t0 = a.cu_seqlens[n], t1 = a.cu_seqlens[n + 1];
    if (a.workspace && blockIdx.x == 0 && tid == 0) *reinterpret_cast<int*>(a.workspace) = 0;   // no error: nothing waits here

    __shared__ float s_k[D], s_q[D], s_u[COLS], s_red[3][4];
    __shared__ __align__(16) float s_part[2][NW][COLS];

    const size_t sbase = ((size_t)n * a.Hv + h) * (size_t)D * D + slice * COLS + 4 * cg;
    float4 st[L::RPT];
#pragma unroll
    for (int r = 0; r < L::RPT; ++r)
        st[r] = a.S0 ? *reinterpret_cast<const float4*>(a.S0 + sbase + (size_t)(rg + r * L::RG) * D)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    const float eA = __expf(a.A[h]);
    for (int t = t0; t < t1; ++t) {
        const size_t row = (size_t)t * a.Hv + h, krow = (size_t)t * a.Hk + hk;
        float qi = 0.f, ki = 0.f;
        if (tid < D) {
            qi = load1<BF16>(a.q, krow * D + tid);
            ki = load1<BF16>(a.k, krow * D + tid);
            const float qq = warp_sum(qi * qi), kk = warp_sum(ki * ki), kq = warp_sum(ki * qi);
            if (lane == 0) { s_red[0][warp] = qq; s_red[1][warp] = kk; s_red[2][warp] = kq; }
        }
        const float decay = __expf(log_decay_mode(a.z[row], eA, a.g_min, a.gate_mode));
        __syncthreads();
        float rq = 1.f, rk = 1.f;
        if (a.qk_l2norm) {
            rq = rsqrtf(s_red[0][0] + s_red[0][1] + s_red[0][2] + s_red[0][3] + 1e-6f);
            rk = rsqrtf(s_red[1][0] + s_red[1][1] + s_red[1][2] + s_red[1][3] + 1e-6f);
        }
        const float kq = (s_red[2][0] + s_red[2][1] + s_red[2][2] + s_red[2][3]) * rq * rk;
        if (tid < D) { s_k[tid] = ki * rk; s_q[tid] = qi * rq; }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < L::RPT; ++r) { st[r].x *= decay; st[r].y *= decay; st[r].z *= decay; st[r].w *= decay; }
        slice_products<COLS>(st, s_k, s_q, rg, cg, warp, lane, s_part);
        __syncthreads();
        if (tid < COLS) {
            float w = 0.f, qs = 0.f;
#pragma unroll
            for (int j = 0; j < NW; ++j) { w += s_part[0][j][tid]; qs += s_part[1][j][tid]; }
            const size_t e = row * D + slice * COLS + tid;
            const float u = a.beta[row] * (load1<BF16>(a.v, e) - w);
            s_u[tid] = u;
            if (a.o) {
                const float o = a.scale * (qs + kq * u);
                if (BF16) reinterpret_cast<uint16_t*>(a.o)[e] = f_to_bf16(o);
                else reinterpret_cast<float*>(a.o)[e] = o;
            }
        }
        __syncthreads();
        const float4 u4 = make_float4(s_u[4 * cg], s_u[4 * cg + 1], s_u[4 * cg + 2], s_u[4 * cg + 3]);
#pragma unroll
        for (int r = 0; r < L::RPT; ++r) {
            const float k1 = s_k[rg + r * L::RG];
            st[r].x += k1 * u4.x; st[r].y += k1 * u4.y; st[r].z += k1 * u4.z; st[r].w += k1 * u4.w;
        }
        __syncthreads();   // s_k, s_u and s_part are rewritten by the next token
    }
    if (a.S_T) {
#pragma unroll
        for (int r = 0; r < L::RPT; ++r)
            *reinterpret_cast<float4*>(a.S_T + sbase + (size_t)(rg + r * L::RG) * D) = st[r];
    }
}

template <bool BF16>
__global__ void __launch_bounds__(NT)
gdn_recurrent_kernel(const __grid_constant__ kda_gdn_prefill_args a, const __grid_constant__ Sequences which) {
    recurrence<BF16>(a, which);
    tc::wait_prerequisites();       // beside the scan of other sequences: this grid's end is not to come first
}

cudaError_t launch_recurrent(const kda_gdn_prefill_args& a, const Sequences& which, cudaStream_t s) {
    const long blocks = (long)(which.count ? which.count : a.num_seqs) * a.Hv * 4;
    if (blocks == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = which.count ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, a.qkv_dtype == KDA_BF16 ? gdn_recurrent_kernel<true> : gdn_recurrent_kernel<false>, a, which);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace gdn
}  // namespace kda
