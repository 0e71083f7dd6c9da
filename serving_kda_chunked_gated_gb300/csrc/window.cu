// Sliding-window attention with sinks: the decode step over a ring cache, the
// cache fill after a prefill.
//
// Decode is bound by HBM: per (sequence, key head) it reads the visible rows of
// K and V once.  The query heads of one key head are the 16 rows of an
// m16n8k16 product (padded), so that the arithmetic hides behind the loads
// whatever the group size.  Every warp walks its own 16-key tiles with a running
// maximum and sum (no barrier in the loop); a ring of asynchronous copies per warp
// keeps STAGES tiles in flight.  Warps are merged through shared memory, CTAs that
// share a (sequence, key head) through distributed shared memory of their cluster:
// no workspace and no second launch.  256 sequences x 8 key heads of 128, window
// 4096: 4.1 GB in 577 us, 7.1 TB/s (reads alone run above a copy's rate).
#include "kda_common.cuh"
#include "tcgen05.cuh"

#include <math.h>

#include <atomic>

namespace kda {
namespace win {

KDA_DEV uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
KDA_DEV void cp16(uint32_t dst, const void* src, bool valid) {   // !valid: 16 zero bytes, src not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
KDA_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
KDA_DEV void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
KDA_DEV void ldsm4(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
KDA_DEV void ldsm4t(uint32_t* r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// C += A B, m16n8k16, bf16 inputs, fp32 accumulate
KDA_DEV void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
KDA_DEV uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// x = hi + lo, both bf16: pairs packed with the lower index in the low half
KDA_DEV void split2(float x0, float x1, uint32_t* hi, uint32_t* lo) {
    *hi = pack2(x0, x1);
    *lo = pack2(x0 - __uint_as_float(*hi << 16), x1 - __uint_as_float(*hi & 0xffff0000u));
}
KDA_DEV uint32_t cluster_rank() { uint32_t r; asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r)); return r; }
KDA_DEV uint32_t cluster_size() { uint32_t r; asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r)); return r; }
KDA_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
KDA_DEV float ld_peer(const float* p, uint32_t rank) {   // the float at this address in another CTA of the cluster
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(su32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

constexpr int DEC_STAGES = 3;
constexpr int DEC_KEYS = 16;     // keys per tile

template <int D, int WARPS>
constexpr int dec_smem() { return WARPS * DEC_STAGES * DEC_KEYS * D * 2 * 2; }

// 8 / WARPS CTAs share an SM
template <int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 8 / WARPS)
window_decode_kernel(kda_window_decode_args a, int mtiles) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_m[WARPS][16], s_l[WARPS][16], s_M[16], s_L[16];
    constexpr int TILE = DEC_KEYS * D * 2;          // bytes of one K (or V) tile
    constexpr int CH = D / 8;                       // 16-byte chunks per row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t nsplit = cluster_size(), split = cluster_rank();
    const long unit = blockIdx.x / nsplit;          // (sequence, key head, 16-row tile of its query heads)
    const int mt = (int)(unit % mtiles);
    const int hk = (int)(unit / mtiles % a.Hkv);
    const int n = (int)(unit / mtiles / a.Hkv);
    const int G = a.Hq / a.Hkv;
    const int pos = a.positions[n];
    const int slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots || pos < 0) return;     // the whole cluster: same n

    const int R = a.cache_rows - a.sinks;
    // visible rows: the first `ns` sinks, then the ring from position `first` on
    const int first = max(a.sinks, pos - a.window + 1);
    const int ns = pos < a.sinks ? pos + 1 : a.sinks;
    const int total = ns + max(0, pos - first + 1);
    const int ring0 = pos >= a.sinks ? (first - a.sinks) % R : 0;
    const size_t rstride = (size_t)a.Hkv * D;
    const uint16_t* Kc = reinterpret_cast<const uint16_t*>(a.k_cache) + (size_t)slot * a.cache_rows * rstride + (size_t)hk * D;
    const uint16_t* Vc = reinterpret_cast<const uint16_t*>(a.v_cache) + (size_t)slot * a.cache_rows * rstride + (size_t)hk * D;
    const uint16_t* kn = reinterpret_cast<const uint16_t*>(a.k) + (size_t)n * a.k_stride + (size_t)hk * D;
    const uint16_t* vn = reinterpret_cast<const uint16_t*>(a.v) + (size_t)n * a.v_stride + (size_t)hk * D;

    uint8_t* mine = smem + warp * (DEC_STAGES * 2 * TILE);
    const uint32_t mine_u = su32(mine);
    const int ntiles = (total + DEC_KEYS - 1) / DEC_KEYS;
    const int t0 = split * WARPS + warp, tstep = nsplit * WARPS;

    // The new token is the last visible row; it is read from the inputs, so no CTA
    // depends on the cache row that is being written.
    auto fetch = [&](int tile, int stage) {
        const uint32_t kb = mine_u + stage * 2 * TILE, vb = kb + TILE;
#pragma unroll
        for (int i = 0; i < DEC_KEYS * CH / 32; ++i) {
            const int e = i * 32 + lane, r = e / CH, c = e % CH;
            const int u = tile * DEC_KEYS + r;
            const bool on = u < total;
            int row = u;
            if (u >= ns) { row = ring0 + (u - ns); row = a.sinks + (row >= R ? row - R : row); }
            const bool fresh = u == total - 1;
            const uint16_t* ks = fresh ? kn + c * 8 : Kc + (size_t)row * rstride + c * 8;
            const uint16_t* vs = fresh ? vn + c * 8 : Vc + (size_t)row * rstride + c * 8;
            const uint32_t off = r * (D * 2) + ((c ^ (r & 7)) << 4);
            cp16(kb + off, on ? ks : kn, on);
            cp16(vb + off, on ? vs : vn, on);
        }
    };
#pragma unroll
    for (int s = 0; s < DEC_STAGES - 1; ++s) {
        if (t0 + s * tstep < ntiles) fetch(t0 + s * tstep, s);
        cp_commit();
    }
    // query rows: row g of the tile is query head hk G + 16 mt + g, rows >= G are zero
    const int g = lane >> 2, t4 = lane & 3;
    uint32_t qf[D / 16][4];
    {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q) + (size_t)n * a.q_stride + (size_t)hk * G * D;
        const int r0 = mt * 16 + g, r1 = r0 + 8;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            const int c = k * 16 + t4 * 2;
            qf[k][0] = r0 < G ? *reinterpret_cast<const uint32_t*>(q + (size_t)r0 * D + c) : 0u;
            qf[k][1] = r1 < G ? *reinterpret_cast<const uint32_t*>(q + (size_t)r1 * D + c) : 0u;
            qf[k][2] = r0 < G ? *reinterpret_cast<const uint32_t*>(q + (size_t)r0 * D + c + 8) : 0u;
            qf[k][3] = r1 < G ? *reinterpret_cast<const uint32_t*>(q + (size_t)r1 * D + c + 8) : 0u;
        }
    }
    if (split == 0 && mt == 0 && tid < 2 * CH) {      // the token's row of the caches
        const int row = pos < a.sinks ? pos : a.sinks + (pos - a.sinks) % R;
        const size_t at = ((size_t)slot * a.cache_rows + row) * rstride + (size_t)hk * D;
        const int c = (tid % CH) * 8;
        uint16_t* dst = reinterpret_cast<uint16_t*>(tid < CH ? a.k_cache : a.v_cache) + at + c;
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>((tid < CH ? kn : vn) + c);
    }
    const float sc = a.scale * 1.4426950408889634f;    // scores in powers of two
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    int stage = 0;
    for (int tile = t0; tile < ntiles; tile += tstep) {
        cp_wait<DEC_STAGES - 2>();
        __syncwarp();
        {
            const int nt = tile + (DEC_STAGES - 1) * tstep;
            int ps = stage + DEC_STAGES - 1;
            if (ps >= DEC_STAGES) ps -= DEC_STAGES;
            if (nt < ntiles) fetch(nt, ps);
            cp_commit();
        }
        const uint32_t kb = mine_u + stage * 2 * TILE, vb = kb + TILE;
        float s[2][4] = {};
        const int mrow = (lane & 7) + ((lane >> 4) << 3), mch = (lane >> 3) & 1;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldsm4(b, kb + mrow * (D * 2) + (((2 * k + mch) ^ (mrow & 7)) << 4));
            mma16816(s[0], qf[k], b[0], b[1]);
            mma16816(s[1], qf[k], b[2], b[3]);
        }
        const int left = total - tile * DEC_KEYS;
        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool on = j * 8 + t4 * 2 + (i & 1) < left;
                s[j][i] = on ? s[j][i] * sc : -INFINITY;
            }
            x0 = fmaxf(x0, fmaxf(s[j][0], s[j][1]));
            x1 = fmaxf(x1, fmaxf(s[j][2], s[j][3]));
        }
        x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, 1)); x0 = fmaxf(x0, __shfl_xor_sync(~0u, x0, 2));
        x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, 1)); x1 = fmaxf(x1, __shfl_xor_sync(~0u, x1, 2));
        const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
        // a row whose scores are all -inf so far: subtract 0, its exponentials are 0
        const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;
        if (__any_sync(~0u, n0 != m0 || n1 != m1)) {
            const float c0 = exp2f(m0 - b0), c1 = exp2f(m1 - b1);
            l0 *= c0; l1 *= c1;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) { o[i][0] *= c0; o[i][1] *= c0; o[i][2] *= c1; o[i][3] *= c1; }
            m0 = n0; m1 = n1;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            s[j][0] = exp2f(s[j][0] - b0); s[j][1] = exp2f(s[j][1] - b0);
            s[j][2] = exp2f(s[j][2] - b1); s[j][3] = exp2f(s[j][3] - b1);
            l0 += s[j][0] + s[j][1];
            l1 += s[j][2] + s[j][3];
        }
        // Weights in [0, 1] as two bf16 parts (2^-17 left): o is then off by its own rounding alone, 1.7e-3,
        // rather than 2.1e-3 with one part.  256 sequences, window 4096, us with one part and two: 32/8 heads
        // of 128 586, 589; of 64 307, 316; window 512, 16/8 of 128: 88, 90; 64 sequences, 32 query heads to
        // a key head (arithmetic counts there): 60, 68.
        uint32_t p[4], pl[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            split2(s[j][0], s[j][1], &p[2 * j], &pl[2 * j]);
            split2(s[j][2], s[j][3], &p[2 * j + 1], &pl[2 * j + 1]);
        }
        const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vch = lane >> 4;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t b[4];
            ldsm4t(b, vb + vrow * (D * 2) + (((2 * k + vch) ^ (vrow & 7)) << 4));
            mma16816(o[2 * k], p, b[0], b[1]);
            mma16816(o[2 * k + 1], p, b[2], b[3]);
            mma16816(o[2 * k], pl, b[0], b[1]);
            mma16816(o[2 * k + 1], pl, b[2], b[3]);
        }
        if (++stage == DEC_STAGES) stage = 0;
        __syncwarp();          // the tile is read before its stage is filled again
    }
    cp_wait<0>();
    l0 += __shfl_xor_sync(~0u, l0, 1); l0 += __shfl_xor_sync(~0u, l0, 2);
    l1 += __shfl_xor_sync(~0u, l1, 1); l1 += __shfl_xor_sync(~0u, l1, 2);
    // warps -> CTA: each warp's rows in its own tile ring (16 x D floats <= the ring)
    static_assert(16 * D * 4 <= DEC_STAGES * 2 * TILE, "a warp's partial rows fit its ring");
    __syncwarp();
    float* po = reinterpret_cast<float*>(mine);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        *reinterpret_cast<float2*>(po + g * D + i * 8 + t4 * 2) = make_float2(o[i][0], o[i][1]);
        *reinterpret_cast<float2*>(po + (g + 8) * D + i * 8 + t4 * 2) = make_float2(o[i][2], o[i][3]);
    }
    if (t4 == 0) { s_m[warp][g] = m0; s_m[warp][g + 8] = m1; s_l[warp][g] = l0; s_l[warp][g + 8] = l1; }
    __syncthreads();
    if (tid < 16) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_m[w][tid]);
        const float b = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = exp2f(s_m[w][tid] - b);
            L += f * s_l[w][tid];
            s_m[w][tid] = f;                              // from here on: the warp's weight
        }
        s_M[tid] = M;
        s_L[tid] = L;
    }
    __syncthreads();
    const int rows = min(16, G - mt * 16);
    float* acc = reinterpret_cast<float*>(smem);          // the CTA's rows replace warp 0's (same thread, same place)
    for (int e = tid; e < rows * D; e += WARPS * 32) {
        const int r = e / D;
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
            x += s_m[w][r] * reinterpret_cast<const float*>(smem + w * (DEC_STAGES * 2 * TILE))[e];
        acc[e] = x;
    }
    uint16_t* out = reinterpret_cast<uint16_t*>(a.o) + ((size_t)n * a.Hq + (size_t)hk * G + mt * 16) * D;
    if (nsplit == 1) {
        for (int e = tid; e < rows * D; e += WARPS * 32) out[e] = f_to_bf16(acc[e] / s_L[e / D]);
        return;
    }
    cluster_sync();
    for (int e = split * (WARPS * 32) + tid; e < rows * D; e += nsplit * WARPS * 32) {
        const int r = e / D;
        float M = -INFINITY, x = 0.f, L = 0.f;
        for (uint32_t c = 0; c < nsplit; ++c) M = fmaxf(M, ld_peer(&s_M[r], c));
        const float b = M == -INFINITY ? 0.f : M;
        for (uint32_t c = 0; c < nsplit; ++c) {
            const float f = exp2f(ld_peer(&s_M[r], c) - b);
            L += f * ld_peer(&s_L[r], c);
            x += f * ld_peer(&acc[e], c);
        }
        out[e] = f_to_bf16(x / L);
    }
    cluster_sync();                                       // no CTA leaves while its shared memory is read
}

// CTAs of a cluster at most (the portable size) and devices whose counts are kept
constexpr int DEC_SPLIT = 8, DEC_DEVICES = 64;

template <int D, int WARPS>
static void decode_shape(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, long units, int split, cudaStream_t s) {
    *cfg = {};
    cfg->gridDim = dim3((unsigned)(units * split));
    cfg->blockDim = dim3(WARPS * 32);
    cfg->dynamicSmemBytes = dec_smem<D, WARPS>();
    cfg->stream = s;
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = split;
    attr->val.clusterDim.y = attr->val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
}

// How many clusters of `split` CTAs the current device holds at once: a property of the
// device (clusters stay inside a group of SMs, and groups differ in size), asked once.
template <int D>
static cudaError_t resident_clusters(int split, int* count) {
    static std::atomic<int> held[DEC_DEVICES][DEC_SPLIT + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool keep = dev < DEC_DEVICES;
    if (keep && (*count = held[dev][split].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    decode_shape<D, 8>(&cfg, &attr, 1, split, nullptr);
    e = cudaOccupancyMaxActiveClusters(count, window_decode_kernel<D, 8>, &cfg);
    if (e == cudaSuccess && keep) held[dev][split].store(*count, std::memory_order_relaxed);
    return e;
}

template <int D, int WARPS>
static cudaError_t decode_go(const kda_window_decode_args& a, int mtiles, long units, cudaStream_t s) {
    cudaError_t e =
        cudaFuncSetAttribute(window_decode_kernel<D, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, dec_smem<D, WARPS>());
    if (e != cudaSuccess) return e;
    int split = 1;
    if constexpr (WARPS == 8) {
        // CTAs per unit: as many as leave all clusters resident at once, at most one per 16-key tile of
        // each warp.  Window of 4096, d = 128, us: 14 units 30.2 alone, 12.3 by fours, 9.6 by eights;
        // 36 units 30.6, 12.9, but 27.0 by eights, whose clusters then come in turns; 100 units
        // 35.6, 45.4 by twos.
        const long most = ((long)a.sinks + a.window + DEC_KEYS * WARPS - 1) / (DEC_KEYS * WARPS);
        for (int c = DEC_SPLIT; c > 1 && split == 1; --c) {
            if (c > most || units * c > 152) continue;
            int fit = 0;
            if ((e = resident_clusters<D>(c, &fit)) != cudaSuccess) return e;
            if (units <= fit) split = c;
        }
    }
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    decode_shape<D, WARPS>(&cfg, &attr, units, split, s);
    e = cudaLaunchKernelEx(&cfg, window_decode_kernel<D, WARPS>, a, mtiles);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return cudaSuccess;
}

template <int D>
static cudaError_t decode_d(const kda_window_decode_args& a, cudaStream_t s) {
    const int mtiles = (a.Hq / a.Hkv + 15) / 16;
    const long units = (long)a.N * a.Hkv * mtiles;          // (sequence, key head, 16 of its query heads)
    // Eight warps an SM in all, in smaller CTAs where there are units enough to fill it with them: a
    // CTA's start and end then pass beside others' loads.  d = 128, us with 8, 4, 2 warps: 152 units,
    // window 4096: 50, 52, 76; 300 units, 2000: 51, 49, 52; 1160 units, 101 + 64 sinks: 31, 19, 14;
    // 2048 units, 512: 109, 92, 91; 1024: 170, 160, 163; 4096: 587, 586, 607 (more pages of
    // memory open at a time).
    const long rows = (long)a.sinks + a.window;
    if (units > 2 * 152 && rows <= 512) return decode_go<D, 2>(a, mtiles, units, s);
    // also where eight warps would not have a tile each (82 units, 6 + 64 rows, d = 64: 3.6, 3.3, 3.2)
    if (units > 152 || rows < 8 * DEC_KEYS) return decode_go<D, 4>(a, mtiles, units, s);
    return decode_go<D, 8>(a, mtiles, units, s);
}

cudaError_t launch_decode(const kda_window_decode_args& a, cudaStream_t s) {
    if (a.N == 0) return cudaSuccess;
    return a.d == 64 ? decode_d<64>(a, s) : decode_d<128>(a, s);
}

// ---------------------------------------------------------------------------
// cache fill after a prefill: the sinks and the last `window` positions of each
// sequence, one 16-byte piece of K and of V per thread
// ---------------------------------------------------------------------------
KDA_DEV void fill_piece(const kda_window_prefill_args& a, long per_seq) {
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    const long n = i / per_seq;
    if (n >= a.num_seqs) return;
    const int slot = a.slots ? a.slots[n] : (int)n;
    if (slot < 0 || slot >= a.num_slots) return;
    const int pieces = a.Hkv * a.d / 8;
    const int u = (int)((i - n * per_seq) / pieces), c = (int)((i - n * per_seq) % pieces) * 8;
    const int k0 = a.cu_seqlens_k[n], len = a.cu_seqlens_k[n + 1] - k0;
    const int ns = min(a.sinks, len), first = max(a.sinks, len - a.window);
    int p;
    if (u < a.sinks) { if (u >= ns) return; p = u; }
    else { p = first + (u - a.sinks); if (p >= len) return; }
    const int R = a.cache_rows - a.sinks;
    const int row = p < a.sinks ? p : a.sinks + (p - a.sinks) % R;
    const size_t dst = ((size_t)slot * a.cache_rows + row) * (size_t)(a.Hkv * a.d) + c;
    const size_t t = (size_t)(k0 + p);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.k_cache) + dst) =
        *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.k) + t * a.k_stride + c);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.v_cache) + dst) =
        *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.v) + t * a.v_stride + c);
}

__global__ void __launch_bounds__(256)
window_fill_kernel(const __grid_constant__ kda_window_prefill_args a, long per_seq) {
    fill_piece(a, per_seq);
    // Nothing here depends on the prefill's outputs: only the end of this grid is not to come first.
    tc::wait_prerequisites();
}

cudaError_t launch_fill(const kda_window_prefill_args& a, bool beside_prefill, cudaStream_t s) {
    int longest = 0;
    for (int n = 0; n < a.num_seqs; ++n) {
        const int len = a.cu_seqlens_k_host[n + 1] - a.cu_seqlens_k_host[n];
        longest = len > longest ? len : longest;
    }
    const long ring = longest < a.window ? longest : a.window;   // ring rows any sequence writes
    const long per_seq = ((long)a.sinks + ring) * (a.Hkv * a.d / 8);
    const long blocks = (per_seq * a.num_seqs + 255) / 256;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    // beside the prefill: six ragged sequences, window 1000: 55 -> 49 us back to back
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = beside_prefill ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, window_fill_kernel, a, per_seq);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

}  // namespace win
}  // namespace kda
