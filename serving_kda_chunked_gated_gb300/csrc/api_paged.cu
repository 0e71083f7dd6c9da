// Host side of the paged key/value cache declared in include/kda.h: argument validation and
// dispatch.  Nothing is enqueued when validation fails.
#include <math.h>

#include "kda_common.cuh"

namespace kda {
namespace paged {
cudaError_t launch_write(const kda_paged_write_args& a, cudaStream_t s);
cudaError_t launch_read(const kda_paged_read_args& a, cudaStream_t s);
size_t prefill_workspace_size(const kda_paged_prefill_args& a);
cudaError_t launch_prefill(const kda_paged_prefill_args& a, cudaStream_t s);
size_t decode_workspace_size(const kda_paged_decode_args& a);
cudaError_t launch_decode(const kda_paged_decode_args& a, cudaStream_t s);
}  // namespace paged
}  // namespace kda

namespace {

constexpr long MAX_INT = 0x7fffffffL;

bool misaligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }

kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : kda::cuda_failure(e); }

// `work`: the call has something to do with the pages
kda_status check_cache(const kda_paged_cache& c, bool work) {
    if (c.num_pages < 0 || c.num_seqs < 0 || c.max_pages < 0 || c.Hkv <= 0 || (c.d != 64 && c.d != 128)) return KDA_ERR_SHAPE;
    if (c.page_size <= 0 || c.page_size % 16 != 0) return KDA_ERR_SHAPE;
    // rows and positions, a tile past them included, stay in 32 bits
    if ((long)c.num_pages * c.page_size > MAX_INT - 256 || (long)c.max_pages * c.page_size > 1L << 30) return KDA_ERR_SHAPE;
    if (c.Hkv > 1 << 20) return KDA_ERR_SHAPE;
    if (c.dtype != KDA_BF16 && c.dtype != KDA_E4M3) return KDA_ERR_DTYPE;
    if (work) {
        if (c.num_seqs == 0 || c.num_pages == 0) return KDA_ERR_SHAPE;
        if (!c.k || !c.v || !c.lens || (c.max_pages > 0 && !c.tables)) return KDA_ERR_NULL;
        if (c.dtype == KDA_E4M3 && (!c.k_scale || !c.v_scale)) return KDA_ERR_NULL;
    }
    if (misaligned(c.k) || misaligned(c.v) || misaligned(c.tables) || misaligned(c.lens)) return KDA_ERR_ALIGN;
    if (c.dtype == KDA_E4M3 && (misaligned(c.k_scale) || misaligned(c.v_scale))) return KDA_ERR_ALIGN;
    return KDA_OK;
}

// T tokens in rows of the cache's heads, with or without bounds
template <typename A>
kda_status check_tokens(const A& a) {
    if (a.T < 0 || a.T > MAX_INT - 256) return KDA_ERR_SHAPE;
    const kda_status st = check_cache(a.cache, a.T > 0);
    if (st != KDA_OK) return st;
    if (a.dtype != KDA_BF16 && a.dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (a.T > 0 && (!a.k || !a.v)) return KDA_ERR_NULL;
    if (misaligned(a.k) || misaligned(a.v) || misaligned(a.cu_seqlens)) return KDA_ERR_ALIGN;
    if (a.T > 0 && !a.cu_seqlens && a.cache.num_seqs != 1 && a.cache.num_seqs != a.T) return KDA_ERR_SEQLENS;
    return KDA_OK;
}

kda_status check_heads(int Hq, const kda_paged_cache& c, kda_dtype dtype, long q_stride, float scale) {
    if (Hq <= 0 || Hq % c.Hkv != 0 || Hq > 1 << 20) return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16) return KDA_ERR_DTYPE;
    if (q_stride < (long)Hq * c.d) return KDA_ERR_SHAPE;
    if (q_stride % 8 != 0) return KDA_ERR_ALIGN;
    if (!isfinite(scale)) return KDA_ERR_SHAPE;
    return KDA_OK;
}

kda_status check(const kda_paged_prefill_args* a) {
    if (!a) return KDA_ERR_NULL;
    if (a->T_total < 0 || a->T_total > 1L << 30) return KDA_ERR_SHAPE;
    kda_status st = check_cache(a->cache, a->T_total > 0);
    if (st == KDA_OK) st = check_heads(a->Hq, a->cache, a->dtype, a->q_stride, a->scale);
    if (st != KDA_OK) return st;
    if (!a->cu_seqlens || !a->cu_seqlens_host) return KDA_ERR_NULL;
    if (a->T_total > 0 && (!a->q || !a->o)) return KDA_ERR_NULL;
    if (misaligned(a->cu_seqlens) || misaligned(a->q) || misaligned(a->o) || misaligned(a->lse) ||
        misaligned(a->error))
        return KDA_ERR_ALIGN;
    const int32_t* cu = a->cu_seqlens_host;
    if (cu[0] != 0 || cu[a->cache.num_seqs] != a->T_total) return KDA_ERR_SEQLENS;
    for (int n = 0; n < a->cache.num_seqs; ++n)
        if (cu[n + 1] < cu[n]) return KDA_ERR_SEQLENS;
    if ((long)a->T_total > MAX_INT / a->Hq) return KDA_ERR_SHAPE;
    return KDA_OK;
}

kda_status check(const kda_paged_decode_args* a) {
    if (!a) return KDA_ERR_NULL;
    const bool work = a->cache.num_seqs > 0;
    kda_status st = check_cache(a->cache, work);
    if (st == KDA_OK) st = check_heads(a->Hq, a->cache, a->dtype, a->q_stride, a->scale);
    if (st != KDA_OK) return st;
    if (work && (!a->q || !a->o)) return KDA_ERR_NULL;
    if (!a->k != !a->v) return KDA_ERR_NULL;
    if (a->k) {
        const long row = (long)a->cache.Hkv * a->cache.d;
        if (a->k_stride < row || a->v_stride < row) return KDA_ERR_SHAPE;
        if (a->k_stride % 8 != 0 || a->v_stride % 8 != 0) return KDA_ERR_ALIGN;
    }
    if (misaligned(a->q) || misaligned(a->k) || misaligned(a->v) || misaligned(a->o) || misaligned(a->lse)) return KDA_ERR_ALIGN;
    if ((long)a->cache.num_seqs > MAX_INT / a->Hq) return KDA_ERR_SHAPE;
    return KDA_OK;
}

template <typename A>
kda_status check_workspace(const A& a, size_t need) {
    if (!a.workspace || a.workspace_bytes < need) return KDA_ERR_WORKSPACE;
    return misaligned(a.workspace) ? KDA_ERR_ALIGN : KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_paged_write(const kda_paged_write_args* a, void* stream) {
    if (!a) return KDA_ERR_NULL;
    const kda_status st = check_tokens(*a);
    if (st != KDA_OK) return st;
    const long row = (long)a->cache.Hkv * a->cache.d, piece = a->dtype == KDA_BF16 ? 8 : 4;     // elements in 16 bytes
    if (a->k_stride < row || a->v_stride < row) return KDA_ERR_SHAPE;
    if (a->k_stride % piece != 0 || a->v_stride % piece != 0) return KDA_ERR_ALIGN;
    if (a->T == 0) return KDA_OK;
    return done(kda::paged::launch_write(*a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_paged_read(const kda_paged_read_args* a, void* stream) {
    if (!a) return KDA_ERR_NULL;
    const kda_status st = check_tokens(*a);
    if (st != KDA_OK) return st;
    if (a->T == 0) return KDA_OK;
    return done(kda::paged::launch_read(*a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_paged_prefill_workspace_size(const kda_paged_prefill_args* a) {
    return check(a) == KDA_OK ? kda::paged::prefill_workspace_size(*a) : 0;
}

kda_status kda_paged_prefill(const kda_paged_prefill_args* a, void* stream) {
    kda_status st = check(a);
    if (st == KDA_OK) st = check_workspace(*a, kda::paged::prefill_workspace_size(*a));
    if (st != KDA_OK) return st;
    if (a->T_total == 0) return KDA_OK;
    return done(kda::paged::launch_prefill(*a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_paged_decode_workspace_size(const kda_paged_decode_args* a) {
    return check(a) == KDA_OK ? kda::paged::decode_workspace_size(*a) : 0;
}

kda_status kda_paged_decode(const kda_paged_decode_args* a, void* stream) {
    kda_status st = check(a);
    if (st == KDA_OK) st = check_workspace(*a, kda::paged::decode_workspace_size(*a));
    if (st != KDA_OK) return st;
    if (a->cache.num_seqs == 0) return KDA_OK;
    return done(kda::paged::launch_decode(*a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
