// Host side of the hybrid stack's token mixers declared in include/kda.h (scalar
// gated delta rule, per-head norm with rotation, window attention): argument
// validation and dispatch.  Nothing is enqueued when validation fails.
#include <math.h>

#include "gdn.cuh"
#include "kda_common.cuh"

namespace kda {
namespace gdn {
cudaError_t launch_decode(const kda_gdn_decode_args& a, cudaStream_t s);
size_t chunked_workspace_size(const kda_gdn_prefill_args& a);
cudaError_t launch_chunked(const kda_gdn_prefill_args& a, cudaStream_t s);
}  // namespace gdn
namespace qknr {
cudaError_t launch(const kda_qk_norm_rope_args& a, cudaStream_t s);
}
namespace win {
cudaError_t launch_prefill(const kda_window_prefill_args& a, cudaStream_t s);
cudaError_t launch_fill(const kda_window_prefill_args& a, bool beside_prefill, cudaStream_t s);
cudaError_t launch_decode(const kda_window_decode_args& a, cudaStream_t s);
}  // namespace win
}  // namespace kda

namespace {

constexpr long MAX_BLOCKS = 0x7fffffffL;     // of a one-dimensional grid

bool misaligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }

template <int N>
bool any_misaligned(const void* const (&ptrs)[N]) {
    for (const void* p : ptrs)
        if (misaligned(p)) return true;
    return false;
}

// first 0, non-decreasing, last `total`
bool seqlens_ok(const int32_t* cu, int num_seqs, int total) {
    if (cu[0] != 0 || cu[num_seqs] != total) return false;
    for (int n = 0; n < num_seqs; ++n)
        if (cu[n + 1] < cu[n]) return false;
    return true;
}

bool gate_ok(int mode) { return mode == KDA_GATE_BOUNDED || mode == KDA_GATE_SOFTPLUS; }

kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : kda::cuda_failure(e); }

kda_status check(const kda_gdn_prefill_args* a) {
    if (!a) return KDA_ERR_NULL;
    if (a->num_seqs < 0 || a->T_total < 0 || a->Hk <= 0 || a->Hv <= 0 || a->Hv % a->Hk != 0) return KDA_ERR_SHAPE;
    if (a->dk != 128 || a->dv != 128) return KDA_ERR_SHAPE;
    if (a->qkv_dtype != KDA_BF16 && a->qkv_dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (!a->cu_seqlens || !a->cu_seqlens_host || !a->A) return KDA_ERR_NULL;
    if (a->T_total > 0 && (!a->q || !a->k || !a->v || !a->z || !a->beta)) return KDA_ERR_NULL;
    if (a->T_total > 0 && !a->o && !a->S_T) return KDA_ERR_NULL;
    if (any_misaligned({a->cu_seqlens, a->q, a->k, a->v, (const void*)a->z, (const void*)a->beta, (const void*)a->A,
                        (const void*)a->S0, a->o, (const void*)a->S_T}))
        return KDA_ERR_ALIGN;
    if (!seqlens_ok(a->cu_seqlens_host, a->num_seqs, a->T_total)) return KDA_ERR_SEQLENS;
    if (!gate_ok(a->gate_mode)) return KDA_ERR_UNSUPPORTED;
    // one CTA per (sequence, head, slice), per (chunk, head) at most
    if ((long)a->num_seqs * a->Hv > MAX_BLOCKS / 8 || ((long)a->T_total / 128 + a->num_seqs) * a->Hv > MAX_BLOCKS)
        return KDA_ERR_SHAPE;
    return KDA_OK;
}

}  // namespace

extern "C" {

size_t kda_gdn_prefill_workspace_size(const kda_gdn_prefill_args* a) {
    if (check(a) != KDA_OK || a->qkv_dtype != KDA_BF16) return 0;
    return kda::gdn::chunked_workspace_size(*a);
}

kda_status kda_gdn_prefill(const kda_gdn_prefill_args* a, void* stream) {
    const kda_status st = check(a);
    if (st != KDA_OK) return st;
    if (a->num_seqs == 0 || (!a->o && !a->S_T)) return KDA_OK;      // no tokens and no state asked for
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (a->qkv_dtype == KDA_F32) return kda_gdn_prefill_recurrent(a, stream);
    if (!a->workspace || a->workspace_bytes < kda::gdn::chunked_workspace_size(*a)) return KDA_ERR_WORKSPACE;
    if (misaligned(a->workspace)) return KDA_ERR_ALIGN;
    return done(kda::gdn::launch_chunked(*a, s));
}

kda_status kda_gdn_prefill_recurrent(const kda_gdn_prefill_args* a, void* stream) {
    const kda_status st = check(a);
    if (st != KDA_OK) return st;
    kda_gdn_prefill_args r = *a;
    r.workspace = nullptr;                // has none, whatever the field holds
    kda::gdn::Sequences all;
    all.count = 0;
    return done(kda::gdn::launch_recurrent(r, all, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_gdn_decode_step(const kda_gdn_decode_args* a, void* stream) {
    if (!a) return KDA_ERR_NULL;
    if (a->N < 0 || a->Hk <= 0 || a->Hv <= 0 || a->Hv % a->Hk != 0 || a->num_slots < 0) return KDA_ERR_SHAPE;
    if (a->dk != 128 || a->dv != 128) return KDA_ERR_SHAPE;
    if (!a->slots && a->num_slots < a->N) return KDA_ERR_SHAPE;
    if ((long)a->N * a->Hv > MAX_BLOCKS) return KDA_ERR_SHAPE;
    if (a->N > 0 && (!a->q || !a->k || !a->v || !a->z || !a->beta || !a->A || !a->state || !a->o)) return KDA_ERR_NULL;
    if (any_misaligned({a->q, a->k, a->v, (const void*)a->z, (const void*)a->beta, (const void*)a->A,
                        (const void*)a->state, (const void*)a->slots, (const void*)a->o}))
        return KDA_ERR_ALIGN;
    if (!gate_ok(a->gate_mode)) return KDA_ERR_UNSUPPORTED;
    return done(kda::gdn::launch_decode(*a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_qk_norm_rope(const kda_qk_norm_rope_args* a, void* stream) {
    if (!a) return KDA_ERR_NULL;
    if (a->T < 0 || a->Hq < 0 || a->Hkv < 0 || (a->Hq == 0 && a->Hkv == 0) || a->num_pos < 0) return KDA_ERR_SHAPE;
    if (a->d < 16 || a->d > 256 || a->d % 8 != 0) return KDA_ERR_SHAPE;
    if (a->rot < 16 || a->rot > a->d || a->rot % 16 != 0) return KDA_ERR_SHAPE;
    if (a->dtype != KDA_BF16 && a->dtype != KDA_F32) return KDA_ERR_DTYPE;
    if (a->T > 0) {
        if (!a->cos || !a->sin || !a->positions) return KDA_ERR_NULL;
        if (a->Hq > 0 && (!a->q || !a->q_out)) return KDA_ERR_NULL;
        if (a->Hkv > 0 && (!a->k || !a->k_out)) return KDA_ERR_NULL;
    }
    const long piece = a->dtype == KDA_BF16 ? 8 : 4;        // elements in 16 bytes
    if (a->q_stride < (long)a->Hq * a->d || a->k_stride < (long)a->Hkv * a->d) return KDA_ERR_SHAPE;
    if (a->q_stride % piece != 0 || a->k_stride % piece != 0) return KDA_ERR_ALIGN;
    if ((a->q_out && a->q_out == a->q && a->q_stride != (long)a->Hq * a->d) ||
        (a->k_out && a->k_out == a->k && a->k_stride != (long)a->Hkv * a->d))
        return KDA_ERR_SHAPE;                                // in place needs the dense layout
    if (any_misaligned({a->q, a->k, (const void*)a->q_weight, (const void*)a->k_weight, (const void*)a->cos,
                        (const void*)a->sin, (const void*)a->positions, (const void*)a->q_out, (const void*)a->k_out}))
        return KDA_ERR_ALIGN;
    // the kernel counts heads, and (token, four or more heads), in 32 bits
    if ((long)a->Hq + a->Hkv > 1L << 20 || (long)a->T * ((a->Hq + 3) / 4 + (a->Hkv + 3) / 4) > MAX_BLOCKS) return KDA_ERR_SHAPE;
    return done(kda::qknr::launch(*a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

// what both window calls share: heads, window, strides, scale
kda_status check_window(int Hq, int Hkv, int d, int window, int sinks, kda_dtype dtype, long qs, long ks, long vs,
                        float scale) {
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || (d != 64 && d != 128)) return KDA_ERR_SHAPE;
    if (window < 1 || sinks < 0 || (long)window + sinks > 0x7fffffffL) return KDA_ERR_SHAPE;
    if (dtype != KDA_BF16) return KDA_ERR_DTYPE;
    if (qs < (long)Hq * d || ks < (long)Hkv * d || vs < (long)Hkv * d) return KDA_ERR_SHAPE;
    if (qs % 8 != 0 || ks % 8 != 0 || vs % 8 != 0) return KDA_ERR_ALIGN;
    if (!isfinite(scale)) return KDA_ERR_SHAPE;
    return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_window_prefill(const kda_window_prefill_args* a, void* stream) {
    if (!a) return KDA_ERR_NULL;
    if (a->num_seqs < 0 || a->T_total < 0 || a->Tk_total < 0) return KDA_ERR_SHAPE;
    const kda_status st = check_window(a->Hq, a->Hkv, a->d, a->window, a->sinks, a->dtype, a->q_stride, a->k_stride,
                                       a->v_stride, a->scale);
    if (st != KDA_OK) return st;
    if (!a->cu_seqlens || !a->cu_seqlens_host || !a->cu_seqlens_k || !a->cu_seqlens_k_host) return KDA_ERR_NULL;
    if (a->T_total > 0 && (!a->q || !a->o)) return KDA_ERR_NULL;
    if (a->Tk_total > 0 && (!a->k || !a->v)) return KDA_ERR_NULL;
    if (!a->k_cache != !a->v_cache) return KDA_ERR_NULL;
    if (any_misaligned({a->cu_seqlens, a->cu_seqlens_k, a->q, a->k, a->v, (const void*)a->o, (const void*)a->lse,
                        (const void*)a->k_cache, (const void*)a->v_cache, (const void*)a->slots, (const void*)a->error}))
        return KDA_ERR_ALIGN;
    const int32_t *cq = a->cu_seqlens_host, *ck = a->cu_seqlens_k_host;
    if (!seqlens_ok(cq, a->num_seqs, a->T_total) || !seqlens_ok(ck, a->num_seqs, a->Tk_total)) return KDA_ERR_SEQLENS;
    for (int n = 0; n < a->num_seqs; ++n)
        if (ck[n + 1] - ck[n] < cq[n + 1] - cq[n]) return KDA_ERR_SEQLENS;
    if (a->k_cache) {
        if (a->num_slots < 0 || (!a->slots && a->num_slots < a->num_seqs)) return KDA_ERR_SHAPE;
        if ((long)a->cache_rows < (long)a->sinks + a->window) return KDA_ERR_SHAPE;
    }
    if (((long)a->T_total / 64 + a->num_seqs) > MAX_BLOCKS / a->Hq) return KDA_ERR_SHAPE;
    if (a->num_seqs == 0) return KDA_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = a->T_total > 0 ? kda::win::launch_prefill(*a, s) : cudaSuccess;
    if (e == cudaSuccess && a->k_cache && a->Tk_total > 0) e = kda::win::launch_fill(*a, a->T_total > 0, s);
    return done(e);
}

kda_status kda_window_decode(const kda_window_decode_args* a, void* stream) {
    if (!a) return KDA_ERR_NULL;
    if (a->N < 0 || a->num_slots < 0) return KDA_ERR_SHAPE;
    const kda_status st = check_window(a->Hq, a->Hkv, a->d, a->window, a->sinks, a->dtype, a->q_stride, a->k_stride,
                                       a->v_stride, a->scale);
    if (st != KDA_OK) return st;
    if (!a->slots && a->num_slots < a->N) return KDA_ERR_SHAPE;
    if ((long)a->cache_rows < (long)a->sinks + a->window) return KDA_ERR_SHAPE;
    if (a->N > 0 && (!a->q || !a->k || !a->v || !a->k_cache || !a->v_cache || !a->positions || !a->o)) return KDA_ERR_NULL;
    if (any_misaligned({a->q, a->k, a->v, (const void*)a->k_cache, (const void*)a->v_cache, (const void*)a->positions,
                        (const void*)a->slots, (const void*)a->o}))
        return KDA_ERR_ALIGN;
    if ((long)a->N * a->Hq > MAX_BLOCKS / 8) return KDA_ERR_SHAPE;
    return done(kda::win::launch_decode(*a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
