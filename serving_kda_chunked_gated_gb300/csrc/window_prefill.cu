// Sliding-window attention with sinks over packed sequences, on tcgen05.
//
// Work unit: 256 rows of one key head's attention, two tiles A and B of 128 rows.
// Row r of a tile is query r / GP and head r % GP, GP the largest power of two that
// divides the group (at most 16): the heads that share a key head share its tiles,
// and a unit covers few queries, so its key range is hardly wider than the window
// itself.  The unit's keys are the window's union [lo, p_last] in tiles of 128 (the
// last one only as wide as needed, in steps of 32), then the sinks before lo.
//
//   S = Q K^T (TMEM, 128 x 128 fp32 per tile), P = exp2(c S - m) in registers with the
//   running row maximum m and sum l, P back to TMEM as bf16 over S, O += P V (TMEM).
// A new maximum rescales O only when it exceeds the reference by more than 2^8 (the
// weights then stay below 2^8, which costs bf16 and fp32 nothing): O is rarely touched.
//
// Roles of the 16 warps: 0-3 the softmax of tile A, 4-7 that of tile B (one thread per
// row), 8-11 the output rows of both, 12 the TMA loads, 13 and 14 the MMAs of a tile each
// (15 only fills its warpgroup).  While one tile is in its softmax the tensor core works on
// the other, and one issuing warp's waits hide behind the other's MMAs;
// the first half of a tile's P V runs while the second half of its P is being made.  CTAs
// are persistent: the loads and the first S of the next unit run while this unit's rows
// are written.
//
// V is the B operand straight from the TMA tile (MN-major), Q and K are K-major; no
// thread touches an operand but for zeroing the unseen rows of edge tiles (0 x NaN).
//
// Two bounds meet: a round (both tiles' P V and Q K^T, d = 128) keeps the tensor core busy for
// 2068 cycles, and its 2 x 128 x 128 exponentials the special-function units (16 a cycle) for
// 2048.  Measured: 8192 tokens, 32 / 8 heads of 128, window 4096: 331 us, some 3600 cycles a
// round (TMEM reads slow down while products run, instructions arrive late), 1.24 PFLOP/s; 131072
// tokens, window 512: 1.39 ms, where a unit has 5 rounds and its change (queries in, rows out)
// costs another.
#include <math.h>

#include <algorithm>

#include "kda_common.cuh"
#include "tcgen05.cuh"
#include "tma_host.cuh"

namespace kda {
namespace win {

constexpr int PF_THREADS = 512;
constexpr int KT = 128;                     // keys per tile
// The tiles stream through a ring of slots in the order K0, V0 K1, V1 K2, ..., over all
// units of a CTA.  Round 0 consumes K0 (the first S), round r >= 1 the values V of the
// r-th softmax step and the keys K of the next one: one full and one empty barrier per
// round, ROUNDS of them in turn (more rounds than the ring holds).
constexpr int ROUNDS = 8;
// Unit geometries ahead of their readers.  The loads of a unit wait for the last S of the
// unit before, whose products waited for the output rows of the third before it: four do.
constexpr int UNITS = 4;

template <int D>
struct PF {
    static constexpr int QB = 128 * D * 2;          // bytes of one Q tile
    static constexpr int SB = KT * D * 2;           // bytes of one K or V tile (ring slot)
    static constexpr int SLOTS = D == 128 ? 5 : 9;
    static constexpr int SMEM = 2 * QB + SLOTS * SB + 1024;   // + alignment slack
    // TMEM columns: S of both tiles, O of both, and P where there is room beside them: S of the next
    // step is then formed while this step's weights are, and the tiles take no turns (16384 tokens, 24 / 8
    // heads of 64, window 512: 165 -> 154 us; window 4096, where the exponentials decide, no
    // change).  Otherwise P takes the place of S.
    static constexpr bool EARLY = D == 64;
    static constexpr int P0 = EARLY ? 384 : 0, PSTEP = EARLY ? 64 : 128;
};

__device__ int g_window_error;              // ERR_ bits of calls without a word of their own (sticky until read)

struct PfParams {
    kda_window_prefill_args a;
    int gp, subs;                           // rows' heads per tile; head subgroups per key head
    int qpt;                                // queries per tile (128 / gp)
    uint32_t units;                         // at most 2^31 - 1
    float c;                                // |scale| log2 e
    int neg;                                // scale < 0: S = -Q K^T
    int wide;                               // o is 32-byte aligned
    uint32_t wait_limit;
};

// One unit's geometry, from its index; called by whole warps.
struct Unit {
    int q0, q1;        // packed query rows [q0, q1) of the unit
    int p0;            // position of query q0 in its sequence
    int k0;            // packed key row of position 0
    int lo, hi;        // window keys: positions [lo, hi]
    int nsink;         // sink keys before lo: positions [0, nsink)
    int nwin, ntiles;  // window tiles, all tiles
    int hk, h0;        // key head, first query head
    // tile i: first position and width (a multiple of 32, at most KT)
    KDA_DEV void tile(int i, int* j0, int* width) const {
        const bool w = i < nwin;
        *j0 = w ? lo + i * KT : (i - nwin) * KT;
        const int left = (w ? hi + 1 : nsink) - *j0;
        *width = left >= KT ? KT : (left + 31) & ~31;
    }
    // rows of tile i that some query of the unit sees
    KDA_DEV int seen(int i) const {
        const bool w = i < nwin;
        const int left = w ? hi + 1 - (lo + i * KT) : nsink - (i - nwin) * KT;
        return left < KT ? left : KT;
    }
};

// The unit of a CTA's turn r.  Units get cheaper as they go (below), and every other turn deals them
// the other way round, which leaves the CTAs even: 4096 tokens, window 2048: 114 -> 105 us.
KDA_DEV uint32_t unit_of(uint32_t r) {
    const uint32_t g = gridDim.x, k = blockIdx.x;
    return r * g + (r & 1 ? g - 1 - k : k);
}

// A place in the list of query blocks (2 qpt queries each).  The list takes 32 sequences at a time,
// the last ones first, and of these the blocks at the highest positions first, where windows
// are full.  It moves with the units: none is before the last one.
struct Place {
    int base;              // the sequences are base .. base + 31, one per lane:
    int first, end;        // their blocks' levels, in blocks from position 0
    int q0, q1, k0, hist;  // packed query rows, first key row, keys before the queries
    int level, left;       // the level to come, blocks of these sequences from it down
    int before;            // blocks in front of it
};

KDA_DEV void enter(const PfParams& p, Place& at) {
    const int m = at.base + (int)(threadIdx.x & 31), per = 2 * p.qpt;
    at.q0 = at.q1 = at.k0 = at.hist = 0;
    if (m < p.a.num_seqs) {
        at.q0 = p.a.cu_seqlens[m];
        at.q1 = p.a.cu_seqlens[m + 1];
        at.k0 = p.a.cu_seqlens_k[m];
        at.hist = p.a.cu_seqlens_k[m + 1] - at.k0 - (at.q1 - at.q0);
    }
    const int blocks = (at.q1 - at.q0 + per - 1) / per;
    at.first = at.hist / per;
    at.end = at.first + blocks;
    at.level = __reduce_max_sync(~0u, blocks ? at.end - 1 : 0);
    at.left = __reduce_add_sync(~0u, blocks);
}

KDA_DEV Unit unit_at(const PfParams& p, uint32_t u, Place& at) {
    const uint32_t heads = p.a.Hkv * p.subs;
    const int hs = (int)(u % heads), idx = (int)(u / heads), per = 2 * p.qpt;      // idx: block in the list
    const int lane = threadIdx.x & 31;
    int f = 0, b = 0;                       // lane of the sequence, block in it
    for (;;) {
        while (at.left == 0 && at.base > 0) {
            at.base -= 32;
            enter(p, at);
        }
        if (at.left == 0) break;            // (not for u < units)
        // the sequences at this level, and down to which level they are the same ones
        const bool at_it = at.first <= at.level && at.level < at.end;
        const unsigned here = __ballot_sync(~0u, at_it);
        const int low = __reduce_max_sync(~0u, at_it ? at.first : at.first < at.end && at.end <= at.level ? at.end : 0);
        const int many = __popc(here), levels = at.level - low + 1;
        const int rank = idx - at.before, down = rank < levels * many ? rank / many : levels;
        at.before += down * many;
        at.left -= down * many;
        at.level -= down;
        if (down < levels) {
            const bool mine = at_it && __popc(here & ((1u << lane) - 1)) == idx - at.before;
            f = __ffs(__ballot_sync(~0u, mine)) - 1;
            b = at.level - __shfl_sync(~0u, at.first, f);
            break;
        }
    }
    Unit x;
    x.k0 = __shfl_sync(~0u, at.k0, f);
    x.q0 = __shfl_sync(~0u, at.q0, f) + b * per;
    x.q1 = min(__shfl_sync(~0u, at.q1, f), x.q0 + per);
    x.p0 = __shfl_sync(~0u, at.hist, f) + b * per;
    x.hi = x.p0 + (x.q1 - x.q0) - 1;
    x.lo = max(0, x.p0 - p.a.window + 1);
    x.nsink = min(p.a.sinks, x.lo);
    x.nwin = (x.hi - x.lo + KT) / KT;
    x.ntiles = x.nwin + (x.nsink + KT - 1) / KT;
    x.hk = hs / p.subs;
    x.h0 = x.hk * (p.a.Hq / p.a.Hkv) + (hs % p.subs) * p.gp;
    return x;
}

// A wait of a whole warp: every lane gets the same answer.  The first poll stands apart:
// most waits end with it (3 % on the whole kernel).
KDA_DEV bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t limit, volatile int* abort) {
    if (limit && __all_sync(~0u, tc::mbar_try_wait(bar, parity))) return true;
    return __all_sync(~0u, tc::mbar_wait_role(bar, parity, limit, abort));
}

// lane 0's value, which the compiler then knows to be the same in every lane
KDA_DEV uint32_t uniform(uint32_t x) { return __shfl_sync(~0u, x, 0); }

// two float32 operations in one instruction: d = x c + b, and l += e
KDA_DEV void fma2(float& d0, float& d1, float x0, float x1, float c, float b) {
    asm("{\n\t.reg .b64 x, c, b, d;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 c, {%4, %4};\n\tmov.b64 b, {%5, %5};\n\t"
        "fma.rn.ftz.f32x2 d, x, c, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(x0), "f"(x1), "f"(c), "f"(b));
}
// The registers of an asynchronous TMEM load are the compiler's to use only behind the wait.
KDA_DEV void after_wait(float* s, int n) {
#pragma unroll
    for (int i = 0; i < n; ++i) asm volatile("" : "+f"(s[i]));
}
KDA_DEV void add2(float& l0, float& l1, float e0, float e1) {
    asm("{\n\t.reg .b64 l, e;\n\t"
        "mov.b64 l, {%0, %1};\n\tmov.b64 e, {%2, %3};\n\t"
        "add.rn.ftz.f32x2 l, l, e;\n\tmov.b64 {%0, %1}, l;\n\t}"
        : "+f"(l0), "+f"(l1) : "f"(e0), "f"(e1));
}

template <int D>
__global__ void __launch_bounds__(PF_THREADS, 1)
window_prefill_kernel(const __grid_constant__ PfParams p, const __grid_constant__ CUtensorMap mq,
                      const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using L = PF<D>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[ROUNDS], empty[ROUNDS], edge, q_full, q_empty, s_full[2], p_full[2][2], o_full[2],
        l_full[2], o_empty[2], u_full[UNITS], turn[2], s_free[2], pv_done[2], drained;
    __shared__ Unit s_unit[UNITS];
    __shared__ float s_l[2][128];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sq = sm;
    uint8_t* ring = sm + 2 * L::QB;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int* abort = &s_abort;

    if (p.a.k_cache) tc::launch_dependents();      // the cache fill, on the SMs that this grid leaves
    if (tid == 0) {
        for (int i = 0; i < ROUNDS; ++i) { tc::mbar_init(&full[i], 2); tc::mbar_init(&empty[i], 2); }
        for (int i = 0; i < UNITS; ++i) tc::mbar_init(&u_full[i], 1);
        tc::mbar_init(&edge, 1);
        tc::mbar_init(&q_full, 1);
        tc::mbar_init(&q_empty, 2);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s_full[i], 1);
            tc::mbar_init(&turn[i], 1);
            tc::mbar_init(&s_free[i], 4);          // warps
            tc::mbar_init(&pv_done[i], 1);
            tc::mbar_init(&p_full[i][0], 4);
            tc::mbar_init(&p_full[i][1], 4);
            tc::mbar_init(&o_full[i], 1);
            tc::mbar_init(&l_full[i], 4);
            tc::mbar_init(&o_empty[i], 4);
        }
        tc::mbar_init(&drained, 2);
        tc::mbar_fence_init();
        s_abort = 0;
    }
    if (warp == 13) {
        tc::tmem_alloc(&s_tmem, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = s_tmem;
    const uint32_t limit = p.wait_limit;
    // The launch has 128 registers for each of the 512 threads (65536); a softmax thread
    // holds a whole row: 2 x 128 x 184 + 2 x 128 x 72 = 65536.
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 12) {
            // ---------------- loads: Q of a unit, then K and V tiles through the ring ----------------
            uint32_t it = 0, edges = 0, nu = 0, nq = 0;     // items, zeroed tiles, units, Q loads so far
            bool ok = true, direct = true;         // direct: the last item counts on its round's barrier
            Place place;
            place.base = (p.a.num_seqs - 1) & ~31;
            place.before = 0;
            enter(p, place);
            for (uint32_t u; (u = unit_of(nu)) < p.units && ok; ++nu) {
                const Unit x = unit_at(p, u, place);
                for (int i = 0; i < x.ntiles && ok; ++i) {
                    int j0, width;
                    x.tile(i, &j0, &width);
                    const int seen = x.seen(i);
                    if (i == 0) {
                        if (nu > 0) ok = wait_warp(&q_empty, (nu - 1) & 1, limit, abort);
                        if (!ok) break;
                        if (lane == 0) {
                            s_unit[nu % UNITS] = x;
                            tc::mbar_arrive(&u_full[nu % UNITS]);
                            tc::mbar_arrive_expect_tx(&q_full, 2 * L::QB);
                            for (int t = 0; t < 2; ++t)
                                for (int s = 0; s < D / 64; ++s)
                                    tc::tma_load_3d(sq + t * L::QB + s * 16384, &mq, s * 64, x.h0, x.q0 + t * p.qpt, &q_full);
                        }
                        ++nq;
                    }
                    for (int kv = 0; kv < 2; ++kv) {       // item `it`: even K, odd V, consumed in round ceil(it / 2)
                        const int slot = it % L::SLOTS;
                        if (it >= L::SLOTS) {
                            const uint32_t r = (it - L::SLOTS + 1) >> 1;     // the round that frees the slot
                            ok = wait_warp(&empty[r % ROUNDS], (r / ROUNDS) & 1, limit, abort);
                        }
                        if (!ok) break;
                        uint8_t* dst = ring + slot * L::SB;
                        uint64_t* round = &full[((it + 1) >> 1) % ROUNDS];
                        const bool zero = kv == 1 && seen < width;    // V rows that nothing sees are multiplied by 0
                        uint64_t* bar = zero ? &edge : round;
                        if (lane == 0) {
                            tc::mbar_arrive_expect_tx(bar, L::SB);
                            if (it == 0) tc::mbar_arrive(bar);        // round 0 has no values
                            for (int s = 0; s < D / 64; ++s)
                                tc::tma_load_3d(dst + s * 16384, kv ? &mv : &mk, s * 64, x.hk, x.k0 + j0, bar);
                        }
                        ++it;
                        direct = !zero;
                        if (zero) {
                            ok = wait_warp(&edge, edges & 1, limit, abort);
                            ++edges;
                            if (!ok) break;
                            // 16-byte pieces of rows [seen, width); the swizzle permutes pieces within a row only
                            for (int e = lane; e < (width - seen) * (D / 8); e += 32) {
                                const int r = seen + e / (D / 8), c = e % (D / 8);
                                *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                            }
                            tc::fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) tc::mbar_arrive(round);
                        }
                    }
                }
            }
            if (ok && it > 0 && lane == 0) tc::mbar_arrive(&full[(it >> 1) % ROUNDS]);   // the last round has no keys
            if (!ok && lane == 0) {
                // Give up.  The copies issued so far land before the CTA leaves: those of Q and of the
                // zeroed tiles complete their phases; a round's phase may stay open for want of its
                // other half, so its bytes are given the default bound of a wait, too.
                bool d = tc::drain_phase(&q_full, nq) && tc::drain_phase(&edge, edges);
                const uint32_t whole = (it + 1) >> 1;          // rounds 0 .. whole - 1 have both halves
                for (uint32_t r = whole > ROUNDS ? whole - ROUNDS : 0; r < whole; ++r)
                    d = tc::mbar_wait_bounded(&full[r % ROUNDS], (r / ROUNDS) & 1, tc::WAIT_POLLS) && d;
                if (it > 0 && (it & 1) == 0 && direct) {         // values without their keys: supply the arrival
                    tc::mbar_arrive(&full[whole % ROUNDS]);
                    d = tc::mbar_wait_bounded(&full[whole % ROUNDS], (whole / ROUNDS) & 1, tc::WAIT_POLLS) && d;
                }
                atomicOr(p.a.error, d ? tc::ERR_WAIT : tc::ERR_WAIT | tc::ERR_DRAIN);
            }
        } else if (warp < 15) {
            // ---------------- MMAs of tile t: the warp computes together, one lane issues ----------------
            // d = 128: the tiles take turns: A's products of a round, B's, A's of the next round, handed on by the
            // barriers `turn`.  One tile's S is so ready while the other's products run, and the two
            // softmaxes stay half a round apart; with the products interleaved both S arrive together
            // and the softmaxes share the issue slots while the tensor core waits (4600 cycles a round).
            // Two warps, because the waits and the commits of one hide behind the other's products.
            const int t = warp - 13;
            uint32_t rd = 0, nu = 0, np = 0;       // rounds, units, softmax steps
            bool ok = true;
            const uint32_t ra = uniform(tc::smem_u32(ring)), tmu = uniform(tm);
            const uint64_t qd = tc::sw128_desc(uniform(tc::smem_u32(sq)) + t * L::QB);
            auto qk = [&](uint32_t slot, int width) {
                const uint32_t id = tc::idesc_bf16(128, width, false, false, p.neg != 0);
                const uint64_t kd = tc::sw128_desc(ra + slot * L::SB);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;      // descriptors count 16 bytes
                    tc::mma_f16_ss_elect(tmu + t * 128, qd + off, kd + off, id, k > 0);
                }
            };
            auto pv = [&](uint32_t slot, int half, int steps, bool first) {
                const uint32_t id = tc::idesc_bf16(128, D, false, true);
                const uint64_t vd = tc::sw128_desc_mn(ra + slot * L::SB, 16384);
                const int k0 = 4 * half;
                if (steps >= k0 + 4) {              // without a test between the products
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tc::mma_f16_ts_elect(tmu + 256 + t * D, tmu + L::P0 + t * L::PSTEP + (k0 + k) * 8, vd + (k0 + k) * (2048 >> 4), id,
                                             !(first && k0 + k == 0));
                } else {
#pragma unroll 1
                    for (int k = k0; k < steps; ++k)
                        tc::mma_f16_ts_elect(tmu + 256 + t * D, tmu + L::P0 + t * L::PSTEP + k * 8, vd + k * (2048 >> 4), id,
                                             !(first && k == 0));
                }
            };
            // Round r of A waits for B's round r - 1, that of B for A's round r.
            auto my_turn = [&](uint32_t r) { return L::EARLY ? true : t ? wait_warp(&turn[1], r & 1, limit, abort) : r == 0 || wait_warp(&turn[0], (r - 1) & 1, limit, abort); };
            auto hand_on = [&] {
                if (L::EARLY) return;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&turn[1 - t]);
            };
            // widths of a unit's tiles, uniform over the warp
            struct Tiles { int nwin, ntiles, wlast, slast; };
            auto tiles_of = [&](uint32_t n) {
                const Unit x = s_unit[n % UNITS];
                Tiles r;
                int j0, w;
                r.nwin = uniform(x.nwin);
                r.ntiles = uniform(x.ntiles);
                x.tile(x.nwin - 1, &j0, &w);
                r.wlast = uniform(w);
                x.tile(x.ntiles - 1, &j0, &w);
                r.slast = uniform(w);
                return r;
            };
            auto width_of = [&](const Tiles& r, int i) { return i == r.ntiles - 1 ? r.slast : i == r.nwin - 1 ? r.wlast : KT; };
            Tiles x = {0, 0, 0, 0};
            uint32_t vs = L::SLOTS - 1, ks = 0;    // slots of this round's values and keys
            if (unit_of(0) < p.units) {
                ok = wait_warp(&u_full[0], 0, limit, abort) && wait_warp(&q_full, 0, limit, abort) &&
                     wait_warp(&full[0], 0, limit, abort) && my_turn(0);
                tc::fence_after_sync();
                if (ok) {
                    x = tiles_of(0);
                    qk(0, width_of(x, 0));
                    tc::mma_commit_elect(&s_full[t]);
                    hand_on();
                    tc::mma_commit_elect(&empty[0]);
                    if (x.ntiles == 1) tc::mma_commit_elect(&q_empty);
                }
                rd = 1;
            }
#pragma unroll 1
            for (; unit_of(nu) < p.units && ok; ++nu) {
                const bool next_unit = unit_of(nu + 1) < p.units;
                Tiles y = x;
#pragma unroll 1
                for (int i = 0; i < x.ntiles; ++i, ++np, ++rd) {
                    const bool last = i + 1 == x.ntiles, more = !last || next_unit;
                    vs = vs + 2 >= L::SLOTS ? vs + 2 - L::SLOTS : vs + 2;
                    ks = ks + 2 >= L::SLOTS ? ks + 2 - L::SLOTS : ks + 2;
                    const int steps = width_of(x, i) / 16;
                    ok = wait_warp(&full[rd % ROUNDS], (rd / ROUNDS) & 1, limit, abort);
                    if (L::EARLY && !last) {           // S has been read: the next one
                        ok = ok && wait_warp(&s_free[t], np & 1, limit, abort);
                        tc::fence_after_sync();
                        if (!ok) break;
                        qk(ks, width_of(x, i + 1));
                        tc::mma_commit_elect(&s_full[t]);
                        if (i + 2 == x.ntiles) tc::mma_commit_elect(&q_empty);
                    }
                    if (ok && i == 0 && nu > 0) ok = wait_warp(&o_empty[t], (nu - 1) & 1, limit, abort);
                    ok = ok && my_turn(rd) && wait_warp(&p_full[t][0], np & 1, limit, abort);
                    tc::fence_after_sync();
                    if (ok) pv(vs, 0, steps, i == 0);
                    ok = ok && wait_warp(&p_full[t][1], np & 1, limit, abort);
                    tc::fence_after_sync();
                    if (ok) pv(vs, 1, steps, i == 0);
                    if (!ok) break;
                    if (L::EARLY) tc::mma_commit_elect(&pv_done[t]);
                    if (last) {
                        tc::mma_commit_elect(&o_full[t]);
                        if (next_unit) {
                            ok = wait_warp(&u_full[(nu + 1) % UNITS], ((nu + 1) / UNITS) & 1, limit, abort) &&
                                 wait_warp(&q_full, (nu + 1) & 1, limit, abort);
                            if (!ok) break;
                            y = tiles_of(nu + 1);
                        }
                    }
                    if (L::EARLY ? last && more : more) {
                        qk(ks, last ? width_of(y, 0) : width_of(x, i + 1));
                        tc::mma_commit_elect(&s_full[t]);
                    }
                    hand_on();
                    tc::mma_commit_elect(&empty[rd % ROUNDS]);
                    // the S issued in this round was a unit's last: its Q may be overwritten
                    if (last ? more && y.ntiles == 1 : !L::EARLY && i + 2 == x.ntiles) tc::mma_commit_elect(&q_empty);
                }
                x = y;
            }
            // everything issued has finished before TMEM and shared memory are given back
            __syncwarp();
            tc::mma_commit_elect(&drained);
            if (lane == 0) {
                const bool d = tc::mbar_wait_bounded(&drained, 0, tc::WAIT_POLLS);
                if (!ok || !d) atomicOr(p.a.error, d ? tc::ERR_WAIT : tc::ERR_WAIT | tc::ERR_DRAIN);
            }
            __syncwarp();
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // ---------------- output rows: O / l, one row per thread ----------------
        const int r = tid & 127;
        uint32_t nu = 0;
        bool ok = true;
        for (; unit_of(nu) < p.units && ok; ++nu) {
            ok = wait_warp(&u_full[nu % UNITS], (nu / UNITS) & 1, limit, abort);
            if (!ok) break;
            const Unit x = s_unit[nu % UNITS];
            for (int t = 0; t < 2; ++t) {
                ok = wait_warp(&l_full[t], nu & 1, limit, abort) && wait_warp(&o_full[t], nu & 1, limit, abort);
                if (!ok) break;
                tc::fence_after_sync();
                const uint32_t to = tm + 256 + t * D + ((uint32_t)(warp & 3) << 21);
                const float inv = 1.0f / s_l[t][r];
                const int q = x.q0 + t * p.qpt + r / p.gp;
                const bool live = q < x.q1;
                const size_t row = (size_t)q * p.a.Hq + x.h0 + r % p.gp;
                uint16_t* out = reinterpret_cast<uint16_t*>(p.a.o) + row * D;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    float o[32];
                    tc::tmem_ld32(to + k * 32, o);
                    tc::tmem_ld_wait();
                    if (k == D / 32 - 1) {        // O and l have been read: the next unit may write them
                        tc::fence_before_sync();
                        tc::mbar_arrive_warp(&o_empty[t]);
                    }
                    if (live) {
#pragma unroll
                        for (int c = 0; c < 32; c += 16) {            // 32 bytes, a whole sector, per store where o allows it
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(o[c + 2 * e] * inv, o[c + 2 * e + 1] * inv);
                                v[e] = __uint_as_float(*reinterpret_cast<const uint32_t*>(&h));
                            }
                            if (p.wide) {
                                st_stream_f8(reinterpret_cast<float*>(out + k * 32 + c), v);
                            } else {
                                st_stream_f4(reinterpret_cast<float*>(out + k * 32 + c), make_float4(v[0], v[1], v[2], v[3]));
                                st_stream_f4(reinterpret_cast<float*>(out + k * 32 + c + 8), make_float4(v[4], v[5], v[6], v[7]));
                            }
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ---------------- softmax of tile t, one row per thread ----------------
        const int t = warp >> 2, r = tid & 127;
        const uint32_t ts = tm + t * 128 + ((uint32_t)(warp & 3) << 21);        // this warp's 32 lanes of S (and P)
        const uint32_t to = tm + 256 + t * D + ((uint32_t)(warp & 3) << 21);
        const uint32_t tp = tm + L::P0 + t * L::PSTEP + ((uint32_t)(warp & 3) << 21);
        uint32_t np = 0, nu = 0;
        bool ok = true;
        for (; unit_of(nu) < p.units && ok; ++nu) {
            ok = wait_warp(&u_full[nu % UNITS], (nu / UNITS) & 1, limit, abort);
            if (!ok) break;
            const Unit x = s_unit[nu % UNITS];
            const int pos = x.p0 + t * p.qpt + r / p.gp;          // position of this row's query
            float ref = -INFINITY, l0 = 0.f, l1 = 0.f;            // reference (scaled), sum in two parts
            // the tile's rows see everything between these positions without a mask
            const int pmin = x.p0 + t * p.qpt, pmax = min(x.hi, pmin + p.qpt - 1);
            for (int i = 0; i < x.ntiles; ++i, ++np) {
                int j0, width;
                x.tile(i, &j0, &width);
                ok = wait_warp(&s_full[t], np & 1, limit, abort);
                if (!ok) break;
                tc::fence_after_sync();
                float s[KT];
                const bool window = i < x.nwin;
                const bool whole = window && j0 + width - 1 <= pmin && j0 > pmax - p.a.window;
                // columns [a, b] of the window and columns below z of the sinks are seen
                const int b = window ? pos - j0 : -1, a = window ? max(0, pos - p.a.window + 1 - j0) : 0;
                const int z = window ? min(p.a.sinks - j0, b + 1) : x.nsink - j0;
                // masks 32 columns.  A warp's rows are few queries, so most chunks of an edge tile are
                // seen by all of them.
                auto mask = [&](int k) {
                    if (!whole) {
                        const int hi = min(31, b - 32 * k), lo = max(0, a - 32 * k), zz = min(32, z - 32 * k);
                        uint32_t seen = hi >= lo && lo < 32 ? (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo) : 0u;
                        if (zz > 0) seen |= 0xffffffffu >> (32 - zz);
                        if (!__all_sync(~0u, seen == 0xffffffffu)) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) s[32 * k + c] = (seen >> c) & 1u ? s[32 * k + c] : -INFINITY;
                        }
                    }
                };
                auto largest = [&](int k, float m) {
                    float m0 = m, m1 = s[32 * k];
#pragma unroll
                    for (int c = 1; c < 31; c += 4) {
                        m0 = fmaxf(fmaxf(m0, s[32 * k + c]), s[32 * k + c + 1]);
                        m1 = fmaxf(fmaxf(m1, s[32 * k + c + 2]), c + 3 < 32 ? s[32 * k + c + 3] : m1);
                    }
                    return fmaxf(fmaxf(m0, m1), s[32 * k + 31]);
                };
                // exp2(c s - ref) of 32 columns, their sum, and P in bf16 over S (S is in registers)
                auto weigh = [&](int k, float base, float& l0, float& l1) {
                    uint32_t w[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        float e0, e1;
                        fma2(e0, e1, s[32 * k + c], s[32 * k + c + 1], p.c, base);
                        e0 = exp2f(e0);
                        e1 = exp2f(e1);
                        add2(l0, l1, e0, e1);
                        // weights rounded to bf16 for the product (its operands share a type, and V is
                        // bf16; a second part would double P V and the stores of P); l keeps float32
                        const __nv_bfloat162 h = __floats2bfloat162_rn(e0, e1);
                        w[c >> 1] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    tc::tmem_st16u(tp + k * 16, w);
                };
                // The row's reference is the largest score known before this tile (on the first tile: its
                // own first half's), so the exponentials need not wait for the tile's maximum, nor for its
                // last columns: TMEM reads crawl while the other tile's products run (64 columns in some
                // 700 cycles).  Where the maximum outgrows the reference by 2^8 the tile is done again.
                tc::tmem_ld64(ts, s);              // one load of 64 columns: two of 32 cost 8 % of the kernel
                tc::tmem_ld_wait();
                after_wait(s, 64);
                if (64 < width) tc::tmem_ld64(ts + 64, s + 64);
                mask(0);
                if (32 < width) mask(1);
                float m01 = largest(0, -INFINITY);     // of the first half: in the tile's maximum, too (2 %)
                if (32 < width) m01 = largest(1, m01);
                if (i == 0) ref = m01 * p.c;
                if (L::EARLY && np > 0) {              // P and O of the step before are the row's again
                    ok = wait_warp(&pv_done[t], (np - 1) & 1, limit, abort);
                    if (!ok) {
                        tc::tmem_ld_wait();            // the second half of S is still on its way
                        break;
                    }
                    tc::fence_after_sync();
                }
                for (bool again = false;; again = true) {
                    const float base = ref == -INFINITY ? 0.f : -ref;   // nothing seen yet: every weight is exp2(-inf) = 0
                    float n0 = 0.f, n1 = 0.f;
                    weigh(0, base, n0, n1);
                    if (32 < width) weigh(1, base, n0, n1);
                    if (!again) {
                        tc::tmem_ld_wait();
                        after_wait(s + 64, 64);
                        if (L::EARLY) {
                            tc::fence_before_sync();
                            tc::mbar_arrive_warp(&s_free[t]);
                        }
                        if (64 < width) mask(2);
                        if (96 < width) mask(3);
                        float m = m01;
                        if (64 < width) m = largest(2, m);
                        if (96 < width) m = largest(3, m);
                        m *= p.c;
                        const bool grow = m > ref + 8.f;                // (always from no reference)
                        if (__any_sync(~0u, grow)) {
                            const float nref = grow ? m : ref;
                            const float f = ref == -INFINITY ? 0.f : exp2f(ref - nref);
                            l0 *= f;
                            l1 *= f;
                            ref = nref;
                            if (i > 0) {
#pragma unroll 1
                                for (int k = 0; k < D / 16; ++k) {
                                    float o[16];
                                    tc::tmem_ld16(to + k * 16, o);
                                    tc::tmem_ld_wait();
#pragma unroll
                                    for (int c = 0; c < 16; ++c) o[c] *= f;
                                    tc::tmem_st16(to + k * 16, o);
                                }
                            }
                            continue;
                        }
                    }
                    tc::tmem_st_wait();
                    tc::fence_before_sync();
                    tc::mbar_arrive_warp(&p_full[t][0]);
                    if (64 < width) weigh(2, base, n0, n1);
                    if (96 < width) weigh(3, base, n0, n1);
                    l0 += n0;
                    l1 += n1;
                    tc::tmem_st_wait();
                    tc::fence_before_sync();
                    tc::mbar_arrive_warp(&p_full[t][1]);
                    break;
                }
            }
            if (!ok) break;
            if (nu > 0) ok = wait_warp(&o_empty[t], (nu - 1) & 1, limit, abort);   // the last unit's l has been read
            if (!ok) break;
            s_l[t][r] = l0 + l1;
            tc::mbar_arrive_warp(&l_full[t]);
            const int q = x.q0 + t * p.qpt + r / p.gp;
            if (p.a.lse && q < x.q1)
                p.a.lse[(size_t)q * p.a.Hq + x.h0 + r % p.gp] = 0.6931471805599453f * ref + logf(l0 + l1);
            __syncwarp();
        }
    }
    __syncthreads();
    if (warp == 13) tc::tmem_dealloc(tm, 512);
}

cudaError_t error_word(void** out) { return cudaGetSymbolAddress(out, g_window_error); }

template <int D>
static cudaError_t prefill_d(const kda_window_prefill_args& a, cudaStream_t s) {
    PfParams p;
    p.a = a;
    p.a.window = std::min(a.window, a.Tk_total);       // as wide as any sequence: sums of positions stay in 32 bits
    const int G = a.Hq / a.Hkv;
    p.gp = G & -G;
    if (p.gp > 16) p.gp = 16;
    p.subs = G / p.gp;
    p.qpt = 128 / p.gp;
    long blocks = 0;
    for (int n = 0; n < a.num_seqs; ++n)
        blocks += (a.cu_seqlens_host[n + 1] - a.cu_seqlens_host[n] + 2 * p.qpt - 1) / (2 * p.qpt);
    p.units = (uint32_t)(blocks * a.Hkv * p.subs);
    if (p.units == 0) return cudaSuccess;
    // a zero scale keeps exp2(fma(-inf, c, ...)) at 0 for masked scores
    p.c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-37f);
    p.neg = a.scale < 0.f;
    p.wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
    p.wait_limit = wait_limit();
    CUtensorMap mq, mk, mv;
    cudaError_t e = make_map_heads(&mq, a.q, D, a.Hq, a.T_total, a.q_stride, p.gp, p.qpt);
    if (e == cudaSuccess) e = make_map_heads(&mk, a.k, D, a.Hkv, a.Tk_total, a.k_stride, 1, KT);
    if (e == cudaSuccess) e = make_map_heads(&mv, a.v, D, a.Hkv, a.Tk_total, a.v_stride, 1, KT);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(window_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, PF<D>::SMEM);
    void* shared = nullptr;
    if (e == cudaSuccess && !a.error && (e = error_word(&shared)) == cudaSuccess) p.a.error = static_cast<int32_t*>(shared);
    int dev = 0, sms = 0;
    if (e == cudaSuccess) e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const unsigned grid = std::min(p.units, (uint32_t)sms);
    window_prefill_kernel<D><<<grid, PF_THREADS, PF<D>::SMEM, s>>>(p, mq, mk, mv);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_prefill(const kda_window_prefill_args& a, cudaStream_t s) {
    return a.d == 64 ? prefill_d<64>(a, s) : prefill_d<128>(a, s);
}

}  // namespace win
}  // namespace kda
