// Attention of packed new tokens over the paged key/value cache, on tcgen05.
//
// Work unit: 256 rows of one key head's attention, two tiles A and B of 128 rows; row r of a tile is query r / GP
// and head r % GP, GP the largest power of two that divides the group (at most 16).  Its keys are the positions
// 0 .. p_last in tiles of 128, whose rows the page table names piece by piece.
//
//   S = Q K^T (TMEM, 128 x 128 fp32 per tile), P = exp2(c S - m) in registers with the
//   running row maximum m and sum l, P back to TMEM as bf16, O += P V (TMEM).
// A new maximum rescales O only when it exceeds the reference by more than 2^8 (the
// weights then stay below 2^8, which costs bf16 and fp32 nothing): O is rarely touched.
//
// The key tiles of all units, one unit after the other, are cut into even ranges, one per CTA (a CTA per SM): batches of
// any shape come out even, from a few tokens after a long history to packed prompts, and the cuts need the lengths on
// the device only.  A unit that a cut splits leaves its parts (O, m, l) in the workspace; a second kernel, whose
// launch overlaps this one, joins those.
//
// Roles of the 16 warps: 0-3 the softmax of tile A, 4-7 that of tile B (one thread per row), 12 the list
// and the TMA loads, 13 and 14 the MMAs of a tile each (15 only fills its warpgroup); 8-11 the output
// rows of both tiles, or, where the pages are 8-bit, the operands: they turn a tile of codes
// into bf16 with its rows' powers of two (exact), and the softmax warps write their rows themselves.
// While one tile is in its softmax the tensor core works on the other.
//
// V is the B operand as it lies in memory (MN-major), Q and K are K-major; bf16 pages reach the operands by TMA alone
// but for zeroing the unseen rows of a last tile (0 x NaN).
//
// Bounds and measurements (GB300): a round (both tiles' P V and Q K^T, d = 128) keeps the tensor core busy for 2068 cycles
// and takes some 3300: a tile's products wait for its softmax, 900 instructions of a warp, and the two tiles' turns
// follow one another.  8192 tokens, 32 / 8 heads of 128: 417 us, 1.32 PFLOP/s.  2048 tokens after 63488 over 8-bit pages: 2.04 ms,
// 1.06 PFLOP/s: the operands' warpgroup takes 1400 cycles for each of a round's two tiles, in shared memory that the
// products read at its full rate.  Five tokens of 16 sequences of 3000 to 13500: 115 us, 4.7 TB/s.
#include <math.h>

#include <algorithm>

#include "attn.cuh"
#include "paged.cuh"
#include "tma_host.cuh"

namespace kda {
namespace paged {

constexpr int PF_THREADS = 512;
constexpr int PF_CTAS = 152;                // at most: one per SM
constexpr int KT = 128;                     // keys per tile
// The tiles stream through a ring of slots in the order K0, V0 K1, V1 K2, ..., over all
// units of a CTA.  Round 0 consumes K0 (the first S), round r >= 1 the values V of the
// r-th softmax step and the keys K of the next one: one full and one empty barrier per
// round, ROUNDS of them in turn (more rounds than the ring holds).
constexpr int ROUNDS = 8;
// Unit records ahead of their readers.  The loads of a unit wait for the last S of the
// unit before, whose products waited for the output rows of the third before it: four do.
constexpr int UNITS = 4;
// What a unit costs beside its tiles, in tiles.  4096 tokens, 32 / 8 heads of 128, with 1, 2, 4: 123, 126, 128 us, over 8-bit pages
// 164, 171, 175.
constexpr int OVERHEAD = 1;
// Cost of a range at least.  A CTA's first product comes some 5 us after its start, beside the others', so short lists are
// spread: with 2 and 5 one token takes 10 and 13 us, 16 after 500 14 and 18, over 8-bit pages 15 and 22, 512 20 and 23; longer ones the same.
constexpr int RANGE = 2;

template <int D, bool Q8>
struct PF {
    static constexpr int QB = 128 * D * 2;          // bytes of one Q tile
    static constexpr int SB = KT * D * 2;           // bytes of one K or V tile (ring slot)
    static constexpr int RB = KT * D;               // bytes of one tile of codes
    static constexpr int RAW = !Q8 ? 0 : D == 128 ? 2 : 4;         // tiles of codes in flight
    static constexpr int SLOTS = D == 128 ? 5 - Q8 : 9 - 2 * Q8;
    static constexpr int SMEM = 2 * QB + SLOTS * SB + RAW * RB + 1024;   // + alignment slack
    // arrivals that complete a round: its two copies, or four warps for each
    static constexpr int FULL = Q8 ? 8 : 2;
    // TMEM columns: S of both tiles, O of both, and P where there is room beside them (then S of the next
    // step is formed while this step's weights are); otherwise P takes the place of S.
    static constexpr bool EARLY = D == 64;
    static constexpr int P0 = EARLY ? 384 : 0, PSTEP = EARLY ? 64 : 128;
};

struct Split { int q0, q1, h0, first, last, pad[3]; };      // a split unit and the CTAs that have its parts; q0 < 0: none

struct PfParams {
    kda_paged_prefill_args a;
    int gp, subs;                           // rows' heads per tile; head subgroups per key head
    int qpt;                                // queries per tile (128 / gp)
    int per_log;                            // log2 of the queries of a unit (2 qpt)
    int piece;                              // rows of a page that one copy takes
    float c;                                // |scale| log2 e
    int neg;                                // scale < 0: S = -Q K^T
    int wide;                               // o is 32-byte aligned
    uint32_t wait_limit;
    int* error;                             // the call's error word (a.error: the caller's, for many calls)
    int* errors;                            // [CTAs]: what each has to report
    Split* split;                           // [CTAs]: of the unit that the range's start splits, where it is the first start in it
    float* parts;                           // [CTAs][2]: 256 rows of O, then m and l
};

// One unit, or the part of it that is the CTA's: key tiles t0 .. t1 - 1.
struct Unit {
    int n;             // sequence
    int q0, q1;        // packed query rows [q0, q1)
    int p0;            // position of query q0 in its sequence (negative: before the first)
    int hi;            // the last position that a query of the unit sees (negative: none)
    int hk, h0;        // key head, first query head
    int t0, t1;
    int whole;         // all tiles of the unit
    int more;          // another unit follows
    // tile t: rows of it that some query sees, and its width (a multiple of 32, at most KT)
    KDA_DEV int seen(int t) const { return min(KT, max(0, hi + 1 - t * KT)); }
    KDA_DEV int width(int t) const { return max(32, (seen(t) + 31) & ~31); }
};

// ---------------------------------------------------------------------------
// the list of units: sequence after sequence, head after head, block after block of queries
// ---------------------------------------------------------------------------

KDA_DEV int tiles_to(int keys) { return keys <= KT ? 1 : (keys + KT - 1) / KT; }

// sum of floor(k / 2^s) over k < x
KDA_DEV long floor_sum(long x, int s) {
    const long q = x >> s;
    return ((q * (q - 1) / 2) << s) + q * (x - (q << s));
}

// Cost of the first b blocks of a sequence of m queries after `hist` keys (negative: queries before position 0).
KDA_DEV long cost_before(const PfParams& p, long hist, int m, int b) {
    const int lg = p.per_log, nb = (m + (1 << lg) - 1) >> lg;
    long sum = (long)OVERHEAD * b;
    int full = b;
    if (b == nb && b > 0) {                                   // the last block may be short
        sum += tiles_to((int)(hist + m));
        --full;
    }
    // block i, full, sees hist + (i + 1) 2^lg keys; the first `one` of them a tile at most
    const int one = (int)min((long)full, max(0L, (KT - hist) >> lg));
    sum += one;
    const long n = full - one, y = hist + ((long)(one + 1) << lg) + KT - 1;     // > 2 KT - 1 where n > 0
    if (n > 0) {
        if (lg <= 7) {
            const long k = y >> lg;
            sum += floor_sum(k + n, 7 - lg) - floor_sum(k, 7 - lg);
        } else {
            sum += n * (y >> 7) + (n * (n - 1) / 2 << (lg - 7));
        }
    }
    return sum;
}

// The loading warp's place in the list; the same in every lane.
struct Place {
    int n, hs, b;              // sequence, head subgroup, block
    int q0, m, nb;             // the sequence's first query row, queries, blocks
    long hist;
    long s;                    // the unit's start in the list; its tiles begin OVERHEAD later
    int tiles;

    KDA_DEV void unit(const PfParams& p) { tiles = tiles_to((int)(hist + min(m, (b + 1) << p.per_log))); }
    KDA_DEV void sequence(const PfParams& p, int at) {
        n = at;
        q0 = p.a.cu_seqlens[n];
        m = p.a.cu_seqlens[n + 1] - q0;
        const int len = p.a.cache.lens[n];
        if (!len_ok(p.a.cache, len)) m = 0;                   // skipped
        hist = (long)len - m;
        nb = (m + (1 << p.per_log) - 1) >> p.per_log;
    }
    // to the unit that holds x, which lies in the list
    KDA_DEV void seek(const PfParams& p, long x) {
        const int lane = threadIdx.x & 31, heads = p.a.cache.Hkv * p.subs;
        long before = 0;
        for (int base = 0; base < p.a.cache.num_seqs; base += 32) {
            Place mine;
            mine.m = mine.nb = 0;
            if (base + lane < p.a.cache.num_seqs) mine.sequence(p, base + lane);
            const long w = mine.nb ? heads * cost_before(p, mine.hist, mine.m, mine.nb) : 0;
            long sum = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long y = __shfl_up_sync(~0u, sum, o);
                if (lane >= o) sum += y;
            }
            const unsigned past = __ballot_sync(~0u, before + sum > x);
            if (past) {
                const int f = __ffs(past) - 1;
                sequence(p, base + f);
                s = before + __shfl_sync(~0u, sum - w, f);
                const long head = cost_before(p, hist, m, nb);
                hs = (int)((x - s) / head);
                s += hs * head;
                int lo = 0, up = nb;                          // cost_before(lo) <= x - s < cost_before(up)
                while (up - lo > 1) {
                    const int mid = (lo + up) >> 1;
                    if (cost_before(p, hist, m, mid) <= x - s) lo = mid; else up = mid;
                }
                b = lo;
                s += cost_before(p, hist, m, b);
                unit(p);
                return;
            }
            before += __shfl_sync(~0u, sum, 31);
        }
    }
    // to the next unit; false: there is none
    KDA_DEV bool next(const PfParams& p) {
        s += tiles + OVERHEAD;
        if (++b == nb) {
            b = 0;
            if (++hs == p.a.cache.Hkv * p.subs) {
                hs = 0;
                do {
                    if (n + 1 == p.a.cache.num_seqs) return false;
                    sequence(p, n + 1);
                } while (nb == 0);
            }
        }
        unit(p);
        return true;
    }
};

KDA_DEV long total_cost(const PfParams& p) {
    long w = 0;
    for (int n = threadIdx.x & 31; n < p.a.cache.num_seqs; n += 32) {
        Place x;
        x.sequence(p, n);
        if (x.nb) w += cost_before(p, x.hist, x.m, x.nb);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(~0u, w, o);
    return w * p.a.cache.Hkv * p.subs;
}

// 32 channels of a row as bf16, streamed out
KDA_DEV void store_row32(uint16_t* out, const float* o, float inv, bool zero, int wide) {
#pragma unroll
    for (int c = 0; c < 32; c += 16) {            // 32 bytes, a whole sector, per store where o allows it
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(o[c + 2 * e] * inv, o[c + 2 * e + 1] * inv);
            v[e] = zero ? 0.f : __uint_as_float(*reinterpret_cast<const uint32_t*>(&h));
        }
        if (wide) {
            st_stream_f8(reinterpret_cast<float*>(out + c), v);
        } else {
            st_stream_f4(reinterpret_cast<float*>(out + c), make_float4(v[0], v[1], v[2], v[3]));
            st_stream_f4(reinterpret_cast<float*>(out + c + 8), make_float4(v[4], v[5], v[6], v[7]));
        }
    }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(PF_THREADS, 1)
prefill_kernel(const __grid_constant__ PfParams p, const __grid_constant__ CUtensorMap mq,
               const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using L = PF<D, Q8>;
    extern __shared__ uint8_t raw[];
    __shared__ __align__(8) uint64_t full[ROUNDS], empty[ROUNDS], edge, q_full, q_empty, s_full[2], p_full[2][2], o_full[2],
        l_full[2], o_empty[2], u_full[UNITS], turn[2], s_free[2], pv_done[2], drained, raw_full[4], raw_empty[4];
    __shared__ Unit s_unit[UNITS];
    __shared__ float s_l[2][128];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_error;
    __shared__ uint32_t s_issued[2];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* sq = sm;
    uint8_t* ring = sm + 2 * L::QB;
    uint8_t* codes = ring + L::SLOTS * L::SB;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    volatile int* abort = &s_abort;

    tc::launch_dependents();                       // the joining kernel, on the SMs that this grid leaves
    if (tid == 0) {
        for (int i = 0; i < ROUNDS; ++i) { tc::mbar_init(&full[i], L::FULL); tc::mbar_init(&empty[i], 2); }
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
        for (int i = 0; i < 4; ++i) { tc::mbar_init(&raw_full[i], 1); tc::mbar_init(&raw_empty[i], 4); }
        tc::mbar_init(&drained, 2);
        tc::mbar_fence_init();
        s_abort = s_error = 0;
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
    // A tile's output rows, one per thread of a warpgroup (row r): O / l, or the part as it is
    auto write_rows = [&](const Unit& x, int t, int r, float l) {
        const uint32_t to = tm + 256 + t * D + ((uint32_t)(warp & 3) << 21);
        const int q = x.q0 + t * p.qpt + r / p.gp;
        const bool live = q < x.q1;
        const size_t row = (size_t)q * p.a.Hq + x.h0 + r % p.gp;
        float* part = p.parts + (size_t)(blockIdx.x * 2 + (x.t0 == 0)) * 256 * D + (t * 128 + r) * 4;     // four channels of all rows, the next four, ...
        const float inv = 1.0f / l;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
            float o[32];
            tc::tmem_ld32(to + k * 32, o);
            tc::tmem_ld_wait();
            if (k == D / 32 - 1) {                // O and l have been read: the next unit may write them
                tc::fence_before_sync();
                tc::mbar_arrive_warp(&o_empty[t]);
            }
            if (live && x.whole) {
                store_row32(reinterpret_cast<uint16_t*>(p.a.o) + row * D + k * 32, o, inv, l == 0.f, p.wide);
            } else if (live) {
#pragma unroll
                for (int c = 0; c < 32; c += 4) st_stream_f4(part + (k * 32 + c) * 256, make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]));
            }
            __syncwarp();
        }
    };
    // The launch has 128 registers for each of the 512 threads (65536); a softmax thread
    // holds a whole row: 2 x 128 x 184 + 2 x 128 x 72 = 65536.
    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 12 || (!Q8 && warp == 15)) {
            // ---------------- the list, and the loads: Q of a unit, K and V tiles through the ring ----------------
            // bf16 pages: one warp loads Q and K, the other V.  A copy takes its warp some 100 cycles, and a tile of 16-row pieces has
            // 8 or 16 of them: by one warp 4096 tokens, 32 / 8 heads of 128, pages of 16, take 172 us, by two 126; heads of 64, pages
            // of 64 108 and 93.
            const int role = warp == 15;
            const long W = total_cost(p);
            const int ctas = (int)max(1L, min((long)gridDim.x, W / RANGE));
            const long x0 = W * blockIdx.x / ctas, x1 = W * (blockIdx.x + 1) / ctas;
            Place at;
            bool have = (int)blockIdx.x < ctas && x0 < x1;
            if (have) at.seek(p, x0);
            Split sp = {-1, 0, 0, 0, 0, {0, 0, 0}};
            const int G = p.a.Hq / p.a.cache.Hkv;
            // The CTA's part of the unit at `at`, or of the first one behind it that has any; false: none
            int t0 = 0, t1 = 0;
            auto enter = [&] {
                for (;;) {
                    t0 = (int)max(0L, x0 - at.s - OVERHEAD);
                    t1 = (int)min((long)at.tiles, x1 - at.s - OVERHEAD);
                    if (t0 < t1) return true;
                    if (at.s >= x1 || !at.next(p)) return false;
                }
            };
            auto record = [&] {
                Unit x;
                x.n = at.n;
                x.q0 = at.q0 + (at.b << p.per_log);
                x.q1 = min(at.q0 + at.m, x.q0 + (1 << p.per_log));
                x.p0 = (int)at.hist + (at.b << p.per_log);
                x.hi = x.p0 + (x.q1 - x.q0) - 1;
                x.hk = at.hs / p.subs;
                x.h0 = x.hk * G + (at.hs % p.subs) * p.gp;
                x.t0 = t0;
                x.t1 = t1;
                x.whole = t0 == 0 && t1 == at.tiles;
                x.more = 0;
                return x;
            };
            have = have && enter();
            Unit x;
            if (have) {
                x = record();
                if (t0 > 0) {                      // is this start the first one in its unit?
                    const long first_tile = at.s + OVERHEAD;
                    const int first = (int)(((first_tile + 1) * ctas + W - 1) / W) - 1;     // the CTA that has tile 0
                    if (first == (int)blockIdx.x - 1)
                        sp = {x.q0, x.q1, x.h0, first, (int)(((first_tile + at.tiles) * ctas + W - 1) / W) - 1, {0, 0, 0}};
                }
            } else {
                x.t0 = x.t1 = 0;
                if (lane == 0 && !role) {
                    s_unit[0] = x;
                    tc::mbar_arrive(&u_full[0]);
                }
            }
            if (lane == 0 && !role) p.split[blockIdx.x] = sp;
            uint32_t nt = 0, edges = 0, nu = 0, nq = 0;     // tiles, zeroed tiles, units, Q loads so far
            uint32_t issued = 0;                   // items of this warp that have arrived at their barriers
            bool ok = true;
            const int pieces = KT / p.piece;       // of a tile; lane i knows the page row of piece i % pieces
            const int absent = p.a.cache.num_pages * p.a.cache.page_size;       // behind the last row: reads as zeros
            auto look_up = [&](const Unit& u, int t) {
                const int pos = t * KT + (lane & (pieces - 1)) * p.piece;
                return pos <= u.hi ? entry_of(p.a.cache, u.n, pos) : Entry{-1, 0};
            };
            Entry ahead = {-1, 0};                 // of the tile to come
            if (have) ahead = look_up(x, t0);
            while (have && ok) {
                Unit y = x;                        // the next one
                const bool more = at.s + OVERHEAD + at.tiles < x1 && at.next(p) && enter();
                if (more) y = record();
                x.more = more;
                for (int t = x.t0; t < x.t1 && ok; ++t, ++nt) {
                    const int seen = x.seen(t), width = x.width(t);
                    const int live = (seen + p.piece - 1) / p.piece;          // pieces to load
                    const int found = row(p.a.cache, ahead), here = found < 0 ? absent : found;
                    const bool turn_over = t + 1 == x.t1;
                    if (!turn_over || more) ahead = look_up(turn_over ? y : x, turn_over ? y.t0 : t + 1);
                    if (t == x.t0 && !role) {
                        if (nu > 0) ok = wait_warp(&q_empty, (nu - 1) & 1, limit, abort);
                        if (!ok) break;
                        if (lane == 0) {
                            s_unit[nu % UNITS] = x;
                            tc::mbar_arrive(&u_full[nu % UNITS]);
                            tc::mbar_arrive_expect_tx(&q_full, 2 * L::QB);
                            for (int i = 0; i < 2; ++i)
                                for (int s = 0; s < D / 64; ++s)
                                    tc::tma_load_3d(sq + i * L::QB + s * 16384, &mq, s * 64, x.h0, x.q0 + i * p.qpt, &q_full);
                        }
                        ++nq;
                    }
                    for (int kv = role; kv < (Q8 ? 2 : role + 1); ++kv) {
                        const uint32_t it = 2 * nt + kv;   // the item: even K, odd V, consumed in round ceil(it / 2)
                        if constexpr (Q8) {
                            const int slot = it % (L::RAW ? L::RAW : 1);
                            if (it >= L::RAW) ok = wait_warp(&raw_empty[slot], (it / (L::RAW ? L::RAW : 1) - 1) & 1, limit, abort);
                            if (!ok) break;
                            if (lane == 0) tc::mbar_arrive_expect_tx(&raw_full[slot], live * p.piece * D);
                            __syncwarp();
                            if (lane < live)
                                tc::tma_load_3d(codes + slot * L::RB + lane * p.piece * D, kv ? &mv : &mk, 0, x.hk, here, &raw_full[slot]);
                            __syncwarp();
                            ++issued;
                        } else {
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
                                tc::mbar_arrive_expect_tx(bar, live * p.piece * D * 2);
                                if (it == 0) tc::mbar_arrive(bar);        // round 0 has no values
                            }
                            __syncwarp();
                            const int s = lane / pieces, i = lane & (pieces - 1);     // channels, piece
                            if (s < D / 64 && i < live)
                                tc::tma_load_3d(dst + s * 16384 + i * p.piece * 128, kv ? &mv : &mk, s * 64, x.hk, here, bar);
                            __syncwarp();
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
                            ++issued;
                        }
                    }
                }
                have = more;
                x = y;
                ++nu;
            }
            if (!Q8 && ok && nt > 0 && !role) {    // the last round has no keys
                if (lane == 0) tc::mbar_arrive(&full[nt % ROUNDS]);
                ++issued;
            }
            if constexpr (!Q8) {
                if (lane == 0) s_issued[role] = issued;
                asm volatile("bar.sync 1, 64;" ::: "memory");      // the two loading warps
            }
            if (lane == 0) {
                // The copies issued so far land before the CTA leaves, whoever gave up: those of Q, of the
                // zeroed tiles and of codes complete their phases; a round's phase may want its
                // other half, whose arrival is made up for.
                bool d = role ? tc::drain_phase(&edge, edges) : tc::drain_phase(&q_full, nq);
                if constexpr (Q8) {
                    for (uint32_t i = issued > L::RAW ? issued - L::RAW : 0; i < issued; ++i)
                        d = tc::mbar_wait_bounded(&raw_full[i % (L::RAW ? L::RAW : 1)], (i / (L::RAW ? L::RAW : 1)) & 1, tc::WAIT_POLLS) && d;
                } else if (!role) {
                    const uint32_t nk = s_issued[0], nv = s_issued[1];       // keys are rounds 0 .. nk - 1, values 1 .. nv
                    const uint32_t rounds = nk == 0 && nv == 0 ? 0 : max(nk, nv + 1);
                    for (uint32_t r = rounds > ROUNDS ? rounds - ROUNDS : 0; r < rounds; ++r) {
                        if (r >= nk) tc::mbar_arrive(&full[r % ROUNDS]);
                        if (r >= nk && r == 0) tc::mbar_arrive(&full[0]);
                        if (r > nv) tc::mbar_arrive(&full[r % ROUNDS]);
                        d = tc::mbar_wait_bounded(&full[r % ROUNDS], (r / ROUNDS) & 1, tc::WAIT_POLLS) && d;
                    }
                }
                if (!ok || !d) atomicOr(&s_error, d ? tc::ERR_WAIT : tc::ERR_WAIT | tc::ERR_DRAIN);
            }
        } else if (warp < 15) {
            // ---------------- MMAs of tile t: the warp computes together, one lane issues ----------------
            // d = 128: the tiles take turns: A's products of a round, B's, A's of the next round, handed on by the
            // barriers `turn`.  One tile's S is so ready while the other's products run, and the two
            // softmaxes stay half a round apart.
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
            // a unit's tiles: all but the last one are whole.  Uniform over the warp.
            struct Tiles { int n, last, more; };
            auto tiles_of = [&](uint32_t i) {
                const Unit x = s_unit[i % UNITS];
                Tiles r;
                r.n = uniform(x.t1 - x.t0);
                r.last = uniform(r.n ? x.width(x.t1 - 1) : 0);
                r.more = uniform(x.more);
                return r;
            };
            auto width_of = [&](const Tiles& r, int i) { return i == r.n - 1 ? r.last : KT; };
            Tiles x = {0, 0, 0};
            uint32_t vs = L::SLOTS - 1, ks = 0;    // slots of this round's values and keys
            ok = wait_warp(&u_full[0], 0, limit, abort);
            if (ok) x = tiles_of(0);
            bool have = ok && x.n > 0;
            if (have) {
                ok = wait_warp(&q_full, 0, limit, abort) && wait_warp(&full[0], 0, limit, abort) && my_turn(0);
                tc::fence_after_sync();
                if (ok) {
                    qk(0, width_of(x, 0));
                    tc::mma_commit_elect(&s_full[t]);
                    hand_on();
                    tc::mma_commit_elect(&empty[0]);
                    if (x.n == 1) tc::mma_commit_elect(&q_empty);
                }
                rd = 1;
            }
#pragma unroll 1
            for (; have && ok; ++nu) {
                Tiles y = {0, 0, 0};
#pragma unroll 1
                for (int i = 0; i < x.n; ++i, ++np, ++rd) {
                    const bool last = i + 1 == x.n, more = !last || x.more;
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
                        if (i + 2 == x.n) tc::mma_commit_elect(&q_empty);
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
                        if (x.more) {
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
                    if (last ? more && y.n == 1 : !L::EARLY && i + 2 == x.n) tc::mma_commit_elect(&q_empty);
                }
                have = x.more;
                x = y;
            }
            // everything issued has finished before TMEM and shared memory are given back
            __syncwarp();
            tc::mma_commit_elect(&drained);
            if (lane == 0) {
                const bool d = tc::mbar_wait_bounded(&drained, 0, tc::WAIT_POLLS);
                if (!ok || !d) atomicOr(&s_error, d ? tc::ERR_WAIT : tc::ERR_WAIT | tc::ERR_DRAIN);
            }
            __syncwarp();
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int r = tid & 127;
        bool ok = true;
        if constexpr (!Q8) {
            // ---------------- output rows of both tiles ----------------
            for (uint32_t nu = 0; ok; ++nu) {
                ok = wait_warp(&u_full[nu % UNITS], (nu / UNITS) & 1, limit, abort);
                if (!ok) break;
                const Unit x = s_unit[nu % UNITS];
                if (x.t0 >= x.t1) break;
                for (int t = 0; t < 2; ++t) {
                    ok = wait_warp(&l_full[t], nu & 1, limit, abort) && wait_warp(&o_full[t], nu & 1, limit, abort);
                    if (!ok) break;
                    tc::fence_after_sync();
                    write_rows(x, t, r, s_l[t][r]);
                }
                if (!x.more) break;
            }
        } else {
            // ---------------- operands: row r of a tile of codes as bf16, times its power of two ----------------
            uint32_t it = 0;
            for (uint32_t nu = 0; ok; ++nu) {
                ok = wait_warp(&u_full[nu % UNITS], (nu / UNITS) & 1, limit, abort);
                if (!ok) break;
                const Unit x = s_unit[nu % UNITS];
                if (x.t0 >= x.t1) break;
                // The row's place is looked up two tiles ahead, the scale bytes of its key and value one.
                auto look_up = [&](int t) {
                    const int pos = t * KT + r;
                    return t < x.t1 && pos <= x.hi ? entry_of(p.a.cache, x.n, pos) : Entry{-1, 0};
                };
                uint32_t kb, vb;
                auto load_scales = [&](Entry e) {
                    const int at_row = row(p.a.cache, e);
                    kb = vb = 127u;
                    if (at_row >= 0) {
                        const size_t at = (size_t)at_row * p.a.cache.Hkv + x.hk;
                        kb = p.a.cache.k_scale[at];
                        vb = p.a.cache.v_scale[at];
                    }
                };
                load_scales(look_up(x.t0));
                Entry ahead = look_up(x.t0 + 1);
                for (int t = x.t0; t < x.t1 && ok; ++t) {
                    const float k_scale = scale_of(kb), v_scale = scale_of(vb);
                    const int seen = x.seen(t);
                    load_scales(ahead);
                    ahead = look_up(t + 2);
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv, ++it) {
                        const int from = it % (L::RAW ? L::RAW : 1), slot = it % L::SLOTS;
                        const float scale = kv ? v_scale : k_scale;
                        ok = wait_warp(&raw_full[from], (it / (L::RAW ? L::RAW : 1)) & 1, limit, abort);
                        if (ok && it >= L::SLOTS) {
                            const uint32_t rd = (it - L::SLOTS + 1) >> 1;     // the round that frees the slot
                            ok = wait_warp(&empty[rd % ROUNDS], (rd / ROUNDS) & 1, limit, abort);
                        }
                        if (!ok) break;
                        const uint8_t* src = codes + from * L::RB + r * D;
                        uint8_t* dst = ring + slot * L::SB + r * 128;
                        const int turn = D == 128 ? r & 7 : (r >> 1) & 3;      // the copies' swizzle of a row of codes
                        // few instructions, so that they stay in the cache nearest to the issue beside the softmax
#pragma unroll 2
                        for (int c = 0; c < D / 16; ++c) {
                            uint4 w = *reinterpret_cast<const uint4*>(src + ((c ^ turn) << 4));
                            if (r >= seen) w = make_uint4(0, 0, 0, 0);
                            const uint2 a = values4_bf16(w.x, scale), b = values4_bf16(w.y, scale);
                            const uint2 e = values4_bf16(w.z, scale), f = values4_bf16(w.w, scale);
                            uint8_t* to = dst + (c >> 2) * 16384;
                            const int at = 2 * (c & 3);
                            *reinterpret_cast<uint4*>(to + ((at ^ (r & 7)) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
                            *reinterpret_cast<uint4*>(to + (((at + 1) ^ (r & 7)) << 4)) = make_uint4(e.x, e.y, f.x, f.y);
                        }
                        tc::fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) {
                            uint64_t* round = &full[((it + 1) >> 1) % ROUNDS];
                            tc::mbar_arrive(&raw_empty[from]);
                            tc::mbar_arrive(round);
                            if (it == 0) tc::mbar_arrive(round);              // round 0 has no values
                        }
                    }
                }
                if (!x.more) break;
            }
            if (ok && it > 0 && lane == 0) tc::mbar_arrive(&full[(it >> 1) % ROUNDS]);        // the last round has no keys
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ---------------- softmax of tile t, one row per thread ----------------
        const int t = warp >> 2, r = tid & 127;
        const uint32_t ts = tm + t * 128 + ((uint32_t)(warp & 3) << 21);        // this warp's 32 lanes of S (and P)
        const uint32_t to = tm + 256 + t * D + ((uint32_t)(warp & 3) << 21);
        const uint32_t tp = tm + L::P0 + t * L::PSTEP + ((uint32_t)(warp & 3) << 21);
        uint32_t np = 0;
        bool ok = true;
        for (uint32_t nu = 0; ok; ++nu) {
            ok = wait_warp(&u_full[nu % UNITS], (nu / UNITS) & 1, limit, abort);
            if (!ok) break;
            const Unit x = s_unit[nu % UNITS];
            if (x.t0 >= x.t1) break;
            const int pos = min(x.hi, x.p0 + t * p.qpt + r / p.gp);          // position of this row's query
            float ref = -INFINITY, l0 = 0.f, l1 = 0.f;            // reference (scaled), sum in two parts
            const int pmin = min(x.hi, x.p0 + t * p.qpt);         // the tile's rows see everything up to here
            for (int i = x.t0; i < x.t1; ++i, ++np) {
                const int j0 = i * KT, width = x.width(i);
                ok = wait_warp(&s_full[t], np & 1, limit, abort);
                if (!ok) break;
                tc::fence_after_sync();
                float s[KT];
                const bool whole = j0 + KT - 1 <= pmin;           // (a narrower tile's other columns hold anything)
                const int b = pos - j0;                           // columns up to b are seen
                // masks 32 columns.  A warp's rows are few queries, so most chunks of an edge tile are
                // seen by all of them.
                auto mask = [&](int k) {
                    if (!whole) {
                        const int hi = min(31, b - 32 * k);
                        const uint32_t seen = hi >= 0 ? 0xffffffffu >> (31 - hi) : 0u;
                        if (!__all_sync(~0u, seen == 0xffffffffu)) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) s[32 * k + c] = (seen >> c) & 1u ? s[32 * k + c] : -INFINITY;
                        }
                    }
                };
                // The whole row first, and its maximum: the reference is settled before the exponentials, and nothing is done
                // twice (the first half's weights under the reference so far, the tile again where it was outgrown: 430 us).
                tc::tmem_ld64(ts, s);
                tc::tmem_ld64(ts + 64, s + 64);
                tc::tmem_ld_wait();
                after_wait(s, KT);
                if (L::EARLY) {
                    tc::fence_before_sync();
                    tc::mbar_arrive_warp(&s_free[t]);
                }
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) mask(k);
                }
                float mx[8];                       // eight chains
#pragma unroll
                for (int e = 0; e < 8; ++e) mx[e] = fmaxf(s[e], s[e + 8]);
#pragma unroll
                for (int c = 16; c < KT; c += 16) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) mx[e] = fmaxf(fmaxf(mx[e], s[c + e]), s[c + 8 + e]);
                }
                const float m = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * p.c;
                if (L::EARLY && np > 0) {              // P and O of the step before are the row's again
                    ok = wait_warp(&pv_done[t], (np - 1) & 1, limit, abort);
                    if (!ok) break;
                    tc::fence_after_sync();
                }
                const bool grow = m > ref + 8.f;                // (always from no reference)
                if (__any_sync(~0u, grow)) {
                    const float nref = grow ? m : ref;
                    const float f = ref == nref ? 1.f : exp2f(ref - nref);
                    l0 *= f;
                    l1 *= f;
                    ref = nref;
                    if (i > x.t0) {
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
                }
                const float base = ref == -INFINITY ? 0.f : -ref;   // nothing seen yet: every weight is exp2(-inf) = 0
                float l2 = 0.f, l3 = 0.f;
                // exp2(c s - ref), their sum in four parts, and P in bf16: weights are rounded to bf16 for the product (its
                // operands share a type, and V is bf16; a second part would double P V and the stores of P); l keeps float32
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 0 || width > 64) {
                        uint32_t w[32];
#pragma unroll
                        for (int j = 0; j < 64; j += 4) {
                            const int c = 64 * h + j;
                            float e0, e1, e2, e3;
                            fma2(e0, e1, s[c], s[c + 1], p.c, base);
                            fma2(e2, e3, s[c + 2], s[c + 3], p.c, base);
                            e0 = exp2f(e0);
                            e1 = exp2f(e1);
                            e2 = exp2f(e2);
                            e3 = exp2f(e3);
                            add2(l0, l1, e0, e1);
                            add2(l2, l3, e2, e3);
                            w[j / 2] = pack2(e0, e1);
                            w[j / 2 + 1] = pack2(e2, e3);
                        }
                        tc::tmem_st16u(tp + h * 32, w);
                        tc::tmem_st16u(tp + h * 32 + 16, w + 16);
                        tc::tmem_st_wait();
                    }
                    tc::fence_before_sync();
                    tc::mbar_arrive_warp(&p_full[t][h]);
                }
                l0 += l2;
                l1 += l3;
            }
            if (!ok) break;
            const float l = l0 + l1;
            const int q = x.q0 + t * p.qpt + r / p.gp;
            if (x.whole) {
                if (p.a.lse && q < x.q1) p.a.lse[(size_t)q * p.a.Hq + x.h0 + r % p.gp] = 0.6931471805599453f * ref + logf(l);
            } else {
                float* ml = p.parts + (size_t)gridDim.x * 512 * D + (blockIdx.x * 2 + (x.t0 == 0)) * 512 + t * 128 + r;
                ml[0] = ref;
                ml[256] = l;
            }
            if constexpr (Q8) {
                ok = wait_warp(&o_full[t], nu & 1, limit, abort);
                if (!ok) break;
                tc::fence_after_sync();
                write_rows(x, t, r, l);
            } else {
                if (nu > 0) ok = wait_warp(&o_empty[t], (nu - 1) & 1, limit, abort);   // the last unit's l has been read
                if (!ok) break;
                s_l[t][r] = l;
                tc::mbar_arrive_warp(&l_full[t]);
            }
            __syncwarp();
            if (!x.more) break;
        }
    }
    __syncthreads();
    if (warp == 13) tc::tmem_dealloc(tm, 512);
    if (tid == 0) p.errors[blockIdx.x] = s_error;
}

// Joins the parts of the units that were split, 8 channels of a row to a thread; the first CTA also gathers the error reports.
// Neighbouring threads have neighbouring rows, and the parts lie four channels of all rows after four channels of all rows,
// so that the parts' loads and stores are dense.  (A row to a warp, rows as they are: 4096 tokens, 32 / 8 heads of 128, 131 us in
// all, this 128; one token after 100000, one key head, 68 and 44, with two parts at once and not four 65.)
constexpr int JOIN_THREADS = 512;

template <int D>
__global__ void __launch_bounds__(JOIN_THREADS, 2)
join_rows_kernel(const __grid_constant__ PfParams p, int ctas) {
    tc::wait_prerequisites();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 32) {
        int e = 0;
        for (int i = threadIdx.x; i < ctas; i += 32) e |= p.errors[i];
        e = __reduce_or_sync(~0u, (unsigned)e);
        if (threadIdx.x == 0) {
            *p.error = e;
            if (e && p.a.error) atomicOr(p.a.error, e);
        }
    }
    if ((int)blockIdx.x + 1 >= ctas) return;
    const Split d = p.split[blockIdx.x + 1];
    if (d.q0 < 0) return;
    constexpr int B = 4;               // parts at once
    const int parts = d.last - d.first + 1, rows = (d.q1 - d.q0) * p.gp, items = rows * (D / 8);       // the unit's first rows have queries
    // Many parts and few items: the unit's CTAs share the items, and threads of a CTA the parts of an item (one token after 100000,
    // one key head, 152 parts: 44 us in all without, 26 with).
    int per = JOIN_THREADS, slices = 1;
    if (parts > B) {
        per = (items + gridDim.y - 1) / gridDim.y;
        while (2 * slices * per <= JOIN_THREADS && slices * B < parts) slices *= 2;
    }
    const int slice = threadIdx.x / per, item = blockIdx.y * per + threadIdx.x % per;
    const bool on = slice < slices && item < items;
    const int r = on ? item % rows : 0, c0 = on ? item / rows * 8 : 0;
    // (numbers of floats stay below 2^24)
    const uint32_t at_m = ctas * 512 * D + r, at_o = c0 * 256 + r * 4;
    float m = -INFINITY, l = 0.f, acc[8] = {};
    for (int i0 = on ? slice * B : parts; i0 < parts; i0 += slices * B) {
        float pm[B], pl[B], n = m;
        float4 o[B][2];
#pragma unroll
        for (int u = 0; u < B; ++u) {
            pm[u] = -INFINITY;
            pl[u] = 0.f;
            o[u][0] = o[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int i = i0 + u;
            if (i < parts) {
                // the first begins its unit (second half of its CTA's room), the others continue it
                const uint32_t room = (d.first + i) * 2 + (i == 0);
                pm[u] = p.parts[at_m + room * 512];
                pl[u] = p.parts[at_m + room * 512 + 256];
                o[u][0] = *reinterpret_cast<const float4*>(p.parts + (at_o + room * 256 * D));
                o[u][1] = *reinterpret_cast<const float4*>(p.parts + (at_o + room * 256 * D + 1024));
            }
        }
#pragma unroll
        for (int u = 0; u < B; ++u) n = fmaxf(n, pm[u]);
        const float base = n == -INFINITY ? 0.f : n, f = exp2f(m - base);
        l *= f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= f;
#pragma unroll
        for (int u = 0; u < B; ++u) {
            const float g = exp2f(pm[u] - base);
            const float x[8] = {o[u][0].x, o[u][0].y, o[u][0].z, o[u][0].w, o[u][1].x, o[u][1].y, o[u][1].z, o[u][1].w};
            l += g * pl[u];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += g * x[e];
        }
        m = n;
    }
    if (slices > 1) {                  // the same in all threads
        __shared__ float s_m[JOIN_THREADS], s_l[JOIN_THREADS], s_o[8][JOIN_THREADS];
        s_m[threadIdx.x] = m;
        s_l[threadIdx.x] = l;
#pragma unroll
        for (int e = 0; e < 8; ++e) s_o[e][threadIdx.x] = acc[e];
        __syncthreads();
        if (slice == 0) {
            for (int i = 1; i < slices; ++i) m = fmaxf(m, s_m[threadIdx.x + i * per]);
            const float base = m == -INFINITY ? 0.f : m, f = exp2f(s_m[threadIdx.x] - base);
            l *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] *= f;
            for (int i = 1; i < slices; ++i) {
                const int at = threadIdx.x + i * per;
                const float g = exp2f(s_m[at] - base);
                l += g * s_l[at];
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += g * s_o[e][at];
            }
        }
    }
    if (!on || slice > 0) return;
    const size_t row = (size_t)(d.q0 + r / p.gp) * p.a.Hq + d.h0 + r % p.gp;
    const float inv = 1.f / l;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = l == 0.f ? 0u : pack2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p.a.o) + row * D + c0) = make_uint4(w[0], w[1], w[2], w[3]);
    if (p.a.lse && c0 == 0) p.a.lse[row] = 0.6931471805599453f * m + logf(l);
}

// ---------------------------------------------------------------------------

// workspace: the error word; the CTAs' reports; the split units; their parts
constexpr size_t ERRORS_AT = 256, SPLIT_AT = 1024, PARTS_AT = SPLIT_AT + ((sizeof(Split) * PF_CTAS + 255) & ~(size_t)255);
static_assert(ERRORS_AT + PF_CTAS * 4 <= SPLIT_AT, "the reports' room");

static int ctas_of(const kda_paged_prefill_args& a) {
    // never more than the list can have ranges
    const long tiles = ((long)a.cache.max_pages * a.cache.page_size + KT - 1) / KT + 1 + OVERHEAD;
    const long units = ((long)a.T_total / 16 + a.cache.num_seqs) * a.Hq;
    if (units >= PF_CTAS || tiles >= (1L << 24)) return PF_CTAS;
    return (int)std::max(1L, std::min((long)PF_CTAS, units * tiles / RANGE + 1));
}

size_t prefill_workspace_size(const kda_paged_prefill_args& a) {
    return PARTS_AT + (size_t)ctas_of(a) * 512 * (a.cache.d + 2) * 4;
}

template <int D, bool Q8>
static cudaError_t prefill_d(const kda_paged_prefill_args& a, cudaStream_t s) {
    PfParams p;
    p.a = a;
    const kda_paged_cache& c = a.cache;
    const int G = a.Hq / c.Hkv;
    p.gp = std::min(G & -G, 16);
    p.subs = G / p.gp;
    p.qpt = 128 / p.gp;
    for (p.per_log = 0; 1 << p.per_log < 2 * p.qpt;) ++p.per_log;
    p.piece = std::min(c.page_size & -c.page_size, KT);
    // a zero scale keeps exp2(fma(-inf, c, ...)) at 0 for masked scores
    p.c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-37f);
    p.neg = a.scale < 0.f;
    p.wide = (reinterpret_cast<uintptr_t>(a.o) & 31u) == 0;
    p.wait_limit = wait_limit();
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.error = reinterpret_cast<int*>(ws);
    p.errors = reinterpret_cast<int*>(ws + ERRORS_AT);
    p.split = reinterpret_cast<Split*>(ws + SPLIT_AT);
    p.parts = reinterpret_cast<float*>(ws + PARTS_AT);
    CUtensorMap mq, mk, mv;
    const uint64_t rows = (uint64_t)c.num_pages * c.page_size;
    cudaError_t e = make_map_heads(&mq, a.q, D, a.Hq, a.T_total, a.q_stride, p.gp, p.qpt);
    if (e == cudaSuccess) e = make_map_pages(&mk, c.k, Q8, D, c.Hkv, rows, p.piece);
    if (e == cudaSuccess) e = make_map_pages(&mv, c.v, Q8, D, c.Hkv, rows, p.piece);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(prefill_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, PF<D, Q8>::SMEM);
    if (e != cudaSuccess) return e;
    const int ctas = ctas_of(a);
    prefill_kernel<D, Q8><<<ctas, PF_THREADS, PF<D, Q8>::SMEM, s>>>(p, mq, mk, mv);
    count_launches(1);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::max(1, ctas - 1), 256 * (D / 8) / JOIN_THREADS);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, join_rows_kernel<D>, p, ctas);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

cudaError_t launch_prefill(const kda_paged_prefill_args& a, cudaStream_t s) {
    if (a.cache.dtype == KDA_E4M3) return a.cache.d == 128 ? prefill_d<128, true>(a, s) : prefill_d<64, true>(a, s);
    return a.cache.d == 128 ? prefill_d<128, false>(a, s) : prefill_d<64, false>(a, s);
}

}  // namespace paged
}  // namespace kda
