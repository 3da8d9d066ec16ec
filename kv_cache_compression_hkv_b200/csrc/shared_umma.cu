// shared_umma.cu -- shared-prefix attention of many query rows on the
// 5th-generation tensor cores (tcgen05), bf16.
//
// A block takes NT tiles of 128 query rows that share their keys and walks a
// list of 64-key tiles, prefix first, then own keys up to the rows' causal
// limit.  Per (row tile X, key tile j):
//   S = Q_X K_j^T   (M 128, N 64, fp32 in TMEM)
//   P = 2^(c S - m) as the sum of two bf16 in TMEM: its first bits, and of what
//       they leave
//   O_X += P V_j    (two products; A from TMEM, V as the MN-major operand, fp32 in TMEM)
// so that outputs are off by their own rounding alone.  (With P's rounding alone
// their error was 2.1e-3 to 2.3e-3 relative, instead of 1.7e-3, and not the same in
// every split of a call; the tensor cores had a third less to do.)
// Rows: thread = query row = TMEM lane.  m is a reference maximum that is
// raised (and O rescaled in TMEM) only when a logit passes it by more than
// 16, so weights stay below 2^16 and bf16's relative rounding is unaffected;
// the sum l is of the unrounded weights in fp32.
// Roles: 4 NT softmax warps; a copy warp (TMA into a ring of pairs K0, V0 K1,
// V1 K2, ... as they are used together); an MMA warp a row tile, one lane of
// which waits and issues.
// S of tile j + 1 is issued as soon as the rows hold S of tile j in registers,
// so a softmax warp finds its next logits ready.  (With P over S's own place S of
// tile j + 2 had to wait for the product of tile j behind the other row tile's.)
//
// d = 128: 16004 rows of 16 heads over 2834 keys on average 457 us (0.81 PFLOP/s,
// 1.22 with the second product of the weights: those products are most of it, the
// rest the softmax's exponentials and the hand-over; 367 us with one product),
// 512 heads of 256 rows over 384 keys 63 us with the weights, 512 heads of 49 rows
// over 49 to 462 and 128 42 us: there each block's beginning and end, two blocks an
// SM to hide them.
#include <math.h>

#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"
#include "shared.cuh"
#include "umma.cuh"

namespace hkv {
namespace shared {

namespace {

using ptx::mbar_expect_tx;
using ptx::mbar_init;
using ptx::mbar_wait;
using ptx::smem_u32;

constexpr int QT = 128;
constexpr int UK = 64;  // keys of a tile
constexpr float RAISE = 16.f;
constexpr uint64_t WAIT_NS = 2000000000ull;

template <int D, int NT> struct Shape {
    static constexpr int NS = NT == 2 ? (D == 128 ? 4 : 6) : (D == 128 ? 2 : 3);  // (V, K) pairs in the ring
    static constexpr int ROWS = 128 * NT;
    static constexpr int THREADS = ROWS + 32 + 32 * NT;
    static constexpr int COPY_WARP = 4 * NT, MMA_WARP = 4 * NT + 1;  // MMA_WARP + x issues for row tile x
    static constexpr uint32_t O_COL = 128 * NT;  // before it, a row tile: 64 columns of S, two times 32 of P
    static constexpr uint32_t TMEM = NT == 2 ? 512 : 256;
    static constexpr int Q_BYTES = QT * D * 2, KV_BYTES = UK * D * 2;
    enum { B_Q, B_FULL, B_FREE = B_FULL + NS, B_S = B_FREE + NS, B_SF = B_S + NT, B_P = B_SF + NT, B_PV = B_P + 2 * NT,
           B_T = B_PV + 2 * NT, B_TF = B_T + NT, B_COUNT = B_TF + NT };
    static constexpr int TAIL = B_COUNT * 8 + 16 + 16 + (QT + 4) * 4 + ROWS * 4;
    static constexpr int SMEM = 1024 + NT * Q_BYTES + NS * 2 * KV_BYTES + TAIL;
};

}  // namespace

// sum over 128 columns from taddr (a thread's lane) of 2^(c S + nl), for the
// columns [from, to) (all of them: ALL).  Columns past the last query hold no
// zeros where a key is infinite.
template <bool ALL>
__device__ __forceinline__ float column_weights(uint32_t taddr, const float* nl, float c, int from, int to) {
    float total = 0.f;
    const unsigned span = max(0, to - from);
#pragma unroll
    for (int c0 = 0; c0 < QT; c0 += 32) {
        if (!ALL && c0 >= to) break;
        uint32_t o[32];
        tc::ld32(taddr + c0, o);
        tc::ld_wait();
        float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
            const float4 e = *reinterpret_cast<const float4*>(nl + c0 + u);
#pragma unroll
            for (int v = 0; v < 4; v += 2) {
                const float2 y = tc::fma2(make_float2(__uint_as_float(o[u + v]), __uint_as_float(o[u + v + 1])), make_float2(c, c),
                                          v == 0 ? make_float2(e.x, e.y) : make_float2(e.z, e.w));
                float2 p = make_float2(tc::ex2(y.x), tc::ex2(y.y));
                if (!ALL) {
                    p.x = (unsigned)(c0 + u + v - from) < span ? p.x : 0.f;
                    p.y = (unsigned)(c0 + u + v + 1 - from) < span ? p.y : 0.f;
                }
                acc[v >> 1] = tc::add2(acc[v >> 1], p);
            }
        }
        acc[0] = tc::add2(acc[0], acc[1]);
        total += acc[0].x + acc[0].y;
    }
    return total;
}

// MODE 0: every key of a row tile of one (sequence, KV head), prefix, then own;
//         final results.  With a.sum_tiles (and one row tile a block) the block
//         also sums the weights its own keys get from its rows: S once more,
//         transposed (128 keys on the M side, the rows as N), into the places of
//         S and P, so that a thread sums 2^(x - lse) of its key.  A block with
//         all rows of its (sequence, KV head) adds them to the accumulated
//         weights; several leave theirs for add_sums_kernel, which adds them in
//         their order.
// MODE 2: the same keys cut in `splits` pieces of the tile list; partial
//         results (slot = piece).
// MODE 1: rows of all sequences of a prefix over the prefix's keys, cut in
//         a.np ranges; partial results (slot = range).
template <int D, int NT, int MODE>
__global__ void __launch_bounds__(Shape<D, NT>::THREADS, NT == 2 ? 1 : 2)
    attend_umma_kernel(const __grid_constant__ View a, const __grid_constant__ CUtensorMap km,
                       const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap pkm,
                       const __grid_constant__ CUtensorMap pvm, int row_tiles, int splits) {
    using C = Shape<D, NT>;
    extern __shared__ unsigned char raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    unsigned char* q_s = base;
    unsigned char* ring = q_s + NT * C::Q_BYTES;  // pairs: V, then K
    float* nl_s = reinterpret_cast<float*>(ring + C::NS * 2 * C::KV_BYTES);  // [ROWS] -log2 of the rows' sums
    uint64_t* bars = reinterpret_cast<uint64_t*>(nl_s + C::ROWS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::B_COUNT);
    int* res = reinterpret_cast<int*>(tmem_slot + 4);
    int* list = res + 4;
    constexpr int NSUB = D / 64;

    const int tid = threadIdx.x, warp = tc::uniform(tid >> 5), lane = tid & 31;
    const int rps = a.rep * a.T;
    const int64_t R = (int64_t)a.S * a.H * a.T;

    ptx::grid_dep_wait();
    ptx::grid_dep_trigger();
    // what this block works on
    int hk, s = 0, g, first, rows, piece, p_tiles, t0, t1, p_len, n_own = 0, p_lo = 0;
    // this thread's row (warps of the rows): sequence, row within (sequence, KV head), query head, query
    int sq = 0, ri = 0, h = 0, t = 0;
    bool live = false;
    constexpr int CH = D / 8, RPI = 32 / CH;  // 16-byte pieces of a row; rows a warp covers at once
    // Where piece c of row r of a row tile lies in the swizzled K-major tile.
    auto q_off = [](int r, int c) { return (c / 8) * (QT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4); };
    // Starts the copies of the warp's rows of Q into the swizzled tile, whole
    // rows at a time, so that they run while the lengths are looked up.  Threads
    // past the last row take that row (zeros would give NaN with a key that is
    // infinite, in the sums over all of a tile's columns).
    auto load_q = [&]() {
        if (warp >= 4 * NT) return;
        live = tid < rows;
        const int f = first + min(tid, rows - 1);
        if constexpr (MODE != 1) {
            sq = s;
            ri = f;
        } else {
            sq = list[f / rps - first / rps];
            ri = f % rps;
        }
        t = query_of(a, ri);
        h = hk * a.rep + ri - t * a.rep;
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
        const int64_t at = sq * a.qs[0] + h * a.qs[1] + t * a.qs[2];
        const uint32_t tile = smem_u32(q_s + (warp >> 2) * C::Q_BYTES);
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            const int r = e * RPI + lane / CH, c = lane % CH;
            const int64_t o = __shfl_sync(FULL_MASK, at, r);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tile + q_off((warp & 3) * 32 + r, c)), "l"(q + o + c * 8)
                         : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (MODE != 1) {
        // longest row tiles (the last queries) first
        const int b = blockIdx.x, per = a.S * a.Hk * splits;
        const int tile = row_tiles - 1 - b / per;
        piece = b % per % splits;
        const int sh = b % per / splits;
        s = sh / a.Hk;
        hk = sh % a.Hk;
        first = tile * C::ROWS;
        rows = min(C::ROWS, rps - first);
        load_q();
        g = prefix_of(a, s);
        p_len = prefix_len(a, g);
        n_own = own_len(a, s, hk);
        p_tiles = (p_len + UK - 1) / UK;
        const int all = p_tiles + (n_own + UK - 1) / UK;
        const int per_piece = (all + splits - 1) / splits;
        t0 = min(all, piece * per_piece);
        t1 = min(all, t0 + per_piece);
        if (MODE == 2 && t0 >= t1) {  // the joining kernel knows
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            return;
        }
    } else {
        const int b = blockIdx.x;
        piece = b % a.np;
        hk = b / a.np % a.Hk;
        if (!find_prefix_tile(a, b / a.np / a.Hk, C::ROWS, g, first, rows, reinterpret_cast<int*>(ring), res, list))
            return;
        load_q();
        p_len = prefix_len(a, g);
        int lo, hi;
        split_range(p_len, a.np, piece, lo, hi);
        if (lo >= hi) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            return;
        }
        p_lo = lo;
        p_len = hi;
        ptx::fence_proxy_async();  // (the ring held the counts just now)
        t0 = 0;
        t1 = p_tiles = (hi - lo + UK - 1) / UK;
    }
    // key tiles of each row tile within [t0, t1)
    int nx[NT], n = 0;
#pragma unroll
    for (int x = 0; x < NT; ++x) {
        const int last = min(rows, (x + 1) * QT) - 1;
        nx[x] = 0;
        if (last >= x * QT) {
            const int vis = MODE != 1 ? p_tiles + (own_limit(a, n_own, first + last) + UK - 1) / UK : t1;
            nx[x] = max(0, min(vis, t1) - t0);
        }
        n = max(n, nx[x]);
    }

    if (tid == 0) {
        for (int i = 0; i < C::B_COUNT; ++i)
            mbar_init(bars + i, i == C::B_Q ? 4 * NT : i >= C::B_FREE && i < C::B_S ? NT : ((i >= C::B_SF && i < C::B_PV) || i >= C::B_TF) ? 4 : 1);
        ptx::fence_mbar_init();
    }
    if (warp == 0) tc::alloc(tmem_slot, C::TMEM);
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    bool fail = false;

    // own keys that some row sees, and their blocks of 128, for the sums
    const int seen = MODE == 0 && NT == 1 && a.sum_tiles ? min(n_own, own_limit(a, n_own, first + rows - 1)) : 0;
    const int n2 = (seen + QT - 1) / QT;

    // list tile t0 + j: where its keys start, and how many of 64 are keys
    auto tile_at = [&](int j, bool& pre, int& k0, int& valid) {
        const int t = t0 + j;
        pre = t < p_tiles;
        k0 = pre ? p_lo + t * UK : (t - p_tiles) * UK;
        valid = min(UK, (pre ? p_len : n_own) - k0);
    };
    if (warp == C::COPY_WARP) {
        if (lane == 0) {
            // pair i: V of tile i - 1 and K of tile i
            int issued = 0;
            for (int i = 0; i <= n && n > 0; ++i) {
                const int slot = i % C::NS, use = i / C::NS;
                if (use > 0 && !mbar_wait(bars + C::B_FREE + slot, (use - 1) & 1, WAIT_NS)) { fail = true; break; }
                unsigned char* dst = ring + slot * 2 * C::KV_BYTES;
                mbar_expect_tx(bars + C::B_FULL + slot, (i > 0 && i < n ? 2 : 1) * C::KV_BYTES);
                bool pre;
                int k0, valid;
                if (i < n) {
                    tile_at(i, pre, k0, valid);
                    for (int sub = 0; sub < NSUB; ++sub)
                        tc::tma_load_4d(dst + C::KV_BYTES + sub * UK * 128, pre ? &pkm : &km, bars + C::B_FULL + slot,
                                        sub * 64, k0, hk, pre ? g : s);
                }
                if (i > 0) {
                    tile_at(i - 1, pre, k0, valid);
                    for (int sub = 0; sub < NSUB; ++sub)
                        tc::tma_load_4d(dst + sub * UK * 128, pre ? &pvm : &vm, bars + C::B_FULL + slot, sub * 64, k0, hk,
                                        pre ? g : s);
                }
                issued = i + 1;
            }
            for (int kb = 0; kb < n2 && !fail; ++kb) {
                const int i = n + 1 + kb, slot = i % C::NS, use = i / C::NS;
                if (use > 0 && !mbar_wait(bars + C::B_FREE + slot, (use - 1) & 1, WAIT_NS)) { fail = true; break; }
                unsigned char* dst = ring + slot * 2 * C::KV_BYTES;
                mbar_expect_tx(bars + C::B_FULL + slot, 2 * C::KV_BYTES);
                for (int sub = 0; sub < NSUB; ++sub)
                    for (int e = 0; e < 2; ++e)
                        tc::tma_load_4d(dst + sub * QT * 128 + e * UK * 128, &km, bars + C::B_FULL + slot, sub * 64,
                                        kb * QT + e * UK, hk, s);
                issued = i + 1;
            }
            if (fail)  // the block's own copies land before its shared memory goes
                for (int i = max(0, issued - C::NS); i < issued; ++i)
                    mbar_wait(bars + C::B_FULL + i % C::NS, (i / C::NS) & 1, WAIT_NS);
        }
    } else if (warp >= C::MMA_WARP) {
        // All that an MMA's operands come from is made uniform first (with
        // addresses in per-thread registers an issue took 84 cycles, up to
        // three times the product), and one lane does the waiting too (with
        // votes of the warp around each wait the products were 1260 cycles of
        // the 2150 that a key tile of two row tiles took).
        constexpr uint32_t IS = tc::idesc_bf16(UK, false), IO = tc::idesc_bf16(D, true);
        const uint32_t tm = tc::uniform(tmem);
        const int nn = tc::uniform(n);
        const int x = NT == 1 ? 0 : warp - C::MMA_WARP;
        const int nu = tc::uniform(NT == 1 || x == 0 ? nx[0] : nx[NT - 1]);
        const uint32_t ring_u = tc::uniform(smem_u32(ring)), q_u = tc::uniform(smem_u32(q_s));
        const uint64_t q_desc = tc::sw128_desc(q_u + x * C::Q_BYTES, 16, 1024), k_desc = tc::sw128_desc(ring_u + C::KV_BYTES, 16, 1024),
                       v_desc = tc::sw128_desc(ring_u, UK * 128, 1024);
        if (tc::elect()) {
            // Pair i: S of tile i once it has landed and the rows have read S of
            // tile i - 1, then P V of tile i - 1 once its weights are written.
            // (One warp for both row tiles kept S of one waiting for the weights
            // of the other.)
            const uint32_t t_s = tm + x * 128, t_o = tm + C::O_COL + x * D;
            int s_done = -1, pv_done = -1, freed = 0, sums = 0;
            auto full = [&](int i) { return mbar_wait(bars + C::B_FULL + i % C::NS, (i / C::NS) & 1, WAIT_NS); };
            auto give_back = [&](int i) {
                tc::commit(bars + C::B_FREE + i % C::NS);
                ++freed;
            };
            if (!mbar_wait(bars + C::B_Q, 0, WAIT_NS)) fail = true;
            for (int i = 0; i <= nn && nn > 0 && !fail; ++i) {
                if (!full(i)) { fail = true; break; }
                const uint32_t pair = (i % C::NS) * (2 * C::KV_BYTES / 16);
                if (i < nu) {
                    if (i > 0 && !mbar_wait(bars + C::B_SF + x, (i - 1) & 1, WAIT_NS)) { fail = true; break; }
                    tc::fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)  // descriptors count 16-byte units
                        tc::mma_ss(t_s, q_desc + (kk / 4) * (QT * 8) + (kk % 4) * 2,
                                   k_desc + pair + (kk / 4) * (UK * 8) + (kk % 4) * 2, IS, kk > 0);
                    tc::commit(bars + C::B_S + x);
                    s_done = i;
                }
                if (i > 0 && i <= nu) {
                    const int j = i - 1;
                    if (!mbar_wait(bars + C::B_P + 2 * x + (j & 1), (j >> 1) & 1, WAIT_NS)) { fail = true; break; }
                    tc::fence_after();
#pragma unroll
                    for (int kk = 0; kk < UK / 16; ++kk)
                        tc::mma_ts(t_o, t_s + UK + kk * 8, v_desc + pair + kk * 128, IO, (j > 0 || kk > 0));
#pragma unroll
                    for (int kk = 0; kk < UK / 16; ++kk)
                        tc::mma_ts(t_o, t_s + UK + 32 + kk * 8, v_desc + pair + kk * 128, IO, 1);
                    tc::commit(bars + C::B_PV + 2 * x + (j & 1));
                    pv_done = j;
                }
                give_back(i);
            }
            if (n2 > 0 && !fail) {
                constexpr uint32_t IT = tc::idesc_bf16(QT, false);
                const uint64_t t_desc = tc::sw128_desc(ring_u, 16, 1024);
                // the places of S and P are free once the last product is done
                if (pv_done >= 0 && !mbar_wait(bars + C::B_PV + 2 * x + (pv_done & 1), (pv_done >> 1) & 1, WAIT_NS)) fail = true;
                for (int kb = 0; kb < n2 && !fail; ++kb) {
                    const int i = nn + 1 + kb;
                    if (!full(i) || (kb > 0 && !mbar_wait(bars + C::B_TF + x, (kb - 1) & 1, WAIT_NS))) { fail = true; break; }
                    tc::fence_after();
                    const uint32_t pair = (i % C::NS) * (2 * C::KV_BYTES / 16);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk)
                        tc::mma_ss(t_s, t_desc + pair + (kk / 4) * (QT * 8) + (kk % 4) * 2, q_desc + (kk / 4) * (QT * 8) + (kk % 4) * 2,
                                   IT, kk > 0);
                    tc::commit(bars + C::B_T + x);
                    give_back(i);
                    ++sums;
                }
            }
            // The tensor cores finish what was issued before TMEM is freed, and
            // the last commits' arrivals land before the shared memory goes.
            if (s_done > pv_done) mbar_wait(bars + C::B_S + x, s_done & 1, WAIT_NS);
            if (pv_done >= 0) mbar_wait(bars + C::B_PV + 2 * x + (pv_done & 1), (pv_done >> 1) & 1, WAIT_NS);
            if (sums > 0) mbar_wait(bars + C::B_T + x, (sums - 1) & 1, WAIT_NS);
            if (freed > 0) mbar_wait(bars + C::B_FREE + (freed - 1) % C::NS, ((freed - 1) / C::NS) & 1, WAIT_NS);
        }
        __syncwarp();
    } else {
        // --- rows ----------------------------------------------------------
        const int x = warp >> 2;  // row tile
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (a.qscale < 0.f) {
            // negated where the scale is negative (exact), so that the
            // reference maximum is of the scaled logits: every lane the pieces it copied
            for (int e = 0; e < CH; ++e) {
                uint4* w = reinterpret_cast<uint4*>(q_s + x * C::Q_BYTES + q_off((warp & 3) * 32 + e * RPI + lane / CH, lane % CH));
                uint4 y = *w;
                y.x ^= 0x80008000u; y.y ^= 0x80008000u; y.z ^= 0x80008000u; y.w ^= 0x80008000u;
                *w = y;
            }
        }
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::arrive(bars + C::B_Q);
        const float c = fabsf(a.qscale);
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = t_lane + x * 128, t_o = t_lane + C::O_COL + x * D;
        // own keys this row sees; what threads past the last row make is not used
        const int lim = MODE != 1 ? (live ? own_limit(a, n_own, ri) : 0x7fffffff) : 0;
        const int lim_warp = __shfl_sync(FULL_MASK, lim, 0);  // the least of the warp's
        const int nt = NT == 2 ? (x == 0 ? nx[0] : nx[NT - 1]) : nx[0];
        // reference maximum (before c), the logit above which it is raised, what a
        // tile's logits are lowered by, and the sum
        float ref = -INFINITY, above = -INFINITY, mb = 0.f, l = 0.f;
        // Some row's c ref is so large that c S - c ref would be off by its
        // rounding: the warp comes to the raise with every tile, and S - ref is formed.
        bool far = false;
        const bool idle = !__any_sync(FULL_MASK, live);  // no row of the warp is one: it only keeps the barriers' counts
        // every branch around the warp-wide TMEM accesses is taken by the whole warp
        for (int j = 0; j < nt; ++j) {
            if (__any_sync(FULL_MASK, !mbar_wait(bars + C::B_S + x, j & 1, WAIT_NS))) { fail = true; break; }
            tc::fence_after();
            if (idle) {
                if (lane == 0) {
                    tc::arrive(bars + C::B_SF + x);
                    tc::arrive(bars + C::B_P + 2 * x + (j & 1));
                }
                continue;
            }
            uint32_t sr[2][32];
            tc::ld32(t_s, sr[0]);
            tc::ld32(t_s + 32, sr[1]);
            bool pre;
            int k0, valid;
            tile_at(j, pre, k0, valid);
            tc::ld_wait();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::arrive(bars + C::B_SF + x);
            if (valid < UK) {
                // V's rows past the last key hold whatever the memory held, and
                // 0 x NaN must not be formed: they are cleared before the
                // weights are announced (by each row tile's warps: the same zeros)
                if (__any_sync(FULL_MASK, !mbar_wait(bars + C::B_FULL + (j + 1) % C::NS, ((j + 1) / C::NS) & 1, WAIT_NS))) {
                    fail = true;
                    break;
                }
                // (warps past the last row do not take part: the first warp of a row tile with keys has one)
                const int busy = min(4, (rows - x * QT + 31) / 32);
                unsigned char* vt = ring + ((j + 1) % C::NS) * 2 * C::KV_BYTES;
                for (int e = tid & 127; e < (UK - valid) * 8 * NSUB; e += 32 * busy) {
                    const int sub = e / ((UK - valid) * 8), w = e % ((UK - valid) * 8);
                    *reinterpret_cast<uint4*>(vt + sub * UK * 128 + valid * 128 + w * 16) = make_uint4(0, 0, 0, 0);
                }
                ptx::fence_proxy_async();
            }
            if (valid < UK || (!pre && k0 + UK > lim_warp)) {
                const int end = pre ? valid : min(valid, lim - k0);
#pragma unroll
                for (int u = 0; u < UK; ++u)
                    if (u >= end) sr[u >> 5][u & 31] = 0xff800000u;  // -inf
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int u = 0; u < UK; ++u) mx[u & 3] = fmaxf(mx[u & 3], __uint_as_float(sr[u >> 5][u & 31]));
            const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            if (__any_sync(FULL_MASK, most * c > above)) {
                const float rn = fmaxf(ref, most), m = rn * c;
                const float alpha = rn == -INFINITY ? 1.f : exp2f((ref - rn) * c);
                if (j > 0) {
                    const int jp = j - 1;
                    if (__any_sync(FULL_MASK, !mbar_wait(bars + C::B_PV + 2 * x + (jp & 1), (jp >> 1) & 1, WAIT_NS))) {
                        fail = true;
                        break;
                    }
                    tc::fence_after();
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tc::ld32(t_o + c0, o);
                        tc::ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tc::st32(t_o + c0, o);
                    }
                    tc::st_wait();
                }
                l *= alpha;
                ref = rn;
                far = __any_sync(FULL_MASK, far || (fabsf(m) > BIG && m != -INFINITY));
                mb = m == -INFINITY || far ? 0.f : m;
                above = far ? -INFINITY : m + RAISE;
                if (far) {
                    const float r = rn == -INFINITY ? 0.f : rn;
#pragma unroll
                    for (int u = 0; u < UK; ++u) sr[u >> 5][u & 31] = __float_as_uint(__uint_as_float(sr[u >> 5][u & 31]) - r);
                }
            }
            uint32_t w[32];
            float2 ls[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) ls[u] = make_float2(0.f, 0.f);
#pragma unroll
            for (int u = 0; u < 32; ++u) {
                const float2 y = tc::fma2(make_float2(__uint_as_float(sr[u >> 4][2 * u & 31]), __uint_as_float(sr[u >> 4][(2 * u & 31) + 1])),
                                          make_float2(c, c), make_float2(-mb, -mb));
                const float2 p = make_float2(tc::ex2(y.x), tc::ex2(y.y));
                ls[u & 3] = tc::add2(ls[u & 3], p);
                split_weights(p.x, p.y, w[u], sr[0][u]);  // (over S's registers: logits 0 .. 2 u + 1 have been used)
            }
            ls[0] = tc::add2(tc::add2(ls[0], ls[1]), tc::add2(ls[2], ls[3]));
            l += ls[0].x + ls[0].y;
            // (P's place is free once the last product is done)
            if (j > 0 && __any_sync(FULL_MASK, !mbar_wait(bars + C::B_PV + 2 * x + ((j - 1) & 1), ((j - 1) >> 1) & 1, WAIT_NS))) {
                fail = true;
                break;
            }
            tc::fence_after();
            tc::st32(t_s + UK + 32, sr[0]);
            tc::st32(t_s + UK, w);
            tc::st_wait();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::arrive(bars + C::B_P + 2 * x + (j & 1));
        }
        if (!fail && nt > 0) {
            const int jl = nt - 1;
            if (__any_sync(FULL_MASK, !mbar_wait(bars + C::B_PV + 2 * x + (jl & 1), (jl >> 1) & 1, WAIT_NS))) fail = true;
        }
        const float m = ref == -INFINITY ? ref : ref * c;
        if (MODE == 0 && NT == 1 && n2 > 0) {
            // every row thread comes here, failed or not
            nl_s[tid] = live && !(m == -INFINITY && l == 0.f) ? less_sum(m + log2f(l)) : -INFINITY;
            asm volatile("bar.sync 1, %0;" ::"n"(C::ROWS) : "memory");
            const int shift = n_own - a.T;  // key j is seen by the queries t >= j - shift
            const int sh = s * a.Hk + hk;
            float* wrow = a.weight + (int64_t)sh * a.cap;
            float* prow = a.part_sum + ((int64_t)(first / QT) * a.S * a.Hk + sh) * a.cap;
            for (int kb = 0; kb < n2 && !fail; ++kb) {
                const int key = kb * QT + tid;
                const float old = a.sum_tiles == 1 && key < seen ? wrow[key] : 0.f;
                if (__any_sync(FULL_MASK, !mbar_wait(bars + C::B_T, kb & 1, WAIT_NS))) { fail = true; break; }
                tc::fence_after();
                // rows of the block before it do not see the key (the first slots of a long head, which
                // every row sees, lie far below shift: times rep that would pass 32 bits)
                const int from = max(0, key - shift) * a.rep - first;
                const bool whole = __shfl_sync(FULL_MASK, from, 31) <= 0;
                float total = 0.f;
#pragma unroll
                for (int c0 = 0; c0 < QT; c0 += 32) {
                    if (c0 >= rows) break;
                    uint32_t o[32];
                    tc::ld32(t_s + c0, o);
                    tc::ld_wait();
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int u = 0; u < 32; u += 4) {
                        const float4 e = *reinterpret_cast<const float4*>(nl_s + c0 + u);
                        const float ee[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const float p = tc::ex2(fmaf(__uint_as_float(o[u + v]), c, ee[v]));
                            acc[v] += whole || c0 + u + v >= from ? p : 0.f;
                        }
                    }
                    total += (acc[0] + acc[1]) + (acc[2] + acc[3]);
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::arrive(bars + C::B_TF);
                if (key < seen) {
                    if (a.sum_tiles == 1) wrow[key] = old + total;
                    else prow[key] = total;
                }
            }
        }
        if (!fail) {
            tc::fence_after();
            const int64_t row = live ? row_index(a, sq, h, t) : 0;
            const bool some = nt > 0 && !(m == -INFINITY && l == 0.f);
            constexpr bool final = MODE == 0;
            const float f = !final ? 1.f : some ? 1.f / l : 0.f;
            // The rows go out through Q's place (every product that read it is
            // done), 2 D bytes of a row at a time, so that a warp stores whole
            // rows and not 16 bytes of 32 of them.
            const int64_t dst = !live ? -1 : final ? sq * a.os[0] + h * a.os[1] + t * a.os[2] : (piece * R + row) * D;
            unsigned char* tile = q_s + x * C::Q_BYTES;
            constexpr int PASSES = final ? 1 : 2, FW = D / PASSES;  // values of a pass
#pragma unroll
            for (int pass = 0; pass < PASSES; ++pass) {
                if (idle) break;
                __syncwarp();
#pragma unroll
                for (int c0 = pass * FW; c0 < (pass + 1) * FW; c0 += 32) {
                    uint32_t o[32];
                    if (nt > 0) {
                        tc::ld32(t_o + c0, o);
                        tc::ld_wait();
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = some ? __float_as_uint(__uint_as_float(o[e]) * f) : 0u;
                    const int r = (warp & 3) * 32 + lane;
                    if constexpr (final) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(o[8 * e + 2 * u]), __uint_as_float(o[8 * e + 2 * u + 1]));
                                w[u] = *reinterpret_cast<uint32_t*>(&h2);
                            }
                            *reinterpret_cast<uint4*>(tile + q_off(r, c0 / 8 + e)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<uint4*>(tile + q_off(r, (c0 - pass * FW) / 4 + e)) =
                                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    const int r = e * RPI + lane / CH, c = lane % CH;
                    const int64_t o = __shfl_sync(FULL_MASK, dst, r);
                    const uint4 w = *reinterpret_cast<const uint4*>(tile + q_off((warp & 3) * 32 + r, c));
                    if (o >= 0) {
                        if constexpr (final) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + o + c * 8) = w;
                        else *reinterpret_cast<uint4*>(a.part_o + o + pass * FW + c * 4) = w;
                    }
                }
            }
            if (live) {
                if (final) {
                    const float l2 = some ? m + log2f(l) : -INFINITY;
                    if (a.lse) a.lse[row] = l2 * 0.6931471805599453f;
                    if (a.row_nl) a.row_nl[row] = less_sum(l2);
                } else {
                    a.part_ml[ml_index(a, row, piece)] = make_float2(l != l && m == -INFINITY ? 0.f : m, l);
                }
            }
        }
    }
    tc::fence_before();
    if (__syncthreads_or(fail)) {
        if (tid == 0 && a.status && atomicCAS(a.status, 0, HKV_ERR_TIMEOUT) == 0) atomicExch(a.status + 1, (int)blockIdx.x);
    }
    tc::fence_after();
    if (warp == 0) tc::dealloc(tmem, C::TMEM);
}

// weight += the sums that the row tiles' blocks left, in their order: those of
// the tiles whose last row sees the slot.  One thread a slot.
__global__ void __launch_bounds__(256) add_sums_kernel(const __grid_constant__ View a) {
    const int chunks = (a.cap + 255) / 256, sh = blockIdx.x / chunks, key = blockIdx.x % chunks * 256 + threadIdx.x;
    const int n = own_len(a, sh / a.Hk, sh % a.Hk), rps = a.rep * a.T;
    ptx::grid_dep_wait();
    if (key >= n) return;
    float* w = a.weight + (int64_t)sh * a.cap + key;
    float sum = 0.f;
    for (int t = 0; t < a.sum_tiles; ++t)
        if (key < own_limit(a, n, min(rps, (t + 1) * QT) - 1)) sum += a.part_sum[((int64_t)t * a.S * a.Hk + sh) * a.cap + key];
    *w += sum;
}

// ---------------------------------------------------------------------------
// accumulated weights of many rows
// ---------------------------------------------------------------------------

namespace {

template <int D> struct SumShape {
    static constexpr int KB = 128;      // keys of a block (MMA M)
    static constexpr int QN = 128;      // queries of a tile (MMA N)
    static constexpr int NS = 2;        // query tiles in shared memory, and S slots in TMEM
    static constexpr int NL = 4;        // places of the rows' sums
    static constexpr int THREADS = 256 + 64, COPY_WARP = 8, MMA_WARP = 9;
    static constexpr uint32_t TMEM = NS * QN;
    static constexpr int K_BYTES = KB * D * 2, Q_BYTES = QN * D * 2;
    enum { B_K, B_FULL, B_FREE = B_FULL + NS, B_S = B_FREE + NS, B_SF = B_S + NS, B_COUNT = B_SF + NS };
    static constexpr int SMEM = 1024 + K_BYTES + NS * Q_BYTES + NL * QN * 4 + KB * 4 + B_COUNT * 8 + 16;
};

}  // namespace

// weight[key] += sum over rows of 2^(c q.k - lse2[row]), the log2 of the row
// sums (row_nl: its negative) being known: the logits once more, keys on the M side, so that a
// thread owns a key (TMEM lane) and sums along its own columns.  One block
// per (sequence, KV head, 128 keys) walks 128-query tiles of each query head
// in turn, from the first query that sees its first key on; two groups of
// four warps take every other tile.  (With 64 queries a tile an MMA waits for
// shared memory, which gives it the 128 keys again for every 64 queries: 408
// cycles instead of 256.)  A row that is not to be counted has -lse2 = -inf.
// 16004 rows of 16 heads, 4001 keys, d = 128: 209 us, of exponentials (16 a cycle
// an SM) as much as of products.
template <int D>
__global__ void __launch_bounds__(SumShape<D>::THREADS, 2)
    column_sums_umma_kernel(const __grid_constant__ View a, const __grid_constant__ CUtensorMap km,
                            const __grid_constant__ CUtensorMap qm) {
    using C = SumShape<D>;
    extern __shared__ unsigned char raw[];
    unsigned char* k_s = reinterpret_cast<unsigned char*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    unsigned char* q_s = k_s + C::K_BYTES;
    float* nl_s = reinterpret_cast<float*>(q_s + C::NS * C::Q_BYTES);  // [NL][QN]
    float* half = nl_s + C::NL * C::QN;                                // [KB]
    uint64_t* bars = reinterpret_cast<uint64_t*>(half + C::KB);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::B_COUNT);
    constexpr int NSUB = D / 64;
    const int tid = threadIdx.x, warp = tc::uniform(tid >> 5), lane = tid & 31;
    // the first keys, which the most queries see, first
    const int heads = a.S * a.Hk, sh = blockIdx.x % heads, k0 = blockIdx.x / heads * C::KB;
    const int s = sh / a.Hk, hk = sh % a.Hk;
    ptx::grid_dep_wait();
    const int n = own_len(a, s, hk);
    if (k0 >= n) return;
    // key j is seen by the queries t >= j - (n - T)
    const int shift = n - a.T;
    const int tile0 = max(0, k0 - shift) / C::QN, per_head = (a.T + C::QN - 1) / C::QN - tile0;
    const int tiles = per_head * a.rep;

    if (warp == 0) tc::alloc(tmem_slot, C::TMEM);
    if (tid == 0) {
        for (int i = 0; i < C::B_COUNT; ++i) mbar_init(bars + i, i >= C::B_SF ? 4 : 1);
        ptx::fence_mbar_init();
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_slot;
    bool fail = false;
    float total = 0.f;

    if (warp == C::COPY_WARP) {
        if (lane == 0) {
            mbar_expect_tx(bars + C::B_K, C::K_BYTES);
            for (int sub = 0; sub < NSUB; ++sub) tc::tma_load_4d(k_s + sub * C::KB * 128, &km, bars + C::B_K, sub * 64, k0, hk, s);
        }
        int issued = 0;
        // The sums of the next tile's rows are read a tile ahead.  Their places
        // are free: Q's place is given back once S of tile j - 2 is done, and that
        // S was issued after the rows had finished with tile j - 4.
        float nl[C::QN / 32];
        auto fetch = [&](int j) {
            const float* src = a.row_nl + row_index(a, s, hk * a.rep + j / per_head, 0);
#pragma unroll
            for (int u = 0; u < C::QN / 32; ++u) {
                const int t = (tile0 + j % per_head) * C::QN + u * 32 + lane;
                nl[u] = j < tiles && t < a.T ? src[t] : -INFINITY;
            }
        };
        if (tiles > 0) fetch(0);
        for (int j = 0; j < tiles; ++j) {
            const int slot = j % C::NS, use = j / C::NS;
            if (use > 0 && __any_sync(FULL_MASK, !mbar_wait(bars + C::B_FREE + slot, (use - 1) & 1, WAIT_NS))) { fail = true; break; }
            const int h = hk * a.rep + j / per_head, t0 = (tile0 + j % per_head) * C::QN;
#pragma unroll
            for (int u = 0; u < C::QN / 32; ++u) nl_s[j % C::NL * C::QN + u * 32 + lane] = nl[u];
            __syncwarp();
            if (lane == 0) {
                mbar_expect_tx(bars + C::B_FULL + slot, C::Q_BYTES);
                for (int sub = 0; sub < NSUB; ++sub)
                    tc::tma_load_4d(q_s + slot * C::Q_BYTES + sub * C::QN * 128, &qm, bars + C::B_FULL + slot, sub * 64, t0, h, s);
            }
            issued = j + 1;
            fetch(j + 1 < tiles ? j + 1 : j);
        }
        if (fail && lane == 0) {
            mbar_wait(bars + C::B_K, 0, WAIT_NS);
            for (int j = max(0, issued - C::NS); j < issued; ++j)
                mbar_wait(bars + C::B_FULL + j % C::NS, (j / C::NS) & 1, WAIT_NS);
        }
    } else if (warp == C::MMA_WARP) {
        constexpr uint32_t IS = tc::idesc_bf16(C::QN, false);
        const uint32_t tm = tc::uniform(tmem);
        const uint64_t k_desc = tc::sw128_desc(tc::uniform(smem_u32(k_s)), 16, 1024),
                       q_desc = tc::sw128_desc(tc::uniform(smem_u32(q_s)), 16, 1024);
        const int nt = tc::uniform(tiles);
        if (tc::elect()) {
            int done = -1;
            if (!mbar_wait(bars + C::B_K, 0, WAIT_NS)) fail = true;
            for (int j = 0; j < nt && !fail; ++j) {
                const int slot = j % C::NS;
                if (!mbar_wait(bars + C::B_FULL + slot, (j / C::NS) & 1, WAIT_NS) ||
                    (j >= C::NS && !mbar_wait(bars + C::B_SF + slot, (j / C::NS - 1) & 1, WAIT_NS))) {
                    fail = true;
                    break;
                }
                tc::fence_after();
                const uint64_t qd = q_desc + slot * (C::Q_BYTES / 16);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc::mma_ss(tm + slot * C::QN, k_desc + (kk / 4) * (C::KB * 8) + (kk % 4) * 2,
                               qd + (kk / 4) * (C::QN * 8) + (kk % 4) * 2, IS, kk > 0);
                tc::commit(bars + C::B_S + slot);
                tc::commit(bars + C::B_FREE + slot);
                done = j;
            }
            if (done >= 0) {
                mbar_wait(bars + C::B_S + done % C::NS, (done / C::NS) & 1, WAIT_NS);
                mbar_wait(bars + C::B_FREE + done % C::NS, (done / C::NS) & 1, WAIT_NS);
            }
        }
        __syncwarp();
    } else {
        const int grp = warp >> 2, key = k0 + (tid & 127);
        const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const float c = a.qscale;
        const int last = __shfl_sync(FULL_MASK, key, 31) - shift;  // first query that the warp's last key is seen by
        for (int j = grp; j < tiles; j += 2) {
            const int slot = j % C::NS, t0 = (tile0 + j % per_head) * C::QN;
            if (__any_sync(FULL_MASK, !mbar_wait(bars + C::B_S + slot, (j / C::NS) & 1, WAIT_NS))) { fail = true; break; }
            tc::fence_after();
            const float* nl = nl_s + j % C::NL * C::QN;
            const uint32_t at = t_lane + slot * C::QN;
            // (columns before key - shift - t0 do not see the key)
            total += t0 >= last && t0 + C::QN <= a.T ? column_weights<true>(at, nl, c, 0, C::QN)
                                                     : column_weights<false>(at, nl, c, key - shift - t0, min(C::QN, a.T - t0));
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::arrive(bars + C::B_SF + slot);
        }
        if (grp == 1) half[tid & 127] = total;
    }
    tc::fence_before();
    if (__syncthreads_or(fail)) {
        if (tid == 0 && a.status && atomicCAS(a.status, 0, HKV_ERR_TIMEOUT) == 0) atomicExch(a.status + 1, (int)blockIdx.x);
    } else if (tid < C::KB && k0 + tid < n) {
        a.weight[(int64_t)sh * a.cap + k0 + tid] += total + half[tid];
    }
    tc::fence_after();
    if (warp == 0) tc::dealloc(tmem, C::TMEM);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// Tensor map of bf16 rows [n2][n1][n0] of d elements at strides st (elements:
// outermost, middle, row): boxes of 64 columns x box rows, 128-byte swizzle,
// zeros past the ends.
static bool make_map(CUtensorMap* m, const void* ptr, int d, int n0, int n1, int n2, const int64_t* st, int box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    // a dimension of one element may come with any stride: give it a lawful one
    auto bytes = [&](int n, int64_t e) { return (cuuint64_t)(n == 1 ? (int64_t)d * 2 : e * 2); };
    cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n0, (cuuint64_t)n1, (cuuint64_t)n2};
    cuuint64_t strides[3] = {bytes(n0, st[2]), bytes(n1, st[1]), bytes(n2, st[0])};
    cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, bx, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, int MODE>
static cudaError_t go(const View& a, const CUtensorMap* m, int64_t blocks, int row_tiles, int splits, cudaStream_t st) {
    using C = Shape<D, NT>;
    return launch(attend_umma_kernel<D, NT, MODE>, blocks, C::THREADS, C::SMEM, st, a, m[0], m[1], m[2], m[3], row_tiles,
                  splits);
}

static bool own_maps(const View& a, int d, CUtensorMap* m) {
    return make_map(m, a.k, d, a.cap, a.Hk, a.S, a.ks, UK) && make_map(m + 1, a.v, d, a.cap, a.Hk, a.S, a.vs, UK);
}
static bool prefix_maps(const View& a, int d, CUtensorMap* m) {
    return make_map(m, a.pk, d, a.pcap, a.Hk, a.G, a.pks, UK) && make_map(m + 1, a.pv, d, a.pcap, a.Hk, a.G, a.pvs, UK);
}

cudaError_t launch_attend_umma(const View& a, int d, cudaStream_t st) {
    CUtensorMap m[4];
    if (!own_maps(a, d, m)) return cudaErrorInvalidValue;
    if (a.G == 0) {  // never read
        m[2] = m[0];
        m[3] = m[1];
    } else if (!prefix_maps(a, d, m + 2)) {
        return cudaErrorInvalidValue;
    }
    const int rps = a.rep * a.T, nt = umma_row_tiles(rps), splits = a.no;
    const int tiles = (rps + QT * nt - 1) / (QT * nt);
    const int64_t blocks = (int64_t)tiles * a.S * a.Hk * splits;
    auto run = [&](auto dim, auto mode) {
        constexpr int D = decltype(dim)::value, MODE = decltype(mode)::value;
        return nt == 2 ? go<D, 2, MODE>(a, m, blocks, tiles, splits, st) : go<D, 1, MODE>(a, m, blocks, tiles, splits, st);
    };
    using Final = std::integral_constant<int, 0>;
    using Pieces = std::integral_constant<int, 2>;
    if (d == 128) {
        using Dim = std::integral_constant<int, 128>;
        return splits == 1 ? run(Dim(), Final()) : run(Dim(), Pieces());
    }
    using Dim = std::integral_constant<int, 64>;
    return splits == 1 ? run(Dim(), Final()) : run(Dim(), Pieces());
}

cudaError_t launch_add_sums(const View& a, cudaStream_t st) {
    return launch(add_sums_kernel, (int64_t)a.S * a.Hk * ((a.cap + 255) / 256), 256, 0, st, a);
}

cudaError_t launch_prefix_umma(const View& a, int d, cudaStream_t st) {
    CUtensorMap m[4];
    if (!prefix_maps(a, d, m + 2)) return cudaErrorInvalidValue;
    m[0] = m[2];  // never read
    m[1] = m[3];
    const int rps = a.rep * a.T;
    const int64_t tiles = max_prefix_tiles(a.S, a.G, rps, QT);
    const int64_t blocks = tiles * a.Hk * a.np;
    return d == 128 ? go<128, 1, 1>(a, m, blocks, (int)tiles, 1, st) : go<64, 1, 1>(a, m, blocks, (int)tiles, 1, st);
}

cudaError_t launch_column_sums_umma(const View& a, int d, cudaStream_t st) {
    CUtensorMap km, qm;
    if (!make_map(&km, a.k, d, a.cap, a.Hk, a.S, a.ks, 128) || !make_map(&qm, a.q, d, a.T, a.H, a.S, a.qs, 128))
        return cudaErrorInvalidValue;
    const int64_t blocks = (int64_t)a.S * a.Hk * ((a.cap + 127) / 128);
    if (d == 128) return launch(column_sums_umma_kernel<128>, blocks, SumShape<128>::THREADS, SumShape<128>::SMEM, st, a, km, qm);
    return launch(column_sums_umma_kernel<64>, blocks, SumShape<64>::THREADS, SumShape<64>::SMEM, st, a, km, qm);
}

cudaError_t prepare_shared_umma() {
    cudaError_t e = cudaSuccess;
    auto set = [&](auto kernel, int smem) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    };
    auto all = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        set(attend_umma_kernel<D, 1, 0>, Shape<D, 1>::SMEM);
        set(attend_umma_kernel<D, 2, 0>, Shape<D, 2>::SMEM);
        set(attend_umma_kernel<D, 1, 1>, Shape<D, 1>::SMEM);
        set(attend_umma_kernel<D, 1, 2>, Shape<D, 1>::SMEM);
        set(attend_umma_kernel<D, 2, 2>, Shape<D, 2>::SMEM);
    };
    all(std::integral_constant<int, 64>());
    all(std::integral_constant<int, 128>());
    set(column_sums_umma_kernel<128>, SumShape<128>::SMEM);
    set(column_sums_umma_kernel<64>, SumShape<64>::SMEM);
    return e;
}

}  // namespace shared
}  // namespace hkv
