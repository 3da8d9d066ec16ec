// shared_evict.cu -- eviction by accumulated weight from a shared-prefix cache.
//
// A due head (len n >= budget B + slack) loses the E = n - B tokens lowest in
// (recent, weight, position, slot).  The first two fields fold into 32 bits
// that order like them (ordered float bits; all recent tokens share the
// highest value) and the position into 32 more.  The E-th smallest of these
// 64-bit keys is found digit by digit from the top (histograms of 11 or 10
// bits in shared memory); as soon as at most CAND tokens are left to choose
// from they are ranked against each other by (key, slot): at once in a short
// head, after the first or second digit in a long one whose weights differ.
// Tokens at or below the threshold are evicted.  The head's weights and
// positions are read once, into shared memory where they fit.
//
// What bounds it: a short head (a few hundred tokens) the chain of block-wide
// steps, so one small block a head and as many heads as fit at once; a long
// one the rows that move, which a second launch spreads over the GPU.  d = 128,
// bf16: 64 of 477 tokens of 512 heads 14 us, one of 28 to 107 of 1024 heads 9 us;
// 8192 of 24576 of 64 heads 42 us for the selection, 64 us for 257 MB of rows
// (launches alone).
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"
#include "shared.cuh"

namespace hkv {
namespace shared {

namespace {

constexpr int BINS = 2048;
constexpr int CAND = 64;        // candidates ranked against each other (with 256, 512 heads of 477 slots took 40 us instead of 23)
constexpr int LIST = 512;       // moves whose slots stay in shared memory
// Blocks of 128 threads that also move the rows, up to SHORT_CAP slots where
// there are more heads than SMs, else up to half as many; more: blocks of 1024,
// and a launch for the rows.  (us, 128 / 1024 threads: 1024 heads of 2000 slots
// 58.8 / 106.5, 256 of 2000 29.2 / 31.8, 148 of 1400 22.4 / 20.5; 32 heads of 477
// 13.0 / 15.6, of 1000 18.6 / 17.8, of 2000 26.6 / 20.0.)
constexpr int SHORT_CAP = 2048;
// Capacities up to this: weights and positions in shared memory (200 KB; 64 heads
// of up to 24576 slots: 157 us held, 178 read again for every step).
constexpr int HELD_CAP = 24576;

// Bits that order as (recent, weight): recent tokens highest, then NaN, then
// the numbers (-0 as +0).
__device__ __forceinline__ uint32_t class_bits(float w, bool recent) {
    if (recent) return 0xffffffffu;
    if (w != w) return 0xfffffffeu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

template <int THREADS> struct EvictSmem {
    // bins a thread adds up lie PER apart, and a word further each thread
    static constexpr int PER = BINS / THREADS;
    int hist[BINS + THREADS];
    __device__ int& bin_at(int b) { return hist[b + b / PER]; }
    uint64_t cand_key[CAND];
    int cand_slot[CAND];
    int list[2 * LIST];
    int warp_a[THREADS / 32], warp_b[THREADS / 32];
    int newest, digit, below, n_cand, thr_slot;
    uint64_t thr_key;
};

// Moves rows (16-byte pieces), positions and weights from movers to holes:
// entries first, first + step, ... of the lists.
__device__ __forceinline__ void move_rows(const View& a, int head, const int* holes, const int* movers, int count,
                                          int first, int step, int row_bytes, int es) {
    const int s = head / a.Hk, hk = head % a.Hk;
    unsigned char* kb = static_cast<unsigned char*>(a.k) + (s * a.ks[0] + hk * a.ks[1]) * es;
    unsigned char* vb = static_cast<unsigned char*>(a.v) + (s * a.vs[0] + hk * a.vs[1]) * es;
    const int64_t kst = a.ks[2] * es, vst = a.vs[2] * es;
    int32_t* pos = a.pos + (int64_t)head * a.cap;
    float* weight = a.weight + (int64_t)head * a.cap;
    const int pieces = row_bytes / 16, per = (int)blockDim.x / pieces;  // rows a block moves at once
    const int c = threadIdx.x % pieces * 16, lead = threadIdx.x / pieces;
    // four rows' pieces in flight a thread
    for (int i0 = first * per * 4 + lead; i0 < count; i0 += step * per * 4) {
        uint4 x[4], y[4];
        int to[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * per;
            to[u] = i < count ? holes[i] : -1;
            if (to[u] < 0) continue;
            const int from = movers[i];
            x[u] = *reinterpret_cast<const uint4*>(kb + from * kst + c);
            y[u] = *reinterpret_cast<const uint4*>(vb + from * vst + c);
            if (c == 0) {
                pos[to[u]] = pos[from];
                weight[to[u]] = weight[from];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (to[u] < 0) continue;
            *reinterpret_cast<uint4*>(kb + to[u] * kst + c) = x[u];
            *reinterpret_cast<uint4*>(vb + to[u] * vst + c) = y[u];
        }
    }
}

}  // namespace

// One block per (sequence, KV head).  move: the block moves its rows itself;
// otherwise it leaves the lists in `lists` (holes from 0, movers from B, the
// counts in `counts`) for move_kernel.
template <int THREADS, bool HELD>
__global__ void __launch_bounds__(THREADS) select_kernel(const __grid_constant__ View a,
                                                         const int32_t* budget, int recent, int slack,
                                                         int row_bytes, int es, int move, int32_t* lists,
                                                         int2* counts) {
    __shared__ EvictSmem<THREADS> sm;
    extern __shared__ __align__(16) unsigned char held_raw[];
    constexpr int WARPS = THREADS / 32;
    const int head = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ptx::grid_dep_wait();
    const int n = own_len(a, head / a.Hk, head % a.Hk), B = max(0, budget[head]);
    if ((int64_t)n < (int64_t)B + slack) {
        if (!move && tid == 0) counts[head] = make_int2(0, 0);
        return;
    }
    const int E = n - B;
    const int32_t* pos = a.pos + (int64_t)head * a.cap;
    const float* weight = a.weight + (int64_t)head * a.cap;
    if (tid == 0) {
        sm.newest = INT32_MIN;
        sm.n_cand = 0;
    }
    // what is held: positions, and weights until the first look at the keys
    // turns them into their class bits; then a bit a slot: evicted
    int32_t* hpos = reinterpret_cast<int32_t*>(held_raw);
    uint32_t* hclass = reinterpret_cast<uint32_t*>(held_raw) + a.cap;
    uint32_t* hgone = hclass + a.cap;
    int nw = INT32_MIN;
    for (int i0 = tid; i0 < n; i0 += 4 * THREADS) {
        int32_t p[4];
        float w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * THREADS;
            p[u] = i < n ? pos[i] : INT32_MIN;
            w[u] = HELD && i < n ? weight[i] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * THREADS;
            nw = max(nw, p[u]);
            if (HELD && i < n) {
                hpos[i] = p[u];
                hclass[i] = __float_as_uint(w[u]);
            }
        }
    }
    nw = __reduce_max_sync(FULL_MASK, nw);
    __syncthreads();
    if (lane == 0) atomicMax(&sm.newest, nw);
    __syncthreads();
    const int64_t newest = sm.newest;
    if (HELD) {
        for (int i = tid; i < n; i += THREADS) hclass[i] = class_bits(__uint_as_float(hclass[i]), newest - hpos[i] < recent);
        __syncthreads();
    }
    auto key = [&](int i) {
        const int p = HELD ? hpos[i] : pos[i];
        const uint32_t c = HELD ? hclass[i] : class_bits(weight[i], newest - p < recent);
        return ((uint64_t)c << 32) | ((uint32_t)p ^ 0x80000000u);
    };

    // the threshold: (thr_key, thr_slot), the last to go
    uint64_t prefix = 0, mask = 0;
    int want = E, found = 0, count = n;
    for (int d = 0; d <= 6 && !found; ++d) {
        // `count` tokens share the digits so far, `want` of them go
        if (count == want) {
            if (tid == 0) {
                sm.thr_key = prefix | ~mask;
                sm.thr_slot = INT32_MAX;
            }
            found = 1;
            break;
        }
        if (count <= CAND) {
            for (int i = tid; i < n; i += THREADS) {
                const uint64_t k = key(i);
                if ((k & mask) == prefix) {
                    const int c = atomicAdd(&sm.n_cand, 1);
                    sm.cand_key[c] = k;
                    sm.cand_slot[c] = i;
                }
            }
            __syncthreads();
            for (int c = tid; c < count; c += THREADS) {
                const uint64_t k = sm.cand_key[c];
                const int i = sm.cand_slot[c];
                int rank = 0;
#pragma unroll 4
                for (int e = 0; e < count; ++e) {
                    const uint64_t ke = sm.cand_key[e];
                    rank += (int)(ke < k) | ((int)(ke == k) & (int)(sm.cand_slot[e] < i));
                }
                if (rank == want - 1) {
                    sm.thr_key = k;
                    sm.thr_slot = i;
                }
            }
            found = 1;
            break;
        }
        if (d == 6) break;
        // digits of 11, 11 and 10 bits in each half
        const int bits = d == 2 || d == 5 ? 10 : 11, shift = (d < 3 ? 32 : 0) + (d % 3 == 0 ? 21 : d % 3 == 1 ? 10 : 0);
        for (int i = tid; i < BINS + THREADS; i += THREADS) sm.hist[i] = 0;
        __syncthreads();
        for (int i0 = 0; i0 < n; i0 += THREADS) {
            const int i = i0 + tid;
            const uint64_t k = i < n ? key(i) : 0;
            const bool in = i < n && (k & mask) == prefix;
            const int dig = (int)(k >> shift) & ((1 << bits) - 1);
            // lanes that share the first lane's digit count together: equal
            // weights and recent tokens would queue up at one address
            const unsigned on = __ballot_sync(FULL_MASK, in);
            if (on == 0) continue;
            const int lead = __ffs(on) - 1, ldig = __shfl_sync(FULL_MASK, dig, lead);
            const unsigned same = __ballot_sync(FULL_MASK, in && dig == ldig);
            if (lane == lead) atomicAdd(&sm.bin_at(ldig), __popc(same));
            else if (in && dig != ldig) atomicAdd(&sm.bin_at(dig), 1);
        }
        __syncthreads();
        constexpr int PER = EvictSmem<THREADS>::PER;
        int own = 0;
#pragma unroll
        for (int u = 0; u < PER; ++u) own += sm.bin_at(tid * PER + u);
        int incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL_MASK, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sm.warp_a[warp] = incl;
        __syncthreads();
        int before = incl - own;
        for (int w = 0; w < warp; ++w) before += sm.warp_a[w];
        if (before < want && want <= before + own) {
            int u = 0;
            while (want > before + sm.bin_at(tid * PER + u)) before += sm.bin_at(tid * PER + u++);
            sm.digit = tid * PER + u;
            sm.below = before;
        }
        __syncthreads();
        const int digit = sm.digit;
        count = sm.bin_at(digit);
        want -= sm.below;
        prefix |= (uint64_t)digit << shift;
        mask |= (uint64_t)((1 << bits) - 1) << shift;
        __syncthreads();  // (the bins are cleared next)
    }
    // slots are dealt to the warps in contiguous runs
    const int seg = (n + WARPS * 32 - 1) / (WARPS * 32) * 32;
    const int lo = min(n, warp * seg), hi = min(n, lo + seg);
    if (!found) {
        // more than CAND tokens share the key: the lowest `want` slots of them go
        int c = 0;
        for (int i0 = lo; i0 < hi; i0 += 32) c += __popc(__ballot_sync(FULL_MASK, i0 + lane < hi && key(i0 + lane) == prefix));
        if (lane == 0) sm.warp_a[warp] = c;
        __syncthreads();
        int before = 0;
        for (int w = 0; w < warp; ++w) before += sm.warp_a[w];
        for (int i0 = lo; i0 < hi && before < want; i0 += 32) {
            const bool eq = i0 + lane < hi && key(i0 + lane) == prefix;
            const unsigned b = __ballot_sync(FULL_MASK, eq);
            if (eq && before + __popc(b & ((1u << lane) - 1)) == want - 1) {
                sm.thr_key = prefix;
                sm.thr_slot = i0 + lane;
            }
            before += __popc(b);
        }
    }
    __syncthreads();
    const uint64_t thr_key = sm.thr_key;
    const int thr_slot = sm.thr_slot;
    auto gone = [&](int i) {
        const uint64_t k = key(i);
        return k < thr_key || (k == thr_key && i <= thr_slot);
    };
    // holes (evicted below B) and movers (survivors from B on) in slot order
    int nh = 0, nm = 0;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const unsigned g = __ballot_sync(FULL_MASK, i < hi && gone(i));
        // (bit masks of the 32 slots from i0: those below B, those below the end)
        const unsigned below = B >= i0 + 32 ? FULL_MASK : B <= i0 ? 0u : (1u << (B - i0)) - 1;
        const unsigned in = hi >= i0 + 32 ? FULL_MASK : (1u << (hi - i0)) - 1;
        nh += __popc(g & below);
        nm += __popc(in & ~g & ~below);
        if (HELD && lane == 0) hgone[i0 >> 5] = g;
    }
    __syncwarp();
    if (lane == 0) {
        sm.warp_a[warp] = nh;
        sm.warp_b[warp] = nm;
    }
    __syncthreads();
    int bh = 0, bm = 0, moves = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) {
            bh += sm.warp_a[w];
            bm += sm.warp_b[w];
        }
        moves += sm.warp_b[w];
    }
    // (as many movers as holes; both lists fit a row of `lists`: B + moves <= n)
    int* hl = move && moves <= LIST ? sm.list : lists + (int64_t)head * a.cap;
    int* ml = move && moves <= LIST ? sm.list + LIST : hl + B;
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const unsigned g = HELD ? hgone[i0 >> 5] : __ballot_sync(FULL_MASK, i < hi && gone(i));
        const unsigned below = B >= i0 + 32 ? FULL_MASK : B <= i0 ? 0u : (1u << (B - i0)) - 1;
        const unsigned in = hi >= i0 + 32 ? FULL_MASK : (1u << (hi - i0)) - 1;
        const unsigned b = g & below, m = in & ~g & ~below, lt = (1u << lane) - 1;
        if (b >> lane & 1) hl[bh + __popc(b & lt)] = i;
        if (m >> lane & 1) ml[bm + __popc(m & lt)] = i;
        bh += __popc(b);
        bm += __popc(m);
    }
    __syncthreads();
    if (move) {
        move_rows(a, head, hl, ml, moves, 0, 1, row_bytes, es);
    } else if (tid == 0) {
        counts[head] = make_int2(moves, B);
    }
    if (tid == 0) a.len[head] = B;
}

// Block (head, part): every parts-th group of the head's moves.
__global__ void __launch_bounds__(256) move_kernel(const __grid_constant__ View a, int parts, int row_bytes, int es,
                                                   const int32_t* lists, const int2* counts) {
    const int head = blockIdx.x / parts;
    ptx::grid_dep_wait();
    const int2 c = counts[head];
    const int32_t* hl = lists + (int64_t)head * a.cap;
    move_rows(a, head, hl, hl + c.y, c.x, blockIdx.x % parts, parts, row_bytes, es);
}

// positions, classes and the evicted slots' bits of a head
static size_t held_bytes(int cap) { return (size_t)cap * 8 + (size_t)(cap + 31) / 32 * 4; }

cudaError_t prepare_shared_evict() {
    return cudaFuncSetAttribute(select_kernel<1024, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)held_bytes(HELD_CAP));
}

size_t evict_bytes(int heads, int cap) {
    return (size_t)heads * cap * 4 + ((size_t)heads * 8 + 255) / 256 * 256;
}

cudaError_t launch_evict(const View& a, int dtype, int d, const int32_t* budget, int recent, int slack,
                         unsigned char* scratch, cudaStream_t st) {
    const int es = dtype == HKV_DTYPE_F32 ? 4 : 2, heads = a.S * a.Hk, row = d * es;
    int2* counts = reinterpret_cast<int2*>(scratch);
    int32_t* lists = reinterpret_cast<int32_t*>(scratch + ((size_t)heads * 8 + 255) / 256 * 256);
    const size_t held = held_bytes(a.cap);
    if (a.cap <= (heads > SMS ? SHORT_CAP : SHORT_CAP / 2))
        return launch(select_kernel<128, true>, heads, 128, held, st, a, budget, recent, slack, row, es, 1, lists, counts);
    const cudaError_t e =
        a.cap <= HELD_CAP
            ? launch(select_kernel<1024, true>, heads, 1024, held, st, a, budget, recent, slack, row, es, 0, lists, counts)
            : launch(select_kernel<1024, false>, heads, 1024, 0, st, a, budget, recent, slack, row, es, 0, lists, counts);
    if (e != cudaSuccess) return e;
    const int parts = std::max(1, (SMS * 8 + heads - 1) / heads);
    return launch(move_kernel, (int64_t)heads * parts, 256, 0, st, a, parts, row, es, lists, counts);
}

}  // namespace shared
}  // namespace hkv
