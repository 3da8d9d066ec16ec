// shared.cuh -- device view of a shared-prefix cache and what its kernels
// agree on: how rows are numbered, how key ranges are split, and the partial
// results that the combining kernel joins.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/hkv.h"
#include "hkv_internal.cuh"

namespace hkv {
namespace shared {

constexpr int SMS = 148;         // of the GPU
constexpr int KEY_STEP = 64;     // key ranges start at multiples of this
constexpr int MAX_SPLITS = 64;   // splits of the own keys, and of the prefix keys
constexpr int MAX_PREFIXES = 1024;
// Own tokens of at most this many query rows (query heads of a KV head x
// queries) are streamed once with every row's logits kept for the accumulated
// weights, bf16 as one M side of mma.sync; more rows go to the tcgen05 tiles and
// recompute the logits.  (16 rows, d = 128, streamed / tiles: 12 heads of 9000 to
// 32001 slots 45.5 / 213 us, 512 heads of 56 to 477 37.6 / 42.8 us.)
constexpr int STREAM_ROWS = 16;
constexpr int STREAM_ROWS_F32 = 8;  // see shared_stream_f32.cu

// The cache and one call's tensors, by value.
struct View {
    int32_t S, H, Hk, rep, cap, G, pcap, T;
    uint64_t rep_inv;  // ceil(2^40 / rep), see query_of
    void *k, *v;
    int64_t ks[3], vs[3];
    int32_t* pos;
    float* weight;
    int32_t* len;
    int32_t* next_pos;
    const void *pk, *pv;
    int64_t pks[3], pvs[3];
    const int32_t* plen;
    const int32_t* pof;
    int32_t* status;
    const void* q;
    void* out;
    int64_t qs[3], os[3];
    float* lse;
    float qscale;     // scale * log2(e): logits are in the exp2 domain
    // partial results of a row: slots [0, np) the prefix's splits, [np, np + no) its own keys'
    int32_t np, no;
    // 1 (np is 0): the slots are no pieces of one list of 64-key tiles, the prefix's and then the own ones
    int32_t listed;
    float2* part_ml;  // [R][np + no] (max, sum)
    float* part_o;    // [np + no][R][d]
    float* logit;     // [S][Hk][rep T][lcap] exp2-domain logits of the own keys (few rows, accumulate)
    int32_t lcap;     // capacity rounded up to 4
    int32_t sum_tiles;  // row tiles of a (sequence, KV head) whose blocks sum the weights themselves (0: they do not)
    float* part_sum;    // [sum_tiles][S][Hk][cap] their sums, where there are several
    float* row_nl;    // [R] less_sum of the rows (weights summed in a pass of their own)
};

// 2^24: logits from here on are off by one and more.
constexpr float BIG = 16777216.f;

// What the sums of the weights add to a row's logits: minus the log2 of its sum
// (l2 = -inf: the row has no weights).  Beyond BIG that is off by more than one
// and would let weights be infinite: there it is lowered by more than its own
// and the logits' rounding.
__device__ __forceinline__ float less_sum(float l2) {
    return l2 == -INFINITY ? l2 : fabsf(l2) > BIG ? -l2 - fabsf(l2) * 0x1p-21f : -l2;
}

__device__ __forceinline__ int clamp_len(int n, int cap) { return n < 0 ? 0 : (n > cap ? cap : n); }
__device__ __forceinline__ int own_len(const View& a, int s, int hk) {
    return clamp_len(a.len[(size_t)s * a.Hk + hk], a.cap);
}
// Prefix of a sequence (-1: none) and its length.
__device__ __forceinline__ int prefix_of(const View& a, int s) {
    if (a.G == 0) return -1;
    const int g = a.pof[s];
    return (unsigned)g < (unsigned)a.G ? g : -1;
}
__device__ __forceinline__ int prefix_len(const View& a, int g) {
    return g < 0 ? 0 : clamp_len(a.plen[g], a.pcap);
}
// Split j of n keys cut in ns: [lo, hi), empty when lo >= hi.
__device__ __forceinline__ int split_size(int n, int ns) {
    const int c = (n + ns - 1) / ns;
    return (c + KEY_STEP - 1) / KEY_STEP * KEY_STEP;
}
__device__ __forceinline__ void split_range(int n, int ns, int j, int& lo, int& hi) {
    const int64_t c = split_size(n, ns);
    lo = (int)min((int64_t)n, c * j);
    hi = (int)min((int64_t)n, c * (j + 1));
}
// Piece j of `no` of a list of 64-key tiles, those of pl prefix keys and then
// those of n own keys: prefix keys [pa, pb), own keys [oa, ob).
struct Piece {
    int pa, pb, oa, ob;
    __device__ bool empty() const { return pa >= pb && oa >= ob; }
};
__device__ __forceinline__ Piece list_piece(int pl, int n, int no, int j) {
    const int pt = (pl + KEY_STEP - 1) / KEY_STEP, all = pt + (n + KEY_STEP - 1) / KEY_STEP;
    const int64_t per = (all + no - 1) / no;
    const int t0 = (int)min((int64_t)all, per * j), t1 = (int)min((int64_t)all, per * j + per);
    Piece p;
    p.pa = min(pl, t0 * KEY_STEP);
    p.pb = min(pl, t1 * KEY_STEP);
    p.oa = min(n, max(0, t0 - pt) * KEY_STEP);
    p.ob = min(n, max(0, t1 - pt) * KEY_STEP);
    return p;
}
// Whether slot j of the partial results of a row with pk prefix keys and ok own keys was written.
__device__ __forceinline__ bool slot_valid(const View& a, int j, int pk, int ok) {
    if (a.listed) return !list_piece(pk, ok, a.no, j).empty();
    if (j >= a.np) return !list_piece(0, ok, a.no, j - a.np).empty();
    int lo, hi;
    split_range(pk, a.np, j, lo, hi);
    return lo < hi;
}
// Row of (sequence, query head, query) in lse and the partial arrays.
__device__ __forceinline__ int64_t row_index(const View& a, int s, int h, int t) {
    return ((int64_t)s * a.H + h) * a.T + t;
}
__device__ __forceinline__ int64_t ml_index(const View& a, int64_t row, int slot) { return row * (a.np + a.no) + slot; }
// Rows of one (sequence, KV head) are numbered i = t * rep + (query head within
// the KV head).  i / rep by multiplication (exact for i < 2^24 and rep < 2^16:
// the product is too large by less than i rep / 2^40 < 1 / rep); kernels that
// divided spent more on their rows' places than on reading them.
__device__ __forceinline__ int query_of(const View& a, int i) { return (int)((uint64_t)i * a.rep_inv >> 40); }
__device__ __forceinline__ int64_t row_of(const View& a, int s, int hk, int i) {
    const int t = query_of(a, i);
    return row_index(a, s, hk * a.rep + i - t * a.rep, t);
}
// Own slots row i sees: those before len - T + t + 1.
__device__ __forceinline__ int own_limit(const View& a, int n, int i) {
    const int lim = n - a.T + query_of(a, i) + 1;
    return lim < 0 ? 0 : lim;
}

// 16 bytes from global to shared memory, asynchronously; zeros where not `on`.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// Adds the weights 2^(x - M) / l of a head's kept logits to its accumulated
// ones, rows in order: slots k0, k0 + step, ..., four at once.  ml: the rows' (M, 1 / l).
__device__ __forceinline__ void add_kept(const View& a, int sh, int n, const float2* ml, int k0, int step) {
    const int rps = a.rep * a.T;
    const float* lg = a.logit + (int64_t)sh * rps * a.lcap;
    float* w = a.weight + (int64_t)sh * a.cap;
    for (; k0 < n; k0 += 4 * step) {
        float sum[4], old[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            sum[v] = 0.f;
            old[v] = k0 + step * v < n ? w[k0 + step * v] : 0.f;
        }
        for (int i = 0; i < rps; ++i) {
            const float2 y = ml[i];
            if (y.x == -INFINITY) continue;
            const float* x = lg + (int64_t)i * a.lcap + k0;
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (k0 + step * v < n) sum[v] += exp2f(x[step * v] - y.x) * y.y;
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (k0 + step * v < n) w[k0 + step * v] = old[v] + sum[v];
    }
}

// Finds the `tile`-th tile of `rt` rows among the prefixes' row lists: the
// rows of prefix g are those of the sequences that continue it (ascending),
// rep * T each, and every prefix starts a new tile.  Gives the prefix, the
// first row and the number of rows, and in `list` the sequences of the rows:
// list[o - first / (rep T)] for the o-th sequence of the prefix (at most rt
// + 1 of them).  False: there is no such tile.  Called by the whole block;
// cnt: G ints of shared memory, res: four.
__device__ inline bool find_prefix_tile(const View& a, int tile, int rt, int& g, int& first, int& rows,
                                        int* cnt, int* res, int* list) {
    const int tid = threadIdx.x, rps = a.rep * a.T;
    for (int i = tid; i < a.G; i += blockDim.x) cnt[i] = 0;
    if (tid < 4) res[tid] = -1;
    __syncthreads();
    for (int i = tid; i < a.S; i += blockDim.x) {
        const int p = prefix_of(a, i);
        if (p >= 0) atomicAdd(cnt + p, 1);
    }
    __syncthreads();
    if (tid < 32) {
        // running tile counts over the prefixes, 32 at a time
        int base = 0;
        for (int g0 = 0; g0 < a.G; g0 += 32) {
            const int gi = g0 + tid;
            const int64_t r = gi < a.G ? (int64_t)cnt[gi] * rps : 0;
            const int nt = (int)((r + rt - 1) / rt);
            int incl = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(FULL_MASK, incl, o);
                if (tid >= o) incl += y;
            }
            const int lo = base + incl - nt;
            if (tile >= lo && tile < lo + nt) {
                res[0] = gi;
                res[1] = (tile - lo) * rt;
                res[2] = (int)min((int64_t)rt, r - (int64_t)(tile - lo) * rt);
            }
            base += __shfl_sync(FULL_MASK, incl, 31);
            if (base > tile) break;
        }
        __syncwarp();
        if (res[0] >= 0) {
            const int gg = res[0], o0 = res[1] / rps, o1 = (res[1] + res[2] - 1) / rps;
            int ord = 0;
            for (int i0 = 0; i0 < a.S && ord <= o1; i0 += 32) {
                const int i = i0 + tid;
                const bool mine = i < a.S && prefix_of(a, i) == gg;
                const unsigned b = __ballot_sync(FULL_MASK, mine);
                const int o = ord + __popc(b & ((1u << tid) - 1));
                if (mine && o >= o0 && o <= o1) list[o - o0] = i;
                ord += __popc(b);
            }
        }
    }
    __syncthreads();
    g = res[0];
    first = res[1];
    rows = res[2];
    return g >= 0;
}

// Upper bound of the prefix tiles of a call (the groups are on the device).
inline int64_t max_prefix_tiles(int S, int G, int rows_per_seq, int rt) {
    if (G == 0) return 0;
    const int64_t full = (int64_t)S * rows_per_seq / rt;
    return full + (G < S ? G : S);
}

// Row tiles of 128 that a tensor-core block takes.  With one, two blocks share
// an SM and hide each other's beginnings and ends, and the block can sum its
// keys' weights; with two, the row tiles share the copies of K and V.  (d = 128,
// with the weights, one / two: 512 heads of 256 rows 64.1 / 81.9 us, 256 heads of
// 512 rows 80 / 88; 128 heads of 1024 110 / 111; 16 heads of 16004 679 / 649.)
constexpr int ONE_TILE_ROWS = 512;
inline int umma_row_tiles(int64_t rows_per_seq) { return rows_per_seq > ONE_TILE_ROWS ? 2 : 1; }

// Two weights p >= 0 as sums of two bf16 each, hi + lo, packed in pairs: off by at
// most 2^-15 of p (of weights below 2^-119, 2^-134).  hi is cut off from a little less
// than p, so that lo lies between 2^-9 p (less its rounding) and 2^-7 p 5/4, and both
// are above zero wherever p is (down to 2^-124): a product with an infinite value is
// that infinity, where a lo of zero or below gave NaN.
__device__ __forceinline__ void split_weights(float p0, float p1, uint32_t& hi, uint32_t& lo) {
    constexpr float LESS = 1.f - 0x1p-9f;
    hi = __byte_perm(__float_as_uint(p0 * LESS), __float_as_uint(p1 * LESS), 0x7632);
    const __nv_bfloat162 rest = __floats2bfloat162_rn(p0 - __uint_as_float(hi << 16), p1 - __uint_as_float(hi & 0xffff0000u));
    lo = *reinterpret_cast<const uint32_t*>(&rest);
}

// Launches a kernel as a programmatic dependent: its blocks may be set up while
// the kernel in front of it in the stream drains, so it executes
// griddepcontrol.wait before it touches memory, and lets the next launch begin
// only after that.  (The streaming kernel beside the prefixes' one is the
// exception: it starts on that kernel's word.)  A kernel's lifetime so begins before
// what it reads is written: its parameters are not __restrict__ and nothing is read
// by __ldg, which promise data that do not change during the kernel and may be
// moved in front of the wait.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t blocks, int threads, size_t smem, cudaStream_t st, A... args) {
    if (blocks < 1 || blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// launchers (host)
cudaError_t prepare_shared_umma();
cudaError_t launch_attend_umma(const View& a, int d, cudaStream_t st);
cudaError_t launch_column_sums_umma(const View& a, int d, cudaStream_t st);
cudaError_t launch_add_sums(const View& a, cudaStream_t st);
cudaError_t launch_prefix_umma(const View& a, int d, cudaStream_t st);
cudaError_t launch_append(const View& a, int dtype, int d, const void* k_t, const int64_t* kts, const void* v_t,
                          const int64_t* vts, const float* w_t, cudaStream_t st);
// rows_too: the own keys of every row, else the prefixes' tiles alone
cudaError_t launch_attend_f32(const View& a, int d, bool rows_too, cudaStream_t st);
cudaError_t prepare_shared_stream_f32();
cudaError_t launch_stream_f32(const View& a, int d, int warps_per_head, bool beside, cudaStream_t st);
cudaError_t prepare_shared_stream();
// beside: launched right behind the prefixes' kernel, whose end this launch's end includes
cudaError_t launch_stream(const View& a, int d, int warps_per_head, bool beside, cudaStream_t st);
cudaError_t launch_combine(const View& a, int dtype, int d, cudaStream_t st);
cudaError_t launch_column_sums_f32(const View& a, int d, cudaStream_t st);
cudaError_t prepare_shared_f32();
cudaError_t prepare_shared_evict();
size_t evict_bytes(int heads, int cap);
cudaError_t launch_evict(const View& a, int dtype, int d, const int32_t* budget, int recent, int slack,
                         unsigned char* scratch, cudaStream_t st);

}  // namespace shared
}  // namespace hkv
