// shared_evict.cu -- eviction by accumulated weight from a shared-prefix cache.
//
// A due head (len n >= budget B + slack) loses the E = n - B tokens lowest in
// (recent, weight, position, slot).  The first two fields fold into 32 bits
// that order like them (ordered float bits; all recent tokens share the
// highest value), the position into 32 more: the E-th smallest of these
// 64-bit keys is found by a most-significant-digit radix select, and among
// tokens with that same key the lower slots go.
#include "kernels.h"
#include "shared.cuh"

namespace hkv {
namespace shared {

// Bits that order as (recent, weight): recent tokens highest, then NaN, then
// the numbers (-0 as +0).
__device__ __forceinline__ uint32_t class_bits(float w, bool recent) {
    if (recent) return 0xffffffffu;
    if (w != w) return 0xfffffffeu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr int ET = 256;

__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(FULL_MASK, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < ET / 32; ++w) {
        const int v = warp_sums[w];
        if (w < warp) before += v;
        all += v;
    }
    total = all;
    return before + incl - x;
}

// One block per (sequence, KV head).
__global__ void __launch_bounds__(ET) evict_simple_kernel(View a, const int32_t* __restrict__ budget, int recent,
                                                          int slack, int row_bytes, int es,
                                                          int32_t* __restrict__ holes) {
    __shared__ int hist[256];
    __shared__ int warp_sums[ET / 32];
    __shared__ int newest_s, digit_s, below_s;
    const int head = blockIdx.x, s = head / a.Hk, hk = head % a.Hk, tid = threadIdx.x;
    const int n = own_len(a, s, hk), B = max(0, budget[head]);
    if ((int64_t)n < (int64_t)B + slack) return;
    const int E = n - B;
    int32_t* pos = a.pos + (int64_t)head * a.cap;
    float* weight = a.weight + (int64_t)head * a.cap;
    if (tid == 0) newest_s = INT32_MIN;
    __syncthreads();
    int nw = INT32_MIN;
    for (int i = tid; i < n; i += ET) nw = max(nw, pos[i]);
    atomicMax(&newest_s, nw);
    __syncthreads();
    const int64_t newest = newest_s;
    auto key = [&](int i) {
        const int p = pos[i];
        return ((uint64_t)class_bits(weight[i], newest - p < recent) << 32) | ((uint32_t)p ^ 0x80000000u);
    };
    // the E-th smallest key, digit by digit
    uint64_t prefix = 0, mask = 0;
    int want = E;
    for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += ET) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += ET) {
            const uint64_t k = key(i);
            if ((k & mask) == prefix) atomicAdd(hist + (int)(k >> shift & 255), 1);
        }
        __syncthreads();
        int total;
        const int c = hist[tid], below = block_scan(c, warp_sums, total);
        if (below < want && want <= below + c) {
            digit_s = tid;
            below_s = below;
        }
        __syncthreads();
        want -= below_s;
        prefix |= (uint64_t)digit_s << shift;
        mask |= (uint64_t)255 << shift;
    }
    // evicted: key < prefix, or key == prefix and among the first `want` of
    // those by slot.  Holes (evicted below B) are listed in slot order; the
    // survivors at or above B take them in slot order.
    int32_t* hl = holes + (int64_t)head * a.cap;
    int eq_seen = 0, n_holes = 0, n_movers = 0;
    unsigned char* kb = static_cast<unsigned char*>(a.k) + (s * a.ks[0] + hk * a.ks[1]) * es;
    unsigned char* vb = static_cast<unsigned char*>(a.v) + (s * a.vs[0] + hk * a.vs[1]) * es;
    for (int i0 = 0; i0 < n; i0 += ET) {
        const int i = i0 + tid;
        const uint64_t k = i < n ? key(i) : ~0ull;
        const bool eq = i < n && k == prefix;
        int total;
        const int er = block_scan(eq, warp_sums, total);
        const bool gone = i < n && (k < prefix || (eq && eq_seen + er < want));
        eq_seen += total;
        const bool hole = gone && i < B;
        const int hr = block_scan(hole, warp_sums, total);
        if (hole) hl[n_holes + hr] = i;
        n_holes += total;
        const bool mover = i < n && !gone && i >= B;
        const int mr = block_scan(mover, warp_sums, total);
        if (mover) hl[B + n_movers + mr] = i;
        n_movers += total;
    }
    __syncthreads();
    // (as many movers as holes, at most min(B, E))
    for (int i = tid; i < n_movers; i += ET) {
        const int from = hl[B + i], to = hl[i];
        pos[to] = pos[from];
        weight[to] = weight[from];
    }
    const int pieces = row_bytes / 16;
    for (int e = tid; e < n_movers * pieces; e += ET) {
        const int i = e / pieces, c = e % pieces * 16;
        const int64_t from = hl[B + i], to = hl[i];
        *reinterpret_cast<uint4*>(kb + to * a.ks[2] * es + c) = *reinterpret_cast<uint4*>(kb + from * a.ks[2] * es + c);
        *reinterpret_cast<uint4*>(vb + to * a.vs[2] * es + c) = *reinterpret_cast<uint4*>(vb + from * a.vs[2] * es + c);
    }
    if (tid == 0) a.len[head] = B;
}

cudaError_t launch_evict(const View& a, int dtype, int d, const int32_t* budget, int recent, int slack,
                         int32_t* holes, cudaStream_t st) {
    const int es = dtype == HKV_DTYPE_F32 ? 4 : 2;
    evict_simple_kernel<<<a.S * a.Hk, ET, 0, st>>>(a, budget, recent, slack, d * es, es, holes);
    return cudaGetLastError();
}

}  // namespace shared
}  // namespace hkv
