// shared_stream.cu -- attention of few query rows (up to 16 of one (sequence,
// KV head)) over the own keys of a shared-prefix cache, bf16: the decode step.
//
// Every key and value row is read once and used for at most 16 rows, so the
// kernel is bound by HBM: a warp keeps three stages of 16 rows of K and V in
// flight (cp.async, 16-byte pieces at a swizzled place; TMA boxes of 16 rows
// took 16.1 us where these take 11.0, on 1024 heads of 28 to 138 tokens of
// d = 128) and works on the oldest with mma.sync m16n8k16: S = Q K^T with the rows on the M side, the
// weights straight from S's registers as the A operand of O += P V.  (A
// tcgen05 tile would compute 128 rows for these 16 and pass the weights
// through TMEM; at 8 KB of keys and values a step the legacy instruction's
// rate is a third of what HBM leaves time for.)
#include <math.h>

#include "kernels.h"
#include "ptx.cuh"
#include "shared.cuh"
#include "umma.cuh"

namespace hkv {
namespace shared {

namespace {

constexpr int SK = 16;   // keys of a step
constexpr int SN = 3;    // stages of a warp
constexpr int SW = 4;    // warps of a block
constexpr float RAISE = 16.f;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float x, float y) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t*>(&h);
}

}  // namespace

template <int D> constexpr int stream_smem() { return SW * SN * 2 * SK * D * 2; }

// WPH warps of a block work on one (sequence, KV head, key range): 1 (four
// heads a block, nothing to join) or 4 (steps dealt out in turn, joined in
// shared memory).  LOW: at most 8 rows, the upper half of the M side is empty.
// Where the item has all of the rows' keys (no splits, the prefix listed with
// the own keys) the results are final, the accumulated weights too.
template <int D, int WPH, bool LOW>
__global__ void __launch_bounds__(32 * SW) stream_attend_kernel(const __grid_constant__ View a, int beside) {
    extern __shared__ __align__(1024) unsigned char raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!beside) ptx::grid_dep_wait();
    ptx::grid_dep_trigger();  // the joining kernel waits for this grid's end
    const int item = blockIdx.x * (SW / WPH) + warp / WPH, wi = warp % WPH;
    const int rps = a.rep * a.T;
    const int64_t R = (int64_t)a.S * a.H * a.T;
    const bool on = item < a.S * a.Hk * a.no;
    const int j = on ? item % a.no : 0, sh = on ? item / a.no : 0;
    const int s = sh / a.Hk, hk = sh % a.Hk;
    const int n = own_len(a, s, hk);
    // this item's keys: a piece of the prefix's (where they are listed with the
    // own ones, see the caller) and of the own
    const int pg = a.listed ? prefix_of(a, s) : -1;
    const Piece pc = list_piece(prefix_len(a, pg), n, a.no, j);
    const bool final = a.np + a.no == 1;
    const bool work = on && !pc.empty();
    constexpr int CH = D / 8;  // 16-byte pieces of a row
    constexpr int NT = LOW ? 1 : 2;

    // accumulators: 16 rows x D, fragments of 8 columns
    float o[D / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    const int g = lane >> 2, q2 = (lane & 3) * 2;  // this thread's rows g, g + 8; columns q2, q2 + 1

    if (work) {
        const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(a.k) + s * a.ks[0] + hk * a.ks[1];
        const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(a.v) + s * a.vs[0] + hk * a.vs[1];
        const uint32_t stage0 = ptx::smem_u32(raw) + warp * SN * 2 * SK * D * 2;
        const __nv_bfloat16* pkb = static_cast<const __nv_bfloat16*>(a.pk) + (pg < 0 ? 0 : pg) * a.pks[0] + hk * a.pks[1];
        const __nv_bfloat16* pvb = static_cast<const __nv_bfloat16*>(a.pv) + (pg < 0 ? 0 : pg) * a.pvs[0] + hk * a.pvs[1];
        const int psteps = (pc.pb - pc.pa + SK - 1) / SK, steps = psteps + (pc.ob - pc.oa + SK - 1) / SK;
        const int mine = wi < steps ? (steps - wi + WPH - 1) / WPH : 0;
        auto load = [&](int i) {  // this warp's i-th step
            if (i < mine) {
                const int st = i * WPH + wi;
                const bool pre = st < psteps;
                const int k0 = pre ? pc.pa + st * SK : pc.oa + (st - psteps) * SK, hi = pre ? pc.pb : pc.ob;
                const __nv_bfloat16 *kp = pre ? pkb : kb, *vp = pre ? pvb : vb;
                const int64_t kst = pre ? a.pks[2] : a.ks[2], vst = pre ? a.pvs[2] : a.vs[2];
                const uint32_t kd = stage0 + (i % SN) * 2 * SK * D * 2, vd = kd + SK * D * 2;
#pragma unroll
                for (int e = 0; e < SK * CH / 32; ++e) {
                    const int idx = e * 32 + lane, r = idx / CH, c = idx % CH;
                    const bool in = k0 + r < hi;
                    const int64_t key = in ? k0 + r : k0;
                    const uint32_t off = r * (D * 2) + ((c ^ (r & 7)) << 4);
                    cp16(kd + off, kp + key * kst + c * 8, in);
                    cp16(vd + off, vp + key * vst + c * 8, in);
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < SN - 1; ++i) load(i);
        // Q fragments
        uint32_t qa[D / 16][4];
        int lim[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = g + 8 * u;
            const bool live = i < rps && u < NT;
            lim[u] = live ? min(pc.ob, own_limit(a, n, i)) : 0;
            const int t = query_of(a, i);
            const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + s * a.qs[0] +
                                      (hk * a.rep + i - t * a.rep) * a.qs[1] + t * a.qs[2];
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qa[kk][u] = live ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + q2) : 0u;
                qa[kk][2 + u] = live ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + q2 + 8) : 0u;
            }
        }
        float* lrow[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
            lrow[u] = a.logit && g + 8 * u < rps && u < NT ? a.logit + ((int64_t)sh * rps + g + 8 * u) * a.lcap : nullptr;
        for (int i = 0; i < mine; ++i) {
            cp_wait<SN - 2>();
            __syncwarp();
            load(i + SN - 1);  // into the stage of step i - 1, which every lane has left
            const int st = i * WPH + wi;
            const bool pre = st < psteps;
            const int k0 = pre ? pc.pa + st * SK : pc.oa + (st - psteps) * SK, hi = pre ? pc.pb : pc.ob;
            const uint32_t ks = stage0 + (i % SN) * 2 * SK * D * 2, vs = ks + SK * D * 2;
            float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            {
                const int r = ((lane >> 4) << 3) + (lane & 7), cb = (lane >> 3) & 1;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b[4];
                    ldsm4(ks + r * (D * 2) + (((kk * 2 + cb) ^ (r & 7)) << 4), b);
                    mma16816(x[0], qa[kk], b[0], b[1]);
                    mma16816(x[1], qa[kk], b[2], b[3]);
                }
            }
            // x[h][2u + e]: row g + 8u, key k0 + 8h + q2 + e
            float mt[2];
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                mt[u] = -INFINITY;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int key = k0 + 8 * h + q2;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float& y = x[h][2 * u + e];
                        y = key + e < (pre ? hi : lim[u]) ? y * a.qscale : -INFINITY;
                        mt[u] = fmaxf(mt[u], y);
                    }
                    if (lrow[u] && !pre && key < hi)
                        *reinterpret_cast<float2*>(lrow[u] + key) = make_float2(x[h][2 * u], x[h][2 * u + 1]);
                }
            }
            bool up = mt[0] > m[0] + RAISE;
            if (NT == 2) up |= mt[NT - 1] > m[NT - 1] + RAISE;
            if (__any_sync(FULL_MASK, up)) {
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    float t = mt[u];
                    t = fmaxf(t, __shfl_xor_sync(FULL_MASK, t, 1));
                    t = fmaxf(t, __shfl_xor_sync(FULL_MASK, t, 2));
                    const float mn = fmaxf(m[u], t);
                    const float alpha = mn == -INFINITY ? 1.f : exp2f(m[u] - mn);
                    l[u] *= alpha;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c) {
                        o[c][2 * u] *= alpha;
                        o[c][2 * u + 1] *= alpha;
                    }
                    m[u] = mn;
                }
            }
            uint32_t pa[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const float mb = m[u] == -INFINITY ? 0.f : m[u];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = tc::ex2(x[h][2 * u] - mb), p1 = tc::ex2(x[h][2 * u + 1] - mb);
                    l[u] += p0 + p1;
                    pa[2 * h + u] = pack(p0, p1);
                }
            }
            {
                const int r = ((lane >> 3) & 1) * 8 + (lane & 7), cb = lane >> 4;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t b[4];
                    ldsm4t(vs + r * (D * 2) + (((c * 2 + cb) ^ (r & 7)) << 4), b);
                    mma16816(o[2 * c], pa, b[0], b[1]);
                    mma16816(o[2 * c + 1], pa, b[2], b[3]);
                }
            }
        }
        cp_wait<0>();
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            l[u] += __shfl_xor_sync(FULL_MASK, l[u], 1);
            l[u] += __shfl_xor_sync(FULL_MASK, l[u], 2);
            // (a sum of NaN logits alone must not pass for an empty row)
            if (l[u] != l[u] && m[u] == -INFINITY) m[u] = 0.f;
        }
    }
    const int slot = a.np + j;
    const float* lg = a.logit + (int64_t)sh * rps * a.lcap;
    float* w = a.weight + (int64_t)sh * a.cap;
    if constexpr (WPH == 1) {
        if (final) {
            // the warp has all of its rows' keys
            float inv[2] = {0.f, 0.f};
            if (on) {
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    const int i = g + 8 * u;
                    if (i >= rps) continue;
                    const bool some = !(m[u] == -INFINITY);
                    inv[u] = some ? 1.f / l[u] : 0.f;
                    const int t = query_of(a, i), h = hk * a.rep + i - t * a.rep;
                    __nv_bfloat16* po = static_cast<__nv_bfloat16*>(a.out) + s * a.os[0] + h * a.os[1] + t * a.os[2] + q2;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        *reinterpret_cast<uint32_t*>(po + c * 8) = pack(o[c][2 * u] * inv[u], o[c][2 * u + 1] * inv[u]);
                    if ((lane & 3) == 0 && a.lse)
                        a.lse[row_index(a, s, h, t)] = some ? (m[u] + log2f(l[u])) * 0.6931471805599453f : -INFINITY;
                }
                if (a.logit) {
                    __syncwarp();  // the logits that other lanes kept
                    for (int k0 = 0; k0 < n; k0 += 32) {
                        const int key = k0 + lane;
                        float sum = 0.f;
                        for (int i = 0; i < rps; ++i) {
                            const float M = __shfl_sync(FULL_MASK, i < 8 ? m[0] : m[1], (i & 7) * 4);
                            const float f = __shfl_sync(FULL_MASK, i < 8 ? inv[0] : inv[1], (i & 7) * 4);
                            if (key < n && M != -INFINITY) sum += exp2f(lg[(int64_t)i * a.lcap + key] - M) * f;
                        }
                        if (key < n) w[key] += sum;
                    }
                }
            }
        } else if (work) {
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const int i = g + 8 * u;
                if (i >= rps) continue;
                const int64_t row = row_of(a, s, hk, i);
                if ((lane & 3) == 0) a.part_ml[ml_index(a, row, slot)] = make_float2(m[u], l[u]);
                float* po = a.part_o + (slot * R + row) * D + q2;
#pragma unroll
                for (int c = 0; c < D / 8; ++c)
                    *reinterpret_cast<float2*>(po + c * 8) = make_float2(o[c][2 * u], o[c][2 * u + 1]);
            }
        }
    } else {
        // the four warps' states of the rows, joined by the block
        constexpr int ROWS = LOW ? 8 : 16, PITCH = D + 8;
        static_assert(SW * ROWS * PITCH * 4 <= stream_smem<D>(), "the states fit the stages");
        __shared__ float2 ml[SW][ROWS], joined[ROWS];
        float* st = reinterpret_cast<float*>(raw);
        __syncthreads();  // every warp has left its stages
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            const int i = g + 8 * u;
            if ((lane & 3) == 0) ml[warp][i] = make_float2(m[u], l[u]);
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                *reinterpret_cast<float2*>(st + (warp * ROWS + i) * PITCH + c * 8 + q2) =
                    make_float2(o[c][2 * u], o[c][2 * u + 1]);
        }
        __syncthreads();
        if (work || (final && on)) {
            for (int e = tid; e < min(ROWS, rps) * (D / 4); e += 32 * SW) {
                const int i = e / (D / 4), c = e % (D / 4) * 4;
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int w = 0; w < SW; ++w) M = fmaxf(M, ml[w][i].x);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < SW; ++w) {
                    const float2 y = ml[w][i];
                    const float f = y.x == -INFINITY ? 0.f : exp2f(y.x - M);
                    const float4 z = *reinterpret_cast<const float4*>(st + (w * ROWS + i) * PITCH + c);
                    if (f != 0.f) {
                        L = fmaf(y.y, f, L);
                        acc.x = fmaf(z.x, f, acc.x);
                        acc.y = fmaf(z.y, f, acc.y);
                        acc.z = fmaf(z.z, f, acc.z);
                        acc.w = fmaf(z.w, f, acc.w);
                    }
                }
                const int64_t row = row_of(a, s, hk, i);
                if (final) {
                    const bool some = !(M == -INFINITY);
                    const float inv = some ? 1.f / L : 0.f;
                    const int t = query_of(a, i);
                    __nv_bfloat16* po = static_cast<__nv_bfloat16*>(a.out) + s * a.os[0] +
                                        (hk * a.rep + i - t * a.rep) * a.os[1] + t * a.os[2] + c;
                    *reinterpret_cast<uint2*>(po) = make_uint2(pack(acc.x * inv, acc.y * inv), pack(acc.z * inv, acc.w * inv));
                    if (c == 0) {
                        if (a.lse) a.lse[row] = some ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
                        joined[i] = make_float2(M, inv);
                    }
                } else {
                    *reinterpret_cast<float4*>(a.part_o + (slot * R + row) * D + c) = acc;
                    if (c == 0) a.part_ml[ml_index(a, row, slot)] = make_float2(M, L);
                }
            }
        }
        if (final && a.logit) {  // (the same for the whole block)
            __syncthreads();
            if (on)
                for (int key = tid; key < n; key += 32 * SW) {
                    float sum = 0.f;
                    for (int i = 0; i < rps; ++i) {
                        const float2 y = joined[i];
                        if (y.x != -INFINITY) sum += exp2f(lg[(int64_t)i * a.lcap + key] - y.x) * y.y;
                    }
                    w[key] += sum;
                }
        }
    }
    // this grid ends after the one it was launched beside (the prefixes')
    if (beside) ptx::grid_dep_wait();
}

cudaError_t launch_stream(const View& a, int d, int warps_per_head, bool beside, cudaStream_t st) {
    const int rps = a.rep * a.T;
    const int64_t items = (int64_t)a.S * a.Hk * a.no, per = SW / warps_per_head;
    const int64_t blocks = (items + per - 1) / per;
    auto run = [&](auto kernel) {
        return launch(kernel, blocks, 32 * SW, d == 128 ? stream_smem<128>() : stream_smem<64>(), st, a, (int)beside);
    };
    const bool low = rps <= 8, one = warps_per_head == 1;
    if (d == 128)
        return one ? (low ? run(stream_attend_kernel<128, 1, true>) : run(stream_attend_kernel<128, 1, false>))
                   : (low ? run(stream_attend_kernel<128, 4, true>) : run(stream_attend_kernel<128, 4, false>));
    return one ? (low ? run(stream_attend_kernel<64, 1, true>) : run(stream_attend_kernel<64, 1, false>))
               : (low ? run(stream_attend_kernel<64, 4, true>) : run(stream_attend_kernel<64, 4, false>));
}

cudaError_t prepare_shared_stream() {
    cudaError_t e = cudaSuccess;
    auto set = [&](auto kernel, int smem) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    };
    set(stream_attend_kernel<128, 1, true>, stream_smem<128>());
    set(stream_attend_kernel<128, 1, false>, stream_smem<128>());
    set(stream_attend_kernel<128, 4, true>, stream_smem<128>());
    set(stream_attend_kernel<128, 4, false>, stream_smem<128>());
    set(stream_attend_kernel<64, 1, true>, stream_smem<64>());
    set(stream_attend_kernel<64, 1, false>, stream_smem<64>());
    set(stream_attend_kernel<64, 4, true>, stream_smem<64>());
    set(stream_attend_kernel<64, 4, false>, stream_smem<64>());
    return e;
}

}  // namespace shared
}  // namespace hkv
