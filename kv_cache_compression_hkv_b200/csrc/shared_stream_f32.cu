// shared_stream_f32.cu -- attention of up to 8 query rows of one (sequence, KV
// head) over the own keys of a shared-prefix cache, fp32: the decode step.
//
// As in the bf16 kernel every key and value row is read once, so HBM bounds
// it while there are few rows, but products of fp32 stay fp32, on the CUDA
// cores.  A row of K lies across the lanes (16 bytes each; two rows a warp where
// d = 64), and a warp takes eight rows a lane at once.  The lanes' parts of the
// eight dot products are summed by a butterfly that halves the number of
// products with the number of lanes that share one: nine shuffles for eight
// products of 32 lanes, after which a lane holds one key's logit.  Three steps
// of 8 KB a warp are in flight or in use, each lane copying what it uses itself.
//
// d = 128: 1024 heads of 28 to 138 tokens and 64 shared ones 23.9 us (the blocks
// of 16 rows that more rows use: 47.1), 128 heads of 4 rows over 700 to 1000 and
// 512 34.5 (57.8), 12 heads of 8 rows over 9000 to 16001 and 777 52.4 (71.0): 154
// MB, or 3.0 TB/s.  With 8 rows the shuffles and the products (about 900
// instructions for 8 KB) take longer than HBM, with 16 they would take longer
// than those blocks, so they end at 8.  Registers in the place of the stages
// left too little in flight (64.6 us on the first of these).
#include <math.h>

#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"
#include "shared.cuh"

namespace hkv {
namespace shared {

namespace {

constexpr int SW = 4;  // warps of a block
constexpr int NK = 8;  // rows of K and V of a step that a lane holds parts of
constexpr int SN = 3;  // stages of a warp
constexpr int STAGE = 2 * NK * 512;

// v[i]: this lane's part of key i's product.  Returns the whole product of key
// (lane % LPK) / (LPK / NK), summed over the LPK lanes that share the keys.
template <int LPK> __device__ __forceinline__ float butterfly(float (&v)[NK], int lane) {
    int width = LPK / 2;
#pragma unroll
    for (int n = NK / 2; n >= 1; n /= 2, width /= 2) {
        const bool up = lane & width;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(FULL_MASK, give, width);
        }
    }
    for (; width >= 1; width /= 2) v[0] += __shfl_xor_sync(FULL_MASK, v[0], width);
    return v[0];
}

}  // namespace

// WPH warps of a block work on one (sequence, KV head, key range), 1 or 4, as
// in the bf16 kernel; RW: rows of a head, at most.
template <int D, int WPH, int RW>
__global__ void __launch_bounds__(32 * SW, 2) stream_f32_kernel(const __grid_constant__ View a, int beside) {
    constexpr int LPK = D / 4, PER = 32 / LPK, KS = NK * PER;  // lanes of a key, keys side by side, keys of a step
    extern __shared__ __align__(16) unsigned char raw[];
    static_assert(sizeof(float) * RW * D <= SN * STAGE, "a warp's states fit its stages");
    auto state = [&](int w, int u, int c) { return reinterpret_cast<float4*>(raw + w * SN * STAGE + (u * D + c) * 4); };
    __shared__ float2 ml[SW][RW], joined[SW / WPH][RW];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (!beside) ptx::grid_dep_wait();
    ptx::grid_dep_trigger();  // the joining kernel waits for this grid's end
    const int item = blockIdx.x * (SW / WPH) + warp / WPH, wi = warp % WPH;
    const int rps = a.rep * a.T;
    const int64_t R = (int64_t)a.S * a.H * a.T;
    const bool on = item < a.S * a.Hk * a.no;
    const int j = on ? item % a.no : 0, sh = on ? item / a.no : 0;
    const int s = sh / a.Hk, hk = sh % a.Hk;
    const int c0 = lane % LPK * 4, side = lane / LPK;
    float4 q[RW];
#pragma unroll
    for (int u = 0; u < RW; ++u) {
        q[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u < rps) {
            const int t = query_of(a, u);
            const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + s * a.qs[0] +
                                                              (hk * a.rep + u - t * a.rep) * a.qs[1] + t * a.qs[2] + c0);
            q[u] = make_float4(x.x * a.qscale, x.y * a.qscale, x.z * a.qscale, x.w * a.qscale);
        }
    }
    const int n = own_len(a, s, hk);
    const int pg = a.listed ? prefix_of(a, s) : -1;
    const Piece pc = list_piece(prefix_len(a, pg), n, a.no, j);
    const bool final = a.np + a.no == 1;
    const bool work = on && !pc.empty();
    float m[RW], l[RW];
    float4 o[RW];
#pragma unroll
    for (int u = 0; u < RW; ++u) {
        m[u] = -INFINITY;
        l[u] = 0.f;
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (work) {
        const float* kb = static_cast<const float*>(a.k) + s * a.ks[0] + hk * a.ks[1] + c0;
        const float* vb = static_cast<const float*>(a.v) + s * a.vs[0] + hk * a.vs[1] + c0;
        const float* pkb = static_cast<const float*>(a.pk) + (pg < 0 ? 0 : pg) * a.pks[0] + hk * a.pks[1] + c0;
        const float* pvb = static_cast<const float*>(a.pv) + (pg < 0 ? 0 : pg) * a.pvs[0] + hk * a.pvs[1] + c0;
        const int psteps = (pc.pb - pc.pa + KS - 1) / KS, steps = psteps + (pc.ob - pc.oa + KS - 1) / KS;
        // A lane copies the pieces that it uses itself: piece e of a step is of key
        // e PER + side; zeros past the last key.
        const uint32_t ring = ptx::smem_u32(raw) + warp * SN * STAGE + lane * 16;
        auto load = [&](int i) {  // this warp's i-th step
            const int st = i * WPH + wi;
            if (st < steps) {
                const bool pre = st < psteps;
                const int k0 = (pre ? pc.pa + st * KS : pc.oa + (st - psteps) * KS) + side, hi = pre ? pc.pb : pc.ob;
                const int64_t kst = pre ? a.pks[2] : a.ks[2], vst = pre ? a.pvs[2] : a.vs[2];
                const float *kp = (pre ? pkb : kb) + k0 * kst, *vp = (pre ? pvb : vb) + k0 * vst;
                const uint32_t dst = ring + i % SN * STAGE;
#pragma unroll
                for (int e = 0; e < NK; ++e) {
                    const bool in = k0 + e * PER < hi;
                    cp16(dst + e * 512, in ? kp + e * PER * kst : kb, in);
                    cp16(dst + (NK + e) * 512, in ? vp + e * PER * vst : vb, in);
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
#pragma unroll
        for (int i = 0; i < SN - 1; ++i) load(i);
        // the key of a step whose logit this lane comes to hold, and whether it is the first such lane
        const int mine = lane % LPK / (LPK / NK) * PER + side;
        const bool first = lane % (LPK / NK) == 0;
        for (int i = 0; i * WPH + wi < steps; ++i) {
            const int at = i * WPH + wi;
            const bool pre = at < psteps;
            const int k0 = pre ? pc.pa + at * KS : pc.oa + (at - psteps) * KS, hi = pre ? pc.pb : pc.ob, key = k0 + mine;
            asm volatile("cp.async.wait_group %0;" ::"n"(SN - 2) : "memory");
            load(i + SN - 1);  // into the stage of step i - 1
            const float4* kr = reinterpret_cast<const float4*>(raw + (warp * SN + i % SN) * STAGE) + lane;
            const float4* vr = kr + NK * 32;
            float x[RW], mx[RW];
            float4 y[NK];
#pragma unroll
            for (int e = 0; e < NK; ++e) y[e] = kr[e * 32];
#pragma unroll
            for (int u = 0; u < RW; ++u) {
                float v[NK];
#pragma unroll
                for (int e = 0; e < NK; ++e)
                    v[e] = fmaf(y[e].x, q[u].x, fmaf(y[e].y, q[u].y, fmaf(y[e].z, q[u].z, y[e].w * q[u].w)));
                x[u] = butterfly<LPK>(v, lane);
            }
#pragma unroll
            for (int e = 0; e < NK; ++e) y[e] = vr[e * 32];
#pragma unroll
            for (int u = 0; u < RW; ++u) {
                x[u] = key < hi && (pre || key < own_limit(a, n, u)) ? x[u] : -INFINITY;
                if (a.logit && first && !pre && key < hi && u < rps) a.logit[((int64_t)sh * rps + u) * a.lcap + key] = x[u];
                mx[u] = x[u];
            }
#pragma unroll
            for (int off = 16; off >= LPK / NK; off /= 2)
#pragma unroll
                for (int u = 0; u < RW; ++u) mx[u] = fmaxf(mx[u], __shfl_xor_sync(FULL_MASK, mx[u], off));
#pragma unroll
            for (int u = 0; u < RW; ++u) {
                const float mn = fmaxf(mx[u], m[u]);
                const float mb = mn == -INFINITY ? 0.f : mn, alpha = exp2f(m[u] - mb);
                m[u] = mn;
                x[u] = exp2f(x[u] - mb);
                l[u] = fmaf(l[u], alpha, x[u]);  // each lane its own keys; summed at the end
                o[u].x *= alpha; o[u].y *= alpha; o[u].z *= alpha; o[u].w *= alpha;
            }
#pragma unroll
            for (int e = 0; e < NK; ++e) {
#pragma unroll
                for (int u = 0; u < RW; ++u) {
                    const float p = __shfl_sync(FULL_MASK, x[u], side * LPK + e * (LPK / NK));
                    o[u].x = fmaf(p, y[e].x, o[u].x);
                    o[u].y = fmaf(p, y[e].y, o[u].y);
                    o[u].z = fmaf(p, y[e].z, o[u].z);
                    o[u].w = fmaf(p, y[e].w, o[u].w);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
        for (int u = 0; u < RW; ++u) {
#pragma unroll
            for (int off = 16; off >= 1; off /= 2)
                if (off >= LPK / NK) l[u] += __shfl_xor_sync(FULL_MASK, l[u], off);
            if (PER == 2) {
                o[u].x += __shfl_xor_sync(FULL_MASK, o[u].x, 16);
                o[u].y += __shfl_xor_sync(FULL_MASK, o[u].y, 16);
                o[u].z += __shfl_xor_sync(FULL_MASK, o[u].z, 16);
                o[u].w += __shfl_xor_sync(FULL_MASK, o[u].w, 16);
            }
            // (a sum of NaN logits alone must not pass for an empty row)
            if (l[u] != l[u] && m[u] == -INFINITY) m[u] = 0.f;
        }
    }
    // the warps' states of the rows, joined by the warps of the head
    __syncwarp();  // (into the warp's stages: every lane has left them)
#pragma unroll
    for (int u = 0; u < RW; ++u) {
        if (lane == 0) ml[warp][u] = make_float2(m[u], l[u]);
        if (side == 0) *state(warp, u, c0) = o[u];
    }
    if (WPH == 1) __syncwarp();
    else __syncthreads();
    if (work || (final && on)) {
        const int w0 = warp / WPH * WPH, slot = a.np + j;  // w0: the head's first warp
        for (int e = wi * 32 + lane; e < rps * LPK; e += 32 * WPH) {
            const int i = e / LPK, c = e % LPK * 4;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int v = 0; v < WPH; ++v) M = fmaxf(M, ml[w0 + v][i].x);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < WPH; ++v) {
                const float2 y = ml[w0 + v][i];
                const float f = y.x == -INFINITY ? 0.f : exp2f(y.x - M);
                const float4 z = *state(w0 + v, i, c);
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
                float* po = static_cast<float*>(a.out) + s * a.os[0] + (hk * a.rep + i - t * a.rep) * a.os[1] + t * a.os[2] + c;
                *reinterpret_cast<float4*>(po) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
                if (c == 0) {
                    if (a.lse) a.lse[row] = some ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
                    joined[warp / WPH][i] = make_float2(M, inv);
                }
            } else {
                *reinterpret_cast<float4*>(a.part_o + (slot * R + row) * D + c) = acc;
                if (c == 0) a.part_ml[ml_index(a, row, slot)] = make_float2(M, L);
            }
        }
    }
    if (final && a.logit) {  // (the same for the whole block)
        __syncthreads();     // the kept logits too
        if (on) add_kept(a, sh, n, joined[warp / WPH], wi * 32 + lane, 32 * WPH);
    }
    // this grid ends after the one it was launched beside (the prefixes')
    if (beside) ptx::grid_dep_wait();
}

cudaError_t launch_stream_f32(const View& a, int d, int warps_per_head, bool beside, cudaStream_t st) {
    const int rps = a.rep * a.T;
    const int64_t items = (int64_t)a.S * a.Hk * a.no, per = SW / warps_per_head;
    const int64_t blocks = (items + per - 1) / per;
    auto rows = [&](auto dim, auto wph) {
        constexpr int D = decltype(dim)::value, W = decltype(wph)::value;
        auto go = [&](auto kernel) { return launch(kernel, blocks, 32 * SW, SW * SN * STAGE, st, a, (int)beside); };
        if (rps == 1) return go(stream_f32_kernel<D, W, 1>);
        if (rps == 2) return go(stream_f32_kernel<D, W, 2>);
        return rps <= 4 ? go(stream_f32_kernel<D, W, 4>) : go(stream_f32_kernel<D, W, STREAM_ROWS_F32>);
    };
    auto warps = [&](auto dim) {
        return warps_per_head == 1 ? rows(dim, std::integral_constant<int, 1>()) : rows(dim, std::integral_constant<int, 4>());
    };
    return d == 128 ? warps(std::integral_constant<int, 128>()) : warps(std::integral_constant<int, 64>());
}

cudaError_t prepare_shared_stream_f32() {
    cudaError_t e = cudaSuccess;
    auto set = [&](auto kernel) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SW * SN * STAGE);
    };
    auto all = [&](auto dim, auto wph) {
        constexpr int D = decltype(dim)::value, W = decltype(wph)::value;
        set(stream_f32_kernel<D, W, 1>);
        set(stream_f32_kernel<D, W, 2>);
        set(stream_f32_kernel<D, W, 4>);
        set(stream_f32_kernel<D, W, STREAM_ROWS_F32>);
    };
    all(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    all(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
    all(std::integral_constant<int, 128>(), std::integral_constant<int, 1>());
    all(std::integral_constant<int, 128>(), std::integral_constant<int, 4>());
    return e;
}

}  // namespace shared
}  // namespace hkv
