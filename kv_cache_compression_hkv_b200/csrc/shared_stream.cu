// shared_stream.cu -- attention of few query rows (up to 16 of one (sequence,
// KV head)) over the own keys of a shared-prefix cache, bf16: the decode step.
//
// Every key and value row is read once and used for at most 16 rows, so the
// kernel is bound by HBM: a warp keeps three stages of 16 rows of K and V in
// flight (cp.async, 16-byte pieces at a swizzled place; TMA boxes of 16 rows
// took 16.1 us where these take 11.0, on 1024 heads of 28 to 138 tokens of
// d = 128) and works on the oldest with mma.sync m16n8k16: S = Q K^T with the
// rows on the M side, the weights straight from S's registers as the A operand
// of O += P V.  (A tcgen05 tile would compute 128 rows for these 16 and pass
// the weights through TMEM; at 8 KB of keys and values a step the legacy
// instruction takes a third of the time that HBM leaves for it.)
// d = 128: 1024 heads of 28 to 138 own tokens and 64 shared ones 12.8 us, 512 of
// 56 to 477 and 128 17.0 us (15.4 and 20.3 with their rows in HBM); 12 heads of 8
// rows over 9000 to 32001 30.3 us with the joining, 126 MB.
#include <math.h>

#include <type_traits>

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
// shared memory).  LOW: at most 8 rows; the upper half of the M side takes what
// the weights' first 8 bits leave (as weights of their own, added up at the
// end), which with more rows is a second product.  With the weights rounded alone
// the outputs were off by as much again as by their own rounding.
// Where the item has all of the rows' keys (no splits, the prefix listed with
// the own keys) the results are final, the accumulated weights too.
template <int D, int WPH, bool LOW>
__global__ void __launch_bounds__(32 * SW, 2) stream_attend_kernel(const __grid_constant__ View a, int beside) {
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
    constexpr int NT = LOW ? 1 : 2;
    const int g = lane >> 2, q2 = (lane & 3) * 2;  // this thread's rows g, g + 8; columns q2, q2 + 1
    // Q fragments (on their way while the lengths are looked up)
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = g + 8 * u;
        const bool live = on && i < rps && u < NT;
        const int t = query_of(a, i);
        const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(a.q) + s * a.qs[0] + (hk * a.rep + i - t * a.rep) * a.qs[1] +
                                  t * a.qs[2];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            qa[kk][u] = live ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + q2) : 0u;
            qa[kk][2 + u] = live ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + q2 + 8) : 0u;
        }
    }
    const int n = own_len(a, s, hk);
    // this item's keys: a piece of the prefix's (where they are listed with the
    // own ones, see the caller) and of the own
    const int pg = a.listed ? prefix_of(a, s) : -1;
    const Piece pc = list_piece(prefix_len(a, pg), n, a.no, j);
    const bool final = a.np + a.no == 1;
    const bool work = on && !pc.empty();
    constexpr int CH = D / 8;  // 16-byte pieces of a row

    // accumulators: 16 rows x D, fragments of 8 columns
    float o[D / 8][4];
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][e] = 0.f;

    if (work) {
        const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(a.k) + s * a.ks[0] + hk * a.ks[1];
        const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(a.v) + s * a.vs[0] + hk * a.vs[1];
        const uint32_t stage0 = ptx::smem_u32(raw) + warp * SN * 2 * SK * D * 2;
        const __nv_bfloat16* pkb = static_cast<const __nv_bfloat16*>(a.pk) + (pg < 0 ? 0 : pg) * a.pks[0] + hk * a.pks[1];
        const __nv_bfloat16* pvb = static_cast<const __nv_bfloat16*>(a.pv) + (pg < 0 ? 0 : pg) * a.pvs[0] + hk * a.pvs[1];
        const int psteps = (pc.pb - pc.pa + SK - 1) / SK, steps = psteps + (pc.ob - pc.oa + SK - 1) / SK;
        const int mine = wi < steps ? (steps - wi + WPH - 1) / WPH : 0;
        // A lane's pieces of a step: piece c0 of rows r0, r0 + RPI, ...; in shared
        // memory piece c of row r lies at r (2 D) + ((c ^ (r & 7)) << 4).  Rows are
        // a power of two apart, so both come from one place by adding and xoring
        // constants (with a multiplication for each piece the step took 500
        // instructions instead of 370).
        constexpr int RPI = 32 / CH, ITER = SK / RPI;
        const int r0 = lane / CH, c0 = lane % CH;
        const uint32_t dst0 = stage0 + r0 * (D * 2) + ((c0 ^ r0) << 4);
        auto load = [&](int i) {  // this warp's i-th step
            if (i < mine) {
                const int st = i * WPH + wi;
                const bool pre = st < psteps;
                const int k0 = pre ? pc.pa + st * SK : pc.oa + (st - psteps) * SK, hi = pre ? pc.pb : pc.ob;
                const int64_t kst = pre ? a.pks[2] : a.ks[2], vst = pre ? a.pvs[2] : a.vs[2];
                const __nv_bfloat16* kp = (pre ? pkb : kb) + (k0 + r0) * kst + c0 * 8;
                const __nv_bfloat16* vp = (pre ? pvb : vb) + (k0 + r0) * vst + c0 * 8;
                const uint32_t kd = dst0 + (i % SN) * 2 * SK * D * 2;
                if (k0 + SK <= hi) {
#pragma unroll
                    for (int e = 0; e < ITER; ++e) {
                        const uint32_t d = (kd ^ ((e * RPI & 7) << 4)) + e * RPI * (D * 2);
                        cp16(d, kp, true);
                        cp16(d + SK * D * 2, vp, true);
                        kp += RPI * kst;
                        vp += RPI * vst;
                    }
                } else {  // rows past the last key: zeros
#pragma unroll
                    for (int e = 0; e < ITER; ++e) {
                        const uint32_t d = (kd ^ ((e * RPI & 7) << 4)) + e * RPI * (D * 2);
                        const bool in = k0 + r0 + e * RPI < hi;
                        cp16(d, in ? kp + e * RPI * kst : kb, in);
                        cp16(d + SK * D * 2, in ? vp + e * RPI * vst : vb, in);
                    }
                }
            }
            cp_commit();
        };
#pragma unroll
        for (int i = 0; i < SN - 1; ++i) load(i);
        int lim[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) lim[u] = g + 8 * u < rps && u < NT ? min(pc.ob, own_limit(a, n, g + 8 * u)) : 0;
        // where a lane's row addresses of K's and V's fragments start: pieces 2 kk + cb of row r
        const int kr = ((lane >> 4) << 3) + (lane & 7), vr = ((lane >> 3) & 1) * 8 + (lane & 7);
        const uint32_t k_frag = kr * (D * 2) + ((((lane >> 3) & 1) ^ (kr & 7)) << 4);
        const uint32_t v_frag = vr * (D * 2) + (((lane >> 4) ^ (vr & 7)) << 4);
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
                const uint32_t k_at = ks + k_frag;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t b[4];
                    ldsm4(k_at ^ (kk << 5), b);
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
                        if (LOW) {
                            o[c][2] *= alpha;
                            o[c][3] *= alpha;
                        }
                    }
                    m[u] = mn;
                }
            }
            // a weight as the sum of two bf16: its first bits, and of what they leave
            uint32_t pa[4], pl[4];
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const float mb = m[u] == -INFINITY ? 0.f : m[u];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float p0 = tc::ex2(x[h][2 * u] - mb), p1 = tc::ex2(x[h][2 * u + 1] - mb);
                    l[u] += p0 + p1;
                    split_weights(p0, p1, pa[2 * h + u], (LOW ? pa : pl)[2 * h + (LOW ? 1 : u)]);
                }
            }
            {
                const uint32_t v_at = vs + v_frag;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t b[4];
                    ldsm4t(v_at ^ (c << 5), b);
                    mma16816(o[2 * c], pa, b[0], b[1]);
                    mma16816(o[2 * c + 1], pa, b[2], b[3]);
                    if (!LOW) {
                        mma16816(o[2 * c], pl, b[0], b[1]);
                        mma16816(o[2 * c + 1], pl, b[2], b[3]);
                    }
                }
            }
        }
        if (LOW)
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                o[c][0] += o[c][2];
                o[c][1] += o[c][3];
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
                    for (int k0 = lane; k0 - lane < n; k0 += 128) {
                        float sum[4], old[4];
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            sum[v] = 0.f;
                            old[v] = k0 + 32 * v < n ? w[k0 + 32 * v] : 0.f;
                        }
                        for (int i = 0; i < rps; ++i) {
                            const float M = __shfl_sync(FULL_MASK, i < 8 ? m[0] : m[1], (i & 7) * 4);
                            const float f = __shfl_sync(FULL_MASK, i < 8 ? inv[0] : inv[1], (i & 7) * 4);
                            if (M == -INFINITY) continue;
                            const float* x = lg + (int64_t)i * a.lcap + k0;
#pragma unroll
                            for (int v = 0; v < 4; ++v)
                                if (k0 + 32 * v < n) sum[v] += exp2f(x[32 * v] - M) * f;
                        }
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (k0 + 32 * v < n) w[k0 + 32 * v] = old[v] + sum[v];
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
        // the warps' states of the rows, joined by the warps of the head
        constexpr int ROWS = LOW ? 8 : 16, PITCH = D + 8;
        static_assert(SW * ROWS * PITCH * 4 <= stream_smem<D>(), "the states fit the stages");
        __shared__ float2 ml[SW][ROWS], joined[SW / WPH][ROWS];
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
            const int w0 = warp / WPH * WPH;  // the head's first warp
            for (int e = wi * 32 + lane; e < min(ROWS, rps) * (D / 4); e += 32 * WPH) {
                const int i = e / (D / 4), c = e % (D / 4) * 4;
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int v = 0; v < WPH; ++v) M = fmaxf(M, ml[w0 + v][i].x);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int v = 0; v < WPH; ++v) {
                    const float2 y = ml[w0 + v][i];
                    const float f = y.x == -INFINITY ? 0.f : exp2f(y.x - M);
                    const float4 z = *reinterpret_cast<const float4*>(st + ((w0 + v) * ROWS + i) * PITCH + c);
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
                        joined[warp / WPH][i] = make_float2(M, inv);
                    }
                } else {
                    *reinterpret_cast<float4*>(a.part_o + (slot * R + row) * D + c) = acc;
                    if (c == 0) a.part_ml[ml_index(a, row, slot)] = make_float2(M, L);
                }
            }
        }
        if (final && a.logit) {  // (the same for the whole block)
            __syncthreads();
            if (on) add_kept(a, sh, n, joined[warp / WPH], wi * 32 + lane, 32 * WPH);
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
    const bool low = rps <= 8;
    auto by_warps = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (warps_per_head == 1) return low ? run(stream_attend_kernel<D, 1, true>) : run(stream_attend_kernel<D, 1, false>);
        return low ? run(stream_attend_kernel<D, 4, true>) : run(stream_attend_kernel<D, 4, false>);
    };
    return d == 128 ? by_warps(std::integral_constant<int, 128>()) : by_warps(std::integral_constant<int, 64>());
}

cudaError_t prepare_shared_stream() {
    cudaError_t e = cudaSuccess;
    auto set = [&](auto kernel, int smem) {
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    };
    auto all = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        set(stream_attend_kernel<D, 1, true>, stream_smem<D>());
        set(stream_attend_kernel<D, 1, false>, stream_smem<D>());
        set(stream_attend_kernel<D, 4, true>, stream_smem<D>());
        set(stream_attend_kernel<D, 4, false>, stream_smem<D>());
    };
    all(std::integral_constant<int, 64>());
    all(std::integral_constant<int, 128>());
    return e;
}

}  // namespace shared
}  // namespace hkv
