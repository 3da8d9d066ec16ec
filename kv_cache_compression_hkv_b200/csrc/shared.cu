// shared.cu -- shared-prefix cache: append, attention in fp32 on the CUDA
// cores, the joining of partial results, and the accumulated weights.
//
// A row (sequence s, query head h, query t) attends over the n_p keys of its
// prefix and its own keys j < lim:
//     x_j = log2(e) scale q.k_j,   m = max x_j,   l = sum 2^(x_j - m),
//     o = sum 2^(x_j - m) v_j / l,   weight_j += 2^(x_j - m) / l.
// Keys are cut into ranges that different blocks take; each leaves (m, l,
// sum 2^(x - m) v) of its range, all in fp32, and a last kernel joins them:
// with M = max m_i, o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"
#include "shared.cuh"

namespace hkv {
namespace shared {

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------

// One block per (sequence, KV head, slice of the new tokens): rows are copied
// as 16-byte pieces.  With more than one slice per head the lengths are
// advanced by bump_kernel behind this launch (another block may not have read
// them yet); with one, here.
template <typename T, int D>
__global__ void __launch_bounds__(256) append_rows_kernel(View a, const T* __restrict__ kt, int64_t k0, int64_t k1,
                                                          int64_t k2, const T* __restrict__ vt, int64_t v0,
                                                          int64_t v1, int64_t v2, const float* __restrict__ wt,
                                                          int n_new, int slices) {
    const int head = blockIdx.x / slices, part = blockIdx.x % slices;
    const int s = head / a.Hk, hk = head % a.Hk;
    ptx::grid_dep_wait();
    const int len = own_len(a, s, hk), np0 = a.next_pos ? a.next_pos[head] : 0;
    if (n_new > a.cap - len) {
        if (a.status && part == 0 && threadIdx.x == 0 && atomicCAS(a.status, 0, HKV_ERR_CAPACITY) == 0)
            atomicExch(a.status + 1, head);
        return;
    }
    if (slices == 1) __syncthreads();  // everyone has read the length
    const int per = (n_new + slices - 1) / slices;
    const int lo = part * per, hi = min(n_new, lo + per);
    constexpr int PIECES = D * (int)sizeof(T) / 16;
    const T* ksrc = kt + s * k0 + hk * k1;
    const T* vsrc = vt + s * v0 + hk * v1;
    T* kd = static_cast<T*>(a.k) + s * a.ks[0] + hk * a.ks[1];
    T* vd = static_cast<T*>(a.v) + s * a.vs[0] + hk * a.vs[1];
    constexpr int EP = 16 / (int)sizeof(T);
    for (int e = lo * PIECES + threadIdx.x; e < hi * PIECES; e += 256) {
        const int i = e / PIECES, c = (e % PIECES) * EP;
        const uint4 x = *reinterpret_cast<const uint4*>(ksrc + i * k2 + c);
        const uint4 y = *reinterpret_cast<const uint4*>(vsrc + i * v2 + c);
        *reinterpret_cast<uint4*>(kd + (int64_t)(len + i) * a.ks[2] + c) = x;
        *reinterpret_cast<uint4*>(vd + (int64_t)(len + i) * a.vs[2] + c) = y;
    }
    const int64_t row0 = (int64_t)head * a.cap + len;
    for (int i = lo + threadIdx.x; i < hi; i += 256) {
        if (a.pos) a.pos[row0 + i] = np0 + i;
        if (a.weight) a.weight[row0 + i] = wt ? wt[(int64_t)head * n_new + i] : 0.f;
    }
    if (slices == 1 && threadIdx.x == 0) {
        a.len[head] = len + n_new;
        if (a.next_pos) a.next_pos[head] = np0 + n_new;
    }
}

__global__ void bump_kernel(View a, int n_new) {
    const int head = blockIdx.x * blockDim.x + threadIdx.x;
    ptx::grid_dep_wait();
    if (head >= a.S * a.Hk) return;
    const int len = clamp_len(a.len[head], a.cap);
    if (n_new > a.cap - len) return;
    a.len[head] = len + n_new;
    if (a.next_pos) a.next_pos[head] += n_new;
}

cudaError_t launch_append(const View& a, int dtype, int d, const void* k_t, const int64_t* ks, const void* v_t,
                          const int64_t* vs, const float* w_t, cudaStream_t st) {
    const int heads = a.S * a.Hk, n_new = a.T;
    int slices = 1;
    while (heads * slices < 592 && n_new / slices > 64) slices *= 2;
    auto go = [&](auto tag, auto dim) {
        using E = decltype(tag);
        constexpr int D = decltype(dim)::value;
        return launch(append_rows_kernel<E, D>, (int64_t)heads * slices, 256, 0, st, a, (const E*)k_t, ks[0], ks[1], ks[2],
                      (const E*)v_t, vs[0], vs[1], vs[2], w_t, n_new, slices);
    };
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    cudaError_t e;
    if (dtype == HKV_DTYPE_F32) e = d == 64 ? go(float(), I64()) : go(float(), I128());
    else e = d == 64 ? go(__nv_bfloat16(), I64()) : go(__nv_bfloat16(), I128());
    if (e == cudaSuccess && slices > 1) e = launch(bump_kernel, (heads + 255) / 256, 256, 0, st, a, n_new);
    return e;
}

// ---------------------------------------------------------------------------
// attention in fp32, on the CUDA cores (fp32 products stay fp32)
// ---------------------------------------------------------------------------

constexpr int RT = 16;   // rows of a block
constexpr int KT = 32;   // keys a step

template <int D> struct F32Smem {
    static constexpr int KP = D + 4;  // padded rows: float4 reads of 32 rows spread over the banks
    float q[RT][KP];
    float k[2][KT][KP];
    float v[2][KT][D];
    float p[KT][RT];
    float2 ml[RT];
    int list[RT + 1];
    int res[4];
};

__device__ __forceinline__ void cp16(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}

// One block per (tile of 16 rows, keys): first the prefixes' tiles, whose rows
// come from all their sequences (np > 0), then tiles of one (sequence, KV
// head) over a piece of its list of keys.  Steps of 32 keys, the next one's on
// their way.  Warp w owns rows 4w .. 4w + 3: lane = key for the logits, lanes
// across d for the weighted sum.  Where a block has all of its rows' keys the
// result is final, and, with the logits kept (one tile has all the head's
// rows), so are the accumulated weights.
template <int D>
__global__ void __launch_bounds__(128) attend_f32_kernel(const __grid_constant__ View a, int ptiles, int otiles) {
    extern __shared__ __align__(16) unsigned char raw[];
    F32Smem<D>& sm = *reinterpret_cast<F32Smem<D>*>(raw);
    int* cnt = reinterpret_cast<int*>(raw + sizeof(F32Smem<D>));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rps = a.rep * a.T;
    const int64_t R = (int64_t)a.S * a.H * a.T;
    const bool final = a.np + a.no == 1;
    ptx::grid_dep_wait();
    ptx::grid_dep_trigger();
    const int n_prefix = ptiles * a.Hk * a.np;
    const bool is_prefix = (int)blockIdx.x < n_prefix;
    int slot, rows, hk, s = 0, first = 0, n_own = 0, g;
    Piece pc;
    if (is_prefix) {
        const int b = blockIdx.x;
        slot = b % a.np;
        hk = b / a.np % a.Hk;
        if (!find_prefix_tile(a, b / a.np / a.Hk, RT, g, first, rows, cnt, sm.res, sm.list)) return;
        split_range(prefix_len(a, g), a.np, slot, pc.pa, pc.pb);
        pc.oa = pc.ob = 0;
    } else {
        // the rows with the most keys (the last queries) first
        const int b = blockIdx.x - n_prefix, heads = a.S * a.Hk;
        const int j = b % a.no, sh = b / a.no % heads, tile = otiles - 1 - b / a.no / heads;
        s = sh / a.Hk;
        hk = sh % a.Hk;
        first = tile * RT;
        rows = min(RT, rps - first);
        g = prefix_of(a, s);
        n_own = own_len(a, s, hk);
        pc = list_piece(a.listed ? prefix_len(a, g) : 0, n_own, a.no, j);
        slot = a.np + j;
    }
    if (pc.empty() && !final) return;  // the joining kernel knows
    const int o0 = first / rps;
    auto seq_row = [&](int r, int& sq, int& i) {  // row r of the tile -> sequence, row within (sequence, KV head)
        const int f = first + r;
        sq = is_prefix ? sm.list[f / rps - o0] : s;
        i = is_prefix ? f % rps : f;
    };
    // own keys past the last row's limit are needed only where their logits are kept
    const bool keep = !is_prefix && a.logit;
    if (!is_prefix && !keep) pc.ob = min(pc.ob, own_limit(a, n_own, first + rows - 1));
    const int psteps = (pc.pb - pc.pa + KT - 1) / KT, steps = psteps + max(0, pc.ob - pc.oa + KT - 1) / KT;
    const float* pkb = static_cast<const float*>(a.pk) + (g < 0 ? 0 : g) * a.pks[0] + hk * a.pks[1];
    const float* pvb = static_cast<const float*>(a.pv) + (g < 0 ? 0 : g) * a.pvs[0] + hk * a.pvs[1];
    const float* kb = static_cast<const float*>(a.k) + s * a.ks[0] + hk * a.ks[1];
    const float* vb = static_cast<const float*>(a.v) + s * a.vs[0] + hk * a.vs[1];
    auto load = [&](int st) {
        if (st < steps) {
            const bool pre = st < psteps;
            const int k0 = pre ? pc.pa + st * KT : pc.oa + (st - psteps) * KT, hi = pre ? pc.pb : pc.ob;
            const float *kp = pre ? pkb : kb, *vp = pre ? pvb : vb;
            const int64_t kst = pre ? a.pks[2] : a.ks[2], vst = pre ? a.pvs[2] : a.vs[2];
#pragma unroll
            for (int e = 0; e < KT * (D / 4) / 128; ++e) {
                const int idx = e * 128 + tid, r = idx / (D / 4), c = idx % (D / 4) * 4;
                const bool on = k0 + r < hi;
                const int64_t key = on ? k0 + r : k0;
                cp16(&sm.k[st & 1][r][c], kp + key * kst + c, on);
                cp16(&sm.v[st & 1][r][c], vp + key * vst + c, on);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load(0);
    for (int e = tid; e < RT * (D / 4); e += 128) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            int sq, i;
            seq_row(r, sq, i);
            x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + sq * a.qs[0] +
                                                 (hk * a.rep + i % a.rep) * a.qs[1] + i / a.rep * a.qs[2] + c);
        }
        *reinterpret_cast<float4*>(&sm.q[r][c]) = make_float4(x.x * a.qscale, x.y * a.qscale, x.z * a.qscale, x.w * a.qscale);
    }
    constexpr int V = D / 32;
    float m[4], l[4], o[4][V];
    int lim[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int r = warp * 4 + u;
        m[u] = -INFINITY;
        l[u] = 0.f;
#pragma unroll
        for (int c = 0; c < V; ++c) o[u][c] = 0.f;
        lim[u] = r >= rows || is_prefix ? 0 : own_limit(a, n_own, first + r);
    }
    float* lrow = keep ? a.logit + ((int64_t)(s * a.Hk + hk) * rps + warp * 4) * a.lcap : nullptr;
    const bool idle = warp * 4 >= rows;
    for (int st = 0; st < steps; ++st) {
        load(st + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        if (!idle) {
            const bool pre = st < psteps;
            const int k0 = pre ? pc.pa + st * KT : pc.oa + (st - psteps) * KT, hi = pre ? pc.pb : pc.ob;
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
            for (int c = 0; c < D; c += 4) {
                const float4 kk = *reinterpret_cast<const float4*>(&sm.k[st & 1][lane][c]);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float4 qq = *reinterpret_cast<const float4*>(&sm.q[warp * 4 + u][c]);
                    x[u] = fmaf(kk.x, qq.x, fmaf(kk.y, qq.y, fmaf(kk.z, qq.z, fmaf(kk.w, qq.w, x[u]))));
                }
            }
            const int key = k0 + lane;
            float pw[4], mt[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const bool in = key < hi && (pre ? warp * 4 + u < rows : key < lim[u]);
                x[u] = in ? x[u] : -INFINITY;
                if (lrow && !pre && key < hi && warp * 4 + u < rows) lrow[(int64_t)u * a.lcap + key] = x[u];
                mt[u] = x[u];
            }
#pragma unroll
            for (int off = 16; off; off >>= 1)
#pragma unroll
                for (int u = 0; u < 4; ++u) mt[u] = fmaxf(mt[u], __shfl_xor_sync(FULL_MASK, mt[u], off));
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float mn = fmaxf(m[u], mt[u]);
                const float mb = mn == -INFINITY ? 0.f : mn;
                const float alpha = exp2f(m[u] - mb);
                pw[u] = exp2f(x[u] - mb);
                l[u] = l[u] * alpha + pw[u];  // each lane its own keys; summed at the end
                m[u] = mn;
#pragma unroll
                for (int c = 0; c < V; ++c) o[u][c] *= alpha;
            }
            *reinterpret_cast<float4*>(&sm.p[lane][warp * 4]) = make_float4(pw[0], pw[1], pw[2], pw[3]);
            __syncwarp();
#pragma unroll 8
            for (int kk = 0; kk < KT; ++kk) {
                const float4 p4 = *reinterpret_cast<const float4*>(&sm.p[kk][warp * 4]);
                const float pr[4] = {p4.x, p4.y, p4.z, p4.w};
                float vv[V];
                if constexpr (V == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(&sm.v[st & 1][kk][lane * 4]);
                    vv[0] = y.x; vv[1] = y.y; vv[2] = y.z; vv[3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2*>(&sm.v[st & 1][kk][lane * 2]);
                    vv[0] = y.x; vv[1] = y.y;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int c = 0; c < V; ++c) o[u][c] = fmaf(pr[u], vv[c], o[u][c]);
            }
        }
        __syncthreads();  // the stage is loaded again next
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!idle) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = warp * 4 + u;
            float ls = l[u];
#pragma unroll
            for (int off = 16; off; off >>= 1) ls += __shfl_xor_sync(FULL_MASK, ls, off);
            if (r >= rows) continue;
            int sq, i;
            seq_row(r, sq, i);
            const int64_t row = row_of(a, sq, hk, i);
            // (a sum that is NaN, of NaN logits alone, must not pass for an empty row)
            if (ls != ls && m[u] == -INFINITY) m[u] = 0.f;
            const bool some = !(m[u] == -INFINITY);
            const float f = !final ? 1.f : some ? 1.f / ls : 0.f;
            float* po = final ? static_cast<float*>(a.out) + s * a.os[0] + (hk * a.rep + i % a.rep) * a.os[1] + i / a.rep * a.os[2]
                              : a.part_o + (slot * R + row) * D;
            if constexpr (V == 4)
                *reinterpret_cast<float4*>(po + lane * 4) = make_float4(o[u][0] * f, o[u][1] * f, o[u][2] * f, o[u][3] * f);
            else
                *reinterpret_cast<float2*>(po + lane * 2) = make_float2(o[u][0] * f, o[u][1] * f);
            if (lane == 0) {
                if (final) {
                    const float l2 = some ? m[u] + log2f(ls) : -INFINITY;
                    if (a.lse) a.lse[row] = l2 * 0.6931471805599453f;
                    if (a.row_lse) a.row_lse[row] = l2;
                    sm.ml[r] = make_float2(m[u], f);
                } else {
                    a.part_ml[ml_index(a, row, slot)] = make_float2(m[u], ls);
                }
            }
        }
    }
    if (!final || !keep) return;
    __syncthreads();
    const float* lg = a.logit + (int64_t)(s * a.Hk + hk) * rps * a.lcap;
    float* w = a.weight + (int64_t)(s * a.Hk + hk) * a.cap;
    for (int j = tid; j < n_own; j += 128) {
        float sum = 0.f;
        for (int i = 0; i < rps; ++i) {
            const float2 y = sm.ml[i];
            if (y.x != -INFINITY) sum += exp2f(lg[(int64_t)i * a.lcap + j] - y.x) * y.y;
        }
        w[j] += sum;
    }
}

// ---------------------------------------------------------------------------
// joining the partial results; accumulated weights from kept logits
// ---------------------------------------------------------------------------

// A row's partial results as the calling warp holds them: lane j % 32,
// register j / 32 has 2^(m_j - M) of slot j (0 where it was not written).
struct RowJoin {
    float f[2 * MAX_SPLITS / 32];
    float M, L;  // maximum and sum over the slots
};
// The loads of a row's (max, sum) pairs go out together, and with those of
// the lengths that say which of them were written.
__device__ __forceinline__ RowJoin join_row(const View& a, int64_t row, int pk, int ok) {
    const int lane = threadIdx.x & 31, ns = a.np + a.no;
    constexpr int N = 2 * MAX_SPLITS / 32;
    float2 ml[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
        const int j = u * 32 + lane;
        ml[u] = j < ns ? a.part_ml[ml_index(a, row, j)] : make_float2(-INFINITY, 0.f);
    }
    RowJoin r;
    r.M = -INFINITY;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        if (u * 32 >= ns) break;
        if (!slot_valid(a, u * 32 + lane, pk, ok)) ml[u] = make_float2(-INFINITY, 0.f);
        r.M = fmaxf(r.M, ml[u].x);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) r.M = fmaxf(r.M, __shfl_xor_sync(FULL_MASK, r.M, off));
    r.L = 0.f;
#pragma unroll
    for (int u = 0; u < N; ++u) {
        r.f[u] = 0.f;
        if (u * 32 >= ns) continue;
        if (ml[u].x != -INFINITY) {
            r.f[u] = exp2f(ml[u].x - r.M);
            r.L = fmaf(ml[u].y, r.f[u], r.L);
        }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) r.L += __shfl_xor_sync(FULL_MASK, r.L, off);
    return r;
}

// The calling warp adds up the joined row's partial sums (eight slots' loads in
// flight) and writes the row.
template <typename T, int D>
__device__ __forceinline__ void write_row(const View& a, const RowJoin& j, int64_t row, int s, int h, int t) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, ns = a.np + a.no;
    const int64_t R = (int64_t)a.S * a.H * a.T;
    float acc[V];
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] = 0.f;
    const float* po = a.part_o + row * D + lane * V;
#pragma unroll
    for (int u = 0; u < 2 * MAX_SPLITS / 32; ++u) {
        if (u * 32 >= ns) break;
        for (int e0 = 0; e0 < 32 && u * 32 + e0 < ns; e0 += 8) {
            float x[8][V], f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = __shfl_sync(FULL_MASK, j.f[u], e0 + e);
                const float* p = po + (u * 32 + e0 + e) * R * D;
                if constexpr (V == 4) {
                    const float4 y = f[e] != 0.f ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
                    x[e][0] = y.x; x[e][1] = y.y; x[e][2] = y.z; x[e][3] = y.w;
                } else {
                    const float2 y = f[e] != 0.f ? *reinterpret_cast<const float2*>(p) : make_float2(0.f, 0.f);
                    x[e][0] = y.x; x[e][1] = y.y;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int c = 0; c < V; ++c) acc[c] = fmaf(x[e][c], f[e], acc[c]);
        }
    }
    const bool some = !(j.M == -INFINITY);
    const float inv = some ? 1.f / j.L : 0.f;
    T* orow = static_cast<T*>(a.out) + s * a.os[0] + h * a.os[1] + t * a.os[2] + lane * V;
#pragma unroll
    for (int c = 0; c < V; ++c) acc[c] *= inv;
    if constexpr (sizeof(T) == 4) {
        if constexpr (V == 4) *reinterpret_cast<float4*>(orow) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        else *reinterpret_cast<float2*>(orow) = make_float2(acc[0], acc[1]);
    } else {
#pragma unroll
        for (int c = 0; c < V; c += 2) *reinterpret_cast<__nv_bfloat162*>(orow + c) = __floats2bfloat162_rn(acc[c], acc[c + 1]);
    }
    if (lane == 0) {
        const float l2 = some ? j.M + log2f(j.L) : -INFINITY;
        if (a.lse) a.lse[row] = l2 * 0.6931471805599453f;
        if (a.row_lse) a.row_lse[row] = l2;
    }
}

// Blocks [0, row_blocks): one warp per row.  Blocks beyond: 128 slots of one
// (sequence, KV head) each, weight += the kept logits' weights in row order;
// the logits are on their way while the block joins the head's rows for itself
// (waiting for the other blocks' rows instead would cost another launch).
template <typename T, int D, int MAXR>
__global__ void __launch_bounds__(128, 8) combine_kernel(const __grid_constant__ View a, int row_blocks) {
    __shared__ float2 ml_s[MAXR];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if ((int)blockIdx.x < row_blocks) {
        const int R = a.S * a.H * a.T, row = blockIdx.x * 4 + warp;
        const int t = row % a.T, sh = row / a.T, h = sh % a.H, s = sh / a.H;
        int pk = 0, ok = 0;
        if (row < R) {
            pk = prefix_len(a, prefix_of(a, s));
            ok = own_len(a, s, h / a.rep);
        }
        ptx::grid_dep_wait();
        if (row >= R) return;
        const RowJoin j = join_row(a, row, pk, ok);
        write_row<T, D>(a, j, row, s, h, t);
        return;
    }
    const int chunks = (a.cap + 127) / 128;
    const int b = blockIdx.x - row_blocks, sh = b / chunks;
    const int s = sh / a.Hk, hk = sh % a.Hk, rps = a.rep * a.T;
    const int n = own_len(a, s, hk);
    if (b % chunks * 128 >= n) {
        ptx::grid_dep_wait();
        return;
    }
    const int pk = prefix_len(a, prefix_of(a, s));
    const int j = b % chunks * 128 + tid;
    float* w = a.weight + (int64_t)sh * a.cap + j;
    const float old = j < n ? *w : 0.f;
    ptx::grid_dep_wait();
    float x[MAXR];
    const float* lg = a.logit + (int64_t)sh * rps * a.lcap + j;
#pragma unroll
    for (int i = 0; i < MAXR; ++i) x[i] = i < rps && j < n ? lg[(int64_t)i * a.lcap] : -INFINITY;
    for (int i = warp; i < rps; i += 4) {
        const RowJoin r = join_row(a, row_of(a, s, hk, i), pk, n);
        if (lane == 0) ml_s[i] = make_float2(r.M, r.M == -INFINITY ? 0.f : 1.f / r.L);
    }
    __syncthreads();
    if (j >= n) return;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < MAXR; ++i)
        if (i < rps) {
            const float2 y = ml_s[i];
            if (y.x != -INFINITY) sum += exp2f(x[i] - y.x) * y.y;
        }
    *w = old + sum;
}

// ---------------------------------------------------------------------------
// accumulated weights of many rows: the logits once more, summed by key
// ---------------------------------------------------------------------------

// One block per (sequence, KV head, 32 keys): lane = key, warp w takes rows
// 4w .. 4w + 3 of every tile of 16; a key's weight 2^(x - lse) over the rows
// that see it, per tile, then over the tiles, then over the warps.
template <int D> struct SumSmem {
    float q[RT][D + 4];
    float k[KT][D + 4];
    float p[4][KT];
};

template <int D>
__global__ void __launch_bounds__(128) column_sums_f32_kernel(const __grid_constant__ View a) {
    extern __shared__ __align__(16) unsigned char raw[];
    SumSmem<D>& sm = *reinterpret_cast<SumSmem<D>*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int chunks = (a.cap + KT - 1) / KT;
    const int sh = blockIdx.x / chunks, k0 = blockIdx.x % chunks * KT;
    const int s = sh / a.Hk, hk = sh % a.Hk, rps = a.rep * a.T;
    ptx::grid_dep_wait();
    const int n = own_len(a, s, hk);
    if (k0 >= n) return;
    const float* kb = static_cast<const float*>(a.k) + s * a.ks[0] + hk * a.ks[1];
    for (int e = tid; e < KT * (D / 4); e += 128) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + r < n) x = *reinterpret_cast<const float4*>(kb + (int64_t)(k0 + r) * a.ks[2] + c);
        *reinterpret_cast<float4*>(&sm.k[r][c]) = x;
    }
    // the first row that sees key k0: n - T + t + 1 > k0
    const int t0 = max(0, k0 - (n - a.T));
    const int key = k0 + lane;
    float total = 0.f;
    for (int f = t0 * a.rep / RT * RT; f < rps; f += RT) {
        __syncthreads();
        const int rows = min(RT, rps - f);
        for (int e = tid; e < RT * (D / 4); e += 128) {
            const int r = e / (D / 4), c = e % (D / 4) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int i = f + r;
                x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + s * a.qs[0] +
                                                     (hk * a.rep + i % a.rep) * a.qs[1] + i / a.rep * a.qs[2] + c);
            }
            sm.q[r][c] = x.x * a.qscale;
            sm.q[r][c + 1] = x.y * a.qscale;
            sm.q[r][c + 2] = x.z * a.qscale;
            sm.q[r][c + 3] = x.w * a.qscale;
        }
        __syncthreads();
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int c = 0; c < D; c += 4) {
            const float4 kk = *reinterpret_cast<const float4*>(&sm.k[lane][c]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 qq = *reinterpret_cast<const float4*>(&sm.q[warp * 4 + u][c]);
                x[u] = fmaf(kk.x, qq.x, fmaf(kk.y, qq.y, fmaf(kk.z, qq.z, fmaf(kk.w, qq.w, x[u]))));
            }
        }
        float tile = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = warp * 4 + u;
            if (r >= rows) continue;
            const float e = a.row_lse[row_of(a, s, hk, f + r)];
            if (key < n && key < own_limit(a, n, f + r) && e != -INFINITY) tile += exp2f(x[u] - e);
        }
        total += tile;
    }
    __syncthreads();
    float* red = &sm.p[0][0];
    red[warp * 32 + lane] = total;
    __syncthreads();
    if (warp == 0 && key < n)
        a.weight[(int64_t)sh * a.cap + key] += (red[lane] + red[32 + lane]) + (red[64 + lane] + red[96 + lane]);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

namespace {

template <typename F> cudaError_t by_type(int dtype, int d, F&& f) {
    using I64 = std::integral_constant<int, 64>;
    using I128 = std::integral_constant<int, 128>;
    if (dtype == HKV_DTYPE_F32) return d == 64 ? f(float(), I64()) : f(float(), I128());
    return d == 64 ? f(__nv_bfloat16(), I64()) : f(__nv_bfloat16(), I128());
}

}  // namespace

cudaError_t launch_attend_f32(const View& a, int d, cudaStream_t st) {
    const int rps = a.rep * a.T, otiles = (rps + RT - 1) / RT;
    const int64_t ptiles = a.np ? max_prefix_tiles(a.S, a.G, rps, RT) : 0;
    const int64_t blocks = ptiles * a.Hk * a.np + (int64_t)a.S * a.Hk * otiles * a.no;
    auto go = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        return launch(attend_f32_kernel<D>, blocks, 128, sizeof(F32Smem<D>) + (size_t)a.G * 4, st, a, (int)ptiles, otiles);
    };
    return d == 64 ? go(std::integral_constant<int, 64>()) : go(std::integral_constant<int, 128>());
}

cudaError_t prepare_shared_f32() {
    cudaError_t e = cudaFuncSetAttribute(attend_f32_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(F32Smem<64>) + MAX_PREFIXES * 4);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(attend_f32_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(F32Smem<128>) + MAX_PREFIXES * 4);
    return e;
}

cudaError_t launch_combine(const View& a, int dtype, int d, cudaStream_t st) {
    const int64_t R = (int64_t)a.S * a.H * a.T, rb = (R + 3) / 4;
    const int64_t blocks = rb + (a.logit ? (int64_t)a.S * a.Hk * ((a.cap + 127) / 128) : 0);
    return by_type(dtype, d, [&](auto tag, auto dim) {
        using E = decltype(tag);
        constexpr int D = decltype(dim)::value;
        const int rps = a.rep * a.T;
        if (rps == 1) return launch(combine_kernel<E, D, 1>, blocks, 128, 0, st, a, (int)rb);
        if (rps <= 8) return launch(combine_kernel<E, D, 8>, blocks, 128, 0, st, a, (int)rb);
        return launch(combine_kernel<E, D, STREAM_ROWS>, blocks, 128, 0, st, a, (int)rb);
    });
}

cudaError_t launch_column_sums_f32(const View& a, int d, cudaStream_t st) {
    const int64_t blocks = (int64_t)a.S * a.Hk * ((a.cap + KT - 1) / KT);
    if (d == 64) return launch(column_sums_f32_kernel<64>, blocks, 128, sizeof(SumSmem<64>), st, a);
    return launch(column_sums_f32_kernel<128>, blocks, 128, sizeof(SumSmem<128>), st, a);
}

}  // namespace shared
}  // namespace hkv
