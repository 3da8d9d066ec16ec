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
// them yet); with one, here.  8192 tokens of 64 heads, d = 128, bf16: 98 us, 537
// MB or 5.5 TB/s.
template <typename T, int D>
__global__ void __launch_bounds__(256) append_rows_kernel(View a, const T* kt, int64_t k0, int64_t k1, int64_t k2,
                                                          const T* vt, int64_t v0, int64_t v1, int64_t v2,
                                                          const float* wt, int n_new, int slices) {
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
    while (heads * slices < 4 * SMS && n_new / slices > 64) slices *= 2;
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

// A block's shape: four warps of RW rows each, steps of 32 KPL keys in ST
// stages.  Few rows (9 to 16 of a head, and the prefixes' rows beside the
// streaming kernel): 4 x 4 rows, two stages.  More: 4 x 8
// rows, and two keys a lane where d = 64 leaves the shared memory for it: a
// warp then reads 10 times from shared memory for 64 fused multiply-adds
// instead of 5 for 16; one stage, so that four blocks share an SM and hide each
// other's loads.
template <int D, int RW_, int KPL_, int ST_> struct F32Shape {
    static constexpr int WARPS = 4, RW = RW_, KPL = KPL_, ST = ST_, THREADS = 32 * WARPS;
    static constexpr int RT = WARPS * RW, KT = 32 * KPL;
    static constexpr int KP = D + 4;  // padded rows: float4 reads of 32 rows spread over the banks
    struct Smem {
        float q[RT][KP];
        float k[ST][KT][KP];
        float v[ST][KT][D];
        float p[KT][RT];
        float2 ml[RT];
        int list[RT + 1];
        int res[4];
    };
    struct SumSmem {
        float q[RT][KP];
        float k[KT][KP];
        float part[WARPS][KT];
    };
};
template <int D> using FewF32 = F32Shape<D, 4, 1, 2>;
template <int D> using ManyF32 = F32Shape<D, 8, D == 64 ? 2 : 1, 1>;

// x[u][p] = q row u . k row lane + 32 p, for a warp's rows and p < N (0 beyond).
template <int D, int N, int RW, int KPL, int KP>
__device__ __forceinline__ void dots(float (&x)[RW][KPL], const float (*q)[KP], const float (*k)[KP], int lane) {
#pragma unroll
    for (int u = 0; u < RW; ++u)
#pragma unroll
        for (int p = 0; p < KPL; ++p) x[u][p] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 kk[N];
#pragma unroll
        for (int p = 0; p < N; ++p) kk[p] = *reinterpret_cast<const float4*>(&k[lane + 32 * p][c]);
#pragma unroll
        for (int u = 0; u < RW; ++u) {
            const float4 qq = *reinterpret_cast<const float4*>(&q[u][c]);
#pragma unroll
            for (int p = 0; p < N; ++p)
                x[u][p] = fmaf(kk[p].x, qq.x, fmaf(kk[p].y, qq.y, fmaf(kk[p].z, qq.z, fmaf(kk[p].w, qq.w, x[u][p]))));
        }
    }
}

// One block per (tile of RT rows, keys): first the prefixes' tiles, whose rows
// come from all their sequences (np > 0), then tiles of one (sequence, KV
// head) over a piece of its list of keys.  The next step's keys are on their
// way.  A warp owns RW rows: lane = key for the logits, lanes across d for the
// weighted sum.  Where a block has all of its rows' keys the
// result is final, and, with the logits kept (one tile has all the head's
// rows), so are the accumulated weights.  160 heads of 96 rows over 129 keys, d =
// 64: 36 us, a quarter of the fp32 rate; shared memory is read for as long as the
// products take.
template <int D, typename C>
__global__ void __launch_bounds__(C::THREADS, 4) attend_f32_kernel(const __grid_constant__ View a, int ptiles, int otiles) {
    extern __shared__ __align__(16) unsigned char raw[];
    constexpr int RT = C::RT, KT = C::KT, RW = C::RW, KPL = C::KPL, THREADS = C::THREADS;
    typename C::Smem& sm = *reinterpret_cast<typename C::Smem*>(raw);
    int* cnt = reinterpret_cast<int*>(raw + sizeof(typename C::Smem));
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
    constexpr int ST = C::ST;
    auto load = [&](int st) {
        if (st < steps) {
            const bool pre = st < psteps;
            const int k0 = pre ? pc.pa + st * KT : pc.oa + (st - psteps) * KT, hi = pre ? pc.pb : pc.ob;
            const float *kp = pre ? pkb : kb, *vp = pre ? pvb : vb;
            const int64_t kst = pre ? a.pks[2] : a.ks[2], vst = pre ? a.pvs[2] : a.vs[2];
#pragma unroll
            for (int e = 0; e < KT * (D / 4) / THREADS; ++e) {
                const int idx = e * THREADS + tid, r = idx / (D / 4), c = idx % (D / 4) * 4;
                const bool on = k0 + r < hi;
                const int64_t key = on ? k0 + r : k0;
                cp16(ptx::smem_u32(&sm.k[st % ST][r][c]), kp + key * kst + c, on);
                cp16(ptx::smem_u32(&sm.v[st % ST][r][c]), vp + key * vst + c, on);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load(0);
    for (int e = tid; e < RT * (D / 4); e += THREADS) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < rows) {
            int sq, i;
            seq_row(r, sq, i);
            const int t = query_of(a, i);
            x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + sq * a.qs[0] +
                                                 (hk * a.rep + i - t * a.rep) * a.qs[1] + t * a.qs[2] + c);
        }
        *reinterpret_cast<float4*>(&sm.q[r][c]) = make_float4(x.x * a.qscale, x.y * a.qscale, x.z * a.qscale, x.w * a.qscale);
    }
    constexpr int V = D / 32;
    float m[RW], l[RW], o[RW][V];
    int lim[RW];
#pragma unroll
    for (int u = 0; u < RW; ++u) {
        const int r = warp * RW + u;
        m[u] = -INFINITY;
        l[u] = 0.f;
#pragma unroll
        for (int c = 0; c < V; ++c) o[u][c] = 0.f;
        lim[u] = r >= rows || is_prefix ? 0 : own_limit(a, n_own, first + r);
    }
    float* lrow = keep ? a.logit + ((int64_t)(s * a.Hk + hk) * rps + warp * RW) * a.lcap : nullptr;
    const bool idle = warp * RW >= rows;
    int lim_last = 0;
#pragma unroll
    for (int u = 0; u < RW; ++u) lim_last = max(lim_last, lim[u]);
    for (int st = 0; st < steps; ++st) {
        if constexpr (ST == 2) {
            load(st + 1);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        __syncthreads();
        const bool pre = st < psteps;
        const int k0 = pre ? pc.pa + st * KT : pc.oa + (st - psteps) * KT, hi = pre ? pc.pb : pc.ob;
        // keys that some row of the warp sees (the last row sees the most)
        const int need = (pre || keep ? hi : min(hi, lim_last)) - k0;
        if (!idle && need > 0) {
            float x[RW][KPL], mt[RW];
            const int groups = KPL == 1 || need <= 32 ? 1 : KPL;  // of 32 keys
            if (groups == KPL) dots<D, KPL>(x, &sm.q[warp * RW], sm.k[st % ST], lane);
            else dots<D, 1>(x, &sm.q[warp * RW], sm.k[st % ST], lane);
#pragma unroll
            for (int u = 0; u < RW; ++u) {
                mt[u] = -INFINITY;
#pragma unroll
                for (int p = 0; p < KPL; ++p) {
                    const int key = k0 + lane + 32 * p;
                    const bool in = key < hi && (pre ? warp * RW + u < rows : key < lim[u]);
                    x[u][p] = in ? x[u][p] : -INFINITY;
                    if (lrow && !pre && key < hi && warp * RW + u < rows) lrow[(int64_t)u * a.lcap + key] = x[u][p];
                    mt[u] = fmaxf(mt[u], x[u][p]);
                }
            }
#pragma unroll
            for (int off = 16; off; off >>= 1)
#pragma unroll
                for (int u = 0; u < RW; ++u) mt[u] = fmaxf(mt[u], __shfl_xor_sync(FULL_MASK, mt[u], off));
#pragma unroll
            for (int u = 0; u < RW; ++u) {
                const float mn = fmaxf(m[u], mt[u]);
                const float mb = mn == -INFINITY ? 0.f : mn;
                const float alpha = exp2f(m[u] - mb);
                l[u] *= alpha;  // each lane its own keys; summed at the end
#pragma unroll
                for (int p = 0; p < KPL; ++p) {
                    x[u][p] = exp2f(x[u][p] - mb);
                    l[u] += x[u][p];
                }
                m[u] = mn;
#pragma unroll
                for (int c = 0; c < V; ++c) o[u][c] *= alpha;
            }
#pragma unroll
            for (int p = 0; p < KPL; ++p)
#pragma unroll
                for (int u = 0; u < RW; u += 4)
                    *reinterpret_cast<float4*>(&sm.p[lane + 32 * p][warp * RW + u]) =
                        make_float4(x[u][p], x[u + 1][p], x[u + 2][p], x[u + 3][p]);
            __syncwarp();
#pragma unroll 4
            for (int kk = 0; kk < 32 * groups; ++kk) {
                float pr[RW], vv[V];
#pragma unroll
                for (int u = 0; u < RW; u += 4) {
                    const float4 p4 = *reinterpret_cast<const float4*>(&sm.p[kk][warp * RW + u]);
                    pr[u] = p4.x; pr[u + 1] = p4.y; pr[u + 2] = p4.z; pr[u + 3] = p4.w;
                }
                if constexpr (V == 4) {
                    const float4 y = *reinterpret_cast<const float4*>(&sm.v[st % ST][kk][lane * 4]);
                    vv[0] = y.x; vv[1] = y.y; vv[2] = y.z; vv[3] = y.w;
                } else {
                    const float2 y = *reinterpret_cast<const float2*>(&sm.v[st % ST][kk][lane * 2]);
                    vv[0] = y.x; vv[1] = y.y;
                }
#pragma unroll
                for (int u = 0; u < RW; ++u)
#pragma unroll
                    for (int c = 0; c < V; ++c) o[u][c] = fmaf(pr[u], vv[c], o[u][c]);
            }
        }
        __syncthreads();  // the stage is loaded again next
        if constexpr (ST == 1) load(st + 1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (!idle) {
#pragma unroll
        for (int u = 0; u < RW; ++u) {
            const int r = warp * RW + u;
            float ls = l[u];
#pragma unroll
            for (int off = 16; off; off >>= 1) ls += __shfl_xor_sync(FULL_MASK, ls, off);
            if (r >= rows) continue;
            int sq, i;
            seq_row(r, sq, i);
            const int t = query_of(a, i), h = hk * a.rep + i - t * a.rep;
            const int64_t row = row_index(a, sq, h, t);
            // (a sum that is NaN, of NaN logits alone, must not pass for an empty row)
            if (ls != ls && m[u] == -INFINITY) m[u] = 0.f;
            const bool some = !(m[u] == -INFINITY);
            const float f = !final ? 1.f : some ? 1.f / ls : 0.f;
            float* po = final ? static_cast<float*>(a.out) + s * a.os[0] + h * a.os[1] + t * a.os[2]
                              : a.part_o + (slot * R + row) * D;
            if constexpr (V == 4)
                *reinterpret_cast<float4*>(po + lane * 4) = make_float4(o[u][0] * f, o[u][1] * f, o[u][2] * f, o[u][3] * f);
            else
                *reinterpret_cast<float2*>(po + lane * 2) = make_float2(o[u][0] * f, o[u][1] * f);
            if (lane == 0) {
                if (final) {
                    const float l2 = some ? m[u] + log2f(ls) : -INFINITY;
                    if (a.lse) a.lse[row] = l2 * 0.6931471805599453f;
                    if (a.row_nl) a.row_nl[row] = less_sum(l2);
                    sm.ml[r] = make_float2(m[u], f);
                } else {
                    a.part_ml[ml_index(a, row, slot)] = make_float2(m[u], ls);
                }
            }
        }
    }
    if (!final || !keep) return;
    __syncthreads();
    add_kept(a, s * a.Hk + hk, n_own, sm.ml, tid, THREADS);
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
        if (a.row_nl) a.row_nl[row] = less_sum(l2);
    }
}

// Blocks [0, row_blocks): one warp per row.  Blocks beyond: sum_slots(MAXR)
// slots of one (sequence, KV head) each, weight += the kept logits' weights in
// row order; the logits are on their way while the block joins the head's rows
// for itself (waiting for the other blocks' rows instead would cost another
// launch).  Several slots a thread, so that the blocks of a call fit the GPU at
// once (12 heads of 32001 slots: 11.6 us with one, 7.2).
constexpr int sum_slots(int max_rows) { return max_rows <= 8 ? 512 : 256; }
template <typename T, int D, int MAXR>
__global__ void __launch_bounds__(128, MAXR > 1 ? 5 : 8) combine_kernel(const __grid_constant__ View a, int row_blocks) {
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
    constexpr int SLOTS = sum_slots(MAXR), V = SLOTS / 128;
    const int chunks = (a.cap + SLOTS - 1) / SLOTS;
    const int b = blockIdx.x - row_blocks, sh = b / chunks, j0 = b % chunks * SLOTS;
    const int s = sh / a.Hk, hk = sh % a.Hk, rps = a.rep * a.T;
    const int n = own_len(a, s, hk);
    if (j0 >= n) {
        ptx::grid_dep_wait();
        return;
    }
    const int pk = prefix_len(a, prefix_of(a, s));
    const int j = j0 + tid;
    float* w = a.weight + (int64_t)sh * a.cap + j;
    float old[V], x[MAXR][V];
#pragma unroll
    for (int v = 0; v < V; ++v) old[v] = j + 128 * v < n ? w[128 * v] : 0.f;
    ptx::grid_dep_wait();
    const float* lg = a.logit + (int64_t)sh * rps * a.lcap + j;
#pragma unroll
    for (int i = 0; i < MAXR; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) x[i][v] = i < rps && j + 128 * v < n ? lg[(int64_t)i * a.lcap + 128 * v] : -INFINITY;
    for (int i = warp; i < rps; i += 4) {
        const RowJoin r = join_row(a, row_of(a, s, hk, i), pk, n);
        if (lane == 0) ml_s[i] = make_float2(r.M, r.M == -INFINITY ? 0.f : 1.f / r.L);
    }
    __syncthreads();
    float sum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.f;
#pragma unroll
    for (int i = 0; i < MAXR; ++i)
        if (i < rps) {
            const float2 y = ml_s[i];
            if (y.x == -INFINITY) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) sum[v] += exp2f(x[i][v] - y.x) * y.y;
        }
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (j + 128 * v < n) w[128 * v] = old[v] + sum[v];
}

// ---------------------------------------------------------------------------
// accumulated weights of many rows: the logits once more, summed by key
// ---------------------------------------------------------------------------

// One block per (sequence, KV head, KT keys): lane = key, the warps share the
// rows of each tile; a key's weight 2^(x - lse) over the rows that see it, per
// tile, then over the tiles, then over the warps.  The next rows are on their
// way.
template <int D, typename C>
__global__ void __launch_bounds__(C::THREADS, 4) column_sums_f32_kernel(const __grid_constant__ View a) {
    extern __shared__ __align__(16) unsigned char raw[];
    constexpr int RT = C::RT, KT = C::KT, RW = C::RW, KPL = C::KPL, THREADS = C::THREADS;
    typename C::SumSmem& sm = *reinterpret_cast<typename C::SumSmem*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // the first keys, which the most queries see, first
    const int heads = a.S * a.Hk, sh = blockIdx.x % heads, k0 = blockIdx.x / heads * KT;
    const int s = sh / a.Hk, hk = sh % a.Hk, rps = a.rep * a.T;
    ptx::grid_dep_wait();
    const int n = own_len(a, s, hk);
    if (k0 >= n) return;
    const float* kb = static_cast<const float*>(a.k) + s * a.ks[0] + hk * a.ks[1];
    for (int e = tid; e < KT * (D / 4); e += THREADS) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        cp16(ptx::smem_u32(&sm.k[r][c]), kb + (int64_t)(k0 + r < n ? k0 + r : k0) * a.ks[2] + c, k0 + r < n);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // the first row that sees key k0: n - T + t + 1 > k0
    const int t0 = max(0, k0 - (n - a.T));
    constexpr int Q4 = RT * (D / 4) / THREADS;
    float4 next[Q4];
    auto fetch = [&](int f) {
#pragma unroll
        for (int e = 0; e < Q4; ++e) {
            const int idx = e * THREADS + tid, i = f + idx / (D / 4), c = idx % (D / 4) * 4;
            const int t = query_of(a, i);
            next[e] = i < rps ? *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + s * a.qs[0] +
                                                                 (hk * a.rep + i - t * a.rep) * a.qs[1] + t * a.qs[2] + c)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    const int f0 = t0 * a.rep / RT * RT;
    fetch(f0);
    float total[KPL];
#pragma unroll
    for (int p = 0; p < KPL; ++p) total[p] = 0.f;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (int f = f0; f < rps; f += RT) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < Q4; ++e) {
            const int idx = e * THREADS + tid;
            const float4 y = next[e];
            *reinterpret_cast<float4*>(&sm.q[idx / (D / 4)][idx % (D / 4) * 4]) =
                make_float4(y.x * a.qscale, y.y * a.qscale, y.z * a.qscale, y.w * a.qscale);
        }
        __syncthreads();
        if (f + RT < rps) fetch(f + RT);
        float nl[RW];
#pragma unroll
        for (int u = 0; u < RW; ++u) {
            const int i = f + warp * RW + u;
            nl[u] = i < rps ? a.row_nl[row_of(a, s, hk, i)] : -INFINITY;
        }
        if (f + warp * RW >= rps) continue;
        float x[RW][KPL], tile[KPL];
        dots<D, KPL>(x, &sm.q[warp * RW], sm.k, lane);
#pragma unroll
        for (int p = 0; p < KPL; ++p) tile[p] = 0.f;
#pragma unroll
        for (int u = 0; u < RW; ++u)
#pragma unroll
            for (int p = 0; p < KPL; ++p)
                if (nl[u] != -INFINITY && k0 + lane + 32 * p < own_limit(a, n, f + warp * RW + u))
                    tile[p] += exp2f(x[u][p] + nl[u]);
#pragma unroll
        for (int p = 0; p < KPL; ++p) total[p] += tile[p];
    }
#pragma unroll
    for (int p = 0; p < KPL; ++p) sm.part[warp][lane + 32 * p] = total[p];
    __syncthreads();
    if (tid < KT && k0 + tid < n) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) sum += sm.part[w][tid];
        a.weight[(int64_t)sh * a.cap + k0 + tid] += sum;
    }
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

namespace {

template <int D, typename C> cudaError_t attend_f32(const View& a, bool rows_too, cudaStream_t st) {
    const int rps = a.rep * a.T, otiles = rows_too ? (rps + C::RT - 1) / C::RT : 0;
    const int64_t ptiles = a.np ? max_prefix_tiles(a.S, a.G, rps, C::RT) : 0;
    const int64_t blocks = ptiles * a.Hk * a.np + (int64_t)a.S * a.Hk * otiles * a.no;
    return launch(attend_f32_kernel<D, C>, blocks, C::THREADS, sizeof(typename C::Smem) + (size_t)a.G * 4, st, a,
                  (int)ptiles, otiles);
}
template <int D, typename C> cudaError_t prepare_f32() {
    cudaError_t e = cudaFuncSetAttribute(attend_f32_kernel<D, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(typename C::Smem) + MAX_PREFIXES * 4);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(column_sums_f32_kernel<D, ManyF32<D>>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sizeof(typename ManyF32<D>::SumSmem));
    return e;
}
template <int D> cudaError_t sums_f32(const View& a, cudaStream_t st) {
    using C = ManyF32<D>;
    return launch(column_sums_f32_kernel<D, C>, (int64_t)a.S * a.Hk * ((a.cap + C::KT - 1) / C::KT), C::THREADS,
                  sizeof(typename C::SumSmem), st, a);
}

}  // namespace

cudaError_t launch_attend_f32(const View& a, int d, bool rows_too, cudaStream_t st) {
    if (a.rep * a.T <= STREAM_ROWS)
        return d == 64 ? attend_f32<64, FewF32<64>>(a, rows_too, st) : attend_f32<128, FewF32<128>>(a, rows_too, st);
    return d == 64 ? attend_f32<64, ManyF32<64>>(a, rows_too, st) : attend_f32<128, ManyF32<128>>(a, rows_too, st);
}

cudaError_t launch_column_sums_f32(const View& a, int d, cudaStream_t st) {
    return d == 64 ? sums_f32<64>(a, st) : sums_f32<128>(a, st);
}

cudaError_t prepare_shared_f32() {
    cudaError_t e = prepare_f32<64, FewF32<64>>();
    if (e == cudaSuccess) e = prepare_f32<128, FewF32<128>>();
    if (e == cudaSuccess) e = prepare_f32<64, ManyF32<64>>();
    if (e == cudaSuccess) e = prepare_f32<128, ManyF32<128>>();
    return e;
}

cudaError_t launch_combine(const View& a, int dtype, int d, cudaStream_t st) {
    const int64_t R = (int64_t)a.S * a.H * a.T, rb = (R + 3) / 4;
    const int rps = a.rep * a.T, slots = sum_slots(rps);
    const int64_t blocks = rb + (a.logit ? (int64_t)a.S * a.Hk * ((a.cap + slots - 1) / slots) : 0);
    return by_type(dtype, d, [&](auto tag, auto dim) {
        using E = decltype(tag);
        constexpr int D = decltype(dim)::value;
        if (rps == 1) return launch(combine_kernel<E, D, 1>, blocks, 128, 0, st, a, (int)rb);
        if (rps <= 8) return launch(combine_kernel<E, D, 8>, blocks, 128, 0, st, a, (int)rb);
        return launch(combine_kernel<E, D, STREAM_ROWS>, blocks, 128, 0, st, a, (int)rb);
    });
}

}  // namespace shared
}  // namespace hkv
