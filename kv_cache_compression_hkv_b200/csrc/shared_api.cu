// shared_api.cu -- the C entry points of the shared-prefix cache: argument
// checks, how a call is split over blocks, and launches.
#include <math.h>
#include <string.h>

#include "kernels.h"
#include "shared.cuh"

using hkv::shared::View;

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxSlots = 1 << 24;    // capacity, prefix_capacity
constexpr int kMaxRows = 1 << 24;     // S * Hkv, and query rows of one (sequence, KV head)

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Row bases and strides on 16-byte boundaries (a negative or zero stride is
// the caller's: a zero one repeats rows, which only inputs may).
bool rows_ok(const void* p, const int64_t* st, int64_t es) {
    if (!p || !aligned(p, 16)) return false;
    for (int i = 0; i < 3; ++i)
        if (st[i] * es % 16 != 0 || st[i] < 0) return false;
    return true;
}

bool cache_ok(const hkv_shared_cache* c) {
    if (!c) return false;
    if (c->dtype != HKV_DTYPE_F32 && c->dtype != HKV_DTYPE_BF16) return false;
    if (c->head_dim != 64 && c->head_dim != 128) return false;
    if (c->num_seqs < 1 || c->num_heads < 1 || c->num_kv_heads < 1 || c->num_heads % c->num_kv_heads) return false;
    if ((int64_t)c->num_seqs * c->num_heads > kMaxRows) return false;
    if (c->capacity < 1 || c->capacity > kMaxSlots) return false;
    if (c->num_prefixes < 0 || c->num_prefixes > hkv::shared::MAX_PREFIXES) return false;
    const int64_t es = c->dtype == HKV_DTYPE_F32 ? 4 : 2;
    if (!rows_ok(c->k, c->k_stride, es) || !rows_ok(c->v, c->v_stride, es)) return false;
    if (c->k_stride[2] < c->head_dim || c->v_stride[2] < c->head_dim) return false;
    if (!c->len || !aligned(c->len, 4) || !aligned(c->pos, 4) || !aligned(c->weight, 4) || !aligned(c->next_pos, 4) ||
        !aligned(c->status, 4))
        return false;
    if (c->num_prefixes > 0) {
        if (c->prefix_capacity < 1 || c->prefix_capacity > kMaxSlots) return false;
        if (!rows_ok(c->prefix_k, c->prefix_k_stride, es) || !rows_ok(c->prefix_v, c->prefix_v_stride, es)) return false;
        if (!c->prefix_len || !c->prefix_of || !aligned(c->prefix_len, 4) || !aligned(c->prefix_of, 4)) return false;
    }
    return true;
}

View view_of(const hkv_shared_cache* c) {
    View a;
    memset(&a, 0, sizeof(a));
    a.S = c->num_seqs; a.H = c->num_heads; a.Hk = c->num_kv_heads; a.rep = c->num_heads / c->num_kv_heads;
    a.cap = c->capacity; a.G = c->num_prefixes; a.pcap = c->prefix_capacity;
    a.k = c->k; a.v = c->v;
    a.pos = c->pos; a.weight = c->weight; a.len = c->len; a.next_pos = c->next_pos;
    a.pk = c->prefix_k; a.pv = c->prefix_v; a.plen = c->prefix_len; a.pof = c->prefix_of;
    a.status = c->status;
    for (int i = 0; i < 3; ++i) {
        a.ks[i] = c->k_stride[i]; a.vs[i] = c->v_stride[i];
        a.pks[i] = c->prefix_k_stride[i]; a.pvs[i] = c->prefix_v_stride[i];
    }
    return a;
}

// How an attention call is split, and its scratch carved from `base` (sizes
// alone when base is null).
size_t plan_attend(View& a, int d, int T, int accumulate, unsigned char* base) {
    a.T = T;
    a.accumulate = accumulate;
    const int64_t rps = (int64_t)a.rep * T, R = (int64_t)a.S * a.H * T;
    const bool stream = rps <= hkv::shared::STREAM_ROWS;
    // enough blocks for every SM to hold several, ranges of 64 keys at least
    auto splits = [&](int64_t tiles, int64_t keys) {
        int64_t n = (148 * 6 + tiles - 1) / tiles;
        n = n < (keys + 127) / 128 ? n : (keys + 127) / 128;
        return (int)(n < 1 ? 1 : n > hkv::shared::MAX_SPLITS ? hkv::shared::MAX_SPLITS : n);
    };
    a.no = splits((int64_t)a.S * a.Hk * ((rps + 15) / 16), a.cap);
    a.np = a.G ? splits(a.Hk * ((int64_t)a.S * rps / 16 + 1), a.pcap) : 0;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        unsigned char* p = base ? base + o : nullptr;
        o = align_up(o + bytes);
        return p;
    };
    const size_t ns = a.np + a.no;
    a.part_ml = (float2*)take(ns * R * sizeof(float2));
    a.part_o = (float*)take(ns * R * d * sizeof(float));
    if (accumulate && stream) a.logit = (float*)take((size_t)a.S * a.Hk * rps * a.cap * 4);
    if (accumulate && !stream) a.row_lse = (float*)take((size_t)R * 4);
    return o;
}

bool queries_ok(const hkv_shared_cache* c, int T) {
    return T >= 1 && T <= c->capacity && (int64_t)T * (c->num_heads / c->num_kv_heads) <= kMaxRows &&
           (int64_t)c->num_seqs * c->num_heads * T <= (int64_t)1 << 30;
}

hkv_status cuda_status(cudaError_t e) { return e == cudaSuccess ? HKV_OK : HKV_ERR_CUDA; }

}  // namespace

extern "C" {

hkv_status hkv_shared_append(const hkv_shared_cache* c, const void* k_t, const int64_t* k_stride, const void* v_t,
                             const int64_t* v_stride, const float* weight_t, int32_t num_tokens, void* stream) {
    if (!cache_ok(c) || !k_stride || !v_stride || num_tokens < 0 || num_tokens > c->capacity || !aligned(weight_t, 4))
        return HKV_ERR_INVALID_ARG;
    const int64_t es = c->dtype == HKV_DTYPE_F32 ? 4 : 2;
    if (!rows_ok(k_t, k_stride, es) || !rows_ok(v_t, v_stride, es)) return HKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return HKV_OK;
    View a = view_of(c);
    a.T = num_tokens;
    return cuda_status(hkv::shared::launch_append(a, c->dtype, c->head_dim, k_t, k_stride, v_t, v_stride, weight_t,
                                                  (cudaStream_t)stream));
}

hkv_status hkv_shared_attend_bytes(const hkv_shared_cache* c, int32_t num_queries, int32_t accumulate, size_t* bytes) {
    if (!bytes || !cache_ok(c) || !queries_ok(c, num_queries) || (accumulate != 0 && accumulate != 1))
        return HKV_ERR_INVALID_ARG;
    View a = view_of(c);
    *bytes = plan_attend(a, c->head_dim, num_queries, accumulate, nullptr);
    return HKV_OK;
}

hkv_status hkv_shared_attend(const hkv_shared_cache* c, const void* q, const int64_t* q_stride, void* out,
                             const int64_t* out_stride, float* lse, int32_t num_queries, double scale,
                             int32_t accumulate, void* scratch, size_t scratch_bytes, void* stream) {
    if (!cache_ok(c) || !queries_ok(c, num_queries) || !q_stride || !out_stride || !aligned(lse, 4) ||
        (accumulate != 0 && accumulate != 1) || (accumulate && !c->weight) || !isfinite(scale))
        return HKV_ERR_INVALID_ARG;
    const int64_t es = c->dtype == HKV_DTYPE_F32 ? 4 : 2;
    if (!rows_ok(q, q_stride, es) || !rows_ok(out, out_stride, es)) return HKV_ERR_INVALID_ARG;
    View a = view_of(c);
    if (scratch_bytes < plan_attend(a, c->head_dim, num_queries, accumulate, nullptr)) return HKV_ERR_CAPACITY;
    if (!scratch || !aligned(scratch, kAlign)) return HKV_ERR_INVALID_ARG;
    plan_attend(a, c->head_dim, num_queries, accumulate, (unsigned char*)scratch);
    a.q = q;
    a.out = out;
    a.lse = lse;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = q_stride[i];
        a.os[i] = out_stride[i];
    }
    a.qscale = (float)((scale == 0.0 ? 1.0 / sqrt((double)c->head_dim) : scale) * 1.4426950408889634);
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = hkv::shared::launch_attend_simt(a, c->dtype, c->head_dim, st);
    if (e == cudaSuccess) e = hkv::shared::launch_combine(a, c->dtype, c->head_dim, st);
    if (e == cudaSuccess && a.row_lse) e = hkv::shared::launch_column_sums_simt(a, c->dtype, c->head_dim, st);
    return cuda_status(e);
}

hkv_status hkv_shared_evict_bytes(const hkv_shared_cache* c, size_t* bytes) {
    if (!bytes || !cache_ok(c)) return HKV_ERR_INVALID_ARG;
    *bytes = (size_t)c->num_seqs * c->num_kv_heads * c->capacity * 4;
    return HKV_OK;
}

hkv_status hkv_shared_evict(const hkv_shared_cache* c, const int32_t* budget, int32_t recent, int32_t slack,
                            void* scratch, size_t scratch_bytes, void* stream) {
    if (!cache_ok(c) || !c->pos || !c->weight || !budget || !aligned(budget, 4) || recent < 0 || slack < 1)
        return HKV_ERR_INVALID_ARG;
    size_t need = 0;
    hkv_shared_evict_bytes(c, &need);
    if (scratch_bytes < need) return HKV_ERR_CAPACITY;
    if (!scratch || !aligned(scratch, kAlign)) return HKV_ERR_INVALID_ARG;
    View a = view_of(c);
    return cuda_status(hkv::shared::launch_evict(a, c->dtype, c->head_dim, budget, recent, slack, (int32_t*)scratch,
                                                 (cudaStream_t)stream));
}

}  // extern "C"
