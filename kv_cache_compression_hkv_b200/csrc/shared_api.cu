// shared_api.cu -- the C entry points of the shared-prefix cache: argument
// checks, how a call is split over blocks, and launches.
#include <math.h>
#include <string.h>

#include <atomic>

#include "kernels.h"
#include "shared.cuh"

using hkv::shared::SMS;
using hkv::shared::View;

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxSlots = 1 << 24;    // capacity, prefix_capacity
constexpr int64_t kMaxStride = (int64_t)1 << 37;  // elements
constexpr int kMaxRows = 1 << 24;     // S * Hkv, and query rows of one (sequence, KV head)

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Row bases and strides on 16-byte boundaries.
bool rows_ok(const void* p, const int64_t* st, int64_t es) {
    if (!p || !aligned(p, 16)) return false;
    for (int i = 0; i < 3; ++i)
        if (st[i] < 0 || st[i] > kMaxStride || st[i] * es % 16 != 0) return false;
    return true;
}
// The same for rows that are held: no dimension of more than one element repeats its rows.
bool held_ok(const void* p, const int64_t* st, int64_t es, int n0, int n1, int n2) {
    return rows_ok(p, st, es) && (n0 == 1 || st[0] > 0) && (n1 == 1 || st[1] > 0) && (n2 == 1 || st[2] > 0);
}

bool cache_ok(const hkv_shared_cache* c) {
    if (!c) return false;
    if (c->dtype != HKV_DTYPE_F32 && c->dtype != HKV_DTYPE_BF16) return false;
    if (c->head_dim != 64 && c->head_dim != 128) return false;
    if (c->num_seqs < 1 || c->num_heads < 1 || c->num_kv_heads < 1 || c->num_heads % c->num_kv_heads) return false;
    if ((int64_t)c->num_seqs * c->num_heads > kMaxRows || c->num_heads / c->num_kv_heads > 0xffff) return false;
    if (c->capacity < 1 || c->capacity > kMaxSlots) return false;
    if (c->num_prefixes < 0 || c->num_prefixes > hkv::shared::MAX_PREFIXES) return false;
    const int64_t es = c->dtype == HKV_DTYPE_F32 ? 4 : 2;
    if (!held_ok(c->k, c->k_stride, es, c->num_seqs, c->num_kv_heads, c->capacity) ||
        !held_ok(c->v, c->v_stride, es, c->num_seqs, c->num_kv_heads, c->capacity))
        return false;
    if (c->capacity > 1 && (c->k_stride[2] < c->head_dim || c->v_stride[2] < c->head_dim)) return false;
    if (!c->len || !aligned(c->len, 4) || !aligned(c->pos, 4) || !aligned(c->weight, 4) || !aligned(c->next_pos, 4) ||
        !aligned(c->status, 4))
        return false;
    if (c->num_prefixes > 0) {
        if (c->prefix_capacity < 1 || c->prefix_capacity > kMaxSlots) return false;
        if (!held_ok(c->prefix_k, c->prefix_k_stride, es, c->num_prefixes, c->num_kv_heads, c->prefix_capacity) ||
            !held_ok(c->prefix_v, c->prefix_v_stride, es, c->num_prefixes, c->num_kv_heads, c->prefix_capacity))
            return false;
        if (!c->prefix_len || !c->prefix_of || !aligned(c->prefix_len, 4) || !aligned(c->prefix_of, 4)) return false;
    }
    return true;
}

View view_of(const hkv_shared_cache* c) {
    View a;
    memset(&a, 0, sizeof(a));
    a.S = c->num_seqs; a.H = c->num_heads; a.Hk = c->num_kv_heads; a.rep = c->num_heads / c->num_kv_heads;
    a.rep_inv = (((uint64_t)1 << 40) + a.rep - 1) / a.rep;
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

// The kernels of an attention call, and how its keys are split over blocks.
// Few rows a (sequence, KV head) (STREAM_ROWS): the own keys are streamed; the
// prefix's either with them (folded: each sequence reads it again, from L2) or
// once for the rows of all its sequences, by tiles that leave partial results
// for the joining kernel.  Folding saves that kernel and the joining, and costs
// the re-reads: see FOLD_BYTES.  More rows: prefix and own keys in one pass, cut
// only where there are too few row tiles.
struct Plan {
    bool umma_prefix, umma_rows, stream;
    int warps_per_head;  // of the stream kernel
    size_t bytes;
};

// Bytes of prefix rows that all sequences together read up to which they are
// folded.  (us, d = 128, folded / once: 1024 heads over 64, 192, 384 shared keys
// 13.9 / 20.4, 19.0 / 21.2, 26.5 / 23.0, which is 34, 101, 201 MB; 128 heads of
// four query heads over 1024, 2048: 13.9 / 16.8, 19.2 / 18.4, or 67, 134 MB.)
// fp32 up to half of that, as its rows cost arithmetic (1024 heads over 64: 23.9 /
// 30.8, 67 MB; 640 heads, d = 64, over 300: 32.0 / 24.2, 98 MB).
constexpr int64_t FOLD_BYTES = 128 << 20;

// Row tiles from which on their keys are not cut, so that no joining follows.
// (us, whole / two pieces.  bf16, one tile of 49 rows a block: 84 blocks over 590 keys
// 19.8 / 25.7, over 16000 343 / 294; 104 blocks 20.2 / 26.8, 362 / 349; 120 over 16000
// 370 / 393; two tiles a block over up to 1280 keys: 60 blocks 40.7 / 45.1, 80 41.2 /
// 50.9, 120 42.4 / 71.0, 160 44.6 / 87.2; over up to 4352: 96 121 / 107, 128 123 / 122.
// fp32, 32 rows a block: 180 over 233 keys 49.1 / 48.7, over 2033 286 / 217; 240 52.5 /
// 58.2, 308 / 270; 300 58.5 / 63.2, 369 / 364; of 16 rows: 200 over 2033 185 / 104, 400
// over 233 34.2 / 41.1.)
constexpr int64_t UNCUT = 100, UNCUT_F32 = 240;

Plan plan_attend(View& a, int dtype, int d, int T, int accumulate, unsigned char* base) {
    a.T = T;
    const int64_t rps = (int64_t)a.rep * T, R = (int64_t)a.S * a.H * T, heads = (int64_t)a.S * a.Hk;
    const bool few = rps <= hkv::shared::STREAM_ROWS, bf16 = dtype == HKV_DTYPE_BF16;
    const bool fold = a.G == 0 || !few || heads * a.pcap * d * (bf16 ? 4 : 8) <= (bf16 ? FOLD_BYTES : FOLD_BYTES / 2);
    const int64_t keys = (int64_t)a.cap + (fold && a.G ? a.pcap : 0);  // of a list of keys, at most
    Plan p;
    p.stream = few && (bf16 || rps <= hkv::shared::STREAM_ROWS_F32);
    p.umma_rows = bf16 && !few;
    p.umma_prefix = bf16 && !fold;
    p.warps_per_head = 1;
    // `want` blocks over `tiles`, at least `least` keys a split
    auto splits = [&](int64_t want, int64_t tiles, int64_t n_keys, int64_t least) {
        int64_t n = (want + tiles - 1) / tiles, most = (n_keys + least - 1) / least;
        n = n < most ? n : most;
        return (int)(n < 1 ? 1 : n > hkv::shared::MAX_SPLITS ? hkv::shared::MAX_SPLITS : n);
    };
    a.listed = fold;
    a.lcap = (a.cap + 3) & ~3;
    if (p.umma_rows) {
        const int nt = hkv::shared::umma_row_tiles(rps);
        const int64_t items = heads * ((rps + 128 * nt - 1) / (128 * nt));
        a.no = items >= UNCUT ? 1 : splits(SMS * (nt == 2 ? 1 : 2), items, keys, 256);
    } else if (p.stream) {
        // eight warps fit an SM: a head goes to as many as fill the GPU, one or
        // several blocks of four (one warp / a block a head: 1024 heads of 28 to
        // 138 tokens 13.8 / 19.6 us, 512 of 56 to 477 24.5 / 18.4)
        const int64_t warps = (SMS * 8 + heads / 2) / heads, most = (keys + 31) / 32;
        const int64_t n = warps < most ? warps : most;
        p.warps_per_head = n > 1 ? 4 : 1;
        a.no = splits((n + 2) / 4, 1, keys, 64);
    } else {
        const int64_t items = heads * (few ? 1 : (rps + 31) / 32);
        a.no = items >= UNCUT_F32 ? 1 : splits(SMS * (few ? 4 : 2), items, keys, 128);
    }
    a.np = 0;
    if (!fold) {
        const int64_t tiles = (a.S * rps + 127) / 128, groups = a.G < a.S ? a.G : a.S;
        // two blocks of tiles fit an SM; a third of the places is left to the
        // streaming kernel's blocks, which need the other resource (48 sequences,
        // 16384 shared keys: 62.9 us in 192 blocks, 65.1 in 304, 65.4 in 144)
        const int64_t items = a.Hk * (tiles > groups ? tiles : groups);
        a.np = bf16 ? splits(items > 200 ? 1 : 200 / items, 1, a.pcap, 128)
                    : splits(SMS * 6, a.Hk * (a.S * rps / 16 + 1), a.pcap, 128);
    }
    size_t o = 0;
    auto take = [&](size_t bytes) {
        unsigned char* q = base ? base + o : nullptr;
        o = align_up(o + bytes);
        return q;
    };
    const size_t ns = a.np + a.no;
    if (ns > 1) {
        a.part_ml = (float2*)take(ns * R * sizeof(float2));
        a.part_o = (float*)take(ns * R * d * sizeof(float));
    }
    a.sum_tiles = accumulate && p.umma_rows && a.no == 1 && rps <= hkv::shared::ONE_TILE_ROWS ? (int)((rps + 127) / 128) : 0;
    if (accumulate && few) a.logit = (float*)take((size_t)heads * rps * a.lcap * 4);
    if (a.sum_tiles > 1) a.part_sum = (float*)take((size_t)a.sum_tiles * heads * a.cap * 4);
    if (accumulate && !few && !a.sum_tiles) a.row_nl = (float*)take((size_t)R * 4);
    p.bytes = o;
    return p;
}

// Raises the kernels' shared-memory limits, once per device.
cudaError_t prepare() {
    static std::atomic<unsigned long long> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (ready.load() & bit) return cudaSuccess;
    e = hkv::shared::prepare_shared_umma();
    if (e == cudaSuccess) e = hkv::shared::prepare_shared_stream();
    if (e == cudaSuccess) e = hkv::shared::prepare_shared_stream_f32();
    if (e == cudaSuccess) e = hkv::shared::prepare_shared_evict();
    if (e == cudaSuccess) e = hkv::shared::prepare_shared_f32();
    if (e == cudaSuccess && dev < 64) ready.fetch_or(bit);
    return e;
}

bool queries_ok(const hkv_shared_cache* c, int T) {
    return T >= 1 && T <= c->capacity && (int64_t)T * (c->num_heads / c->num_kv_heads) < kMaxRows &&
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
    *bytes = plan_attend(a, c->dtype, c->head_dim, num_queries, accumulate, nullptr).bytes;
    return HKV_OK;
}

hkv_status hkv_shared_attend(const hkv_shared_cache* c, const void* q, const int64_t* q_stride, void* out,
                             const int64_t* out_stride, float* lse, int32_t num_queries, double scale,
                             int32_t accumulate, void* scratch, size_t scratch_bytes, void* stream) {
    if (!cache_ok(c) || !queries_ok(c, num_queries) || !q_stride || !out_stride || !aligned(lse, 4) ||
        (accumulate != 0 && accumulate != 1) || (accumulate && !c->weight) || !isfinite(scale))
        return HKV_ERR_INVALID_ARG;
    const int64_t es = c->dtype == HKV_DTYPE_F32 ? 4 : 2;
    if (!held_ok(q, q_stride, es, c->num_seqs, c->num_heads, num_queries) ||
        !held_ok(out, out_stride, es, c->num_seqs, c->num_heads, num_queries))
        return HKV_ERR_INVALID_ARG;
    View a = view_of(c);
    const double sc = (scale == 0.0 ? 1.0 / sqrt((double)c->head_dim) : scale) * 1.4426950408889634;
    if (!(fabs(sc) >= 1e-30 && fabs(sc) <= 1e30)) return HKV_ERR_INVALID_ARG;
    const Plan p = plan_attend(a, c->dtype, c->head_dim, num_queries, accumulate, nullptr);
    if (scratch_bytes < p.bytes) return HKV_ERR_CAPACITY;
    if (p.bytes && (!scratch || !aligned(scratch, kAlign))) return HKV_ERR_INVALID_ARG;
    plan_attend(a, c->dtype, c->head_dim, num_queries, accumulate, p.bytes ? (unsigned char*)scratch : nullptr);
    a.q = q;
    a.out = out;
    a.lse = lse;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = q_stride[i];
        a.os[i] = out_stride[i];
    }
    a.qscale = (float)sc;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = prepare();
    const int d = c->head_dim;
    if (e == cudaSuccess && p.umma_rows) e = hkv::shared::launch_attend_umma(a, d, st);
    if (e == cudaSuccess && p.umma_prefix) e = hkv::shared::launch_prefix_umma(a, d, st);
    if (e == cudaSuccess && c->dtype == HKV_DTYPE_F32 && (!p.stream || a.np))
        e = hkv::shared::launch_attend_f32(a, d, !p.stream, st);
    if (e == cudaSuccess && p.stream)
        e = c->dtype == HKV_DTYPE_F32 ? hkv::shared::launch_stream_f32(a, d, p.warps_per_head, a.np > 0, st)
                                      : hkv::shared::launch_stream(a, d, p.warps_per_head, a.np > 0, st);
    if (e == cudaSuccess && a.part_ml) e = hkv::shared::launch_combine(a, c->dtype, d, st);
    if (e == cudaSuccess && a.part_sum) e = hkv::shared::launch_add_sums(a, st);
    if (e == cudaSuccess && a.row_nl)
        e = p.umma_rows ? hkv::shared::launch_column_sums_umma(a, d, st)
                        : hkv::shared::launch_column_sums_f32(a, d, st);
    return cuda_status(e);
}

hkv_status hkv_shared_evict_bytes(const hkv_shared_cache* c, size_t* bytes) {
    if (!bytes || !cache_ok(c)) return HKV_ERR_INVALID_ARG;
    *bytes = align_up(hkv::shared::evict_bytes(c->num_seqs * c->num_kv_heads, c->capacity));
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
    cudaError_t e = prepare();
    if (e == cudaSuccess)
        e = hkv::shared::launch_evict(a, c->dtype, c->head_dim, budget, recent, slack, (unsigned char*)scratch,
                                      (cudaStream_t)stream);
    return cuda_status(e);
}

}  // extern "C"
