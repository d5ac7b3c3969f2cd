// Host side of the attention operators (include/colibri_attn.h): argument
// checks, the split of the keys, the launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "attn.h"
#include "colibri_attn.h"
#include "common.cuh"
#include "kernels.h"

using namespace colibri;

namespace {

// The grids are sized for the GPU this library is built for, so that a
// workspace's size does not depend on the machine that asks for it.
constexpr int kSms = 152;
constexpr int kMaxSplits = 64;

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

constexpr int kCodes = -8;         // dtype of a view of 8-bit pages
int elem_size(int dtype) { return dtype == COLIBRI_DTYPE_BF16 ? 2 : dtype == kCodes ? 1 : 4; }
int rows_of(int dtype) { return dtype == kCodes ? (int)COLIBRI_DTYPE_BF16 : dtype; }      // dtype of q and o
DType dtype_of(int dtype) { return rows_of(dtype) == COLIBRI_DTYPE_BF16 ? DType::BF16 : DType::F32; }

// A row tensor [rows, heads, d] with `stride` elements from row to row.
bool rows_ok(const void* p, int64_t stride, int heads, int d, int esz) {
    return p && aligned16(p) && stride >= (int64_t)heads * d && (stride * esz) % 16 == 0 &&
           stride * esz < ((int64_t)1 << 40);
}

bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
    return pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

// Rows of a tensor: `rows` times `width` bytes, `stride` bytes apart.
struct Rows {
    const void* p;
    int64_t stride, width;
    int64_t extent(int64_t rows) const { return (rows - 1) * stride + width; }
};
Rows row_bytes(const void* p, int64_t stride, int heads, int d, int esz) {
    return {p, stride * esz, (int64_t)heads * d * esz};
}
// They share a byte.  Column ranges of one tensor's rows (equal strides) may lie
// between each other; other tensors may not.
bool clash(const Rows& a, const Rows& b, int64_t rows) {
    if (rows <= 0 || !overlap(a.p, a.extent(rows), b.p, b.extent(rows))) return false;
    if (a.stride != b.stride) return true;
    int64_t off = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p) % a.stride;
    if (off < 0) off += a.stride;
    return off < a.width || off + b.width > a.stride;
}

colibri_status_t check_heads(int n_q_heads, int n_kv_heads, int head_dim, int dtype) {
    if (dtype != COLIBRI_DTYPE_FP32 && dtype != COLIBRI_DTYPE_BF16) return COLIBRI_ERR_INVALID_ARG;
    if (n_q_heads <= 0 || n_kv_heads <= 0 || head_dim <= 0 || n_q_heads % n_kv_heads)
        return COLIBRI_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || n_q_heads / n_kv_heads > 128 || n_kv_heads > 65535 ||
        n_q_heads > 65535)
        return COLIBRI_ERR_UNSUPPORTED;
    return COLIBRI_OK;
}

// paged: the sizes of pages too (keys without pages: check_prompt).
colibri_status_t check_kv(const colibri_kv_pages_t* kv, bool paged) {
    if (!kv || !kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return COLIBRI_ERR_INVALID_ARG;
    if (kv->num_pages <= 0 || kv->page_size <= 0) return COLIBRI_ERR_INVALID_ARG;
    const int esz = elem_size(kv->dtype);
    for (const int64_t s : {kv->page_stride, kv->head_stride, kv->row_stride})
        if (s < 0 || (s * esz) % 16 || s >= ((int64_t)1 << 37)) return COLIBRI_ERR_INVALID_ARG;
    if (kv->row_stride < kv->head_dim || (kv->n_kv_heads > 1 && kv->head_stride < kv->head_dim) ||
        (kv->num_pages > 1 && kv->page_stride < kv->head_dim))
        return COLIBRI_ERR_INVALID_ARG;
    if (paged && (kv->page_size < 8 || kv->page_size > 65536 || (kv->page_size & (kv->page_size - 1))))
        return COLIBRI_ERR_UNSUPPORTED;
    return COLIBRI_OK;
}

// Bytes from the first to behind the last element of k (or v).
int64_t kv_extent(const colibri_kv_pages_t* kv) {
    return ((int64_t)(kv->num_pages - 1) * kv->page_stride +
            (int64_t)(kv->n_kv_heads - 1) * kv->head_stride +
            (int64_t)(kv->page_size - 1) * kv->row_stride + kv->head_dim) * elem_size(kv->dtype);
}

colibri_status_t check_seqs(const colibri_seqs_t* s, int n_q_heads) {
    if (!s || s->n_seqs < 0 || s->n_rows < 0 || s->table_stride < 0) return COLIBRI_ERR_INVALID_ARG;
    if (!s->seq_start && s->n_rows != s->n_seqs) return COLIBRI_ERR_INVALID_ARG;
    // (without sequences the arrays have no entries, and may be NULL)
    if (s->n_seqs > 0 && s->page_table && (!s->kv_len || s->table_stride <= 0)) return COLIBRI_ERR_INVALID_ARG;
    for (const int32_t* p : {s->seq_start, s->kv_len, s->page_table})
        if ((uintptr_t)p & 3) return COLIBRI_ERR_INVALID_ARG;
    if (((int64_t)s->n_rows + s->n_seqs) * std::max(n_q_heads, 128) > INT32_MAX) return COLIBRI_ERR_INVALID_ARG;
    return COLIBRI_OK;
}

colibri_status_t check_rope(const colibri_rope_t* r, int head_dim) {
    if (!r) return COLIBRI_OK;
    if (!r->freq || ((uintptr_t)r->freq & 7) || r->rot_dim <= 0 || r->rot_dim > head_dim ||
        r->rot_dim % 16 || !(std::isfinite(r->mscale)))
        return COLIBRI_ERR_INVALID_ARG;
    if (r->style != COLIBRI_ROPE_HALF && r->style != COLIBRI_ROPE_INTERLEAVED)
        return COLIBRI_ERR_INVALID_ARG;
    return COLIBRI_OK;
}

colibri_status_t check_positions(const colibri_positions_t* p, const colibri_rope_t* rope, int n_rows) {
    if (!p) return COLIBRI_OK;
    if (!rope || p->n_axes < 1 || p->n_axes > 8 || ((uintptr_t)p->at & 3) || (n_rows > 0 && !p->at) ||
        (p->n_axes > 1 && p->axis_stride < 0) || p->axis_stride >= ((int64_t)1 << 37))
        return COLIBRI_ERR_INVALID_ARG;
    return COLIBRI_OK;
}

void set_rope(AppendArgs& a, const colibri_rope_t* rope, const colibri_positions_t* p) {
    if (!rope) return;
    a.freq = rope->freq, a.rot_dim = rope->rot_dim, a.mscale = rope->mscale;
    a.interleaved = rope->style == COLIBRI_ROPE_INTERLEAVED;
    if (p) a.positions = p->at, a.axis_stride = p->axis_stride, a.axis = p->axis, a.n_axes = p->n_axes;
}

int shift_of(int n) {
    int s = 0;
    while ((1 << s) < n) ++s;
    return s;
}

// 8-bit pages as pages whose elements are bytes.
colibri_kv_pages_t view(const colibri_kv_pages8_t* c) {
    return {c->k, c->v, c->page_stride, c->head_stride, c->row_stride, c->num_pages,
            c->page_size, c->n_kv_heads, c->head_dim, kCodes};
}
int64_t scale_bytes(const colibri_kv_pages8_t* c) {
    return (int64_t)c->num_pages * c->n_kv_heads * (c->page_size / c->block) * 4;
}

colibri_status_t check_kv8(const colibri_kv_pages8_t* c) {
    if (!c) return COLIBRI_ERR_INVALID_ARG;
    if (!c->k_scale || !c->v_scale || ((uintptr_t)c->k_scale & 3) || ((uintptr_t)c->v_scale & 3) || c->block <= 0 ||
        (c->code != COLIBRI_CODE_E4M3 && c->code != COLIBRI_CODE_INT8))
        return COLIBRI_ERR_INVALID_ARG;
    colibri_status_t st = check_heads(c->n_kv_heads, c->n_kv_heads, c->head_dim, COLIBRI_DTYPE_BF16);
    const colibri_kv_pages_t kv = view(c);
    if (st == COLIBRI_OK) st = check_kv(&kv, true);
    if (st != COLIBRI_OK) return st;
    if ((c->block != 16 && c->block != 32 && c->block != 64) || c->block > c->page_size) return COLIBRI_ERR_UNSUPPORTED;
    return COLIBRI_OK;
}

ValuesArgs values_args(const colibri_kv_pages8_t* c) {
    ValuesArgs a{};
    a.k = c->k, a.v = c->v, a.k_scale = c->k_scale, a.v_scale = c->v_scale;
    a.page_stride = c->page_stride, a.head_stride = c->head_stride, a.row_stride = c->row_stride;
    a.num_pages = c->num_pages, a.page_size = c->page_size, a.page_shift = shift_of(c->page_size);
    a.block_shift = shift_of(c->block), a.hkv = c->n_kv_heads;
    return a;
}

// The rows of an append.
struct Projection {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const void *q_norm, *k_norm;
    float eps;
    void* q_out;
    int64_t q_out_stride;
};

// Checks an append of rows of `dtype` and describes it; a->n_rows is 0 where there is
// nothing to do.
colibri_status_t check_append(const colibri_kv_pages_t* cache, int dtype, const colibri_seqs_t* seqs,
                              const colibri_rope_t* rope, const colibri_positions_t* positions, int n_q_heads,
                              const Projection& p, AppendArgs* out_args) {
    if (!seqs || (seqs->n_seqs > 0 && (!seqs->page_table || !seqs->kv_len))) return COLIBRI_ERR_INVALID_ARG;
    colibri_status_t st = check_heads(n_q_heads, cache->n_kv_heads, cache->head_dim, dtype);
    if (st == COLIBRI_OK) st = check_seqs(seqs, n_q_heads);
    if (st == COLIBRI_OK) st = check_kv(cache, true);
    if (st == COLIBRI_OK) st = check_rope(rope, cache->head_dim);
    if (st == COLIBRI_OK) st = check_positions(positions, rope, seqs->n_rows);
    if (st != COLIBRI_OK) return st;
    const int d = cache->head_dim, esz = elem_size(dtype), hkv = cache->n_kv_heads;
    if (!rows_ok(p.q, p.q_stride, n_q_heads, d, esz) || !rows_ok(p.k, p.k_stride, hkv, d, esz) ||
        !rows_ok(p.v, p.v_stride, hkv, d, esz) || !rows_ok(p.q_out, p.q_out_stride, n_q_heads, d, esz) ||
        !aligned16(p.q_norm) || !aligned16(p.k_norm) || !(p.eps >= 0.f))
        return COLIBRI_ERR_INVALID_ARG;
    if (p.q_out == p.q && p.q_out_stride != p.q_stride) return COLIBRI_ERR_INVALID_ARG;
    const Rows out = row_bytes(p.q_out, p.q_out_stride, n_q_heads, d, esz);
    if ((p.q_out != p.q && clash(row_bytes(p.q, p.q_stride, n_q_heads, d, esz), out, seqs->n_rows)) ||
        clash(row_bytes(p.k, p.k_stride, hkv, d, esz), out, seqs->n_rows) ||
        clash(row_bytes(p.v, p.v_stride, hkv, d, esz), out, seqs->n_rows))
        return COLIBRI_ERR_INVALID_ARG;
    for (const void* pages : {(const void*)cache->k, (const void*)cache->v})
        for (const Rows& r : {row_bytes(p.q, p.q_stride, n_q_heads, d, esz), row_bytes(p.k, p.k_stride, hkv, d, esz),
                              row_bytes(p.v, p.v_stride, hkv, d, esz), out})
            if (seqs->n_rows > 0 && overlap(pages, kv_extent(cache), r.p, r.extent(seqs->n_rows)))
                return COLIBRI_ERR_INVALID_ARG;
    if (seqs->n_rows == 0 || seqs->n_seqs == 0) return COLIBRI_OK;
    AppendArgs& a = *out_args;
    a.q = p.q, a.k = p.k, a.v = p.v;
    a.q_stride = p.q_stride, a.k_stride = p.k_stride, a.v_stride = p.v_stride;
    a.q_norm = p.q_norm, a.k_norm = p.k_norm, a.eps = p.eps;
    set_rope(a, rope, positions);
    a.seq_start = seqs->seq_start, a.kv_len = seqs->kv_len, a.table = seqs->page_table;
    a.n_seqs = seqs->n_seqs, a.n_rows = seqs->n_rows, a.table_stride = seqs->table_stride;
    a.hq = n_q_heads, a.hkv = hkv;
    a.q_out = p.q_out, a.q_out_stride = p.q_out_stride;
    a.k_out = cache->k, a.v_out = cache->v;
    a.page_stride = cache->page_stride, a.head_stride = cache->head_stride;
    a.row_stride = cache->row_stride, a.num_pages = cache->num_pages;
    a.page_shift = shift_of(cache->page_size);
    return COLIBRI_OK;
}


// How a call's keys are split: ranges of the shared prefix and of the
// sequences' own keys, each leaving a partial row per (row, head).  shares: the
// own keys run in equal shares per CTA (launch_attn_decode), which leaves at
// most one partial row per (row, head) and the pieces of the cut ones.
struct Plan {
    int prefix = 0;      // ranges of the prefix (0: no prefix launch)
    int own = 1;         // ranges of the sequences' own keys
    bool shares = false;
    int tile_rows = 0, piece_rows = 0;         // of launch_attn_decode8
    size_t rows = 0, pieces = 0;     // partial rows of a slot; piece rows
    int slots() const { return prefix == 0 && own == 1 ? 0 : prefix + own; }
    size_t lse_bytes() const { return ((slots() * rows + pieces) * 4 + 255) & ~(size_t)255; }
    size_t bytes(int d) const { return lse_bytes() + (slots() * rows + pieces) * d * 4; }
};

// Key ranges per row tile of a launch with `items` tiles over up to `keys`
// keys, in `slots` CTAs: as many as those take, of at least two steps of `step` keys
// each.  `keys` is what the page table could hold, since lengths are on the device: a
// prompt of 37 rows takes 8.4 us (in a graph) with a table of 2 pages of 32 keys and
// 13.9 with one of 1024, for which it is cut into 19 ranges and joined.  More
// tiles than slots are not split: the
// partial rows' way through memory costs more than an even last wave gives
// (2560 rows in 3 chunks over up to 9000 keys: 233 us in one range, 355 us in
// the number that evened the waves).
int choose_splits(int64_t items, int64_t keys, int slots, int step) {
    const int64_t most = std::max<int64_t>(1, keys / (2 * step));
    return (int)std::max<int64_t>(1, std::min({slots / std::max<int64_t>(items, 1), most, (int64_t)kMaxSplits}));
}

constexpr float kLog2e = 1.44269504088896340736f;

// bf16 prompts and prefixes run on the tensor cores.
bool on_tensor_cores(int dtype, int mode) { return rows_of(dtype) == COLIBRI_DTYPE_BF16 && mode != kAttnSuffix; }

// The slots: one tensor-core CTA per SM.  Two of the CUDA-core kernel, which is what an
// SM holds at d 64 (101 KB of shared memory); at d 128 it holds one (183 KB), but two
// waves of shorter ranges take less than one of longer: 64 rows of 16 heads over 1024
// keys 25 us instead of 33, 600 packed rows 71 instead of 82, 200 rows over a prefix of
// 4096 248 instead of 291 (8 rows of group 64 over 4000 keys 61 instead of 40).
int splits_for(const AttnArgs& a, const colibri_kv_pages_t* kv, int64_t keys) {
    const bool tc = on_tensor_cores(kv->dtype, a.mode);
    return tc ? choose_splits(attn_tc_items(a) * kv->n_kv_heads, keys, kSms, 128)
              : choose_splits(attn_simt_items(a) * kv->n_kv_heads, keys, 2 * kSms, 64);
}

// Prompts over codes whose sequences have few rows each (drafts to be verified): tiles of
// 16 rows read the keys once each, at HBM's rate, where the tensor-core kernel walks
// them with one or two tiles per CTA and waits for one step's chain after another
// (12 sequences of 4500 keys: 33, 50, 64, 69, 92 us for 8, 16, 24, 32, 48 rows each, on the
// tensor cores 76 whatever the rows; 48 of 3000 keys and 16 rows: 117 and 157).  How the rows
// are spread is known on the device only, and one sequence may have nearly all of them: up
// to kMostRows, so that its keys are read 64 times at most.
constexpr int kFewRows = 32, kMostRows = 1024;
bool few_rows(const colibri_kv_pages_t* kv, const colibri_seqs_t* s, int group, int64_t keys) {
    const int64_t rows = (int64_t)s->n_rows * group;
    // (and the list of steps is counted in 64 bits, times the shares, even where every
    // sequence claims all rows)
    return rows <= kFewRows * (int64_t)s->n_seqs && rows <= kMostRows &&
           ((double)keys / 32 + 1) * kv->n_kv_heads * ((double)rows / 8 + 1) * s->n_seqs <= 1e15;
}

Plan make_plan(const colibri_kv_pages_t* kv, const colibri_seqs_t* s, int hq, int mode, int prefix_len) {
    const int64_t keys = s->page_table ? (int64_t)s->table_stride * kv->page_size : s->n_rows;
    AttnArgs a{};
    a.n_rows = s->n_rows, a.n_seqs = s->n_seqs, a.hkv = kv->n_kv_heads, a.group = hq / a.hkv, a.mode = mode;
    a.prefix_len = prefix_len;
    Plan p;
    if (s->n_seqs == 0) return p;
    p.rows = (size_t)s->n_rows * hq;
    if (kv->dtype == kCodes && (mode == kAttnSuffix || few_rows(kv, s, a.group, keys))) {
        const int64_t rows = (int64_t)s->n_rows * a.group;         // (one token each: n_rows sequences)
        p.shares = true;
        p.tile_rows = rows <= 8 * (int64_t)s->n_seqs ? 8 : 16;
        p.piece_rows = mode == kAttnSuffix ? std::min(a.group, p.tile_rows) : p.tile_rows;
        p.pieces = attn_decode8_pieces(p.tile_rows, p.piece_rows);
    } else if (mode == kAttnSuffix && attn_decode_takes(dtype_of(kv->dtype), a.group)) {
        p.shares = true;
        p.pieces = attn_decode_pieces(dtype_of(kv->dtype), a.group);
    } else {
        p.own = splits_for(a, kv, std::max<int64_t>(keys - prefix_len, 1));
    }
    if (prefix_len > 0) {
        a.mode = kAttnPrefix;
        p.prefix = splits_for(a, kv, prefix_len);
    }
    return p;
}

cudaError_t launch_attention(int dtype, int d, const AttnArgs& a, cudaStream_t s) {
    if (on_tensor_cores(dtype, a.mode)) return launch_attn_tc(d, a, s);
    return launch_attn_simt(d, a, s);
}

// The bound of the tensor-core kernel's waits, and where copies stop in the
// failure-detection tests (colibri_attention_waits).  The environment gives what they
// start with and is read once: a getenv per call would race with other threads' setenv.
constexpr uint64_t kWaitLimitNs = 2000000000ull;
struct Waits {
    std::atomic<uint64_t> limit_ns{kWaitLimitNs};
    std::atomic<int> stall{0};
    Waits() {
        if (const char* e = std::getenv("COLIBRI_WAIT_LIMIT_NS")) limit_ns = std::strtoull(e, nullptr, 10);
        if (const char* e = std::getenv("COLIBRI_TEST_STALL_TMA")) stall = std::atoi(e);
    }
};
Waits& waits() {
    static Waits w;
    return w;
}

AttnArgs make_args(const colibri_kv_pages_t* kv, const colibri_seqs_t* s, int hq, const void* q,
                   int64_t q_stride, float scale, void* o, int64_t o_stride, float* lse) {
    AttnArgs a{};
    a.q = q, a.k = kv->k, a.v = kv->v, a.o = o, a.lse = lse;
    a.seq_start = s->seq_start, a.kv_len = s->kv_len, a.table = s->page_table;
    a.q_stride = q_stride, a.o_stride = o_stride;
    a.page_stride = kv->page_stride, a.head_stride = kv->head_stride, a.row_stride = kv->row_stride;
    a.mode = s->seq_start ? kAttnPrompt : kAttnSuffix;
    a.n_seqs = s->n_seqs, a.n_rows = s->n_rows;
    a.hq = hq, a.hkv = kv->n_kv_heads, a.group = hq / kv->n_kv_heads;
    a.table_stride = s->table_stride;
    a.num_pages = kv->num_pages, a.page_size = kv->page_size;
    a.page_shift = shift_of(kv->page_size);
    a.scale_log2 = scale * kLog2e;
    a.splits = 1;
    a.wait_limit_ns = waits().limit_ns.load(std::memory_order_relaxed);
    a.stall_tma = waits().stall.load(std::memory_order_relaxed);
    return a;
}

colibri_status_t check_attention(const colibri_kv_pages_t* kv, const colibri_seqs_t* s, int hq,
                                 const void* q, int64_t q_stride, float scale, const void* o,
                                 int64_t o_stride, const float* lse) {
    const int esz = elem_size(rows_of(kv->dtype)), d = kv->head_dim;
    if (!rows_ok(q, q_stride, hq, d, esz) || !rows_ok(o, o_stride, hq, d, esz) || ((uintptr_t)lse & 3))
        return COLIBRI_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !std::isfinite(scale * kLog2e)) return COLIBRI_ERR_INVALID_ARG;
    if (s->n_rows == 0) return COLIBRI_OK;
    const Rows out = row_bytes(o, o_stride, hq, d, esz);
    if (clash(row_bytes(q, q_stride, hq, d, esz), out, s->n_rows)) return COLIBRI_ERR_INVALID_ARG;
    if (!s->page_table && s->n_seqs == 0) return COLIBRI_OK;      // no keys, of pages or rows
    for (const void* p : {(const void*)kv->k, (const void*)kv->v}) {
        const Rows packed = {p, kv->row_stride * esz, ((int64_t)(kv->n_kv_heads - 1) * kv->head_stride + d) * esz};
        if (s->page_table ? overlap(p, kv_extent(kv), o, out.extent(s->n_rows)) : clash(packed, out, s->n_rows))
            return COLIBRI_ERR_INVALID_ARG;
    }
    return COLIBRI_OK;
}

void place_workspace(AttnArgs& a, const Plan& p, int d, void* ws) {
    if (p.slots() + p.pieces == 0) return;
    float* lse = static_cast<float*>(ws);
    float* o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + p.lse_bytes());
    a.piece_lse = lse + p.slots() * p.rows;
    a.piece_o = o + p.slots() * p.rows * d;
    if (p.slots() > 0) a.part_lse = lse, a.part_o = o;
}

// The status of a call's launches.  A launch returns its own errors, so one that an
// earlier call left behind is not asked for, and none is left to later calls.
colibri_status_t launched(cudaError_t e) {
    if (e == cudaSuccess) return COLIBRI_OK;
    cudaGetLastError();
    return COLIBRI_ERR_CUDA;
}

colibri_status_t run_attention(AttnArgs a, const Plan& p, int dtype, int d, int prefix_len,
                               const int32_t* prefix_table, void* ws, cudaStream_t s) {
    place_workspace(a, p, d, ws);
    a.prefix_len = prefix_len;
    cudaError_t e = cudaSuccess;
    if (p.prefix > 0) {
        AttnArgs f = a;
        f.mode = kAttnPrefix;
        f.causal = 0;
        f.table = prefix_table;
        f.splits = p.prefix;
        f.part_slot = 0;
        e = launch_attention(dtype, d, f, s);
    }
    a.splits = p.own;
    a.tile_rows = p.tile_rows, a.piece_rows = p.piece_rows;
    const int tile = p.tile_rows ? p.tile_rows : attn_decode_tile(dtype_of(dtype), a.group);
    a.group_tiles = (a.group + tile - 1) / tile;
    a.seq_items = a.group_tiles * a.hkv;
    a.part_slot = p.prefix;
    a.beside_prefix = p.prefix > 0;
    if (e == cudaSuccess)
        e = !p.shares   ? launch_attention(dtype, d, a, s)
            : a.k_scale ? launch_attn_decode8(d, a, s)
                        : launch_attn_decode(dtype_of(dtype), d, a, s);
    if (e == cudaSuccess && (p.shares || p.slots() > 0))
        e = launch_attn_join(dtype_of(dtype), d, a, p.shares ? p.prefix : p.slots(), p.shares, s);
    return launched(e);
}

// The pages can be named by the tensor-core kernel's tensor map.
bool mappable(const colibri_kv_pages_t* kv) {
    AttnArgs a{};
    a.hkv = kv->n_kv_heads, a.num_pages = kv->num_pages;
    a.page_stride = kv->page_stride, a.head_stride = kv->head_stride;
    int64_t unit;
    int per_page, per_head, count;
    return attn_tc_units(a, &unit, &per_page, &per_head, &count);
}

// The list of all keys of all heads is counted in 64 bits, times the CTAs.
bool countable(const colibri_kv_pages_t* kv, const colibri_seqs_t* s, int n_q_heads) {
    return (double)s->n_seqs * s->table_stride * kv->page_size * n_q_heads <= 1e15;
}

colibri_status_t check_prompt(const colibri_kv_pages_t* kv, const colibri_seqs_t* seqs, int n_q_heads) {
    if (!kv || !seqs) return COLIBRI_ERR_INVALID_ARG;
    colibri_status_t st = check_heads(n_q_heads, kv->n_kv_heads, kv->head_dim, rows_of(kv->dtype));
    if (st == COLIBRI_OK) st = check_seqs(seqs, n_q_heads);
    if (st == COLIBRI_OK) st = check_kv(kv, seqs->page_table != nullptr);
    if (st != COLIBRI_OK) return st;
    if (seqs->page_table && !(countable(kv, seqs, n_q_heads) && mappable(kv))) return COLIBRI_ERR_UNSUPPORTED;
    // packed keys: the call's own rows
    if (!seqs->page_table && seqs->n_seqs > 0 &&
        (seqs->kv_len || kv->num_pages != 1 || (seqs->n_rows > 0 && kv->page_size != seqs->n_rows)))
        return COLIBRI_ERR_INVALID_ARG;
    return COLIBRI_OK;
}

colibri_status_t check_decode(const colibri_kv_pages_t* kv, const colibri_seqs_t* seqs, int n_q_heads,
                              int prefix_len) {
    if (!kv || !seqs || seqs->seq_start || (seqs->n_seqs > 0 && (!seqs->page_table || !seqs->kv_len)))
        return COLIBRI_ERR_INVALID_ARG;
    colibri_status_t st = check_heads(n_q_heads, kv->n_kv_heads, kv->head_dim, rows_of(kv->dtype));
    if (st == COLIBRI_OK) st = check_seqs(seqs, n_q_heads);
    if (st == COLIBRI_OK) st = check_kv(kv, true);
    if (st != COLIBRI_OK) return st;
    if (prefix_len < 0 || prefix_len % kv->page_size) return COLIBRI_ERR_INVALID_ARG;
    if (prefix_len > kMaxKeys || !countable(kv, seqs, n_q_heads) || !mappable(kv))
        return COLIBRI_ERR_UNSUPPORTED;
    return COLIBRI_OK;
}

// o shares no byte with the scales.
bool apart_from_scales(const colibri_kv_pages8_t* c, int hq, const void* o, int64_t o_stride, int rows) {
    if (rows <= 0) return true;
    const int64_t n = row_bytes(o, o_stride, hq, c->head_dim, 2).extent(rows);
    return !overlap(c->k_scale, scale_bytes(c), o, n) && !overlap(c->v_scale, scale_bytes(c), o, n);
}

// The caller's description of pages of rows' elements: kCodes is this file's own.
bool describes_codes(const colibri_kv_pages_t* kv) { return kv && kv->dtype == kCodes; }

colibri_status_t check_prompt8(const colibri_kv_pages8_t* c, const colibri_seqs_t* s, int hq) {
    const colibri_status_t st = check_kv8(c);
    if (st != COLIBRI_OK) return st;
    if (!s || (s->n_seqs > 0 && (!s->page_table || !s->kv_len))) return COLIBRI_ERR_INVALID_ARG;
    const colibri_kv_pages_t kv = view(c);
    return check_prompt(&kv, s, hq);
}

colibri_status_t check_attention8(const colibri_kv_pages8_t* c, const colibri_seqs_t* s, int hq, const void* q,
                                  int64_t q_stride, float scale, const void* o, int64_t o_stride, const float* lse) {
    const colibri_kv_pages_t kv = view(c);
    const colibri_status_t st = check_attention(&kv, s, hq, q, q_stride, scale, o, o_stride, lse);
    if (st != COLIBRI_OK) return st;
    return apart_from_scales(c, hq, o, o_stride, s->n_rows) ? COLIBRI_OK : COLIBRI_ERR_INVALID_ARG;
}

// make_args for a cache of codes.
AttnArgs make_args8(const colibri_kv_pages8_t* c, const colibri_seqs_t* s, int hq, const void* q, int64_t q_stride,
                    float scale, void* o, int64_t o_stride, float* lse) {
    const colibri_kv_pages_t kv = view(c);
    AttnArgs a = make_args(&kv, s, hq, q, q_stride, scale, o, o_stride, lse);
    a.k_scale = c->k_scale, a.v_scale = c->v_scale;
    a.block_shift = shift_of(c->block), a.int8 = c->code == COLIBRI_CODE_INT8;
    return a;
}

}  // namespace

extern "C" {

colibri_status_t colibri_rope_frequencies(int32_t rot_dim, double theta, int32_t scaling, double factor,
                                          int32_t trained, double beta_fast, double beta_slow,
                                          double* freq, float* mscale) {
    if (!freq || !mscale || rot_dim <= 0 || rot_dim % 16 || !(theta > 1.0) || !std::isfinite(theta))
        return COLIBRI_ERR_INVALID_ARG;
    if (scaling < COLIBRI_ROPE_SCALE_NONE || scaling > COLIBRI_ROPE_SCALE_YARN)
        return COLIBRI_ERR_INVALID_ARG;
    if (scaling != COLIBRI_ROPE_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
        return COLIBRI_ERR_INVALID_ARG;
    const bool yarn = scaling == COLIBRI_ROPE_SCALE_YARN;
    if (yarn && (trained <= 0 || !(beta_slow > 0.0) || !(beta_fast > beta_slow)))
        return COLIBRI_ERR_INVALID_ARG;
    const int half = rot_dim / 2;
    if (scaling == COLIBRI_ROPE_SCALE_NTK)
        theta *= std::pow(factor, (double)rot_dim / (double)(rot_dim - 2));
    double lo = 0.0, hi = 0.0;
    if (yarn) {
        // the pair that turns `turns` times in the trained context
        const auto at = [&](double turns) {
            return rot_dim * std::log(trained / (turns * 2.0 * 3.14159265358979323846)) /
                   (2.0 * std::log(theta));
        };
        lo = std::max(std::floor(at(beta_fast)), 0.0);
        hi = std::min(std::ceil(at(beta_slow)), (double)(rot_dim - 1));
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(theta, -2.0 * i / rot_dim);
        if (scaling == COLIBRI_ROPE_SCALE_LINEAR) {
            f /= factor;
        } else if (yarn) {
            const double ramp = std::min(1.0, std::max(0.0, (i - lo) / std::max(hi - lo, 1e-3)));
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        freq[i] = f;
    }
    *mscale = yarn ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
    return COLIBRI_OK;
}

colibri_status_t colibri_append_qkv(const colibri_kv_pages_t* cache, const colibri_seqs_t* seqs,
                                    const colibri_rope_t* rope, int32_t n_q_heads, const void* q,
                                    int64_t q_stride, const void* k, int64_t k_stride,
                                    const void* v, int64_t v_stride, const void* q_norm,
                                    const void* k_norm, float eps, void* q_out,
                                    int64_t q_out_stride, void* stream) {
    return colibri_append_qkv_at(cache, seqs, rope, nullptr, n_q_heads, q, q_stride, k, k_stride, v, v_stride, q_norm,
                                 k_norm, eps, q_out, q_out_stride, stream);
}

colibri_status_t colibri_append_qkv_at(const colibri_kv_pages_t* cache, const colibri_seqs_t* seqs,
                                       const colibri_rope_t* rope, const colibri_positions_t* positions,
                                       int32_t n_q_heads, const void* q, int64_t q_stride, const void* k,
                                       int64_t k_stride, const void* v, int64_t v_stride,
                                       const void* q_norm, const void* k_norm, float eps, void* q_out,
                                       int64_t q_out_stride, void* stream) {
    if (!cache) return COLIBRI_ERR_INVALID_ARG;
    const Projection p = {q, k, v, q_stride, k_stride, v_stride, q_norm, k_norm, eps, q_out, q_out_stride};
    AppendArgs a{};
    const colibri_status_t st = check_append(cache, cache->dtype, seqs, rope, positions, n_q_heads, p, &a);
    if (st != COLIBRI_OK || a.n_rows == 0) return st;
    return launched(launch_append(dtype_of(cache->dtype), cache->head_dim, a, (cudaStream_t)stream));
}

colibri_status_t colibri_append_qkv8(const colibri_kv_pages8_t* cache, const colibri_seqs_t* seqs,
                                     const colibri_rope_t* rope, const colibri_positions_t* positions,
                                     int32_t n_q_heads, const void* q, int64_t q_stride, const void* k,
                                     int64_t k_stride, const void* v, int64_t v_stride,
                                     const void* q_norm, const void* k_norm, float eps, void* q_out,
                                     int64_t q_out_stride, void* stream) {
    colibri_status_t st = check_kv8(cache);
    if (st != COLIBRI_OK) return st;
    const colibri_kv_pages_t kv = view(cache);
    const Projection p = {q, k, v, q_stride, k_stride, v_stride, q_norm, k_norm, eps, q_out, q_out_stride};
    AppendArgs a{};
    st = check_append(&kv, COLIBRI_DTYPE_BF16, seqs, rope, positions, n_q_heads, p, &a);
    if (st != COLIBRI_OK) return st;
    const int d = kv.head_dim, hkv = kv.n_kv_heads;
    for (const float* scale : {cache->k_scale, cache->v_scale})
        for (const Rows& r : {row_bytes(q, q_stride, n_q_heads, d, 2), row_bytes(k, k_stride, hkv, d, 2),
                              row_bytes(v, v_stride, hkv, d, 2), row_bytes(q_out, q_out_stride, n_q_heads, d, 2)})
            if (seqs->n_rows > 0 && overlap(scale, scale_bytes(cache), r.p, r.extent(seqs->n_rows)))
                return COLIBRI_ERR_INVALID_ARG;
    // (what is written in one part of the cache is not another part)
    if (overlap(cache->k_scale, scale_bytes(cache), cache->v_scale, scale_bytes(cache))) return COLIBRI_ERR_INVALID_ARG;
    for (const float* scale : {cache->k_scale, cache->v_scale})
        for (const void* codes : {cache->k, cache->v})
            if (overlap(scale, scale_bytes(cache), codes, kv_extent(&kv))) return COLIBRI_ERR_INVALID_ARG;
    if (a.n_rows == 0) return COLIBRI_OK;
    a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
    a.block_shift = shift_of(cache->block);
    return launched(launch_append8(cache->code == COLIBRI_CODE_INT8, d, a, (cudaStream_t)stream));
}

colibri_status_t colibri_values8(const colibri_kv_pages8_t* cache, const int32_t* pages, int32_t n_pages,
                                 void* k_out, void* v_out, void* stream) {
    const colibri_status_t st = check_kv8(cache);
    if (st != COLIBRI_OK) return st;
    if (n_pages < 0 || ((uintptr_t)pages & 3) || (!pages && n_pages > cache->num_pages)) return COLIBRI_ERR_INVALID_ARG;
    if (n_pages == 0) return COLIBRI_OK;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return COLIBRI_ERR_INVALID_ARG;
    if ((int64_t)n_pages * cache->n_kv_heads > INT32_MAX) return COLIBRI_ERR_UNSUPPORTED;
    const colibri_kv_pages_t kv = view(cache);
    const int64_t bytes = (int64_t)n_pages * kv.n_kv_heads * kv.page_size * kv.head_dim * 2;
    if (overlap(k_out, bytes, v_out, bytes)) return COLIBRI_ERR_INVALID_ARG;
    for (const void* to : {k_out, v_out}) {
        for (const void* p : {(const void*)kv.k, (const void*)kv.v})
            if (overlap(p, kv_extent(&kv), to, bytes)) return COLIBRI_ERR_INVALID_ARG;
        for (const float* p : {cache->k_scale, cache->v_scale})
            if (overlap(p, scale_bytes(cache), to, bytes)) return COLIBRI_ERR_INVALID_ARG;
    }
    ValuesArgs a = values_args(cache);
    a.pages = pages, a.n_pages = n_pages;
    a.k_out = k_out, a.v_out = v_out;
    return launched(launch_values8(cache->code == COLIBRI_CODE_INT8, kv.head_dim, a, (cudaStream_t)stream));
}

colibri_status_t colibri_qk_norm_rope(const colibri_seqs_t* seqs, const colibri_rope_t* rope,
                                      int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                      int32_t dtype, const void* q, int64_t q_stride,
                                      const void* k, int64_t k_stride, const void* q_norm,
                                      const void* k_norm, float eps, void* q_out,
                                      int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                      void* stream) {
    return colibri_qk_norm_rope_at(seqs, rope, nullptr, n_q_heads, n_kv_heads, head_dim, dtype, q, q_stride, k, k_stride,
                                   q_norm, k_norm, eps, q_out, q_out_stride, k_out, k_out_stride, stream);
}

colibri_status_t colibri_qk_norm_rope_at(const colibri_seqs_t* seqs, const colibri_rope_t* rope,
                                         const colibri_positions_t* positions, int32_t n_q_heads,
                                         int32_t n_kv_heads, int32_t head_dim, int32_t dtype,
                                         const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                         const void* q_norm, const void* k_norm, float eps, void* q_out,
                                         int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                         void* stream) {
    if (!seqs) return COLIBRI_ERR_INVALID_ARG;
    colibri_status_t st = check_heads(n_q_heads, n_kv_heads, head_dim, dtype);
    if (st == COLIBRI_OK) st = check_seqs(seqs, n_q_heads);
    if (st == COLIBRI_OK) st = check_rope(rope, head_dim);
    if (st == COLIBRI_OK) st = check_positions(positions, rope, seqs->n_rows);
    if (st != COLIBRI_OK) return st;
    const int d = head_dim, esz = elem_size(dtype);
    if (!rows_ok(q, q_stride, n_q_heads, d, esz) || !rows_ok(k, k_stride, n_kv_heads, d, esz) ||
        !rows_ok(q_out, q_out_stride, n_q_heads, d, esz) ||
        !rows_ok(k_out, k_out_stride, n_kv_heads, d, esz) || !aligned16(q_norm) ||
        !aligned16(k_norm) || !(eps >= 0.f))
        return COLIBRI_ERR_INVALID_ARG;
    if ((q_out == q && q_out_stride != q_stride) || (k_out == k && k_out_stride != k_stride))
        return COLIBRI_ERR_INVALID_ARG;
    const Rows qi = row_bytes(q, q_stride, n_q_heads, d, esz), ki = row_bytes(k, k_stride, n_kv_heads, d, esz);
    const Rows qo = row_bytes(q_out, q_out_stride, n_q_heads, d, esz), ko = row_bytes(k_out, k_out_stride, n_kv_heads, d, esz);
    if ((q_out != q && clash(qi, qo, seqs->n_rows)) || (k_out != k && clash(ki, ko, seqs->n_rows)) ||
        clash(qi, ko, seqs->n_rows) || clash(ki, qo, seqs->n_rows) || clash(qo, ko, seqs->n_rows))
        return COLIBRI_ERR_INVALID_ARG;
    if (seqs->n_rows == 0 || seqs->n_seqs == 0) return COLIBRI_OK;
    AppendArgs a{};
    a.q = q, a.k = k;
    a.q_stride = q_stride, a.k_stride = k_stride;
    a.q_norm = q_norm, a.k_norm = k_norm, a.eps = eps;
    set_rope(a, rope, positions);
    a.seq_start = seqs->seq_start, a.kv_len = seqs->kv_len;
    a.n_seqs = seqs->n_seqs, a.n_rows = seqs->n_rows;
    a.hq = n_q_heads, a.hkv = n_kv_heads;
    a.q_out = q_out, a.q_out_stride = q_out_stride;
    a.k_out = k_out, a.row_stride = k_out_stride, a.head_stride = d;
    return launched(launch_append(dtype_of(dtype), d, a, (cudaStream_t)stream));
}

colibri_status_t colibri_attention_waits(uint64_t limit_ns, int32_t stall) {
    if (stall < 0) return COLIBRI_ERR_INVALID_ARG;
    waits().limit_ns = limit_ns ? limit_ns : kWaitLimitNs;
    waits().stall = stall;
    return COLIBRI_OK;
}

colibri_status_t colibri_attention_check(void* stream) {
    int status = DEV_OK;
    const colibri_status_t st = launched(attn_tc_status(&status, (cudaStream_t)stream));
    return st == COLIBRI_OK && status != DEV_OK ? COLIBRI_ERR_TIMEOUT : st;
}

colibri_status_t colibri_attention_prompt_workspace(const colibri_kv_pages_t* kv,
                                                    const colibri_seqs_t* seqs, int32_t n_q_heads,
                                                    size_t* bytes) {
    if (!bytes || describes_codes(kv)) return COLIBRI_ERR_INVALID_ARG;
    const colibri_status_t st = check_prompt(kv, seqs, n_q_heads);
    if (st != COLIBRI_OK) return st;
    const int mode = seqs->seq_start ? kAttnPrompt : kAttnSuffix;
    *bytes = make_plan(kv, seqs, n_q_heads, mode, 0).bytes(kv->head_dim);
    return COLIBRI_OK;
}

colibri_status_t colibri_attention_prompt(const colibri_kv_pages_t* kv, const colibri_seqs_t* seqs,
                                          int32_t n_q_heads, const void* q, int64_t q_stride,
                                          float scale, int32_t causal, void* o, int64_t o_stride,
                                          float* lse, void* workspace, size_t workspace_bytes,
                                          void* stream) {
    if (describes_codes(kv)) return COLIBRI_ERR_INVALID_ARG;
    colibri_status_t st = check_prompt(kv, seqs, n_q_heads);
    if (st == COLIBRI_OK) st = check_attention(kv, seqs, n_q_heads, q, q_stride, scale, o, o_stride, lse);
    if (st != COLIBRI_OK) return st;
    const int mode = seqs->seq_start ? kAttnPrompt : kAttnSuffix;
    const Plan p = make_plan(kv, seqs, n_q_heads, mode, 0);
    const size_t need = p.bytes(kv->head_dim);
    if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255)))
        return COLIBRI_ERR_INVALID_ARG;
    if (seqs->n_rows == 0 || seqs->n_seqs == 0) return COLIBRI_OK;
    AttnArgs a = make_args(kv, seqs, n_q_heads, q, q_stride, scale, o, o_stride, lse);
    a.causal = causal != 0;
    return run_attention(a, p, kv->dtype, kv->head_dim, 0, nullptr, workspace, (cudaStream_t)stream);
}

colibri_status_t colibri_attention_decode_workspace(const colibri_kv_pages_t* cache,
                                                    const colibri_seqs_t* seqs, int32_t n_q_heads,
                                                    int32_t prefix_len, size_t* bytes) {
    if (!bytes || describes_codes(cache)) return COLIBRI_ERR_INVALID_ARG;
    const colibri_status_t st = check_decode(cache, seqs, n_q_heads, prefix_len);
    if (st != COLIBRI_OK) return st;
    *bytes = make_plan(cache, seqs, n_q_heads, kAttnSuffix, prefix_len)
                 .bytes(cache->head_dim);
    return COLIBRI_OK;
}

colibri_status_t colibri_attention_decode(const colibri_kv_pages_t* cache, const colibri_seqs_t* seqs,
                                          int32_t n_q_heads, const void* q, int64_t q_stride,
                                          float scale, int32_t prefix_len,
                                          const int32_t* prefix_table, void* o, int64_t o_stride,
                                          float* lse, void* workspace, size_t workspace_bytes,
                                          void* stream) {
    if (describes_codes(cache)) return COLIBRI_ERR_INVALID_ARG;
    colibri_status_t st = check_decode(cache, seqs, n_q_heads, prefix_len);
    if (st == COLIBRI_OK)
        st = check_attention(cache, seqs, n_q_heads, q, q_stride, scale, o, o_stride, lse);
    if (st != COLIBRI_OK) return st;
    if ((prefix_len > 0) != (prefix_table != nullptr) || ((uintptr_t)prefix_table & 3))
        return COLIBRI_ERR_INVALID_ARG;
    const Plan p = make_plan(cache, seqs, n_q_heads, kAttnSuffix, prefix_len);
    const size_t need = p.bytes(cache->head_dim);
    if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255)))
        return COLIBRI_ERR_INVALID_ARG;
    if (seqs->n_rows == 0) return COLIBRI_OK;
    AttnArgs a = make_args(cache, seqs, n_q_heads, q, q_stride, scale, o, o_stride, lse);
    return run_attention(a, p, cache->dtype, cache->head_dim, prefix_len, prefix_table, workspace,
                         (cudaStream_t)stream);
}

colibri_status_t colibri_attention_prompt8_workspace(const colibri_kv_pages8_t* cache, const colibri_seqs_t* seqs,
                                                     int32_t n_q_heads, size_t* bytes) {
    if (!bytes) return COLIBRI_ERR_INVALID_ARG;
    const colibri_status_t st = check_prompt8(cache, seqs, n_q_heads);
    if (st != COLIBRI_OK) return st;
    const colibri_kv_pages_t kv = view(cache);
    *bytes = make_plan(&kv, seqs, n_q_heads, seqs->seq_start ? kAttnPrompt : kAttnSuffix, 0).bytes(kv.head_dim);
    return COLIBRI_OK;
}

colibri_status_t colibri_attention_prompt8(const colibri_kv_pages8_t* cache, const colibri_seqs_t* seqs,
                                           int32_t n_q_heads, const void* q, int64_t q_stride, float scale,
                                           int32_t causal, void* o, int64_t o_stride, float* lse,
                                           void* workspace, size_t workspace_bytes, void* stream) {
    colibri_status_t st = check_prompt8(cache, seqs, n_q_heads);
    if (st == COLIBRI_OK) st = check_attention8(cache, seqs, n_q_heads, q, q_stride, scale, o, o_stride, lse);
    if (st != COLIBRI_OK) return st;
    const colibri_kv_pages_t kv = view(cache);
    const Plan p = make_plan(&kv, seqs, n_q_heads, seqs->seq_start ? kAttnPrompt : kAttnSuffix, 0);
    const size_t need = p.bytes(kv.head_dim);
    if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255)))
        return COLIBRI_ERR_INVALID_ARG;
    if (seqs->n_rows == 0 || seqs->n_seqs == 0) return COLIBRI_OK;
    AttnArgs a = make_args8(cache, seqs, n_q_heads, q, q_stride, scale, o, o_stride, lse);
    a.causal = causal != 0;
    return run_attention(a, p, kCodes, kv.head_dim, 0, nullptr, workspace, (cudaStream_t)stream);
}

colibri_status_t colibri_attention_decode8_workspace(const colibri_kv_pages8_t* cache, const colibri_seqs_t* seqs,
                                                     int32_t n_q_heads, int32_t prefix_len, size_t* bytes) {
    if (!bytes) return COLIBRI_ERR_INVALID_ARG;
    colibri_status_t st = check_kv8(cache);
    if (st != COLIBRI_OK) return st;
    const colibri_kv_pages_t kv = view(cache);
    st = check_decode(&kv, seqs, n_q_heads, prefix_len);
    if (st != COLIBRI_OK) return st;
    *bytes = make_plan(&kv, seqs, n_q_heads, kAttnSuffix, prefix_len).bytes(kv.head_dim);
    return COLIBRI_OK;
}

colibri_status_t colibri_attention_decode8(const colibri_kv_pages8_t* cache, const colibri_seqs_t* seqs,
                                           int32_t n_q_heads, const void* q, int64_t q_stride, float scale,
                                           int32_t prefix_len, const int32_t* prefix_table, void* o,
                                           int64_t o_stride, float* lse, void* workspace,
                                           size_t workspace_bytes, void* stream) {
    size_t need;
    colibri_status_t st = colibri_attention_decode8_workspace(cache, seqs, n_q_heads, prefix_len, &need);
    if (st == COLIBRI_OK) st = check_attention8(cache, seqs, n_q_heads, q, q_stride, scale, o, o_stride, lse);
    if (st != COLIBRI_OK) return st;
    if ((prefix_len > 0) != (prefix_table != nullptr) || ((uintptr_t)prefix_table & 3))
        return COLIBRI_ERR_INVALID_ARG;
    if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255)))
        return COLIBRI_ERR_INVALID_ARG;
    if (seqs->n_rows == 0) return COLIBRI_OK;
    const colibri_kv_pages_t kv = view(cache);
    const Plan p = make_plan(&kv, seqs, n_q_heads, kAttnSuffix, prefix_len);
    const AttnArgs a = make_args8(cache, seqs, n_q_heads, q, q_stride, scale, o, o_stride, lse);
    return run_attention(a, p, kCodes, kv.head_dim, prefix_len, prefix_table, workspace, (cudaStream_t)stream);
}

}  // extern "C"
