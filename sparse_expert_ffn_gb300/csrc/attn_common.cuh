// Device helpers of the attention kernels: which rows and keys a work item
// covers.  Every value that comes from a device array is cut to the bounds the
// launch knows, so whatever the arrays hold, every access stays in bounds.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace colibri {

// kEarly: read before the kernel has waited for the launch before it (the
// sequences' own keys beside a prefix, the join's lengths).  What is read then was
// left by the launch before that one, which is complete, its writes in L2: its
// successor waited for it before it let this kernel start.  But only a grid that has
// itself waited is promised to see other grids' writes in L1, so early reads come
// from L2 (keys and values by cp.async.cg in any case).  Kernels that wait first
// read through L1 (everything from L2: 53 instead of 48 us on 65421 keys).
template <bool kEarly, typename T>
__device__ __forceinline__ T ld_early(const T* p) {
    return kEarly ? __ldcg(p) : __ldg(p);
}

// One sequence of a launch: rows row0 .. row0 + n - 1, keys kv0 .. kv - 1.
struct AttnSeq {
    int row0, n, kv0, kv, raw;
};

template <bool kEarly = false>
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
    AttnSeq s;
    if (a.mode == kAttnPrefix) {
        s.row0 = 0, s.n = a.n_seqs, s.kv0 = 0, s.kv = s.raw = a.prefix_len;
        return s;
    }
    if (a.mode == kAttnSuffix) {
        s.row0 = b, s.n = 1, s.kv0 = a.prefix_len;
    } else {
        s.row0 = min(max(__ldg(a.seq_start + b), 0), a.n_rows);
        s.n = min(max(__ldg(a.seq_start + b + 1), s.row0), a.n_rows) - s.row0;
        s.kv0 = 0;
    }
    s.raw = !a.kv_len ? s.n : max(ld_early<kEarly>(a.kv_len + b), 0);
    const int64_t cap = a.table ? (int64_t)a.table_stride << a.page_shift : (int64_t)s.n;
    s.kv = (int)min(min((int64_t)s.raw, cap), (int64_t)kMaxKeys);
    return s;
}

// Keys that row i of the sequence sees: kv0 .. attn_limit - 1.
__device__ __forceinline__ int attn_limit(const AttnArgs& a, const AttnSeq& s, int i) {
    if (a.mode == kAttnPrefix) return min(max(__ldg(a.kv_len + i), 0), s.kv);
    if (!a.causal) return s.kv;
    return min(max(s.raw - (s.n - 1 - i), 0), s.kv);
}

// Largest limit of rows i0 .. i1 - 1 (i0 < i1); called by a whole warp.  Of a prefix
// that is where a tile's keys end, however long the prefix is: values that no row of
// the tile sees are not read (or cleared), whatever they hold.
__device__ __forceinline__ int attn_limit_max(const AttnArgs& a, const AttnSeq& s, int i0, int i1) {
    if (a.mode != kAttnPrefix) return attn_limit(a, s, i1 - 1);
    int most = 0;
    for (int i = i0 + (threadIdx.x & 31); i < i1; i += 32) most = max(most, attn_limit(a, s, i));
    return __reduce_max_sync(0xffffffffu, most);
}

// Page id of keys at page index `p` of sequence b, -1 where there is none.
template <bool kEarly = false>
__device__ __forceinline__ int attn_page(const AttnArgs& a, int b, int p) {
    const int64_t at = a.mode == kAttnPrefix ? (int64_t)p : (int64_t)b * a.table_stride + p;
    const int id = ld_early<kEarly>(a.table + at);
    return (unsigned)id < (unsigned)a.num_pages ? id : -1;
}

// Item number `item` of a prompt launch with tiles of `per` of a sequence's
// n * mul rows, the tiles that see the most keys first whatever sequence they are
// of, so that the last ones to start are short (in the order of the sequences,
// packed prompts of head_dim 64 took 56 us, so 49 us).  Tile r from the end of a
// sequence has the key  top - r * per  (causal; else its kv length), in rows; the
// item is found by bisection of the number of tiles whose key is at least c.
// Called by a whole warp, up to 32 * kKept sequences.
constexpr int kKept = 4;
__device__ __forceinline__ bool longest_first(const AttnArgs& a, int item, int mul, int per, int* b, int* tile) {
    const int lane = threadIdx.x & 31;
    int tiles[kKept], top[kKept], most = 0, sum = 0;
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int q = lane + 32 * k;
        tiles[k] = top[k] = 0;
        if (q < a.n_seqs) {
            const AttnSeq s = attn_seq(a, q);
            tiles[k] = (int)(((uint32_t)s.n * (uint32_t)mul + (uint32_t)per - 1u) / (uint32_t)per);
            // (an order only: lengths past 2^23 count as that)
            const int past = min(max((a.causal ? s.raw - s.n : s.kv), 0), 1 << 23) * mul;
            top[k] = a.causal ? past + tiles[k] * per : past;
        }
        if (tiles[k] > 0) most = max(most, top[k]);
        sum += tiles[k];
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (item >= __reduce_add_sync(0xffffffffu, sum)) return false;
    // (keys below 0 count as 0: the threshold 0 takes every tile)
    const auto mine = [&](int k, int c) {
        if (tiles[k] == 0) return 0;
        if (c == 0) return tiles[k];
        if (top[k] < c) return 0;
        return a.causal ? min(tiles[k], (top[k] - c) / per + 1) : tiles[k];
    };
    const auto count = [&](int c) {
        int n = 0;
#pragma unroll
        for (int k = 0; k < kKept; ++k) n += mine(k, c);
        return __reduce_add_sync(0xffffffffu, n);
    };
    int lo = 0, hi = most + 1;                                  // count(lo) > item >= count(hi)
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (count(mid) > item) lo = mid;
        else hi = mid;
    }
    // tiles of key lo exactly, in the order of the sequences
    int left = item - count(hi);
#pragma unroll
    for (int k = 0; k < kKept; ++k) {
        const int from = mine(k, hi), here = mine(k, lo) - from;
        int upto = here;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned holds = __ballot_sync(0xffffffffu, left < upto);
        if (holds) {
            const int src = __ffs(holds) - 1;
            *b = src + 32 * k;
            *tile = __shfl_sync(0xffffffffu, tiles[k] - 1 - from - (left - (upto - here)), src);
            return true;
        }
        left -= __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;                                               // (not reached)
}

// Work item `item` of the launch as (sequence, tile), tiles of `per` rows of a
// sequence's n * mul; called by a whole warp.  The last tiles of a sequence,
// which see the most keys, come first, or with `sorted` those of any sequence.
// False: no such item.
__device__ __forceinline__ bool attn_item(const AttnArgs& a, int item, int mul, int per, bool sorted, int* b,
                                          int* tile) {
    const int lane = threadIdx.x & 31;
    const int count = a.mode == kAttnPrefix ? 1 : a.n_seqs;
    if (a.mode != kAttnPrompt) {
        const int tiles = ((a.mode == kAttnPrefix ? a.n_seqs : 1) * mul + per - 1) / per;
        *b = item / tiles;
        *tile = item % tiles;
        return *b < count;
    }
    // (tiles of up to 128 sequences, whatever seq_start holds, add up in 32 bits)
    if (sorted && count > 1 && count <= 32 * kKept && (int64_t)a.n_rows * mul / per < 1 << 23)
        return longest_first(a, item, mul, per, b, tile);
    int64_t done = 0;
    for (int base = 0; base < count; base += 32) {
        int mine = 0;
        if (base + lane < count) {
            const int s0 = min(max(__ldg(a.seq_start + base + lane), 0), a.n_rows);
            const int s1 = min(max(__ldg(a.seq_start + base + lane + 1), s0), a.n_rows);
            mine = (int)(((uint32_t)(s1 - s0) * (uint32_t)mul + (uint32_t)per - 1u) / (uint32_t)per);
            if (a.kv_len) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.kv_len + base + lane));   // for attn_seq
        }
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned holds = __ballot_sync(0xffffffffu, item - done < upto);
        if (holds) {
            const int src = __ffs(holds) - 1;
            *b = base + src;
            const int into = (int)(item - done) - __shfl_sync(0xffffffffu, upto - mine, src);
            *tile = __shfl_sync(0xffffffffu, mine, src) - 1 - into;
            return true;
        }
        done += __shfl_sync(0xffffffffu, upto, 31);
    }
    return false;
}

// Keys of split `sp` of the tile range kv0 .. end: whole tiles of `kt` keys,
// the same number for every split but the last ones.
__device__ __forceinline__ void attn_split(const AttnArgs& a, int sp, int kt, int kv0, int end,
                                           int* lo, int* hi) {
    const int tiles = end > kv0 ? (end - kv0 + kt - 1) / kt : 0;
    const int per = (tiles + a.splits - 1) / a.splits;
    *lo = min(end, kv0 + min(tiles, sp * per) * kt);
    *hi = min(end, kv0 + min(tiles, (sp + 1) * per) * kt);
}

// Equal shares of the key list (attn_decode.cu).  The list is made of steps of
// 4 KB of keys of one (sequence, key head, row tile), one after another; a share
// goes to one warp.
template <typename T>
__host__ __device__ constexpr int row_tile(int group) {
    return sizeof(T) == 4 ? 4 : group <= 16 ? 16 : 32;
}
template <typename T>
__host__ __device__ constexpr int row_tiles(int group) {
    return (group + row_tile<T>(group) - 1) / row_tile<T>(group);
}
// rows of a piece in the workspace
template <typename T>
__host__ __device__ constexpr int piece_rows(int group) {
    return group < row_tile<T>(group) ? group : row_tile<T>(group);
}
template <typename T, int D> constexpr int kStepKeys = 4096 / (D * (int)sizeof(T));
constexpr int kShareWarps = 4;                    // per CTA
constexpr int kShares = 2 * 152 * kShareWarps;    // 2 CTAs per SM
constexpr int kMinSteps = 4;                      // steps of a share at least

// Steps of sequence b per (head, row tile).
template <typename T, int D, bool kEarly>
__device__ __forceinline__ int seq_steps(const AttnArgs& a, int b) {
    const AttnSeq s = attn_seq<kEarly>(a, b);
    return s.kv > s.kv0 ? (s.kv - s.kv0 + kStepKeys<T, D> - 1) / kStepKeys<T, D> : 0;
}

// The whole list: its length, and the steps before sequence `upto`.  Called by
// a whole warp.
template <typename T, int D, bool kEarly>
__device__ __forceinline__ void count_steps(const AttnArgs& a, int per_seq, int upto, int64_t* total,
                                            int64_t* before) {
    int64_t all = 0, part = 0;
    for (int b = threadIdx.x & 31; b < a.n_seqs; b += 32) {
        const int64_t u = (int64_t)seq_steps<T, D, kEarly>(a, b) * per_seq;
        all += u;
        if (b < upto) part += u;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        all += __shfl_xor_sync(0xffffffffu, all, o);
        part += __shfl_xor_sync(0xffffffffu, part, o);
    }
    *total = all;
    *before = part;
}

// Shares of the list, share c's first step, and the share that step u falls into.
__device__ __forceinline__ int share_count(int64_t total) {
    const int64_t most = (total + kMinSteps - 1) / kMinSteps;
    return most < kShares ? (int)most : kShares;
}
// (in 32 bits where the products fit them: a 64-bit division is some 100 instructions)
constexpr int64_t kSmallList = 1 << 21;
static_assert(kSmallList * kShares < ((int64_t)1 << 32), "fits 32 bits");
__device__ __forceinline__ int64_t share_begin(int64_t total, int shares, int c) {
    return total < kSmallList ? (uint32_t)total * (uint32_t)c / (uint32_t)shares : total * c / shares;
}
__device__ __forceinline__ int share_of(int64_t total, int shares, int64_t u) {
    return total < kSmallList ? (int)(((uint32_t)(u + 1) * (uint32_t)shares - 1u) / (uint32_t)total)
                              : (int)(((u + 1) * shares - 1) / total);
}

constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two f32 operations per instruction.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// 16 bytes into shared memory, asynchronously; zeros where there is nothing.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
    const int n = there ? 16 : 0;
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

}  // namespace colibri
