// Equal shares of the list of all keys, one per warp: the frame of the kernels for
// single rows (attn_decode.cu).  A kernel brings `Rows`: the rows of
// a group, what a step of keys adds to them, and how they are written.
#pragma once

#include "attn_common.cuh"
#include "kernels.h"

namespace colibri {
namespace {

constexpr int kDecThreads = 32 * kShareWarps;
constexpr int kStageBytes = 8192;                                 // K then V of one step

__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16x2(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// A position in a warp's share: the piece it is in, step by step.
template <typename T, int D, bool kEarly>
struct Walk {
    int b, units, tiles;       // sequence, its steps per (head, row tile), its row tiles per head
    int64_t end;               // its steps
    int64_t in_seq;            // steps of sequence b before the piece
    int item;                  // (head, row tile) of the sequence
    int lo, hi;                // keys of the piece
    int step, count;           // steps of the piece: done, all
    bool whole;                // the piece is all of the sequence's steps

    // The piece at in_seq, of at most `left` steps.  False: nothing there.
    __device__ __forceinline__ bool piece(const AttnArgs& a, int64_t left) {
        if (in_seq == end) {
            in_seq = 0, units = 0;
            while (++b < a.n_seqs && (units = seq_steps<T, D, kEarly>(a, b)) == 0) {}
            if (units == 0) return false;                          // (not reached: left > 0)
            tiles = seq_tiles<T, kEarly>(a, b);
            end = units * seq_items<T, kEarly>(a, b);
        }
        const AttnSeq s = attn_seq<kEarly>(a, b);
        item = (int)(in_seq / units);
        const int first = (int)(in_seq - (int64_t)item * units);
        count = (int)min((int64_t)(units - first), left);
        whole = count == units;
        lo = s.kv0 + first * kStepKeys<T, D>;
        hi = min(s.kv, lo + count * kStepKeys<T, D>);
        step = 0;
        in_seq += count;
        return true;
    }
};

// Chunk c of a 128-byte row of codes lies at c ^ code_turn(row), so that chunk c of 8
// rows and four neighbouring chunks of two rows each cover all banks.
__host__ __device__ constexpr int code_turn(int row) { return (row & 1) << 2 | (row >> 1 & 3); }

// One warp's copies.  The page ids of up to 32 page parts ahead lie one per lane.
template <typename T, int D, bool kEarly>
struct Stream {
    static constexpr int kRowBytes = D * (int)sizeof(T);
    static constexpr int kChunks = kRowBytes / 16;                 // 16-byte chunks of a row
    static constexpr int kRowsPer = 32 / kChunks;                  // rows that a pass of the warp covers
    static constexpr int kPasses = kStepKeys<T, D> / kRowsPer;
    int b, lo, hi;             // sequence, keys of the piece
    int parts;                 // pages that a step touches
    int window;                // first step whose page parts the lanes hold
    int id;
    int head;
    // codes: lane 4 kind + s has the scale of keys 16 s .. 16 s + 15 of a step, of keys
    // (kind 0) or values, of the step just asked for, the one before and the one before that
    float asked, waiting, scale;
    const T* k;                // this lane's chunk of row 0 of the head in page 0 (packed: key 0)
    const T* v;
    uint32_t dst;              // this lane's place in a stage, pass 0

    __device__ __forceinline__ void begin(const AttnArgs& a, int seq, int h, int first, int end) {
        const int lane = threadIdx.x & 31, chunk = lane % kChunks, row = lane / kChunks;
        b = seq, lo = first, hi = end, head = h;
        int64_t at = (int64_t)h * a.head_stride + chunk * (16 / (int)sizeof(T));
        if (!a.table) at += (int64_t)b * a.row_stride;             // packed rows: the row's own key
        k = static_cast<const T*>(a.k) + at;
        v = static_cast<const T*>(a.v) + at;
        dst = row * kRowBytes + (kRowBytes == 64 ? (chunk ^ ((row >> 1) & 3)) << 4
                                                 : (chunk ^ (sizeof(T) == 1 ? code_turn(row) : row)) << 4);
        parts = a.page_size < kStepKeys<T, D> ? kStepKeys<T, D> / a.page_size : 1;
        if (a.table) fill(a, 0);
    }
    __device__ __forceinline__ int first_key(int step) const { return lo + step * kStepKeys<T, D>; }
    __device__ __forceinline__ void fill(const AttnArgs& a, int step) {
        const int lane = threadIdx.x & 31;
        window = step;
        const int key = first_key(step + lane / parts) + (lane % parts) * (kStepKeys<T, D> / parts);
        id = key < hi ? attn_page<kEarly>(a, b, key >> a.page_shift) : -1;
    }
    // (a register's copy waits for the load that fills it: by then, a step later, it is there)
    __device__ __forceinline__ void shift_scales() { scale = waiting, waiting = asked; }
    __device__ __forceinline__ void ask_scale(const AttnArgs& a, int step, int key0) {
        const int lane = threadIdx.x & 31, sub = lane & 3, key = key0 + 16 * sub;
        const int part = parts > 1 ? (16 * sub & (kStepKeys<T, D> - 1)) / (kStepKeys<T, D> / parts) : 0;
        const int page = __shfl_sync(0xffffffffu, id, (step - window) * parts + part);
        const bool there = lane < 8 && 16 * sub < kStepKeys<T, D> && key < hi && page >= 0;
        const int64_t at = (((int64_t)page * a.hkv + head) << (a.page_shift - a.block_shift)) +
                           ((key & (a.page_size - 1)) >> a.block_shift);
        asked = there ? ld_early<kEarly>((lane & 4 ? a.v_scale : a.k_scale) + at) : 0.f;
    }
    __device__ __forceinline__ void copy(const AttnArgs& a, int step, uint32_t stage) {
        const int lane = threadIdx.x & 31, key0 = first_key(step), row0 = lane / kChunks;
        if (a.table && step >= window + 32 / parts) fill(a, step);
        if constexpr (sizeof(T) == 1) ask_scale(a, step, key0);
        // rows of one pass lie kRowsPer apart: their swizzle differs by that in
        // the row's low three bits (64-byte rows: not at all)
        const auto place = [&](int i) {
            const int turn = kRowBytes == 64 ? 0 : sizeof(T) == 1 ? code_turn(i * kRowsPer) : (i * kRowsPer) & 7;
            return stage + ((dst + i * kRowsPer * kRowBytes) ^ (turn << 4));
        };
        if (a.table && parts > 1) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int row = i * kRowsPer + row0, key = key0 + row;
                const int page = __shfl_sync(0xffffffffu, id, (step - window) * parts + row / (kStepKeys<T, D> / parts));
                const bool there = key < hi && page >= 0;
                const int64_t at = there ? (int64_t)page * a.page_stride +
                                               (int64_t)(key & (a.page_size - 1)) * a.row_stride : 0;
                cp16(place(i), k + at, there);
                cp16(place(i) + kStageBytes / 2, v + at, there);
            }
            return;
        }
        // the whole step lies in one page (or in packed rows)
        int64_t at = (int64_t)row0 * a.row_stride;
        bool page_there = true;
        if (a.table) {
            const int page = __shfl_sync(0xffffffffu, id, step - window);
            page_there = page >= 0;
            at += (int64_t)max(page, 0) * a.page_stride + (int64_t)(key0 & (a.page_size - 1)) * a.row_stride;
        }
        const int64_t pass = (int64_t)kRowsPer * a.row_stride;
        if (page_there && key0 + kStepKeys<T, D> <= hi) {
            const T *kp = k + at, *vp = v + at;
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                cp16(place(i), kp, true);
                cp16(place(i) + kStageBytes / 2, vp, true);
                kp += pass, vp += pass;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const bool there = page_there && key0 + i * kRowsPer + row0 < hi;
                const int64_t off = there ? at + i * pass : 0;
                cp16(place(i), k + off, there);
                cp16(place(i) + kStageBytes / 2, v + off, there);
            }
        }
    }
};

template <typename Rows, bool kEarly>
__device__ __forceinline__ void decode_share(const AttnArgs& a, uint8_t* smem) {
    using T = typename Rows::T;
    constexpr int D = Rows::kD, KS = Rows::KS, kStages = Rows::kStages, kRingBytes = kStages * kStageBytes;
    const int lane = threadIdx.x & 31, share = blockIdx.x * kShareWarps + (threadIdx.x >> 5);
    // this warp's share of the list, and the sequence that its first step lies in
    int64_t total, left, before = 0, u0;
    count_steps<T, D, kEarly>(a, 0, &total, &left);
    if (total == 0) return;
    const int shares = share_count(total, most_shares<T>(tile_rows<T>(a)));
    if (share >= shares) return;
    u0 = share_begin(total, shares, share);
    left = share_begin(total, shares, share + 1) - u0;             // (at least one)
    Walk<T, D, kEarly> load;
    for (int base = 0;; base += 32) {
        const int mine = base + lane < a.n_seqs ? seq_steps<T, D, kEarly>(a, base + lane) : 0;
        const int64_t own = mine ? mine * seq_items<T, kEarly>(a, base + lane) : 0;
        int64_t upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        const unsigned holds = __ballot_sync(0xffffffffu, u0 - before < upto);
        if (holds) {
            const int src = __ffs(holds) - 1;
            load.b = base + src;
            load.units = __shfl_sync(0xffffffffu, mine, src);
            load.tiles = seq_tiles<T, kEarly>(a, load.b);
            load.end = __shfl_sync(0xffffffffu, own, src);
            load.in_seq = u0 - before - (__shfl_sync(0xffffffffu, upto, src) - load.end);
            break;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    Walk<T, D, kEarly> at = load;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + (threadIdx.x >> 5) * kRingBytes;
    [[maybe_unused]] const uint32_t scratch = (uint32_t)__cvta_generic_to_shared(smem) + kShareWarps * kRingBytes +
                             (threadIdx.x >> 5) * Rows::kScratch;
    int64_t to_load = left;
    Stream<T, D, kEarly> st;
    int slot_in = 0, slot_out = 0;
    load.step = load.count = 0;
    st.asked = st.waiting = st.scale = 0.f;
    const auto copy_next = [&]() {
        if constexpr (sizeof(T) == 1) st.shift_scales();
        if (to_load > 0) {
            if (load.step == load.count) {
                if (!load.piece(a, to_load)) return;
                st.begin(a, load.b, load.item / load.tiles, load.lo, load.hi);
            }
            st.copy(a, load.step++, ring + slot_in * kStageBytes);
            --to_load;
        }
        slot_in = slot_in == kStages - 1 ? 0 : slot_in + 1;
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) copy_next(), cp_commit();
    bool first_piece = true;
#pragma unroll 1
    while (left > 0 && at.piece(a, left)) {
        const int b = at.b, h = at.item / at.tiles, r0 = (at.item % at.tiles) * Rows::kRows;
        Rows rows;
        // the sequence's first row and its rows times heads of the group
        int first_row = b, count = a.group;
        if constexpr (sizeof(T) == 1) {
            AttnSeq s = {b, 1, 0, 0, 0};
            if constexpr (Rows::kMany) s = attn_seq<kEarly>(a, b);
            first_row = s.row0, count = s.n * a.group;
            rows.template begin<kEarly>(a, s, h, r0);
        } else {
            rows.template begin<kEarly>(a, b, h, r0);
        }
#pragma unroll 1
        for (int step = 0; step < at.count; ++step) {
            cp_wait<kStages - 2>();
            __syncwarp();
            // (the stage that this copy fills was read in the previous step)
            copy_next();
            cp_commit();
            const uint32_t ks = ring + slot_out * kStageBytes, vs = ks + kStageBytes / 2;
            slot_out = slot_out == kStages - 1 ? 0 : slot_out + 1;
            if constexpr (sizeof(T) == 1) rows.step(a, ks, vs, at.hi, at.lo + step * KS, kStages == 2 ? st.waiting : st.scale);
            else rows.step(a, ks, vs, at.hi - (at.lo + step * KS), scratch);
        }
        left -= at.count;
        // the piece's rows: the result, or a part of it
        rows.end([&](int row, float m, float sum, bool writes_sum, auto write) {
            int g = r0 + row, to_row = first_row;
            if (g >= count) return;
            if (Rows::kMany) to_row += g / a.group, g %= a.group;
            const float inv = sum > 0.f ? 1.f / sum : sum;         // no key: 0; NaN stays
            const float lse2 = sum == 0.f ? -INFINITY : m + log2f(sum);
            const int head = h * a.group + g;
            const int64_t flat = (int64_t)to_row * a.hq + head;
            if (at.whole && !a.part_o) {
                write(static_cast<typename Rows::Out*>(a.o) + (int64_t)to_row * a.o_stride + (int64_t)head * D, inv);
                if (writes_sum && a.lse) a.lse[flat] = lse2 * kLn2;
                return;
            }
            const int64_t to = at.whole ? (int64_t)a.part_slot * a.n_rows * a.hq + flat
                                        : ((int64_t)share * 2 + (first_piece ? 0 : 1)) *
                                                  (sizeof(T) == 1 ? a.piece_rows : piece_rows<T>(a.group)) + row;
            write((at.whole ? a.part_o : a.piece_o) + to * D, inv);
            if (writes_sum) (at.whole ? a.part_lse : a.piece_lse)[to] = lse2;
        });
        first_piece = false;
    }
    cp_wait<0>();
}

}  // namespace
}  // namespace colibri
