// Attention on the tensor cores (tcgen05, TMEM, TMA) for bf16: prompts, and
// the shared prefix of a decode batch.
//
// One CTA takes two tiles of up to 128 rows of one sequence and key head and
// walks its keys 128 at a time.  A tile's rows are (token, head of the group)
// pairs, tokens * group of them, so the heads that share a key head share its
// keys in shared memory, and a decode batch over a shared prefix is the same
// kernel with the batch as the tokens.  Per tile and 128 keys:
//   S = Q K^T   (128 x 128 x d, f32 in tensor memory)
//   P = 2^(c S - m')  (bf16, written over S),  l += sum P
//   O += P V    (128 x d x 128, P read from tensor memory)
// with c = scale * log2(e), and instead of the running maximum a reference m'
// that stands as long as the weights are not above 2^24 (nor below 2^-64 while
// the row has none): bf16 and f32 hold weights up to 2^24 as exactly as those up
// to 1.  Whether it stands shows in the sum of the weights, so a maximum is taken,
// S read again, and O, which stays in tensor memory, multiplied by 2^(m - m'),
// only in the few steps that move the reference.
//
// Roles: warps 0-3 and 4-7 the softmax of the two tiles (one row per thread,
// no shuffles; they take over registers of the others, since a row's 128
// scores stay in registers), warps 8 and 10 issue the MMAs of one tile each
// (a wait costs about 150 cycles even when it is over; one warp for both tiles
// held the tensor pipe up between them), warps 9 and 11 the TMA copies (K and V
// tiles alternate in a ring; with pages, one box per page) and the work list.  A
// box costs the warp that issues it about 65 cycles, so that K and V of 16-key
// pages, from one warp, took 2700 cycles of a step's 3000 (chunks of prompts over a
// cache: 160 us, with a warp each 149).  The MMAs
// of one tile run while the other tile is in its softmax.  A commit after S(j + 1) also covers
// the O += P V of step j issued before it, so the one barrier per tile tells the
// softmax warps both that S is there and that O may be rescaled.
//
// The grid has a CTA per work item, those that see the most keys first; a
// running CTA takes over the next CTA that has not started (cluster launch
// control) while it works on its own item, so that the next item's copies and
// first scores overlap the end of the last one, and the tensor memory and
// barriers are set up once.
//
// P is rounded to bf16 because the MMA takes both operands in one 16-bit type;
// l adds the unrounded f32 values.
#include <cuda.h>
#include <cuda_runtime.h>

#include <numeric>

#include "attn_common.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace colibri {
namespace {

using namespace tc;

constexpr int kTcThreads = 384;               // 2 softmax warpgroups, 1 of MMA issue and copies
constexpr int kTileKeys = 128;
constexpr uint32_t kHalfBytes = 128 * 128;      // 128 rows of one 128-byte swizzle atom

// Ring slots of 128 keys: 5 of 32 KB, 8 of 16 KB (d = 64).
template <int D> constexpr int kSlots = D == 128 ? 5 : 8;
template <int D> constexpr uint32_t kTileBytes = (D / 64) * kHalfBytes;

// d = 64 leaves tensor memory for P in columns of its own: S(j + 1) is then formed
// as soon as S(j) is no longer needed, during the softmax of step j, and the order
// of the two tiles is left to the pipe.
template <int D> constexpr bool kOwnP = D == 64;

// DEV_TIMEOUT once a wait of any launch on this device has given up
// (colibri_attention_check).
__device__ int wait_status;

// A work item, as every role needs it.
struct Item {
    int b;                    // sequence, < 0: no more items
    int h, split, tok0;       // key head, key range, first token of tile 0
    int lo, hi;               // keys
    int steps[2];             // 128-key steps of each tile
    AttnSeq seq;
};

struct TcBars {
    alignas(16) uint8_t taken[16];   // the hardware's answer: which CTA was taken over
    uint64_t q_full[2];
    uint64_t q_empty[2];      // the item's last scores of the tile are done
    uint64_t s_full[2];       // S of the tile's next step is there, its O is up to date
    uint64_t p_most[2];       // O rescaled, P's first 96 keys written
    uint64_t p_ready[2];      // P's last 32 keys written
    uint64_t o_done[2];       // the item's last product of the tile is done (kOwnP: a step's)
    uint64_t s_read[2];       // kOwnP: the softmax is done with S
    uint64_t kv_full[8];
    uint64_t kv_empty[8];     // both tiles are done with the slot
    uint64_t tail[2];         // item n & 1's last value tile is cleared behind its last row
    uint64_t turn[2];         // the other tile's batch of MMAs has been issued
    uint64_t item_full[2];
    uint64_t item_empty[2];
    uint64_t taken_full;
    uint64_t drain[2];
    uint64_t never;           // failure-detection tests: nothing arrives
    uint32_t tmem;
    int abort;
    int announced;            // items that the copying warp has handed out
    uint32_t filled[2];       // K and V tiles copied
    int orphan;               // item[2] was taken over and not handed out
    Item item[3];
};

template <int D>
constexpr size_t tc_smem_bytes() {
    return 1024 + 2 * kTileBytes<D> + kSlots<D> * kTileBytes<D> + sizeof(TcBars);
}
static_assert(tc_smem_bytes<128>() <= 232448 && tc_smem_bytes<64>() <= 232448, "fits an SM");

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            int c3, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// 16 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}

// 32 bytes to a 32-byte boundary.
__device__ __forceinline__ void store32(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// One lane of the (whole) warp; the form that lets the compiler keep what the
// lane issues in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// A value that every lane holds, as a uniform one.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                            int c3, int c4, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

// A K or V tile in shared memory is made of atoms of 8 keys x 64 columns (1024
// bytes, 128-byte swizzle).  Packed keys: one copy per 64-column half, the
// halves behind each other.  Pages: one copy brings all columns of a page's
// keys, so the halves of 8 keys lie next to each other, whatever part of the
// tile the page is (16-key pages with one copy per half: 4850 cycles per step
// against 2700 without pages).
template <int D, bool kPaged> constexpr uint32_t kGroupBytes = kPaged ? (D / 64) * 1024 : 1024;   // next 8 keys
template <bool kPaged> constexpr uint32_t kColumnBytes = kPaged ? 1024 : kHalfBytes;              // next 64 columns

// K: K-major.  V: B operand with the MN index contiguous (its rows, the keys,
// are the MMA's K).
template <int D, bool kPaged>
__device__ __forceinline__ uint64_t smem_desc_k(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;                                     // (leading offset, unused)
    d |= (uint64_t)(kGroupBytes<D, kPaged> >> 4) << 32;         // stride offset: next 8 keys
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;                                     // 128-byte swizzle
    return d;
}
template <int D, bool kPaged>
__device__ __forceinline__ uint64_t smem_desc_v(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kColumnBytes<kPaged> >> 4) << 16;           // leading offset: next 64 columns
    d |= (uint64_t)(kGroupBytes<D, kPaged> >> 4) << 32;         // stride offset: next 8 keys
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Pages and heads as one dimension of the tensor map: page p, head h is unit
// p * per_page + h * per_head of `count`.
struct Units {
    int per_page, per_head, count;
};

// mbar_wait for a chain of short waits: the clock and the abort flag are looked
// at once in 64 tries (reading the global timer takes longer than most waits).
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                             uint64_t limit_ns) {
    uint64_t t0 = 0;
    for (int i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (i & 63) continue;
        if (*abort_flag) return false;
        const uint64_t now = globaltimer();
        if (t0 == 0) t0 = now;
        if (now - t0 > limit_ns) {
            *abort_flag = 1;
            return false;
        }
    }
}

// Asks for the next CTA that has not started; the answer arrives on `bar`.
__device__ __forceinline__ void take_over(uint32_t answer, uint32_t bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     answer),
                 "r"(bar)
                 : "memory");
}
// The answer: true and the CTA's index, or false when none was left.
__device__ __forceinline__ bool taken_over(uint32_t answer, int* x, int* y) {
    uint32_t got, cx, cy;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%3];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\tmov.u32 %2, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, _, _}, r;\n\t}"
        : "=&r"(got), "=&r"(cx), "=&r"(cy)
        : "r"(answer)
        : "memory");
    *x = (int)cx, *y = (int)cy;
    return got != 0;
}

// CTA (x, y) of the grid as a work item; called by a whole warp.
__device__ __forceinline__ Item work_item(const AttnArgs& a, int x, int y, int tokens) {
    Item it;
    int tile = 0;
    it.b = -1;
    it.h = x % a.hkv, it.split = y;
    if (!attn_item(a, x / a.hkv, 1, 2 * tokens, gridDim.x * gridDim.y > 152, &it.b, &tile)) {
        it.b = -1;
        return it;
    }
    it.seq = attn_seq(a, it.b);
    it.tok0 = tile * 2 * tokens;
    int ends[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = it.tok0 + t * tokens, last = min(first + tokens, it.seq.n);
        ends[t] = first < it.seq.n ? attn_limit_max(a, it.seq, first, last) : 0;
    }
    attn_split(a, y, kTileKeys, it.seq.kv0, max(ends[0], ends[1]), &it.lo, &it.hi);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int end = min(it.hi, ends[t]);
        it.steps[t] = end > it.lo ? (end - it.lo + kTileKeys - 1) / kTileKeys : 0;
    }
    return it;
}

template <int D, bool kPaged>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, AttnArgs a, int tokens, int box, Units units) {
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* skv = smem + 2 * kTileBytes<D>;
    TcBars& bars = *reinterpret_cast<TcBars*>(skv + kSlots<D> * kTileBytes<D>);
    const uint32_t q0 = smem_u32(smem), kv0 = smem_u32(skv);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

    if (tid == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&bars.q_full[t]), 1);
            mbar_init(smem_u32(&bars.q_empty[t]), 1);
            mbar_init(smem_u32(&bars.s_full[t]), 1);
            mbar_init(smem_u32(&bars.p_most[t]), 4);
            mbar_init(smem_u32(&bars.p_ready[t]), 4);
            mbar_init(smem_u32(&bars.o_done[t]), 1);
            mbar_init(smem_u32(&bars.s_read[t]), 4);
            mbar_init(smem_u32(&bars.item_full[t]), 1);
            mbar_init(smem_u32(&bars.item_empty[t]), 11);       // softmax and MMA warps, V's copies
            mbar_init(smem_u32(&bars.drain[t]), 1);
            mbar_init(smem_u32(&bars.tail[t]), 2);
            mbar_init(smem_u32(&bars.turn[t]), 1);
        }
        for (int s = 0; s < kSlots<D>; ++s) {
            mbar_init(smem_u32(&bars.kv_full[s]), 1);
            mbar_init(smem_u32(&bars.kv_empty[s]), 2);
        }
        mbar_init(smem_u32(&bars.taken_full), 1);
        for (const CUtensorMap* m : {&tm_q, &tm_k, &tm_v})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
        mbar_init(smem_u32(&bars.never), 1);
        bars.abort = bars.announced = bars.orphan = 0;
        bars.filled[0] = bars.filled[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_enter();
    if (warp == 9) {
        const Item it = work_item(a, blockIdx.x, blockIdx.y, tokens);
        if (lane == 0) bars.item[0] = it;
    }
    __syncthreads();
    if (bars.item[0].b < 0) return;                             // (and so are all later CTAs)
    if (warp == 8) tmem_alloc<false>(smem_u32(&bars.tmem), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = uniform(bars.tmem);
    volatile int* abort_flag = &bars.abort;
    const uint64_t limit = a.wait_limit_ns;
    // S0 0, S1 128, O0 256, O1 256 + D; P over S, or P0 384, P1 448
    constexpr uint32_t kColO = 256, kColP = kOwnP<D> ? 384 : 0, kStepP = kOwnP<D> ? 64 : 128;
    // one outcome for the whole warp, so that no collective runs without its lanes
    const auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, bounded_wait(smem_u32(bar), parity, abort_flag, limit)) != 0;
    };
    // item n of this CTA (the first one is there from the start)
    const auto item_there = [&](int n) { return n == 0 || warp_wait(&bars.item_full[n & 1], ((n >> 1) - !(n & 1)) & 1); };
    const auto item_left = [&](int n) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.item_empty[n & 1]));
    };
    int item_no = 0;                                            // items that this warp is done with

    const bool wide_rows = (reinterpret_cast<uintptr_t>(a.o) % 32 | (uint64_t)a.o_stride % 16) == 0;
    // Output rows of an item's tile t: this thread's row times inv, or NaN.
    const auto write_row = [&](const Item& it, int t, bool ok, bool keys, float l, float m, uint32_t to) {
        const int r = tid & 127, i = it.tok0 + t * tokens + r / a.group, g = r % a.group;
        const bool live = r < tokens * a.group && i < it.seq.n;
        // o / l; a row without keys has l = 0
        const float inv = !ok ? __int_as_float(0x7fc00000) : l > 0.f ? 1.f / l : l;
        const int row = it.seq.row0 + i;
        const int64_t flat = (int64_t)row * a.hq + it.h * a.group + g;
        const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);
        const int64_t at = (int64_t)(a.part_slot + it.split) * a.n_rows * a.hq + flat;
        if (live) {
            if (a.part_o) a.part_lse[at] = ok ? lse2 : inv;
            else if (a.lse) a.lse[flat] = ok ? lse2 * kLn2 : inv;
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            uint32_t o[32];
            if (keys) {
                tmem_ld32(to + 32 * x, o);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = 0;
            }
            if (!live) continue;
            // (a row that saw no key may stand in a tile that did)
#pragma unroll
            for (int y = 0; y < 32; ++y) o[y] = l == 0.f && ok ? 0 : __float_as_uint(__uint_as_float(o[y]) * inv);
            // (a row per thread: every store of a warp touches 32 cache lines, so
            // few wide ones; 16-byte stores took 3550 cycles per item, as many as 1.3
            // steps)
            if (a.part_o) {
#pragma unroll
                for (int y = 0; y < 4; ++y) store32(a.part_o + at * D + 32 * x + 8 * y, o + 8 * y);
            } else {
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (int64_t)row * a.o_stride +
                                     (int64_t)(it.h * a.group + g) * D + 32 * x;
                uint32_t w[16];
#pragma unroll
                for (int y = 0; y < 16; ++y) w[y] = pack_h2<false>(__uint_as_float(o[2 * y]), __uint_as_float(o[2 * y + 1]));
                if (wide_rows) {
                    store32(dst, w);
                    store32(dst + 16, w + 8);
                } else {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        reinterpret_cast<uint4*>(dst)[y] = make_uint4(w[4 * y], w[4 * y + 1], w[4 * y + 2], w[4 * y + 3]);
                }
            }
        }
    };

    if (warp < 8) {
        // ------------------------------------------------ softmax, one row per thread
        // (384 x 168 registers at launch = 256 x 208 + 128 x 88)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int t = warp >> 2, r = tid & 127;
        const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lane_base + t * 128, to = lane_base + kColO + t * D, tp = lane_base + kColP + t * kStepP;
        const float c = a.scale_log2;
        const auto hand_over = [&](uint64_t* bar) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(bar));
        };
        uint32_t step_no = 0, done_no = 0;                      // of this tile, over all items
        // The warp stays together whatever a wait says: a lane whose wait gave up
        // goes on without waiting, to the end of the item, whose rows become NaN.
        bool ok = true;
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok) ok = bounded_wait(smem_u32(bar), parity, abort_flag, limit);
            __syncwarp();
            tc_fence_after();
        };
        while (ok) {
            ok = item_there(item_no);
            if (!ok) break;
            const Item& it = bars.item[item_no & 1];
            if (it.b < 0) break;
            const int i = it.tok0 + t * tokens + r / a.group;
            const bool live = r < tokens * a.group && i < it.seq.n;
            const int steps = uniform(it.steps[t]), lo = uniform(it.lo);
            // (a thread without a row computes what nobody reads; it masks nothing
            // and never moves its reference)
            const int lim = live ? min(it.hi, attn_limit(a, it.seq, i)) : it.hi;
            float m = 0.f, l = 0.f;            // reference (in units of log2), sum of the weights
            for (int j = 0; j < steps; ++j, ++step_no) {
                wait(&bars.s_full[t], step_no & 1);
                const int left = lim - (lo + j * kTileKeys);       // keys of this step that the row sees
                uint32_t s[4][32], p[3][16];
                uint64_t sum[4], c2 = pack2(c, c), ref2;
                const auto weights = [&](const uint32_t (&sx)[32], uint32_t (&px)[16]) {
#pragma unroll
                    for (int y = 0; y < 16; ++y) {
                        const float2 e =
                            unpack2(fma2(pack2(__uint_as_float(sx[2 * y]), __uint_as_float(sx[2 * y + 1])), c2, ref2));
                        const float p0 = ex2(e.x), p1 = ex2(e.y);
                        sum[y & 3] = add2(sum[y & 3], pack2(p0, p1));
                        px[y] = pack_h2<false>(p0, p1);
                    }
                };
                // S of the step, -infinity where the row sees no key
                const auto load_scores = [&]() {
#pragma unroll
                    for (int x = 0; x < 4; ++x) tmem_ld32(ts + 32 * x, s[x]);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        if (left >= 32 * x + 32) continue;         // (rows of a warp differ by few keys)
#pragma unroll
                        for (int y = 0; y < 32; ++y)
                            if (x * 32 + y >= left) s[x][y] = 0xff800000u;
                    }
                };
                // largest of chunks from .. 3, times c
                const auto largest = [&](int from) {
                    float top[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) top[x] = -INFINITY;
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (x >= from) {
#pragma unroll
                            for (int y = 0; y < 32; y += 2)
                                top[y / 2 % 8] = max3(top[y / 2 % 8], __uint_as_float(s[x][y]), __uint_as_float(s[x][y + 1]));
                        }
                    return max3(max3(top[0], top[1], top[2]), max3(top[3], top[4], top[5]), fmaxf(top[6], top[7])) * c;
                };
                bool waited = false;                               // for the last step's product
#pragma unroll 1
                for (int pass = 0;; ++pass) {
                    load_scores();
                    // The weights are formed on the reference as it is.  Whether it
                    // stands shows in their sum (of the first 96; of the last 32, not
                    // formed yet, in the largest score): a maximum is taken only in
                    // the few steps where it does not
                    ref2 = pack2(-m, -m);
                    sum[0] = sum[1] = sum[2] = sum[3] = 0;
#pragma unroll
                    for (int x = 0; x < 3; ++x) weights(s[x], p[x]);
                    const float2 some = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                    const float most = largest(3), weight = some.x + some.y;
                    const bool high = !(weight <= 16777216.f) || most > m + 24.f;
                    const bool low = l == 0.f && left > 0 && weight < 5.421010862427522e-20f && most < m - 64.f;   // 2^-64
                    if (pass > 0 || !__any_sync(0xffffffffu, live && (high || low))) break;
                    load_scores();
                    const float mn = largest(0);
                    // (a sum above 2^24 has a weight above 2^17)
                    const bool move = live && (mn > m + 16.f || (l == 0.f && mn < m - 64.f && mn != -INFINITY));
                    if (!__any_sync(0xffffffffu, move)) break;
                    // (a row without weight yet has O = 0, or none before the first product)
                    const float keep = move && l != 0.f ? ex2(m - mn) : 1.f;
                    if (move) m = mn;
                    l *= keep;
                    if (j > 0) {
                        if (kOwnP<D>) {
                            wait(&bars.o_done[t], (step_no - 1) & 1);
                            waited = true;
                        }
#pragma unroll
                        for (int x = 0; x < D / 16; ++x) {
                            uint32_t o[16];
                            tmem_ld16(to + 16 * x, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * keep);
                            tmem_st16(to + 16 * x, o);
                        }
                    }
                }
                if (kOwnP<D>) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&bars.s_read[t]));
                    // P's columns are free once the last step's product is done
                    if (j > 0 && !waited) wait(&bars.o_done[t], (step_no - 1) & 1);
                }
#pragma unroll
                for (int x = 0; x < 3; ++x) tmem_st16(tp + 16 * x, p[x]);
                hand_over(&bars.p_most[t]);                        // the product with V starts on these
                weights(s[3], p[0]);
                tmem_st16(tp + 48, p[0]);
                hand_over(&bars.p_ready[t]);
                const float2 sums = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                l += sums.x + sums.y;
            }
            if (steps > 0) wait(&bars.o_done[t], (kOwnP<D> ? step_no - 1 : done_no++) & 1);
            ok = __all_sync(0xffffffffu, ok);
            write_row(it, t, ok, steps > 0, l, m, to);
            item_left(item_no++);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp == 8 || warp == 10) {
            // ------------------------------------------------ MMA issue, one tile each
            const int t = warp == 8 ? 0 : 1;
            constexpr uint32_t kIdS = idesc_bf16(128, kTileKeys);
            constexpr uint32_t kIdO = idesc_bf16(128, D) | (1u << 16);   // V: MN-major
            const uint32_t ts = tmem + t * 128, to = tmem + kColO + t * D, tp = tmem + kColP + t * kStepP;
            const uint32_t qt = q0 + t * kTileBytes<D>;
            const bool leader = elect_one();
            // The warp stays together whatever a wait says: a lane whose wait gave
            // up goes on without waiting, and the leader issues nothing more.
            bool ok = true;
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                if (ok) ok = bounded_wait(smem_u32(bar), parity, abort_flag, limit);
                __syncwarp();
            };
            const auto scores = [&](int slot) {
                const uint32_t k = kv0 + slot * kTileBytes<D>;
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    mma_bf16<false>(ts, smem_desc_sw128(qt + (x / 4) * kHalfBytes + (x % 4) * 32),
                                    smem_desc_k<D, kPaged>(k + (x / 4) * kColumnBytes<kPaged> + (x % 4) * 32), kIdS, x > 0);
                }
                mma_commit<false>(smem_u32(&bars.s_full[t]));
            };
            // slots in the order K(0), V(0), K(1), ...; `next` waits for the one after the last
            int slot = -1;
            uint32_t lap = 0;
            const auto next = [&]() {
                if (++slot == kSlots<D>) slot = 0, lap ^= 1;
                wait(&bars.kv_full[slot], lap);
                return slot;
            };
            // The two tiles' batches (the product of a step and the next scores) go to
            // the tensor pipe in turn.  Left alone, the pipe shares itself between
            // them, both tiles then finish and start their softmax together, and the
            // pipe waits for both (8192 tokens: 439 us instead of 356).
            uint32_t batch = 0;
            const auto my_turn = [&]() {
                if (kOwnP<D>) return;
                if (t == 1) wait(&bars.turn[1], batch & 1);
                else if (batch > 0) wait(&bars.turn[0], (batch - 1) & 1);
                ++batch;
            };
            const auto pass_on = [&]() {
                if (!kOwnP<D>) mbar_arrive(smem_u32(&bars.turn[t ^ 1]));
            };
            uint32_t step_no = 0, q_no = 0, tail_laps = 0, s_no = 0;
            // kOwnP: the scores before these are no longer needed
            const auto s_free = [&]() {
                if (!kOwnP<D>) return;
                if (s_no > 0) {
                    wait(&bars.s_read[t], (s_no - 1) & 1);
                    tc_fence_after();
                }
                ++s_no;
            };
            while (__all_sync(0xffffffffu, ok)) {
                if (!item_there(item_no)) {
                    ok = false;
                    break;
                }
                const Item& it = bars.item[item_no & 1];
                if (uniform(it.b) < 0) break;
                const int mine = uniform(it.steps[t]), nsteps = max(mine, uniform(it.steps[t ^ 1]));
                const int have = uniform((it.hi - it.lo) % kTileKeys);      // keys of the last tile, 0: all
                int kslot = 0, vslot = 0;
                if (nsteps > 0) {
                    kslot = next();
                    if (mine > 0) {
                        wait(&bars.q_full[t], q_no++ & 1);
                        s_free();
                    }
                    my_turn();
                    if (leader && ok) {
                        if (mine > 0) {
                            scores(kslot);
                            if (mine == 1) mma_commit<false>(smem_u32(&bars.q_empty[t]));
                        }
                        pass_on();
                        mma_commit<false>(smem_u32(&bars.kv_empty[kslot]));
                    }
                    __syncwarp();
                }
                for (int j = 0; j < nsteps; ++j) {
                    vslot = next();
                    if (j + 1 < nsteps) kslot = next();
                    const uint32_t v = kv0 + vslot * kTileBytes<D>;
                    if (j + 1 == nsteps && have > 0) {
                        // rows behind the last key: their weights are 0, and 0
                        // times whatever lies there has to be 0.  Each of the
                        // two warps clears half of them.
                        for (int e = lane + 32 * t; e < (kTileKeys - have) * (D / 8); e += 64) {
                            const int row = have + e / (D / 8), c = e % (D / 8);
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             v + (row >> 3) * kGroupBytes<D, kPaged> + (c >> 3) * kColumnBytes<kPaged> +
                                             (row & 7) * 128 + (c & 7) * 16),
                                         "r"(0)
                                         : "memory");
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&bars.tail[item_no & 1]));
                        wait(&bars.tail[item_no & 1], tail_laps >> (item_no & 1) & 1);
                        tail_laps ^= 1u << (item_no & 1);
                    }
                    const auto product = [&](int x) {
                        mma_f16_ta(to, tp + x * 8, smem_desc_v<D, kPaged>(v + x * 2 * kGroupBytes<D, kPaged>), kIdO, j > 0 || x > 0);
                    };
                    if (kOwnP<D> && j + 1 < mine) {
                        s_free();
                        if (leader && ok) {
                            scores(kslot);
                            if (j + 2 == mine) mma_commit<false>(smem_u32(&bars.q_empty[t]));
                        }
                        __syncwarp();
                    }
                    my_turn();
                    if (j < mine) {
                        wait(&bars.p_most[t], step_no & 1);
                        tc_fence_after();
                        if (leader && ok) {
#pragma unroll
                            for (int x = 0; x < 6; ++x) product(x);
                        }
                        __syncwarp();
                        wait(&bars.p_ready[t], step_no & 1);
                        ++step_no;
                        tc_fence_after();
                    }
                    if (leader && ok) {
                        if (j < mine) {
                            product(6);
                            product(7);
                            if (kOwnP<D> || j + 1 == mine) mma_commit<false>(smem_u32(&bars.o_done[t]));
                        }
                        if (!kOwnP<D> && j + 1 < mine) {
                            scores(kslot);
                            if (j + 2 == mine) mma_commit<false>(smem_u32(&bars.q_empty[t]));
                        }
                        pass_on();
                        mma_commit<false>(smem_u32(&bars.kv_empty[vslot]));
                        if (j + 1 < nsteps) mma_commit<false>(smem_u32(&bars.kv_empty[kslot]));
                    }
                    __syncwarp();
                }
                item_left(item_no++);
            }
            // wait, bounded, for all that was issued: no arrival is outstanding
            // when the CTA ends
            if (leader) {
                mma_commit<false>(smem_u32(&bars.drain[t]));
                mbar_wait_drain(smem_u32(&bars.drain[t]), 0, kDrainLimitNs);
            }
            __syncwarp();
        } else {
            // ------------------------------------------------ TMA copies: warp 9 Q and K, and
            // the work list; warp 11 V.  Tile i of K is number 2 i of the ring, of V
            // 2 i + 1.  (One code for both warps: a kernel as short as a prefix's takes
            // 2 us more with two, which have to be fetched.)
            const int kind = warp == 11;
            uint32_t filled = 0;                                    // tiles so far, over all items
            uint32_t q_no[2] = {0, 0};
            const uint32_t answer = smem_u32(bars.taken), answer_bar = smem_u32(&bars.taken_full);
            const CUtensorMap* map = kind ? &tm_v : &tm_k;
            const bool leader = elect_one();
            // (failure-detection tests: no Q and K are copied from item stall_tma on)
            bool ok = kind || a.stall_tma != 1 || warp_wait(&bars.never, 0);
            bool asked = false;
            if (!kind && lane == 0) bars.announced = 1;
            while (ok) {
                if (kind) {
                    ok = item_there(item_no);
                    if (!ok || uniform(bars.item[item_no & 1].b) < 0) break;
                }
                const Item& it = bars.item[item_no & 1];
                const int lo = uniform(it.lo), hi = uniform(it.hi), h = uniform(it.h);
                const int nsteps = uniform(max(it.steps[0], it.steps[1]));
                const auto ask = [&]() {
                    if (lane == 0) {
                        mbar_expect_tx(answer_bar, 16);
                        take_over(answer, answer_bar);
                    }
                    asked = true;
                };
                for (int t = 0; t < 2 && ok && !kind; ++t) {
                    if (uniform(it.steps[t]) == 0) continue;
                    if (q_no[t] > 0) ok = warp_wait(&bars.q_empty[t], (q_no[t] - 1) & 1);
                    if (!ok) break;
                    ++q_no[t];
                    if (lane == 0) {
                        const uint32_t bar = smem_u32(&bars.q_full[t]);
                        mbar_expect_tx(bar, tokens * a.group * 128 * (D / 64));
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_4d(q0 + t * kTileBytes<D> + x * kHalfBytes, &tm_q, 64 * x, 0,
                                        it.seq.row0 + it.tok0 + t * tokens, h, bar);
                    }
                    __syncwarp();
                }
                // page ids of 32 boxes, one per lane, and of the 32 after them
                const int per_step = kTileKeys / box;
                const auto look = [&](int first) {
                    const int key = lo + (first + lane) * box;
                    return kPaged && key < hi ? attn_page(a, it.b, key >> a.page_shift) : -1;
                };
                int ids = look(0), ids_ahead = look(32), page = -1;
                for (int j = 0; j < nsteps && ok; ++j) {
                    const uint32_t n = 2 * filled + kind, slot = n % kSlots<D>;
                    const int base = lo + j * kTileKeys;
                    if (kPaged) {
                        const int first = j * per_step;
                        if (first > 0 && (first & 31) == 0) ids = ids_ahead, ids_ahead = look(first + 32);
                        page = __shfl_sync(0xffffffffu, ids, (first + lane) & 31);
                    }
                    // the next item is taken as late as its copies can still follow
                    // this one's: whoever is free first takes the longest left
                    if (!kind && j == nsteps - 1) {
                        ask();
                        if (a.stall_tma > 1 && item_no + 1 >= a.stall_tma) ok = warp_wait(&bars.never, 0);
                        if (!ok) break;
                    }
                    if (n >= kSlots<D>) ok = warp_wait(&bars.kv_empty[slot], (n / kSlots<D> - 1) & 1);
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&bars.kv_full[slot]);
                    const uint32_t dst = kv0 + slot * kTileBytes<D>;
                    if (kPaged) {
                        // one box per page, lane l has box l; a page that does not
                        // exist lies outside the tensor and gives zeros
                        const int boxes = (min(kTileKeys, hi - base) + box - 1) / box;
                        if (lane == 0) mbar_expect_tx(bar, boxes * box * D * 2);
                        __syncwarp();
                        if (lane < boxes)
                            tma_load_5d(dst + lane * box * D * 2, map, 0, 0, 0, ((base + lane * box) & (a.page_size - 1)) >> 3,
                                        page < 0 ? units.count : page * units.per_page + h * units.per_head, bar);
                    } else if (leader) {
                        mbar_expect_tx(bar, kTileBytes<D>);
#pragma unroll
                        for (int x = 0; x < D / 64; ++x)
                            tma_load_4d(dst + x * kHalfBytes, map, 64 * x, it.seq.row0 + base, h, 0, bar);
                    }
                    __syncwarp();
                    ++filled;
                }
                if (!ok) break;
                if (kind) {
                    item_left(item_no++);
                    continue;
                }
                if (nsteps == 0) ask();
                // the next item
                ok = warp_wait(&bars.taken_full, item_no & 1);
                if (!ok) break;
                asked = false;
                int x, y;
                Item nx;
                nx.b = -1;
                if (taken_over(answer, &x, &y)) nx = work_item(a, x, y, tokens);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (the answer is read before the next)
                const int n = item_no + 1;
                if (n >= 2) ok = warp_wait(&bars.item_empty[n & 1], ((n >> 1) - 1) & 1);
                if (!ok) {
                    if (nx.b >= 0 && lane == 0) bars.item[2] = nx, bars.orphan = 1;
                    break;
                }
                if (lane == 0) {
                    bars.item[n & 1] = nx;
                    bars.announced = n + 1;
                    mbar_arrive(smem_u32(&bars.item_full[n & 1]));
                }
                __syncwarp();
                item_no = n;
                if (uniform(nx.b) < 0) break;
            }
            // a CTA that gave up leaves none of its copies in flight, and none of the
            // work it took over unanswered
            if (!kind && *abort_flag) {
                if (asked) {
                    mbar_wait_drain(answer_bar, item_no & 1, kDrainLimitNs);
                    __syncwarp();
                    int x, y;
                    if (mbar_try_wait(answer_bar, item_no & 1) && taken_over(answer, &x, &y)) {
                        const Item nx = work_item(a, x, y, tokens);
                        if (lane == 0 && nx.b >= 0) bars.item[2] = nx, bars.orphan = 1;
                    }
                }
                if (lane == 0) {
                    for (int t = 0; t < 2; ++t)
                        if (q_no[t] > 0) mbar_wait_drain(smem_u32(&bars.q_full[t]), (q_no[t] - 1) & 1, kDrainLimitNs);
                }
                __syncwarp();
            }
            if (lane == 0) bars.filled[kind] = filled;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (bars.abort && tid == 0) {
        atomicExch(&wait_status, DEV_TIMEOUT);
        // none of the copies stays in flight: each slot's last one
        for (uint32_t slot = 0; slot < kSlots<D>; ++slot) {
            int last = -1;
            for (int kind = 0; kind < 2; ++kind)
                for (int i = max((int)bars.filled[kind] - kSlots<D>, 0); i < (int)bars.filled[kind]; ++i)
                    if ((2 * i + kind) % kSlots<D> == (int)slot) last = max(last, 2 * i + kind);
            if (last >= 0) mbar_wait_drain(smem_u32(&bars.kv_full[slot]), (last / kSlots<D>) & 1, kDrainLimitNs);
        }
    }
    if (bars.abort && warp < 8) {
        // rows of items that were handed out or taken over, and that this warp
        // has not come to
        for (int n = item_no; n < bars.announced; ++n)
            if (bars.item[n & 1].b >= 0) write_row(bars.item[n & 1], warp >> 2, false, false, 0.f, 0.f, 0);
        if (bars.orphan) write_row(bars.item[2], warp >> 2, false, false, 0.f, 0.f, 0);
    }
    if (warp == 8) tmem_dealloc<false>(tmem, 512);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// bf16 tensor of `rank` dimensions (innermost first, contiguous) with strides in
// elements, 128-byte swizzle, zeros outside.
bool encode(CUtensorMap* m, const void* p, int rank, const int64_t* dims, const int64_t* strides, const int* boxes) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[5], s[4];
    cuuint32_t b[5], ones[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = (cuuint64_t)dims[i], b[i] = (cuuint32_t)boxes[i], ones[i] = 1;
        // (the stride of a dimension of one entry is never used, but has to be valid)
        if (i > 0) s[i - 1] = (cuuint64_t)(dims[i] > 1 ? strides[i - 1] : dims[0]) * 2;
    }
    const auto call = [&]() {
        return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(p), d, s, b, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (call()) return true;
    // a driver call needs the device's context current, which a thread that has
    // not called the runtime yet does not have
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess && call();
}

template <int D, bool kPaged>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    const int tokens = 128 / a.group;
    CUtensorMap tq, tk, tv;
    const int64_t qd[4] = {D, a.group, a.n_rows, a.hkv}, qs[3] = {D, a.q_stride, (int64_t)a.group * D};
    const int qb[4] = {64, a.group, tokens, 1};
    bool ok = encode(&tq, a.q, 4, qd, qs, qb);
    int box = kTileKeys;
    Units units{};
    if (kPaged) {
        box = a.page_size < kTileKeys ? a.page_size : kTileKeys;
        int64_t unit;
        if (!attn_tc_units(a, &unit, &units.per_page, &units.per_head, &units.count)) return cudaErrorInvalidValue;
        const int64_t kd[5] = {64, 8, D / 64, a.page_size / 8, units.count},
                      ks[4] = {a.row_stride, 64, 8 * a.row_stride, unit};
        const int kb[5] = {64, 8, D / 64, box / 8, 1};
        ok = ok && encode(&tk, a.k, 5, kd, ks, kb) && encode(&tv, a.v, 5, kd, ks, kb);
    } else {
        const int64_t kd[4] = {D, a.page_size, a.hkv, 1}, ks[3] = {a.row_stride, a.head_stride, 0};
        const int kb[4] = {64, box, 1, 1};
        ok = ok && encode(&tk, a.k, 4, kd, ks, kb) && encode(&tv, a.v, 4, kd, ks, kb);
    }
    if (!ok) return cudaErrorInvalidValue;
    auto kern = attn_tc_kernel<D, kPaged>;
    const int bytes = (int)tc_smem_bytes<D>();
    cudaError_t e = smem_attr((const void*)kern, bytes);
    if (e != cudaSuccess) return e;
    const int64_t items = attn_tc_items(a);
    return launch_pdl(kern, dim3((unsigned)(items * a.hkv), a.splits), dim3(kTcThreads), bytes, s, tq, tk, tv, a, tokens,
                      box, units);
}

}  // namespace

int64_t attn_tc_items(const AttnArgs& a) {
    const int per = 2 * (128 / a.group);
    return a.mode == kAttnPrompt ? a.n_rows / per + a.n_seqs : (a.n_seqs + per - 1) / per;
}

// Pages and heads in units of the greatest common divisor of their strides.
bool attn_tc_units(const AttnArgs& a, int64_t* unit, int* per_page, int* per_head, int* count) {
    const int64_t g = a.hkv > 1 && a.num_pages > 1 ? std::gcd(a.page_stride, a.head_stride)
                      : a.hkv > 1                  ? a.head_stride
                                                   : a.page_stride;
    const int64_t pp = a.num_pages > 1 ? a.page_stride / g : 0, ph = a.hkv > 1 ? a.head_stride / g : 0;
    const int64_t n = (a.num_pages - 1) * pp + (a.hkv - 1) * ph + 1;
    if (n > 0x7fffffff) return false;
    *unit = g, *per_page = (int)pp, *per_head = (int)ph, *count = (int)n;
    return true;
}

cudaError_t attn_tc_status(int* status, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(status, wait_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || *status == DEV_OK) return e;
    const int ok = DEV_OK;
    e = cudaMemcpyToSymbolAsync(wait_status, &ok, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    return e != cudaSuccess ? e : cudaStreamSynchronize(s);
}

cudaError_t launch_attn_tc(int d, const AttnArgs& a, cudaStream_t s) {
    if (a.table) return d == 64 ? launch<64, true>(a, s) : launch<128, true>(a, s);
    return d == 64 ? launch<64, false>(a, s) : launch<128, false>(a, s);
}

}  // namespace colibri
