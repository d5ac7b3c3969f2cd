// Joins the partial rows of key ranges: with w_i = 2^(log2-sum_i - largest),
//   o = sum_i w_i o_i / sum_i w_i,   ln-sum = ln2 (largest + log2 sum_i w_i)
// in a fixed order, so that results do not depend on timing.
//
// One CTA per (row, head).  Bound by latency: every warp takes every so-manieth
// part and reads the log2-sums and rows of eight parts at once, keeping its own
// largest log2-sum; the warps' sums are joined at the end.  A range that held no
// key of the row has log2-sum -infinity, so weight 0, and left zeros.  A NaN
// log2-sum (scores that are NaN, rows whose wait gave up) makes the row NaN.
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "kernels.h"

namespace colibri {
namespace {

constexpr int kBatch = 8;

// Where a row's parts are.
struct Place {
    int live;             // the row belongs to a sequence, and has parts to join
    int c0, c1;           // shares that hold its keys
    int first_is_last;    // its piece of share c0 is that share's last
};

// Called by a whole warp.
template <typename T, int D, bool kEarly>
__device__ __forceinline__ Place row_parts(const AttnArgs& a, int row, int head, int slots, int shares_per_seq) {
    Place p = {1, 0, -1, 0};
    if (shares_per_seq) {
        int64_t total, first;
        count_steps<T, D, kEarly>(a, shares_per_seq, row, &total, &first);
        const int steps = seq_steps<T, D, kEarly>(a, row);
        if (steps > 0) {
            const int shares = share_count(total);
            first += (int64_t)((head / a.group) * row_tiles<T>(a.group) + (head % a.group) / row_tile<T>(a.group)) * steps;
            p.c0 = share_of(total, shares, first);
            p.c1 = share_of(total, shares, first + steps - 1);
            p.first_is_last = share_begin(total, shares, p.c0) < first;
        }
        p.live = p.c0 != p.c1 || slots > 0;                        // (else written by the one share)
    } else if (a.mode == kAttnPrompt) {
        p.live = 0;
        for (int b = threadIdx.x & 31; b < a.n_seqs; b += 32)
            p.live |= row >= max(ld_early<kEarly>(a.seq_start + b), 0) && row < ld_early<kEarly>(a.seq_start + b + 1);
        p.live = __any_sync(0xffffffffu, p.live);
    }
    return p;
}

// Lengths are read before the wait, from L2 (ld_early), while they are few: the long
// sequence of 65421 keys takes 48 us instead of 50, 64 sequences 50 instead of 51.
// Every CTA reads all of them, and many come faster through L1: 256 sequences of 1000
// keys 183 instead of 185 us, 4096 3960 instead of 5550.
constexpr int kEarlySeqs = 128;

template <typename T, int D, int kThreads>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(const __grid_constant__ AttnArgs a, int slots,
                                                             int shares_per_seq) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float4 rows[kWarps][D / 4];
    __shared__ float tops[kWarps], sums[kWarps];
    __shared__ Place place;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t flat = blockIdx.x;
    const int64_t total_rows = (int64_t)a.n_rows * a.hq;
    const int row = (int)(flat / (uint32_t)a.hq), head = (int)(flat % (uint32_t)a.hq);
    const int tile_row = (head % a.group) % row_tile<T>(a.group);
    const bool early = a.n_seqs <= kEarlySeqs;
    if (!early) pdl_enter();
    if (warp == 0) {
        const Place p = early ? row_parts<T, D, true>(a, row, head, slots, shares_per_seq)
                              : row_parts<T, D, false>(a, row, head, slots, shares_per_seq);
        if (lane == 0) place = p;
    }
    if (early) pdl_enter();
    __syncthreads();
    if (!place.live) return;
    const int c0 = place.c0, c1 = place.c1;
    const bool one = shares_per_seq && c0 == c1;                   // whole, in slot part_slot
    const int in_slots = slots + (one ? 1 : 0), parts = in_slots + (one ? 0 : c1 - c0 + 1);
    float top = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = warp; i0 < parts; i0 += kWarps * kBatch) {
        float w[kBatch], most = top;
        float4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * kWarps;
            w[k] = -INFINITY, v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < parts) {
                const int c = c0 + i - in_slots;
                const bool slot = i < in_slots;
                const int64_t at = slot ? i * total_rows + flat
                                        : ((int64_t)c * 2 + (c == c0 && place.first_is_last)) * piece_rows<T>(a.group) + tile_row;
                w[k] = (slot ? a.part_lse : a.piece_lse)[at];
                if (lane < D / 4)
                    v[k] = *reinterpret_cast<const float4*>((slot ? a.part_o : a.piece_o) + at * D + lane * 4);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) most = fmaxf(most, w[k]);
        const float ref = most == -INFINITY ? 0.f : most, keep = ex2(top - ref);
        top = most;
        sum *= keep;
        acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float f = ex2(w[k] - ref);
            sum += f;
            acc.x = fmaf(f, v[k].x, acc.x), acc.y = fmaf(f, v[k].y, acc.y);
            acc.z = fmaf(f, v[k].z, acc.z), acc.w = fmaf(f, v[k].w, acc.w);
        }
    }
    if (lane < D / 4) rows[warp][lane] = acc;
    if (lane == 0) tops[warp] = top, sums[warp] = sum;
    __syncthreads();
    top = tops[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, tops[w]);
    const float ref = top == -INFINITY ? 0.f : top;
    float v = 0.f;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(tops[w] - ref);
        sum = fmaf(f, sums[w], sum);
        if (tid < D) v = fmaf(f, reinterpret_cast<const float*>(rows[w])[tid], v);
    }
    const float inv = sum > 0.f ? 1.f / sum : sum;                 // no key: 0; NaN stays
    if (tid < D) static_cast<T*>(a.o)[(int64_t)row * a.o_stride + (int64_t)head * D + tid] = from_f32<T>(v * inv);
    if (tid == 0 && a.lse) a.lse[flat] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * kLn2;
}

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, int slots, bool shares, cudaStream_t s) {
    const int64_t rows = (int64_t)a.n_rows * a.hq;
    if (rows == 0) return cudaSuccess;
    const int per_seq = shares ? a.hkv * row_tiles<T>(a.group) : 0;
    // few rows may have many pieces each (one sequence: 32 rows of 152), many rows few
    if (rows <= 2 * 152)
        return launch_pdl(attn_join_kernel<T, D, 512>, dim3((unsigned)rows), dim3(512), 0, s, a, slots, per_seq);
    return launch_pdl(attn_join_kernel<T, D, 128>, dim3((unsigned)rows), dim3(128), 0, s, a, slots, per_seq);
}

}  // namespace

cudaError_t launch_attn_join(DType dt, int d, const AttnArgs& a, int slots, bool shares, cudaStream_t s) {
    if (dt == DType::F32) return d == 64 ? launch<float, 64>(a, slots, shares, s) : launch<float, 128>(a, slots, shares, s);
    return d == 64 ? launch<__nv_bfloat16, 64>(a, slots, shares, s) : launch<__nv_bfloat16, 128>(a, slots, shares, s);
}

}  // namespace colibri
