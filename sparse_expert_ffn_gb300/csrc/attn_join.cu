// Joins the partial rows of key ranges: with w_i = 2^(log2-sum_i - largest),
//   o = sum_i w_i o_i / sum_i w_i,   ln-sum = ln2 (largest + log2 sum_i w_i)
// in a fixed order, so that results do not depend on timing.
//
// One CTA per (row, head).  Bound by latency: the log2-sums are read all at
// once, then every warp adds its own share of the rows with independent loads,
// and the shares are added at the end.  A range that held no key of the
// row has log2-sum -infinity, so weight 0, and left zeros.
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "kernels.h"

namespace colibri {
namespace {

constexpr int kMaxParts = kShares + 72;   // 64 + 1 slots and a piece per share at most

template <typename T, int D, int kThreads>
__global__ void __launch_bounds__(kThreads) attn_join_kernel(AttnArgs a, int slots, int shares_per_seq) {
    __shared__ float weight[kMaxParts];
    constexpr int kWarps = kThreads / 32;
    __shared__ float4 share[kWarps][D / 4];
    __shared__ int place[5];
    pdl_enter();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t total_rows = (int64_t)a.n_rows * a.hq, flat = blockIdx.x;
    const int row = (int)(flat / a.hq), head = (int)(flat % a.hq), g = head % a.group;
    const int ROWS = row_tile(a.group);
    if (warp == 0) {
        // live: the row belongs to a sequence; c0 .. c1: the shares that hold its keys
        int live = 1, c0 = 0, c1 = -1, first_is_last = 0;
        if (shares_per_seq) {
            int64_t total, first;
            count_steps<D>(a, shares_per_seq, row, &total, &first);
            const int units = seq_steps<D>(a, row);
            if (units > 0) {
                const int shares = share_count(total);
                first += (int64_t)((head / a.group) * row_tiles(a.group) + g / ROWS) * units;
                c0 = share_of(total, shares, first);
                c1 = share_of(total, shares, first + units - 1);
                first_is_last = share_begin(total, shares, c0) < first;
            }
            live = c0 != c1 || slots > 0;                          // (else written by the one share)
        } else if (a.mode == kAttnPrompt) {
            live = 0;
            for (int b = lane; b < a.n_seqs; b += 32)
                live |= row >= max(__ldg(a.seq_start + b), 0) && row < __ldg(a.seq_start + b + 1);
            live = __any_sync(0xffffffffu, live);
        }
        if (lane == 0) place[0] = live, place[1] = c0, place[2] = c1, place[3] = first_is_last;
    }
    __syncthreads();
    if (!place[0]) return;
    const int c0 = place[1], c1 = place[2];
    const bool one = shares_per_seq && c0 == c1;                   // whole, in slot part_slot
    const int in_slots = slots + (one ? 1 : 0), parts = min(in_slots + (one ? 0 : c1 - c0 + 1), kMaxParts);
    // part i: its index among the slots' or the pieces' rows
    const auto piece = [&](int i) {
        const int c = c0 + i - in_slots;
        return ((int64_t)c * 2 + (c == c0 && place[3])) * piece_rows(a.group) + g % ROWS;
    };
    float top = -INFINITY;
    bool bad = false;
    for (int i = tid; i < parts; i += kThreads) {
        const float v = i < in_slots ? a.part_lse[i * total_rows + flat] : a.piece_lse[piece(i)];
        weight[i] = v;
        top = fmaxf(top, v);
        bad |= isnan(v);
    }
    __shared__ float tops[kWarps], sums[kWarps];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) tops[warp] = top;
    // a NaN log2-sum (scores that are NaN, rows whose wait gave up) makes the row NaN
    if (__syncthreads_or(bad)) {
        top = __int_as_float(0x7fc00000);
    } else {
        top = tops[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, tops[w]);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    if (top != -INFINITY) {
#pragma unroll 8
        for (int i = warp; i < parts; i += kWarps) {
            const float w = ex2(weight[i] - top);
            sum += w;
            if (lane < D / 4) {
                const float* p = i < in_slots ? a.part_o + (i * total_rows + flat) * D : a.piece_o + piece(i) * D;
                const float4 v = *reinterpret_cast<const float4*>(p + lane * 4);
                acc.x = fmaf(w, v.x, acc.x), acc.y = fmaf(w, v.y, acc.y);
                acc.z = fmaf(w, v.z, acc.z), acc.w = fmaf(w, v.w, acc.w);
            }
        }
    }
    if (lane < D / 4) share[warp][lane] = acc;
    if (lane == 0) sums[warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sums[w];
    const float inv = sum > 0.f ? 1.f / sum : sum;                 // no key: 0; NaN stays
    if (tid < D) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += reinterpret_cast<const float*>(share[w])[tid];
        static_cast<T*>(a.o)[(int64_t)row * a.o_stride + (int64_t)head * D + tid] = from_f32<T>(v * inv);
    }
    if (tid == 0 && a.lse) a.lse[flat] = top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <typename T, int D>
cudaError_t launch(const AttnArgs& a, int slots, bool shares, cudaStream_t s) {
    const int64_t rows = (int64_t)a.n_rows * a.hq;
    if (rows == 0) return cudaSuccess;
    const int per_seq = shares ? a.hkv * row_tiles(a.group) : 0;
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
