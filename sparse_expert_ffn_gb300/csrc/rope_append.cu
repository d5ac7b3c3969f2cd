// Rows of a q/k/v projection made ready for attention, in one pass: RMSNorm of
// every query and key head, rotation to the row's position, keys and values
// placed in the pages of a cache (or key rows of a tensor).
//
// Mathematics, per head x of a row at position t:
//   y = x / sqrt(mean(x^2) + eps) * w
//   (a, b) -> mscale (a cos t f_i - b sin t f_i, b cos t f_i + a sin t f_i)
// for the pairs (a, b) of y; float32, rounded once at the end.
//
// The angle: f_i / 2 pi, formed in double, as a 64-bit fraction of a turn; t times
// it, wrapped by the integer product itself, of which the top 32 bits are taken:
// off by at most 2^-32 turn and t (f_i 2^-55 + 2^-64) turns (the double product and
// its constant, and the fraction's end).  That is 2^-32 turn at positions that
// contexts have and 2^-24 at 2^31, where a float32 product would be off by 2^-24 of
// t f_i radians.  sin and cos of it are good to float32 rounding.  One set of
// angles serves every head of a row.
//
// Bound by HBM (each element is read once and written once), and close to it by
// instruction issue, so the work per element is kept small: a head is held by
// head_dim / 16 lanes, each with the first elements of eight pairs and their
// second ones, so that the rotation needs no exchange; the norm is a butterfly
// over those lanes; and a lane group takes several heads of one row, whose
// cosines and sines, times the norm weights, stay in registers.
#include <cuda_runtime.h>

#include "kernels.h"
#include "rope_common.cuh"

namespace colibri {
namespace {

constexpr int kThreads = 256;

// heads of a lane group in flight (64 bytes per lane)
template <typename T> constexpr int kBatch = sizeof(T) == 2 ? 2 : 1;
// float32: the first key and value heads are loaded during the kind before them
// (1852 rows of 48 heads 17.3 -> 15.5 us).  For bf16 the registers that this takes
// cost more (15373 rows 71 -> 78 us); its heads are fetched into L2 two batches
// ahead, which takes none (71 -> 64 us; all of a row at once: 71).
template <typename T> constexpr bool kAhead = sizeof(T) == 4;
template <typename T> using Vecs = Vec8<T>[kBatch<T>][2];

// A CTA takes kGroups / per_row rows, `per_row` lane groups each (a power of two);
// group `sub` of a row takes heads sub, sub + step, ... of q's, of k's and of v's
// (step: per_row times the CTAs that share the row).
template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const __grid_constant__ AppendArgs a, int per_row) {
    constexpr int kLanes = D / 16;                 // lanes of a head
    constexpr int kGroups = kThreads / kLanes;
    __shared__ float2 turn[2 * kThreads];          // rows x pairs: mscale * (cos, sin)
    __shared__ int place[16][2];
    __shared__ uint64_t unit[64];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid % kLanes, grp = tid / kLanes;
    const int rows = kGroups / per_row, r = grp / per_row;
    const int64_t row0 = (int64_t)blockIdx.x * rows, row = row0 + r;
    const int sub = grp % per_row + per_row * blockIdx.y, step = per_row * gridDim.y;
    const int pairs = a.freq ? a.rot_dim >> 1 : 0;
    // this lane's elements.  Half layout: the first and second elements of eight
    // pairs, then the elements that are not rotated; interleaved: sixteen neighbours.
    int c0 = 16 * lane, c1 = 16 * lane + 8;
    const bool turns = 16 * lane < 2 * pairs;
    if (!kInterleaved && turns) c0 = 8 * lane, c1 = pairs + 8 * lane;

    // the first heads are loaded before the row's place and angles are known
    const T* q = static_cast<const T*>(a.q) + row * a.q_stride;
    Vecs<T> x, ahead;
    Vecs<T>& y = *(kAhead<T> ? &ahead : &x);
    const auto load = [&](Vecs<T>& x, const T* p, int h, int heads) {
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c)
            if (h + c * step < heads) {
                x[c][0].load(p + (int64_t)(h + c * step) * D + c0);
                x[c][1].load(p + (int64_t)(h + c * step) * D + c1);
            }
    };
    // a batch fetched into L2 ahead of its load
    const auto touch = [&](const T* p, int h, int heads) {
        if (kAhead<T>) return;
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c)
            if (h + c * step < heads) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (int64_t)(h + c * step) * D + c0));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p + (int64_t)(h + c * step) * D + c1));
            }
    };
    if (row < a.n_rows) load(x, q, sub, a.hq);
    if (row < a.n_rows) touch(q, sub + kBatch<T> * step, a.hq);
    if (tid >= kThreads - 64 && tid - (kThreads - 64) < pairs) unit[tid - (kThreads - 64)] = pair_unit(a, tid - (kThreads - 64));
    for (int w = tid >> 5; w < rows; w += kThreads / 32) {
        int seq = -1, pos = 0;
        if (row0 + w < a.n_rows) row_place(a, (int)(row0 + w), &seq, &pos);
        if ((tid & 31) == 0) place[w][0] = seq, place[w][1] = pos;
    }
    __syncthreads();
    for (int e = tid; e < rows * pairs; e += kThreads) {
        turn[e] = row_turn(a, row0 + e / pairs, place[e / pairs][1], e % pairs, unit[e % pairs]);
    }
    __syncthreads();
    const int seq = place[r][0], pos = place[r][1];
    if (seq < 0) return;

    // the row's place in the cache
    int64_t at = -1;
    if (a.v_out) {
        if (pos >= 0 && (pos >> a.page_shift) < a.table_stride) {
            const int id = __ldg(a.table + (int64_t)seq * a.table_stride + (pos >> a.page_shift));
            if ((unsigned)id < (unsigned)a.num_pages)
                at = (int64_t)id * a.page_stride + (int64_t)(pos & ((1 << a.page_shift) - 1)) * a.row_stride;
        }
    } else {
        at = row * a.row_stride;
    }
    Heads<T, D, kInterleaved> hd;
    hd.prepare(static_cast<const T*>(a.q_norm), a.eps, turn + r * pairs, lane, turns, c0, c1);
    T* q_out = static_cast<T*>(a.q_out) + row * a.q_out_stride;
    const T* k = static_cast<const T*>(a.k) + row * a.k_stride;
    if (kAhead<T> && at >= 0) load(y, k, sub, a.hkv);
    for (int h = sub; h < a.hq; h += kBatch<T> * step) {
        if (h != sub) load(x, q, h, a.hq);
        if (h + 2 * kBatch<T> * step < a.hq) touch(q, h + 2 * kBatch<T> * step, a.hq);
        else if (h + kBatch<T> * step < a.hq) touch(k, sub, a.hkv);
        else if (a.v_out) touch(static_cast<const T*>(a.v) + row * a.v_stride, sub, a.hkv);
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c) {
            if (h + c * step >= a.hq) break;
            hd.apply(x[c]);
            x[c][0].store(q_out + (int64_t)(h + c * step) * D + c0);
            x[c][1].store(q_out + (int64_t)(h + c * step) * D + c1);
        }
    }
    if (at < 0) return;
    const T* v = static_cast<const T*>(a.v) + row * a.v_stride;
    if (kAhead<T> && a.v_out) load(x, v, sub, a.hkv);
    T* k_out = static_cast<T*>(a.k_out) + at;
    if (sub < a.hkv) hd.prepare(static_cast<const T*>(a.k_norm), a.eps, turn + r * pairs, lane, turns, c0, c1);
    for (int h = sub; h < a.hkv; h += kBatch<T> * step) {
        if (!kAhead<T> || h != sub) load(y, k, h, a.hkv);
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c) {
            if (h + c * step >= a.hkv) break;
            hd.apply(y[c]);
            y[c][0].store(k_out + (int64_t)(h + c * step) * a.head_stride + c0);
            y[c][1].store(k_out + (int64_t)(h + c * step) * a.head_stride + c1);
        }
    }
    if (!a.v_out) return;
    T* v_out = static_cast<T*>(a.v_out) + at;
    for (int h = sub; h < a.hkv; h += kBatch<T> * step) {
        if (!kAhead<T> || h != sub) load(x, v, h, a.hkv);
#pragma unroll
        for (int c = 0; c < kBatch<T>; ++c) {
            if (h + c * step >= a.hkv) break;
            x[c][0].store(v_out + (int64_t)(h + c * step) * a.head_stride + c0);
            x[c][1].store(v_out + (int64_t)(h + c * step) * a.head_stride + c1);
        }
    }
}

template <typename T, int D, bool kInterleaved>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
    constexpr int kGroups = kThreads / (D / 16);
    auto kern = append_kernel<T, D, kInterleaved>;
    // four groups per row while that gives three CTAs per SM; fewer rows are
    // spread over more groups, and a few over as many CTAs as give every group
    // one head (they are bound by latency)
    int per_row = 4;
    while (per_row < kGroups && (int64_t)a.n_rows * per_row < (int64_t)3 * 152 * kGroups) per_row *= 2;
    const int rows = kGroups / per_row;
    const int slices = rows == 1 && a.n_rows < 3 * 152 ? (a.hq + kGroups - 1) / kGroups : 1;
    return launch_pdl(kern, dim3((unsigned)(((int64_t)a.n_rows + rows - 1) / rows), slices), dim3(kThreads), 0, s, a,
                      per_row);
}

}  // namespace

cudaError_t launch_append(DType dt, int d, const AppendArgs& a, cudaStream_t s) {
    if (a.n_rows <= 0) return cudaSuccess;
    const bool il = a.freq && a.interleaved;
    if (dt == DType::F32)
        return d == 64 ? (il ? launch<float, 64, true>(a, s) : launch<float, 64, false>(a, s))
                       : (il ? launch<float, 128, true>(a, s) : launch<float, 128, false>(a, s));
    return d == 64 ? (il ? launch<__nv_bfloat16, 64, true>(a, s) : launch<__nv_bfloat16, 64, false>(a, s))
                   : (il ? launch<__nv_bfloat16, 128, true>(a, s) : launch<__nv_bfloat16, 128, false>(a, s));
}

}  // namespace colibri
