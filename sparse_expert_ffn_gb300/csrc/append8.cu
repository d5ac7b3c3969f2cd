// Rows of a q/k/v projection written to a cache of 8-bit codes with a scale for
// each block of tokens and key head, and the values of such pages in bf16.
//
// Mathematics: rows are normalised and rotated as in rope_append.cu, in float32.
// Of the elements that a call brings to a block of tokens of one head let `most`
// be the largest magnitude.  The block's scale s stays as it is where it had rows
// before and most <= largest code * s; otherwise it becomes the smallest power of
// two that `most` fits under, and the codes of the rows before, if any, are
// rounded again: code' = round(code * s_old / s).  New codes are round(y * (1 / s)).
// Powers of two, because then y * (1 / s) is exact and so is code * s_old / s but
// for e4m3's subnormal numbers and whole numbers that lose a bit: every value is
// rounded once, not once per token that the block grows by.
//
// A CTA takes the rows of one block of tokens of a sequence and a slice of the
// heads, so the scale needs nothing from another CTA.  A block's keys are read
// twice, for `most` and for the codes (the second time from the caches), rather
// than held: blocks of 64 tokens do not fit the registers.  Bound by HBM in the end
// (2 bytes of each element read, 2 of q and 1 of k and v written), but short of it: 15373
// rows of 32 / 8 heads of 128 take 97 us, where their bytes take 51, waiting on loads and
// on the chain length -> place -> angle -> head -> scale -> code of each CTA, four barriers
// long.  Heads are cut into slices so that CTAs are many and short (one slice 137 us with
// the pages' values read back, two 117, four 118, eight 141, which form each row's angles
// eight times).  One decode step of 32 sequences takes 8 us of the GPU, that chain.
#include <cuda_runtime.h>

#include <algorithm>

#include "codes.cuh"
#include "kernels.h"
#include "rope_common.cuh"

namespace colibri {
namespace {

constexpr int kThreads = 256;
constexpr int kSliceHeads = 32;               // key heads of a CTA at most

using BF = __nv_bfloat16;

// The rows of a CTA: positions lo .. lo + rows - 1 of sequence seq, rows row0 ..
struct Span {
    int seq, lo, rows, row0;
};

// Block of tokens number `item` over all sequences; called by a whole warp.
__device__ __forceinline__ Span find_span(const AppendArgs& a, int item) {
    const int lane = threadIdx.x & 31, shift = a.block_shift;
    Span s = {-1, 0, 0, 0};
    int64_t done = 0;
    for (int base = 0; base < a.n_seqs; base += 32) {
        const int b = base + lane;
        int r0 = 0, n = 0, first = 0, mine = 0;
        if (b < a.n_seqs) {
            r0 = a.seq_start ? min(max(__ldg(a.seq_start + b), 0), a.n_rows) : b;
            n = a.seq_start ? min(max(__ldg(a.seq_start + b + 1), r0), a.n_rows) - r0 : 1;
            first = max(__ldg(a.kv_len + b), 0) - n;
            if (n > 0) mine = ((first + n - 1) >> shift) - (first >> shift) + 1;
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
            const int into = (int)(item - done) - __shfl_sync(0xffffffffu, upto - mine, src);
            first = __shfl_sync(0xffffffffu, first, src), n = __shfl_sync(0xffffffffu, n, src);
            r0 = __shfl_sync(0xffffffffu, r0, src);
            const int start = ((first >> shift) + into) << shift;
            s.seq = base + src;
            s.lo = max(start, first);
            s.rows = (int)(min((int64_t)start + (1 << shift), (int64_t)first + n) - s.lo);
            s.row0 = r0 + (s.lo - first);
            return s;
        }
        done += __shfl_sync(0xffffffffu, upto, 31);
    }
    return s;
}

template <typename Code, int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3) append8_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kLanes = D / 16;                 // lanes of a head
    constexpr int kGroups = kThreads / kLanes;
    extern __shared__ float2 turn[];               // rows x pairs: mscale * (cos, sin)
    __shared__ Span span;
    __shared__ uint32_t most[2][kSliceHeads];
    __shared__ float2 fit[2][kSliceHeads];         // 1 / scale, old scale / scale
    __shared__ uint64_t unit[64];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid % kLanes, grp = tid / kLanes;
    const int pairs = a.freq ? a.rot_dim >> 1 : 0;
    if (tid < 32) {
        const Span s = find_span(a, blockIdx.x);
        if (tid == 0) span = s;
    } else if (tid >= kThreads - 64 && tid - (kThreads - 64) < pairs) {
        unit[tid - (kThreads - 64)] = pair_unit(a, tid - (kThreads - 64));
    }
    for (int i = tid; i < 2 * kSliceHeads; i += kThreads) most[i / kSliceHeads][i % kSliceHeads] = 0;
    __syncthreads();
    const Span sp = span;
    if (sp.seq < 0) return;
    // heads y, y + slices, ...; lane groups take units (query heads, then keys, then
    // values) of one row in turn, `per` groups a row (a power of two)
    const int slices = gridDim.y, y0 = blockIdx.y;
    const int nq = (a.hq - y0 + slices - 1) / slices;
    int per = 1;
    while (2 * per * sp.rows <= kGroups) per *= 2;
    const int sub = grp % per;
    const auto first_of = [&](int base) { return (sub - base) & (per - 1); };   // of the units from base on
    // rows' heads are fetched into L2 ahead of their loads
    const auto touch = [&](const BF* row, int h, int heads) {
        if (h < heads) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + (int64_t)(y0 + h * slices) * D + 16 * lane));
    };
    if (grp / per < sp.rows) {
        const int64_t row = sp.row0 + grp / per;
#pragma unroll
        for (int c = 0; c < 4; ++c) touch(static_cast<const BF*>(a.q) + row * a.q_stride, sub + c * per, nq);
    }
    for (int e = tid; e < sp.rows * pairs; e += kThreads)
        turn[e] = row_turn<true>(a, sp.row0 + e / pairs, sp.lo + e / pairs, e % pairs, unit[e % pairs]);
    // the block's place
    int page = -1;
    if (sp.lo >= 0 && (sp.lo >> a.page_shift) < a.table_stride) {
        const int id = __ldg(a.table + (int64_t)sp.seq * a.table_stride + (sp.lo >> a.page_shift));
        if ((unsigned)id < (unsigned)a.num_pages) page = id;
    }
    __syncthreads();

    const int nk = page >= 0 ? (a.hkv - y0 + slices - 1) / slices : 0;
    // this lane's elements (rope_append.cu)
    int c0 = 16 * lane, c1 = 16 * lane + 8;
    const bool turns = 16 * lane < 2 * pairs;
    if (!kInterleaved && turns) c0 = 8 * lane, c1 = pairs + 8 * lane;
    const uint32_t mine = (((1ull << kLanes) - 1) << (tid & 31 & ~(kLanes - 1)));
    const auto note = [&](int kind, int h, float top) {
        // (as whole numbers: NaN above infinity above all others)
        uint32_t bits = __float_as_uint(top);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) bits = max(bits, __shfl_xor_sync(mine, bits, o));
        if (lane == 0) atomicMax(&most[kind][h], bits);
    };
    const auto abs_top = [](const float (&v)[8], float top) {
        // (a NaN has to come through: fmaxf would drop it)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = __uint_as_float(max(__float_as_uint(top), __float_as_uint(fabsf(v[i]))));
        return top;
    };
    Heads<BF, D, kInterleaved> hd;
    for (int r = grp / per; r < sp.rows; r += kGroups / per) {
        const int64_t row = sp.row0 + r;
        const BF* q = static_cast<const BF*>(a.q) + row * a.q_stride;
        const BF* k = static_cast<const BF*>(a.k) + row * a.k_stride;
        const BF* v = static_cast<const BF*>(a.v) + row * a.v_stride;
        BF* q_out = static_cast<BF*>(a.q_out) + row * a.q_out_stride;
        hd.prepare(static_cast<const BF*>(a.q_norm), a.eps, turn + r * pairs, lane, turns, c0, c1);
        for (int h = sub; h < nq; h += 2 * per) {
            Vec8<BF> x[2][2];
#pragma unroll
            for (int c = 4; c < 6; ++c) touch(q, h + c * per, nq);
            // (keys and values behind the last query heads)
            if (h + 4 * per >= nq) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    touch(k, first_of(nq) + (h / per + c) % 8 * per, nk);
                    touch(v, first_of(nq + nk) + (h / per + c) % 8 * per, nk);
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (h + c * per < nq) {
                    const int at = (y0 + (h + c * per) * slices) * D;
                    x[c][0].load(q + at + c0), x[c][1].load(q + at + c1);
                }
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (h + c * per < nq) {
                    const int at = (y0 + (h + c * per) * slices) * D;
                    hd.apply(x[c]);
                    x[c][0].store(q_out + at + c0), x[c][1].store(q_out + at + c1);
                }
        }
        if (nk == 0) continue;
        hd.template prepare<true>(static_cast<const BF*>(a.k_norm), a.eps, turn + r * pairs, lane, turns, c0, c1);
        for (int h = first_of(nq); h < nk; h += per) {
            Vec8<BF> x[2];
            float y[2][8];
            const int at = (y0 + h * slices) * D;
            x[0].load(k + at + c0), x[1].load(k + at + c1);
            hd.template turned<true>(x, y);
            note(0, h, abs_top(y[1], abs_top(y[0], 0.f)));
        }
        for (int h = first_of(nq + nk); h < nk; h += per) {
            Vec8<BF> x[2];
            float y[2][8];
            const int at = (y0 + h * slices) * D;
            x[0].load(v + at + c0), x[1].load(v + at + c1);
            x[0].get(y[0]), x[1].get(y[1]);
            note(1, h, abs_top(y[1], abs_top(y[0], 0.f)));
        }
    }
    if (nk == 0) return;
    __syncthreads();
    const int block = 1 << a.block_shift, kept = sp.lo & (block - 1);
    const int in_page = sp.lo & ((1 << a.page_shift) - 1);
    for (int u = tid; u < 2 * nk; u += kThreads) {
        const int kind = u >= nk, h = u - kind * nk;
        float* at = (kind ? a.v_scale : a.k_scale) +
                    (((int64_t)page * a.hkv + y0 + h * slices) << (a.page_shift - a.block_shift)) + (in_page >> a.block_shift);
        const uint32_t bits = most[kind][h];
        float old = 0.f, s = fitting_scale<Code>(bits);
        if (kept > 0) {
            old = *at;
            if (bits < 0x7f800000u && (old != old || __uint_as_float(bits) <= Code::kMost * old)) s = old;
        }
        *at = s;
        fit[kind][h] = make_float2(1.f / s, kept > 0 ? old / s : 1.f);
    }
    __syncthreads();
    const int64_t base = (int64_t)page * a.page_stride;
    for (int r = grp / per; r < sp.rows; r += kGroups / per) {
        const int64_t row = sp.row0 + r, place = base + (int64_t)(in_page + r) * a.row_stride;
        const BF* k = static_cast<const BF*>(a.k) + row * a.k_stride;
        const BF* v = static_cast<const BF*>(a.v) + row * a.v_stride;
        const auto put = [&](void* to, int kind, int h, float (&y)[2][8]) {
            const float inv = fit[kind][h].x;
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i / 8][i % 8] *= inv;
            uint8_t* p = static_cast<uint8_t*>(to) + place + (int64_t)(y0 + h * slices) * a.head_stride;
            *reinterpret_cast<uint2*>(p + c0) = make_uint2(Code::encode4(y[0]), Code::encode4(y[0] + 4));
            *reinterpret_cast<uint2*>(p + c1) = make_uint2(Code::encode4(y[1]), Code::encode4(y[1] + 4));
        };
        if (sp.rows > kGroups)                                     // (else the row's are there from above)
            hd.template prepare<true>(static_cast<const BF*>(a.k_norm), a.eps, turn + r * pairs, lane, turns, c0, c1);
        for (int h = first_of(nq); h < nk; h += per) {
            Vec8<BF> x[2];
            float y[2][8];
            const int at = (y0 + h * slices) * D;
            x[0].load(k + at + c0), x[1].load(k + at + c1);
            hd.template turned<true>(x, y);
            put(a.k_out, 0, h, y);
        }
        for (int h = first_of(nq + nk); h < nk; h += per) {
            Vec8<BF> x[2];
            float y[2][8];
            const int at = (y0 + h * slices) * D;
            x[0].load(v + at + c0), x[1].load(v + at + c1);
            x[0].get(y[0]), x[1].get(y[1]);
            put(a.v_out, 1, h, y);
        }
    }
    // the rows before them, where the scale has grown
    for (int u = grp; u < 2 * nk; u += kGroups) {
        const int kind = u >= nk, h = u - kind * nk;
        const float ratio = fit[kind][h].y;
        if (ratio == 1.f) continue;
        uint8_t* p = static_cast<uint8_t*>(kind ? a.v_out : a.k_out) + base + (int64_t)(y0 + h * slices) * a.head_stride +
                     (int64_t)(in_page - kept) * a.row_stride + 16 * lane;
        for (int r = 0; r < kept; ++r, p += a.row_stride) {
            const uint4 c = *reinterpret_cast<const uint4*>(p);
            const uint32_t in[4] = {c.x, c.y, c.z, c.w};
            uint32_t out[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[4];
                Code::decode4(in[i], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] *= ratio;
                out[i] = Code::encode4(f);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
}

template <typename Code, int D, bool kInterleaved>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
    auto kern = append8_kernel<Code, D, kInterleaved>;
    const int block = 1 << a.block_shift;
    // a sequence of n rows touches at most (n - 2) / block + 2 blocks of tokens, and n
    const int64_t items = std::min<int64_t>(a.n_rows, a.n_rows / block + 2 * (int64_t)a.n_seqs);
    int slices = (a.hkv + kSliceHeads - 1) / kSliceHeads;
    // a few rows are spread over the SMs; of many, enough CTAs that the last ones to start
    // are a small part (three run on an SM)
    while (items * slices < (items < 152 ? 152 : 4 * 3 * 152) && 2 * slices <= a.hkv) slices *= 2;
    const int bytes = a.freq ? std::min(block, a.n_rows) * (a.rot_dim / 2) * (int)sizeof(float2) : 0;
    return launch_pdl(kern, dim3((unsigned)items, slices), dim3(kThreads), bytes, s, a);
}

// (16-byte boundaries are what is asked of the outputs)
__device__ __forceinline__ void store32(BF* to, const uint32_t (&w)[8]) {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// 16 codes of a row of k and of v per thread.
template <typename Code, int D>
__global__ void __launch_bounds__(256) values8_kernel(const __grid_constant__ ValuesArgs a) {
    constexpr int kChunks = D / 16;
    pdl_enter();
    const int chunk = threadIdx.x % kChunks, r = threadIdx.x / kChunks;
    const int per = 256 / kChunks;                                  // rows of a CTA's pass
    const int rows = a.page_size;
    const int64_t all = (int64_t)a.n_pages * a.hkv * rows;          // (page, head), below 2^31, times rows
    for (int64_t e = (int64_t)blockIdx.x * per + r; e < all; e += (int64_t)gridDim.x * per) {
        const int row = (int)(e & (rows - 1));
        const uint32_t piece = (uint32_t)(e >> a.page_shift), i = piece / (uint32_t)a.hkv;
        const int h = (int)(piece - i * (uint32_t)a.hkv), id = a.pages ? __ldg(a.pages + i) : (int)i;
        const bool there = (unsigned)id < (unsigned)a.num_pages;
        const int64_t to = ((int64_t)piece * rows + row) * D + 16 * chunk;
        const int64_t from = there ? (int64_t)id * a.page_stride + (int64_t)h * a.head_stride + (int64_t)row * a.row_stride + 16 * chunk : 0;
        const int64_t at = there ? (((int64_t)id * a.hkv + h) << (a.page_shift - a.block_shift)) + (row >> a.block_shift) : 0;
        uint4 c[2];
        float s[2];
        c[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.k) + from));
        c[1] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.v) + from));
        s[0] = __ldg(a.k_scale + at), s[1] = __ldg(a.v_scale + at);
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
            const uint32_t in[4] = {c[kind].x, c[kind].y, c[kind].z, c[kind].w};
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float f[4];
                Code::decode4(in[j], f);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * x] * s[kind], f[2 * x + 1] * s[kind]);
                    w[2 * j + x] = there ? *reinterpret_cast<const uint32_t*>(&p) : 0u;
                }
            }
            store32(static_cast<BF*>(kind ? a.v_out : a.k_out) + to, w);
        }
    }
}

template <typename Code, int D>
cudaError_t launch_values(const ValuesArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.n_pages * a.hkv * a.page_size, per = 256 / (D / 16);
    const int64_t ctas = std::min<int64_t>((rows + per - 1) / per, 152 * 8);
    return launch_pdl(values8_kernel<Code, D>, dim3((unsigned)ctas), dim3(256), 0, s, a);
}

}  // namespace

cudaError_t launch_append8(bool int8, int d, const AppendArgs& a, cudaStream_t s) {
    if (a.n_rows <= 0) return cudaSuccess;
    const auto pick = [&](auto code) {
        using C = decltype(code);
        if (a.freq && a.interleaved) return d == 64 ? launch<C, 64, true>(a, s) : launch<C, 128, true>(a, s);
        return d == 64 ? launch<C, 64, false>(a, s) : launch<C, 128, false>(a, s);
    };
    return int8 ? pick(I8{}) : pick(E4M3{});
}

cudaError_t launch_values8(bool int8, int d, const ValuesArgs& a, cudaStream_t s) {
    if (a.n_pages <= 0) return cudaSuccess;
    if (int8) return d == 64 ? launch_values<I8, 64>(a, s) : launch_values<I8, 128>(a, s);
    return d == 64 ? launch_values<E4M3, 64>(a, s) : launch_values<E4M3, 128>(a, s);
}

}  // namespace colibri
