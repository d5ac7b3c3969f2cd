// Attention of single rows over a paged cache (bf16): the decode step, and the
// sequences' own keys behind a shared prefix.
//
// Bound by HBM: every key and value is read once and meets only the rows of
// its head group, so the products are few and what counts is that all SMs
// stream all the time, whatever the lengths of the sequences are.
//
// Work is cut into units of kUnitKeys keys of one (sequence, key head, row
// tile), laid out one after another, and every CTA takes an equal share of the
// whole list: a CTA's share may end inside a sequence and begin inside another
// one.  A (sequence, head) that falls to one CTA is written directly; the
// pieces of one that is cut go to the workspace, at most two per CTA (its first
// and its last), and the join adds them in key order.  Nothing depends on the
// order in which CTAs run.
//
// Each of a CTA's 4 warps streams its own keys (2048 / d at a time, 8 KB of K
// and V) through its own ring of 3 stages with cp.async, so no warp waits for
// another until the end of a piece.  The rows of the group are the 16 rows of
// mma.sync m16n8k16 (2 tiles up to 32 rows): tensor-memory MMAs would pad them
// to 64 or 128 and spend most of the time of a 16-key step on that padding.
// Scores stay in registers and become the A operand of the product with V as
// they lie.  The running maximum and sum are f32 per row, P is rounded to bf16
// for the product (its operands share one 16-bit type).
#include <cuda_runtime.h>

#include "attn_common.cuh"
#include "kernels.h"

namespace colibri {
namespace {

constexpr int kWarps = 4;
constexpr int kDecThreads = 32 * kWarps;
constexpr int kStages = 3;
template <int D> constexpr int kStepKeys = 2048 / D;              // keys of a warp's step
static_assert(kUnitKeys<64> == kWarps * kStepKeys<64> && kUnitKeys<128> == kWarps * kStepKeys<128>, "a unit is a step of every warp");
constexpr int kStageBytes = 8192;                                 // K then V of one step
constexpr int kRingBytes = kStages * kStageBytes;
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool there) {
    const int n = there ? 16 : 0;                                  // 0: the 16 bytes become zeros
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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

// One warp's stream over the keys of a piece: which step is copied next.  The
// page ids of up to 32 page parts ahead lie one per lane.
template <int D>
struct Stream {
    static constexpr int kChunks = D / 8;                          // 16-byte chunks of a row
    static constexpr int kRowsPer = 32 / kChunks;                  // rows that a pass of the warp covers
    static constexpr int kPasses = kStepKeys<D> / kRowsPer;
    int b, lo, hi;             // sequence, keys of the piece
    int parts;                 // pages that a step touches
    int window;                // first step whose page parts the lanes hold
    int id;
    const __nv_bfloat16* k;    // this lane's chunk of row 0 of the head in page 0 (packed: key 0)
    const __nv_bfloat16* v;
    uint32_t dst;              // this lane's place in a stage, pass 0

    __device__ __forceinline__ void begin(const AttnArgs& a, int seq, int h, int first, int end) {
        const int lane = threadIdx.x & 31, chunk = lane % kChunks, row = lane / kChunks;
        b = seq, lo = first, hi = end;
        int64_t at = (int64_t)h * a.head_stride + chunk * 8;
        if (!a.table) at += (int64_t)b * a.row_stride;             // packed rows: the row's own key
        k = static_cast<const __nv_bfloat16*>(a.k) + at;
        v = static_cast<const __nv_bfloat16*>(a.v) + at;
        // (the chunk's swizzled place: the row's low bits of later passes are xored in copy())
        dst = row * (D * 2) + ((chunk ^ row) << 4);
        parts = a.page_size < kStepKeys<D> ? kStepKeys<D> / a.page_size : 1;
        if (a.table) fill(a, 0);
    }
    __device__ __forceinline__ int first_key(int step) const {
        return lo + (step * kWarps + (int)(threadIdx.x >> 5)) * kStepKeys<D>;
    }
    __device__ __forceinline__ void fill(const AttnArgs& a, int step) {
        const int lane = threadIdx.x & 31;
        window = step;
        const int key = first_key(step + lane / parts) + (lane % parts) * (kStepKeys<D> / parts);
        id = key < hi ? attn_page(a, b, key >> a.page_shift) : -1;
    }
    __device__ __forceinline__ void copy(const AttnArgs& a, int step, uint32_t stage) {
        const int lane = threadIdx.x & 31, key0 = first_key(step), row0 = lane / kChunks;
        if (a.table && step >= window + 32 / parts) fill(a, step);
        // rows of one pass lie kRowsPer apart: their swizzle differs by that in
        // the row's low three bits
        const auto place = [&](int i) {
            return stage + ((dst + i * kRowsPer * (D * 2)) ^ (((i * kRowsPer) & 7) << 4));
        };
        if (a.table && parts > 1) {
#pragma unroll
            for (int i = 0; i < kPasses; ++i) {
                const int row = i * kRowsPer + row0, key = key0 + row;
                const int page = __shfl_sync(0xffffffffu, id, (step - window) * parts + row / (kStepKeys<D> / parts));
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
        if (page_there && key0 + kStepKeys<D> <= hi) {
            const __nv_bfloat16 *kp = k + at, *vp = v + at;
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

template <int D, int MT>
__global__ void __launch_bounds__(kDecThreads, 2) attn_decode_kernel(AttnArgs a, int per_seq) {
    constexpr int KS = kStepKeys<D>, ROWS = 16 * MT, kAcc = D + 4;
    static_assert(ROWS * (kAcc + 2) * 4 <= kRingBytes, "a warp's rows fit its ring");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t place[4];
    pdl_enter();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = row_tiles(a.group);
    // this CTA's share u0 .. u1 - 1, and the sequence that u0 lies in
    if (warp == 0) {
        int64_t total, unused;
        count_units<D>(a, per_seq, 0, &total, &unused);
        int64_t u0 = 0, u1 = 0, before = 0;
        if (total > 0) {
            const int shares = share_count(total, gridDim.x);
            if ((int)blockIdx.x < shares) {
                u0 = share_begin(total, shares, blockIdx.x);
                u1 = share_begin(total, shares, blockIdx.x + 1);
            }
        }
        int seq = 0;
        if (u1 > u0) {
            for (int base = 0;; base += 32) {
                int64_t upto = base + lane < a.n_seqs ? (int64_t)seq_units<D>(a, base + lane) * per_seq : 0;
                const int64_t mine = upto;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += v;
                }
                const unsigned holds = __ballot_sync(0xffffffffu, u0 < before + upto);
                if (holds) {
                    const int src = __ffs(holds) - 1;
                    seq = base + src;
                    before += __shfl_sync(0xffffffffu, upto - mine, src);
                    break;
                }
                before += __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        if (lane == 0) place[0] = u0, place[1] = u1, place[2] = seq, place[3] = u0 - before;
    }
    __syncthreads();
    const int64_t u1 = place[1];
    int64_t u = place[0];
    if (u >= u1) return;
    int b = (int)place[2];
    int64_t in_seq = place[3];                                     // units of sequence b before u
    const int64_t begin = u;
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * kRingBytes;
    float* own = reinterpret_cast<float*>(smem + warp * kRingBytes);

    while (u < u1) {
        int units = 0;
        while (b < a.n_seqs && (units = seq_units<D>(a, b)) == 0) ++b;
        if (units == 0) return;                                    // (not reached: u < u1)
        const AttnSeq sq = attn_seq(a, b);
        const int item = (int)(in_seq / units), step0 = (int)(in_seq % units);
        const int h = item / tiles, r0 = (item % tiles) * ROWS;
        const int count = (int)min((int64_t)(units - step0), u1 - u);   // units of this piece
        Stream<D> st;
        st.begin(a, b, h, sq.kv0 + step0 * kUnitKeys<D>,
                 min(sq.kv, sq.kv0 + (step0 + count) * kUnitKeys<D>));
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            if (s < count) st.copy(a, s, ring + s * kStageBytes);
            cp_commit();
        }
        // the group's rows as A operands: row lane / 4 (+ 8), columns 2 (lane % 4) (+ 8)
        uint32_t qf[MT][D / 16][4];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int g = r0 + 16 * t + 8 * half + (lane >> 2);
                const uint32_t* q = reinterpret_cast<const uint32_t*>(
                    static_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.q_stride + (int64_t)(h * a.group + g) * D);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    qf[t][x][half] = g < a.group ? __ldg(q + x * 8 + (lane & 3)) : 0u;
                    qf[t][x][half + 2] = g < a.group ? __ldg(q + x * 8 + 4 + (lane & 3)) : 0u;
                }
            }
        float o[MT][D / 8][4], m[MT][2], l[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int x = 0; x < D / 8; ++x) o[t][x][0] = o[t][x][1] = o[t][x][2] = o[t][x][3] = 0.f;
        }
        for (int step = 0; step < count; ++step) {
            cp_wait<kStages - 2>();
            __syncwarp();
            // (the stage that this copy fills was read in the previous step)
            if (step + kStages - 1 < count)
                st.copy(a, step + kStages - 1, ring + (step + kStages - 1) % kStages * kStageBytes);
            cp_commit();
            const uint32_t ks = ring + step % kStages * kStageBytes, vs = ks + kStageBytes / 2;
            float s[MT][KS / 8][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int n = 0; n < KS / 8; ++n) s[t][n][0] = s[t][n][1] = s[t][n][2] = s[t][n][3] = 0.f;
#pragma unroll
            for (int n = 0; n < KS / 16; ++n)
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    uint32_t kf[4];
                    const int key = n * 16 + ((lane >> 4) << 3) + (lane & 7), chunk = 2 * x + ((lane >> 3) & 1);
                    ldm4(ks + key * (D * 2) + ((chunk ^ (key & 7)) << 4), kf);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        mma16816(s[t][2 * n], qf[t][x], kf[0], kf[1]);
                        mma16816(s[t][2 * n + 1], qf[t][x], kf[2], kf[3]);
                    }
                }
            const int left = st.hi - st.first_key(step);           // keys of this step
            uint32_t pf[MT][KS / 16][4];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                float top[2] = {-INFINITY, -INFINITY};
                if (left < KS) {
#pragma unroll
                    for (int n = 0; n < KS / 8; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n * 8 + 2 * (lane & 3) + (e & 1) >= left) s[t][n][e] = -INFINITY;
                }
#pragma unroll
                for (int n = 0; n < KS / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[t][n][e]);
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                    top[r] *= a.scale_log2;
                }
                // the reference maximum moves only when a row's has grown by
                // more than 2^8 (weights below 2^8 are held as exactly)
                if (__any_sync(0xffffffffu, top[0] > m[t][0] + 8.f || top[1] > m[t][1] + 8.f)) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const bool grow = top[r] > m[t][r];
                        const float keep = grow ? ex2(m[t][r] - top[r]) : 1.f;
                        if (grow) m[t][r] = top[r];
                        l[t][r] *= keep;
#pragma unroll
                        for (int x = 0; x < D / 8; ++x) o[t][x][2 * r] *= keep, o[t][x][2 * r + 1] *= keep;
                    }
                }
                const float ref[2] = {m[t][0] == -INFINITY ? 0.f : m[t][0], m[t][1] == -INFINITY ? 0.f : m[t][1]};
#pragma unroll
                for (int n = 0; n < KS / 8; ++n) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[t][n][e] = ex2(fmaf(s[t][n][e], a.scale_log2, -ref[e >> 1]));
                        l[t][e >> 1] += s[t][n][e];
                    }
                    pf[t][n / 2][(n & 1) * 2] = bf16x2(s[t][n][0], s[t][n][1]);
                    pf[t][n / 2][(n & 1) * 2 + 1] = bf16x2(s[t][n][2], s[t][n][3]);
                }
            }
#pragma unroll
            for (int n = 0; n < KS / 16; ++n)
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    uint32_t vf[4];
                    const int key = n * 16 + (((lane >> 3) & 1) << 3) + (lane & 7), chunk = 2 * x + (lane >> 4);
                    ldm4t(vs + key * (D * 2) + ((chunk ^ (key & 7)) << 4), vf);
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        mma16816(o[t][2 * x], pf[t][n], vf[0], vf[1]);
                        mma16816(o[t][2 * x + 1], pf[t][n], vf[2], vf[3]);
                    }
                }
        }
        cp_wait<0>();
        __syncwarp();
        // the warps' rows, added in warp order
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 1);
                l[t][r] += __shfl_xor_sync(0xffffffffu, l[t][r], 2);
                const int row = 16 * t + 8 * r + (lane >> 2);
#pragma unroll
                for (int x = 0; x < D / 8; ++x)
                    *reinterpret_cast<float2*>(own + row * kAcc + x * 8 + 2 * (lane & 3)) =
                        make_float2(o[t][x][2 * r], o[t][x][2 * r + 1]);
                if ((lane & 3) == 0) own[ROWS * kAcc + row] = m[t][r], own[ROWS * (kAcc + 1) + row] = l[t][r];
            }
        __syncthreads();
        const bool whole = step0 == 0 && count == units;           // the (sequence, head) is this CTA's alone
        for (int e = threadIdx.x; e < ROWS * (D / 4); e += kDecThreads) {
            const int row = e / (D / 4), c = (e % (D / 4)) * 4, g = r0 + row;
            if (g >= a.group) continue;
            float top = -INFINITY, sum = 0.f;
            const float* all = reinterpret_cast<const float*>(smem);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, all[w * (kRingBytes / 4) + ROWS * kAcc + row]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float* p = all + w * (kRingBytes / 4);
                const float mw = p[ROWS * kAcc + row], f = mw == -INFINITY ? 0.f : ex2(mw - top);
                const float4 v = *reinterpret_cast<const float4*>(p + row * kAcc + c);
                sum += f * p[ROWS * (kAcc + 1) + row];
                acc.x = fmaf(f, v.x, acc.x), acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z), acc.w = fmaf(f, v.w, acc.w);
            }
            const float inv = sum > 0.f ? 1.f / sum : sum;
            acc.x *= inv, acc.y *= inv, acc.z *= inv, acc.w *= inv;
            const float lse2 = sum == 0.f ? -INFINITY : top + log2f(sum);
            const int head = h * a.group + g;
            const int64_t flat = (int64_t)b * a.hq + head;
            if (whole && !a.part_o) {
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o) + (int64_t)b * a.o_stride + (int64_t)head * D + c;
                *reinterpret_cast<uint2*>(out) = make_uint2(bf16x2(acc.x, acc.y), bf16x2(acc.z, acc.w));
                if (c == 0 && a.lse) a.lse[flat] = lse2 * kLn2;
            } else if (whole) {
                const int64_t at = (int64_t)a.part_slot * a.n_rows * a.hq + flat;
                *reinterpret_cast<float4*>(a.part_o + at * D + c) = acc;
                if (c == 0) a.part_lse[at] = lse2;
            } else {
                const int64_t at = ((int64_t)blockIdx.x * 2 + (u == begin ? 0 : 1)) * ROWS + row;
                *reinterpret_cast<float4*>(a.piece_o + at * D + c) = acc;
                if (c == 0) a.piece_lse[at] = lse2;
            }
        }
        __syncthreads();
        u += count;
        in_seq += count;
        if (in_seq == (int64_t)units * per_seq) ++b, in_seq = 0;
    }
}

template <int D, int MT>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    auto kern = attn_decode_kernel<D, MT>;
    const int bytes = kWarps * kRingBytes, per_seq = a.hkv * row_tiles(a.group);
    cudaError_t e = smem_attr((const void*)kern, bytes);
    return e != cudaSuccess ? e : launch_pdl(kern, dim3(kShareCtas), dim3(kDecThreads), bytes, s, a, per_seq);
}

}  // namespace

size_t attn_decode_pieces(int group) { return (size_t)kShareCtas * 2 * row_tile(group); }

cudaError_t launch_attn_decode(int d, const AttnArgs& a, cudaStream_t s) {
    if (d == 64) return a.group <= 16 ? launch<64, 1>(a, s) : launch<64, 2>(a, s);
    return a.group <= 16 ? launch<128, 1>(a, s) : launch<128, 2>(a, s);
}

}  // namespace colibri
