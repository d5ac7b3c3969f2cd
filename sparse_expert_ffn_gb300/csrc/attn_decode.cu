// Attention of single rows over a paged cache (bf16, and float32 groups of up to
// 32 heads): the decode step, and the sequences' own keys behind a shared prefix.
//
// Bound by HBM: every key and value is read once and meets only the rows of
// its head group, so the products are few and what counts is that all SMs
// stream all the time, whatever the lengths of the sequences are.
//
// Work is cut into steps of 8 KB of K and V (2048 / d keys of bf16, 1024 / d of
// float32) of one (sequence, key head, row tile), laid out one after another, and
// every warp of the grid takes an equal share of the whole list: a share may end
// inside a sequence and begin inside another one.  A (sequence, head) that falls to one warp is
// written directly; the pieces of one that is cut go to the workspace, at most
// two per warp (its first and its last), and attn_join.cu adds them in key
// order.  Nothing depends on the order in which warps run, and no warp waits
// for another: each streams its share through its own ring of 3 stages with
// cp.async, two steps ahead of the products, across the ends of its pieces.
//
// bf16: the rows of the group are the 16 rows of mma.sync m16n8k16 (2 tiles up to 32
// rows): tensor-memory MMAs would pad them to 64 or 128 and spend most of the
// time of a 16-key step on that padding.  Scores stay in registers and become
// the A operand of the product with V as they lie.  The reference maximum and
// the sum are f32 per row, P is rounded to bf16 for the product (its operands
// share one 16-bit type).
//
// float32: products in f32, two to an instruction.  A lane has one key of a step
// and a quarter (d 128) or half (d 64) of its columns in the scores, whose query
// rows lie in registers, and d / 32 columns of all keys in the product with V.  A
// step of 4 rows takes a quarter of the issue slots that its 8 KB leave: 48
// sequences of 4000 keys of 16 heads of 128 take 447 to 458 us, 6.9 TB/s (tiles of 16
// rows of a CTA, which read K and V from shared memory for every row, 2135 us).  More
// rows' queries do not fit a warp's registers, so a group is cut into tiles of 4, and
// since every warp streams for itself, the keys are read once per tile (4 key heads of
// d 128: groups of 4 take 120 us, of 8 236 instead of 716 in one tile of attn_simt.cu,
// of 32 865 instead of 1007).
#include <cuda_runtime.h>

#include "attn_rows8.cuh"
#include "attn_share.cuh"

namespace colibri {
namespace {

// Up to 16 MT rows of a group on mma.sync.
template <int D, int MT>
struct TensorRows {
    using T = __nv_bfloat16;
    using Out = T;
    static constexpr int kD = D, kRows = 16 * MT, KS = kStepKeys<T, D>, kScratch = 0, kStages = 3, kCtas = 2;
    static constexpr bool kMany = false;
    uint32_t qf[MT][D / 16][4];
    float o[MT][D / 8][4], m[MT][2], l[MT][2];

    template <bool kEarly>
    __device__ __forceinline__ void begin(const AttnArgs& a, int b, int h, int r0) {
        const int lane = threadIdx.x & 31;
        // the group's rows as A operands: row lane / 4 (+ 8), columns 2 (lane % 4) (+ 8)
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int g = r0 + 16 * t + 8 * half + (lane >> 2);
                const uint32_t* q = reinterpret_cast<const uint32_t*>(
                    static_cast<const __nv_bfloat16*>(a.q) + (int64_t)b * a.q_stride + (int64_t)(h * a.group + g) * D);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    qf[t][x][half] = g < a.group ? ld_early<kEarly>(q + x * 8 + (lane & 3)) : 0u;
                    qf[t][x][half + 2] = g < a.group ? ld_early<kEarly>(q + x * 8 + 4 + (lane & 3)) : 0u;
                }
            }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;
#pragma unroll
            for (int x = 0; x < D / 8; ++x) o[t][x][0] = o[t][x][1] = o[t][x][2] = o[t][x][3] = 0.f;
        }
    }
    // K and V of `keys` keys at ks and vs
    __device__ __forceinline__ void step(const AttnArgs& a, uint32_t ks, uint32_t vs, int keys, uint32_t) {
        const int lane = threadIdx.x & 31;
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
        uint32_t pf[MT][KS / 16][4];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            float top[2] = {-INFINITY, -INFINITY};
            if (keys < KS) {
#pragma unroll
                for (int n = 0; n < KS / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n * 8 + 2 * (lane & 3) + (e & 1) >= keys) s[t][n][e] = -INFINITY;
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
    // put(row of the tile, reference, sum, whether this lane writes the sum, how it
    // writes its columns) for every row
    template <typename Put>
    __device__ __forceinline__ void end(Put put) {
        const int lane = threadIdx.x & 31, c = 2 * (lane & 3);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float sum = l[t][r];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                put(16 * t + 8 * r + (lane >> 2), m[t][r], sum, c == 0, [&](auto* out, float inv) {
#pragma unroll
                    for (int x = 0; x < D / 8; ++x) {
                        const float u = o[t][x][2 * r] * inv, w = o[t][x][2 * r + 1] * inv;
                        if constexpr (sizeof(*out) == 2) *reinterpret_cast<uint32_t*>(out + x * 8 + c) = bf16x2(u, w);
                        else *reinterpret_cast<float2*>(out + x * 8 + c) = make_float2(u, w);
                    }
                });
            }
    }
};

__device__ __forceinline__ ulonglong2 lds2x2(uint32_t addr) {
    ulonglong2 v;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t lds2(uint32_t addr) {
    uint64_t v;
    asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

// Up to G rows of a group on the f32 pipes.
template <int D, int G>
struct FloatRows {
    using T = float;
    using Out = T;
    static constexpr int kD = D, kRows = row_tile<T>(0), KS = kStepKeys<T, D>, kParts = 32 / KS, kStages = 3, kCtas = 2;
    static constexpr bool kMany = false;
    static constexpr int kScratch = G * KS * 4;                    // a step's weights
    static constexpr int kPairs = D / 64;                          // column pairs of a lane
    uint64_t q[G][16], o[G][kPairs];                               // columns 32 (lane / KS) .. + 31 of q
    float m[G], l[G];                                              // l: of this lane's keys

    template <bool kEarly>
    __device__ __forceinline__ void begin(const AttnArgs& a, int b, int h, int r0) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float* row = static_cast<const float*>(a.q) + (int64_t)b * a.q_stride +
                               (int64_t)(h * a.group + r0 + g) * D + lane / KS * 32;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 v = r0 + g < a.group ? ld_early<kEarly>(reinterpret_cast<const float4*>(row) + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                q[g][2 * i] = pack2(v.x, v.y), q[g][2 * i + 1] = pack2(v.z, v.w);
            }
            m[g] = -INFINITY, l[g] = 0.f;
#pragma unroll
            for (int x = 0; x < kPairs; ++x) o[g][x] = 0;
        }
    }
    __device__ __forceinline__ void step(const AttnArgs& a, uint32_t ks, uint32_t vs, int keys, uint32_t weights) {
        const int lane = threadIdx.x & 31, key = lane % KS, part = lane / KS;
        uint64_t acc[G];
#pragma unroll
        for (int g = 0; g < G; ++g) acc[g] = 0;
        // (8 lanes of a pass read 8 keys, whose chunks the swizzle spreads over the banks)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const ulonglong2 k = lds2x2(ks + key * (D * 4) + (((part * 8 + i) ^ (key & 7)) << 4));
#pragma unroll
            for (int g = 0; g < G; ++g) acc[g] = fma2(q[g][2 * i + 1], k.y, fma2(q[g][2 * i], k.x, acc[g]));
        }
        float s[G];
        bool grown = false;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float2 half = unpack2(acc[g]);
            s[g] = half.x + half.y;
#pragma unroll
            for (int off = KS; off < 32; off <<= 1) s[g] += __shfl_xor_sync(0xffffffffu, s[g], off);
            s[g] = key < keys ? s[g] * a.scale_log2 : -INFINITY;
            grown |= s[g] > m[g] + 8.f;
        }
        // the reference maximum moves only when a row's has grown by more than 2^8
        // (f32 holds weights below 2^8 as exactly as those below 1)
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                float top = s[g];
#pragma unroll
                for (int off = 1; off < KS; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                const bool grow = top > m[g];
                const float keep = grow ? ex2(m[g] - top) : 1.f;
                if (grow) m[g] = top;
                l[g] *= keep;
#pragma unroll
                for (int x = 0; x < kPairs; ++x) o[g][x] = mul2(o[g][x], pack2(keep, keep));
            }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const float p = ex2(s[g] - (m[g] == -INFINITY ? 0.f : m[g]));
            l[g] += p;
            if (part == g % kParts)
                asm volatile("st.shared.f32 [%0], %1;" ::"r"(weights + (g * KS + key) * 4), "f"(p) : "memory");
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < KS; j += 4) {
            float2 p[G][2];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const ulonglong2 w = lds2x2(weights + (g * KS + j) * 4);
                p[g][0] = unpack2(w.x), p[g][1] = unpack2(w.y);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                uint64_t v[kPairs];
                const uint32_t row = vs + (j + y) * (D * 4);
                if constexpr (kPairs == 2) {
                    const ulonglong2 w = lds2x2(row + ((lane ^ ((j + y) & 7)) << 4));
                    v[0] = w.x, v[1] = w.y;
                } else {
                    v[0] = lds2(row + (((lane >> 1) ^ ((j + y) & 7)) << 4) + (lane & 1) * 8);
                }
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float w = y & 1 ? p[g][y >> 1].y : p[g][y >> 1].x;
#pragma unroll
                    for (int x = 0; x < kPairs; ++x) o[g][x] = fma2(pack2(w, w), v[x], o[g][x]);
                }
            }
        }
    }
    template <typename Put>
    __device__ __forceinline__ void end(Put put) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float sum = l[g];
#pragma unroll
            for (int off = 1; off < KS; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            put(g, m[g], sum, lane == 0, [&](float* out, float inv) {
#pragma unroll
                for (int x = 0; x < kPairs; ++x) {
                    const float2 u = unpack2(o[g][x]);
                    reinterpret_cast<float2*>(out)[lane * kPairs + x] = make_float2(u.x * inv, u.y * inv);
                }
            });
        }
    }
};

// kEarly: behind a prefix launch the kernel starts on the SMs that this one has left;
// it needs nothing of it (48 rows over a prefix of 16384 keys: 58 us, 69 waiting
// first; what it reads: ld_early).  It waits for it at the end, so that the join,
// which waits for this kernel, finds both done.
template <typename Rows, bool kEarly>
__global__ void __launch_bounds__(kDecThreads, Rows::kCtas) attn_decode_kernel(const __grid_constant__ AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    if constexpr (kEarly) pdl_launch_dependents();
    else pdl_enter();
    decode_share<Rows, kEarly>(a, smem);
    if constexpr (kEarly) pdl_wait();
}

template <typename Rows>
cudaError_t launch(const AttnArgs& a, cudaStream_t s) {
    auto kern = a.beside_prefix ? attn_decode_kernel<Rows, true> : attn_decode_kernel<Rows, false>;
    using T = typename Rows::T;
    const int bytes = kShareWarps * (Rows::kStages * kStageBytes + Rows::kScratch);
    cudaError_t e = smem_attr((const void*)kern, bytes);
    return e != cudaSuccess ? e : launch_pdl(kern, dim3(most_shares<T>(Rows::kRows) / kShareWarps), dim3(kDecThreads), bytes, s, a);
}

}  // namespace

size_t attn_decode8_pieces(int tile_rows, int piece_rows) {
    return (size_t)most_shares<uint8_t>(tile_rows) * 2 * piece_rows;
}

size_t attn_decode_pieces(DType dt, int group) {
    return dt == DType::BF16 ? (size_t)most_shares<__nv_bfloat16>(group) * 2 * piece_rows<__nv_bfloat16>(group)
                             : (size_t)most_shares<float>(group) * 2 * piece_rows<float>(group);
}

int attn_decode_tile(DType dt, int group) {
    return dt == DType::BF16 ? row_tile<__nv_bfloat16>(group) : row_tile<float>(group);
}

// (a float32 group of 64 would be read 16 times)
bool attn_decode_takes(DType dt, int group) { return dt == DType::BF16 || group <= 32; }

template <int D>
static cudaError_t launch_rows(DType dt, const AttnArgs& a, cudaStream_t s) {
    if (dt == DType::BF16)
        return a.group <= 16 ? launch<TensorRows<D, 1>>(a, s) : launch<TensorRows<D, 2>>(a, s);
    return a.group == 1   ? launch<FloatRows<D, 1>>(a, s)
           : a.group == 2 ? launch<FloatRows<D, 2>>(a, s)
                          : launch<FloatRows<D, 4>>(a, s);
}

cudaError_t launch_attn_decode(DType dt, int d, const AttnArgs& a, cudaStream_t s) {
    return d == 64 ? launch_rows<64>(dt, a, s) : launch_rows<128>(dt, a, s);
}

template <int D>
static cudaError_t launch_codes(const AttnArgs& a, cudaStream_t s) {
    const auto pick = [&](auto code) {
        using C = decltype(code);
        if (a.mode == kAttnPrompt)
            return a.tile_rows == 8 ? launch<CodeRows<C, D, 1, true>>(a, s) : launch<CodeRows<C, D, 2, true>>(a, s);
        return a.tile_rows == 8 ? launch<CodeRows<C, D, 1, false>>(a, s) : launch<CodeRows<C, D, 2, false>>(a, s);
    };
    return a.int8 ? pick(I8{}) : pick(E4M3{});
}

cudaError_t launch_attn_decode8(int d, const AttnArgs& a, cudaStream_t s) {
    return d == 64 ? launch_codes<64>(a, s) : launch_codes<128>(a, s);
}

}  // namespace colibri
