// Attention operators: kernel arguments and launchers (internal to the library).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace colibri {

enum class DType : int;

// Keys of a sequence, and of a shared prefix, at most, so that a tile behind the
// last one still has int32 positions.
constexpr int kMaxKeys = 0x7ff00000;

// What the rows and keys of a launch are.
enum AttnMode : int {
    kAttnPrompt = 0,   // rows of seq_start, keys 0 .. kv_len[b] - 1
    kAttnPrefix = 1,   // all n_seqs rows as one sequence over the shared prefix;
                       // row i sees its first min(kv_len[i], prefix_len) keys
    kAttnSuffix = 2    // row b over keys prefix_len .. kv_len[b] - 1
};

struct AttnArgs {
    const void* q;
    const void* k;
    const void* v;
    void* o;
    float* lse;                  // [n_rows, hq] or null
    const int32_t* seq_start;    // prompt
    const int32_t* kv_len;       // null: the sequence's row count
    const int32_t* table;        // null: packed keys
    int64_t q_stride, o_stride;
    int64_t page_stride, head_stride, row_stride;
    int mode;
    int n_seqs, n_rows;
    int hq, hkv, group;
    int table_stride;            // entries per sequence
    int num_pages, page_size, page_shift;
    int prefix_len;
    int causal;
    float scale_log2;            // scale * log2(e)
    // work split over the keys: `splits` ranges per row tile.  part_o null:
    // one range, the kernel writes o and lse; otherwise range s of this launch
    // writes its normalised rows and log2-sums to slot part_slot + s
    int splits;
    int part_slot;
    float* part_o;               // [slots][n_rows * hq][d]
    float* part_lse;             // [slots][n_rows * hq]
    int beside_prefix;           // launch_attn_decode: the launch before it is the prefix's
    // launch_attn_decode: the cut rows' pieces (attn_decode_pieces() rows)
    float* piece_o;
    float* piece_lse;
    // keys and values as 8-bit codes: scales [num_pages][hkv][page_size >> block_shift]
    // (null: k and v are of the rows' type)
    const float* k_scale;
    const float* v_scale;
    int block_shift, int8;
    // launch_attn_decode8: rows (token, head of the group) of a sequence that meet a key at
    // once, 8 or 16, and of a piece
    int tile_rows, piece_rows;
    // launch_attn_decode(8) and the join, where rows are one token's: tiles per key head, and
    // of all of them (divided on the host: on the device 2 us of a step of some 20)
    int group_tiles, seq_items;
    uint64_t wait_limit_ns;      // bound of every mbarrier wait
    int stall_tma;               // failure-detection tests only: a CTA's copies of Q and K stop at
                                 // this item of its work (1: the first), 0 never
};

// CUDA-core attention of float32 rows (every mode).
int64_t attn_simt_items(const AttnArgs& a);  // row tiles of the launch, per key head
cudaError_t launch_attn_simt(int d, const AttnArgs& a, cudaStream_t s);

// Tensor-core attention of bf16 rows (prompt and prefix modes): row tiles of
// 2 * (128 / group) tokens of one sequence.
int64_t attn_tc_items(const AttnArgs& a);    // row tiles of the launch, per key head
// Pages and heads as one dimension of a tensor map; false: more than 2^31 - 1 of them.
bool attn_tc_units(const AttnArgs& a, int64_t* unit, int* per_page, int* per_head, int* count);
cudaError_t launch_attn_tc(int d, const AttnArgs& a, cudaStream_t s);
// Waits for s; *status is DEV_TIMEOUT when a wait has given up since the last time.
cudaError_t attn_tc_status(int* status, cudaStream_t s);

// Rows of suffix mode, equal shares of the key list per warp (bf16, and float32
// groups of up to 32 heads).  part_o null: no prefix; otherwise slot part_slot
// takes the rows written in one piece.
bool attn_decode_takes(DType dt, int group);
int attn_decode_tile(DType dt, int group);   // rows of a group that meet a key at once
size_t attn_decode_pieces(DType dt, int group);
cudaError_t launch_attn_decode(DType dt, int d, const AttnArgs& a, cudaStream_t s);
// The same over codes (bf16 rows), in suffix mode or prompt mode: tiles of tile_rows rows
// of a sequence; its pieces.
size_t attn_decode8_pieces(int tile_rows, int piece_rows);
cudaError_t launch_attn_decode8(int d, const AttnArgs& a, cudaStream_t s);

// o, lse from the partial rows of `slots` slots, and of the pieces that
// launch_attn_decode left (shares; slot part_slot then holds the rows it wrote
// whole, and without a prefix those are not touched).
cudaError_t launch_attn_join(DType dt, int d, const AttnArgs& a, int slots, bool shares, cudaStream_t s);

// Norm, rotation and placement of q, k, v rows.
struct AppendArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const void *q_norm, *k_norm;     // or null
    float eps;
    const double* freq;              // null: no rotation
    // null: positions follow from the lengths; otherwise row r's on axis x is
    // positions[x * axis_stride + r], and pair i turns by axis[i]'s (null: axis 0)
    const int32_t* positions;
    int64_t axis_stride;
    const uint8_t* axis;
    int n_axes;
    int rot_dim, interleaved;
    float mscale;
    const int32_t *seq_start, *kv_len, *table;
    int n_seqs, n_rows, table_stride;
    int hq, hkv;
    void* q_out;
    int64_t q_out_stride;
    // paged keys and values, or (v_out null) rows of k_out
    void *k_out, *v_out;
    int64_t page_stride, head_stride, row_stride;
    int num_pages, page_shift;
    // codes: scales [num_pages][hkv][page >> block_shift]
    float *k_scale, *v_scale;
    int block_shift;
};
cudaError_t launch_append(DType dt, int d, const AppendArgs& a, cudaStream_t s);
// The same into pages of 8-bit codes (k_out, v_out; bf16 rows).
cudaError_t launch_append8(bool int8, int d, const AppendArgs& a, cudaStream_t s);

// Pages of 8-bit codes as bf16 [n_pages, hkv, page_size, d]; ids that no page has
// give zeros.
struct ValuesArgs {
    const void *k, *v;
    const float *k_scale, *v_scale;
    int64_t page_stride, head_stride, row_stride;
    int num_pages, page_size, page_shift, block_shift, hkv;
    const int32_t* pages;            // [n_pages], null: 0 .. n_pages - 1
    int n_pages;
    void *k_out, *v_out;
};
cudaError_t launch_values8(bool int8, int d, const ValuesArgs& a, cudaStream_t s);

}  // namespace colibri
