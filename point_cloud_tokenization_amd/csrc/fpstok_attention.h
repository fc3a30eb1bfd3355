// Internal interface between the C ABI (fpstok_attention_api.cpp) and the
// gfx950 kernels of attention (fpstok_attention.hip) and rotary positions
// (fpstok_rope.hip).  Not installed; not part of the ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <hip/hip_vector_types.h>
#include <stddef.h>
#include <stdint.h>

namespace fpstok {

constexpr int kMaxAxes = 4;

// Rows of the sequences of a batch (fpstok_seqs).
struct SeqArgs {
    const int32_t* cu;     // packed: [B+1], or null
    const int32_t* count;  // padded: [B], or null
    int64_t rows;
    int32_t B;
    int32_t cap;
};

struct HeadsArg {
    void* data;
    int64_t row, head;  // strides in elements
};

struct AttnArgs {
    SeqArgs qs, ks;
    HeadsArg q, k, v, out, grad_out, grad_q, grad_k, grad_v;
    float* lse;    // [q rows][H], or null (forward)
    float* lse2;   // [H][q rows] log2(e) lse (backward)
    float* delta;  // the same shape: sum of grad_out * out (or its exact value)
    int32_t H, Hk, D, dtype;
    int32_t G, g_shift;  // H / Hk; its logarithm if it is a power of two, else -1
    int32_t same_seqs;   // ks is qs
    int32_t left, right, sinks;
    float scale;
    // keys of a row split over `splits` workgroups (forward): their partial
    // results, [splits][Hk][q rows * H / Hk] of D floats and of (maximum * c, sum)
    int32_t splits;
    float* part;
    float2* part_ml;
    // rows that see a sequence's sinks from behind its first key tile's window
    // (backward): walked in chunks of 2^sink_shift queries, whose parts of the
    // sinks' gradients are [slots][Hk][2][sinks][D] (grad_k, grad_v)
    int32_t sink_shift;
    // a key's walk split over `k_splits` workgroups (backward): their parts,
    // [k_splits][grad_k, grad_v][Hk][k rows][D]
    int32_t k_splits;
    float* k_part;
    float* sink_part;
};

// A learned bias of the scores by buckets of distance (fpstok_rel_bias).
struct BiasArgs {
    const void* q_pos;  // [q rows][axes], float32 or (ints) int32
    const void* k_pos;
    const float* table;  // [H][entries]
    int32_t axes, ints, entries;
    int32_t first[kMaxAxes], top[kMaxAxes];  // an axis's first entry and its last bucket
    int32_t log_shift[kMaxAxes];             // bits below a step of a log axis, -1: linear
    float rate[kMaxAxes], shift[kMaxAxes];
    int32_t spans;  // look for blocks of pairs in one bucket
    // gradient: the entries from .. from + count - 1 (all there are, or a part of
    // many), and the workgroups' parts, [row tiles][Hk][G][count]
    int32_t from, count;
    float* grad;  // [H][entries], or null
    float* part;
    // the pairs' entries, found once for all heads, at [q row * pitch + key] for
    // sequences of up to `pitch` keys.  plane: two axes at a time, in bytes of a table of
    // their sums ([bucket of the first * buckets of the second + that of the second]):
    // axes 0 and 1 in the lower half of a word, 2 and 3, behind them in the table, in the
    // upper one.  bytes: 4 times the entry of axis a in byte a (for the gradient).
    uint32_t* plane;  // null: every head finds its own
    uint32_t* bytes;
    int32_t pitch;
    int32_t joint[2];  // sizes of the two tables of sums
};
constexpr int kGroupEntries = 4096;  // table entries of one key head's query heads (16 KB of LDS)
constexpr int kTableEntries = 64;  // entries whose gradients one launch forms

// The pitch of the entries' plane, 0 without one.
int32_t plan_plane(const AttnArgs& a, const BiasArgs& b, bool few, int32_t k_len);

// How a call is laid out on the device, from the shapes alone.
struct AttnPlan {
    bool few;        // at most 32 rows per sequence and key head: waves split the keys
    int32_t splits;  // workgroups a row's keys are split over
    int64_t blocks;  // workgroups of the largest launch
};

struct RopeArgs {
    SeqArgs seqs;
    HeadsArg in[2], out[2];
    int32_t heads[2];
    const void* positions;
    const float* freqs;
    int32_t D, dtype, int_positions, axes, R, interleaved, inverse;
    int32_t block_rows;  // rows per workgroup (set by the launch)
    int32_t first_pair[kMaxAxes + 1];  // pairs of axis a: first_pair[a] .. first_pair[a+1]-1
};

// Slots of 2^shift rows that cover every sequence (their numbering: slot_of).
int64_t row_slots(const SeqArgs& s, int G, int shift);
// Workgroups that the walk of 128 keys' gradients is split over.
int plan_key_parts(const AttnArgs& a, int32_t q_len);
AttnPlan plan_attention(const AttnArgs& a, int32_t q_len, int32_t k_len);
hipError_t launch_attention(const AttnArgs& a, const AttnPlan& plan, hipStream_t s);
hipError_t launch_attention_backward(const AttnArgs& a, hipStream_t s);
// The same with a bias (fpstok_attention_bias.hip).
hipError_t launch_attention_bias(const AttnArgs& a, const BiasArgs& b, const AttnPlan& plan,
                                 hipStream_t s);
hipError_t launch_attention_bias_backward(const AttnArgs& a, const BiasArgs& b, hipStream_t s);
// Joins of split walks.
void launch_join(const AttnArgs& a, hipStream_t s);
void launch_join_dkv(const AttnArgs& a, hipStream_t s);
hipError_t launch_rope(const RopeArgs& a, hipStream_t s);

}  // namespace fpstok
