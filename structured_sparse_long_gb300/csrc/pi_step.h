// pi_step.h -- host-side launch descriptors of rotary positions and of a speculative serving step, shared by the C ABI and the
// kernel files.
#pragma once

#include "pi_paged.h"

namespace pi {

constexpr int kTreeMax = 256;  // nodes of a drafted tree (PI_ATTN_TREE_MAX)

// Which elements of a row turn (pi_attn_rotary_t).
struct Rotary {
    const unsigned long long *step;  // [rot / 2] turns per position, in 2^-64
    int rot, interleaved;
    float scale;
};

// A [B, heads, N, d] tensor and where its rows go.
struct RotaryTensor {
    const void *x;
    void *y;
    long long x_batch, x_head, x_pos, y_batch, y_head, y_pos;  // strides in elements
    int heads;
};

struct RotaryArgs {
    RotaryTensor t[2];  // queries, keys (heads = 0: none)
    Rotary r;
    const int *pos;  // [B, N] or null: start + row
    int start, B, N, d;
    bool f32, back;
};

struct RotaryAppendArgs {
    AppendArgs a;  // keys, values, cache, batch
    Rotary r;
    const __nv_bfloat16 *q;  // [T, H, d], tokens q_stride elements apart
    long long q_stride;
    __nv_bfloat16 *q_out;
    long long q_out_stride;
    const int *parent;  // [T] or null
    int H;
};

struct ExtendTreeArgs {
    ExtendArgs e;
    const int *parent;  // [T]
    bool few;           // tree_few()
};

struct VerifyArgs {
    const float *target, *draft;  // [T, V], rows *_stride elements apart; draft may be null
    long long target_stride, draft_stride;
    const int *tokens, *cu, *parent;
    const float *u, *u_next;
    int B, T, V;
    int *path, *count, *next;
    int *index_word;
};

constexpr int kKeepLayers = 64;  // layers of a launch

struct KeepArgs {
    PagedCache cache;  // sizes and type; the layers' pages:
    void *k[kKeepLayers], *v[kKeepLayers];
    uint8_t *k_scale[kKeepLayers], *v_scale[kKeepLayers];
    int layers, chunks;  // chunks: CTAs per sequence, set at the launch
    PagedBatch batch;
    const int *path, *count;
    int *index_word;
};

// 16-byte pieces (and one for the scales of an 8-bit row) of a sequence's row in one layer, and whether a launch holds those of B sequences.
inline int keep_pieces(const PagedCache &c) {
    return 2 * c.Hkv * (c.kv_type == kKvBf16 ? c.d / 8 : c.d / 16 + 1);
}
inline bool keep_fits(const PagedCache &c, long long B, int layers) { return B * (((long long)keep_pieces(c) * layers + 255) / 256) <= 0x7fffffffLL; }

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t st);               // pi_verify.cu
cudaError_t launch_keep(const KeepArgs &a, cudaStream_t st);                   // pi_keep.cu
// Query heads of a KV group in a block of 128 rows of the trees' tensor-core kernel: as many as divide the group, so that a block has
// few nodes.
inline int tree_heads(int G) {
    int heads = 1;
    while (heads < 16 && G % (2 * heads) == 0) heads *= 2;
    return heads;
}

bool tree_few(const ExtendTreeArgs &a, bool &fits);  // pi_decode_paged.cu
cudaError_t launch_tree_tc(const ExtendTreeArgs &a, cudaStream_t st);          // pi_tree_tc.cu
cudaError_t launch_extend_tree(const ExtendTreeArgs &a, cudaStream_t st);      // pi_decode_paged.cu
cudaError_t launch_rotary(const RotaryArgs &a, cudaStream_t st);               // pi_rotary.cu
cudaError_t launch_rotary_append(const RotaryAppendArgs &a, cudaStream_t st);  // pi_rotary.cu
bool rotary_append_fits(const RotaryAppendArgs &a);                             // whether a launch holds it

}  // namespace pi
