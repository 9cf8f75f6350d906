/*
 * libgdn.h -- C ABI of libgdn, hand-written HIP kernels (AMD Instinct MI355X,
 * gfx950) for the gated-delta-rule (GDN) linear-attention mixer of the
 * Qwen3.5 hybrid models.
 *
 * The mixer, per layer and per stream: a depthwise causal conv1d of width 4
 * over the packed q/k/v channels, whose last three raw input rows are the
 * stream's conv tail; SiLU on every channel; q and k L2-normalised per key
 * head (q also scaled by dk^-1/2); then, per value head, the gated delta rule
 * (Yang, Kautz and Hatamizadeh, "Gated Delta Networks", 2024)
 *     S <- alpha S (I - beta k k^T) + beta v k^T,     o = S q,
 *     alpha = exp(-exp(A_log) softplus(a + dt_bias)), beta = sigmoid(b).
 * The engine on the pages keeps this glue (gated delta rule and causal
 * convolution) in qwen35.cu: page "perf(qwen3_5 cuda): deliver the first
 * token before drafting", commit note on the MLX affine 4-bit checkpoint.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensor pointers are DEVICE pointers owned by the caller; libgdn never
 *    allocates, frees or keeps them, and keeps no state between calls.
 *    bf16 values travel as their 16-bit patterns (uint16_t).
 *  - Channels of a packed row: C = 2*hk*dk + hv*dv, ordered [q | k | v], each
 *    head-major.  Value head h reads key head h / (hv / hk).
 *  - The recurrent state of a stream is fp32 [hv][dk][dv] with dv contiguous:
 *    it stores S^T, so element [h][i][j] is S_h[j][i].
 *  - The conv tail of a stream is bf16 [3][C]: the last three raw (pre-conv)
 *    rows, oldest first.  Conv weights are fp32 [C][4]; tap 3 multiplies the
 *    current row, tap j the row 3 - j before it.  There is no conv bias.
 *  - Every call is asynchronous on `stream` (a hipStream_t; NULL = the null
 *    stream).  All host-visible arguments are checked before anything is
 *    launched: a refused call returns a negative status and touches no
 *    output.  gdn_last_error() then describes the refusal (per thread).
 *  - Arguments that live on the device (row starts, parents, accepted rows)
 *    cannot be checked without a synchronisation.  Their rules are stated
 *    per call; a stream whose device-side layout breaks them is skipped by
 *    the kernels (its outputs are left untouched).  gdn_check_layout() checks
 *    host copies of them.
 *  - Supported geometry: dk in {64, 128}; dv in {64, 128}; hv % hk == 0;
 *    conv_width == 4.  Windows hold at most 16 rows.
 */
#ifndef LIBGDN_H
#define LIBGDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_MAX_WINDOW_ROWS 16

typedef struct gdn_shape {
    int32_t hk;          /* key heads                        */
    int32_t hv;          /* value heads, a multiple of hk    */
    int32_t dk;          /* key (and query) head size        */
    int32_t dv;          /* value head size                  */
    int32_t conv_width;  /* must be 4                        */
} gdn_shape;

typedef struct gdn_params {
    const float *conv_w;   /* [C][4] fp32, device */
    const float *a_log;    /* [hv]   fp32, device */
    const float *dt_bias;  /* [hv]   fp32, device */
} gdn_params;

enum gdn_status {
    GDN_OK = 0,
    GDN_EINVAL = -1,        /* malformed argument (null pointer, bad size) */
    GDN_EUNSUPPORTED = -2,  /* well-formed but outside the supported shapes */
    GDN_EWORKSPACE = -3,    /* workspace missing or too small               */
    GDN_EHIP = -4           /* the HIP runtime refused a launch             */
};

/* Name of a status code ("GDN_OK", "GDN_EINVAL", ...); never NULL. */
const char *gdn_status_name(int status);

/* Text of the last refusal on the calling thread ("" if none). */
const char *gdn_last_error(void);

/* Number of conv channels C of a shape, or -1 if the shape is refused. */
int32_t gdn_channels(const gdn_shape *shape);

/*
 * One-row decode step for n_streams streams, updating state and tail in
 * place (one-row steps and prompt passes update a stream's state in place:
 * page "perf(qwen3_5 cuda): deliver the first token before drafting", commit
 * note on tree-shaped verify windows).
 *   qkv       [n][C] bf16      row of each stream
 *   a, b      [n][hv] bf16     gate inputs
 *   conv_tail [n][3][C] bf16   in/out
 *   state     [n][hv][dk][dv]  fp32 in/out
 *   out       [n][hv][dv] fp32 o of each value head
 * The result equals, bit for bit, a one-row gdn_recur_window followed by
 * gdn_commit of that row.  Extra limit: (hv/hk) * dv <= 512.
 */
int gdn_conv_step(const gdn_shape *shape, const gdn_params *params, int32_t n_streams,
                  const uint16_t *qkv, const uint16_t *a, const uint16_t *b,
                  uint16_t *conv_tail, float *state, float *out, void *stream);

/*
 * Verify windows of several streams in one pass, recording every row's state
 * and conv tail.  Windows hold up to 16 rows, every stream's window is packed
 * back to back (up to 16 streams of 16 rows were taken together on the page
 * "perf(qwen27 cuda): reduce repeated-prompt TTFT", commit note on the
 * qwen3_5 checkpoint with the 27B's shapes), and each row's recurrence and
 * conv tail are recorded so that any prefix can be kept (page "perf(qwen3_5
 * cuda): deliver the first token before drafting", commit note on the MLX
 * affine 4-bit checkpoint).  Row t of stream s is packed row row_start[s]+t
 * and follows row t-1 (row 0 follows the stream's state and tail).
 *   row_start  [n+1] int32, device: 0 <= row_start[s] <= row_start[s+1]
 *              <= total_rows and row_start[s+1] - row_start[s] <= max_rows
 *   max_rows   1..16, a bound on every window's length
 *   qkv        [total_rows][C] bf16;  a, b [total_rows][hv] bf16
 *   conv_tail  [n][3][C] bf16, state [n][hv][dk][dv] fp32: read only
 *   out        [total_rows][hv][dv] fp32
 *   tail_snap  [total_rows][3][C] bf16: the tail after each row
 *   state_snap [total_rows][hv][dk][dv] fp32: the state after each row
 * Each row's results equal, bit for bit, gdn_conv_step applied row by row,
 * whatever the other streams in the pass and whatever the packing offset.
 */
int gdn_recur_window(const gdn_shape *shape, const gdn_params *params, int32_t n_streams,
                     int32_t total_rows, int32_t max_rows, const int32_t *row_start,
                     const uint16_t *qkv, const uint16_t *a, const uint16_t *b,
                     const uint16_t *conv_tail, const float *state, float *out,
                     uint16_t *tail_snap, float *state_snap, void *stream);

/*
 * Tree-shaped verify windows: each row names its parent, and the conv taps
 * and the delta rule follow that row's own branch (page "perf(qwen3_5 cuda):
 * deliver the first token before drafting", commit note on tree-shaped verify
 * windows).  Same arguments as gdn_recur_window, plus
 *   parent [total_rows] int32, device: the parent's local index within its
 *          stream's window, -1 for a row that follows the stream's own state
 *          and tail; -1 <= parent[row_start[s]+t] < t.
 * A row's state starts from its parent's recorded state, and its conv taps are
 * its three nearest ancestors' raw rows, continuing into the stream's tail.
 * Every root-to-row path equals, bit for bit, gdn_recur_window over that path.
 */
int gdn_recur_tree(const gdn_shape *shape, const gdn_params *params, int32_t n_streams,
                   int32_t total_rows, int32_t max_rows, const int32_t *row_start,
                   const int32_t *parent, const uint16_t *qkv, const uint16_t *a,
                   const uint16_t *b, const uint16_t *conv_tail, const float *state,
                   float *out, uint16_t *tail_snap, float *state_snap, void *stream);

/*
 * Commit of the accepted rows: only each stream's accepted path is kept (page
 * "perf(qwen27 cuda): reduce repeated-prompt TTFT", commit note on the qwen3_5
 * checkpoint with the 27B's shapes).  Copies the accepted row's recorded state
 * and tail over the stream's state and conv_tail.
 *   row_start  [n+1] int32, device: the layout of the gdn_recur_window /
 *              gdn_recur_tree call that recorded the snapshots
 *   accept_row [n] int32, device: the packed index of the stream's accepted
 *              row, within its own window [row_start[s], row_start[s+1]), or
 *              -1 to keep the stream as it is.  Any other value, or a window
 *              that ends past total_rows, skips the stream (a row of another
 *              stream's window is never copied).
 *   tail_snap [total_rows][3][C], state_snap [total_rows][hv][dk][dv]: read
 */
int gdn_commit(const gdn_shape *shape, int32_t n_streams, int32_t total_rows,
               const int32_t *row_start, const int32_t *accept_row, const uint16_t *tail_snap,
               const float *state_snap, uint16_t *conv_tail, float *state, void *stream);

/*
 * Verify windows or trees that LOG every row instead of recording its state
 * and tail: a verify logs its rows' decay, write and key, and keeping a row
 * replays the kept path onto the recurrence (page "perf(qwen3_5 cuda):
 * deliver the first token before drafting", commit note on tree-shaped verify
 * windows).  Same arguments as gdn_recur_tree, with parent == NULL for chain
 * windows, and in place of tail_snap / state_snap:
 *   log_alpha [total_rows][hv] fp32      alpha of each (row, value head)
 *   log_delta [total_rows][hv][dv] fp32  the row's write delta, with
 *             M_row = alpha M_parent + khat delta^T in the stored form M = S^T
 *             (delta = beta (v - alpha M_parent^T khat))
 *   log_key   [total_rows][hk][dk] fp32  khat of each (row, key head)
 * out equals, bit for bit, what gdn_recur_window / gdn_recur_tree write; the
 * log is about 1/100 of the recorded states' bytes at dk = dv = 128, and no
 * per-row state is ever written.
 */
int gdn_recur_log(const gdn_shape *shape, const gdn_params *params, int32_t n_streams,
                  int32_t total_rows, int32_t max_rows, const int32_t *row_start,
                  const int32_t *parent, const uint16_t *qkv, const uint16_t *a,
                  const uint16_t *b, const uint16_t *conv_tail, const float *state, float *out,
                  float *log_alpha, float *log_delta, float *log_key, void *stream);

/*
 * Commit by replay after gdn_recur_log (same page and note: keeping a row
 * replays its path in one pass and carries the path's own entries into
 * place).
 * accept_row [n] int32, device: the packed index of the stream's kept row,
 * within its window [row_start[s], row_start[s+1]), or -1 to keep the stream
 * as it is; any other value, or a layout that breaks gdn_recur_log's rules,
 * skips the stream.  The kept path (the row and its ancestors, root first) is
 * replayed onto state, and the path's last three raw rows from qkv,
 * continuing into the old tail, become conv_tail.  row_start, parent, qkv and
 * the log are those of the gdn_recur_log call.  The result equals, bit for
 * bit, gdn_commit of the same row after gdn_recur_window / gdn_recur_tree.
 */
int gdn_commit_replay(const gdn_shape *shape, int32_t n_streams, int32_t total_rows,
                      int32_t max_rows, const int32_t *row_start, const int32_t *parent,
                      const int32_t *accept_row, const uint16_t *qkv, const float *log_alpha,
                      const float *log_delta, const float *log_key, uint16_t *conv_tail,
                      float *state, void *stream);

/*
 * Bytes of device workspace gdn_prefill_chunked needs for n_seqs prompts of
 * total_rows rows in all (0 if the shape is refused).
 */
size_t gdn_prefill_workspace_bytes(const gdn_shape *shape, int32_t n_seqs, int32_t total_rows);

/*
 * Prompt passes of several prompts packed in one call (prompts that arrive
 * together share one pass: page "perf(qwen27 cuda): reduce repeated-prompt
 * TTFT", commit note on the lane host admitting every queued request), in
 * the chunkwise WY form with chunks of 64 rows, updating each prompt's state
 * and tail in place.  Chunks never cross prompts.  Geometry: dk == dv == 128
 * and hv / hk <= 8 (GDN_EUNSUPPORTED otherwise).
 *   seq_start [n+1] int32, device: 0 <= seq_start[s] <= seq_start[s+1] <= total_rows
 *   max_len   a bound on every prompt's length (sizes the launch)
 *   qkv [total_rows][C] bf16; a, b [total_rows][hv] bf16
 *   conv_tail [n][3][C] bf16 in/out; state [n][hv][dk][dv] fp32 in/out
 *   out [total_rows][hv][dv] fp32
 *   workspace: device memory of at least gdn_prefill_workspace_bytes()
 * Results match the row-by-row recurrence within the rounding of its bf16
 * matrix-core operands; they are not bitwise equal to one-row steps.
 */
int gdn_prefill_chunked(const gdn_shape *shape, const gdn_params *params, int32_t n_seqs,
                        int32_t total_rows, int32_t max_len, const int32_t *seq_start,
                        const uint16_t *qkv, const uint16_t *a, const uint16_t *b,
                        uint16_t *conv_tail, float *state, float *out, void *workspace,
                        size_t workspace_bytes, void *stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation):
 * gdn_prefill_chunked with its workspace in a fixed device array of
 * GDN_PREFILL_SCRATCH_BYTES (128 MiB) that the library holds on every GPU it
 * runs on until the process ends.  Same arguments as gdn_prefill_chunked
 * without the workspace, and bit for bit the same results.  Allocates
 * nothing.
 *  - A pass whose workspace (gdn_prefill_workspace_bytes) exceeds the array
 *    is refused with GDN_EWORKSPACE before anything is launched: at 48 value
 *    heads of 128 that is a pass of more than about 43 chunks of 64 rows
 *    (one prompt of 2,752 rows).
 *    Longer prompts can be passed in pieces cut at multiples of 64 rows,
 *    which give the same bits as one pass.
 *  - `stream` must belong to the calling thread's current device; the
 *    array's address on that device is looked up on the first call there.
 *  - Every call on a GPU shares that GPU's array.  A pass writes every byte
 *    of it that it reads, so nothing has to be cleared between calls, but
 *    calls that overlap on one GPU (on different streams, or from threads
 *    without ordering) race and give undefined results.
 */
#define GDN_PREFILL_SCRATCH_BYTES (128u * 1024u * 1024u)
int gdn_prefill_chunked_noalloc(const gdn_shape *shape, const gdn_params *params, int32_t n_seqs,
                                int32_t total_rows, int32_t max_len, const int32_t *seq_start,
                                const uint16_t *qkv, const uint16_t *a, const uint16_t *b,
                                uint16_t *conv_tail, float *state, float *out, void *stream);

/*
 * The in-projection before the mixer: its packed rows qkv and gate inputs a,
 * b from hidden rows x, y = x W^T, with W in affine 4-bit form (the
 * projections of the MLX affine 4-bit checkpoint run through affine-4
 * kernels: page "perf(qwen3_5 cuda): deliver the first token before
 * drafting", note on that checkpoint; the format read as MLX's affine
 * quantisation).  Output features are [qkv (C) | a (hv) | b (hv)], C =
 * 2*hk*dk + hv*dv; weight w[n][k] = scale[n][k/group] * q[n][k] +
 * bias[n][k/group].  Weights are repacked once (at load) into a tiled layout
 * for these kernels: gdn_inproj_pack_affine4.
 *
 * gdn_inproj_padded_features: NP = 16 * ceil((C + 2 hv) / 16), or -1 for a
 * bad shape.
 *
 * gdn_inproj_pack_affine4: MLX layout in, tiled layout out (device arrays,
 * 16-byte aligned, all on `stream`):
 *   wq     [C + 2 hv][hidden/8] packed codes: code j of word w (bits
 *          4j..4j+3) is q[n][8w + j]
 *   scales, biases [C + 2 hv][hidden/group] bf16
 *   wq_tiled [NP * hidden / 8] words; scales_tiled, biases_tiled
 *          [NP * hidden / group] bf16 (the padded features get zeros)
 *
 * gdn_inproj_affine4:
 *   x      [rows][hidden] bf16, device, 16-byte aligned
 *   wq_tiled, scales_tiled, biases_tiled from gdn_inproj_pack_affine4
 *   qkv    [rows][C] bf16 out (16-byte aligned); a, b [rows][hv] bf16 out
 * hidden must be a multiple of 128 and group_size 32, 64 or 128
 * (GDN_EUNSUPPORTED otherwise).  Weights are rounded to bf16 before the
 * matrix-core products, which accumulate in fp32; outputs are rounded to
 * bf16.  rows == 0 does nothing.
 */
int32_t gdn_inproj_padded_features(const gdn_shape *shape);
int gdn_inproj_pack_affine4(const gdn_shape *shape, int32_t hidden, int32_t group_size, const uint32_t *wq,
                            const uint16_t *scales, const uint16_t *biases, uint32_t *wq_tiled,
                            uint16_t *scales_tiled, uint16_t *biases_tiled, void *stream);
int gdn_inproj_affine4(const gdn_shape *shape, int32_t rows, int32_t hidden, int32_t group_size,
                       const uint16_t *x, const uint32_t *wq_tiled, const uint16_t *scales_tiled,
                       const uint16_t *biases_tiled, uint16_t *qkv, uint16_t *a, uint16_t *b, void *stream);

/*
 * Attention layers
 * ----------------
 * A hybrid model's other layers are gated full attention over a growing
 * key-value cache.  The calls below run them beside the mixer's: the same
 * packed rows, windows, trees and accepted rows, every count read on the
 * device.  gdn_kv_tables and gdn_attn_prep take prompts, too, and
 * gdn_attn_prompt attends over them.  (The engine on the pages keeps its gated
 * attention in qwen35.cu, cuts decode attention into key chunks at logical
 * positions, and stores e4m3 cache rows with an fp32 scale of amax / 448.)
 *
 * The cache is paged.  K and V are [n_pages][hkv][page_size][d] (bf16, or
 * e4m3 codes with one fp32 scale a row in [n_pages][hkv][page_size], or 4-bit
 * codes with an exponent byte for every 32 channels of a row); a
 * stream's cache row i is row i % page_size of page block_table[s][i /
 * page_size], block_table [n][max_blocks] int32.  Slot numbers are page *
 * page_size + row.  page_size is 16, 32, 64, 128 or 256, d is 64, 128 or 256,
 * and n_pages * hkv * page_size < 2^31 (GDN_EUNSUPPORTED otherwise).  Query
 * head h reads kv head h / (hq / hkv).  A step is a window of one row.
 *
 * row_start must not fall.  Every stream is looked at by itself: one whose own
 * two entries break the rules is skipped, the others are served as ever.  Where
 * a fall makes the windows of two streams overlap instead, what their common
 * rows get (slots, positions, results) is undefined, and with it what these
 * streams' next rows see; streams without common rows are not touched by it
 * (but gdn_kv_tables takes pages for every window as it stands), and no access
 * leaves the arrays.  gdn_check_layout finds both on the host.
 */
enum gdn_kv_format {
    GDN_KV_BF16 = 0,
    GDN_KV_E4M3 = 1,  /* OCP e4m3, value = code * scale of its row */
    GDN_KV_MXFP4 = 4  /* OCP MXFP4, value = code * 2^(e - 127) of its block */
};

/*
 * GDN_KV_MXFP4 rows are those of the OCP Microscaling Formats 1.0: e2m1 codes
 * (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two a byte with the even
 * channel in the low half, and exponent bytes e in [n_pages][hkv][page_size]
 * [d / 32], whose addresses go into k_scale and v_scale.  e is 1..252, or 255
 * where the block's values are all NaN (253 and 254 are read as 255); so every
 * value is a bf16 number, and the calls that read it round nothing.  4.25 bits a
 * value: 136 bytes for a key of 256 channels instead of 512.
 */
typedef struct gdn_kv_cache {
    void *k, *v;                /* [n_pages][hkv][page_size][d], 16-byte aligned  */
    float *k_scale, *v_scale;   /* [n_pages][hkv][page_size], 16-byte aligned, GDN_KV_E4M3 only;
                                   GDN_KV_MXFP4: exponent bytes (cast) */
    int32_t n_pages, page_size;
    int32_t hkv, d;
    int32_t format;             /* enum gdn_kv_format */
} gdn_kv_cache;

/*
 * Block tables and slot maps from the streams' lengths.  Stream s is to hold
 * kv_len[s] cache rows and its row_start[s+1] - row_start[s] packed rows of
 * this pass, in ceil of their sum / page_size pages; a stream with kv_len[s] <
 * 0 has finished and holds none.
 *   row_start  [n+1] int32; parent [total_rows] int32 or NULL (chains of any
 *              length; with parents a window has at most 16 rows)
 *   kv_len, page_count [n] int32: cached rows, and pages held so far
 *   free_count [1], free_pages [n_pages] int32: a stack of unused pages
 *   block_table [n][max_blocks] int32, in/out
 *   slots, positions [total_rows] int32 out: the slot of each packed row, cache
 *              row kv_len + (its place in the window), and its position,
 *              kv_len + (its number of ancestors in the window)
 *   page_count_out [n], free_count_out [1]: may be page_count and free_count
 * Pages that streams no longer need go onto the stack in stream order; then
 * the streams that grow take theirs from its top, in stream order, and the
 * first one whose pages are not all there, with every later one that grows,
 * takes none.  Rows of a stream that got none, has finished, would need more
 * than max_blocks pages, or breaks the layout rules, and rows of no stream, get
 * slot and position -1.  Entries of block_table past a stream's pages and
 * entries of free_pages past those pushed are left as they were, except that a
 * stream that got none has no room for this pass's rows: of the entries that
 * its pages would have taken, those that name a page of the pool (perhaps
 * another stream's by now) become -1.  gdn_attn_window and gdn_attn_commit then
 * skip the stream, and its kv_len stays.  The mixer's commits do not look at
 * pages: give them accept_row -1 for a stream whose slots are -1.
 * Pages are not counted: each is on the stack or one stream's.  A page that the
 * tables of two streams hold (gdn_attn_window reads such pages like any other)
 * would go to the stack with the first stream that lets it go, while the other
 * still reads it; streams that share pages need a caller that takes them out of
 * this call's hands.
 * n <= 4096, total_rows and n * max_blocks <= 2^30.
 */
int gdn_kv_tables(int32_t n_streams, int32_t total_rows, int32_t page_size, int32_t n_pages,
                  int32_t max_blocks, const int32_t *row_start, const int32_t *parent,
                  const int32_t *kv_len, const int32_t *page_count, const int32_t *free_count,
                  int32_t *free_pages, int32_t *block_table, int32_t *slots, int32_t *positions,
                  int32_t *page_count_out, int32_t *free_count_out, void *stream);

/*
 * What lies between the projections and attention, for any number of packed
 * rows: RMS norm of every query and key head, rotation of its first rot_dim
 * channels by the row's position, queries to q_out, keys and values to the
 * row's slot of the cache.
 *     y = x / sqrt(mean(x^2) + eps) * norm,
 *     (a, b) -> rot_scale (a cos t - b sin t, b cos t + a sin t),
 *     t = positions[r] * inv_freq[i],  i < rot_dim / 2,
 * with (a, b) channels (i, i + rot_dim/2), or (2i, 2i+1) if interleaved.  A
 * scaling for long contexts is in the caller's inv_freq and rot_scale.  Values
 * are stored as they are.
 *   q [rows] x [hq][d], k, v [rows] x [hkv][d] bf16 with row and head strides
 *     in elements (multiples of 8; 16-byte aligned), so that they may lie in
 *     one projection's rows
 *   q_norm, k_norm [d] fp32, or NULL for no norm;  inv_freq [rot_dim/2] fp32
 *   positions, slots [rows] int32 (gdn_kv_tables); a row whose slot is outside
 *     the cache stores no key and value
 *   q_out [rows][hq][d] bf16
 * GDN_KV_E4M3 rows get scale = max(max|y|, 2^-100) / 448 and codes y / scale,
 * an fp32 quotient, rounded to nearest.  GDN_KV_MXFP4 blocks get, from the bits
 * of amax = max|y| over their 32 channels in fp32,
 *     e = min(max(((bits(amax) + 2^21) >> 23) - 2, 25), 252)
 * (so that amax / 2^(e - 127) is in [3.5, 7), what rounds to 4 or 6) and codes
 * y / 2^(e - 127) rounded to nearest, ties to even, at most 6; a block with an
 * infinite or NaN value gets e = 255 and codes 0.  There y is a key's norm and
 * rotation in fp64 from the bf16 inputs, with one rounding to fp32.  No two rows
 * may have the same slot.  rows < 2^24.
 */
typedef struct gdn_rope {
    const float *inv_freq;   /* [rot_dim / 2], device */
    int32_t rot_dim;         /* even, 0 .. d          */
    int32_t interleaved;
    float rot_scale;
} gdn_rope;

int gdn_attn_prep(const gdn_kv_cache *cache, int32_t rows, int32_t hq, const uint16_t *q,
                  int64_t q_row_stride, int64_t q_head_stride, const uint16_t *k,
                  int64_t k_row_stride, int64_t k_head_stride, const uint16_t *v,
                  int64_t v_row_stride, int64_t v_head_stride, const float *q_norm,
                  const float *k_norm, float eps, const gdn_rope *rope, const int32_t *positions,
                  const int32_t *slots, uint16_t *q_out, void *stream);

/*
 * Attention of one-row steps, verify windows and draft trees over the cache,
 * whose rows of this pass are already stored (gdn_attn_prep).  Row t of stream
 * s sees the stream's kv_len[s] cached rows, itself, and the rows before it in
 * the window, or, with parents, its ancestors:
 *     out = sigmoid(gate) * softmax(scale q K^T) V.
 *   q, out [total_rows][hq][d] bf16;  gate bf16 with row and head strides in
 *     elements (multiples of 4; 8-byte aligned), or NULL
 *   max_rows 1..16 and max_kv (at most 2^21): bounds on every window's rows and
 *     on kv_len[s] + its rows; they size the launch, and total_rows is at most
 *     n_streams * max_rows (a max_kv far above all lengths costs some time)
 *   workspace: gdn_attn_workspace_bytes() of device memory, 16-byte aligned
 *     (NULL where that is 0); its contents need not be kept between calls, and
 *     calls that may overlap need their own.  A size serves every call with the
 *     same hq, hkv and d whose n_streams, total_rows, max_rows and max_kv are no
 *     larger (a call may need less than it); 0 also for what is refused
 * A stream that breaks a rule (window, parents, lengths over max_kv or
 * max_blocks, a page outside the cache) is skipped: its rows of out are left as
 * they were, and so are rows of no stream.  Scores, softmax statistics and sums
 * are in fp32; the weights go into the product with the values to 2^-15 where a
 * window has up to 16 columns (max_rows * hq / hkv), and in bf16 (2^-8, as the
 * result's own rounding) where it has more.  A stream's results depend on
 * neither the other streams of the call nor its place in it, bit for bit, for
 * the same max_rows.  A row takes nothing from rows that it does not see,
 * whatever they hold.  total_rows * hq <= 2^26 - 4.
 */
size_t gdn_attn_workspace_bytes(const gdn_kv_cache *cache, int32_t n_streams, int32_t total_rows,
                                int32_t max_rows, int32_t max_kv, int32_t hq);

int gdn_attn_window(const gdn_kv_cache *cache, int32_t n_streams, int32_t total_rows,
                    int32_t max_rows, int32_t max_kv, int32_t max_blocks, int32_t hq,
                    const int32_t *row_start, const int32_t *parent, const int32_t *kv_len,
                    const int32_t *block_table, const uint16_t *q, const uint16_t *gate,
                    int64_t gate_row_stride, int64_t gate_head_stride, float scale, uint16_t *out,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * Attention of whole prompts, fresh (kv_len[s] 0), resumed, or in pieces, packed
 * rows of any lengths whose keys and values are already stored (gdn_attn_prep):
 * row t of stream s sees cache rows 0 .. kv_len[s] + t,
 *     out = sigmoid(gate) * softmax(scale q K^T) V.
 *   q, out [total_rows][hq][d] bf16;  gate as in gdn_attn_window
 *   max_kv (at most 2^21): a bound on kv_len[s] + the stream's rows
 *   workspace: gdn_attn_prompt_workspace_bytes() of device memory, 16-byte
 *     aligned (NULL where that is 0); its contents need not be kept between
 *     calls, and calls that may overlap need their own.  A size serves every call
 *     with the same hq, hkv and d whose total_rows and max_kv are no larger, so it
 *     is what the most chunks of such calls take (up to 271 MB for d 256), also
 *     where the call itself is not cut and uses none of it; 0 also for what is
 *     refused
 * A stream without rows has nothing to do; one that breaks a rule (its window,
 * lengths over max_kv or max_blocks, a page outside the cache) is skipped: its
 * rows of out are left as they were, and so are rows of no stream.  Scores,
 * softmax statistics and sums are in fp32; the weights go into the product with
 * the values in bf16, rounded to nearest (2^-8 at most, as the result's own
 * rounding).  A call of few rows over long streams is cut along the keys, by
 * total_rows, max_kv, the heads and the cache's format alone; given these, a
 * stream's results depend on neither the other streams nor its place in the call,
 * bit for bit.  So bounds far above what the streams have, as a captured pass may
 * need them, leave long streams in few pieces or one: 512 rows over 32,000 keys (24
 * and 4 heads of 256) take 0.38 ms under their own bounds and 1.45 under a max_kv of
 * 262,144, with room for 8,306 rows, or beside as many fresh rows.  A row takes
 * nothing from rows that it does not see, whatever they hold.  Streams of a row or
 * two are taken, but each has tiles of 128 or 256 (row, head) pairs to itself: steps
 * belong into gdn_attn_window.  total_rows * hq <= 2^26 - 4.
 */
size_t gdn_attn_prompt_workspace_bytes(const gdn_kv_cache *cache, int32_t n_streams, int32_t total_rows,
                                       int32_t max_kv, int32_t hq);

int gdn_attn_prompt(const gdn_kv_cache *cache, int32_t n_streams, int32_t total_rows, int32_t max_kv,
                    int32_t max_blocks, int32_t hq, const int32_t *row_start, const int32_t *kv_len,
                    const int32_t *block_table, const uint16_t *q, const uint16_t *gate,
                    int64_t gate_row_stride, int64_t gate_head_stride, float scale, uint16_t *out,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * Cached rows read back, in any format: packed row row_start[s] + t of k_out and
 * v_out gets the values of cache row first[s] + t of stream s (a prompt's rows to
 * be kept outside the pool, or a working copy).  Written again by gdn_attn_prep
 * without norms and rotation, rows of a bf16 cache come back bit for bit.
 *   row_start [n+1], first [n] int32;  k_out, v_out [total_rows][hkv][d] bf16
 * E4M3 values are rounded to bf16 from the fp32 product of code and scale; the
 * other formats' are exact.  A stream whose rows would end past total_rows or its
 * block table, or with first[s] < 0, and a row whose page is outside the cache,
 * are left out: their rows of k_out and v_out stay as they were, and so do rows
 * of no stream.  total_rows < 2^24.
 */
int gdn_kv_read(const gdn_kv_cache *cache, int32_t n_streams, int32_t total_rows, int32_t max_blocks,
                const int32_t *row_start, const int32_t *first, const int32_t *block_table, uint16_t *k_out,
                uint16_t *v_out, void *stream);

/*
 * Commit of the accepted rows in the cache, beside gdn_commit or
 * gdn_commit_replay: the rows of the path that ends at accept_row[s] (a packed
 * row of the stream's window, or -1 to keep none), root first, move to cache
 * rows kv_len[s], kv_len[s] + 1, ..., and kv_len_out[s] = kv_len[s] + their
 * number.  parent NULL: chains (nothing moves).  kv_len_out may be kv_len.  A
 * stream whose accepted row or layout breaks the rules, or whose window has a
 * page outside the cache, keeps its length, and none of its rows move.
 * n_streams < 2^24.
 */
int gdn_attn_commit(const gdn_kv_cache *cache, int32_t n_streams, int32_t total_rows,
                    int32_t max_rows, int32_t max_blocks, const int32_t *row_start,
                    const int32_t *parent, const int32_t *accept_row, const int32_t *kv_len,
                    const int32_t *block_table, int32_t *kv_len_out, void *stream);

/*
 * Host-side check of a window or tree layout (HOST copies of row_start and,
 * for trees, parent; parent may be NULL for chains).  Returns GDN_OK or
 * GDN_EINVAL with gdn_last_error() naming the first broken rule.
 */
int gdn_check_layout(int32_t n_streams, int32_t total_rows, int32_t max_rows,
                     const int32_t *row_start_host, const int32_t *parent_host);

#ifdef __cplusplus
}
#endif

#endif /* LIBGDN_H */
