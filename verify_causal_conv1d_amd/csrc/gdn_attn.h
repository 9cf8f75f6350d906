// Internal declarations of libgdn's attention-layer operators: block tables
// and slot maps, norms + rotation + cache writes, paged attention, commits.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// A paged cache: K and V of [pages][hkv][page_size][d], bf16, e4m3 with one fp32
// scale a row in [pages][hkv][page_size], or e2m1 (two codes a byte) with an
// exponent byte for every 32 channels in [pages][hkv][page_size][d / 32].
struct KvArgs {
    uint8_t *k, *v;
    float *k_scale, *v_scale;   // e4m3 only
    int32_t n_pages, page_shift, hkv, d;
    uint8_t *k_exp, *v_exp;     // e2m1 only
};
enum { FMT_BF16 = 0, FMT_E4M3 = 1, FMT_MXFP4 = 2 };
inline int format_of(const KvArgs &K) { return K.k_exp ? FMT_MXFP4 : K.k_scale ? FMT_E4M3 : FMT_BF16; }

struct TablesArgs {
    int32_t n_streams, total_rows, page_shift, max_blocks, n_pages;
    const int32_t *row_start, *parent, *kv_len, *page_count, *free_count;
    int32_t *free_pages, *table, *slots, *positions, *page_count_out, *free_count_out;
};

struct PrepArgs {
    KvArgs kv;
    int32_t rows, hq, rot, interleaved;
    const uint16_t *q, *k, *v;                        // bf16, strides in elements
    int64_t q_row, q_head, k_row, k_head, v_row, v_head;
    const float *q_norm, *k_norm, *inv_freq;
    float eps, rot_scale;
    const int32_t *positions, *slots;
    uint16_t *q_out;
};

struct AttnArgs {
    KvArgs kv;
    int32_t n_streams, total_rows, max_rows, max_kv, max_blocks;
    int32_t hq, group;           // query heads, and query heads of a kv head
    int32_t chunks;              // chunks the longest stream has: partials are [total_rows][hq][chunks]
    const int32_t *row_start, *parent, *kv_len, *table;
    const uint16_t *q, *gate;    // q [total_rows][hq][d]; gate strided, or NULL
    int64_t gate_row, gate_head;
    float scale;                 // of the scores, with log2(e)
    uint16_t *out;
    float *part;                 // [total_rows][hq][chunks][d]
    float2 *stat;                // [total_rows][hq][chunks]: running maximum (base 2), sum
};

struct AttnCommitArgs {
    KvArgs kv;
    int32_t n_streams, total_rows, max_rows, max_blocks;
    const int32_t *row_start, *parent, *accept, *kv_len, *table;
    int32_t *kv_len_out;
};

struct ReadArgs {
    KvArgs kv;
    int32_t n_streams, total_rows, max_blocks;
    const int32_t *row_start, *first, *table;
    uint16_t *k_out, *v_out;     // [total_rows][hkv][d]
};

constexpr int kMaxAttnKeys = 1 << 21;    // of one stream: a workgroup lists its chunk's pages in LDS
constexpr int kMaxGroups = (1 << 24) - 1;  // workgroups of 256 threads: a launch has less than 2^32 threads
constexpr int kMaxTableStreams = 4096;   // a workgroup keeps six ints of each in LDS

// of a pass with just these bounds; it does not grow with max_rows
size_t attn_workspace_bytes(int hq, int hkv, int d, int total_rows, int max_rows, int max_kv);

bool attn_fits(const AttnArgs &A);   // the launch's workgroups can be numbered

hipError_t launch_tables(const TablesArgs &A, hipStream_t stream);
hipError_t launch_prep(const PrepArgs &A, hipStream_t stream);
hipError_t launch_attn(AttnArgs A, void *workspace, hipStream_t stream);

// Attention of whole prompts: max_rows is not looked at.  The workspace of a call,
// and one that is enough for all calls with no larger sizes.
size_t prompt_workspace_bytes(int hq, int hkv, int d, int fmt, int n_streams, int total_rows, int max_kv);
size_t prompt_workspace_most(int hq, int d, int total_rows, int max_kv);
bool prompt_fits(const AttnArgs &A);
hipError_t launch_prompt(AttnArgs A, void *workspace, hipStream_t stream);
// Windows of more than 16 columns over a 4-bit cache, in the chunks of the others
hipError_t launch_wide4(const AttnArgs &A, long long pieces, hipStream_t stream);
// Merges the chunks of every (row, head); split_keys 0: chunks of windows
hipError_t launch_join(const AttnArgs &A, bool wide, int split_keys, hipStream_t stream);
hipError_t launch_read(const ReadArgs &A, hipStream_t stream);
hipError_t launch_attn_commit(const AttnCommitArgs &A, hipStream_t stream);

}  // namespace gdn
