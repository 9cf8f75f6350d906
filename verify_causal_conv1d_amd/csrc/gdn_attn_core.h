// What the attention kernels share: the rules by which a stream's keys are cut
// into chunks, how a workgroup finds its piece of work, masks, results and
// transposing LDS reads.
#pragma once

#include "gdn_attn.h"
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {

constexpr int kTile = 32;                  // keys of a wave's step
constexpr int kCols = 16;                  // (row, head) pairs of a column tile
constexpr int kMaxChunks = 64;             // of one stream

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// a / b for 0 <= a < 2^22 and 0 < b: on the device by a reciprocal, whose
// quotient is off by one at most, and a correction (the integer sequence is four
// times as long, and a short call is little else).
__host__ __device__ inline int small_div(int a, int b)
{
#ifdef __HIP_DEVICE_COMPILE__
    const int q = (int)((float)a * __builtin_amdgcn_rcpf((float)b)), r = a - q * b;
    return q + (r >= b) - (r < 0);
#else
    return a / b;
#endif
}
__host__ __device__ inline int small_ceil_div(int a, int b) { return small_div(a + b - 1, b); }
__host__ __device__ inline int at_least(int a, int b) { return a > b ? a : b; }
__host__ __device__ inline int at_most(int a, int b) { return a < b ? a : b; }

// The most keys that a chunk of a stream with len keys is to have: at least
// kChunkLeast; more once there are 4 of them, up to chunk_usual; more again once
// there are 32, up to chunk_long; and more than that once there are kMaxChunks.
// Short chunks spread a lone stream over the chip, long ones write fewer parts
// and begin less often: 64 steps of 2,000 to 4,096 keys take 164 us in chunks of
// 256 and 186 in chunks of 128, one step of 500 keys 15.5 and 13.4; 16 steps of
// up to 16,384 keys 82 us in chunks of 256 and 77 of 512; a tree of 8 rows over
// 500 keys 27 us in one wide chunk and 17 in chunks of 128.
constexpr int kChunkLeast = 128;
__host__ __device__ inline int chunk_usual(bool wide) { return wide ? 512 : 256; }
__host__ __device__ inline int chunk_long(bool wide) { return wide ? 1024 : 512; }

__host__ __device__ inline int chunk_most(int len, bool wide)
{
    const int a = at_least(kChunkLeast, at_most(chunk_usual(wide), ceil_div(len, 4)));
    const int b = at_least(a, at_most(chunk_long(wide), ceil_div(len, 32)));
    return at_least(b, ceil_div(len, kMaxChunks));
}

// Its keys: equal chunks, in whole units.  Up to a sixteenth more than the most is
// allowed, so that a few rows past a round number do not make another chunk; but
// in whole units, too, which is nothing before the most is sixteen units (wide:
// from 32,737 keys, else from 131,009).  Below that they do make one: 8,200 keys
// are 16 wide chunks of 512 and one of 8.
__host__ __device__ inline int chunk_unit(bool wide) { return wide ? 64 : 128; }
__host__ __device__ inline int chunk_keys(int len, bool wide)
{
    const int most = chunk_most(len, wide), unit = chunk_unit(wide);
    return unit * ceil_div(small_ceil_div(len, small_ceil_div(len, most + most / 16 / unit * unit)), unit);
}

__host__ __device__ inline int chunk_count(int len, bool wide) { return len <= 0 ? 0 : small_ceil_div(len, chunk_keys(len, wide)); }

// The most chunks that a stream of up to max_kv keys can have.
inline int chunk_bound(int max_kv, bool wide)
{
    const int n = at_least(at_most(4, ceil_div(max_kv, kChunkLeast)), at_most(32, ceil_div(max_kv, chunk_usual(wide))));
    return at_most(kMaxChunks, at_least(n, ceil_div(max_kv, chunk_long(wide))));
}

inline bool is_wide(int max_rows, int group) { return max_rows * group > kCols; }

// A stream's window by the layout rules that need no parents: false skips it.
__device__ __forceinline__ bool stream_window(const AttnArgs &A, int s, int &r0, int &m, int &kv)
{
    r0 = A.row_start[s];
    const int r1 = A.row_start[s + 1];
    kv = A.kv_len[s];
    m = r1 - r0;
    return r0 >= 0 && r1 > r0 && r1 <= A.total_rows && m <= A.max_rows && kv >= 0 && kv <= A.max_kv - m
           && (long long)kv + m <= (long long)A.max_blocks << A.kv.page_shift;
}

// Bits of the window's rows that row t sees (itself and its ancestors);
// ok = false if a parent breaks the rules.  Lane u < m holds row u.
__device__ __forceinline__ uint32_t seen_rows(const AttnArgs &A, int r0, int m, int t, bool &ok)
{
    if (!A.parent) return (2u << t) - 1;
    const int lane = threadIdx.x & 63;
    const int up = lane < m ? A.parent[r0 + lane] : -1;
    ok = ok && !__ballot(lane < m && (up < -1 || up >= lane));
    uint32_t bits = 1u << t;
    if (ok)
        for (int u = m - 1; u >= 0; --u) {     // parents come before their rows
            const int p = __builtin_amdgcn_readlane(up, u);
            if (p >= 0 && (bits >> u & 1)) bits |= 1u << p;
        }
    return bits;
}

// The thread's number, as a value that the compiler cannot trace: what is worked
// out from it inside a loop stays there, instead of taking registers from the
// accumulators all through it.
__device__ __forceinline__ int fresh(int x)
{
    asm volatile("" : "+v"(x));
    return x;
}

__device__ __forceinline__ float max_rows4(float x)     // over lanes l, l ^ 16, l ^ 32, l ^ 48
{
    const uint32_t xi = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane16_swap(xi, xi, false, false);
    const float s = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t si = __float_as_uint(s);
    const auto q = __builtin_amdgcn_permlane32_swap(si, si, false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// the gates of 4 channels (none: all ones, which finish4 does not look at)
__device__ __forceinline__ uint2 gates4(const AttnArgs &A, int r, int head, int d)
{
    return A.gate ? *reinterpret_cast<const uint2 *>(A.gate + r * A.gate_row + head * A.gate_head + d) : make_uint2(0, 0);
}

// the result of one (row, head) column's 4 channels: o / l, gated, in bf16
__device__ __forceinline__ uint2 finish4(const AttnArgs &A, float4 o, float inv, uint2 g)
{
    float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    if (A.gate) {
        x[0] *= sigmoid_f(__uint_as_float(g.x << 16));
        x[1] *= sigmoid_f(__uint_as_float(g.x & 0xffff0000u));
        x[2] *= sigmoid_f(__uint_as_float(g.y << 16));
        x[3] *= sigmoid_f(__uint_as_float(g.y & 0xffff0000u));
    }
    return make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
}

// What a stream's skipped chunk leaves in the workspace for join_kernel: sums
// are never negative.
constexpr float kSkipped = -1.0f;

// Sum over the lanes up to and including this one: row_shr within the 16-lane
// rows, then row_bcast of a row's last lane to the rows after it.
__device__ __forceinline__ int wave_running_sum(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return x;
}

// One piece of work: a chunk of a stream's keys, for one kv head and one tile of
// columns.
struct Chunk {
    int h, rt, c;             // kv head, tile of columns, chunk
    int s, r0, m, kv, len;    // the stream, its window, cached rows, keys in all
    int k0, k1, nch;          // the chunk's keys, and chunks of the stream
    int size;                 // keys of a full chunk
    int cols;                 // (row, head) pairs of the stream
};

// The pieces of all streams, in stream order.  How many there are follows from
// the lengths, which only the device knows.  Every wave finds its pieces by
// itself: lane l holds stream first + l of a block of 64 streams, and the pieces
// of the block up to and including that stream's.  Within a block no workgroup
// for a piece that is not there comes before those that are.  attn_kernel's grid
// has room for max_kv keys of every stream, a row of workgroups a block, and those
// that find nothing end at once, but are not free: 512 steps of 500 keys take 264
// us under a max_kv of 501 and 423 under 262,144, 16 such steps 15.7 and 18.1.
struct Pieces {
    int first = -64, before = 0, incl = 0;    // of the block: first stream, pieces before it, running sum
    int r0 = 0, m = 0, kv = 0;

    __device__ __forceinline__ void load(const AttnArgs &A, bool wide, int tile_cols, int block)
    {
        const int lane = threadIdx.x & 63, s = block + lane;
        first = block;
        int count = 0;
        if (s < A.n_streams && stream_window(A, s, r0, m, kv))
            count = chunk_count(kv + m, wide) * A.kv.hkv * ceil_div(m * A.group, tile_cols);
        incl = wave_running_sum(count);
    }

    // piece `at` of the block's
    __device__ __forceinline__ void get(const AttnArgs &A, bool wide, int at, Chunk &K) const
    {
        const int l = __builtin_ctzll(__ballot(incl > at));
        const int x = at - (l ? __builtin_amdgcn_readlane(incl, l - 1) : 0);
        K.s = first + l;
        K.r0 = __builtin_amdgcn_readlane(r0, l);
        K.m = __builtin_amdgcn_readlane(m, l);
        K.kv = __builtin_amdgcn_readlane(kv, l);
        K.len = K.kv + K.m;
        K.size = chunk_keys(K.len, wide);
        K.nch = small_ceil_div(K.len, K.size);
        K.cols = K.m * A.group;
        // the stream's pieces: chunks innermost (at most 64 * 1024 * 128 of them)
        const int y = x < 1 << 22 ? small_div(x, K.nch) : x / K.nch;
        K.c = x - y * K.nch;
        K.rt = small_div(y, A.kv.hkv);
        K.h = y - K.rt * A.kv.hkv;
        K.k0 = K.c * K.size;
        K.k1 = min(K.k0 + K.size, K.len);
    }

    // piece `at` of the block of 64 streams from `block`; false if it has fewer
    __device__ __forceinline__ bool find_in_block(const AttnArgs &A, bool wide, int tile_cols, int block, int at, Chunk &K)
    {
        load(A, wide, tile_cols, block);
        if (at >= __builtin_amdgcn_readlane(incl, 63)) return false;
        get(A, wide, at, K);
        return true;
    }

    // piece `item` of all (not less than in the call before); false if there is none
    __device__ __forceinline__ bool find(const AttnArgs &A, bool wide, int tile_cols, int item, Chunk &K)
    {
        while (item >= before + __builtin_amdgcn_readlane(incl, 63)) {
            before += __builtin_amdgcn_readlane(incl, 63);
            if (first + 64 >= A.n_streams) return false;
            load(A, wide, tile_cols, first + 64);
        }
        get(A, wide, item - before, K);
        return true;
    }
};

// Cache rows of the chunk's keys, 16 at a time (pages hold multiples of 16) up
// to the chunk's full size: past the stream's end those of its last keys, so
// that every load stays in its pages.  false if a page is not in the cache.
// (For the caller's wave: whether its share of them is.)
__device__ __forceinline__ bool chunk_rows(const AttnArgs &A, const Chunk &K, int *rows16, int threads)
{
    bool ok = true;
    for (int i = threadIdx.x; i < K.size / 16; i += threads) {
        const int key = min(K.k0 + 16 * i, (K.len - 1) & ~15);
        const int id = A.table[(size_t)K.s * A.max_blocks + (key >> A.kv.page_shift)];
        const bool good = id >= 0 && id < A.kv.n_pages;
        ok = ok && good;
        rows16[i] = good ? ((id * A.kv.hkv + K.h) << A.kv.page_shift) + (key & ((1 << A.kv.page_shift) - 1)) : 0;
    }
    return !__ballot(!ok);
}

// Entries of the block table, which nothing writes while the kernel runs, through
// the scalar cache: their addresses are the wave's.
typedef const __attribute__((address_space(4))) int const_int;
__device__ __forceinline__ int table_entry(const int *table, int i) { return ((const_int *)table)[i]; }

// Packed row and query head of a stream's column.
__device__ __forceinline__ int col_row(const AttnArgs &A, const Chunk &K, int col) { return K.r0 + small_div(col, A.group); }
__device__ __forceinline__ int col_head(const AttnArgs &A, const Chunk &K, int col) { return K.h * A.group + col - small_div(col, A.group) * A.group; }
// and its place in the workspace
__device__ __forceinline__ size_t col_part(const AttnArgs &A, const Chunk &K, int col)
{
    return ((size_t)col_row(A, K, col) * A.hq + col_head(A, K, col)) * A.chunks + K.c;
}

// A column's 4 channels from d: the result where the chunk is the stream's only
// one, else its part in the workspace.
template <int D>
__device__ __forceinline__ void put4(const AttnArgs &A, const Chunk &K, int col, float4 a, float l, int d)
{
    const int r = col_row(A, K, col), hd = col_head(A, K, col);
    if (K.nch == 1) *reinterpret_cast<uint2 *>(A.out + ((size_t)r * A.hq + hd) * D + d) = finish4(A, a, 1.0f / l, gates4(A, r, hd, d));
    else *reinterpret_cast<float4 *>(A.part + col_part(A, K, col) * D + d) = a;
}

typedef const __attribute__((address_space(1))) void global_void;
typedef __attribute__((address_space(3))) void lds_void;
constexpr int kOnce = 2;        // the nontemporal bit of a load's cache policy

// Waits until all but the newest N vector memory operations of the wave and all
// of its LDS reads are done, then for the workgroup's other waves.
template <int N>
__device__ __forceinline__ void wait_and_meet()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);     // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

typedef short s4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4v lds_s4v;

// Transposing LDS read: each group of 16 lanes brings four 16-element rows, lane
// 4 r + c elements 4 c .. 4 c + 3 of row r; lane i gets element i of the four.
__device__ __forceinline__ s4v read_transposed(const uint8_t *p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v *)(s4v *)p);
}

// The same of bytes: eight 16-byte rows, lane 2 r + c bytes 8 c .. 8 c + 7 of row
// r; lane i gets byte i of the eight.
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v2i lds_v2i;
__device__ __forceinline__ v2i read_transposed_codes(const uint8_t *p)
{
    return __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(v2i *)p);
}

}  // namespace gdn
