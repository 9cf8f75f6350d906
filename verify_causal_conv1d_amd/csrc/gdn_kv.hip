// The paged key-value cache of the attention layers: block tables and slot
// maps from request lengths (tables_kernel), norms and rotation of queries and
// keys with the cache writes (prep_kernel), and the commit of accepted tree
// paths (attn_commit_kernel), and cached rows read back (read_kernel).  Contracts are
// in include/libgdn.h.
#include "gdn_attn.h"
#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_mxfp4.h"
#include "gdn_once.h"

namespace gdn {
namespace {

// ---- block tables and slot maps ------------------------------------------
//
// Stream s holds have_s pages and needs want_s = ceil((kv_len_s + rows_s) /
// page) (none once it has finished, kv_len_s < 0).  With the exclusive sums
//     D_s = sum_{i<s} max(have_i - want_i, 0),   G_s = sum_{i<s} max(want_i - have_i, 0)
// the released pages go to free_pages[free + D_s ...] and, with avail = free +
// sum of all drops, page have_s + i of a growing stream is
// free_pages[avail - 1 - G_s - i].  A stream with G_s + grow_s > avail gets none,
// and page numbers that earlier rounds left in the entries it asked for become
// -1: they may be pages that other streams hold by now, and attention and commit
// know a stream without room by these entries alone.
//
// Every workgroup computes the sums for itself (n streams are a few KB) and
// takes its share of the pages and rows.  A page taken that is released by the
// same call is read from the releasing stream's table, not from free_pages, so
// no workgroup waits for another's writes: nothing that one of them reads is
// written in the launch, except the counts where they are updated in place.
// Those then come from a second launch (counts only); the last workgroup writes
// them where they go elsewhere, or where a single one does it all.
constexpr int kTablesThreads = 1024, kTablesBlocks = 32;

struct TableStreams {          // LDS, n entries each (start: n + 1)
    int *start, *kv, *have, *want, *drop, *grow;
};

__device__ __forceinline__ int find_last(const int *pre, int n, int x)
{
    // the last index i in [0, n) with pre[i] <= x (pre does not decrease, pre[0] <= x)
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (pre[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ __launch_bounds__(kTablesThreads) void tables_kernel(const TablesArgs A, const int do_counts, const int do_rest)
{
    extern __shared__ int lds[];
    __shared__ long long wave_sum[kTablesThreads / 64];
    __shared__ int falls;                                  // row_start decreases somewhere
    const int n = A.n_streams, tid = threadIdx.x;
    const TableStreams S = {lds, lds + n + 1, lds + 2 * n + 1, lds + 3 * n + 1, lds + 4 * n + 1, lds + 5 * n + 1};
    const int page = 1 << A.page_shift;
    const bool counts_too = do_counts && blockIdx.x == gridDim.x - 1;

    for (int s = tid; s <= n; s += kTablesThreads) S.start[s] = A.row_start[s];
    if (tid == 0) falls = 0;
    __syncthreads();
    // each thread a run of streams: (drop | grow << 32) summed over it
    const int per = (n + kTablesThreads - 1) / kTablesThreads;
    const int s0 = min(tid * per, n), s1 = min(s0 + per, n);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
        const int a = S.start[s], b = S.start[s + 1], kv = A.kv_len[s], have = A.page_count[s];
        const int cap = A.max_blocks << A.page_shift;      // checked on the host to fit 31 bits
        int want = have;
        // a stream that breaks the rules keeps its pages and gets no slots (kv = -1)
        const bool ok = a >= 0 && b >= a && b <= A.total_rows && have >= 0 && have <= A.max_blocks
                        && (kv < 0 || (kv <= cap && b - a <= cap - kv));     // finished: no room needed
        if (ok) want = kv < 0 ? 0 : (kv + (b - a) + page - 1) >> A.page_shift;
        if (b < a) falls = 1;
        S.kv[s] = ok ? kv : -1;
        S.have[s] = have;
        S.want[s] = want;
        mine += (long long)max(have - want, 0) + ((long long)max(want - have, 0) << 32);
    }
    // exclusive sums over the threads, in stream order
    long long incl = mine;
    for (int o = 1; o < 64; o <<= 1) {
        const long long up = __shfl_up(incl, o);
        if ((tid & 63) >= o) incl += up;
    }
    if ((tid & 63) == 63) wave_sum[tid >> 6] = incl;
    __syncthreads();
    long long before = incl - mine, all = 0;
    for (int w = 0; w < kTablesThreads / 64; ++w) {
        if (w < (tid >> 6)) before += wave_sum[w];
        all += wave_sum[w];
    }
    for (int s = s0; s < s1; ++s) {
        S.drop[s] = (int)before;
        S.grow[s] = (int)(before >> 32);
        const int have = S.have[s], want = S.want[s];
        before += (long long)max(have - want, 0) + ((long long)max(want - have, 0) << 32);
    }
    const int drops = (int)all, grows = (int)(all >> 32);
    int free0 = *A.free_count;
    if (free0 < 0 || free0 > A.n_pages) free0 = 0;         // a broken list is taken as empty
    const int avail = (int)min((long long)free0 + drops, (long long)A.n_pages);
    __syncthreads();
    // Streams get pages in order; the first whose run ends past the list, and
    // all that grow after it, get none: grow[s] <= cut says which did.
    auto served = [&](int s) { return S.grow[s] + max(S.want[s] - S.have[s], 0) <= avail || S.want[s] <= S.have[s]; };
    auto free_page = [&](int p) {                          // entry p of the list with the released pages on top
        if (p < free0) return A.free_pages[p];
        const int s = find_last(S.drop, n, p - free0);
        return A.table[(size_t)s * A.max_blocks + S.want[s] + (p - free0 - S.drop[s])];
    };

    if (do_rest) {
        const int step = gridDim.x * kTablesThreads, first = blockIdx.x * kTablesThreads + tid;
        // find_last gives the LAST stream of a run of equal sums: for item i
        // that is the one stream whose run holds i
        for (int i = first; i < drops; i += step) {
            const int s = find_last(S.drop, n, i);
            if (free0 + i < A.n_pages)
                A.free_pages[free0 + i] = A.table[(size_t)s * A.max_blocks + S.want[s] + (i - S.drop[s])];
        }
        for (int i = first; i < grows; i += step) {
            const int s = find_last(S.grow, n, i);
            int32_t &entry = A.table[(size_t)s * A.max_blocks + S.have[s] + (i - S.grow[s])];
            if (served(s)) entry = free_page(avail - 1 - i);
            else if (entry >= 0 && entry < A.n_pages) entry = -1;
        }
        // every packed row: a captured pass with fewer rows than it has room for
        // must not leave the slots of an earlier one behind
        for (int r = first; r < A.total_rows; r += step) {
            int s = n > 0 ? find_last(S.start, n, r) : 0;
            if (falls)               // a broken layout does not hide the streams that keep the rules
                for (s = 0; s < n - 1 && !(S.kv[s] >= 0 && r >= S.start[s] && r < S.start[s + 1]);) ++s;
            const int a = S.start[s], t = r - a;
            int slot = -1, pos = -1;
            if (n > 0 && t >= 0 && r < S.start[s + 1] && S.kv[s] >= 0 && served(s)) {
                const int kv = S.kv[s];
                const int at = kv + t, b = at >> A.page_shift;
                const int id = b < S.have[s] ? A.table[(size_t)s * A.max_blocks + b] : free_page(avail - 1 - S.grow[s] - (b - S.have[s]));
                int depth = t;
                bool ok = id >= 0 && id < A.n_pages;
                if (A.parent) {
                    // the window's parents, each + 1 in four bits (p < u <= 15), then the walk up
                    const int m = S.start[s + 1] - a;
                    ok = ok && m <= kMaxWindowRows;
                    uint64_t up = 0;
#pragma unroll
                    for (int u = 0; u < kMaxWindowRows; ++u)
                        if (ok && u < m) {
                            const int p = A.parent[a + u];
                            ok = p >= -1 && p < u;
                            up |= (uint64_t)((p + 1) & 15) << (4 * u);
                        }
                    depth = 0;
                    for (int u = t; ok && (u = (int)(up >> (4 * u) & 15) - 1) >= 0;) ++depth;
                }
                if (ok) {
                    slot = (id << A.page_shift) + (at & (page - 1));
                    pos = kv + depth;
                }
            }
            A.slots[r] = slot;
            A.positions[r] = pos;
        }
    }
    if (counts_too) {
        // taken = the end of the last served run
        for (int s = s0; s < s1; ++s) {
            A.page_count_out[s] = served(s) ? S.want[s] : S.have[s];
        }
        __shared__ int taken;
        if (tid == 0) taken = 0;
        __syncthreads();
        int mx = 0;
        for (int s = s0; s < s1; ++s)
            if (S.want[s] > S.have[s] && served(s)) mx = max(mx, S.grow[s] + S.want[s] - S.have[s]);
        if (mx) atomicMax(&taken, mx);
        __syncthreads();
        if (tid == 0) *A.free_count_out = avail - taken;
    }
}

// ---- norms, rotation and cache writes ------------------------------------
//
// One workgroup a packed row.  A lane holds 8 consecutive channels of one head
// (one 16-byte load), so d / 8 lanes share a head; the mean square is summed
// over them by lane moves.  The row's cosines and sines are worked out once
// and shared by its heads through LDS: the angle pos * inv_freq needs fp64 (at
// position 2^18 its fp32 rounding alone is 1/64 rad), taken there to
// revolutions and reduced, then sincospif of the fraction.
constexpr int kPrepThreads = 256;
constexpr int kPrepFewRows = 512;
constexpr int kPrepMaxHalf = 128;                  // rotated pairs of a head
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyMax = 0x1p-100f;              // the least row maximum a scale is made from (1 / 2^-100 is finite)

template <int LANES>                               // sum over aligned groups of 8, 16 or 32 lanes
__device__ __forceinline__ float sum_group(float x)
{
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xF, 0xF, false));
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xF, 0xF, false));
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xF, 0xF, false));
    if (LANES > 8) x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x140, 0xF, 0xF, false));
    if (LANES > 16) x += __shfl_xor(x, 16);
    return x;
}

template <int LANES>
__device__ __forceinline__ float max_group(float x)
{
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0xB1, 0xF, 0xF, false)));
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x4E, 0xF, 0xF, false)));
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x141, 0xF, 0xF, false)));
    if (LANES > 8) x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x140, 0xF, 0xF, false)));
    if (LANES > 16) x = fmaxf(x, __shfl_xor(x, 16));
    return x;
}

// A key head's values once more, in fp64 from its bf16 channels up to the last
// rounding: norm, then rotation.  For all lanes of a wave; those of other heads
// keep what they have.
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, false);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int LANES>
__device__ __forceinline__ double sum_group(double x)
{
    x += dpp_f64<0xB1>(x);
    x += dpp_f64<0x4E>(x);
    x += dpp_f64<0x141>(x);
    if (LANES > 8) x += dpp_f64<0x140>(x);
    if (LANES > 16) x += __shfl_xor(x, 16);
    return x;
}

// 1 / sqrt(a), a > 0: the instruction's estimate (2^-22 or better) and two steps of
// Newton's method; 0 of infinity
__device__ __forceinline__ double rsqrt_f64(double a)
{
    const double r0 = __builtin_amdgcn_rsq(a);
    double r = r0 * fma(-0.5 * a * r0, r0, 1.5);
    r = r * fma(-0.5 * a * r, r, 1.5);
    return a < INFINITY ? r : r0;
}

// cos and sin of 2 pi turns, |turns| <= 0.5, to 2^-45: quarter turns off, then the
// Taylor series on [-pi / 4, pi / 4] (their next terms are below 2^-45)
__device__ __forceinline__ void cos_sin_f64(double turns, double &c, double &s)
{
    const double q = rint(4.0 * turns), r = (turns - 0.25 * q) * 6.28318530717958647693, z = r * r;
    const double sn = r * fma(z, fma(z, fma(z, fma(z, fma(z, fma(z, 1.0 / 6227020800.0, -1.0 / 39916800.0), 1.0 / 362880.0), -1.0 / 5040.0), 1.0 / 120.0), -1.0 / 6.0), 1.0);
    const double cn = fma(z, fma(z, fma(z, fma(z, fma(z, fma(z, fma(z, -1.0 / 87178291200.0, 1.0 / 479001600.0), -1.0 / 3628800.0), 1.0 / 40320.0), -1.0 / 720.0), 1.0 / 24.0), -0.5), 1.0);
    const int n = (int)q;
    c = n & 1 ? (n & 2 ? sn : -sn) : (n & 2 ? -cn : cn);
    s = n & 1 ? (n & 2 ? -cn : cn) : (n & 2 ? -sn : sn);
}

// cos and sin of a position's ith angle, times the rotation's scale.  The angle is
// exact in fp64 for positions below 2^29 (times the 24 bits of a frequency; beyond, it
// is the product rounded to fp64), and so, up to 2^-52 of a turn, is what whole turns
// leave of it.
__device__ __forceinline__ void turn_f64(const PrepArgs &A, int pos, int i, double &c, double &s)
{
    const double angle = (double)pos * (double)A.inv_freq[i], n = rint(angle * 0.15915494309189533577);
    const double rest = fma(-n, 2.4492935982947064e-16, fma(-n, 6.28318530717958647693, angle));
    cos_sin_f64(rest * 0.15915494309189533577, c, s);
    c *= (double)A.rot_scale;
    s *= (double)A.rot_scale;
}

// A lane's 8 channels of a row, quantised with the other three lanes of their block
// of 32 (all lanes of a wave call it), and stored
template <int D>
__device__ __forceinline__ void put_block(const float (&x)[8], int lane, bool store, uint8_t *pool, uint8_t *exps, size_t row)
{
    uint32_t top = 0;               // of the bits: a NaN is above infinity
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, false));
    top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, false));
    if (!store) return;
    const bool fin = top < 0x7f800000u;
    const int e = fin ? min(max((int)((top + (1u << 21)) >> 23) - 2, kMxLeast), kMxMost) : kMxNan;
    const float to = __uint_as_float((uint32_t)(254 - e) << 23);         // 2^(127 - e)
    uint32_t codes = 0;
    if (fin) {
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[0] * to, x[1] * to, 1.0f, 0);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[2] * to, x[3] * to, 1.0f, 1);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[4] * to, x[5] * to, 1.0f, 2);
        codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, x[6] * to, x[7] * to, 1.0f, 3);
    }
    *reinterpret_cast<uint32_t *>(pool + row * (D / 2) + 4 * lane) = codes;
    if (lane % 4 == 0) exps[row * (D / kMxBlock) + lane / 4] = (uint8_t)e;
}

// A key head's values in fp64 from its bf16 channels up to the last rounding: norm,
// then rotation.  row: the head's LDS; weight: the norm's, there.
template <int D, int LANES>
__device__ __forceinline__ void exact_key(const PrepArgs &A, uint4 raw, int lane, double *row, const double *weight, const double *cs,
                                          const double *sn, float (&x)[8])
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    double inv = 1.0;
    if (A.k_norm) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double a = (double)__uint_as_float(w[i] << 16), b = (double)__uint_as_float(w[i] & 0xffff0000u);
            ss = fma(b, b, fma(a, a, ss));
        }
        inv = rsqrt_f64(sum_group<LANES>(ss) * (1.0 / D) + (double)A.eps);
    }
    // the head's normed channels change lanes through LDS, within the wave
    double z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        z[i] = (double)__uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16) * (inv * weight[8 * lane + i]);
        if (8 * lane < A.rot) row[8 * lane + i] = z[i];
    }
    __builtin_amdgcn_wave_barrier();
    if (8 * lane < A.rot) {
        const int half = A.rot / 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = 8 * lane + i;
            if (e < A.rot) {
                const bool second = A.interleaved ? e & 1 : e >= half;
                const int p = A.interleaved ? e >> 1 : second ? e - half : e;
                const double other = row[A.interleaved ? e ^ 1 : second ? e - half : e + half] * sn[p];
                z[i] = fma(z[i], cs[p], second ? other : -other);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)z[i];
    __builtin_amdgcn_wave_barrier();
}

// Rows that n (row, kv head) pairs in order belong to, at most, and the doubles that
// a key takes for its lanes' exchange (a lane puts down all of its eight)
__host__ __device__ inline int key_rows(int n, int hkv) { return (n - 1) / hkv + 2 < n ? (n - 1) / hkv + 2 : n; }

__host__ __device__ inline int key_swap(int rot) { return (rot + 7) & ~7; }

// A workgroup's keys of many rows into a 4-bit cache: pairs in order, as many as its
// lanes hold
template <int D>
__device__ __forceinline__ void prep_keys(const PrepArgs &A, const int block, double *lds64)
{
    constexpr int LANES = D / 8, HEADS = kPrepThreads / LANES;
    const int tid = threadIdx.x, lane = tid % LANES, grp = tid / LANES, hkv = A.kv.hkv, half = A.rot / 2;
    double *weight = lds64, *swap = weight + D, *cs64 = swap + HEADS * key_swap(A.rot), *sn64 = cs64 + key_rows(HEADS, hkv) * half;
    const long long first = (long long)block * HEADS, pairs = (long long)A.rows * hkv, pair = first + grp;
    const int row0 = (int)(first / hkv), r = (int)(min(pair, pairs - 1) / hkv), h = (int)(pair - (long long)r * hkv);
    const bool there = pair < pairs;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (there) raw = load_once(A.k + (r * A.k_row + h * A.k_head + 8 * lane));
    const int slot = there ? A.slots[r] : -1, page = slot >> A.kv.page_shift;
    const int rows = (int)(min(first + HEADS, pairs) - 1) / hkv - row0 + 1;
    for (int i = tid; i < rows * half; i += kPrepThreads) turn_f64(A, A.positions[row0 + i / half], i % half, cs64[i], sn64[i]);
    if (tid < D) weight[tid] = A.k_norm ? (double)A.k_norm[tid] : 1.0;
    lds_barrier();
    float x[8];
    exact_key<D, LANES>(A, raw, lane, swap + grp * key_swap(A.rot), weight, cs64 + (r - row0) * half, sn64 + (r - row0) * half, x);
    const size_t at = (((size_t)page * hkv + h) << A.kv.page_shift) + (slot & ((1 << A.kv.page_shift) - 1));
    put_block<D>(x, lane, there && slot >= 0 && page < A.kv.n_pages, A.kv.k, A.kv.k_exp, at);
}

// The rows pass through once, and what is stored is read by other kernels on
// whichever XCD: load_once and store_once (the prompt pass of 8,306 rows takes
// 62 us with them and 68 us without).
//
// Into a 4-bit cache a key's norm and rotation are taken in fp64 up to the fp32 value
// that is quantised: that close to a border between two codes or two scales fp32
// sums would decide by the order of their terms.  Where the rows are few a
// workgroup does its row's keys last (PREP_MX); else workgroups of their own, spread
// among the others, do them (PREP_MX_APART: 8,306 rows 73 us, in the rows' own
// workgroups 88, in a launch after theirs 75).
enum { PREP_ROWS = 0, PREP_MX = 1, PREP_MX_APART = 2 };

template <int D, int MODE>
__global__ __launch_bounds__(kPrepThreads, MODE == PREP_MX_APART ? 8 : 1) void prep_kernel(const PrepArgs A, const int span)
{
    constexpr bool MX = MODE != PREP_ROWS, KEYS = MODE == PREP_MX;
    constexpr int LANES = D / 8, HEADS = kPrepThreads / LANES;   // heads a workgroup handles at once
    constexpr int BATCH = 4;                                     // and loads ahead
    // this workgroup's heads: span of them from span * blockIdx.y
    __shared__ float cs[kPrepMaxHalf], sn[kPrepMaxHalf];
    __shared__ __align__(16) float swap[HEADS][D];
    __shared__ double cs64[KEYS ? kPrepMaxHalf : 1], sn64[KEYS ? kPrepMaxHalf : 1];
    __shared__ double weight[KEYS ? D : 1], swap64[KEYS ? HEADS : 1][D];     // of the keys' norm; their lanes' exchange
    int r = blockIdx.x;
    if constexpr (MODE == PREP_MX_APART) {
        // of gridDim.x workgroups A.rows have a row, as evenly spread as can be
        extern __shared__ double lds64[];
        const long long all = gridDim.x, keys = all - A.rows, before = r * keys / all;
        if ((r + 1) * keys / all > before) {
            prep_keys<D>(A, (int)before, lds64);
            return;
        }
        r -= (int)before;
    }
    const int tid = threadIdx.x, lane = tid % LANES, grp = tid / LANES;
    const int half = A.rot / 2, hkv = A.kv.hkv, first = span * blockIdx.y, heads = min(A.hq + 2 * hkv, first + span);
    const int64_t q_row = r * A.q_row, k_row = r * A.k_row, v_row = r * A.v_row;
    auto source = [&](int h) {
        return h < A.hq ? A.q + (q_row + h * A.q_head)
             : h < A.hq + hkv ? A.k + (k_row + (h - A.hq) * A.k_head) : A.v + (v_row + (h - A.hq - hkv) * A.v_head);
    };
    // into a 4-bit cache the keys come last, by themselves
    const int k_first = max(first, A.hq), k_heads = min(heads, A.hq + hkv);
    uint4 raw[BATCH], raw_k = make_uint4(0, 0, 0, 0);
    if (KEYS && k_first + grp < k_heads) raw_k = load_once(source(k_first + grp) + 8 * lane);
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int h = h0 + i * HEADS + grp;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (h < heads) raw[i] = load_once(source(h) + 8 * lane);
        }
    };
    load(first);
    const int slot = A.slots[r], pos = A.positions[r];
    if (tid < half) {
        const double turns = (double)pos * (double)A.inv_freq[tid] * 0.15915494309189533577;   // 1 / (2 pi)
        float s, c;
        sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
        cs[tid] = c * A.rot_scale;
        sn[tid] = s * A.rot_scale;
        if constexpr (KEYS) turn_f64(A, pos, tid, cs64[tid], sn64[tid]);
    }
    if constexpr (KEYS)
        if (tid < D) weight[tid] = A.k_norm ? (double)A.k_norm[tid] : 1.0;
    const int page = slot >> A.kv.page_shift, off = slot & ((1 << A.kv.page_shift) - 1);
    const bool cached = slot >= 0 && page < A.kv.n_pages;
    lds_barrier();
    // the trip count is the same for every lane of a wave's shuffles: heads past
    // the last are computed on zeros and not stored
    for (int h0 = first; h0 < heads; h0 += BATCH * HEADS) {
        if (h0 > first) load(h0);
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            if (h0 + b * HEADS >= heads) break;
            const int h = h0 + b * HEADS + grp;
            const bool is_q = h < A.hq, is_k = !is_q && h < A.hq + hkv, there = h < heads;
            const int kvh = is_k ? h - A.hq : h - A.hq - hkv;
            float x[8];
            const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            ss = sum_group<LANES>(ss);
            const float *nw = is_q ? A.q_norm : is_k ? A.k_norm : nullptr;
            if (nw) {
                const float inv = __builtin_amdgcn_rsqf(ss * (1.0f / D) + A.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * nw[8 * lane + i];
            }
            if (A.interleaved) {
                if (is_q || is_k) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int p = 4 * lane + i;
                        if (p < half) {
                            const float a = x[2 * i], c = x[2 * i + 1];
                            x[2 * i] = fmaf(a, cs[p], -(c * sn[p]));
                            x[2 * i + 1] = fmaf(c, cs[p], a * sn[p]);
                        }
                    }
                }
            } else if (8 * lane < 2 * half) {
                // partners half a rotation apart change lanes through LDS, within the wave
                float *row = swap[grp];
#pragma unroll
                for (int i = 0; i < 8; ++i) row[8 * lane + i] = x[i];
                __builtin_amdgcn_wave_barrier();
                if (is_q || is_k) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int e = 8 * lane + i;
                        if (e < half) x[i] = fmaf(x[i], cs[e], -(row[e + half] * sn[e]));
                        else if (e < 2 * half) x[i] = fmaf(x[i], cs[e - half], row[e - half] * sn[e - half]);
                    }
                }
                __builtin_amdgcn_wave_barrier();
            }
            if (is_q) {
                const uint4 o = {pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
                store_once(A.q_out + ((size_t)r * A.hq + h) * D + 8 * lane, o);
            }
            const size_t at = (((size_t)page * hkv + kvh) << A.kv.page_shift) + off;
            if constexpr (MX) {
                put_block<D>(x, lane, there && !is_q && !is_k && cached, A.kv.v, A.kv.v_exp, at);
            } else if (A.kv.k_scale) {
                float m = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
                m = fmaxf(max_group<LANES>(m), kTinyMax);
                if (there && !is_q && cached) {
                    const float to = kE4m3Max / m;
                    int lo = 0, hi = 0;
                    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * to, x[1] * to, lo, false);
                    lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * to, x[3] * to, lo, true);
                    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[4] * to, x[5] * to, hi, false);
                    hi = __builtin_amdgcn_cvt_pk_fp8_f32(x[6] * to, x[7] * to, hi, true);
                    *reinterpret_cast<uint2 *>((is_k ? A.kv.k : A.kv.v) + at * D + 8 * lane) = make_uint2(lo, hi);
                    if (lane == 0) (is_k ? A.kv.k_scale : A.kv.v_scale)[at] = m / kE4m3Max;
                }
            } else if (there && !is_q && cached) {
                const uint4 o = is_k ? make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])) : raw[b];
                store_once((is_k ? A.kv.k : A.kv.v) + (at * D + 8 * lane) * 2, o);
            }
        }
    }
    if constexpr (KEYS) {
#pragma unroll 1
        for (int h0 = k_first; h0 < k_heads; h0 += HEADS) {
            const int h = h0 + grp;
            if (h0 > k_first) {
                raw_k = make_uint4(0, 0, 0, 0);
                if (h < k_heads) raw_k = load_once(source(h) + 8 * lane);
            }
            float x[8];
            exact_key<D, LANES>(A, raw_k, lane, swap64[grp], weight, cs64, sn64, x);
            const size_t at = (((size_t)page * hkv + h - A.hq) << A.kv.page_shift) + off;
            put_block<D>(x, lane, h < k_heads && cached, A.kv.k, A.kv.k_exp, at);
        }
    }
}

// ---- commit of accepted paths ----------------------------------------------
//
// One workgroup a stream, 16 trees in 4.6 us on the GPU, one in 2.7: two dependent
// loads (layout, then page numbers), then the rows.  The path's rows i_0 < i_1 < ... move from cache
// rows kv_len + i_j to kv_len + j.  A thread owns 16-byte columns (or one
// scale) of the rows and holds every source in registers before it stores the
// first, so a row that is both source and destination is read in time.
__global__ __launch_bounds__(256) void attn_commit_kernel(const AttnCommitArgs A, const int row_bytes)
{
    __shared__ int src[kMaxWindowRows], dst[kMaxWindowRows], len;
    const int s = blockIdx.x, tid = threadIdx.x;
    int kv = 0, kept = 0;
    if (tid < 64) {
        // lane t: the window's row t, its parent and the page that holds it
        const int a = A.row_start[s], b = A.row_start[s + 1], acc = A.accept[s], m = b - a;
        kv = A.kv_len[s];
        const long long cap = (long long)A.max_blocks << A.kv.page_shift;
        const int mask = (1 << A.kv.page_shift) - 1;
        bool ok = a >= 0 && b >= a && b <= A.total_rows && m <= A.max_rows && kv >= 0 && (long long)kv + m <= cap
                  && acc >= a && acc < b;
        const bool there = ok && tid < m;
        const int up = there ? (A.parent ? A.parent[a + tid] : tid - 1) : -1;
        const int id = there ? A.table[(size_t)s * A.max_blocks + ((kv + tid) >> A.kv.page_shift)] : 0;
        ok = ok && !__ballot(there && (up < -1 || up >= tid));
        uint32_t path = 0;
        if (ok)
            for (int t = acc - a; t >= 0; t = __builtin_amdgcn_readlane(up, t)) path |= 1u << t;
        const int n = __popc(path), rank = __popc(path & ((1u << (tid & 31)) - 1));
        const int id_to = __shfl(id, rank);
        const bool on = tid < kMaxWindowRows && (path >> tid & 1);
        // every page of the window has to be in the cache: a stream that got none
        // for this pass may hold those of a short path
        ok = ok && !__ballot(there && (id < 0 || id >= A.kv.n_pages));
        kept = ok ? n : 0;
        if (on && ok) {
            src[rank] = ((id * A.kv.hkv) << A.kv.page_shift) + ((kv + tid) & mask);
            dst[rank] = ((id_to * A.kv.hkv) << A.kv.page_shift) + ((kv + rank) & mask);
        }
        if (tid == 0) {
            len = kept;
            A.kv_len_out[s] = kv + kept;
        }
    }
    __syncthreads();
    const int n = len, cols = row_bytes / 16, per = A.kv.hkv * cols;
    // the rows before the first that moves stay where they are
    int first = 0;
    while (first < n && src[first] == dst[first]) ++first;
    if (first == n) return;
    for (int i = tid; i < 2 * per; i += 256) {
        const int j = i < per ? i : i - per, h = j / cols;
        uint8_t *pool = (i < per ? A.kv.k : A.kv.v) + (size_t)(j - h * cols) * 16;
        const size_t head = (size_t)h << A.kv.page_shift;
        f4v x[kMaxWindowRows];
#pragma unroll
        for (int t = 0; t < kMaxWindowRows; ++t)
            x[t] = *reinterpret_cast<const f4v *>(pool + (src[min(t, n - 1)] + head) * row_bytes);
#pragma unroll
        for (int t = 0; t < kMaxWindowRows; ++t)
            if (t >= first && t < n) *reinterpret_cast<f4v *>(pool + (dst[t] + head) * row_bytes) = x[t];
    }
    if (A.kv.k_scale) {
        for (int i = tid; i < 2 * A.kv.hkv; i += 256) {
            float *pool = (i < A.kv.hkv ? A.kv.k_scale : A.kv.v_scale) + ((size_t)(i % A.kv.hkv) << A.kv.page_shift);
            float x[kMaxWindowRows];
#pragma unroll
            for (int t = 0; t < kMaxWindowRows; ++t)
                x[t] = pool[src[min(t, n - 1)]];
#pragma unroll
            for (int t = 0; t < kMaxWindowRows; ++t)
                if (t >= first && t < n) pool[dst[t]] = x[t];
        }
    } else if (A.kv.k_exp) {
        const int exps = A.kv.d / kMxBlock;             // bytes of a row
        for (int i = tid; i < 2 * A.kv.hkv * exps; i += 256) {
            const int j = i % (A.kv.hkv * exps), h = j / exps;
            uint8_t *pool = (i == j ? A.kv.k_exp : A.kv.v_exp) + (((size_t)h << A.kv.page_shift) * exps + j % exps);
            uint8_t x[kMaxWindowRows];
#pragma unroll
            for (int t = 0; t < kMaxWindowRows; ++t)
                x[t] = pool[(size_t)src[min(t, n - 1)] * exps];
#pragma unroll
            for (int t = 0; t < kMaxWindowRows; ++t)
                if (t >= first && t < n) pool[(size_t)dst[t] * exps] = x[t];
        }
    }
}

// ---- cached rows read back ---------------------------------------------------
//
// Bounded by memory: 16 packed rows a workgroup, all their kv heads, 16 bytes of
// bf16 a lane and step, so that every wave writes runs of 1 KB (91,000 rows of 4 heads
// of 256: of 4 bits 474 MB in 104 us, 4.5 TB/s, of e4m3 565 MB in 110, of bf16 749 MB
// in 128; 100 rows of 2 heads of 64 in 3.1 to 3.3).
constexpr int kReadRows = 16, kReadThreads = 256;

template <int FMT>
__global__ __launch_bounds__(kReadThreads) void read_kernel(const ReadArgs A)
{
    __shared__ int at[kReadRows];                   // a row's place in the cache (of kv head 0), or -1
    const int tid = threadIdx.x, first = blockIdx.x * kReadRows, rows = min(kReadRows, A.total_rows - first);
    if (tid < 64) {
        // lane i: row first + i of the stream whose rows hold it
        const int r = first + min(tid, rows - 1);
        int stream = -1, t = 0;
        auto look = [&](int block) {
            const int s = block + tid;
            int r0 = 0, r1 = 0;
            if (s < A.n_streams) {
                r0 = A.row_start[s], r1 = A.row_start[s + 1];
                const int f = A.first[s];
                const bool ok = r0 >= 0 && r1 >= r0 && r1 <= A.total_rows && f >= 0 && (long long)f + (r1 - r0) <= (long long)A.max_blocks << A.kv.page_shift;
                if (!ok) r0 = r1 = 0;
            }
            uint64_t some = __ballot(r1 > first && r0 < first + rows);
            while (some) {
                const int l = __builtin_ctzll(some);
                some &= some - 1;
                const int a = __builtin_amdgcn_readlane(r0, l), b = __builtin_amdgcn_readlane(r1, l);
                if (stream < 0 && r >= a && r < b) stream = block + l, t = r - a;
            }
        };
        for (int block = 0; block < A.n_streams && __ballot(stream < 0); block += 64) look(block);
        int row = -1;
        if (stream >= 0) {
            const int key = A.first[stream] + t;
            const int id = A.table[(size_t)stream * A.max_blocks + (key >> A.kv.page_shift)];
            if (id >= 0 && id < A.kv.n_pages) row = ((id * A.kv.hkv) << A.kv.page_shift) + (key & ((1 << A.kv.page_shift) - 1));
        }
        if (tid < rows) at[tid] = row;
    }
    __syncthreads();
    const int d = A.kv.d, per = d / 8, per_row = A.kv.hkv * per;        // 16-byte pieces of a head, and of a row
    for (int i = tid; i < 2 * rows * per_row; i += kReadThreads) {
        const bool is_v = i >= rows * per_row;
        const int j = i - is_v * rows * per_row, r = j / per_row, x = j - r * per_row, h = x / per, p = x - h * per;
        if (at[r] < 0) continue;
        const size_t row = (size_t)at[r] + ((size_t)h << A.kv.page_shift);
        const uint8_t *pool = is_v ? A.kv.v : A.kv.k;
        uint4 y;
        if constexpr (FMT == FMT_BF16) {
            y = load_once(pool + (row * d + 8 * p) * 2);
        } else if constexpr (FMT == FMT_E4M3) {
            const uint2 c = *reinterpret_cast<const uint2 *>(pool + row * d + 8 * p);
            const float f = (is_v ? A.kv.v_scale : A.kv.k_scale)[row];
            float z[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t w = k ? c.y : c.x;
                z[4 * k] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * f, z[4 * k + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * f;
                z[4 * k + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * f, z[4 * k + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * f;
            }
            y = make_uint4(pack2(z[0], z[1]), pack2(z[2], z[3]), pack2(z[4], z[5]), pack2(z[6], z[7]));
        } else {
            const uint32_t c = *reinterpret_cast<const uint32_t *>(pool + row * (d / 2) + 4 * p);
            y = mx_values8(c, mx_scale((is_v ? A.kv.v_exp : A.kv.k_exp)[row * (d / kMxBlock) + p / 4]));
        }
        store_once((is_v ? A.v_out : A.k_out) + ((size_t)(first + r) * per_row + x) * 8, y);
    }
}

}  // namespace

hipError_t launch_tables(const TablesArgs &A, hipStream_t stream)
{
    // A single workgroup for a small call (16 streams of 16 rows: 6.8 us on the GPU,
    // 6.5 with 32 workgroups, but one launch also where the counts are updated in
    // place); 500 streams with 12,163 rows take it 44 us, and 32 workgroups 7.3
    // (8.6 us a call from Python; with the counts in place, in two launches, 12.1).
    const size_t lds = sizeof(int) * (6 * (size_t)A.n_streams + 1);
    if (A.n_streams <= 32 && A.total_rows <= kTablesThreads) {
        tables_kernel<<<1, kTablesThreads, lds, stream>>>(A, 1, 1);
    } else if (A.page_count_out != A.page_count && A.free_count_out != A.free_count) {
        tables_kernel<<<kTablesBlocks, kTablesThreads, lds, stream>>>(A, 1, 1);
    } else {
        tables_kernel<<<kTablesBlocks, kTablesThreads, lds, stream>>>(A, 0, 1);
        tables_kernel<<<1, kTablesThreads, lds, stream>>>(A, 1, 0);
    }
    return hipGetLastError();
}

template <int D>
static void launch_prep_d(const PrepArgs &A, hipStream_t stream)
{
    // A workgroup has all of a row's heads, or where the rows are few, as many as
    // its lanes hold at once (on the GPU, 32 heads of 256: one row 3.7 us instead of
    // 6.8, 249 rows of 48 heads of 128 4.5 instead of 5.3; from about 500 rows on the
    // angles that every workgroup works out again cost more: 1,024 rows 12.5 us
    // instead of 11.0, 8,306 rows 86 instead of 62).  Into a 4-bit cache the border is
    // the same: 24 query and 4 kv heads of 256 so and with the keys in workgroups of
    // their own 256 rows 7.1 and 9.7 us, 400 rows 9.8 and 10.6, 512 rows 11.0 and
    // 10.9, 640 rows 12.0 and 11.3, 1,000 rows 17.3 and 14.0, 2,000 rows 30.7 and 21.7;
    // 32 and 8 heads of 128 400 rows 8.2 and 8.9, 640 rows 11.6 and 10.7.
    const int heads = A.hq + 2 * A.kv.hkv, at_once = kPrepThreads / (D / 8);
    const int span = A.rows <= kPrepFewRows && heads > at_once ? at_once : heads;
    const dim3 grid(A.rows, (heads + span - 1) / span);
    const long long keys = ((long long)A.rows * A.kv.hkv + at_once - 1) / at_once;
    if (!A.kv.k_exp) {
        prep_kernel<D, PREP_ROWS><<<grid, kPrepThreads, 0, stream>>>(A, span);
    } else if (A.rows <= kPrepFewRows || A.rows + keys > kMaxGroups) {
        prep_kernel<D, PREP_MX><<<grid, kPrepThreads, 0, stream>>>(A, span);
    } else {
        const size_t lds = sizeof(double) * (D + at_once * key_swap(A.rot) + key_rows(at_once, A.kv.hkv) * A.rot);
        prep_kernel<D, PREP_MX_APART><<<(unsigned)(A.rows + keys), kPrepThreads, lds, stream>>>(A, heads);
    }
}

hipError_t launch_prep(const PrepArgs &A, hipStream_t stream)
{
    switch (A.kv.d) {
    case 64: launch_prep_d<64>(A, stream); break;
    case 128: launch_prep_d<128>(A, stream); break;
    default: launch_prep_d<256>(A, stream); break;
    }
    return hipGetLastError();
}

hipError_t launch_attn_commit(const AttnCommitArgs &A, hipStream_t stream)
{
    attn_commit_kernel<<<A.n_streams, 256, 0, stream>>>(A, A.kv.k_exp ? A.kv.d / 2 : A.kv.d * (A.kv.k_scale ? 1 : 2));
    return hipGetLastError();
}

hipError_t launch_read(const ReadArgs &A, hipStream_t stream)
{
    const int blocks = (A.total_rows + kReadRows - 1) / kReadRows;
    switch (format_of(A.kv)) {
    case FMT_BF16: read_kernel<FMT_BF16><<<blocks, kReadThreads, 0, stream>>>(A); break;
    case FMT_E4M3: read_kernel<FMT_E4M3><<<blocks, kReadThreads, 0, stream>>>(A); break;
    default: read_kernel<FMT_MXFP4><<<blocks, kReadThreads, 0, stream>>>(A); break;
    }
    return hipGetLastError();
}

}  // namespace gdn
