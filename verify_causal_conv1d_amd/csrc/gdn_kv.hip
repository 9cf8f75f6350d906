// The paged key-value cache of the attention layers: block tables and slot
// maps from request lengths (tables_kernel), norms and rotation of queries and
// keys with the cache writes (prep_kernel), and the commit of accepted tree
// paths (attn_commit_kernel).  Contracts are in include/libgdn.h.
#include "gdn_attn.h"
#include "gdn_device.h"
#include "gdn_internal.h"
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

// The rows pass through once, and what is stored is read by other kernels on
// whichever XCD: load_once and store_once (the prompt pass of 8,306 rows takes
// 62 us with them and 68 us without).
template <int D>
__global__ __launch_bounds__(kPrepThreads) void prep_kernel(const PrepArgs A, const int span)
{
    constexpr int LANES = D / 8, HEADS = kPrepThreads / LANES;   // heads a workgroup handles at once
    constexpr int BATCH = 4;                                     // and loads ahead
    // this workgroup's heads: span of them from span * blockIdx.y
    __shared__ float cs[kPrepMaxHalf], sn[kPrepMaxHalf];
    __shared__ __align__(16) float swap[HEADS][D];
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid % LANES, grp = tid / LANES;
    const int half = A.rot / 2, hkv = A.kv.hkv, first = span * blockIdx.y, heads = min(A.hq + 2 * hkv, first + span);
    const int64_t q_row = r * A.q_row, k_row = r * A.k_row, v_row = r * A.v_row;
    auto source = [&](int h) {
        return h < A.hq ? A.q + (q_row + h * A.q_head)
             : h < A.hq + hkv ? A.k + (k_row + (h - A.hq) * A.k_head) : A.v + (v_row + (h - A.hq - hkv) * A.v_head);
    };
    uint4 raw[BATCH];
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
    }
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
            if (A.kv.k_scale) {
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
    // instead of 11.0, 8,306 rows 86 instead of 62)
    const int heads = A.hq + 2 * A.kv.hkv, at_once = kPrepThreads / (D / 8);
    const int span = A.rows <= kPrepFewRows && heads > at_once ? at_once : heads;
    prep_kernel<D><<<dim3(A.rows, (heads + span - 1) / span), kPrepThreads, 0, stream>>>(A, span);
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
    attn_commit_kernel<<<A.n_streams, 256, 0, stream>>>(A, A.kv.d * (A.kv.k_scale ? 1 : 2));
    return hipGetLastError();
}

}  // namespace gdn
