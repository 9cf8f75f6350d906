// Attention of whole prompts over the paged cache.  Contract in
// include/libgdn.h (gdn_attn_prompt).
//
// Row t of a stream sees its cache rows 0 .. kv_len + t:
//     s_j = scale q . k_j,   o = sum_j e^{s_j} v_j / sum_j e^{s_j},   out = o sigmoid(gate).
// As in the kernels of steps and windows, the (row, query head) pairs of a stream
// and kv head are the columns of S^T = K Q^T and O^T = V^T P^T, with one pass over
// the keys that keeps the running maximum and sum of each column (base-2
// exponentials).  A wave has 32 columns and 32x32x16 matrix instructions, whose
// result gives a lane the weights of one column in just the order in which the
// second product takes them; queries and O stay in registers, a stage of 32 keys and
// their values passes through LDS in bf16 for all waves of the workgroup, the next
// one on its way (bf16 rows by direct loads, the others through registers, where they
// are converted).  A row's page is known a stage before the row is asked for.
//
// What bounds it is the matrix unit and the vector unit beside it: of 256 channels
// a wave's 32 keys are 32 matrix instructions and about 110 others.  16,384 rows of
// 24 query and 4 kv heads of 256 take 2.71 to 2.84 ms in bf16, from card to card
// (1,160 to 1,215 TFLOP/s), 2.66 to 2.77 over 4-bit rows (1,189 to 1,240) and 3.12 to
// 3.22 over e4m3 rows (1,024 to 1,058).  There the scales of the keys take the place of
// the call's in the one fmaf of a score, those of the values are one more
// multiplication of every weight, and both are read from LDS.  Of 32 and 8 heads of
// 128 it is 1,025 to 1,080, 1,058 to 1,101 and 856 to 862 TFLOP/s, of 64 848 to 885,
// 807 to 839 and 669 to 693, as there are half and a quarter as many products to a
// weight.  (A product of two 8,192 x 8,192 matrices reaches 1,254.)
#include "gdn_attn_core.h"
#include "gdn_mxfp4.h"

namespace gdn {
namespace {

__device__ __forceinline__ f16v mfma32(bf8v a, bf8v b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }

// over lanes l and l ^ 32
__device__ __forceinline__ float max_halves(float x)
{
    const uint32_t xi = __float_as_uint(x);
    const auto q = __builtin_amdgcn_permlane32_swap(xi, xi, false, false);
    return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float sum_halves(float x)
{
    const uint32_t xi = __float_as_uint(x);
    const auto q = __builtin_amdgcn_permlane32_swap(xi, xi, false, false);
    return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// The lane's number, worked out anew from a mask that the compiler cannot trace: no
// register holds it through the loop.  (The instructions are the compiler's own, so
// that it waits where a matrix instruction may still use the register that they
// write.)
__device__ __forceinline__ int lane_number()
{
    uint32_t all = ~0u;
    asm volatile("" : "+s"(all));
    return __builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0));
}

// The kernel's arguments, loaded anew: none of them holds scalar registers through
// the loop for the sake of what comes after it (registers that hold spilled scalars
// went to memory, and every wait for one of them waited for all stores before it).
typedef const __attribute__((address_space(4))) AttnArgs const_args;
__device__ __forceinline__ const_args *fresh_args()
{
    auto p = reinterpret_cast<uintptr_t>(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(p));
    return (const_args *)p;
}

__device__ __forceinline__ float uniform(float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x))); }

constexpr int kKeys = 32;      // of a stage: a matrix instruction's tile
constexpr int kAhead = 3;      // operands on their way from LDS

// A stage of keys and values in LDS, in bf16: KEYS rows of K, then of V, in 16-byte
// pieces.  A lane that converts 16 bytes of e4m3 or of 4-bit codes stores 2 or 4
// pieces; those of the same turn lie one after the other, for a row's lanes.  Pieces
// are exchanged by a function of the row, linear in its bits, so that of 16 lanes
// one after the other that store a piece, of 16 rows of K read at one piece, and
// of 32 lanes that read V transposed (4 rows at 64 bytes of channels), each 256 bytes
// of LDS hold every place as often as any other.  (Pieces in order, with the rows
// exchanged as those of bf16: half of the LDS's busy cycles over 4 bits were
// conflicts.)
template <int D, int FMT, int WAVES>
struct PromptShape {
    static constexpr int THREADS = 64 * WAVES, COLS = 32 * WAVES;
    static constexpr int KEYS = kKeys, ROW = 2 * D, HALF = KEYS * ROW, BYTES = 2 * HALF;
    static constexpr int PIECES = ROW / 16, ROWS = 1024 / ROW;    // of a direct load
    static constexpr int TURNS = FMT == FMT_BF16 ? 1 : FMT == FMT_E4M3 ? 2 : 4, LANES = PIECES / TURNS;     // of a row
    static __device__ __forceinline__ int k_place(int c) { return c % TURNS * LANES + c / TURNS; }
    static __device__ __forceinline__ int v_place(int c)
    {
        const int i = c % TURNS, more = D < 256 ? 0 : FMT == FMT_E4M3 ? 8 * i : FMT == FMT_MXFP4 ? (i >> 1) * 4 : 0;
        return (i * LANES + c / TURNS) ^ more;
    }
    static __device__ __forceinline__ int k_swizzle(int r)
    {
        if (FMT == FMT_BF16) return ROW >= 256 ? r & 15 : r >> 1 & 7;
        if (D == 64) return FMT == FMT_E4M3 ? (r & 2) * 2 + (r & 4) / 2 + (r & 8) / 8 : (r & 6) + (r & 8) / 8;
        return FMT == FMT_MXFP4 && D == 128 ? (r & 3) * 4 | (r >> 2 & 3) : (r & 1) * 8 | (r >> 1 & 7);
    }
    static __device__ __forceinline__ int v_swizzle(int r)
    {
        if (FMT == FMT_BF16) return ROW >= 256 ? (r & 3) * 4 : (r & 2) * 2;
        if (D == 64) return FMT == FMT_E4M3 ? (r >> 1 & 1) * 6 : (r >> 1 & 1) * 3 ^ (r & 4);
        if (D == 128) return FMT == FMT_E4M3 ? (r & 1) * 10 ^ (r & 2) * 2 : (r & 3) * 5;
        return FMT == FMT_E4M3 ? (r & 3) * 2 : (r & 1) * 9 ^ (r & 6);
    }
    // `from`, a row's place in bytes, with piece c's place (known at compile time) exchanged into it
    static __device__ __forceinline__ int with_place(int from, int place) { return (from ^ (place & 15) * 16) + (place & ~15) * 16; }
    // cached rows in their own format
    static constexpr int CODES = FMT == FMT_BF16 ? ROW : FMT == FMT_E4M3 ? D : D / 2;
    static constexpr int PER_ROW = CODES / 16;                   // 16-byte units of a row
    static constexpr int UNITS = KEYS * PER_ROW;                 // of a stage's keys, and of its values
    static constexpr int LOADS = (2 * UNITS + THREADS - 1) / THREADS;    // of a thread
    static constexpr int SCALES = FMT == FMT_E4M3 ? 2 * KEYS : 4;
};

struct PromptPiece {
    int h, rt, c;             // kv head, tile of columns, chunk
    int s, r0, m, kv, len;
    int k0, k1, nch, cols;
};

// The pieces of all streams.  Their kv heads are innermost, so that the workgroups
// of a head meet in as few XCDs as can be, and the tiles that see the most keys
// come first, since workgroups begin in their order: of a stream its last rows,
// and where a wave holds all streams and they are not cut into chunks, over all of
// them (a prompt of 4,722 rows packed after three shorter ones begins too late to end
// with them: 391 us, and 375 in order).
template <int COLS, bool WINDOW>
__device__ __forceinline__ bool find_piece(const AttnArgs &A, int split_keys, int item, PromptPiece &K)
{
    const int lane = threadIdx.x & 63;
    for (int first = 0; first < A.n_streams; first += 64) {
        int r0 = 0, m = 0, kv = 0, count = 0, tiles = 0, size = 1;
        const int s = first + lane;
        if (s < A.n_streams && stream_window(A, s, r0, m, kv)) {
            size = WINDOW ? chunk_keys(kv + m, true) : split_keys;
            tiles = ceil_div(m * A.group, COLS);
            count = tiles * ceil_div(kv + m, size) * A.kv.hkv;
        } else {
            kv = 0;         // a skipped stream's may be anything, down to where a level less it overflows
        }
        const int incl = wave_running_sum(count), all = __builtin_amdgcn_readlane(incl, 63);
        if (item >= all) {
            item -= all;
            continue;
        }
        int l, x;
        if (!WINDOW && A.n_streams > 1 && A.n_streams <= 64 && A.chunks == 1) {
            // A tile's level: the cache row of its first pair.  Tiles of the lane's stream
            // above a level; the one looked for has the least level that no more than
            // y tiles are above.
            auto above = [&](int level) {
                const long long from = level < kv ? 0 : ((long long)(level - kv + 1) * A.group + COLS - 1) / COLS;
                return from < tiles ? tiles - (int)from : 0;
            };
            auto total = [&](int level) { return __builtin_amdgcn_readlane(wave_running_sum(above(level)), 63); };
            const int y = item / A.kv.hkv;
            int lo = -1, hi = A.max_kv;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (total(mid) > y) lo = mid;
                else hi = mid;
            }
            const int here = wave_running_sum(above(lo) - above(hi)), nth = y - total(hi);
            l = __builtin_ctzll(__ballot(here > nth));
            const int z = __builtin_amdgcn_readlane(above(lo), l) - 1 - (nth - (l ? __builtin_amdgcn_readlane(here, l - 1) : 0));
            x = z * A.kv.hkv + item - y * A.kv.hkv;
        } else {
            l = __builtin_ctzll(__ballot(incl > item));
            x = item - (l ? __builtin_amdgcn_readlane(incl, l - 1) : 0);
        }
        K.s = first + l;
        K.r0 = __builtin_amdgcn_readlane(r0, l);
        K.m = __builtin_amdgcn_readlane(m, l);
        K.kv = __builtin_amdgcn_readlane(kv, l);
        K.len = K.kv + K.m;
        K.cols = K.m * A.group;
        size = __builtin_amdgcn_readlane(size, l);
        K.nch = ceil_div(K.len, size);
        const int y = x / A.kv.hkv;
        K.h = x - y * A.kv.hkv;
        const int z = y / K.nch;
        K.c = y - z * K.nch;
        K.rt = __builtin_amdgcn_readlane(tiles, l) - 1 - z;
        K.k0 = K.c * size;
        const int last = min((K.rt + 1) * COLS, K.cols) - 1;       // the tile's last column sees the most
        K.k1 = min(K.k0 + size, WINDOW ? K.len : K.kv + last / A.group + 1);
        return true;
    }
    return false;
}

// All pages of the stream are in the cache (for the caller's wave: its share).
__device__ __forceinline__ bool pages_ok(const AttnArgs &A, const PromptPiece &K, int threads)
{
    bool ok = true;
    const int *table = A.table + (size_t)K.s * A.max_blocks;
    for (int i = threadIdx.x; i <= (K.len - 1) >> A.kv.page_shift; i += threads) {
        const int id = table[i];
        ok = ok && id >= 0 && id < A.kv.n_pages;
    }
    return !__ballot(!ok);
}

// Channels d .. d + 3 of the values of a cache row, in bf16 (e4m3: before the row's scale).
template <int D, int FMT>
__device__ __forceinline__ uint2 cached_values4(const uint8_t *pool, const uint8_t *exps, size_t row, int d)
{
    if constexpr (FMT == FMT_BF16) {
        return *reinterpret_cast<const uint2 *>(pool + (row * D + d) * 2);
    } else if constexpr (FMT == FMT_E4M3) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(pool + row * D + d);
        return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)));
    } else {
        const uint32_t w = *reinterpret_cast<const uint16_t *>(pool + (row * D + d) / 2);
        const float f = mx_scale(exps[row * (D / kMxBlock) + d / kMxBlock]);
        return make_uint2(mx_pair<0>(w, f), mx_pair<1>(w, f));
    }
}
// 4 channels of a result in bf16, gated
__device__ __forceinline__ uint2 gated4(float4 o, bool gated, uint2 g)
{
    float x[4] = {o.x, o.y, o.z, o.w};
    if (gated) {
        x[0] *= sigmoid_f(__uint_as_float(g.x << 16));
        x[1] *= sigmoid_f(__uint_as_float(g.x & 0xffff0000u));
        x[2] *= sigmoid_f(__uint_as_float(g.y << 16));
        x[3] *= sigmoid_f(__uint_as_float(g.y & 0xffff0000u));
    }
    return make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
}
__device__ __forceinline__ int wave_int(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ float not_finite(uint32_t bits) { return (bits & 0x7f800000u) == 0x7f800000u ? __uint_as_float(bits) : 0.0f; }

template <int D, int FMT, int WAVES, int PER_SIMD, bool WINDOW>
__global__ __launch_bounds__(64 * WAVES, PER_SIMD) void prompt_kernel(const AttnArgs A, const int split_keys)
{
    using S = PromptShape<D, FMT, WAVES>;
    constexpr int KS = D / 16, NT = D / 32;
    constexpr int PER = 2 * S::HALF / 1024 / WAVES;     // direct loads of a wave
    // Operands of the queries that stay in LDS: with all of them in registers the
    // first three of e4m3 rows of 256 channels went to memory, and reading them back
    // waited for the rows on their way; so did the first of 4-bit rows in workgroups
    // of 4 waves (2,048 rows 114 us, with it in LDS 105).
    constexpr int QL = D < 256 || WINDOW ? 0 : FMT == FMT_E4M3 ? 4 : FMT == FMT_MXFP4 && WAVES == 4 ? 1 : 0;
    __shared__ __align__(16) uint4 q_lds[QL ? WAVES * QL * 64 : 1];
    // separate arrays, so that loads into one are known not to touch the other
    __shared__ __align__(1024) uint8_t st0[S::BYTES], st1[S::BYTES];
    __shared__ __align__(16) float sc0[S::SCALES], sc1[S::SCALES];
    __shared__ int wave_ok[WAVES], bad;
    __shared__ int2 pairs[S::COLS];          // packed row and query head of each column
    __shared__ PromptPiece kept;             // K, for the end
    __shared__ uint32_t seen[WINDOW ? S::COLS : 1];      // rows of a window that each column sees

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 31, g = lane >> 5;
    const float scale = uniform(A.scale);
    // Of up to 128 channels a register is left for it (e4m3 rows of 128, a resumed
    // prompt: 1,256 us, worked out anew 1,309).
    auto this_lane = [&] {
        if constexpr (D < 256) return fresh(lane);
        else return lane_number();
    };
    PromptPiece K;
    for (int item = blockIdx.x; find_piece<S::COLS, WINDOW>(A, split_keys, item, K); item += gridDim.x) {
        if (K.k0 >= K.k1) continue;                 // a chunk past all that the tile sees
        bool ok = true;
        const int col0 = K.rt * S::COLS + wave * 32;            // the wave's first column
        const bool busy = col0 < K.cols;                            // waves without columns only load
        const int t_lo = min(col0, K.cols - 1) / A.group, t_hi = min(col0 + 32, K.cols) - 1;   // rows of the wave
        const int see_lo = K.kv + t_lo, see_hi = K.kv + t_hi / A.group;      // the last key that the first and the last one see
        const int col = min(col0 + n, K.cols - 1);     // past the last one: that one again, not stored
        const int row = col / A.group;
        pairs[wave * 32 + n] = make_int2(K.r0 + row, K.h * A.group + col - row * A.group);     // (both halves the same)
        if constexpr (WINDOW) seen[wave * 32 + n] = seen_rows(A, K.r0, K.m, row, ok);
        // place of a column's (row, head) in q and out
        auto pair_of = [&](int hq) {
            const int2 p = pairs[wave * 32 + (this_lane() & 31)];
            return (size_t)p.x * hq + p.y;
        };
        __builtin_amdgcn_wave_barrier();
        bf8v q[KS];
        const uint16_t *p = A.q + pair_of(A.hq) * D + 8 * (this_lane() >> 5);
#pragma unroll
        for (int k = 0; k < KS; ++k) q[k] = *reinterpret_cast<const bf8v *>(p + 16 * k);
        f16v o[NT];
        float mx = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;
        // keys that every column of the workgroup sees
        const int all_see = WINDOW ? K.kv : K.kv + K.rt * S::COLS / A.group + 1;

        const int *table = A.table + (size_t)K.s * A.max_blocks;
        const int tiles = ceil_div(K.k1 - K.k0, S::KEYS);
        // Pages of the groups of 16 keys of a stage, asked for a step before they are
        // used; then the cache row of the nth group.
        constexpr int GROUPS = S::KEYS / 16;
        int pages[GROUPS], pages_key = 0;
        auto look = [&](int tile) {
            pages_key = K.k0 + min(tile, tiles - 1) * S::KEYS;
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) pages[i] = table_entry(table, min(pages_key + 16 * i, (K.len - 1) & ~15) >> A.kv.page_shift);
        };
        auto group_row = [&](int i) {
            int page = pages[0];
#pragma unroll
            for (int x = 1; x < GROUPS; ++x) page = i == x ? pages[x] : page;
            page = (uint32_t)page < (uint32_t)A.kv.n_pages ? page : 0;
            return ((page * A.kv.hkv + K.h) << A.kv.page_shift) + (min(pages_key + 16 * i, (K.len - 1) & ~15) & ((1 << A.kv.page_shift) - 1));
        };
        uint4 raw[FMT == FMT_BF16 ? 1 : S::LOADS];
        uint32_t raw_scale[FMT == FMT_BF16 ? 1 : S::LOADS];
        float row_scale = 0.0f;
        // unit x of a lane: the wave's are keys or values, whole rows in order
        static_assert(S::UNITS % 64 == 0, "");
        struct Unit {
            bool there, is_v;
            int first;              // the wave's first row
        };
        auto unit = [&](int x) {
            constexpr bool SAME = S::UNITS % S::THREADS == 0, ALL = 2 * S::UNITS % S::THREADS == 0;
            const int u = (x * WAVES + wave) * 64;
            const bool is_v = SAME ? x >= S::LOADS / 2 : u >= S::UNITS;
            return Unit{ALL || u < 2 * S::UNITS, is_v, (is_v ? u - S::UNITS : u) / S::PER_ROW};
        };
        // bf16: straight to a stage; else to registers, for put
        auto load = [&](uint8_t *stage) {
            if constexpr (FMT == FMT_BF16) {
                const int ln = this_lane();
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const bool is_k = j < PER / 2;
                    const int x = j % (PER / 2);
                    const int first = (x * WAVES + wave) * S::ROWS, in = first % 16 + ln / S::PIECES;      // rows of the stage; of its group
                    const uint32_t off = in * S::ROW + (ln % S::PIECES ^ (is_k ? S::k_swizzle(in) : S::v_swizzle(in))) * 16;
                    const uint8_t *p = (is_k ? A.kv.k : A.kv.v) + (size_t)group_row(first / 16) * S::ROW;
                    __builtin_amdgcn_global_load_lds((global_void *)(p + off),
                                                     (lds_void *)(stage + (j * WAVES + wave) * 1024), 16, 0, 0);
                }
            } else {
#pragma unroll
                for (int x = 0; x < S::LOADS; ++x) {
                    const Unit u = unit(x);
                    if (!u.there) continue;
                    // the wave's rows lie one after the other in a group of 16, or in two
                    const uint32_t ln = this_lane();
                    size_t at;
                    uint32_t in;
                    if constexpr (S::PER_ROW < 4) {
                        at = ln < 32 ? group_row(u.first / 16) : group_row(u.first / 16 + 1);
                        in = ln & 31;
                    } else {
                        at = group_row(u.first / 16) + (u.first & 15);
                        in = ln;
                    }
                    raw[x] = *reinterpret_cast<const uint4 *>((u.is_v ? A.kv.v : A.kv.k) + at * S::CODES + 16 * in);
                    if constexpr (FMT == FMT_MXFP4) raw_scale[x] = ((u.is_v ? A.kv.v_exp : A.kv.k_exp) + at * (D / kMxBlock))[in];
                }
                if constexpr (FMT == FMT_E4M3) {        // the first waves: a scale a lane, of the keys and then of the values
                    if (wave < 2) row_scale = (wave == 0 ? A.kv.k_scale : A.kv.v_scale)[(size_t)group_row(this_lane() % S::KEYS / 16) + (this_lane() & 15)];
                }
            }
        };
        // rows in registers, to bf16, to a stage
        auto put = [&](uint8_t *stage, float *scales) {
            if constexpr (FMT != FMT_BF16) {
#pragma unroll
                for (int x = 0; x < S::LOADS; ++x) {
                    __builtin_amdgcn_sched_barrier(0);
                    const Unit u = unit(x);
                    if (!u.there) continue;
                    // the lane's row and its place there
                    const uint32_t ln = this_lane(), r = u.first + ln / S::PER_ROW, p = ln % S::PER_ROW;
                    const int to = r * S::ROW + (p ^ (u.is_v ? S::v_swizzle(r) : S::k_swizzle(r))) * 16;
                    uint8_t *half = stage + u.is_v * S::HALF;
                    const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
                    if constexpr (FMT == FMT_MXFP4) {
                        const float f = mx_scale(raw_scale[x]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(half + S::with_place(to, u.is_v ? S::v_place(i) : S::k_place(i))) = mx_values8(w[i], f);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t y[4];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                y[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + j], 1.0f, false));
                                y[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + j], 1.0f, true));
                            }
                            *reinterpret_cast<uint4 *>(half + S::with_place(to, u.is_v ? S::v_place(i) : S::k_place(i))) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                }
                if constexpr (FMT == FMT_E4M3)
                    if (wave < 2 && this_lane() < S::KEYS) scales[wave * S::KEYS + this_lane()] = wave == 0 ? row_scale * scale : row_scale;
            }
        };

        // The stage's keys, from `first`.  tail: some column does not see all of them.
        auto multiply = [&](bool tail, int first, const uint8_t *stage, const float *scales) {
            f16v s;
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] = 0.0f;

            // Operands are read kAhead steps before the products that take them; the
            // first ones of the values before the weights are worked out.
            // piece 2 k + g of row n
            const int ln = this_lane(), kn = ln & 31;
            const int k_at = kn * S::ROW + (S::k_place(ln >> 5) ^ S::k_swizzle(kn)) * 16;
            auto key = [&](int k) { return *reinterpret_cast<const bf8v *>(stage + S::with_place(k_at, S::k_place(2 * k))); };
            // the operand of channels 32 i .. and keys 16 t + 8 a + 4 g .. + 3 (a < 2),
            // transposed by the reads: this lane brings 4 channels of one of those keys
            const int l16 = ln & 15, vr = 4 * (ln >> 5) + (l16 >> 2), cb = ln >> 4 & 1;
            const uint8_t *vp = stage + S::HALF;
            const int v_at = vr * S::ROW + (l16 & 1) * 8 + (S::v_place(2 * cb + (l16 >> 1 & 1)) ^ S::v_swizzle(vr)) * 16;
            auto value = [&](int x) {
                const int i = x >> 1, t = x & 1, at = S::with_place(v_at, S::v_place(4 * i)) + 16 * t * S::ROW;
                const s4v lo = read_transposed(vp + at), hi = read_transposed(vp + (at + 8 * S::ROW));
                return __builtin_bit_cast(bf8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            };
            // (e4m3 rows' scales: asked for ahead where registers are left)
            constexpr bool EARLY = FMT == FMT_E4M3 && D < 256;
            float4 ks[4], vs[4];
            const float *scale_at = scales + 4 * (ln >> 5);
            bf8v ring[kAhead + 1];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) ring[k] = key(k);
            bf8v q_first[QL + 1];
#pragma unroll
            for (int k = 0; k < QL; ++k) q_first[k] = __builtin_bit_cast(bf8v, q_lds[(wave * QL + k) * 64 + ln]);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (k + kAhead < KS) ring[(k + kAhead) % (kAhead + 1)] = key(k + kAhead);
                if constexpr (EARLY)
                    if (k == KS - kAhead)
#pragma unroll
                        for (int a = 0; a < 4; ++a) ks[a] = *reinterpret_cast<const float4 *>(scale_at + 8 * a);
                __builtin_amdgcn_sched_barrier(0);
                s = mfma32(ring[k % (kAhead + 1)], k < QL ? q_first[k < QL ? k : 0] : q[k], s);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int x = 0; x < kAhead; ++x) ring[x] = value(x);
            if constexpr (EARLY)
#pragma unroll
                for (int a = 0; a < 4; ++a) vs[a] = *reinterpret_cast<const float4 *>(scale_at + S::KEYS + 8 * a);
            __builtin_amdgcn_sched_barrier(0);
            // lane (n, g) has of column n the keys 8 a + 4 g + b (a, b < 4) of the 32
            // (The weights go into the second product in bf16, rounded to nearest, up to
            // 2^-8 of each term, as the bf16 result's own rounding; the sums keep the fp32
            // values.  A second product for what that leaves, as steps have it, whose
            // bound is memory: 2,730 rows over 16,000 keys of 256 channels in bf16 1,386
            // us instead of 1,013, 2,048 of 128 815 instead of 623, of 64 513 instead of
            // 392; the other formats alike.)
            bf8v pb[2];
            // Any base within reach of the maximum does: scores are taken from the one
            // that is there, and it moves, to 2^8 above the maximum, only when that has
            // passed it.  (e4m3: the keys' scales in LDS have the call's in them.)
            const bool unset = mx == -INFINITY;
            const float base = unset ? 0.0f : mx;
            if constexpr (FMT == FMT_E4M3) {
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    float4 f;
                    if constexpr (EARLY) {
                        f = ks[a];
                    } else {
                        __builtin_amdgcn_sched_barrier(0);
                        f = *reinterpret_cast<const float4 *>(scale_at + 8 * a);
                    }
                    s[4 * a] = fmaf(s[4 * a], f.x, -base), s[4 * a + 1] = fmaf(s[4 * a + 1], f.y, -base);
                    s[4 * a + 2] = fmaf(s[4 * a + 2], f.z, -base), s[4 * a + 3] = fmaf(s[4 * a + 3], f.w, -base);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = fmaf(s[e], scale, -base);
            }
            const int from = first + (this_lane() >> 5) * 4 - K.kv;          // the lane's first key's place in the pass
            // bit i: the lane's key i of the 32 (8 a + b), in a window
            uint32_t in_sight = ~0u;
            if constexpr (WINDOW)
                if (tail) {
                    const uint32_t rows = seen[wave * 32 + (this_lane() & 31)];
                    in_sight = from >= kMaxWindowRows ? 0 : from >= 0 ? rows >> from : from <= -32 ? ~0u : rows << -from | ~(~0u << -from);
                }
            auto sees = [&](int e) {
                const int at = 8 * (e / 4) + (e & 3);
                return WINDOW ? (bool)(in_sight >> at & 1) : at <= row - from;
            };
            if (tail)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] = sees(e) ? s[e] : -INFINITY;
            float top = fmaxf(s[0], s[1]);
#pragma unroll
            for (int e = 2; e < 16; ++e) top = fmaxf(top, s[e]);
            top = max_halves(top);
            const bool passed = top > (unset ? -INFINITY : 0.0f);
            if (__ballot(passed)) {
                const float by = passed ? top + 8.0f : 0.0f, back = __builtin_amdgcn_exp2f(mx - (base + by));
#pragma unroll
                for (int e = 0; e < 16; ++e) s[e] -= by;
                if (passed) mx = base + by;
                sum *= back;
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[i][e] *= back;
            }
            float ps = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[e] = __builtin_amdgcn_exp2f(s[e]);
                ps += s[e];
            }
            sum += ps;
            if constexpr (FMT == FMT_E4M3) {
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    float4 f;
                    if constexpr (EARLY) {
                        f = vs[a];
                    } else {
                        __builtin_amdgcn_sched_barrier(0);
                        f = *reinterpret_cast<const float4 *>(scale_at + S::KEYS + 8 * a);
                    }
                    s[4 * a] *= f.x, s[4 * a + 1] *= f.y, s[4 * a + 2] *= f.z, s[4 * a + 3] *= f.w;
                }
                if (tail)                  // a masked row's scale may be anything
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] = sees(e) ? s[e] : 0.0f;
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint4 x = {pack2(s[8 * t], s[8 * t + 1]), pack2(s[8 * t + 2], s[8 * t + 3]), pack2(s[8 * t + 4], s[8 * t + 5]),
                                 pack2(s[8 * t + 6], s[8 * t + 7])};
                pb[t] = __builtin_bit_cast(bf8v, x);
            }
#pragma unroll
            for (int x = 0; x < 2 * NT; ++x) {
                if (x + kAhead < 2 * NT) ring[(x + kAhead) % (kAhead + 1)] = value(x + kAhead);
                __builtin_amdgcn_sched_barrier(0);
                o[x >> 1] = mfma32(ring[x % (kAhead + 1)], pb[x & 1], o[x >> 1]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        auto compute = [&](int tile, const uint8_t *stage, const float *scales) {
            if (!busy) return;
            const int first = K.k0 + tile * S::KEYS;
            if (WINDOW || first <= see_hi) multiply(first + S::KEYS > (WINDOW ? K.kv : see_lo + 1), first, stage, scales);
        };

        // The first stage is on its way while the stream's pages are checked: entries
        // that name no page are taken for page 0 until then.
        look(0);
        load(st0);
        look(1);
        ok = pages_ok(A, K, S::THREADS) && ok;
        if (lane == 0) wave_ok[wave] = ok;
        if (threadIdx.x == 0) {
            bad = 0;
            kept = K;
        }
        lds_barrier();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) ok = ok && wave_ok[w];
        if (!ok) {
            if (K.nch > 1 && g == 0)
                if (col0 + n < K.cols) A.stat[pair_of(A.hq) * A.chunks + K.c] = make_float2(0.0f, kSkipped);
            wait_vmem();
            __syncthreads();
            continue;
        }
        if constexpr (FMT != FMT_BF16) {
            put(st0, sc0);
            load(nullptr);
            look(2);
        }
#pragma unroll
        for (int k = 0; k < QL; ++k) q_lds[(wave * QL + k) * 64 + this_lane()] = __builtin_bit_cast(uint4, q[k]);
        auto step = [&](int tile, uint8_t *stage, float *scales, uint8_t *next, float *next_scales) {
            // Over e4m3 rows of up to 128 channels half of the waves convert the next stage
            // before they multiply this one, the other half afterwards: while one of two
            // waves of a SIMD keeps the vector unit busy, the other has the matrix unit (a
            // resumed prompt of 32 and 8 heads of 128 1,284 and 1,255 us; the other rows,
            // which are converted in fewer steps, gain nothing, or lose 2 %).
            constexpr bool HALVES = FMT == FMT_E4M3 && D < 256;
            const bool late = HALVES && wave >= WAVES / 2;
            auto bring = [&] {
                if (tile + 1 >= tiles) return;
                if constexpr (FMT == FMT_BF16) {
                    load(next);
                    look(tile + 2);
                } else {
                    put(next, next_scales);
                    load(nullptr);
                    look(tile + 3);
                }
            };
            if constexpr (HALVES) lds_barrier();
            else wait_and_meet<0>();
            if (!late) bring();
            // 0 * inf is NaN: a stage with keys that some column does not see (or past
            // the stream's end) has its values that are not finite left out, to be added
            // at the end to the columns that see them (a carry into bits 15 and 31 marks
            // an exponent of all ones)
            const int first = K.k0 + tile * S::KEYS;
            if (first + S::KEYS > all_see) {
                bool found = false;
#pragma unroll
                for (int i = 0; i < S::HALF / 16 / S::THREADS; ++i) {
                    uint4 *at = reinterpret_cast<uint4 *>(stage + S::HALF) + i * S::THREADS + wave * 64 + this_lane(), x = *at;
                    const uint32_t m0 = ((x.x & 0x7f807f80u) + 0x00800080u) & 0x80008000u, m1 = ((x.y & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                    const uint32_t m2 = ((x.z & 0x7f807f80u) + 0x00800080u) & 0x80008000u, m3 = ((x.w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
                    if (m0 | m1 | m2 | m3) {
                        found = true;
                        x.x &= ~((m0 >> 15) * 0xffffu), x.y &= ~((m1 >> 15) * 0xffffu);
                        x.z &= ~((m2 >> 15) * 0xffffu), x.w &= ~((m3 >> 15) * 0xffffu);
                        *at = x;
                    }
                }
                if (found) bad = 1;
                lds_barrier();
            }
            compute(tile, stage, scales);
            if (late) bring();
        };
        for (int tile = 0; tile < tiles; tile += 2) {
            step(tile, st0, sc0, st1, sc1);
            if (tile + 1 < tiles) step(tile + 1, st1, sc1, st0, sc0);
        }

        // Results leave through LDS, up to 128 channels of a wave's 32 columns at a time, so that the gates' and the results' rows are read and written in runs.
        // A column's 16-byte pieces are exchanged by its number.
        __syncthreads();
        const_args *B = fresh_args();
        const PromptPiece E = {wave_int(kept.h), wave_int(kept.rt), wave_int(kept.c), wave_int(kept.s), wave_int(kept.r0), wave_int(kept.m),
                               wave_int(kept.kv), wave_int(kept.len), wave_int(kept.k0), wave_int(kept.k1), wave_int(kept.nch), wave_int(kept.cols)};
        const uint16_t *const gate_at = B->gate;
        const int64_t gate_row = B->gate_row, gate_head = B->gate_head;
        const int first_col = E.rt * S::COLS + wave * 32, hq = B->hq, chunks = B->chunks;
        constexpr int FIT = S::BYTES / (WAVES / 2 * 32 * 4), CH = FIT < D ? FIT : D, PC = CH / 4, LPC = CH / 8;    // channels; pieces of a column; lanes that read it
        static_assert(CH >= 32 && D % CH == 0, "");
        uint8_t *mine = wave < WAVES / 2 ? st0 + wave * (32 * CH * 4) : st1 + (wave - WAVES / 2) * (32 * CH * 4);
        const int ln = this_lane(), en = ln & 31, eg = ln >> 5;
        const int sees = WINDOW ? E.kv : E.kv + E.rt * S::COLS / B->group + 1, bad_from = E.k0 + max(0, (sees - E.k0) / S::KEYS) * S::KEYS;       // the first stage that was looked at
        const float l = sum_halves(sum);
        if (E.nch > 1 && eg == 0 && first_col + en < E.cols) B->stat[pair_of(hq) * chunks + E.c] = make_float2(mx, l);
        if (bad) {
            for (int key = bad_from; key < E.k1; ++key) {
                const int j = key - E.kv;
                if (j >= 0 && !(WINDOW ? seen[first_col + en - E.rt * S::COLS] >> j & 1 : j <= row)) continue;
                const int id = B->table[(size_t)E.s * B->max_blocks + (key >> B->kv.page_shift)];
                const size_t at = (((size_t)id * B->kv.hkv + E.h) << B->kv.page_shift) + (key & ((1 << B->kv.page_shift) - 1));
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const uint2 w = cached_values4<D, FMT>(B->kv.v, B->kv.v_exp, at, 32 * i + 8 * a + 4 * eg);
                        o[i][4 * a] += not_finite(w.x << 16), o[i][4 * a + 1] += not_finite(w.x & 0xffff0000u);
                        o[i][4 * a + 2] += not_finite(w.y << 16), o[i][4 * a + 3] += not_finite(w.y & 0xffff0000u);
                        __builtin_amdgcn_sched_barrier(0);
                    }
            }
        }
        const float inv = E.nch == 1 ? 1.0f / l : 1.0f;
#pragma unroll
        for (int part = 0; part < D / CH; ++part) {
            constexpr int RUNS = 32 * LPC / 64;
            uint2 gate[RUNS][2];
            if (part > 0) __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < CH / 32; ++i)
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const f16v &x = o[part * (CH / 32) + i];
                    *reinterpret_cast<float4 *>(mine + (en * PC + ((8 * i + 2 * a + eg) ^ (en & (PC - 1)))) * 16) =
                        make_float4(x[4 * a] * inv, x[4 * a + 1] * inv, x[4 * a + 2] * inv, x[4 * a + 3] * inv);
                }
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int y = 0; y < RUNS; ++y) gate[y][0] = gate[y][1] = make_uint2(0, 0);
            if (E.nch == 1 && gate_at)
#pragma unroll
                for (int y = 0; y < RUNS; ++y) {
                    const int2 p = pairs[wave * 32 + y * (64 / LPC) + ln / LPC];
                    const uint16_t *from = gate_at + p.x * gate_row + p.y * gate_head + (part * CH + 8 * (ln % LPC));
                    gate[y][0] = reinterpret_cast<const uint2 *>(from)[0], gate[y][1] = reinterpret_cast<const uint2 *>(from)[1];
                }
#pragma unroll
            for (int y = 0; y < RUNS; ++y) {
                const int n = y * (64 / LPC) + ln / LPC, x = ln % LPC, d = part * CH + 8 * x;
                const float4 u = *reinterpret_cast<const float4 *>(mine + (n * PC + ((2 * x) ^ (n & (PC - 1)))) * 16);
                const float4 v = *reinterpret_cast<const float4 *>(mine + (n * PC + ((2 * x + 1) ^ (n & (PC - 1)))) * 16);
                __builtin_amdgcn_sched_barrier(0);
                if (first_col + n >= E.cols) continue;
                const int2 p = pairs[wave * 32 + n];
                const size_t pair = (size_t)p.x * hq + p.y;
                if (E.nch == 1) {
                    const uint2 a = gated4(u, gate_at != nullptr, gate[y][0]), b = gated4(v, gate_at != nullptr, gate[y][1]);
                    *reinterpret_cast<uint4 *>(B->out + pair * D + d) = make_uint4(a.x, a.y, b.x, b.y);
                } else {
                    float *to = B->part + (pair * chunks + E.c) * D + d;
                    *reinterpret_cast<float4 *>(to) = u;
                    *reinterpret_cast<float4 *>(to + 4) = v;
                }
            }
        }
        __syncthreads();
    }
}

// Waves of a workgroup, that is columns that share what is loaded and converted, and
// waves of a SIMD, that is registers of each.  16,384 rows in 8 waves and in 4: 256
// channels (24 query and 4 kv heads) in bf16 2,715 us and 2,905, over 4 bits 2,660 and
// 2,886; 128 channels (32 and 8) in bf16 2,203 and 2,037, over 4 bits 2,119 and
// 1,998, in e4m3 2,550 and 2,600, a resumed prompt 1,255 and 1,351: there what is
// converted weighs most.  Of 256 channels both are here, for calls that leave some of
// the chip empty (prompt_plan): 2,048 fresh rows in bf16 105 and 97 us, over 4 bits
// 114 and 105, 1,024 rows 63 and 54, 64 rows 16 and 14; over cached rows, where pieces
// are cut to fill the chip, 512 rows over 32,000 in 4 bits 386 and 442.
constexpr int prompt_waves(int d, int fmt) { return d == 256 || (d == 128 && fmt == FMT_E4M3) ? 8 : 4; }
constexpr bool prompt_has_both(int d, int fmt) { return d == 256 && fmt != FMT_E4M3; }        // (e4m3: queries in LDS)
constexpr int prompt_per_simd(int d, int fmt) { return d == 64 ? (fmt == FMT_E4M3 ? 3 : 4) : d == 128 && fmt != FMT_E4M3 ? 3 : 2; }

template <int D, int FMT>
hipError_t launch_prompt_d(const AttnArgs &A, int split_keys, int waves, unsigned blocks, hipStream_t stream)
{
    constexpr int WAVES = prompt_waves(D, FMT), PER_SIMD = prompt_per_simd(D, FMT);
    if constexpr (prompt_has_both(D, FMT))
        if (waves == 4) {
            prompt_kernel<D, FMT, 4, PER_SIMD, false><<<blocks, 256, 0, stream>>>(A, split_keys);
            return hipGetLastError();
        }
    prompt_kernel<D, FMT, WAVES, PER_SIMD, false><<<blocks, 64 * WAVES, 0, stream>>>(A, split_keys);
    return hipGetLastError();
}

template <int D>
hipError_t launch_prompt_fmt(const AttnArgs &A, int split_keys, int waves, unsigned blocks, hipStream_t stream)
{
    switch (format_of(A.kv)) {
    case FMT_BF16: return launch_prompt_d<D, FMT_BF16>(A, split_keys, waves, blocks, stream);
    case FMT_E4M3: return launch_prompt_d<D, FMT_E4M3>(A, split_keys, waves, blocks, stream);
    default: return launch_prompt_d<D, FMT_MXFP4>(A, split_keys, waves, blocks, stream);
    }
}

// workgroups that the chip holds at once
int prompt_slots(int d, int fmt, int waves) { return 256 * 4 * prompt_per_simd(d, fmt) / waves; }

// Chunks of the longest stream: by the time that the call would take, in keys of a
// workgroup, if its longest stream were the only one.  A workgroup's beginning and
// end cost as much as 160 keys, a chunk's parts 400 more, and the join 600.  What
// limits the call is its longest piece, or all of them spread over the chip and what
// is left to end on: where the pieces are alike, since most of their keys are cached,
// the rest of a last round (half a piece once the rounds are many), less where the
// last ones are short.  Workgroups that have their CU to themselves are faster.  (24
// query and 4 kv heads of 256 in bf16: a fresh prompt of 2,048 rows takes 97 us whole
// and 130 in two chunks; 512 rows over 32,000 cached keys 1,448 us whole, 373 in 5
// chunks, which are 240 pieces for the chip's 256 places, 570 in 6, 446 in 8, 485 in
// 12 and 419 in 16.)
//
// What is known here is the call's bounds alone, so loose ones cost: those 512 rows
// take 610 us under a max_kv of 65,536 (3 chunks), 1,177 under 131,072 (2), 1,448 under
// 262,144 or with room for 8,306 rows (uncut), and beside 8,306 fresh rows, which take
// 352 by themselves, 1,462; 65 rows over 131,000 4-bit keys 256 us under their own
// bounds, 413 under 262,144, 6,155 with room for 8,306 rows.
constexpr int kPromptRounds = 4;           // pieces of a call that is cut, in workgroups that the chip holds
int most_chunks(int max_kv) { return at_most(kMaxChunks, max_kv / 256); }

int prompt_chunks(long long tiles, int slots, int total_rows, int max_kv)
{
    const double cached = max_kv > total_rows ? max_kv - total_rows : 0, keys = max_kv, mean = (cached + keys) / 2;
    int best = 1;
    double least = 0;
    for (int c = 1; c == 1 || (c <= most_chunks(max_kv) && tiles * c <= (long long)kPromptRounds * slots); ++c) {
        const double parts = c > 1 ? 1 + (c - 1) * mean / keys : 0;       // of a mean tile
        const double rounds = (double)(tiles * c) / slots, full = rounds < 1 ? rounds : 1.0;
        const double left = rounds <= 1 ? 1 - rounds : rounds <= 2 ? 2 - rounds : 0.5;
        const double all = tiles * (mean + 160 + 400 * parts) / slots + (left * cached + (keys - cached) / 8) / c;
        const double one = (keys / c + 160 + (c > 1 ? 400 : 0)) * (0.6 + 0.4 * full);
        const double cost = (all > one ? all : one) + (c > 1 ? 600 : 0);
        if (c == 1 || cost < least) best = c, least = cost;
    }
    return best;
}

struct PromptPlan {
    int waves, chunks, split_keys;
    long long blocks;
};
long long prompt_tiles(int hq, int hkv, int cols, long long total_rows) { return (total_rows * (hq / hkv) + cols - 1) / cols * hkv; }
PromptPlan prompt_plan(int hq, int hkv, int d, int fmt, int n_streams, int total_rows, int max_kv)
{
    const int rows = n_streams < total_rows ? n_streams : total_rows;
    PromptPlan P;
    P.waves = prompt_waves(d, fmt);
    // prompts that are mostly fresh and leave some of the chip empty: twice the workgroups
    if (prompt_has_both(d, fmt) && max_kv / 2 <= total_rows && prompt_tiles(hq, hkv, 32 * P.waves, total_rows) <= prompt_slots(d, fmt, P.waves))
        P.waves = 4;
    const int cols = 32 * P.waves;
    P.chunks = prompt_chunks(prompt_tiles(hq, hkv, cols, total_rows), prompt_slots(d, fmt, P.waves), total_rows, max_kv);
    P.split_keys = ceil_div(ceil_div(max_kv, P.chunks), 64) * 64;
    P.blocks = ((long long)total_rows * (hq / hkv) / cols + rows) * hkv * P.chunks;       // at most
    return P;
}
size_t part_bytes(int hq, int d, int total_rows, int chunks)
{
    return chunks <= 1 ? 0 : (size_t)total_rows * hq * chunks * (sizeof(float) * d + sizeof(float2));
}

}  // namespace

hipError_t launch_wide4(const AttnArgs &A, long long pieces, hipStream_t stream)
{
    const unsigned blocks = (unsigned)(pieces < 2048 ? pieces : 2048);
    switch (A.kv.d) {
    case 64: prompt_kernel<64, FMT_MXFP4, 4, 2, true><<<blocks, 256, 0, stream>>>(A, 0); break;
    case 128: prompt_kernel<128, FMT_MXFP4, 4, 2, true><<<blocks, 256, 0, stream>>>(A, 0); break;
    default: prompt_kernel<256, FMT_MXFP4, 4, 2, true><<<blocks, 256, 0, stream>>>(A, 0); break;
    }
    return hipGetLastError();
}

size_t prompt_workspace_bytes(int hq, int hkv, int d, int fmt, int n_streams, int total_rows, int max_kv)
{
    return part_bytes(hq, d, total_rows, prompt_plan(hq, hkv, d, fmt, n_streams, total_rows, max_kv).chunks);
}

// Of all calls up to these sizes, in any format: one with fewer rows may be cut into
// more chunks, but what is cut has kPromptRounds * slots pieces of as many pairs as
// a tile has columns at most.
size_t prompt_workspace_most(int hq, int d, int total_rows, int max_kv)
{
    const int chunks = most_chunks(max_kv);
    if (chunks <= 1) return 0;
    size_t pairs = 0;
    for (int fmt : {FMT_BF16, FMT_E4M3, FMT_MXFP4}) {
        const size_t held = (size_t)kPromptRounds * prompt_slots(d, fmt, 4) * 32 * 4;      // (with 8 waves the same)
        pairs = held > pairs ? held : pairs;
    }
    const size_t all = (size_t)total_rows * hq * chunks;
    return (all < pairs ? all : pairs) * (sizeof(float) * d + sizeof(float2));
}

bool prompt_fits(const AttnArgs &A)
{
    return prompt_plan(A.hq, A.kv.hkv, A.kv.d, format_of(A.kv), A.n_streams, A.total_rows, A.max_kv).blocks <= kMaxGroups / 2
           && (long long)A.total_rows * A.hq <= (1 << 26) - 4;
}

hipError_t launch_prompt(AttnArgs A, void *workspace, hipStream_t stream)
{
    const PromptPlan P = prompt_plan(A.hq, A.kv.hkv, A.kv.d, format_of(A.kv), A.n_streams, A.total_rows, A.max_kv);
    A.max_rows = A.total_rows;
    A.chunks = P.chunks;
    A.part = static_cast<float *>(workspace);
    A.stat = reinterpret_cast<float2 *>(A.part + (size_t)A.total_rows * A.hq * A.chunks * A.kv.d);
    hipError_t rc;
    switch (A.kv.d) {
    case 64: rc = launch_prompt_fmt<64>(A, P.split_keys, P.waves, (unsigned)P.blocks, stream); break;
    case 128: rc = launch_prompt_fmt<128>(A, P.split_keys, P.waves, (unsigned)P.blocks, stream); break;
    default: rc = launch_prompt_fmt<256>(A, P.split_keys, P.waves, (unsigned)P.blocks, stream); break;
    }
    if (rc != hipSuccess || A.chunks == 1) return rc;
    return launch_join(A, true, P.split_keys, stream);
}

}  // namespace gdn
