// Attention of whole prompts over the paged cache.  Contract in
// include/libgdn.h (gdn_attn_prompt).
//
// Row t of a stream sees its cache rows 0 .. kv_len + t.  As in the kernels of
// steps and windows, the (row, query head) pairs of a stream and kv head are the
// columns of S^T = K Q^T and O^T = V^T P^T, with one pass over the keys that
// keeps the running maximum and sum of each column.
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

constexpr int kSub = 32;       // keys of a matrix instruction's tile

// A stage of keys and values in LDS, in bf16: KEYS rows of K, then of V.  The
// 16-byte pieces of a row of K are exchanged by a function of the row, so that 16
// rows of one operand lie in different banks; rows of V likewise, the 16 channels
// of a transposing read (32 bytes) together.
template <int D, int FMT, int WAVES, int TILES, int KEYS_>
struct PromptShape {
    static constexpr int THREADS = 64 * WAVES, COLS = 32 * TILES * WAVES;
    static constexpr int KEYS = KEYS_, ROW = 2 * D, HALF = KEYS * ROW, BYTES = 2 * HALF;
    static constexpr int PIECES = ROW / 16, ROWS = 1024 / ROW;    // of a direct load
    static __device__ __forceinline__ int k_swizzle(int key) { return ROW >= 256 ? key & 15 : key >> 1 & 7; }
    static __device__ __forceinline__ int v_swizzle(int key) { return 2 * (ROW >= 256 ? key & 7 : key >> 1 & 3); }
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

// The pieces of all streams, in stream order, 64 streams a step; of a stream the
// last rows, which see the most keys, first, and the kv heads innermost, so that
// the workgroups of a head meet in as few XCDs as can be.
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
        }
        const int incl = wave_running_sum(count), all = __builtin_amdgcn_readlane(incl, 63);
        if (item >= all) {
            item -= all;
            continue;
        }
        const int l = __builtin_ctzll(__ballot(incl > item));
        int x = item - (l ? __builtin_amdgcn_readlane(incl, l - 1) : 0);
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
__device__ __forceinline__ uint2 cached_values4(const KvArgs &kv, size_t row, int d)
{
    if constexpr (FMT == FMT_BF16) {
        return *reinterpret_cast<const uint2 *>(kv.v + (row * D + d) * 2);
    } else if constexpr (FMT == FMT_E4M3) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(kv.v + row * D + d);
        return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                          __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)));
    } else {
        const uint32_t w = *reinterpret_cast<const uint16_t *>(kv.v + (row * D + d) / 2);
        const float f = mx_scale(kv.v_exp[row * (D / kMxBlock) + d / kMxBlock]);
        return make_uint2(mx_pair<0>(w, f), mx_pair<1>(w, f));
    }
}
__device__ __forceinline__ float not_finite(uint32_t bits) { return (bits & 0x7f800000u) == 0x7f800000u ? __uint_as_float(bits) : 0.0f; }

template <int D, int FMT, int WAVES, int TILES, int KEYS, bool WINDOW>
__global__ __launch_bounds__(64 * WAVES, 2) void prompt_kernel(const AttnArgs A, const int split_keys)
{
    using S = PromptShape<D, FMT, WAVES, TILES, KEYS>;
    constexpr int KS = D / 16, NT = D / 32, T = TILES;
    constexpr int NK = S::HALF / 1024, PER = 2 * NK / WAVES;     // direct loads of a stage's keys; of a wave, in all
    static_assert(NK % WAVES == 0, "");
    // separate arrays, so that loads into one are known not to touch the other
    __shared__ __align__(1024) uint8_t st0[S::BYTES], st1[S::BYTES];
    __shared__ __align__(16) float sc0[S::SCALES], sc1[S::SCALES];
    __shared__ int wave_ok[WAVES], bad;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, n = lane & 31, g = lane >> 5;
    const float scale = A.scale == 0.0f ? 1.0f : fabsf(A.scale);
    PromptPiece K;
    for (int item = blockIdx.x; find_piece<S::COLS, WINDOW>(A, split_keys, item, K); item += gridDim.x) {
        bool ok = pages_ok(A, K, S::THREADS);
        const int col0 = K.rt * S::COLS + wave * 32 * T;            // the wave's first column
        const bool busy = col0 < K.cols;                            // waves without columns only load
        const int t_lo = min(col0, K.cols - 1) / A.group, t_hi = min(col0 + 32 * T, K.cols) - 1;   // rows of the wave
        const int see_lo = K.kv + t_lo, see_hi = K.kv + t_hi / A.group;      // the last key that the first and the last one see
        int row[T], head[T];
        uint32_t seen[T];
#pragma unroll
        for (int c = 0; c < T; ++c) {
            const int col = min(col0 + 32 * c + n, K.cols - 1);     // past the last one: that one again, not stored
            const int t = col / A.group;
            row[c] = t;
            head[c] = K.h * A.group + col - t * A.group;
            seen[c] = 0;
            if constexpr (WINDOW) seen[c] = seen_rows(A, K.r0, K.m, t, ok);
        }
        if (lane == 0) wave_ok[wave] = ok;
        if (threadIdx.x == 0) bad = 0;
        __syncthreads();
        ok = true;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) ok = ok && wave_ok[w];
        __syncthreads();
        auto part_at = [&](int c) { return ((size_t)(K.r0 + row[c]) * A.hq + head[c]) * A.chunks + K.c; };
        if (!ok) {
            if (K.nch > 1 && g == 0)
#pragma unroll
                for (int c = 0; c < T; ++c)
                    if (col0 + 32 * c + n < K.cols) A.stat[part_at(c)] = make_float2(0.0f, kSkipped);
            continue;
        }
        if (K.k0 >= K.k1) continue;                 // a chunk past all that the tile sees
        bf8v q[T][KS];
#pragma unroll
        for (int c = 0; c < T; ++c) {
            const uint16_t *p = A.q + ((size_t)(K.r0 + row[c]) * A.hq + head[c]) * D + 8 * g;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                uint4 x = *reinterpret_cast<const uint4 *>(p + 16 * k);
                if (A.scale <= 0.0f) {      // scores are multiplied by a positive scale: a negative one changes the queries' signs, 0 makes them 0
                    const uint32_t sign = A.scale < 0.0f ? 0x80008000u : 0u, keep = A.scale < 0.0f ? ~0u : 0u;
                    x = make_uint4((x.x & keep) ^ sign, (x.y & keep) ^ sign, (x.z & keep) ^ sign, (x.w & keep) ^ sign);
                }
                q[c][k] = __builtin_bit_cast(bf8v, x);
            }
        }
        f16v o[T][NT];
        float mx[T], sum[T];
#pragma unroll
        for (int c = 0; c < T; ++c) {
            mx[c] = -INFINITY;
            sum[c] = 0.0f;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[c][i][e] = 0.0f;
        }
        // keys that every column of the workgroup sees
        const int all_see = WINDOW ? K.kv : K.kv + K.rt * S::COLS / A.group + 1;

        // cache row of a key's group of 16 (past the stream's end: of its last keys)
        const int *table = A.table + (size_t)K.s * A.max_blocks;
        auto cache_row = [&](int key) {
            key = min(key, (K.len - 1) & ~15);
            return ((table[key >> A.kv.page_shift] * A.kv.hkv + K.h) << A.kv.page_shift) + (key & ((1 << A.kv.page_shift) - 1));
        };
        const int tiles = ceil_div(K.k1 - K.k0, S::KEYS);
        constexpr int GROUPS = FMT == FMT_BF16 ? PER / 2 : S::LOADS;
        int ahead[GROUPS], ahead_scale = 0;
        uint4 raw[FMT == FMT_BF16 ? 1 : S::LOADS];
        uint32_t raw_scale[FMT == FMT_BF16 ? 1 : S::LOADS];
        float row_scale = 0.0f;
        // unit x of a thread: keys and then values, whole rows in order
        auto unit = [&](int x, int &is_v, int &r, int &p) {
            const int u = x * S::THREADS + threadIdx.x;
            is_v = u >= S::UNITS;
            r = (u - is_v * S::UNITS) / S::PER_ROW;
            p = u % S::PER_ROW;
            return u < 2 * S::UNITS;
        };
        auto look = [&](int tile) {
            const int key = K.k0 + min(tile, tiles - 1) * S::KEYS;
            if constexpr (FMT == FMT_BF16) {
#pragma unroll
                for (int x = 0; x < GROUPS; ++x) ahead[x] = cache_row(key + ((x * WAVES + wave) * S::ROWS & ~15));
            } else {
#pragma unroll
                for (int x = 0; x < GROUPS; ++x) {
                    int is_v, r, p;
                    unit(x, is_v, r, p);
                    ahead[x] = cache_row(key + (r & ~15)) + (r & 15);
                }
                if constexpr (FMT == FMT_E4M3) ahead_scale = cache_row(key + (threadIdx.x % S::KEYS & ~15)) + (threadIdx.x & 15);
            }
        };
        // bf16: straight to a stage; else to registers, for put
        auto load = [&](uint8_t *stage) {
            if constexpr (FMT == FMT_BF16) {
                const int in = wave * S::ROWS % 16 + lane / S::PIECES;         // row in its group
                const uint32_t k_off = in * S::ROW + (lane % S::PIECES ^ S::k_swizzle(in)) * 16, v_off = in * S::ROW + (lane % S::PIECES ^ S::v_swizzle(in)) * 16;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const bool is_k = j < PER / 2;
                    const int x = j % (PER / 2);
                    const uint8_t *p = (is_k ? A.kv.k : A.kv.v) + (size_t)__builtin_amdgcn_readfirstlane(ahead[x]) * S::ROW;
                    __builtin_amdgcn_global_load_lds((global_void *)(p + (is_k ? k_off : v_off)),
                                                     (lds_void *)(stage + (j * WAVES + wave) * 1024), 16, 0, 0);
                }
            } else {
#pragma unroll
                for (int x = 0; x < S::LOADS; ++x) {
                    int is_v, r, p;
                    if (!unit(x, is_v, r, p)) continue;
                    raw[x] = *reinterpret_cast<const uint4 *>((is_v ? A.kv.v : A.kv.k) + ((size_t)ahead[x] * S::CODES + 16 * p));
                    if constexpr (FMT == FMT_MXFP4) raw_scale[x] = (is_v ? A.kv.v_exp : A.kv.k_exp)[(size_t)ahead[x] * (D / kMxBlock) + p];
                }
                if constexpr (FMT == FMT_E4M3)
                    if (threadIdx.x < 2 * S::KEYS) row_scale = (threadIdx.x < S::KEYS ? A.kv.k_scale : A.kv.v_scale)[(size_t)ahead_scale];
            }
        };
        // rows in registers, to bf16, to a stage
        auto put = [&](uint8_t *stage, float *scales) {
            if constexpr (FMT != FMT_BF16) {
#pragma unroll
                for (int x = 0; x < S::LOADS; ++x) {
                    int is_v, r, p;
                    if (!unit(x, is_v, r, p)) continue;
                    uint8_t *to = stage + is_v * S::HALF + r * S::ROW;
                    const int sw = is_v ? S::v_swizzle(r) : S::k_swizzle(r);
                    const uint32_t w[4] = {raw[x].x, raw[x].y, raw[x].z, raw[x].w};
                    if constexpr (FMT == FMT_MXFP4) {
                        const float f = mx_scale(raw_scale[x]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(to + ((4 * p + i) ^ sw) * 16) = mx_values8(w[i], f);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t y[4];
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                y[2 * j] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + j], 1.0f, false));
                                y[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[2 * i + j], 1.0f, true));
                            }
                            *reinterpret_cast<uint4 *>(to + ((2 * p + i) ^ sw) * 16) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                }
                if constexpr (FMT == FMT_E4M3)
                    if (threadIdx.x < 2 * S::KEYS) scales[threadIdx.x] = row_scale;
            }
        };

        // 32 keys from `first`, rows sub * 32 .. of the stage.  tail: some column does not see all of them.
        auto multiply = [&](bool tail, int first, int sub, const uint8_t *stage, const float *scales) {
            f16v acc[T];
#pragma unroll
            for (int c = 0; c < T; ++c)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[c][e] = 0.0f;
            const uint8_t *kr = stage + (sub * kSub + n) * S::ROW;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (k % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                const bf8v a = *reinterpret_cast<const bf8v *>(kr + ((2 * k + g) ^ S::k_swizzle(n)) * 16);
#pragma unroll
                for (int c = 0; c < T; ++c) acc[c] = mfma32(a, q[c][k], acc[c]);
            }
            // lane (n, g) has of column n the keys 8 a + 4 g + b (a, b < 4) of the 32
            bf8v pb[T][2];
#pragma unroll
            for (int c = 0; c < T; ++c) {
                f16v &s = acc[c];
                if constexpr (FMT == FMT_E4M3) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const float4 f = *reinterpret_cast<const float4 *>(scales + sub * kSub + 8 * a + 4 * g);
                        s[4 * a] *= f.x, s[4 * a + 1] *= f.y, s[4 * a + 2] *= f.z, s[4 * a + 3] *= f.w;
                    }
                }
                uint32_t vis = 0xffffu;
                if (tail) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int j = first + 8 * (e / 4) + 4 * g + (e & 3) - K.kv;      // place in the pass
                        const bool sees = WINDOW ? (j < 0) | ((j < kMaxWindowRows) & (seen[c] >> (j & 31))) : j <= row[c];
                        s[e] = sees ? s[e] : -INFINITY;
                        if constexpr (FMT == FMT_E4M3) vis &= ~((uint32_t)!sees << e);
                    }
                }
                float tm = fmaxf(s[0], s[1]);
#pragma unroll
                for (int e = 2; e < 16; ++e) tm = fmaxf(tm, s[e]);
                // Any base within reach of the maximum does: it moves only when the
                // maximum has passed it, and then to 2^8 above that
                tm = max_halves(tm) * scale;
                tm = tm > mx[c] ? tm + 8.0f : mx[c];
                const float base = tm == -INFINITY ? 0.0f : tm;
                const float back = __builtin_amdgcn_exp2f(mx[c] - base);
                const bool moved = __ballot(tm != mx[c] && mx[c] != -INFINITY);
                mx[c] = tm;
                float ps = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], scale, -base));
                    ps += s[e];
                }
                sum[c] = fmaf(sum[c], back, ps);
                if constexpr (FMT == FMT_E4M3) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
                        const float4 f = *reinterpret_cast<const float4 *>(scales + S::KEYS + sub * kSub + 8 * a + 4 * g);
                        s[4 * a] *= f.x, s[4 * a + 1] *= f.y, s[4 * a + 2] *= f.z, s[4 * a + 3] *= f.w;
                    }
                    if (tail)                  // a masked row's scale may be anything
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[e] = vis >> e & 1 ? s[e] : 0.0f;
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const uint4 x = {pack2(s[8 * t], s[8 * t + 1]), pack2(s[8 * t + 2], s[8 * t + 3]), pack2(s[8 * t + 4], s[8 * t + 5]),
                                     pack2(s[8 * t + 6], s[8 * t + 7])};
                    pb[c][t] = __builtin_bit_cast(bf8v, x);
                }
                if (moved) {
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[c][i][e] *= back;
                }
            }
            // the operand of channels 32 i .. and keys 16 t + 8 a + 4 g .. + 3 (a < 2),
            // transposed by the reads: this lane brings 4 channels of one of those keys
            const int l16 = lane & 15, vr = 4 * g + (l16 >> 2), cb = lane >> 4 & 1;
            const uint8_t *vp = stage + S::HALF + (sub * kSub + vr) * S::ROW + (l16 & 3) * 8;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const int at = ((4 * i + 2 * cb) ^ S::v_swizzle(vr)) * 16 + 16 * t * S::ROW;
                    const s4v lo = read_transposed(vp + at), hi = read_transposed(vp + at + 8 * S::ROW);
                    const bf8v v = __builtin_bit_cast(bf8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                    for (int c = 0; c < T; ++c) o[c][i] = mfma32(v, pb[c][t], o[c][i]);
                }
            }
        };
        auto compute = [&](int tile, const uint8_t *stage, const float *scales) {
            if (!busy) return;
#pragma unroll 1
            for (int sub = 0; sub < S::KEYS / kSub; ++sub) {
                const int first = K.k0 + tile * S::KEYS + sub * kSub;
                if (first >= K.k1 || (!WINDOW && first > see_hi)) break;
                multiply(first + kSub > (WINDOW ? K.kv : see_lo + 1), first, sub, stage, scales);
            }
        };

        look(0);
        load(st0);
        look(1);
        if constexpr (FMT != FMT_BF16) {
            put(st0, sc0);
            load(nullptr);
            look(2);
        }
        auto step = [&](int tile, uint8_t *stage, float *scales, uint8_t *next, float *next_scales) {
            wait_and_meet<0>();
            if (tile + 1 < tiles) {
                if constexpr (FMT == FMT_BF16) {
                    load(next);
                    look(tile + 2);
                } else {
                    put(next, next_scales);
                    load(nullptr);
                    look(tile + 3);
                }
            }
            // 0 * inf is NaN: a stage with keys that some column does not see (or past
            // the stream's end) has its values that are not finite left out, to be added
            // at the end to the columns that see them (a carry into bits 15 and 31 marks
            // an exponent of all ones)
            const int first = K.k0 + tile * S::KEYS;
            if (first + S::KEYS > all_see) {
                bool found = false;
#pragma unroll
                for (int i = 0; i < S::HALF / 16 / S::THREADS; ++i) {
                    uint4 *at = reinterpret_cast<uint4 *>(stage + S::HALF) + i * S::THREADS + threadIdx.x, x = *at;
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
        };
        for (int tile = 0; tile < tiles; tile += 2) {
            step(tile, st0, sc0, st1, sc1);
            if (tile + 1 < tiles) step(tile + 1, st1, sc1, st0, sc0);
        }

        const int bad_from = K.k0 + max(0, (all_see - K.k0) / S::KEYS) * S::KEYS;       // the first stage that was looked at
#pragma unroll
        for (int c = 0; c < T; ++c) {
            const float l = sum_halves(sum[c]);
            if (col0 + 32 * c + n >= K.cols) continue;
            if (K.nch > 1 && g == 0) A.stat[part_at(c)] = make_float2(mx[c], l);
            const int r = K.r0 + row[c];
            if (bad) {
                for (int key = bad_from; key < K.k1; ++key) {
                    const int j = key - K.kv;
                    if (j >= 0 && !(WINDOW ? seen[c] >> j & 1 : j <= row[c])) continue;
                    const size_t at = (size_t)cache_row(key & ~15) + (key & 15);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            const uint2 w = cached_values4<D, FMT>(A.kv, at, 32 * i + 8 * a + 4 * g);
                            o[c][i][4 * a] += not_finite(w.x << 16), o[c][i][4 * a + 1] += not_finite(w.x & 0xffff0000u);
                            o[c][i][4 * a + 2] += not_finite(w.y << 16), o[c][i][4 * a + 3] += not_finite(w.y & 0xffff0000u);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                }
            }
            const float inv = 1.0f / l;
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int a = 0; a < 4; ++a) {
                    const int d = 32 * i + 8 * a + 4 * g;
                    const float4 x = make_float4(o[c][i][4 * a], o[c][i][4 * a + 1], o[c][i][4 * a + 2], o[c][i][4 * a + 3]);
                    if (K.nch == 1)
                        *reinterpret_cast<uint2 *>(A.out + ((size_t)r * A.hq + head[c]) * D + d) = finish4(A, x, inv, gates4(A, r, head[c], d));
                    else
                        *reinterpret_cast<float4 *>(A.part + part_at(c) * D + d) = x;
                }
        }
        __syncthreads();
    }
}

constexpr int kPromptCols = 256;
constexpr int kPromptPieces = 512;        // as many as a call is cut into where it has few tiles
constexpr int kPromptLeastKeys = 512;     // but of no fewer keys

// How many chunks the longest stream of a call with these bounds may have.
int prompt_chunks(long long tiles, int max_kv)
{
    const long long want = tiles >= kPromptPieces / 2 ? 1 : kPromptPieces / at_least(1, (int)tiles);
    return at_least(1, at_most((int)(want < kMaxChunks ? want : kMaxChunks), max_kv / kPromptLeastKeys));
}

long long prompt_tiles(int hq, int hkv, int total_rows)
{
    return ((long long)total_rows * (hq / hkv) + kPromptCols - 1) / kPromptCols * hkv;
}

template <int D, int FMT>
hipError_t launch_prompt_d(const AttnArgs &A, int split_keys, unsigned blocks, hipStream_t stream)
{
    if constexpr (D >= 128) prompt_kernel<D, FMT, 8, 1, 64, false><<<blocks, 512, 0, stream>>>(A, split_keys);
    else prompt_kernel<D, FMT, 4, 2, 64, false><<<blocks, 256, 0, stream>>>(A, split_keys);
    return hipGetLastError();
}

template <int D>
hipError_t launch_prompt_fmt(const AttnArgs &A, int split_keys, unsigned blocks, hipStream_t stream)
{
    switch (format_of(A.kv)) {
    case FMT_BF16: return launch_prompt_d<D, FMT_BF16>(A, split_keys, blocks, stream);
    case FMT_E4M3: return launch_prompt_d<D, FMT_E4M3>(A, split_keys, blocks, stream);
    default: return launch_prompt_d<D, FMT_MXFP4>(A, split_keys, blocks, stream);
    }
}

// at most so many pieces
long long prompt_pieces(const AttnArgs &A, int chunks)
{
    const long long tiles = (long long)A.total_rows * A.group / kPromptCols + (A.n_streams < A.total_rows ? A.n_streams : A.total_rows);
    return tiles * A.kv.hkv * chunks;
}

}  // namespace

hipError_t launch_wide4(const AttnArgs &A, long long pieces, hipStream_t stream)
{
    const unsigned blocks = (unsigned)(pieces < 2048 ? pieces : 2048);
    switch (A.kv.d) {
    case 64: prompt_kernel<64, FMT_MXFP4, 4, 1, 32, true><<<blocks, 256, 0, stream>>>(A, 0); break;
    case 128: prompt_kernel<128, FMT_MXFP4, 4, 1, 32, true><<<blocks, 256, 0, stream>>>(A, 0); break;
    default: prompt_kernel<256, FMT_MXFP4, 4, 1, 32, true><<<blocks, 256, 0, stream>>>(A, 0); break;
    }
    return hipGetLastError();
}

size_t prompt_workspace_bytes(int hq, int hkv, int d, int total_rows, int max_kv, bool or_less)
{
    auto bytes = [&](size_t rows, int chunks) { return chunks <= 1 ? 0 : rows * hq * chunks * (sizeof(float) * d + sizeof(float2)); };
    const long long all = prompt_tiles(hq, hkv, total_rows);
    size_t most = bytes(total_rows, prompt_chunks(all, max_kv));
    if (or_less)        // fewer rows may be cut into more chunks: the most rows of each number of tiles
        for (long long tiles = hkv; tiles < all && tiles < kPromptPieces / 2; tiles += hkv) {
            const long long rows = tiles / hkv * kPromptCols / (hq / hkv);
            const size_t b = bytes(rows < total_rows ? rows : total_rows, prompt_chunks(tiles, max_kv));
            most = b > most ? b : most;
        }
    return most;
}

bool prompt_fits(const AttnArgs &A)
{
    return prompt_pieces(A, prompt_chunks(prompt_tiles(A.hq, A.kv.hkv, A.total_rows), A.max_kv)) <= kMaxGroups / 2
           && (long long)A.total_rows * A.hq <= (1 << 26) - 4;
}

hipError_t launch_prompt(AttnArgs A, void *workspace, hipStream_t stream)
{
    A.max_rows = A.total_rows;
    A.chunks = prompt_chunks(prompt_tiles(A.hq, A.kv.hkv, A.total_rows), A.max_kv);
    A.part = static_cast<float *>(workspace);
    A.stat = reinterpret_cast<float2 *>(A.part + (size_t)A.total_rows * A.hq * A.chunks * A.kv.d);
    const int split_keys = ceil_div(ceil_div(A.max_kv, A.chunks), 64) * 64;
    const unsigned blocks = (unsigned)prompt_pieces(A, A.chunks);
    hipError_t rc;
    switch (A.kv.d) {
    case 64: rc = launch_prompt_fmt<64>(A, split_keys, blocks, stream); break;
    case 128: rc = launch_prompt_fmt<128>(A, split_keys, blocks, stream); break;
    default: rc = launch_prompt_fmt<256>(A, split_keys, blocks, stream); break;
    }
    if (rc != hipSuccess || A.chunks == 1) return rc;
    return launch_join(A, true, split_keys, stream);
}

}  // namespace gdn
