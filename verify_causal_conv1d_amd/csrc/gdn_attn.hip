// Attention of steps, verify windows and draft trees over the paged cache.
// Contract in include/libgdn.h (gdn_attn_window).
//
// For row t of a stream, query head h of kv head h / G (G = hq / hkv), and the
// visible keys j (the stream's kv_len cached rows, the row itself and its
// ancestors in the window):
//     s_j = scale q . k_j,   o = sum_j e^{s_j} v_j / sum_j e^{s_j},   out = o sigmoid(gate).
// Keys and values are read once for all rows and query heads of a kv head: the
// (row, head) pairs of a stream and kv head are the columns, 16 to a tile, of
// the matrix products S^T = K Q^T and O^T = V^T P^T.  One pass over the keys
// keeps the running maximum and sum of each column (base-2 exponentials).
//
// A stream's keys are cut into chunks at logical positions, by a rule on its
// own length alone, so that its results do not depend on the other streams of
// the call.  A chunk (of one kv head and up to 16 or 128 columns) is one
// workgroup.  A stream of one chunk ends there; otherwise m, l and O of every
// chunk go to the workspace and join_kernel merges them in chunk order:
//     m = max m_c,   l = sum l_c 2^{m_c - m},   o = sum O_c 2^{m_c - m} / l.
//
// Two kernels, by the columns that a window can have (max_rows * G):
//  - up to 16, attn_kernel: its four waves take tiles of 32 keys in turn, each
//    straight from memory into the registers that feed the matrix
//    instructions, and join through LDS (over 4-bit rows attn4_kernel, whose tiles
//    come by way of LDS);
//  - more, attn_wide_kernel: each wave has a column tile of its own, and K and
//    V pass through LDS once for all of them (over 4-bit rows the kernel of
//    prompts, with a window's masks).
// (16 streams of 700 to 8,191 keys, 24 query and 4 kv heads of 256: with 24
// columns the wide kernel takes 53 us and the other one, reading K and V once a
// tile, 69; with 48 columns 59 and 97.  One stream of 500 keys and 18 columns:
// 15.7 and 14.4.)
#include "gdn_attn_core.h"
#include "gdn_mxfp4.h"
#include "gdn_once.h"

namespace gdn {
namespace {

// ---- operands in registers ---------------------------------------------------

// 8 elements in bf16 of a lane's run of 16 (bf16: 32 bytes, e4m3: 16 bytes)
template <bool F8>
struct Run16;
template <>
struct Run16<false> {
    uint4 a, b;
    __device__ __forceinline__ void load_from_cache(const uint8_t *p)
    {
        a = load_once(p);
        b = load_once(p + 16);
    }
    __device__ __forceinline__ bf8v get(int h) const { return __builtin_bit_cast(bf8v, h ? b : a); }
};

__device__ __forceinline__ uint32_t cvt2(uint32_t codes, bool hi)
{
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, false));
}

template <>
struct Run16<true> {
    uint4 a;
    __device__ __forceinline__ void load_from_cache(const uint8_t *p) { a = load_once(p); }
    __device__ __forceinline__ bf8v get(int h) const
    {
        const uint32_t x = h ? a.z : a.x, y = h ? a.w : a.y;
        const uint4 v = {cvt2(x, false), cvt2(x, true), cvt2(y, false), cvt2(y, true)};
        return __builtin_bit_cast(bf8v, v);
    }
};

// A lane's share of one value row: NL loads of W dwords each.  Column i of
// load h is channel h * 16 * EPL + (lane % 16) * EPL + i.
template <int D, bool F8>
struct VLayout {
    static constexpr int BYTES = D * (F8 ? 1 : 2);
    static constexpr int NL = BYTES > 256 ? 2 : 1;
    static constexpr int W = BYTES / NL / 64;           // dwords of a load: 1, 2 or 4
    static constexpr int EPL = W * (F8 ? 4 : 2);
    static constexpr int NT = NL * EPL;                 // tiles of 16 channels of O^T
};

template <bool F8, int W>
struct VPart {
    typedef uint32_t vec_t __attribute__((ext_vector_type(W)));
    uint32_t w[W];
    __device__ __forceinline__ void set(vec_t x)
    {
        if constexpr (W == 1) {
            w[0] = __builtin_bit_cast(uint32_t, x);
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) w[i] = x[i];
        }
    }
    __device__ __forceinline__ void load(const uint8_t *p) { set(*reinterpret_cast<const vec_t *>(p)); }
    __device__ __forceinline__ void load_from_cache(const uint8_t *p)
    {
        set(__builtin_nontemporal_load(reinterpret_cast<const vec_t *>(p)));
    }
    // a dword's elements that are infinite or NaN, as a mask of their bits
    static __device__ __forceinline__ uint32_t bad(uint32_t x)
    {
        uint32_t m = 0;
        if constexpr (F8) {
#pragma unroll
            for (int b = 0; b < 32; b += 8)
                if ((x >> b & 0x7fu) == 0x7fu) m |= 0xffu << b;
        } else {
            if ((x & 0x7f80u) == 0x7f80u) m |= 0xffffu;
            if ((x & 0x7f800000u) == 0x7f800000u) m |= 0xffff0000u;
        }
        return m;
    }
    __device__ __forceinline__ bool finite() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) m |= bad(w[i]);
        return m == 0;
    }
    __device__ __forceinline__ void drop_bad()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] &= ~bad(w[i]);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
};

// The MFMA operand of column i of a load: that channel of the lane's 8 keys.
template <bool F8, int W>
__device__ __forceinline__ bf8v v_operand(const VPart<F8, W> (&v)[8], int i)
{
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (F8) {
            const uint32_t both = __builtin_amdgcn_perm(v[2 * q + 1].w[i / 4], v[2 * q].w[i / 4], i & 2 ? 0x07030602u : 0x05010400u);
            o[q] = cvt2(both, i & 1);
        } else {
            o[q] = __builtin_amdgcn_perm(v[2 * q + 1].w[i / 2], v[2 * q].w[i / 2], i & 1 ? 0x07060302u : 0x05040100u);
        }
    }
    const uint4 x = {o[0], o[1], o[2], o[3]};
    return __builtin_bit_cast(bf8v, x);
}

__device__ __forceinline__ f4v mfma(bf8v a, bf8v b, f4v c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// Adds the infinite and NaN values that the products of a chunk's keys [k0, k1)
// left out to a column's channels d .. d + 3: those of the rows that it sees (of
// the window, bits of seen) in the tiles that hold rows of the window.
template <int D, bool F8>
__device__ void add_bad(const AttnArgs &A, float4 &a, const int *rows16, uint32_t seen, int kv, int k0, int k1, int d)
{
    for (int key = max(k0, kv & -kTile); key < k1; ++key) {
        if (key >= kv && !(seen >> (key - kv) & 1)) continue;
        const size_t row = (size_t)rows16[(key - k0) >> 4] + (key & 15);
        float v[4];
        if constexpr (F8) {
            const uint32_t x = *reinterpret_cast<const uint32_t *>(A.kv.v + row * D + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (x >> (8 * i) & 0x7fu) == 0x7fu ? NAN : 0.0f;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(A.kv.v + (row * D + d) * 2);
            const float w[4] = {__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                                __uint_as_float(x.y & 0xffff0000u)};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (__float_as_uint(w[i]) & 0x7f800000u) == 0x7f800000u ? w[i] : 0.0f;
        }
        a.x += v[0], a.y += v[1], a.z += v[2], a.w += v[3];
    }
}

// The running state of a wave's column tile.  Lane (n, g) = (lane % 16, lane /
// 16) holds column n: of S^T the keys 16 u + 4 g + i of a tile of 32 (u < 2, i <
// 4), which are also the 8 keys it feeds into O^T's product, and of O^T rows 4 g
// + e of every tile: channels 16 i + 4 g + e where V is transposed by LDS reads,
// else VLayout's, with 4 g + e for lane % 16.
template <int D, bool F8>
struct Column {
    using V = VLayout<D, F8>;
    f4v o[V::NT];
    float mx, sum;
    float back;       // what O is to be multiplied by before a tile's values are added
    bool moved;       // and whether that is not 1 for any column

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < V::NT; ++i) o[i] = f4v{0, 0, 0, 0};
        mx = -INFINITY;
        sum = 0.0f;
    }

    // Weights of a tile's keys from its scores (before scale and k_scale): the
    // maximum and the sum brought up to date, P times v_scale in bf16, and with
    // SPLIT what that rounding leaves of it in rest, in bf16 again.  key0: the
    // lane's first key; seen: the window's rows that the column sees.  TAIL: the
    // tile holds keys of the window or past the end.
    template <bool TAIL, bool SPLIT>
    __device__ __forceinline__ bf8v weights(const f4v (&acc)[2], float scale, const float4 (&ks)[2], const float4 (&vs)[2], int key0,
                                            int kv, uint32_t seen, bf8v &rest)
    {
        float p[8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float k4[4] = {ks[u].x, ks[u].y, ks[u].z, ks[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) p[4 * u + i] = F8 ? acc[u][i] * (scale * k4[i]) : acc[u][i] * scale;
        }
        bool vis[8];
        if constexpr (TAIL)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = key0 + 16 * (i / 4) + (i & 3) - kv;   // place in the window
                vis[i] = (j < 0) | ((j < kMaxWindowRows) & (seen >> (j & 31)));
                p[i] = vis[i] ? p[i] : -INFINITY;
            }
        float tm = p[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) tm = fmaxf(tm, p[i]);
        // Any base within reach of the maximum does: it moves only when the maximum
        // has passed it, and then to 2^8 above that, so that O is rarely scaled again
        // (with the maximum itself, by every second tile of 16 columns).  Weights are
        // at most 1, so that no sum of weighted values overflows that would not with
        // the maximum as the base; P and the sums are floating point.
        tm = max_rows4(tm);
        tm = tm > mx ? tm + 8.0f : mx;
        const float base = tm == -INFINITY ? 0.0f : tm;     // no key seen so far: every p is 0
        back = __builtin_amdgcn_exp2f(mx - base);
        moved = __ballot(tm != mx && mx != -INFINITY);      // before the first key O is zero
        mx = tm;
        float ps = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(p[i] - base);
            ps += p[i];
        }
        sum = fmaf(sum, back, ps);
        if constexpr (F8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                p[4 * u] *= vs[u].x;
                p[4 * u + 1] *= vs[u].y;
                p[4 * u + 2] *= vs[u].z;
                p[4 * u + 3] *= vs[u].w;
            }
            if constexpr (TAIL)        // a masked row's scale may be anything
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = vis[i] ? p[i] : 0.0f;
        }
        // P goes into the product in bf16, rounded to nearest, while the sum keeps the
        // fp32 values: an error of up to 2^-8 of each term.  The rest of each weight
        // in a second product makes that 2^-15, at no cost where memory is the bound
        // (up to 16 columns: 16 steps 76.4 us, without it 76.5; one of 262,143 e4m3
        // keys 104.8 and 103.8).  The wide kernel, which is bound by its own
        // instructions, leaves it out: 16 trees would take 74.6 us instead of 70.4,
        // over e4m3 rows 82.4 instead of 75.8, for an error that is that of the bf16
        // result's own rounding.
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = __float_as_uint(p[2 * i]), hi = __float_as_uint(p[2 * i + 1]);
            w[i] = SPLIT && !F8 ? __builtin_amdgcn_perm(hi, lo, 0x07060302u) : pack2(p[2 * i], p[2 * i + 1]);
        }
        if constexpr (SPLIT) {
            // What is infinite has to stay so.  bf16 values times a rest of 0 or less do
            // not: the weight is cut there, not rounded (its rest is less than 2^-7 of
            // it), and where it is not 0 the rest is at least the least normal number.
            // e4m3 codes have no infinities, but their weights may be infinite with
            // their scale; their rest is that then, not NaN.
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float left = p[i] - __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
                p[i] = F8 ? fminf(left, fabsf(p[i])) : fmaxf(left, fminf(p[i], 0x1p-126f));
            }
            const uint4 x = {pack2(p[0], p[1]), pack2(p[2], p[3]), pack2(p[4], p[5]), pack2(p[6], p[7])};
            rest = __builtin_bit_cast(bf8v, x);
        }
        const uint4 pw = {w[0], w[1], w[2], w[3]};
        if constexpr (!F8) rescale();
        return __builtin_bit_cast(bf8v, pw);
    }

    // O brought up to date, after weights: by the caller for e4m3, once for tiles
    // with and without TAIL (16 trees of 16 e4m3 rows 75.7 us, in weights 80.4), in
    // weights for bf16 (70.1 us, by the caller 71.6)
    __device__ __forceinline__ void rescale()
    {
        if (moved) {
#pragma unroll
            for (int i = 0; i < V::NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= back;
        }
    }
};

// O^T += V^T P^T for the channels of load h, P as the sum of its two parts
template <int D, bool F8>
__device__ __forceinline__ void add_values(Column<D, F8> &C, int h, const VPart<F8, VLayout<D, F8>::W> (&v)[8], bf8v pb, bf8v rest)
{
    constexpr int EPL = VLayout<D, F8>::EPL;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const bf8v a = v_operand(v, i);
        C.o[h * EPL + i] = mfma(a, rest, mfma(a, pb, C.o[h * EPL + i]));
    }
}

// Values of a tile that holds keys of the window or past the end.  Rows past
// the end hold anything: zeros instead.  And 0 * inf is NaN: an infinite or NaN
// value of a window row must not reach the rows that do not see it, so such
// values are left out of the product (true is returned), to be added at the
// end to the results that they belong to (add_bad).
template <class VP>
__device__ __forceinline__ bool clean_values(VP (&v)[8], int key0, int len, int m)
{
    bool fin = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (key0 + 16 * (i / 4) + (i & 3) >= len) v[i].zero();
        fin = fin && v[i].finite();
    }
    if (m == 1 || !__ballot(!fin)) return false;      // every column of a one-row window sees all its keys
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i].drop_bad();
    return true;
}

// ---- up to 16 columns -----------------------------------------------------------

constexpr int kAttnThreads = 256, kAttnWaves = 4;

// Two workgroups a CU (registers and LDS), each wave with the next tile of keys
// and of values in flight: 32 KB a wave at d = 256 in bf16.  K needs no
// transposition (its rows are rows of the A operand); V's 8 x 8 blocks of a lane
// are turned by byte permutes as they are used.  Bounded by memory: 16 streams
// of 1,000 to 16,384 keys (374 MB) take 76 us with the join, 4.9 TB/s; one of
// 262,143 keys in e4m3 (545 MB) 105 us, 5.2 TB/s.  A short stream is bounded by
// the chain of layout, page numbers, first tile and join: 8 us for 100 keys.
template <int D, bool F8>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_kernel(const AttnArgs A)
{
    constexpr int ESZ = F8 ? 1 : 2, ROW = D * ESZ, KS = D / 64;
    using V = VLayout<D, F8>;
    constexpr int OP = D + 4;                      // padded LDS row of a column's channels
    extern __shared__ __align__(16) uint8_t smem[];
    float *o_lds = reinterpret_cast<float *>(smem);                    // [waves][kCols][OP]
    float *m_lds = o_lds + kAttnWaves * kCols * OP;                    // [waves][kCols]
    float *l_lds = m_lds + kAttnWaves * kCols;                         // [waves][kCols]
    uint4 *q_lds = reinterpret_cast<uint4 *>(l_lds + kAttnWaves * kCols);   // [KS][2][64]
    int *bad_lds = reinterpret_cast<int *>(q_lds + KS * 2 * 64);       // whether a window row's value is not finite
    uint32_t *seen_lds = reinterpret_cast<uint32_t *>(bad_lds + 4);    // [kCols]: the window's rows that a column sees
    int *rows16 = bad_lds + 4 + kCols;                                 // [size / 16]

    Pieces pieces;
    Chunk K;
    if (!pieces.find_in_block(A, false, kCols, 64 * blockIdx.y, blockIdx.x, K)) return;
    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, g = lane >> 4;
    const int col0 = K.rt * kCols, ncol = min(K.cols - col0, kCols);
    bool ok = chunk_rows(A, K, rows16, kAttnThreads);
    const uint32_t seen = seen_rows(A, K.r0, K.m, min(small_div(col0 + n, A.group), K.m - 1), ok);
    // the queries, in the order of the lanes' operands: [k-step][half][lane] of
    // 16 bytes (column n, channels 64 k + 16 g + 8 half; zero past the last column)
    for (int i = tid; i < KS * 2 * 64; i += kAttnThreads) {
        const int qc = i & 15, qg = i >> 4 & 3, hh = i >> 6 & 1, k = i >> 7;
        uint4 x = {0, 0, 0, 0};
        if (qc < ncol)
            x = *reinterpret_cast<const uint4 *>(A.q + ((size_t)col_row(A, K, col0 + qc) * A.hq + col_head(A, K, col0 + qc)) * D
                                                 + 64 * k + 16 * qg + 8 * hh);
        q_lds[i] = x;
    }
    static_assert(kAttnWaves == 4, "");
    if (lane == 0) l_lds[wave] = ok ? 1.0f : 0.0f;          // free until the waves join
    if (tid == 0) *bad_lds = 0;
    if (tid < kCols) seen_lds[tid] = seen;
    __syncthreads();
    if (l_lds[0] + l_lds[1] + l_lds[2] + l_lds[3] != 4.0f) {
        if (K.nch > 1 && tid < ncol) A.stat[col_part(A, K, col0 + tid)] = make_float2(0.0f, kSkipped);
        return;
    }

    Column<D, F8> C;
    C.clear();
    Run16<F8> kk[2][KS];
    VPart<F8, V::W> vv[V::NL][8];
    const uint32_t k_off = n * ROW + 16 * g * ESZ, v_off = 4 * g * ROW + n * V::W * 4;
    auto load_k = [&](int tile) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint8_t *p = A.kv.k + (size_t)__builtin_amdgcn_readfirstlane(rows16[2 * tile + u]) * ROW;
#pragma unroll
            for (int k = 0; k < KS; ++k) kk[u][k].load_from_cache(p + (k_off + 64 * k * ESZ));
        }
    };
    auto load_v = [&](int tile) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint8_t *p = A.kv.v + (size_t)__builtin_amdgcn_readfirstlane(rows16[2 * tile + u]) * ROW;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int hh = 0; hh < V::NL; ++hh) vv[hh][4 * u + j].load_from_cache(p + (v_off + j * ROW + hh * 16 * V::W * 4));
        }
    };
    const int tiles = ceil_div(K.k1 - K.k0, kTile);
    if (wave < tiles) {
        load_k(wave);
        load_v(wave);
    }
    for (int tile = wave; tile < tiles; tile += kAttnWaves) {
        const bool more = tile + kAttnWaves < tiles;
        const int key0 = K.k0 + tile * kTile + 4 * g;
        f4v acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const bf8v q = __builtin_bit_cast(bf8v, q_lds[(2 * k + hh) * 64 + lane]);
                acc[0] = mfma(kk[0][k].get(hh), q, acc[0]);
                acc[1] = mfma(kk[1][k].get(hh), q, acc[1]);
            }
        if (more) load_k(tile + kAttnWaves);
        float4 ks[2] = {}, vs[2] = {};
        if constexpr (F8)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const size_t row = __builtin_amdgcn_readfirstlane(rows16[2 * tile + u]);
                ks[u] = *reinterpret_cast<const float4 *>(A.kv.k_scale + row + 4 * g);
                vs[u] = *reinterpret_cast<const float4 *>(A.kv.v_scale + row + 4 * g);
            }
        bf8v pb, rest;
        if (K.k0 + tile * kTile + kTile <= K.kv) {
            pb = C.template weights<false, true>(acc, A.scale, ks, vs, key0, K.kv, seen, rest);
            if constexpr (F8) C.rescale();
#pragma unroll
            for (int hh = 0; hh < V::NL; ++hh) add_values(C, hh, vv[hh], pb, rest);
        } else {
            pb = C.template weights<true, true>(acc, A.scale, ks, vs, key0, K.kv, seen, rest);
            if constexpr (F8) C.rescale();
#pragma unroll
            for (int hh = 0; hh < V::NL; ++hh) {
                if (clean_values(vv[hh], key0, K.len, K.m) && lane == 0) *bad_lds = 1;
                add_values(C, hh, vv[hh], pb, rest);
            }
        }
        if (more) load_v(tile + kAttnWaves);
    }

    // join the waves: the column's maximum over them, each wave's O and l scaled to it
    const float sum = sum_rows4(C.sum);
    if (g == 0) m_lds[wave * kCols + n] = C.mx;
    __syncthreads();
    float top = m_lds[n];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, m_lds[w * kCols + n]);
    const float f = __builtin_amdgcn_exp2f(C.mx - (top == -INFINITY ? 0.0f : top));
    if (g == 0) l_lds[wave * kCols + n] = sum * f;
    if (n < ncol) {
        float *row = o_lds + (wave * kCols + n) * OP;
#pragma unroll
        for (int hh = 0; hh < V::NL; ++hh)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float *p = row + hh * 16 * V::EPL + (4 * g + e) * V::EPL;
                const f4v *o = C.o + hh * V::EPL;
#pragma unroll
                for (int i = 0; i < V::EPL; i += 4)
                    *reinterpret_cast<float4 *>(p + i) = make_float4(o[i][e] * f, o[i + 1][e] * f, o[i + 2][e] * f, o[i + 3][e] * f);
            }
    }
    __syncthreads();
    for (int i = tid; i < ncol * (D / 4); i += kAttnThreads) {
        const int cc = i / (D / 4), d = 4 * (i % (D / 4));
        float4 a = *reinterpret_cast<const float4 *>(o_lds + cc * OP + d);
        float l = l_lds[cc], mm = m_lds[cc];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) {
            const float4 b = *reinterpret_cast<const float4 *>(o_lds + (w * kCols + cc) * OP + d);
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
            l += l_lds[w * kCols + cc];
            mm = fmaxf(mm, m_lds[w * kCols + cc]);
        }
        if (*bad_lds) add_bad<D, F8>(A, a, rows16, seen_lds[cc], K.kv, K.k0, K.k1, d);
        put4<D>(A, K, col0 + cc, a, l, d);
        if (K.nch > 1 && d == 0) A.stat[col_part(A, K, col0 + cc)] = make_float2(mm, l);
    }
}

// ---- up to 16 columns, 4-bit rows ------------------------------------------------

// The same over 4-bit rows.  A tile of 32 keys is a quarter of the bytes, so a
// chunk ends after a few of them, and what counts is how soon they are all on their
// way: each wave keeps its next two tiles in flight, by direct loads into a ring of
// its own in LDS (16 bytes a lane, no registers, no barriers).  Codes
// are converted as they are used: K in blocks of 32 channels, whose exponent is the
// conversion's scale; of V a byte's two channels at once, then set beside the next
// key's.
//
// One stream of 262,143 keys (24 query and 4 kv heads of 256) takes 57 us, 5.0 TB/s:
// memory.  16 streams of 1,000 to 16,384 take 29 us where their bytes are 20: 1,116
// pieces of up to 256 keys on 512 places, each 5 us of loop and 6 of beginning and end
// (the queries through registers: 32).  Loads through registers, as in attn_kernel: 70 and 37.  Three
// workgroups a CU and a ring of one tile: 55 registers of a lane go to memory, 240 and 64.

// Direct loads into LDS, 16 bytes a lane, lane after lane from byte `to` on: of an
// address that is the wave's and an offset, or of the lane's own address.  The
// compiler is not told what they are: it would wait for all of a ring's loads before
// the first read, where the kernel waits itself (the counter that its own waits go
// by counts these loads, too, so that they come no earlier).  It is told that M0
// changes, and warns that M0 is not its to give away.  The wave's address may be
// what a v_readfirstlane has just written: five wait states before a memory
// instruction may read it, which the compiler does not count in front of an asm
// block, are s_mov_b32's and s_nop 3's (M0 needs one of them).
__device__ __forceinline__ uint32_t lds_at(const uint8_t *p) { return (uint32_t)(uintptr_t)(lds_void *)p; }
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds_once(const uint8_t *at, uint32_t off, uint32_t to)
{
    const uint64_t a = reinterpret_cast<uint64_t>(at);
    const uint64_t sa = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)a);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %0 nt" ::"s"(sa), "v"(off), "s"(to) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds_once(const uint8_t *at, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(at), "s"(to) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const void *at, uint32_t to)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(at), "s"(to) : "memory", "m0");
}
#pragma clang diagnostic pop

template <int D>
struct Tile4 {
    static constexpr int ROW = D / 2, EXPS = D / 32, CODES = 32 * ROW;       // bytes of a row, of its exponents, of the tile's keys
    static constexpr int BYTES = 2 * CODES + 64 * EXPS, LOADS = 2 * (CODES / 1024) + 1;     // a tile in LDS: K, V, exponents of both
    // 16-byte pieces of a row are exchanged, so that 16 rows lie in different banks
    static __device__ __forceinline__ int swizzle(int r) { return D == 256 ? r >> 1 & 7 : D == 128 ? r >> 2 & 3 : r >> 3 & 1; }
    static constexpr int VB = D / 32;                       // bytes of a lane's channels of a value row

    // row0, row1: cache rows of the tile's two groups of 16 keys
    static __device__ __forceinline__ void load(const KvArgs &kv, uint32_t to, size_t row0, size_t row1, int lane)
    {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint8_t *pool = x ? kv.v : kv.k;
#pragma unroll
            for (int i = 0; i < CODES / 1024; ++i) {
                const int b = i * 1024 + lane * 16, r = b / ROW, piece = b % ROW / 16 ^ swizzle(r), off = (r & 15) * ROW + piece * 16;
                if constexpr (CODES == 1024) {              // both groups in one load: the second from the first one's address
                    const int64_t apart = (int64_t)(row1 - row0) * ROW;
                    load_to_lds_once(pool + row0 * ROW + (r < 16 ? 0 : apart) + off, to + x * CODES);
                } else {
                    load_to_lds_once(pool + (i * 1024 / ROW < 16 ? row0 : row1) * ROW, off, to + x * CODES + i * 1024);
                }
            }
        }
        constexpr int LE = 2 * EXPS;                        // lanes that bring a pool's exponents
        if (lane < 2 * LE) {
            const int b = lane % LE * 16;
            load_to_lds((lane < LE ? kv.k_exp : kv.v_exp) + (b < 16 * EXPS ? row0 * EXPS + b : row1 * EXPS + (b - 16 * EXPS)), to + 2 * CODES);
        }
    }
    // steps of the product S^T = K Q^T: step s has 8 channels from channel(s, g) on
    static constexpr int STEPS = D / 32;
    static __device__ __forceinline__ int channel(int s, int g) { return D == 64 ? 16 * g + 8 * s : 128 * (s / 4) + 32 * g + 8 * (s & 3); }
};

// The keys of a lane's row, and its channels' values of 8 rows, as they lie in LDS
template <int D>
struct Keys4 {
    using S = Tile4<D>;
    static constexpr int W = D == 64 ? 2 : 4, N = D == 256 ? 2 : 1;
    uint32_t w[N][W];
    float f[N];
    __device__ __forceinline__ void read(const uint8_t *tile, int r, int g)
    {
        const uint8_t *p = tile + r * S::ROW, *x = tile + 2 * S::CODES + r * S::EXPS;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int piece = (D == 64 ? g >> 1 : 4 * j + g) ^ S::swizzle(r);
            if constexpr (D == 64) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p + piece * 16 + (g & 1) * 8);
                w[j][0] = v.x, w[j][1] = v.y;
            } else {
                const uint4 v = *reinterpret_cast<const uint4 *>(p + piece * 16);
                w[j][0] = v.x, w[j][1] = v.y, w[j][2] = v.z, w[j][3] = v.w;
            }
            f[j] = mx_scale(x[D == 64 ? g >> 1 : 4 * j + g]);
        }
    }
    __device__ __forceinline__ bf8v get(int s) const { return __builtin_bit_cast(bf8v, mx_values8(w[s / 4][s % W], f[s / 4])); }
};
template <int D>
struct Values4 {
    using S = Tile4<D>;
    static constexpr int W = D == 256 ? 2 : 1;
    uint32_t w[W], e;
    __device__ __forceinline__ void read(const uint8_t *tile, int r, int n)
    {
        const uint8_t *p = tile + S::CODES + r * S::ROW + (n * S::VB / 16 ^ S::swizzle(r)) * 16 + n * S::VB % 16;
        if constexpr (D == 256) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (D == 128) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(p);
        }
        e = tile[2 * S::CODES + 32 * S::EXPS + r * S::EXPS + n * S::VB / 16];
    }
    __device__ __forceinline__ bool finite() const { return e <= kMxMost; }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
        e = 127;
    }
    __device__ __forceinline__ void drop_bad()
    {
        if (!finite()) zero();
    }
};

// O^T += V^T P^T, P as the sum of its two parts: channel n * D / 16 + i is column i
template <int D>
__device__ __forceinline__ void add_values4(Column<D, false> &C, const Values4<D> (&v)[8], bf8v pb, bf8v rest)
{
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = mx_scale(v[j].e);
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
        uint32_t x[8], lo[4], hi[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = mx_pair(v[j].w[b / 4], f[j], b & 3);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            lo[q] = __builtin_amdgcn_perm(x[2 * q + 1], x[2 * q], 0x05040100u);
            hi[q] = __builtin_amdgcn_perm(x[2 * q + 1], x[2 * q], 0x07060302u);
        }
        const bf8v a = __builtin_bit_cast(bf8v, make_uint4(lo[0], lo[1], lo[2], lo[3])), c = __builtin_bit_cast(bf8v, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        C.o[2 * b] = mfma(a, rest, mfma(a, pb, C.o[2 * b]));
        C.o[2 * b + 1] = mfma(c, rest, mfma(c, pb, C.o[2 * b + 1]));
    }
}

constexpr int kWaves4 = 4, kThreads4 = 64 * kWaves4;

template <int D>
__global__ __launch_bounds__(kThreads4, 2) void attn4_kernel(const AttnArgs A)
{
    using S = Tile4<D>;
    using C4 = Column<D, false>;
    constexpr int OP = D + 4, EPL = D / 16;
    // each wave's next tiles; afterwards their O
    __shared__ __align__(1024) uint8_t ring0[kWaves4 * S::BYTES], ring1[kWaves4 * S::BYTES];
    __shared__ __align__(16) uint4 q_lds[S::STEPS * 64];
    __shared__ float m_lds[kWaves4 * kCols], l_lds[kWaves4 * kCols];
    __shared__ uint32_t seen_lds[kCols];
    __shared__ int ok_lds[kWaves4], bad_lds;
    static_assert(2 * kCols * OP * 4 <= sizeof(ring0), "");

    Pieces pieces;
    Chunk K;
    if (!pieces.find_in_block(A, false, kCols, 64 * blockIdx.y, blockIdx.x, K)) return;
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, n = lane & 15, g = lane >> 4;
    const int col0 = K.rt * kCols, ncol = min(K.cols - col0, kCols), tiles = ceil_div(K.k1 - K.k0, kTile);
    const int *table = A.table + (size_t)K.s * A.max_blocks;
    // cache row of a key's group of 16: past the stream's end that of its last keys,
    // and in place of a page outside the cache page 0's
    auto group_row = [&](int key) -> size_t {
        key = min(key, (K.len - 1) & ~15);
        const int id = table_entry(table, key >> A.kv.page_shift);
        return ((((uint32_t)id < (uint32_t)A.kv.n_pages ? id : 0) * A.kv.hkv + K.h) << A.kv.page_shift) + (key & ((1 << A.kv.page_shift) - 1));
    };
    const uint32_t q_at = __builtin_amdgcn_readfirstlane(lds_at(reinterpret_cast<const uint8_t *>(q_lds)));
    auto issue = [&](int tile, uint8_t *ring) {
        const int key = K.k0 + tile * kTile;
        S::load(A.kv, __builtin_amdgcn_readfirstlane(lds_at(ring)) + wave * S::BYTES, group_row(key), group_row(key + 16), lane);
    };
    // The queries, in the order of the lanes' operands (past the last column the last
    // one's), on their way while the chunk's pages are looked at
#pragma unroll
    for (int s = 0; s < S::STEPS; ++s) {
        if (s % kWaves4 != wave) continue;
        const int col = col0 + min(n, ncol - 1);
        load_to_lds(A.q + ((size_t)col_row(A, K, col) * A.hq + col_head(A, K, col)) * D + S::channel(s, g), q_at + s * 1024);
    }
    bool ok = true;
    for (int i = (K.k0 >> A.kv.page_shift) + tid; i <= (K.k1 - 1) >> A.kv.page_shift; i += kThreads4) {
        const int id = table[i];
        ok = ok && id >= 0 && id < A.kv.n_pages;
    }
    ok = !__ballot(!ok);
    const uint32_t seen = seen_rows(A, K.r0, K.m, min(small_div(col0 + n, A.group), K.m - 1), ok);
    if (lane == 0) ok_lds[wave] = ok;
    if (tid == 0) bad_lds = 0;
    if (tid < kCols) seen_lds[tid] = seen;
    // (the queries have come: the waits for what came before end here)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);
    asm volatile("" ::: "memory");
    if (wave < tiles) issue(wave, ring0);
    if (wave + kWaves4 < tiles) issue(wave + kWaves4, ring1);
    lds_barrier();

    C4 C;
    C.clear();
    auto step = [&](int tile, uint8_t *ring) {
        // this tile is there when no more than the next one's loads are left
        asm volatile("" ::: "memory");
        if (tile + kWaves4 < tiles) __builtin_amdgcn_s_waitcnt(0x0F70 | (S::LOADS & 15) | (S::LOADS >> 4) << 14);
        else __builtin_amdgcn_s_waitcnt(0x0F70);
        asm volatile("" ::: "memory");
        const uint8_t *at = ring + wave * S::BYTES;
        const int key0 = K.k0 + tile * kTile + 4 * g;
        f4v acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
        Keys4<D> kk[2];
        kk[0].read(at, n, g);
        kk[1].read(at, 16 + n, g);
        Values4<D> v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i].read(at, 4 * g + (i & 3) + 16 * (i / 4), n);
#pragma unroll
        for (int s = 0; s < S::STEPS; ++s) {
            const bf8v q = __builtin_bit_cast(bf8v, q_lds[s * 64 + lane]);
            acc[0] = mfma(kk[0].get(s), q, acc[0]);
            acc[1] = mfma(kk[1].get(s), q, acc[1]);
        }
        const float4 none[2] = {};
        bf8v pb, rest;
        if (K.k0 + tile * kTile + kTile <= K.kv) {
            pb = C.template weights<false, true>(acc, A.scale, none, none, key0, K.kv, seen, rest);
        } else {
            pb = C.template weights<true, true>(acc, A.scale, none, none, key0, K.kv, seen, rest);
            if (clean_values(v, key0, K.len, K.m) && lane == 0) bad_lds = 1;
        }
        // the tile's LDS has been read: the ring takes the tile after the next
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0xC07F);
        asm volatile("" ::: "memory");
        if (tile + 2 * kWaves4 < tiles) issue(tile + 2 * kWaves4, ring);
        add_values4(C, v, pb, rest);
    };
    for (int tile = wave; tile < tiles; tile += 2 * kWaves4) {
        step(tile, ring0);
        if (tile + kWaves4 < tiles) step(tile + kWaves4, ring1);
    }

    // join the waves: the column's maximum over them, each wave's O and l scaled to it
    const float sum = sum_rows4(C.sum);
    if (g == 0) m_lds[wave * kCols + n] = C.mx;
    lds_barrier();
    ok = ok_lds[0] && ok_lds[1] && ok_lds[2] && ok_lds[3];
    static_assert(kWaves4 == 4, "");
    if (!ok) {
        if (K.nch > 1 && tid < ncol) A.stat[col_part(A, K, col0 + tid)] = make_float2(0.0f, kSkipped);
        return;
    }
    auto o_at = [&](int w, int c) { return reinterpret_cast<float *>(w < 2 ? ring0 : ring1) + ((w & 1) * kCols + c) * OP; };
    float top = m_lds[n];
#pragma unroll
    for (int w = 1; w < kWaves4; ++w) top = fmaxf(top, m_lds[w * kCols + n]);
    const float f = __builtin_amdgcn_exp2f(C.mx - (top == -INFINITY ? 0.0f : top));
    if (g == 0) l_lds[wave * kCols + n] = sum * f;
    if (n < ncol) {
        float *row = o_at(wave, n);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float *p = row + (4 * g + e) * EPL;
#pragma unroll
            for (int i = 0; i < EPL; i += 4)
                *reinterpret_cast<float4 *>(p + i) = make_float4(C.o[i][e] * f, C.o[i + 1][e] * f, C.o[i + 2][e] * f, C.o[i + 3][e] * f);
        }
    }
    lds_barrier();
    for (int i = tid; i < ncol * (D / 4); i += kThreads4) {
        const int cc = i / (D / 4), d = 4 * (i % (D / 4));
        float4 a = *reinterpret_cast<const float4 *>(o_at(0, cc) + d);
        float l = l_lds[cc], mm = m_lds[cc];
#pragma unroll
        for (int w = 1; w < kWaves4; ++w) {
            const float4 b = *reinterpret_cast<const float4 *>(o_at(w, cc) + d);
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
            l += l_lds[w * kCols + cc];
            mm = fmaxf(mm, m_lds[w * kCols + cc]);
        }
        if (bad_lds)            // blocks of NaN that the products left out, to the columns that see them
            for (int key = max(K.k0, K.kv & -kTile); key < K.k1; ++key) {
                if (key >= K.kv && !(seen_lds[cc] >> (key - K.kv) & 1)) continue;
                const size_t row = (((size_t)table[key >> A.kv.page_shift] * A.kv.hkv + K.h) << A.kv.page_shift) + (key & ((1 << A.kv.page_shift) - 1));
                if (A.kv.v_exp[row * (D / kMxBlock) + d / kMxBlock] > kMxMost) a = make_float4(NAN, NAN, NAN, NAN);
            }
        put4<D>(A, K, col0 + cc, a, l, d);
        if (K.nch > 1 && d == 0) A.stat[col_part(A, K, col0 + cc)] = make_float2(mm, l);
    }
}

// ---- more columns ----------------------------------------------------------------

// Four stages of keys and values in LDS, filled by direct loads (16 bytes a
// lane, 1 KB an instruction): while a stage is multiplied the next three are
// in flight, up to 96 KB a CU, and one barrier a stage separates its readers
// from the loads that fill it again.  K rows are stored with their 16-byte
// pieces exchanged by a function of the row (piece ^ swizzle), so that the 16
// rows of an operand lie in different banks.
//
// One workgroup of 8 waves stays on each CU and goes through its pieces.  16
// draft trees of up to 16 rows over 700 to 8,191 keys (96 columns, 212 MB): 66 us
// with the join (7.5 us).  A tile of 32 keys
// takes a CU about 1.2 us when nothing else runs there (each wave reads the
// tile's 32 KB from LDS, and two of the waves with columns share a SIMD); how
// evenly the pieces fall on the CUs costs the rest.  Over e4m3 rows (110 MB) they
// take 76 us: a wave's chain from the keys through the weights to the values, with
// every code converted on the way, and at most two waves a SIMD to hide it.
template <int D, bool F8>
struct Stage {
    static constexpr int ROW = D * (F8 ? 1 : 2);
    static constexpr int KEYS = ROW == 512 ? 32 : 64;
    static constexpr int BYTES = 2 * KEYS * ROW;
    static constexpr int PIECES = ROW / 16;             // 16-byte pieces of a row
    static constexpr int ROWS = 1024 / ROW;             // rows of one load instruction
    static constexpr int SCALES = F8 ? 2 * KEYS * 4 : 16;
    static __device__ __forceinline__ int swizzle(int key)
    {
        return ROW >= 256 ? key & 15 : ROW == 128 ? key >> 1 & 7 : key >> 2 & 3;
    }
    // V rows likewise, the 16 channels of a tile (32 bytes in bf16) together: the
    // transposing reads take 8 rows at once
    static __device__ __forceinline__ int v_swizzle(int key)
    {
        if (F8) return ROW == 256 ? key & 7 : ROW == 128 ? key >> 1 & 7 : key >> 2 & 3;
        return 2 * (ROW >= 256 ? key & 7 : key >> 1 & 3);
    }
};

// clean_values of one operand in e4m3 codes (byte j: key key0 + 16 (j / 4) + j %
// 4) or in bf16 (element j likewise);
// under the mask `drop`, values that are not finite are left out, and true is
// returned.
__device__ __forceinline__ bool clean_operand(v2i &v, int key0, int len, uint32_t drop)
{
    uint32_t bad = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int left = len - key0 - 16 * u;               // keys of the stream among the four
        const uint32_t x = v[u] & (left >= 4 ? 0xffffffffu : left > 0 ? (1u << 8 * left) - 1 : 0u), b = VPart<true, 1>::bad(x) & drop;
        v[u] = x & ~b;
        bad |= b;
    }
    return bad != 0;
}
__device__ __forceinline__ bool clean_operand(bf8v &v, int key0, int len, uint32_t drop)
{
    uint4 x = __builtin_bit_cast(uint4, v);
    uint32_t w[4] = {x.x, x.y, x.z, x.w}, bad = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int key = key0 + 16 * (q / 2) + 2 * (q & 1);
        w[q] &= key + 1 < len ? 0xffffffffu : key < len ? 0xffffu : 0u;
        const uint32_t b = VPart<false, 1>::bad(w[q]) & drop;
        w[q] &= ~b;
        bad |= b;
    }
    v = __builtin_bit_cast(bf8v, make_uint4(w[0], w[1], w[2], w[3]));
    return bad != 0;
}

constexpr int kWideWaves = 8, kWideThreads = 64 * kWideWaves, kWideTiles = 1;
constexpr int kWideCols = kCols * kWideTiles * kWideWaves;

template <int D, bool F8>
__global__ __launch_bounds__(kWideThreads, 2) void attn_wide_kernel(const AttnArgs A, const int list_size)
{
    using S = Stage<D, F8>;
    using V = VLayout<D, F8>;
    constexpr int ROW = S::ROW, KS = D / 64, T = kWideTiles;
    constexpr int NK = S::KEYS * ROW / 1024;            // load instructions of a stage's keys, and of its values
    constexpr int PER = 2 * NK / kWideWaves;            // of a wave
    constexpr int ALL = PER + (F8 ? 1 : 0);             // with the scales
    static_assert(2 * NK % kWideWaves == 0 && 3 * ALL < 64, "");
    // separate arrays, so that loads into one are known not to touch the others
    __shared__ __align__(1024) uint8_t st0[S::BYTES], st1[S::BYTES], st2[S::BYTES], st3[S::BYTES];
    __shared__ __align__(16) uint8_t sc0[S::SCALES], sc1[S::SCALES], sc2[S::SCALES], sc3[S::SCALES];
    __shared__ int wave_ok[2][kWideWaves];
    extern __shared__ __align__(16) uint8_t smem[];
    int *rows16 = reinterpret_cast<int *>(smem);        // [2][list_size]

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Pieces pieces;
    Chunk K, N;                 // the piece at work and the next one
    int item = blockIdx.x, at = 0;
    if (!pieces.find(A, true, kWideCols, item, K)) return;
    // A piece's list of cache rows is made while the piece before it is at work,
    // and the loads of its first tiles are under way before that one ends.
    int list = 0, next_list = list_size;
    {
        const bool ok = chunk_rows(A, K, rows16 + list, kWideThreads);
        if (threadIdx.x % 64 == 0) wave_ok[at][wave] = ok;
    }
    lds_barrier();

    int tiles = ceil_div(K.k1 - K.k0, S::KEYS);
    // A stage's loads: a wave's instructions bring the same rows of PER / 2 of the
    // stage's groups of 16 (their keys, then their values; rows of 64 bytes: the
    // keys of one group or the values).  The cache rows of the groups are read
    // from the list a stage ahead.
    constexpr int GROUPS = (PER + 1) / 2;
    static_assert(kWideWaves == 8, "");
    int ahead[GROUPS], ahead_scale = 0;
    // the tile after the last one again, where there is none
    auto look = [&](int rows, int tile, int count) {
        const int lane = fresh(threadIdx.x) & 63;
        rows += min(tile, max(count - 1, 0)) * (S::KEYS / 16);
#pragma unroll
        for (int x = 0; x < GROUPS; ++x) ahead[x] = rows16[rows + (x * kWideWaves + wave) % NK * S::ROWS / 16];
        if constexpr (F8) ahead_scale = rows16[rows + lane / 16] + (lane & 15);
    };
    auto fill = [&](uint8_t *stage, uint8_t *scales) {
        const int lane = fresh(threadIdx.x) & 63;
        const int in = wave * S::ROWS % 16 + lane / S::PIECES;             // row in its group
        const uint32_t v_off = in * ROW + (lane % S::PIECES ^ S::v_swizzle(in)) * 16, k_off = in * ROW + (lane % S::PIECES ^ S::swizzle(in)) * 16;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const bool is_k = PER == 1 ? wave < NK : j < PER / 2;
            const int x = PER == 1 ? 0 : j % (PER / 2);
            const uint8_t *p = (is_k ? A.kv.k : A.kv.v) + (size_t)__builtin_amdgcn_readfirstlane(ahead[x]) * ROW;
            __builtin_amdgcn_global_load_lds((global_void *)(p + (is_k ? k_off : v_off)),
                                             (lds_void *)(stage + (j * kWideWaves + wave) * 1024), 16, 0, kOnce);
        }
        if constexpr (F8) {        // even waves the keys' scales, odd ones the values'
            const float *p = (wave & 1 ? A.kv.v_scale : A.kv.k_scale) + (size_t)ahead_scale;
            __builtin_amdgcn_global_load_lds((global_void *)p, (lds_void *)(scales + (wave & 1) * S::KEYS * 4), 4, 0, 0);
        }
    };

    Column<D, F8> C[T];
    uint32_t seen[T];
    bf8v q[T][KS][2];
    int col0 = 0;
    bool busy = false, bad = false;
    auto multiply = [&](int tile, const uint8_t *stage, const uint8_t *scales) {
        const int lane = fresh(threadIdx.x) & 63, n = lane & 15, g = lane >> 4;
        // e4m3: a loop, since in two copies the compiler moves all of O between
        // registers (16 trees 75.8 us, unrolled 77.5); bf16 rows of 128: 69, unrolled 67.4
        constexpr int COPIES = F8 ? 1 : 2;
#pragma unroll COPIES
        for (int sub = 0; sub < S::KEYS / kTile; ++sub) {
            const int first = K.k0 + tile * S::KEYS + sub * kTile;
            if (sub > 0 && first >= K.k1) break;
            const int key0 = first + 4 * g;
            // all reads of the keys first (the products wait for the last of them),
            // then the products, and under them the reads of the first values, to be
            // there when the weights are; over e4m3 rows the weights wait for the
            // scales, and so for the values, whose reads are asked for beside them
            Run16<F8> kk[2][KS];
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int row = (sub * kTile + 16 * u + n) * ROW, sw = S::swizzle(n);
                    if constexpr (F8) {
                        kk[u][k].a = *reinterpret_cast<const uint4 *>(stage + (row + (((4 * k + g) ^ sw) * 16)));
                    } else {
                        kk[u][k].a = *reinterpret_cast<const uint4 *>(stage + (row + (((8 * (k & 1) + 2 * g) ^ sw) + 16 * (k >> 1)) * 16));
                        kk[u][k].b = *reinterpret_cast<const uint4 *>(stage + (row + (((8 * (k & 1) + 2 * g + 1) ^ sw) + 16 * (k >> 1)) * 16));
                    }
                }
            __builtin_amdgcn_sched_barrier(0);
            f4v acc[T][2];
#pragma unroll
            for (int c = 0; c < T; ++c) acc[c][0] = acc[c][1] = f4v{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int c = 0; c < T; ++c) acc[c][u] = mfma(kk[u][k].get(hh), q[c][k][hh], acc[c][u]);
            float4 ks[2] = {}, vs[2] = {};
            if constexpr (F8)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    ks[u] = *reinterpret_cast<const float4 *>(scales + ((sub * kTile + 16 * u + 4 * g) * 4));
                    vs[u] = *reinterpret_cast<const float4 *>(scales + ((S::KEYS + sub * kTile + 16 * u + 4 * g) * 4));
                }
            const bool tail = first + kTile > K.kv;
            bf8v pb[T];
            auto get_weights = [&] {
#pragma unroll
                for (int c = 0; c < T; ++c) {
                    bf8v none;
                    pb[c] = tail ? C[c].template weights<true, false>(acc[c], A.scale, ks, vs, key0, K.kv, seen[c], none)
                                 : C[c].template weights<false, false>(acc[c], A.scale, ks, vs, key0, K.kv, seen[c], none);
                }
                if constexpr (F8)
#pragma unroll
                    for (int c = 0; c < T; ++c) C[c].rescale();
            };
            if constexpr (F8) {
                // the codes of channels 16 i .. 16 i + 15, transposed by the read: this
                // lane brings 8 channels of the (n / 2)th of its 8 keys
                const int vr = 16 * (n >> 3) + 4 * g + (n >> 1 & 3);
                const int base = (S::KEYS + sub * kTile + vr) * ROW + S::v_swizzle(vr & 15) * 16 + (n & 1) * 8;
                v2i v[V::NT];
#pragma unroll
                for (int i = 0; i < V::NT; ++i) v[i] = read_transposed_codes(stage + ((base ^ (i & 7) * 16) + (i & ~7) * 16));
                __builtin_amdgcn_sched_barrier(0);
                get_weights();
                if (tail) {
                    bool any = false;
#pragma unroll
                    for (int i = 0; i < V::NT; ++i) any |= clean_operand(v[i], key0, K.len, K.m > 1 ? ~0u : 0u);
                    bad |= __ballot(any) != 0;
                }
#pragma unroll
                for (int i = 0; i < V::NT; ++i) {
                    const uint4 x = {cvt2(v[i][0], false), cvt2(v[i][0], true), cvt2(v[i][1], false), cvt2(v[i][1], true)};
#pragma unroll
                    for (int c = 0; c < T; ++c) C[c].o[i] = mfma(__builtin_bit_cast(bf8v, x), pb[c], C[c].o[i]);
                }
            } else {
                // the operand of channels 16 i .. 16 i + 15, transposed by the read:
                // row 4 g + n / 4 (and 16 on), channels 4 (n % 4) ..
                const int vr = 4 * g + (n >> 2);
                const int base = (S::KEYS + sub * kTile + vr) * ROW + S::v_swizzle(vr) * 16 + (n & 3) * 8;
                constexpr int HALF = V::NT / 2;
                bf8v v[V::NT];
                auto load_v = [&](int from) {
#pragma unroll
                    for (int i = from; i < from + HALF; ++i) {
                        const int at = (base ^ (i & 7) * 32) + (i & ~7) * 32;
                        const s4v lo = read_transposed(stage + at), hi = read_transposed(stage + (at + 16 * ROW));
                        v[i] = __builtin_bit_cast(bf8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
                    }
                };
                load_v(0);
                __builtin_amdgcn_sched_barrier(0);
                get_weights();
                load_v(HALF);
                if (tail) {
                    bool any = false;
#pragma unroll
                    for (int i = 0; i < V::NT; ++i) any |= clean_operand(v[i], key0, K.len, K.m > 1 ? ~0u : 0u);
                    bad |= __ballot(any) != 0;
                }
#pragma unroll
                for (int i = 0; i < V::NT; ++i)
#pragma unroll
                    for (int c = 0; c < T; ++c) C[c].o[i] = mfma(v[i], pb[c], C[c].o[i]);
            }
        }
    };
    look(list, 0, tiles);
    fill(st0, sc0);
    look(list, 1, tiles);
    fill(st1, sc1);
    look(list, 2, tiles);
    fill(st2, sc2);
    look(list, 3, tiles);
    while (true) {
        const int lane = fresh(threadIdx.x) & 63, n = lane & 15, g = lane >> 4;
        item += gridDim.x;
        const bool more = pieces.find(A, true, kWideCols, item, N);
        // with no next piece (no tiles) the list of this one still names real rows
        const int after = more ? next_list + 0 : list + 0;
        const int next_tiles = more ? ceil_div(N.k1 - N.k0, S::KEYS) : 0;
        if (more) {
            const bool ok = chunk_rows(A, N, rows16 + next_list, kWideThreads);
            if (lane == 0) wave_ok[at ^ 1][wave] = ok;
        }
        col0 = K.rt * kWideCols + wave * kCols * T;         // the wave's first column
        busy = col0 < K.cols;                               // waves without columns only load
        bool ok = true;
#pragma unroll
        for (int c = 0; c < T; ++c) {
            const int col = min(col0 + c * kCols + n, K.cols - 1);      // past the last one: that one again, not stored
            seen[c] = seen_rows(A, K.r0, K.m, small_div(col, A.group), ok);
            const uint16_t *p = A.q + ((size_t)col_row(A, K, col) * A.hq + col_head(A, K, col)) * D + 16 * g;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) q[c][k][hh] = *reinterpret_cast<const bf8v *>(p + 64 * k + 8 * hh);
            C[c].clear();
        }
        bad = false;
        // Steps in fours, so that a piece begins with the first stage.  A tile's
        // loads are done once at most those of the two tiles after it are left;
        // the stage of the tile before it is free when all waves are here.
        const int steps = (tiles + 3) & ~3;
        auto step = [&](int tile, uint8_t *stage, uint8_t *scales, uint8_t *next, uint8_t *next_scales) {
            wait_and_meet<2 * ALL>();
            fill(next, next_scales);                        // tile + 3
            const int f = tile + 4;
            const bool now = f < steps;
            look(now ? list : after, now ? f : f - steps, now ? tiles : next_tiles);
            if (busy && tile < tiles) multiply(tile, stage, scales);
        };
        for (int tile = 0; tile < steps; tile += 4) {
            step(tile, st0, sc0, st3, sc3);
            step(tile + 1, st1, sc1, st0, sc0);
            step(tile + 2, st2, sc2, st1, sc1);
            step(tile + 3, st3, sc3, st2, sc2);
        }

#pragma unroll
        for (int w = 0; w < kWideWaves; ++w) ok = ok && wave_ok[at][w];
        const int end_lane = fresh(threadIdx.x) & 63, en = end_lane & 15, eg = end_lane >> 4;
#pragma unroll
        for (int c = 0; c < T; ++c) {
            const float l = sum_rows4(C[c].sum);
            const int col = col0 + c * kCols + en;
            if (col >= K.cols) continue;
            if (K.nch > 1 && eg == 0) A.stat[col_part(A, K, col)] = ok ? make_float2(C[c].mx, l) : make_float2(0.0f, kSkipped);
            if (!ok) continue;
            auto put = [&](float4 a, int d) {
                if (bad) add_bad<D, F8>(A, a, rows16 + list, seen[c], K.kv, K.k0, K.k1, d);
                put4<D>(A, K, col, a, l, d);
            };
#pragma unroll
            for (int i = 0; i < V::NT; ++i) {
                const f4v o = C[c].o[i];
                put(make_float4(o[0], o[1], o[2], o[3]), 16 * i + 4 * eg);
            }
        }
        if (!more) break;
        lds_barrier();            // the list of this piece is made anew
        K = N;
        tiles = next_tiles;
        at ^= 1;
        list = next_list;
        next_list = list_size - list;
    }
    wait_vmem();      // no load may reach LDS that is no longer this workgroup's
}

// Merges a (row, head)'s chunks, one wave each, D / 64 channels a lane.  Where all
// parts are few bytes, what it reads does not wait for the stream to be found: the
// first parts, the sums and the gates are asked for at once, by the row alone (a
// stream has at most A.chunks chunks; what lies past its own is not used), and the
// streams' windows are looked at 64 at a time.  Of many bytes, whose time it is
// that the kernel takes, only those that are there: of the 16 trees above the longest
// has 17 chunks and ten have 4 to 6, and asked for by the row alone they were 58 MB and
// 12.2 us, where the 25 MB that the chunks wrote take 7.6.  Where every stream has as
// many as are asked for, waiting saves nothing: 64 steps of 16,384 and of 8,192 keys
// 10.9 and 11.2 us (10.2 and 9.9 at once), of calls of 740 and 440; 16 trees of 8,191
// 17.9 and 17.0.
constexpr int kJoinWaves = 4, kJoinBatch = 16;      // loads in flight
constexpr long long kJoinAtOnce = 16 << 20;        // bytes

template <int D, bool PROMPT>
__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(const AttnArgs A, const int is_wide, const int split_keys)
{
    constexpr int VEC = D / 64;
    typedef float part_t __attribute__((ext_vector_type(VEC)));
    typedef uint16_t half_t __attribute__((ext_vector_type(VEC)));
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int item = blockIdx.x * kJoinWaves + wave;
    if (item >= A.total_rows * A.hq) return;
    const int r = item / A.hq, head = item - r * A.hq;
    const size_t at = (size_t)item * A.chunks;
    const part_t *parts = reinterpret_cast<const part_t *>(A.part + at * D) + lane;
    part_t b[kJoinBatch] = {};
    const bool at_once = (long long)A.total_rows * A.hq * at_most(A.chunks, kJoinBatch) * (D * 4) <= kJoinAtOnce;
    if (at_once)
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i)
            if (i < A.chunks) b[i] = parts[(size_t)i * 64];
    static_assert(kMaxChunks == 64, "");
    float2 st = {-INFINITY, 0.0f};
    if (lane < A.chunks) st = A.stat[at + lane];
    half_t gate = {};
    if (A.gate) gate = *reinterpret_cast<const half_t *>(A.gate + r * A.gate_row + head * A.gate_head + VEC * lane);

    int block = 0;
    if (A.n_streams > 64) {                     // the last block that starts at or before r
        int hi = (A.n_streams - 1) / 64;
        while (block < hi) {
            const int mid = (block + hi + 1) >> 1;
            if (A.row_start[64 * mid] <= r) block = mid;
            else hi = mid - 1;
        }
    }
    int r0 = 0, m = 0, kv = 0;
    auto holder = [&](int b) {
        const int s = 64 * b + lane;
        return __ballot(s < A.n_streams && stream_window(A, s, r0, m, kv) && r >= r0 && r < r0 + m);
    };
    uint64_t found = holder(block);
    // not where it should be: a row of no stream, past the last one in the last
    // block, or an entry of row_start is broken and leads elsewhere
    if (!found && A.n_streams > 64) {
        const int s = 64 * block + lane;
        const bool past = block == (A.n_streams - 1) / 64 && r >= A.row_start[A.n_streams]
                          && !__ballot(s < A.n_streams && A.row_start[s + 1] < A.row_start[s]);
        if (!past)
            for (block = 0; !found && 64 * block < A.n_streams; ++block) found = holder(block);
    }
    if (!found) return;
    const int l = __builtin_ctzll(found);
    const int len = __builtin_amdgcn_readlane(kv, l) + __builtin_amdgcn_readlane(m, l);
    int nch;
    if constexpr (PROMPT) {         // of the stream; then those that the row sees
        if (len <= split_keys) return;
        nch = (__builtin_amdgcn_readlane(kv, l) + r - __builtin_amdgcn_readlane(r0, l)) / split_keys + 1;
    } else {
        nch = chunk_count(len, is_wide);
        if (nch <= 1) return;
    }
    if (lane >= nch) st = {-INFINITY, 0.0f};
    if (__ballot(st.y < 0.0f)) return;                      // a chunk was skipped: so is the stream
    float top = st.x;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    top = max_rows4(top);
    const float f = __builtin_amdgcn_exp2f(st.x - (top == -INFINITY ? 0.0f : top));
    const float inv = 1.0f / sum_wave(st.y * f);
    part_t a = {};
    for (int c = 0; c < nch; c += kJoinBatch) {
        if (c > 0 || !at_once)
#pragma unroll
            for (int i = 0; i < kJoinBatch; ++i)
                if (c + i < nch) b[i] = parts[(size_t)(c + i) * 64];
#pragma unroll
        for (int i = 0; i < kJoinBatch; ++i)
            if (c + i < nch) {
                const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), c + i));
#pragma unroll
                for (int e = 0; e < VEC; ++e) a[e] = fmaf(b[i][e], w, a[e]);
            }
    }
    half_t o;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = f2bf(A.gate ? a[e] * inv * sigmoid_f(bf16f(gate[e])) : a[e] * inv);
    *reinterpret_cast<half_t *>(A.out + ((size_t)item * D + VEC * lane)) = o;
}

// Keys of the longest chunk that a stream of up to max_kv keys can have: the
// rule's longest, and what rounding adds.
int longest_chunk(int max_kv, bool wide)
{
    const int most = chunk_most(max_kv, wide);
    return most + most / 16 + chunk_unit(wide);
}

constexpr int kCUs = 256;

template <int D, int FMT>
hipError_t launch_d(const AttnArgs &A, bool wide, long long pieces, hipStream_t stream)
{
    const int list = longest_chunk(A.max_kv, wide) / 16;
    const size_t list_bytes = sizeof(int) * list;
    if (!wide) {
        constexpr size_t lds = sizeof(float) * kAttnWaves * kCols * (D + 4 + 2) + D * 2 * kCols + sizeof(int) * (4 + kCols);
        // 64 streams a grid row
        const unsigned per_row = (unsigned)(pieces / A.n_streams * (A.n_streams < 64 ? A.n_streams : 64));
        const dim3 grid(per_row, ceil_div(A.n_streams, 64));
        if constexpr (FMT == FMT_MXFP4) attn4_kernel<D><<<grid, kThreads4, 0, stream>>>(A);
        else hipLaunchKernelGGL((attn_kernel<D, FMT == FMT_E4M3>), grid, dim3(kAttnThreads), lds + list_bytes, stream, A);
    } else if constexpr (FMT == FMT_MXFP4) {
        const hipError_t rc = launch_wide4(A, pieces, stream);
        if (rc != hipSuccess) return rc;
    } else {
        const unsigned blocks = (unsigned)(pieces < kCUs ? pieces : kCUs);
        hipLaunchKernelGGL((attn_wide_kernel<D, FMT == FMT_E4M3>), dim3(blocks), dim3(kWideThreads), 2 * list_bytes, stream, A, list);
    }
    if (A.chunks > 1) return launch_join(A, wide, 0, stream);
    return hipGetLastError();
}

template <int D>
hipError_t launch_fmt(const AttnArgs &A, bool wide, long long pieces, hipStream_t stream)
{
    switch (format_of(A.kv)) {
    case FMT_BF16: return launch_d<D, FMT_BF16>(A, wide, pieces, stream);
    case FMT_E4M3: return launch_d<D, FMT_E4M3>(A, wide, pieces, stream);
    default: return launch_d<D, FMT_MXFP4>(A, wide, pieces, stream);
    }
}

int column_tiles(int max_rows, int group)
{
    return is_wide(max_rows, group) ? ceil_div(max_rows * group, kWideCols) : 1;
}

}  // namespace

hipError_t launch_join(const AttnArgs &A, bool wide, int split_keys, hipStream_t stream)
{
    const dim3 grid(ceil_div(A.total_rows * A.hq, kJoinWaves)), block(64 * kJoinWaves);
    const int w = wide ? 1 : 0;
    switch (A.kv.d) {
    case 64:
        if (split_keys) join_kernel<64, true><<<grid, block, 0, stream>>>(A, w, split_keys);
        else join_kernel<64, false><<<grid, block, 0, stream>>>(A, w, 0);
        break;
    case 128:
        if (split_keys) join_kernel<128, true><<<grid, block, 0, stream>>>(A, w, split_keys);
        else join_kernel<128, false><<<grid, block, 0, stream>>>(A, w, 0);
        break;
    default:
        if (split_keys) join_kernel<256, true><<<grid, block, 0, stream>>>(A, w, split_keys);
        else join_kernel<256, false><<<grid, block, 0, stream>>>(A, w, 0);
        break;
    }
    return hipGetLastError();
}

size_t attn_workspace_bytes(int hq, int hkv, int d, int total_rows, int max_rows, int max_kv)
{
    const size_t chunks = chunk_bound(max_kv, is_wide(max_rows, hq / hkv));
    if (chunks <= 1) return 0;
    return (size_t)total_rows * hq * chunks * (sizeof(float) * d + sizeof(float2));
}

// at most so many pieces, or -1 if they cannot be numbered
static long long most_pieces(const AttnArgs &A, bool wide)
{
    const long long per = (long long)chunk_bound(A.max_kv, wide) * A.kv.hkv * column_tiles(A.max_rows, A.group);
    return per <= 0x7fffffffLL / A.n_streams - kCUs && A.n_streams <= 64 * 65535 ? per * A.n_streams : -1;
}

bool attn_fits(const AttnArgs &A)
{
    return most_pieces(A, is_wide(A.max_rows, A.group)) >= 0 && (long long)A.total_rows * A.hq <= (long long)kMaxGroups * kJoinWaves;
}

hipError_t launch_attn(AttnArgs A, void *workspace, hipStream_t stream)
{
    const bool wide = is_wide(A.max_rows, A.group);
    const long long pieces = most_pieces(A, wide);
    A.chunks = chunk_bound(A.max_kv, wide);
    A.part = static_cast<float *>(workspace);
    A.stat = reinterpret_cast<float2 *>(A.part + (size_t)A.total_rows * A.hq * A.chunks * A.kv.d);
    switch (A.kv.d) {
    case 64: return launch_fmt<64>(A, wide, pieces, stream);
    case 128: return launch_fmt<128>(A, wide, pieces, stream);
    default: return launch_fmt<256>(A, wide, pieces, stream);
    }
}

}  // namespace gdn
