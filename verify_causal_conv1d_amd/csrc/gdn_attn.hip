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
//    instructions, and join through LDS;
//  - more, attn_wide_kernel: each wave has a column tile of its own, and K and
//    V pass through LDS once for all of them.
// (16 streams of 700 to 8,191 keys, 24 query and 4 kv heads of 256: with 24
// columns the wide kernel takes 53 us and the other one, reading K and V once a
// tile, 69; with 48 columns 59 and 97.  One stream of 500 keys and 18 columns:
// 15.7 and 14.4.)
#include "gdn_attn.h"
#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_once.h"

namespace gdn {
namespace {

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

// What a stream's skipped chunk leaves in the workspace for join_kernel: sums
// are never negative.
constexpr float kSkipped = -1.0f;

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
template <bool F8, int W>
__device__ __forceinline__ bool clean_values(VPart<F8, W> (&v)[8], int key0, int len, int m)
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

// ---- more columns ----------------------------------------------------------------

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

// Four stages of keys and values in LDS, filled by direct loads (16 bytes a
// lane, 1 KB an instruction): while a stage is multiplied the next three are
// in flight, up to 96 KB a CU, and one barrier a stage separates its readers
// from the loads that fill it again.  K rows are stored with their 16-byte
// pieces exchanged by a function of the row (piece ^ swizzle), so that the 16
// rows of an operand lie in different banks.
//
// One workgroup of 8 waves stays on each CU and goes through its pieces.  16
// draft trees of up to 16 rows over 700 to 8,191 keys (96 columns, 212 MB): 70 us
// with the join (11 us, what bounds it is said there).  A tile of 32 keys
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

// Merges a (row, head)'s chunks, one wave each, D / 64 channels a lane.  What it
// reads does not wait for the stream to be found: the first parts, the sums and
// the gates are asked for at once, by the row alone (a stream has at most
// A.chunks chunks; what lies past its own is not used), and the streams' windows
// are looked at 64 at a time.  The price: a (row, head) of a short stream asks for
// more parts than it has.  The 16 trees above, the longest of which has 17 chunks
// and ten of which have 4 to 6, ask for 58 MB where their chunks wrote 25, and the
// kernel's 11 us are the time of those bytes.
constexpr int kJoinWaves = 4, kJoinBatch = 16;      // loads in flight

template <int D>
__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(const AttnArgs A, const int is_wide)
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
    part_t b[kJoinBatch];
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
    const int nch = chunk_count(__builtin_amdgcn_readlane(kv, l) + __builtin_amdgcn_readlane(m, l), is_wide);
    if (nch <= 1) return;
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
        if (c > 0)
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

template <int D, bool F8>
hipError_t launch_d(const AttnArgs &A, bool wide, long long pieces, hipStream_t stream)
{
    const int list = longest_chunk(A.max_kv, wide) / 16;
    const size_t list_bytes = sizeof(int) * list;
    if (!wide) {
        constexpr size_t lds = sizeof(float) * kAttnWaves * kCols * (D + 4 + 2) + D * 2 * kCols + sizeof(int) * (4 + kCols);
        // 64 streams a grid row
        const unsigned per_row = (unsigned)(pieces / A.n_streams * (A.n_streams < 64 ? A.n_streams : 64));
        hipLaunchKernelGGL((attn_kernel<D, F8>), dim3(per_row, ceil_div(A.n_streams, 64)), dim3(kAttnThreads), lds + list_bytes, stream, A);
    } else {
        const unsigned blocks = (unsigned)(pieces < kCUs ? pieces : kCUs);
        hipLaunchKernelGGL((attn_wide_kernel<D, F8>), dim3(blocks), dim3(kWideThreads), 2 * list_bytes, stream, A, list);
    }
    if (A.chunks > 1)
        hipLaunchKernelGGL((join_kernel<D>), dim3(ceil_div(A.total_rows * A.hq, kJoinWaves)), dim3(64 * kJoinWaves), 0, stream, A, wide ? 1 : 0);
    return hipGetLastError();
}

int column_tiles(int max_rows, int group)
{
    return is_wide(max_rows, group) ? ceil_div(max_rows * group, kWideCols) : 1;
}

}  // namespace

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
    const bool wide = is_wide(A.max_rows, A.group), f8 = A.kv.k_scale != nullptr;
    const long long pieces = most_pieces(A, wide);
    A.chunks = chunk_bound(A.max_kv, wide);
    A.part = static_cast<float *>(workspace);
    A.stat = reinterpret_cast<float2 *>(A.part + (size_t)A.total_rows * A.hq * A.chunks * A.kv.d);
    switch (A.kv.d) {
    case 64: return f8 ? launch_d<64, true>(A, wide, pieces, stream) : launch_d<64, false>(A, wide, pieces, stream);
    case 128: return f8 ? launch_d<128, true>(A, wide, pieces, stream) : launch_d<128, false>(A, wide, pieces, stream);
    default: return f8 ? launch_d<256, true>(A, wide, pieces, stream) : launch_d<256, false>(A, wide, pieces, stream);
    }
}

}  // namespace gdn
