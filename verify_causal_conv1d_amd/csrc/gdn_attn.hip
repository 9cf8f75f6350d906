// Attention of steps, verify windows and draft trees over the paged cache.
// Contract in include/libgdn.h (gdn_attn_window).
//
// For row t of a stream, query head h of kv head h / G (G = hq / hkv), and the
// visible keys j (the stream's kv_len cached rows, the row itself and its
// ancestors in the window):
//     s_j = scale q . k_j,   o = sum_j e^{s_j} v_j / sum_j e^{s_j},   out = o sigmoid(gate).
// Keys and values are read once for all rows and query heads of a kv head: the
// (row, head) pairs of a stream and kv head are the 16 columns of the matrix
// products S^T = K Q^T and O^T = V^T P^T.  One pass over the keys keeps the
// running maximum m and sum l of each column (base-2 exponentials).
//
// A stream's keys are cut into chunks at logical positions (a rule on its own
// length alone, so its results do not depend on the other streams of the
// call).  A chunk is one workgroup: its waves take tiles of 32 keys in turn and
// join through LDS.  A stream of one chunk ends there; otherwise m, l and O of
// every chunk go to the workspace and join_kernel merges them in chunk order:
//     m = max m_c,   l = sum l_c 2^{m_c - m},   o = sum O_c 2^{m_c - m} / l.
#include "gdn_attn.h"
#include "gdn_device.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kAttnThreads = 256, kAttnWaves = 4;
constexpr int kTile = 32;                  // keys of a wave's step
constexpr int kCols = 16;                  // (row, head) pairs of a workgroup
constexpr int kChunkUnit = kTile * kAttnWaves;
constexpr int kMaxChunks = 128;            // of one stream

// Keys of a chunk of a stream with len keys: at most kMaxChunks chunks, whole
// steps of the workgroup.
__host__ __device__ inline int chunk_keys(int len)
{
    const int unit = kChunkUnit * kMaxChunks;
    return kChunkUnit * ((len + unit - 1) / unit);
}

__host__ __device__ inline int chunk_count(int len)
{
    return len <= 0 ? 0 : (len + chunk_keys(len) - 1) / chunk_keys(len);
}

// Chunks of the longest stream: the count falls where the chunk grows by a
// step, so the bound is that of the last full step.
inline int chunk_bound(int max_kv)
{
    return max_kv >= kChunkUnit * kMaxChunks ? kMaxChunks : chunk_count(max_kv);
}

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

// ---- operands in registers ---------------------------------------------------

// 8 elements in bf16 of a lane's run of 16 (bf16: 32 bytes, e4m3: 16 bytes)
template <bool F8>
struct Run16;
template <>
struct Run16<false> {
    uint4 a, b;
    __device__ __forceinline__ void load(const uint8_t *p)
    {
        a = reinterpret_cast<const uint4 *>(p)[0];
        b = reinterpret_cast<const uint4 *>(p)[1];
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
    __device__ __forceinline__ void load(const uint8_t *p) { a = reinterpret_cast<const uint4 *>(p)[0]; }
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
struct VRow {
    static constexpr int BYTES = D * (F8 ? 1 : 2);
    static constexpr int NL = BYTES > 256 ? 2 : 1;
    static constexpr int W = BYTES / NL / 64;           // dwords of a load: 1, 2 or 4
    static constexpr int EPL = W * (F8 ? 4 : 2);
    uint32_t w[NL][W];
    __device__ __forceinline__ void load(const uint8_t *base, uint32_t off)
    {
#pragma unroll
        for (int h = 0; h < NL; ++h) {
            const uint8_t *p = base + (off + h * 16 * W * 4);
            if constexpr (W == 4) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p);
                w[h][0] = x.x, w[h][1] = x.y, w[h][2] = x.z, w[h][3] = x.w;
            } else if constexpr (W == 2) {
                const uint2 x = *reinterpret_cast<const uint2 *>(p);
                w[h][0] = x.x, w[h][1] = x.y;
            } else {
                w[h][0] = *reinterpret_cast<const uint32_t *>(p);
            }
        }
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
        for (int h = 0; h < NL; ++h)
#pragma unroll
            for (int i = 0; i < W; ++i) m |= bad(w[h][i]);
        return m == 0;
    }
    __device__ __forceinline__ void drop_bad()
    {
#pragma unroll
        for (int h = 0; h < NL; ++h)
#pragma unroll
            for (int i = 0; i < W; ++i) w[h][i] &= ~bad(w[h][i]);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int h = 0; h < NL; ++h)
#pragma unroll
            for (int i = 0; i < W; ++i) w[h][i] = 0;
    }
};

// The MFMA operand of column i of load h: that channel of the lane's 8 keys.
template <int D, bool F8>
__device__ __forceinline__ bf8v v_operand(const VRow<D, F8> (&v)[8], int h, int i)
{
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if constexpr (F8) {
            const uint32_t both = __builtin_amdgcn_perm(v[2 * q + 1].w[h][i / 4], v[2 * q].w[h][i / 4],
                                                        i & 2 ? 0x07030602u : 0x05010400u);
            o[q] = cvt2(both, i & 1);
        } else {
            o[q] = __builtin_amdgcn_perm(v[2 * q + 1].w[h][i / 2], v[2 * q].w[h][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
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

// the result of one (row, head) column's 4 channels: o / l, gated, in bf16
__device__ __forceinline__ uint2 finish4(const AttnArgs &A, float4 o, float inv, int r, int head, int d)
{
    float x[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    if (A.gate) {
        const uint2 g = *reinterpret_cast<const uint2 *>(A.gate + r * A.gate_row + head * A.gate_head + d);
        x[0] *= sigmoid_f(__uint_as_float(g.x << 16));
        x[1] *= sigmoid_f(__uint_as_float(g.x & 0xffff0000u));
        x[2] *= sigmoid_f(__uint_as_float(g.y << 16));
        x[3] *= sigmoid_f(__uint_as_float(g.y & 0xffff0000u));
    }
    return make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
}

// Adds the infinite and NaN values of the window's rows in [key0, key1) that a
// column sees (bits of seen) to its channels d .. d + 3.
template <int D, bool F8>
__device__ void add_bad(const AttnArgs &A, float4 &a, const int *rows16, uint32_t seen, int key0, int key1, int kv, int k0, int d)
{
    for (int key = key0; key < key1; ++key) {
        if (!(seen >> (key - kv) & 1)) continue;
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

template <int D, bool F8>
__global__ __launch_bounds__(kAttnThreads, 2) void attn_kernel(const AttnArgs A)
{
    constexpr int ESZ = F8 ? 1 : 2, ROW = D * ESZ, KS = D / 64;
    using V = VRow<D, F8>;
    constexpr int NT = V::NL * V::EPL;             // column tiles of O^T (16 channels each)
    constexpr int OP = D + 4;                      // padded LDS row of a column's channels
    extern __shared__ __align__(16) uint8_t smem[];
    float *o_lds = reinterpret_cast<float *>(smem);                    // [waves][kCols][OP]
    float *m_lds = o_lds + kAttnWaves * kCols * OP;                    // [waves][kCols]
    float *l_lds = m_lds + kAttnWaves * kCols;                         // [waves][kCols]
    uint4 *q_lds = reinterpret_cast<uint4 *>(l_lds + kAttnWaves * kCols);   // [KS][2][64]
    int *bad_lds = reinterpret_cast<int *>(q_lds + KS * 2 * 64);       // whether a window row's value is not finite
    uint32_t *seen_lds = reinterpret_cast<uint32_t *>(bad_lds + 4);    // [kCols]: bits of the window's rows a column sees
    int *rows16 = bad_lds + 4 + kCols;                                         // cache row of each 16 keys of the chunk

    const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = lane & 15, g = lane >> 4;
    int x = blockIdx.x;
    const int c = x % A.chunks;
    x /= A.chunks;
    const int h = x % A.kv.hkv;
    x /= A.kv.hkv;
    const int rt = x % A.row_tiles, s = x / A.row_tiles;

    int r0, m, kv;
    if (!stream_window(A, s, r0, m, kv)) return;
    const int len = kv + m, C = chunk_keys(len), k0 = c * C;
    const int cols = m * A.group;                                      // (row, head) pairs of this kv head
    if (k0 >= len || rt * kCols >= cols) return;
    const int k1 = min(k0 + C, len), nch = chunk_count(len);
    const int col = rt * kCols + n, ncol = min(cols - rt * kCols, kCols);
    const int t = min(col / A.group, m - 1);

    static_assert(kAttnWaves == 4, "");
    // cache rows of the chunk's keys, 16 at a time (pages hold multiples of 16)
    bool ok = true;
    for (int i = tid; i < C / 16; i += kAttnThreads) {
        const int key = min(k0 + 16 * i, (len - 1) & ~15);
        const int id = A.table[(size_t)s * A.max_blocks + (key >> A.kv.page_shift)];
        const bool good = id >= 0 && id < A.kv.n_pages;
        ok = ok && good;
        rows16[i] = good ? ((id * A.kv.hkv + h) << A.kv.page_shift) + (key & ((1 << A.kv.page_shift) - 1)) : 0;
    }
    const uint32_t seen = seen_rows(A, r0, m, t, ok);
    // the queries, in the order of the lanes' operands: [k-step][half][lane] of
    // 16 bytes (column n, channels 64 k + 16 g + 8 half; zero past the last column)
    for (int i = tid; i < KS * 2 * 64; i += kAttnThreads) {
        const int qn = i & 15, qg = i >> 4 & 3, hh = i >> 6 & 1, k = i >> 7;
        const int qc = min(rt * kCols + qn, cols - 1);
        uint4 x = {0, 0, 0, 0};
        if (qn < ncol)
            x = *reinterpret_cast<const uint4 *>(A.q + ((size_t)(r0 + qc / A.group) * A.hq + h * A.group + qc % A.group) * D + 64 * k
                                                 + 16 * qg + 8 * hh);
        q_lds[i] = x;
    }
    const bool wave_ok = !__ballot(!ok);
    if (lane == 0) l_lds[wave] = wave_ok ? 1.0f : 0.0f;     // free until the waves join
    if (tid == 0) *bad_lds = 0;
    if (tid < kCols) seen_lds[tid] = seen;
    __syncthreads();
    ok = l_lds[0] + l_lds[1] + l_lds[2] + l_lds[3] == 4.0f;
    if (!ok) {
        if (nch > 1 && tid < ncol)
            A.stat[((size_t)(r0 + (rt * kCols + tid) / A.group) * A.hq + h * A.group + (rt * kCols + tid) % A.group) * A.chunks + c] =
                make_float2(0.0f, kSkipped);
        return;
    }


    f4v o[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i] = f4v{0, 0, 0, 0};
    float mx = -INFINITY, sum = 0.0f;

    Run16<F8> kk[2][KS];
    V vv[8];
    const uint32_t k_off = n * ROW + 16 * g * ESZ, v_off = 4 * g * ROW + n * V::W * 4;
    auto load_k = [&](int tile) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint8_t *p = A.kv.k + (size_t)__builtin_amdgcn_readfirstlane(rows16[2 * tile + u]) * ROW;
#pragma unroll
            for (int k = 0; k < KS; ++k) kk[u][k].load(p + (k_off + 64 * k * ESZ));
        }
    };
    auto load_v = [&](int tile) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint8_t *p = A.kv.v + (size_t)__builtin_amdgcn_readfirstlane(rows16[2 * tile + u]) * ROW;
#pragma unroll
            for (int j = 0; j < 4; ++j) vv[4 * u + j].load(p, v_off + j * ROW);
        }
    };
    const int tiles = (k1 - k0 + kTile - 1) / kTile;
    if (wave < tiles) {
        load_k(wave);
        load_v(wave);
    }
    for (int tile = wave; tile < tiles; tile += kAttnWaves) {
        const bool more = tile + kAttnWaves < tiles;
        const int key0 = k0 + tile * kTile + 4 * g;      // the lane's keys: key0 + 16 u + i
        float p[8];
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
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float4 ks = {1, 1, 1, 1};
            if constexpr (F8)
                ks = *reinterpret_cast<const float4 *>(A.kv.k_scale + __builtin_amdgcn_readfirstlane(rows16[2 * tile + u]) + 4 * g);
            p[4 * u] = acc[u][0] * A.scale * ks.x;
            p[4 * u + 1] = acc[u][1] * A.scale * ks.y;
            p[4 * u + 2] = acc[u][2] * A.scale * ks.z;
            p[4 * u + 3] = acc[u][3] * A.scale * ks.w;
        }
        const bool tail = k0 + tile * kTile + kTile > kv;   // holds keys of the window or past the end
        uint32_t vis = 0xff;
        if (tail) {
            vis = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = key0 + 16 * (i / 4) + (i & 3) - kv;   // place in the window
                if (j < 0 || (j < kMaxWindowRows && (seen >> j & 1))) vis |= 1u << i;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(vis >> i & 1)) p[i] = -INFINITY;
        }
        float tm = p[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) tm = fmaxf(tm, p[i]);
        tm = fmaxf(mx, max_rows4(tm));
        const float base = tm == -INFINITY ? 0.0f : tm;     // no key seen so far: every p is 0
        const float back = __builtin_amdgcn_exp2f(mx - base);
        mx = tm;
        float ps = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(p[i] - base);
            ps += p[i];
        }
        sum = fmaf(sum, back, ps);
        if (__ballot(back != 1.0f)) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][e] *= back;
        }
        if constexpr (F8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float4 vs = *reinterpret_cast<const float4 *>(A.kv.v_scale + __builtin_amdgcn_readfirstlane(rows16[2 * tile + u]) + 4 * g);
                p[4 * u] *= vs.x;
                p[4 * u + 1] *= vs.y;
                p[4 * u + 2] *= vs.z;
                p[4 * u + 3] *= vs.w;
            }
            if (tail)        // a masked row's scale may be anything
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!(vis >> i & 1)) p[i] = 0.0f;
        }
        // P in bf16, rounded to nearest: its error is at most 2^-9 of each term,
        // that of the bf16 result's own rounding; the sum keeps the fp32 values
        const uint4 pw = {pack2(p[0], p[1]), pack2(p[2], p[3]), pack2(p[4], p[5]), pack2(p[6], p[7])};
        const bf8v pb = __builtin_bit_cast(bf8v, pw);
        if (tail) {
            // rows past the end hold anything: zero them
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (key0 + 16 * (i / 4) + (i & 3) >= len) vv[i].zero();
            // 0 * inf is NaN: an infinite or NaN value of a window row must not
            // reach the rows that do not see it.  Such values are left out of the
            // product, and added at the end to the results that they belong to.
            if (m > 1) {
                bool fin = true;
#pragma unroll
                for (int i = 0; i < 8; ++i) fin = fin && vv[i].finite();
                if (__ballot(!fin)) {
                    if (lane == 0) *bad_lds = 1;
#pragma unroll
                    for (int i = 0; i < 8; ++i) vv[i].drop_bad();
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) o[i] = mfma(v_operand<D, F8>(vv, i / V::EPL, i % V::EPL), pb, o[i]);
        if (more) load_v(tile + kAttnWaves);
    }

    // join the waves: the column's maximum over them, each wave's O and l scaled to it
    sum = sum_rows4(sum);
    if (g == 0) m_lds[wave * kCols + n] = mx;
    __syncthreads();
    float top = m_lds[n];
#pragma unroll
    for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, m_lds[w * kCols + n]);
    const float f = __builtin_amdgcn_exp2f(mx - (top == -INFINITY ? 0.0f : top));
    if (g == 0) l_lds[wave * kCols + n] = sum * f;
    if (n < ncol) {
        float *row = o_lds + (wave * kCols + n) * OP;
#pragma unroll
        for (int hh = 0; hh < V::NL; ++hh)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float *p = row + hh * 16 * V::EPL + (4 * g + e) * V::EPL;
#pragma unroll
                for (int i = 0; i < V::EPL; i += 4)
                    *reinterpret_cast<float4 *>(p + i) = make_float4(o[hh * V::EPL + i][e] * f, o[hh * V::EPL + i + 1][e] * f,
                                                                     o[hh * V::EPL + i + 2][e] * f, o[hh * V::EPL + i + 3][e] * f);
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
        const int cg = rt * kCols + cc, r = r0 + cg / A.group, hd = h * A.group + cg % A.group;
        if (*bad_lds) add_bad<D, F8>(A, a, rows16, seen_lds[cc], max(kv, k0), k1, kv, k0, d);
        if (nch == 1) {
            *reinterpret_cast<uint2 *>(A.out + ((size_t)r * A.hq + hd) * D + d) = finish4(A, a, 1.0f / l, r, hd, d);
        } else {
            const size_t at = ((size_t)r * A.hq + hd) * A.chunks + c;
            *reinterpret_cast<float4 *>(A.part + at * D + d) = a;
            if (d == 0) A.stat[at] = make_float2(mm, l);
        }
    }
}

// Merges a (row, head)'s chunks.  D / 4 lanes share the channels, the rest of
// the workgroup splits the chunks.
template <int D>
__global__ __launch_bounds__(256) void join_kernel(const AttnArgs A)
{
    constexpr int LANES = D / 4, PARTS = 256 / LANES;
    __shared__ float w[kMaxChunks];
    __shared__ float4 acc[PARTS][LANES];
    const int r = blockIdx.x / A.hq, head = blockIdx.x % A.hq, tid = threadIdx.x;
    int lo = 0, hi = A.n_streams - 1;           // the last stream that starts at or before r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (A.row_start[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    int r0, m, kv;
    if (!stream_window(A, lo, r0, m, kv) || r < r0 || r >= r0 + m) return;
    const int nch = chunk_count(kv + m);
    if (nch <= 1) return;
    const size_t at = ((size_t)r * A.hq + head) * A.chunks;
    float2 st = {-INFINITY, 0.0f}, st2 = st;
    const int lane = tid & 63;
    if (lane < nch) st = A.stat[at + lane];
    if (lane + 64 < nch) st2 = A.stat[at + 64 + lane];
    if (__ballot(st.y < 0.0f || st2.y < 0.0f)) return;      // a chunk was skipped: so is the stream
    float top = fmaxf(st.x, st2.x);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o));
    const float base = top == -INFINITY ? 0.0f : top;
    const float f = __builtin_amdgcn_exp2f(st.x - base), f2 = __builtin_amdgcn_exp2f(st2.x - base);
    const float l = sum_wave(st.y * f + st2.y * f2);
    if (tid < 64) {
        w[lane] = f;
        w[lane + 64] = f2;
    }
    __syncthreads();
    const int d4 = tid % LANES, part = tid / LANES;
    float4 a = {0, 0, 0, 0};
    for (int c = part; c < nch; c += PARTS) {
        const float4 b = *reinterpret_cast<const float4 *>(A.part + (at + c) * D + 4 * d4);
        const float f0 = w[c];
        a.x = fmaf(b.x, f0, a.x), a.y = fmaf(b.y, f0, a.y), a.z = fmaf(b.z, f0, a.z), a.w = fmaf(b.w, f0, a.w);
    }
    acc[part][d4] = a;
    __syncthreads();
    if (part == 0) {
#pragma unroll
        for (int p = 1; p < PARTS; ++p) {
            const float4 b = acc[p][d4];
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
        }
        *reinterpret_cast<uint2 *>(A.out + ((size_t)r * A.hq + head) * D + 4 * d4) = finish4(A, a, 1.0f / l, r, head, 4 * d4);
    }
}

template <int D, bool F8>
hipError_t launch_d(const AttnArgs &A, hipStream_t stream)
{
    const size_t lds = sizeof(float) * kAttnWaves * kCols * (D + 4 + 2) + D * 2 * kCols
                       + sizeof(int) * (4 + kCols + chunk_keys(A.max_kv) / 16);
    static const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(attn_kernel<D, F8>),
                                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)kRowsMaxLds);
    if (e != hipSuccess) return e;
    const long long blocks = (long long)A.chunks * A.kv.hkv * A.row_tiles * A.n_streams;
    hipLaunchKernelGGL((attn_kernel<D, F8>), dim3((unsigned)blocks), dim3(kAttnThreads), lds, stream, A);
    if (A.chunks > 1)
        hipLaunchKernelGGL((join_kernel<D>), dim3((unsigned)(A.total_rows * A.hq)), dim3(256), 0, stream, A);
    return hipGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(int hq, int hkv, int d, int total_rows, int max_rows, int max_kv)
{
    const size_t chunks = chunk_bound(max_kv);
    if (chunks <= 1) return 0;
    return (size_t)total_rows * hq * chunks * (sizeof(float) * d + sizeof(float2));
}

bool attn_fits(const AttnArgs &A)
{
    const long long tiles = (A.max_rows * A.group + kCols - 1) / kCols;
    return (long long)chunk_bound(A.max_kv) * A.kv.hkv * tiles <= 0x7fffffffLL / A.n_streams
           && (long long)A.total_rows * A.hq <= 0x7fffffffLL;
}

hipError_t launch_attn(AttnArgs A, void *workspace, hipStream_t stream)
{
    A.chunks = chunk_bound(A.max_kv);
    A.row_tiles = (A.max_rows * A.group + kCols - 1) / kCols;
    A.part = static_cast<float *>(workspace);
    A.stat = reinterpret_cast<float2 *>(A.part + (size_t)A.total_rows * A.hq * A.chunks * A.kv.d);
    const bool f8 = A.kv.k_scale != nullptr;
    switch (A.kv.d) {
    case 64: return f8 ? launch_d<64, true>(A, stream) : launch_d<64, false>(A, stream);
    case 128: return f8 ? launch_d<128, true>(A, stream) : launch_d<128, false>(A, stream);
    default: return f8 ? launch_d<256, true>(A, stream) : launch_d<256, false>(A, stream);
    }
}

}  // namespace gdn
