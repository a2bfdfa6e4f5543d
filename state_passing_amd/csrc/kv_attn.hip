// kv_attn.hip -- attention over the paged 8-bit cache (linrec_kv_attn).
#include <hip/hip_runtime.h>

#include <math.h>

#include <algorithm>

#include "kv.hpp"

namespace linrec {
namespace {

struct AttnArgs {
    KvCache c;
    Act<const bf16> q;
    Act<bf16> o;
    float* lse;
    float* part;         // per split: rows of D unnormalised sums, then (max, sum) of every row (part_floats)
    const int* past;
    const int* n_new;
    int B, T, Hq, group, window, nsplit;
    int rows, row_tiles; // query rows of a key/value head (T * group), tiles of them
    float c2;            // |scale| * log2(e)
    bool negate;         // scale < 0: the sign goes into q
};

// The query rows of one key/value head are (token, head of the group) pairs,
// token-major: row r is token r / group, head h * group + r % group.

// Keys are taken 64 at a time (a tile), scores as S^T = K Q^T: the result of a
// 16x16 product gives lane (g, t) four keys of row t, so the softmax of a row
// stays within the 4 lanes of a column and exp(S^T) is, unmoved, the right
// operand of O^T = V^T P^T.  Which keys a tile's 4 products hold is free: product
// i of lane group g holds the keys of KEYS below, chosen so that the 8 values a
// lane contributes to a k32 step of the second product are neighbours in V's
// rows, one 16-byte load.

// What a row sees of a tile: offsets lo .. hi, in the 16-key groups (a group
// lies in one page) whose page is there.
struct Seen {
    int lo, hi;
    unsigned groups;
    __device__ __forceinline__ bool operator()(int key) const
    {
        return key >= lo && key <= hi && (groups >> (key >> 4) & 1);
    }
};

// 8 codes (two words) times 2^e as bf16, exact: e4m3 has 3 mantissa bits.  The
// conversion takes the scale's exponent field, which is all a power of two has.
__device__ __forceinline__ bf16x8 values8(unsigned lo, unsigned hi, float scale)
{
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ Frag<bf16> frag(bf16x8 v)
{
    Frag<bf16> f;
    f.v = v;
    return f;
}

// Running softmax of the 16 rows of a lane column (row t): a bound on the raw
// scores (softmax_tile), this lane's share of the sum, and the sums O^T: tile dt of lane
// (g, t) holds features 16 dt + 4 g + r of row t.
template <int D>
struct RowState {
    float m = -INFINITY, l = 0.f;
    floatx4 acc[D / 16];
    __device__ __forceinline__ void clear()
    {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            acc[i] = zero4();
    }
};

__device__ __forceinline__ float quad_max(float x)
{
    x = fmaxf(x, __shfl_xor(x, 16, 64));
    return fmaxf(x, __shfl_xor(x, 32, 64));
}

__device__ __forceinline__ float quad_sum(float x)
{
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// One tile's scores x (lane (g, t): product i, element r) become the weights'
// fragments p (k32 step s from products 2s, 2s + 1).
//
// The weights enter the second product as bf16, V's type there (exact for its
// codes): each is off by at most 2^-8 of itself, so o by 2^-8 sum_j p_j |v_j|
// before its own rounding.  Of outputs whose rounding alone puts them 0.0017 off
// (relative, root mean square), that makes 0.0019 (one user of 4096 tokens) to 0.0023
// (4096 tokens behind 12K).  Pairs of bf16 would halve the second product's rate,
// on the unit that bounds pieces.  The total l is of the weights before the rounding:
// adding up the rounded ones would take a conversion back for each, so what a row
// really gives its values adds up to 1 within 2^-8.
template <int D>
__device__ __forceinline__ void softmax_tile(RowState<D>& st, floatx4 (&x)[4], Frag<bf16> (&p)[2], float c2)
{
    // (of a NaN this maximum is NaN, which moves nothing: the row ends as NaN whatever
    // st.m is.  One that passed NaN by would take 20 instructions for 8.)
    float mx = __builtin_elementwise_maximum(x[0][0], x[0][1]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = i ? 0 : 2; r < 4; r += 2)
            mx = __builtin_elementwise_maximum(__builtin_elementwise_maximum(mx, x[i][r]), x[i][r + 1]);
    // st.m only has to keep the exponents in range, so it is moved (for all 4
    // lanes of a row together) when a score passes it by 2^8, not at every new
    // maximum: most tiles then need neither the exchange nor the rescaling
    if (__any((mx - st.m) * c2 > 8.f)) {
        mx = fmaxf(st.m, quad_max(mx));
        const float keep = __builtin_amdgcn_exp2f((st.m - (mx == -INFINITY ? 0.f : mx)) * c2);
        st.l *= keep;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
            st.acc[i] *= keep;
        st.m = mx;
    }
    const float off = (st.m == -INFINITY ? 0.f : st.m) * c2;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            x[i][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i][r], c2, -off));
            sum += x[i][r];
        }
    st.l += sum;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            p[s].v[r] = (bf16)x[2 * s][r];
            p[s].v[4 + r] = (bf16)x[2 * s + 1][r];
        }
}

// Query fragments of 16 rows from row r0: element e of k32 step s is feature
// feat(s) + e.  Rows that are not there read as zeros.
template <int D, typename Feat>
__device__ __forceinline__ void load_q(Frag<bf16> (&q)[D / 32], const AttnArgs& a, int b, int h, int row,
                                       int rows, Feat feat)
{
    const bool there = row < rows;
    const int t = there ? row / a.group : 0, hq = h * a.group + (there ? row % a.group : 0);
    const bf16* p = a.q.head(b, hq) + (int64_t)t * a.q.st;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
        u32x4 v = there ? *reinterpret_cast<const u32x4*>(p + feat(s)) : u32x4{0u, 0u, 0u, 0u};
        if (a.negate)
            v ^= u32x4{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
        q[s].v = __builtin_bit_cast(bf16x8, v);
    }
}

// The tiles of keys that a block of rows [r0, r1) reads, and the share of them
// that is this split's.
struct Range {
    int k0, end;         // first key (a multiple of 64), end of the visible keys
    int first, last;     // this split's tiles [first, last)
    __device__ __forceinline__ Range(const AttnArgs& a, const Span& sp, int r0, int r1, int split, int least)
    {
        const int lo = a.window > 0 ? max(0, sp.past + r0 / a.group - a.window + 1) : 0;
        end = min(sp.past + (r1 - 1) / a.group + 1, a.c.max_pages << a.c.shift);
        k0 = lo & ~63;
        const int tiles = end > k0 ? (end - k0 + 63) / 64 : 0;
        const int per = max((tiles + a.nsplit - 1) / a.nsplit, least);
        first = min(tiles, split * per);
        last = min(tiles, first + per);
    }
};

// A tile at the border of what the rows see may hold, for some rows, values
// they do not see.  Their weight is 0, but 0 * NaN is not 0.  Values that are
// not finite (a NaN code, any code under a scale that is not, a code that the
// scale takes past bf16's range) are therefore taken out of a border tile when it
// is loaded, and rows that do see one get a NaN in its feature afterwards.  Both
// are rare, and kept off the registers of the rest.

// The codes that are not finite under `scale` are those whose low 7 bits, as a
// number, reach some border; this is its distance from 0x80, so that adding it
// carries into a code's top bit exactly for them.  Of a scale 2^e below 2^120 that is
// 0x7f, the NaN code (448 * 2^119 is below 2^128); from there on the code of
// 2^(128 - e), which is (128 - e + 7) << 3; of a scale that is not finite every code.
// (With a comparison where the maximum stands the piece kernel takes 485 us for 479.)
__device__ __forceinline__ unsigned nonfinite_lift(float scale)
{
    const int e = (int)(__float_as_uint(scale) >> 23 & 0xffu);   // biased by 127
    return e == 255 ? 0x80u : (unsigned)max(0x80 - ((262 - e) << 3), 1);
}

// 16 codes under `scale`: what is not finite becomes code 0; whether there was
// any.  (finite_scale() of the scale then keeps 0 a 0.)
__device__ __forceinline__ bool take_nonfinite(u32x4& v, float scale)
{
    unsigned any = 0;
    const unsigned lift = nonfinite_lift(scale) * 0x01010101u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned n = ((v[i] & 0x7f7f7f7fu) + lift) & 0x80808080u;
        v[i] &= ~((n >> 7) * 0xffu);
        any |= n;
    }
    return any != 0;
}

__device__ __forceinline__ float finite_scale(float scale)
{
    return (__float_as_uint(scale) & 0x7f800000u) == 0x7f800000u ? 1.f : scale;
}

// Of 8 codes under `scale`, 1 for each that is not finite, as bf16.
__device__ __forceinline__ Frag<bf16> nonfinite8(u32x2 w, float scale)
{
    const unsigned lift = nonfinite_lift(scale) * 0x01010101u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const unsigned n = ((w[i] & 0x7f7f7f7fu) + lift) & 0x80808080u;
        w[i] = (n >> 7) * 0x38u;   // 0x38 is 1
    }
    return frag(values8(w[0], w[1], 1.f));
}

// Gives the rows of st a NaN wherever they see a value that is not finite:
// `codes(key, feature, scale)` reads the 8 codes from a key of the tile on.
template <int D, int NR, typename Codes, typename Key>
__device__ __forceinline__ void give_nonfinite(RowState<D> (&st)[NR], const Seen (&seen)[NR], Codes codes, Key key)
{
    const int t = lane_id() & 15;
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        unsigned hits = 0;   // bit 4 dt + r: the row sees one in feature 16 dt + 4 g + r
#pragma unroll 1
        for (int e = 0; e < D / 8; ++e) {
            const int dt = e >> 1, s = e & 1;
            Frag<bf16> vis;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                vis.v[i] = (bf16)(seen[n](key(2 * s + i / 4, i % 4)) ? 1.f : 0.f);
            float scale;
            const u32x2 w = codes(key(2 * s, 0), 16 * dt + t, scale);
            const floatx4 hit = mma(nonfinite8(w, scale), vis, zero4());
#pragma unroll
            for (int r = 0; r < 4; ++r)
                hits |= (hit[r] > 0.f ? 1u : 0u) << (4 * dt + r);
        }
#pragma unroll
        for (int i = 0; i < D / 4; ++i)
            st[n].acc[i / 4][i % 4] = hits >> i & 1 ? __builtin_nanf("") : st[n].acc[i / 4][i % 4];
    }
}

// Asks the scheduler for the order of a product loop over READS fragments from
// LDS, NR products each: four reads ahead of the products, where it would read
// two, wait, and multiply (piece kernel, 4096 tokens behind 12K: 530 -> 503 us).
template <int NR, int READS>
__device__ __forceinline__ void read_ahead()
{
    constexpr int AHEAD = 4;
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);        // LDS reads
#pragma unroll
    for (int i = 0; i < READS - AHEAD; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, NR, 0);         // matrix instructions
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x8, AHEAD * NR, 0);
}

// Weights and values of one tile, given its scores; LDS: they are read from LDS; vfrag(dt, s): V's fragment.
// whole: every row sees all of the tile (wave-uniform).
template <int D, int NR, bool LDS, typename VFrag, typename Key>
__device__ __forceinline__ void attend(RowState<D> (&st)[NR], floatx4 (&x)[NR][4], float c2, bool whole,
                                       const Seen (&seen)[NR], VFrag vfrag, Key key)
{
    if (!whole) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    x[n][i][r] = seen[n](key(i, r)) ? x[n][i][r] : -INFINITY;
    }
    Frag<bf16> p[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n)
        softmax_tile<D>(st[n], x[n], p[n], c2);
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const Frag<bf16> v = vfrag(dt, s);
#pragma unroll
            for (int n = 0; n < NR; ++n)
                st[n].acc[dt] = mma(v, p[n][s], st[n].acc[dt]);
        }
    if constexpr (LDS)
        read_ahead<NR, D / 8>();
}

// A row's place in o and lse.  No weight at all means that the row sees nothing
// (zeros and -inf).  Where there is a maximum, that or an infinite sum means that
// the maximum passes fp32's range with the scale and took every exponent with it:
// NaN, not an empty row.
template <int D>
__device__ __forceinline__ void write_row(const AttnArgs& a, int b, int h, int row, int f, const floatx4& y, float m,
                                          float l)
{
    const int tok = row / a.group, hq = h * a.group + row % a.group;
    const bool sums = l != 0.f && l != INFINITY, empty = m == -INFINITY;
    const float inv = sums ? 1.f / l : empty ? 0.f : __builtin_nanf("");
    *reinterpret_cast<bf16x4*>(a.o.head(b, hq) + (int64_t)tok * a.o.st + f) =
        bf16x4{(bf16)(y[0] * inv), (bf16)(y[1] * inv), (bf16)(y[2] * inv), (bf16)(y[3] * inv)};
    if (a.lse && f == 0)
        a.lse[((int64_t)b * a.Hq + hq) * a.T + tok] =
            sums ? (m * a.c2 + __log2f(l)) * 0.6931471805599453f : empty ? -INFINITY : __builtin_nanf("");
}

// From one split's part to the next, for n rows: D sums and two statistics each,
// up to whole 16-byte vectors (of an odd n they end 8 bytes into one).
constexpr __host__ __device__ int64_t part_floats(int64_t n, int D) { return (n * (D + 2) + 3) / 4 * 4; }

// A row's sums, and its maximum and total, in a split's part.
template <int D>
__device__ __forceinline__ float* part_row(const AttnArgs& a, int split, int b, int h, int row)
{
    const int64_t n = (int64_t)a.B * a.c.H * a.rows;
    return a.part + split * part_floats(n, D) + (((int64_t)b * a.c.H + h) * a.rows + row) * D;
}

template <int D>
__device__ __forceinline__ float* part_stat(const AttnArgs& a, int split, int b, int h, int row)
{
    const int64_t n = (int64_t)a.B * a.c.H * a.rows;
    return a.part + split * part_floats(n, D) + n * D + (((int64_t)b * a.c.H + h) * a.rows + row) * 2;
}

// ---- few rows: generation -----------------------------------------------
//
// Bound by the cache's bytes (2 D per key).  Four waves take every fourth tile
// of a split's keys each, straight from global memory to registers (no LDS, no
// barrier: a fragment is 16 contiguous bytes of K's or V's rows), the next
// tile's K and its page numbers loaded ahead, and join at the end.  32 sequences
// of 12K-16K tokens, 32 / 8 heads of 128: 167 us, 5.6 TB/s; one sequence of 4096
// tokens: 6.4-8 us, a chain of dependent loads.
// PAGED: a tile may span pages (pages of 16 and 32 tokens); else it lies in one,
// whose number, scales and address are then the wave's, not the lane's.
template <int D, int NR, bool PAGED>
__global__ __launch_bounds__(256, D * NR == 256 ? 1 : 2) void kv_attn_token_kernel(AttnArgs a)
{
    constexpr int KS = D / 64, DT = D / 16;
    __shared__ __align__(16) float red[4][16][D + 4];
    __shared__ float ms[4][16 * NR], ls[4][16 * NR];
    const int tile = blockIdx.x % a.row_tiles, split = blockIdx.x / a.row_tiles, h = blockIdx.y, b = blockIdx.z;
    const Span sp(a.past, a.n_new, b, a.T);
    const int rows = sp.n * a.group, r0 = tile * 16 * NR;
    if (r0 >= rows)
        return;
    const int r1 = min(rows, r0 + 16 * NR);
    const Range rg(a, sp, r0, r1, split, 4);
    const int wave = wave_id(), lane = lane_id(), t = lane & 15, g = lane >> 4;
    const int shift = a.c.shift, P = 1 << shift, H = a.c.H;
    // product i's rows 4 g' + r are the keys 16 g' + 4 i + r of the tile
    auto key = [&](int i, int r) { return 16 * g + 4 * i + r; };

    Frag<bf16> q[NR][D / 32];
    RowState<D> st[NR];
    int pos[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = r0 + 16 * n + t;
        load_q<D>(q[n], a, b, h, row, rows, [&](int s) { return 64 * (s / 2) + 16 * g + 8 * (s % 2); });
        st[n].clear();
        pos[n] = row < rows ? sp.past + row / a.group : -1;   // -1: sees nothing
    }
    // pages of the 16-token groups that this lane loads K (group t / 4) and V (group g) of
    struct Pages {
        int k, v;
    };
    auto pages = [&](int tl) {
        const int k = rg.k0 + 64 * tl;
        const bool in = tl < rg.last;
        if constexpr (!PAGED) {
            const int p = in ? __builtin_amdgcn_readfirstlane(page_of(a.c, b, k >> shift)) : -1;
            return Pages{p, p};
        } else {
            return Pages{in ? page_of(a.c, b, (k + 16 * (t >> 2)) >> shift) : -1,
                         in ? page_of(a.c, b, (k + 16 * g) >> shift) : -1};
        }
    };
    const int k_lane = (16 * (t >> 2) + (t & 3)) * D + 16 * g, v_lane = t * P + 16 * g;
    u32x4 kr[4][KS], vr[DT];
    float ks;
    auto load_k = [&](int tl, int page) {
        const int k = rg.k0 + 64 * tl;
        const int64_t ph = (int64_t)max(page, 0) * H + h;
        const uint8_t* p;
        if constexpr (PAGED)
            p = a.c.k + (ph * P + ((k + 16 * (t >> 2)) & (P - 1)) + (t & 3)) * D + 16 * g;
        else
            p = a.c.k + (ph * P + (k & (P - 1))) * D + k_lane;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < KS; ++j)
                kr[i][j] = *reinterpret_cast<const u32x4*>(p + 4 * i * D + 64 * j);
        ks = a.c.ks[ph];
    };
    int tl = rg.first + wave;
    Pages now = pages(tl), next = pages(tl + 4);
    if (tl < rg.last)
        load_k(tl, now.k);
    for (; tl < rg.last; tl += 4) {
        const int k0 = rg.k0 + 64 * tl;
        const int64_t ph = (int64_t)max(now.v, 0) * H + h;
        const uint8_t* vp;
        if constexpr (PAGED)
            vp = a.c.v + (ph * D + t) * P + ((k0 + 16 * g) & (P - 1));
        else
            vp = a.c.v + (ph * D * P + (k0 & (P - 1))) + v_lane;
#pragma unroll
        for (int i = 0; i < DT; ++i)
            vr[i] = *reinterpret_cast<const u32x4*>(vp + 16 * i * P);
        const float vs = a.c.vs[ph];
        floatx4 x[NR][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int n = 0; n < NR; ++n)
                x[n][i] = zero4();
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                const Frag<bf16> lo = frag(values8(kr[i][j][0], kr[i][j][1], ks));
                const Frag<bf16> hi = frag(values8(kr[i][j][2], kr[i][j][3], ks));
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    x[n][i] = mma(lo, q[n][2 * j], x[n][i]);
                    x[n][i] = mma(hi, q[n][2 * j + 1], x[n][i]);
                }
            }
        }
        // the keys that this lane's scores belong to are its group's
        const bool page_ok = now.v >= 0;
        now = next;
        if (tl + 4 < rg.last)
            load_k(tl + 4, now.k);
        next = pages(tl + 8);
        const bool whole = __all(page_ok) && k0 + 63 <= sp.past + r0 / a.group &&
                           (a.window <= 0 || k0 > sp.past + (r1 - 1) / a.group - a.window);
        Seen seen[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            seen[n].hi = min(pos[n], rg.end - 1) - k0;
            seen[n].lo = a.window > 0 ? pos[n] - a.window + 1 - k0 : 0;
            seen[n].groups = page_ok ? 15u : 0u;
        }
        bool bad = false;
        float vuse = vs;
        if (!whole) {
            vuse = finite_scale(vs);
#pragma unroll
            for (int i = 0; i < DT; ++i)
                bad |= take_nonfinite(vr[i], vs);
        }
        attend<D, NR, false>(st, x, a.c2, whole, seen,
                      [&](int dt, int s) { return frag(values8(vr[dt][2 * s], vr[dt][2 * s + 1], vuse)); }, key);
        if (__any(bad))
            give_nonfinite<D, NR>(st, seen, [&](int k, int f, float& scale) {
                scale = vs;
                return *reinterpret_cast<const u32x2*>(a.c.v + (ph * D + f) * P + ((k0 + k) & (P - 1)));
            }, key);
    }
    // join the four waves
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const float l = quad_sum(st[n].l);
        if (g == 0) {
            ms[wave][16 * n + t] = st[n].m;
            ls[wave][16 * n + t] = l;
        }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int at = 16 * n + t;
        const float m = fmaxf(fmaxf(ms[0][at], ms[1][at]), fmaxf(ms[2][at], ms[3][at]));
        const float f = __builtin_amdgcn_exp2f((st[n].m - (m == -INFINITY ? 0.f : m)) * a.c2);
#pragma unroll
        for (int i = 0; i < DT; ++i)
            *reinterpret_cast<floatx4*>(&red[wave][t][16 * i + 4 * g]) = st[n].acc[i] * f;
        __syncthreads();
        constexpr int LPR = D / 4;                       // lanes per row
        for (int e = threadIdx.x; e < 16 * LPR; e += 256) {
            const int rr = e / LPR, f4 = 4 * (e % LPR), row = r0 + 16 * n + rr, ra = 16 * n + rr;
            if (row >= rows)
                continue;
            const float mr = fmaxf(fmaxf(ms[0][ra], ms[1][ra]), fmaxf(ms[2][ra], ms[3][ra]));
            const float ref = mr == -INFINITY ? 0.f : mr;
            float l = 0.f;
            floatx4 y = zero4();
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                l += ls[w][ra] * __builtin_amdgcn_exp2f((ms[w][ra] - ref) * a.c2);
                y += *reinterpret_cast<const floatx4*>(&red[w][rr][f4]);
            }
            if (a.nsplit == 1) {
                write_row<D>(a, b, h, row, f4, y, mr, l);
            } else {
                *reinterpret_cast<floatx4*>(part_row<D>(a, split, b, h, row) + f4) = y;
                if (f4 == 0) {
                    float* s = part_stat<D>(a, split, b, h, row);
                    s[0] = mr;
                    s[1] = l;
                }
            }
        }
        __syncthreads();
    }
}

// Joins the splits of a row, one wave a row: lane s forms split s's factor, then
// D / 4 lanes take the sums of every (256 / D)-th split, added in a fixed order.
// Latency: 4-5 us for few rows, 10 us for 16384 rows of 4 splits (a workgroup
// a row took 72).
constexpr int MAX_SPLITS = 64;

template <int D>
__global__ __launch_bounds__(256) void kv_attn_join_kernel(AttnArgs a)
{
    constexpr int LPR = D / 4, G = 64 / LPR;
    const int row = blockIdx.x * 4 + wave_id(), h = blockIdx.y, b = blockIdx.z;
    if (row >= a.rows)
        return;
    // the sequence's length, the splits' sums and their first parts are read
    // together (a row that is not there has a place, and nothing of it is used)
    const int lane = lane_id(), grp = lane / LPR, f4 = lane % LPR;
    const float2 stat = *reinterpret_cast<const float2*>(part_stat<D>(a, min(lane, a.nsplit - 1), b, h, row));
    const float* y = part_row<D>(a, 0, b, h, row) + 4 * f4;
    const int64_t next = part_floats((int64_t)a.B * a.c.H * a.rows, D);   // from one split to the next
    constexpr int U = 4;
    floatx4 first[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        first[u] = *reinterpret_cast<const floatx4*>(y + min(grp + G * u, a.nsplit - 1) * next);
    const Span sp(a.past, a.n_new, b, a.T);
    if (row >= sp.n * a.group)
        return;
    const float m = lane < a.nsplit ? stat.x : -INFINITY;
    float l = lane < a.nsplit ? stat.y : 0.f;
    float top = m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        top = fmaxf(top, __shfl_xor(top, off, 64));
    const float f = __builtin_amdgcn_exp2f((m - (top == -INFINITY ? 0.f : top)) * a.c2);
    l *= f;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        l += __shfl_xor(l, off, 64);
    floatx4 sum = zero4();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const float w = __shfl(f, min(grp + G * u, a.nsplit - 1), 64);
        if (grp + G * u < a.nsplit)
            sum += first[u] * w;
    }
#pragma unroll 4
    for (int s0 = G * U; s0 < a.nsplit; s0 += G) {
        const int s = s0 + grp, at = min(s, a.nsplit - 1);
        const floatx4 part = *reinterpret_cast<const floatx4*>(y + at * next);
        const float w = __shfl(f, at, 64);
        if (s < a.nsplit)
            sum += part * w;
    }
#pragma unroll
    for (int off = LPR; off < 64; off <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sum[j] += __shfl_xor(sum[j], off, 64);
    if (grp == 0)
        write_row<D>(a, b, h, row, 4 * f4, sum, top, l);
}

// ---- many rows: pieces of a prompt ------------------------------------------
//
// Bound by the matrix and vector units (4 D flops a score, and about 6 vector
// instructions with one exp), which two waves a SIMD (237 registers) overlap in
// part: 4096 tokens behind 12K, 16 / 4 heads of 128, take 478-484 us (1000 TFLOP/s; a
// library's large product reaches 1210).  Four waves of 32 rows each share every
// tile of 64 keys: the codes are converted once, on the way into LDS ([key][feature]
// and, for V, [feature][key]), two buffers deep, while the loads of the next
// tile are in flight.  64 rows a wave halve the LDS reads but leave one wave a SIMD:
// 939 us; eight waves in two halves, one multiplying while the other forms weights:
// 470, and 230 for 203 us where a head has 68 rows; LDS without bank conflicts: 472.
template <int D, bool PAGED>
__global__ __launch_bounds__(256, 2) void kv_attn_piece_kernel(AttnArgs a)
{
    constexpr int NR = 2, ROWS = 64 * NR, DT = D / 16, KP = D + 16, VP = 64 + 16;
    constexpr int KV = 64 * D / 16 / 256;   // 16-byte vectors of K, and of V, a thread stages
    __shared__ __align__(16) bf16 kt[2][64 * KP];
    __shared__ __align__(16) bf16 vt[2][D * VP];
    __shared__ int there[2][4];              // whether the page of each 16-key group is there
    __shared__ int bad[2];                   // border tile: values were taken out
    const int nbh = a.c.H * a.B;
    const int bh = blockIdx.x % nbh, h = bh % a.c.H, b = bh / a.c.H;
    const int unit = blockIdx.x / nbh, split = unit % a.nsplit;
    // rows of later tokens read more keys: the longest first, and in the second
    // half, which shares the CUs with the first, the shortest first
    const int rank = unit / a.nsplit, half = (a.row_tiles + 1) / 2;
    const int tile = rank < half ? a.row_tiles - 1 - rank : rank - half;
    const Span sp(a.past, a.n_new, b, a.T);
    const int rows = sp.n * a.group, r0 = tile * ROWS;
    if (r0 >= rows)
        return;
    const int r1 = min(rows, r0 + ROWS);
    const Range rg(a, sp, r0, r1, split, 1);
    const int wave = wave_id(), lane = lane_id(), t = lane & 15, g = lane >> 4, tid = threadIdx.x;
    const int shift = a.c.shift, P = 1 << shift, H = a.c.H;
    // product i = 2 s + u: rows 4 g + r are the keys 32 s + 8 g + 4 u + r
    auto key = [&](int i, int r) { return 32 * (i / 2) + 8 * g + 4 * (i % 2) + r; };

    Frag<bf16> q[NR][D / 32];
    RowState<D> st[NR];
    int pos[NR];
    const int w0 = r0 + 16 * NR * wave;      // this wave's rows
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const int row = w0 + 16 * n + t;
        load_q<D>(q[n], a, b, h, row, rows, [&](int s) { return 32 * s + 8 * g; });
        st[n].clear();
        pos[n] = row < rows ? sp.past + row / a.group : -1;
    }
    // staging: K vector v is key kk, features kf; V vector v is feature row vf, keys 16 (tid % 4)
    constexpr int KL = D / 16;               // lanes per key row
    const int kk = tid / KL, kf = 16 * (tid % KL), vf = tid / 4, vg = 16 * (tid % 4);
    // One page a tile: its number and scales are the wave's, but come through vector
    // loads, each used a tile after it is asked for.  A scalar load in flight would
    // make every wait for an LDS read a wait for memory (489 -> 475 us).
    int pk[KV], pv = -1, entry = -1;
    bool entry_in = false;
    auto pages = [&](int tl) {
        const int k = rg.k0 + 64 * tl;
        const bool in = tl < rg.last;
        if constexpr (PAGED) {
#pragma unroll
            for (int v = 0; v < KV; ++v)
                pk[v] = in ? page_of(a.c, b, (k + kk + 256 / KL * v) >> shift) : -1;
            pv = in ? page_of(a.c, b, (k + vg) >> shift) : -1;
        } else {
            int64_t at = b * a.c.table_stride + min(k >> shift, a.c.max_pages - 1);
            asm("" : "+v"(at));
            entry = a.c.table[at];
            entry_in = in && k >> shift < a.c.max_pages;
        }
    };
    const int k_lane = kk * D + kf, v_lane = vf * P + vg;
    u32x4 kr[KV], vr[KV];
    float ks[KV], vs;
    bool v_ok;
    auto load = [&](int tl) {
        const int k = rg.k0 + 64 * tl;
        if constexpr (!PAGED) {
            const int e = __builtin_amdgcn_readfirstlane(entry);
            pv = entry_in && e >= 0 && e < a.c.pages ? e : -1;
        }
        const int64_t ph = (int64_t)max(pv, 0) * H + h;
        if constexpr (PAGED) {
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                const int64_t kh = (int64_t)max(pk[v], 0) * H + h;
                kr[v] = *reinterpret_cast<const u32x4*>(a.c.k + (kh * P + ((k + kk + 256 / KL * v) & (P - 1))) * D + kf);
                ks[v] = a.c.ks[kh];
                vr[v] = *reinterpret_cast<const u32x4*>(a.c.v + (ph * D + vf + 64 * v) * P + ((k + vg) & (P - 1)));
            }
            vs = a.c.vs[ph];
        } else {
            const uint8_t* kp = a.c.k + (ph * P + (k & (P - 1))) * D;
            const uint8_t* vp = a.c.v + (ph * D * P + (k & (P - 1)));
            int none = 0;
            asm("" : "+v"(none));
            ks[0] = a.c.ks[ph + none];
            vs = a.c.vs[ph + none];
#pragma unroll
            for (int v = 0; v < KV; ++v) {
                kr[v] = *reinterpret_cast<const u32x4*>(kp + k_lane + 256 / KL * v * D);
                vr[v] = *reinterpret_cast<const u32x4*>(vp + v_lane + 64 * v * P);
                ks[v] = ks[0];
            }
        }
        v_ok = pv >= 0;
    };
    // whether rows [ra, rb) all see the whole tile from key k0 on
    auto whole_for = [&](int k0, int ra, int rb) {
        return k0 + 63 <= sp.past + ra / a.group && (a.window <= 0 || k0 > sp.past + (rb - 1) / a.group - a.window);
    };
    auto stage = [&](int tl, int buf) {
        bool any = false;
        const bool border = !v_ok || !whole_for(rg.k0 + 64 * tl, r0, r1);
        const float vuse = border ? finite_scale(vs) : vs;
#pragma unroll
        for (int v = 0; v < KV; ++v) {
            bf16* kp = &kt[buf][(kk + 256 / KL * v) * KP + kf];
            *reinterpret_cast<bf16x8*>(kp) = values8(kr[v][0], kr[v][1], ks[v]);
            *reinterpret_cast<bf16x8*>(kp + 8) = values8(kr[v][2], kr[v][3], ks[v]);
            if (border)
                any |= take_nonfinite(vr[v], vs);
            bf16* vp = &vt[buf][(vf + 64 * v) * VP + vg];
            *reinterpret_cast<bf16x8*>(vp) = values8(vr[v][0], vr[v][1], vuse);
            *reinterpret_cast<bf16x8*>(vp + 8) = values8(vr[v][2], vr[v][3], vuse);
        }
        if (PAGED && tid < 4)
            there[buf][tid] = v_ok;
        if (any)
            bad[buf] = tl;
    };
    if (tid < 2)
        bad[tid] = -1;
    __syncthreads();
    int tl = rg.first;
    bool ok = true;   // the page of the tile in LDS is there (one page a tile)
    if (tl < rg.last) {
        pages(tl);
        load(tl);
        pages(tl + 1);
        stage(tl, 0);
        ok = v_ok;
    }
    __syncthreads();
    for (int buf = 0; tl < rg.last; ++tl, buf ^= 1) {
        const int k0 = rg.k0 + 64 * tl;
        const bool more = tl + 1 < rg.last;
        if (more) {
            load(tl + 1);
            pages(tl + 2);
        }
        if (w0 < rows) {
            const bf16* kb = kt[buf];
            const bf16* vb = vt[buf];
            floatx4 x[NR][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    x[n][i] = zero4();
                const bf16* kp = kb + (32 * (i / 2) + 8 * (t >> 2) + 4 * (i % 2) + (t & 3)) * KP + 8 * g;
#pragma unroll
                for (int s = 0; s < D / 32; ++s) {
                    const Frag<bf16> kfr = frag(*reinterpret_cast<const bf16x8*>(kp + 32 * s));
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        x[n][i] = mma(kfr, q[n][s], x[n][i]);
                }
            }
            read_ahead<NR, 4 * (D / 32)>();
            const int w1 = min(rows, w0 + 16 * NR);
            unsigned groups = ok ? 15u : 0u;
            if constexpr (PAGED)
                groups = there[buf][0] | there[buf][1] << 1 | there[buf][2] << 2 | there[buf][3] << 3;
            const bool whole = groups == 15u && whole_for(k0, w0, w1);
            Seen seen[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                seen[n].hi = min(pos[n], rg.end - 1) - k0;
                seen[n].lo = a.window > 0 ? pos[n] - a.window + 1 - k0 : 0;
                seen[n].groups = groups;
            }
            auto vfrag = [&](int dt, int s) {
                return frag(*reinterpret_cast<const bf16x8*>(vb + (16 * dt + t) * VP + 32 * s + 8 * g));
            };
            attend<D, NR, true>(st, x, a.c2, whole, seen, vfrag, key);
            if (bad[buf] == tl)
                give_nonfinite<D, NR>(st, seen, [&](int k, int f, float& scale) {
                    const int64_t ph = (int64_t)max(page_of(a.c, b, (k0 + k) >> shift), 0) * H + h;
                    scale = a.c.vs[ph];
                    return *reinterpret_cast<const u32x2*>(a.c.v + (ph * D + f) * P + ((k0 + k) & (P - 1)));
                }, key);
        }
        if (more) {
            stage(tl + 1, buf ^ 1);
            ok = v_ok;
        }
        __syncthreads();
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
        const float l = quad_sum(st[n].l);
        const int row = w0 + 16 * n + t;
        if (row >= rows)
            continue;
        if (a.nsplit == 1) {
#pragma unroll
            for (int i = 0; i < DT; ++i)
                write_row<D>(a, b, h, row, 16 * i + 4 * g, st[n].acc[i], st[n].m, l);
        } else {
            float* y = part_row<D>(a, split, b, h, row);
#pragma unroll
            for (int i = 0; i < DT; ++i)
                *reinterpret_cast<floatx4*>(y + 16 * i + 4 * g) = st[n].acc[i];
            if (g == 0) {
                float* s = part_stat<D>(a, split, b, h, row);
                s[0] = st[n].m;
                s[1] = l;
            }
        }
    }
}

// ---- host ------------------------------------------------------------------

// How a call is cut: rows of a key/value head, tiles of them, splits of the keys.
struct Plan {
    int rows, row_tiles, nsplit;
    bool token;
};

Plan plan_of(const linrec_kv_cache* c, int B, int T, int Hq)
{
    Plan p;
    p.rows = T * (Hq / c->H);
    // Up to 64 rows the cache's bytes cost more than the products.
    p.token = p.rows <= 64;
    const int tile_rows = p.token ? (p.rows <= 16 ? 16 : 32) : 128;
    p.row_tiles = (p.rows + tile_rows - 1) / tile_rows;
    const int64_t blocks = (int64_t)B * c->H * p.row_tiles;
    const int64_t key_tiles = ((int64_t)c->max_pages * c->page + 63) / 64;
    // Splits bring the workgroups to at least 512, two a CU (of the token kernel with
    // two row tiles at D = 128, whose registers leave one a CU, that is two rounds);
    // whole splits overshoot that, up to 1022 (511 blocks in two).  Their number is
    // bounded by the table's capacity: one tile a wave (token kernel) or 8 tiles
    // (piece kernel) of a sequence that fills it; a shorter one's splits hold fewer,
    // down to 4 tiles (token kernel) or one.  Aiming at 512, 768, 1024, 2048, 4096
    // workgroups: 180, 194, 180, 182, 194 us at 32 sequences of 16K, 15.6, 19.2,
    // 20.8, 23.1, 23.1 at 16 windows of 2048.
    const int64_t want = (512 + blocks - 1) / blocks;
    const int64_t most = std::max<int64_t>(1, key_tiles / (p.token ? 4 : 8));
    p.nsplit = (int)std::min<int64_t>(std::min(want, most), MAX_SPLITS);
    return p;
}

template <int D, bool PAGED>
hipError_t launch_attn(const AttnArgs& a, bool token, hipStream_t s)
{
    if (token) {
        const dim3 grid(a.row_tiles * a.nsplit, a.c.H, a.B);
        if (a.rows <= 16)
            launch_kernel(kv_attn_token_kernel<D, 1, PAGED>, grid, dim3(256), s, a);
        else
            launch_kernel(kv_attn_token_kernel<D, 2, PAGED>, grid, dim3(256), s, a);
    } else {
        launch_kernel(kv_attn_piece_kernel<D, PAGED>, dim3(a.c.H * a.B * a.row_tiles * a.nsplit), dim3(256), s, a);
    }
    if (a.nsplit > 1)
        launch_kernel(kv_attn_join_kernel<D>, dim3((a.rows + 3) / 4, a.c.H, a.B), dim3(256), s, a);
    return hipGetLastError();
}

linrec_status check_attn(const linrec_kv_cache* cache, int32_t B, int32_t T, int32_t Hq)
{
    const linrec_status st = check_kv(cache, B, T);
    if (st != LINREC_OK)
        return st;
    // rows of the whole call are counted in 31 bits
    if (Hq < 1 || Hq > 65535 || Hq % cache->H || (int64_t)B * Hq * T > 0x7fffffff)
        return LINREC_E_SHAPE;
    return LINREC_OK;
}

}  // namespace
}  // namespace linrec

using namespace linrec;

extern "C" {

size_t linrec_kv_attn_workspace_bytes(const linrec_kv_cache* cache, int32_t B, int32_t T, int32_t Hq)
{
    if (check_attn(cache, B, T, Hq) != LINREC_OK || T == 0)
        return 0;
    const Plan p = plan_of(cache, B, T, Hq);
    return p.nsplit == 1 ? 0
                         : (size_t)p.nsplit * part_floats((int64_t)B * cache->H * p.rows, cache->D) * sizeof(float);
}

linrec_status linrec_kv_attn(linrec_ctx* ctx, const linrec_kv_cache* cache, int32_t B, int32_t T, int32_t Hq,
                             linrec_tensor q, const int32_t* past, const int32_t* n_new, float scale,
                             int32_t window, linrec_tensor o, float* lse, void* workspace, void* stream)
{
    linrec_status st;
    if ((st = check_attn(cache, B, T, Hq)) != LINREC_OK)
        return st;
    if (!isfinite(scale))
        return LINREC_E_SHAPE;
    if (T > 0) {
        if ((st = check_kv_ptrs(cache, B, past, n_new)) != LINREC_OK ||
            (st = check_view(q, B, Hq, T, cache->D, 2, false)) != LINREC_OK ||
            (st = check_view(o, B, Hq, T, cache->D, 2, true)) != LINREC_OK)
            return st;
        const Plan p = plan_of(cache, B, T, Hq);
        // a launch holds at most 2^32 - 1 threads along x
        if ((int64_t)B * cache->H * p.row_tiles * p.nsplit > 0xffffff)
            return LINREC_E_SHAPE;
        if (!aligned(lse, 4))
            return LINREC_E_ALIGN;
        if (linrec_kv_attn_workspace_bytes(cache, B, T, Hq) && (st = check_buffer(workspace)) != LINREC_OK)
            return st;
    }
    if ((st = check_ctx(ctx)) != LINREC_OK)
        return st;
    if (T == 0)
        return LINREC_OK;
    AttnArgs a{};
    a.c = kv_arg(cache);
    a.q = Act<const bf16>{(const bf16*)q.ptr, q.sb, q.sh, q.st};
    a.o = Act<bf16>{(bf16*)o.ptr, o.sb, o.sh, o.st};
    a.lse = lse;
    a.past = past;
    a.n_new = n_new;
    a.B = B;
    a.T = T;
    a.Hq = Hq;
    a.group = Hq / cache->H;
    a.window = window < LINREC_MAX_T ? window : 0;   // offsets within a window fit 31 bits
    // the products see q with the scale's sign; a factor of 0 would make
    // 0 * inf of hidden scores
    a.negate = scale < 0.f;
    a.c2 = fmaxf(fabsf(scale) * 1.4426950408889634f, 1e-30f);
    const Plan p = plan_of(cache, B, T, Hq);
    a.rows = p.rows;
    a.row_tiles = p.row_tiles;
    a.nsplit = p.nsplit;
    a.part = (float*)workspace;
    hipStream_t s = (hipStream_t)stream;
    LAUNCH(timed_launch(ctx, LINREC_KERNEL_KV_ATTN, s, [&] {
        if (cache->D == 128)
            return cache->page < 64 ? launch_attn<128, true>(a, p.token, s) : launch_attn<128, false>(a, p.token, s);
        return cache->page < 64 ? launch_attn<64, true>(a, p.token, s) : launch_attn<64, false>(a, p.token, s);
    }));
    return LINREC_OK;
}

}  // extern "C"
