// moe_route.hip -- a router's choice of experts from its logits, and the logits'
// gradient (gfx950).
//
//   p = softmax(l) or 1 / (1 + e^-l), key = p + bias, the best groups, the `top`
//   best keys among them, w = p / sum p (on request) * scale
//   dl = p (dp - sum p dp) or dp p (1 - p), with
//   dp_j = (scale / s) (dw_j - sum_i dw_i p_i / s) for the chosen ones, plus the
//   scores' own gradient
//
// Many tokens of up to 256 experts: four tokens a wave, 16 lanes each; lane l of them
// holds the experts l NPL .. l NPL + NPL - 1, so that the lowest lane among equal keys,
// and there the first, is the lowest index.  Few tokens, more experts, and groups that
// are not a power of two of such lanes, take a wave per token.  The bytes (4 an expert)
// take less time than the instructions: the exponentials and `top` maxima bound it.
//
// Measured for 16384 tokens, 8 experts each: 256 experts by sigmoid, bias, 4 of 8
// groups 16.1 us (its 18 MB would take 3.4; 430 vector instructions a token, a
// third of them fp64; 65536 tokens 45 us), by softmax without bias or groups 10.4 us,
// 64 experts 5.8 us.  The gradient: 64 experts with dscores 6.4 us.
#include "bufio.h"
#include "device_math.h"
#include "launch_moe.h"
#include "wave.h"

namespace mxk {

constexpr int kRouteWaves = 4;

// NPL floats from element `at` on (0 past the descriptor's end; multiples of 4:
// groups of 4, wholly inside or outside).
template <int NPL>
__device__ __forceinline__ void load_floats(rsrc_t r, uint32_t at, bool fours, float (&x)[NPL])
{
    if (NPL % 4 == 0 && fours) {
#pragma unroll
        for (int i = 0; i + 3 < NPL; i += 4) {
            const uint4 v = buf_load16(r, 4 * (at + i));
            x[i] = f32_bits(v.x), x[i + 1] = f32_bits(v.y), x[i + 2] = f32_bits(v.z), x[i + 3] = f32_bits(v.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            x[i] = f32_bits(buf_load4(r, 4 * (at + i)));
    }
}

// Logits of `rows` tokens from t on: this lane's NPL from expert e0 of token
// t + row on, -Inf past the last expert and the last token.
template <int NPL>
__device__ __forceinline__ void load_logits(const void *p, int64_t t, int64_t rows, int row, int e0, int E,
                                            int f32, float (&x)[NPL])
{
    const int size = f32 ? 4 : 2;
    const rsrc_t r = make_rsrc(static_cast<const char *>(p) + t * E * size, 0, rows * E * size);
    const uint32_t at = (uint32_t)(row * E + e0);
    if (f32) {
        load_floats<NPL>(r, at, E % 4 == 0, x);
    } else if (NPL % 4 == 0 && E % 4 == 0) {   // rows of whole 8 bytes
#pragma unroll
        for (int i = 0; i + 3 < NPL; i += 4) {
            const uint2 v = buf_load8(r, 2 * (at + i));
            x[i] = bf16_lo(v.x), x[i + 1] = bf16_hi(v.x), x[i + 2] = bf16_lo(v.y), x[i + 3] = bf16_hi(v.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            x[i] = bf16_lo(buf_load2(r, 2 * (at + i)));
    }
#pragma unroll
    for (int i = 0; i < NPL; i++)
        x[i] = row < rows && e0 + i < E ? x[i] : -__builtin_inff();
}

// e^a for a <= 0 and 1 / d for 1 <= d <= 2 in the three arithmetics of the scores:
// float; double as far as the keys' fixed point needs it, off by less than 2^-36
// (Cody and Waite's reduction, the exponential's series to r^9, |r| <= ln(2) / 2;
// the hardware's reciprocal, measured good to 2^-24, and one Newton step); and double.
struct Quick {
    typedef double type;
    static __device__ __forceinline__ double exp_in_range(double c)
    {
        const double n = __builtin_rint(c * 1.44269504088896340736);
        double r = __builtin_fma(n, -0.693359375, c);              // 355/512
        r = __builtin_fma(n, 2.1219444005469058277e-4, r);         // ln 2 - 355/512
        double p = 1.0 / 362880.0;
        p = __builtin_fma(p, r, 1.0 / 40320.0);
        p = __builtin_fma(p, r, 1.0 / 5040.0);
        p = __builtin_fma(p, r, 1.0 / 720.0);
        p = __builtin_fma(p, r, 1.0 / 120.0);
        p = __builtin_fma(p, r, 1.0 / 24.0);
        p = __builtin_fma(p, r, 1.0 / 6.0);
        p = __builtin_fma(p, r, 0.5);
        p = __builtin_fma(p, r, 1.0);
        p = __builtin_fma(p, r, 1.0);
        return __builtin_ldexp(p, (int)n);
    }
    static __device__ __forceinline__ double exp_nonpos(double a)
    {
        const double p = exp_in_range(__builtin_fmax(a, -1100.0));    // 0 already
        return a != a ? a : p;
    }
    static __device__ __forceinline__ double rcp(double d)
    {
        const double r = __builtin_amdgcn_rcp(d);
        return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
    }
    // 1 / (1 + e^-x), of a number (in double no x needs the other form; past 110 it
    // is 1, and below -110 it rounds to 0 in fp32)
    static __device__ __forceinline__ double sigmoid(float x)
    {
        return rcp(1.0 + exp_in_range((double)__builtin_amdgcn_fmed3f(-x, -110.0f, 110.0f)));
    }
};
struct Single {
    typedef float type;
    static __device__ __forceinline__ float exp_nonpos(float a) { return exp32_nonpos(a); }
    static __device__ __forceinline__ float rcp(float d) { return rcp_1_2(d); }
};
struct Full {
    typedef double type;
    static __device__ __forceinline__ double exp_nonpos(double a) { return exp(a); }
    static __device__ __forceinline__ double rcp(double d) { return 1.0 / d; }
};

// Scores of a token in arithmetic A (ROW: one for each row of 16 lanes): softmax
// (those of -Inf logits 0, all of them where every logit is) or sigmoid (q: 1 - p);
// NaN where they have no value.
template <class A, int NPL, bool ROW>
__device__ __forceinline__ void scores_of(const float (&x)[NPL], bool sigmoid, typename A::type (&p)[NPL],
                                          typename A::type (&q)[NPL])
{
    typedef typename A::type F;
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; i++) {
            const F z = (F)x[i], e = A::exp_nonpos(z < F(0) ? z : -z), r = A::rcp(F(1) + e), s = e * r;
            const bool up = z >= F(0), nan = x[i] != x[i];
            p[i] = nan ? z : up ? r : s;
            q[i] = nan ? z : up ? s : r;
        }
        return;
    }
    float m = x[0];
#pragma unroll
    for (int i = 1; i < NPL; i++)
        m = __builtin_fmaxf(m, x[i]);
    m = ROW ? row_max(m) : wave_max(m);
    m = m == -__builtin_inff() ? 0.0f : m;   // then every exponential is 0 (or NaN)
    F sum = F(0);
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        p[i] = A::exp_nonpos((F)x[i] - (F)m);
        sum += p[i];
    }
    sum = ROW ? row_sum(sum) : wave_sum(sum);
    const F inv = sum > F(0) ? F(1) / sum : sum;
#pragma unroll
    for (int i = 0; i < NPL; i++)
        p[i] *= inv;
}

// Keys as unsigned numbers of the same order; 0 stands for none (a masked expert).
// Logits as keys: their bits, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float k)
{
    const uint32_t u = bits_f32(k + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
// Scores plus a bias: fixed point, 2^-28 apart where no |bias| passes 1 (in general
// 2^(e - 29) where 1 + |bias| < 2^e for all of them), between 1 and 2^30 + 1.  They
// are cut, and the scores are off by far less than a step, so that keys 2 apart are
// in order, and sums of two 3 apart.
constexpr uint32_t kFixedZero = (1u << 29) + 1u;   // a key of 0
struct Fixed {
    double mul;
    bool infinite;      // a bias of +Inf: 64 bits decide
};
template <int NPL, bool ROW>
__device__ __forceinline__ Fixed fixed_point(const float (&bias)[NPL])
{
    uint32_t all = 0u;
#pragma unroll
    for (int i = 0; i < NPL; i++)
        all = max_u32(all, bits_f32(bias[i]) & 0x7FFFFFFFu);
    all = ROW ? row_max(all) : wave_max(all);
    bool inf = false;
    if (__builtin_amdgcn_ballot_w64(all >= 0x7F800000u)) {   // without infinite ones and NaN
        all = 0u;
#pragma unroll
        for (int i = 0; i < NPL; i++) {
            const uint32_t b = bits_f32(bias[i]) & 0x7FFFFFFFu;
            inf |= bias[i] == __builtin_inff();
            all = b < 0x7F800000u ? max_u32(all, b) : all;
        }
        all = ROW ? row_max(all) : wave_max(all);
    }
    const float most = f32_bits(all);
    const int e = __builtin_amdgcn_frexp_exp(1.0 + (double)most);   // 1 + most < 2^e
    return Fixed{__builtin_ldexp(1.0, 29 - e), __builtin_amdgcn_ballot_w64(inf) != 0};
}
__device__ __forceinline__ uint32_t order_of(double score, float bias, const Fixed &f)
{
    return (uint32_t)__builtin_fma(score, f.mul, __builtin_fma((double)bias, f.mul, (double)kFixedZero));
}

// What a token's choice leaves: lane j's expert (-1: none) of slot j; sure: that
// keys off by their rounding give the same choice.
struct Choice {
    int expert;
    bool sure;
};

// A group's best key and second best, of two parts' best and second.
template <class K>
__device__ __forceinline__ void merge_two(K &best, K &second, K b, K s)
{
    const K low = best < b ? best : b;
    second = second > s ? second : s;
    second = second > low ? second : low;
    best = best > b ? best : b;
}

template <int CTRL>
__device__ __forceinline__ void merge_step(uint32_t &best, uint32_t &second)
{
    merge_two(best, second, dpp<CTRL>(0u, best), dpp<CTRL>(0u, second));
}
// Over groups of L lanes, a power of two up to 16.
__device__ __forceinline__ void merge_lanes(int L, uint32_t &best, uint32_t &second)
{
    if (L >= 2)
        merge_step<kDppXor1>(best, second);
    if (L >= 4)
        merge_step<kDppXor2>(best, second);
    if (L >= 8)
        merge_step<kDppHalfMirror>(best, second);
    if (L >= 16)
        merge_step<kDppMirror>(best, second);
}

// Score of a group whose two best keys (fixed point) are added; a missing one adds
// nothing.  0 without any.
__device__ __forceinline__ uint32_t pair_score(uint32_t first, uint32_t second)
{
    const uint32_t more = second != 0u ? second - kFixedZero : 0u;   // may be negative
    return first != 0u ? first + more + (1u << 30) : 0u;
}

// Rank of the score `mine` of group `group` among all; get(g) is group g's.  CERT:
// near tells whether another one is too close to be told apart.
template <bool CERT, class G>
__device__ __forceinline__ int group_rank(int groups, uint32_t mine, int group, G get, bool &near)
{
    int rank = 0, close = 0;
    for (int g = 0; g < groups; g++) {
        const uint32_t k = get(g);
        if constexpr (CERT) {          // equal ones are close: their order does not matter
            rank += k > mine ? 1 : 0;
            close += k - mine + 2u <= 4u ? 1 : 0;
        } else {
            rank += k > mine || (k == mine && g < group) ? 1 : 0;
        }
    }
    near = CERT && close > 1 && mine != 0u;
    return rank;
}

// The best groups: key = 0 in the others.  False where groups are too close to be
// told apart (CERT).  Where a group is a power of two of lanes, at most 16, these
// find its score among themselves; otherwise lane g reads group g's keys from LDS,
// one after the other.
template <int NPL, bool CERT>
__device__ __forceinline__ bool keep_groups(const RouteArgs &a, int lane, uint32_t *keys,
                                            uint32_t (&key)[NPL])
{
    const int S = a.E / a.groups, L = S / NPL;
    // e / S for e, S <= 1024, by a reciprocal that is less than 2^-20 too large
    const uint32_t inv = (1u << 20) / (uint32_t)S + 1;
    const bool lanes = S % NPL == 0 && (L & (L - 1)) == 0 && L <= 16;
    uint32_t first = 0u, second = 0u;
    int group = lane;                  // whose score this lane has
    if (lanes) {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            merge_two(first, second, key[i], 0u);
        merge_lanes(L, first, second);
        group = (int)(((uint32_t)(lane * NPL) * inv) >> 20);
    } else {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            keys[lane * NPL + i] = key[i];
        __builtin_amdgcn_wave_barrier();
        if (lane < a.groups)
            for (int j = 0; j < S; j++)
                merge_two(first, second, keys[lane * S + j], 0u);
    }
    const uint32_t score = a.pair ? pair_score(first, second) : first;
    bool near;
    const int rank = group_rank<CERT>(
        a.groups, score, group,
        [&](int g) { return (uint32_t)__builtin_amdgcn_readlane((int)score, lanes ? g * L : g); }, near);
    if (lanes) {
        const bool kept = rank < a.top_groups;
#pragma unroll
        for (int i = 0; i < NPL; i++)
            key[i] = kept ? key[i] : 0u;
    } else {
        const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && rank < a.top_groups);
#pragma unroll
        for (int i = 0; i < NPL; i++) {
            const uint32_t g = ((uint32_t)(lane * NPL + i) * inv) >> 20;
            key[i] = (kept >> (g & 63)) & 1 ? key[i] : 0u;
        }
    }
    return !CERT || __builtin_amdgcn_ballot_w64(group < a.groups && near) == 0;
}

// A lane's keys, largest first and of equal ones the lowest index first; the
// indices within the lane as bytes of `at`.
struct Sorted4 {
    uint32_t k0, k1, k2, k3, at;
};

__device__ __forceinline__ void in_order(uint32_t &a, uint32_t &b, uint32_t &i, uint32_t &j)
{
    const bool up = b > a;
    const uint32_t k = up ? b : a, n = up ? j : i;
    b = up ? a : b;
    j = up ? i : j;
    a = k;
    i = n;
}

template <int NPL>
__device__ __forceinline__ Sorted4 sort_lane(const uint32_t (&key)[NPL])
{
    Sorted4 s{key[0], 0u, 0u, 0u, 0u};
    uint32_t i0 = 0, i1 = 1, i2 = 2, i3 = 3;
    if constexpr (NPL >= 2) {
        s.k1 = key[1];
        in_order(s.k0, s.k1, i0, i1);
    }
    if constexpr (NPL == 4) {
        s.k2 = key[2];
        s.k3 = key[3];
        in_order(s.k1, s.k2, i1, i2);
        in_order(s.k2, s.k3, i2, i3);
        in_order(s.k0, s.k1, i0, i1);
        in_order(s.k1, s.k2, i1, i2);
        in_order(s.k0, s.k1, i0, i1);
    }
    s.at = i0 | i1 << 8 | i2 << 16 | i3 << 24;
    return s;
}

// The `top` best keys, a maximum over the wave for each.  With up to 4 keys a lane
// they are sorted first, so that a round looks at one and the lane that had it
// moves up; with more, a round looks at all of them.  CERT: `sure` tells whether
// each key is far enough from the next one.
template <int NPL, bool CERT>
__device__ __forceinline__ Choice choose32(const RouteArgs &a, int lane, uint32_t *keys,
                                           uint32_t (&key)[NPL])
{
    Choice c{-1, true};
    if (a.groups > 1)
        c.sure = keep_groups<NPL, CERT>(a, lane, keys, key);
    Sorted4 s{};
    if constexpr (NPL <= 4)
        s = sort_lane<NPL>(key);
    uint32_t got = 0u, extra = 0u;        // lane j: the key of slot j; the first one left over
    for (int j = 0;; j++) {
        uint32_t best, at;
        if constexpr (NPL <= 4) {
            best = s.k0;
            at = s.at & 0xFFu;
        } else {
            best = key[0];
            at = 0;
#pragma unroll
            for (int i = 1; i < NPL; i++) {
                const bool more = key[i] > best;
                best = more ? key[i] : best;
                at = more ? (uint32_t)i : at;
            }
        }
        const uint32_t m = wave_max(best);
        if (j == a.top) {
            extra = m;
            break;
        }
        if (m == 0u)
            break;
        const int owner = __builtin_ctzll(__builtin_amdgcn_ballot_w64(best == m));
        const int i = __builtin_amdgcn_readlane((int)at, owner);
        const bool slot = lane == j, mine = lane == owner;
        c.expert = slot ? owner * NPL + i : c.expert;
        if constexpr (CERT)
            got = slot ? m : got;
        else if (j + 1 == a.top)
            break;
        if constexpr (NPL <= 4) {
            s.k0 = mine ? s.k1 : s.k0;
            s.k1 = mine ? s.k2 : s.k1;
            s.k2 = mine ? s.k3 : s.k2;
            s.k3 = mine ? 0u : s.k3;
            s.at = mine ? s.at >> 8 : s.at;
        } else {
#pragma unroll
            for (int n = 0; n < NPL; n++)
                key[n] = mine && n == i ? 0u : key[n];
        }
    }
    if constexpr (CERT) {
        const uint32_t below = (uint32_t)__shfl_down((int)got, 1, 64);
        const bool close = lane < a.top && got != 0u && got - (lane == a.top - 1 ? extra : below) < 2u;
        c.sure = c.sure && __builtin_amdgcn_ballot_w64(close) == 0;
    }
    return c;
}

// The same in 64 bits, for the few tokens whose fp32 keys do not tell, by a whole
// wave: lane j's expert is slot j's.
template <int NPL>
__device__ __forceinline__ int choose64(const RouteArgs &a, int lane, double *keys, const float (&x)[NPL],
                                        const float (&bias)[NPL])
{
    const double low = -__builtin_inf();
    double key[NPL], q[NPL];
    scores_of<Full, NPL, false>(x, a.sigmoid != 0, key, q);
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        const bool masked = x[i] == -__builtin_inff() || bias[i] == -__builtin_inff();
        key[i] = masked ? low : key[i] + (double)bias[i];
    }
    if (a.groups > 1) {
        const int S = a.E / a.groups;
#pragma unroll
        for (int i = 0; i < NPL; i++)
            keys[lane * NPL + i] = key[i];
        __builtin_amdgcn_wave_barrier();
        double best = low, second = low;
        if (lane < a.groups)
            for (int j = 0; j < S; j++)
                merge_two(best, second, keys[lane * S + j], low);
        if (a.pair && second > low)
            best += second;
        int rank = 0;
        for (int g = 0; g < a.groups; g++) {
            const double k = from_lane(best, g);
            rank += k > best || (k == best && g < lane) ? 1 : 0;
        }
        const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && rank < a.top_groups);
#pragma unroll
        for (int i = 0; i < NPL; i++)
            if (!((kept >> (((lane * NPL + i) / S) & 63)) & 1))
                key[i] = low;
    }
    int expert = -1;
    for (int j = 0; j < a.top; j++) {
        double best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < NPL; i++) {
            const bool more = key[i] > best;
            best = more ? key[i] : best;
            at = more ? i : at;
        }
        const double m = wave_max(best);
        if (m == low)
            break;
        const int owner = __builtin_ctzll(__builtin_amdgcn_ballot_w64(best == m));
        const int i = __builtin_amdgcn_readlane(at, owner);
        expert = lane == j ? owner * NPL + i : expert;
#pragma unroll
        for (int n = 0; n < NPL; n++)
            key[n] = lane == owner && n == i ? low : key[n];
    }
    return expert;
}

// This lane's keys and scores (fp32) of a token, and whether an unmasked one is NaN.
// VALUE: keys are scores plus a bias, or a group's two are added; otherwise the
// logits give the order.  Such keys are compared in fixed point first, and only where
// two of those that decide are within its steps of each other (about one token in
// 10^5, and those with equal keys) once more in 64 bits.
template <int NPL, bool VALUE, bool ROW>
__device__ __forceinline__ bool keys_of(const RouteArgs &a, const float (&x)[NPL], const float (&bias)[NPL],
                                        float (&p)[NPL], uint32_t (&key)[NPL], bool &infinite)
{
    bool nan = false;
    infinite = false;
    if constexpr (VALUE) {
        const Fixed f = fixed_point<NPL, ROW>(bias);
        infinite = f.infinite;
        double s[NPL], q[NPL];
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < NPL; i++) {
                s[i] = Quick::sigmoid(x[i]);
                p[i] = x[i] != x[i] ? x[i] : (float)s[i];
            }
        } else {
            scores_of<Quick, NPL, ROW>(x, false, s, q);
#pragma unroll
            for (int i = 0; i < NPL; i++)
                p[i] = (float)s[i];
        }
#pragma unroll
        for (int i = 0; i < NPL; i++) {
            const bool masked = x[i] == -__builtin_inff() || bias[i] == -__builtin_inff();
            key[i] = masked ? 0u : order_of(s[i], bias[i], f);
            nan |= !masked & __builtin_isunordered(p[i], bias[i]);
        }
    } else {
        float q[NPL];
        scores_of<Single, NPL, ROW>(x, a.sigmoid != 0, p, q);
#pragma unroll
        for (int i = 0; i < NPL; i++) {
            const bool masked = x[i] == -__builtin_inff();
            key[i] = masked ? 0u : order_of(x[i]);
            nan |= !masked & ((p[i] != p[i]) | (x[i] != x[i]));
        }
    }
    return nan;
}

template <int NPL, bool VALUE>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a)
{
    __shared__ double lds[kRouteWaves][64 * NPL];
    __shared__ float ps[kRouteWaves][64 * NPL];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T)
        return;
    float x[NPL], p[NPL], bias[NPL];
    load_logits<NPL>(a.logits, t, 1, 0, lane * NPL, a.E, a.f32, x);
    if (VALUE && a.bias)
        load_floats<NPL>(make_rsrc(a.bias, 0, 4 * a.E), lane * NPL, a.E % 4 == 0, bias);
    else
        for (int i = 0; i < NPL; i++)
            bias[i] = 0.0f;
    uint32_t key[NPL];
    bool infinite;
    const bool nan = keys_of<NPL, VALUE, false>(a, x, bias, p, key, infinite);
#pragma unroll
    for (int i = 0; i < NPL; i++)
        ps[wave][lane * NPL + i] = p[i];
    if (a.scores) {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            if (lane * NPL + i < a.E)
                a.scores[t * a.E + lane * NPL + i] = p[i];
    }
    const bool bad = __builtin_amdgcn_ballot_w64(nan) != 0;
    int expert = -1;
    if (!bad) {
        const Choice c = choose32<NPL, VALUE>(a, lane, reinterpret_cast<uint32_t *>(lds[wave]), key);
        expert = c.expert;
        if (VALUE && (infinite || !c.sure))
            expert = choose64<NPL>(a, lane, lds[wave], x, bias);
    }
    __builtin_amdgcn_wave_barrier();
    float w = expert >= 0 ? ps[wave][expert] : 0.0f;
    if (a.renorm) {
        const float s = wave_sum(w);
        w = s > 0.0f ? w / s : 0.0f;
    }
    w *= a.scale;
    if (lane < a.top) {
        a.experts[t * a.top + lane] = expert;
        a.weights[t * a.top + lane] = bad ? __builtin_nanf("") : w;
    }
}

// ---- four tokens a wave -----------------------------------------------------

// Whether 16 lanes of NPL experts find the groups' scores among themselves.
__host__ __device__ inline bool groups_of_lanes(int E, int groups, int npl)
{
    const int S = E / groups, L = S / npl;
    return groups == 1 || (S % npl == 0 && (L & (L - 1)) == 0 && L <= 16);
}

// As keep_groups, for the rows of 16 lanes; the return value is the row's.
template <int NPL, bool CERT>
__device__ __forceinline__ bool keep_groups16(const RouteArgs &a, int lane, uint32_t (&key)[NPL])
{
    const int L = a.E / a.groups / NPL, group = (lane & 15) / L;   // L a power of two
    uint32_t first = 0u, second = 0u;
#pragma unroll
    for (int i = 0; i < NPL; i++)
        merge_two(first, second, key[i], 0u);
    merge_lanes(L, first, second);
    const uint32_t score = a.pair ? pair_score(first, second) : first;
    bool near;
    const int rank = group_rank<CERT>(
        a.groups, score, group,
        [&](int g) { return (uint32_t)__shfl((int)score, (lane & 48) + g * L, 64); }, near);
    const bool kept = rank < a.top_groups;
#pragma unroll
    for (int i = 0; i < NPL; i++)
        key[i] = kept ? key[i] : 0u;
    if constexpr (!CERT)
        return true;
    const uint64_t m = __builtin_amdgcn_ballot_w64(group < a.groups && near);
    return ((m >> (lane & 48)) & 0xFFFF) == 0;
}

template <int NPL, bool VALUE>
__global__ __launch_bounds__(64 * kRouteWaves) void route16_kernel(RouteArgs a)
{
    constexpr int LISTS = (NPL + 3) / 4, PER = NPL < 4 ? NPL : 4, WIDE = (NPL + 3) / 4;
    __shared__ float ps[kRouteWaves][4][16 * NPL];
    __shared__ uint2 found[kRouteWaves][4][65];   // expert and key of each slot, and the next key
    __shared__ double lds[VALUE ? kRouteWaves : 1][VALUE ? 64 * WIDE : 1];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int row = lane >> 4, l = lane & 15;
    const int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * 4;
    if (t0 >= a.T)
        return;
    const int64_t rows = a.T - t0 < 4 ? a.T - t0 : 4;
    float x[NPL], p[NPL], bias[NPL];
    load_logits<NPL>(a.logits, t0, rows, row, l * NPL, a.E, a.f32, x);
    if (VALUE && a.bias)
        load_floats<NPL>(make_rsrc(a.bias, 0, 4 * a.E), l * NPL, a.E % 4 == 0, bias);
    else
        for (int i = 0; i < NPL; i++)
            bias[i] = 0.0f;
    uint32_t key[NPL];
    bool infinite;
    const bool nan = keys_of<NPL, VALUE, true>(a, x, bias, p, key, infinite);
#pragma unroll
    for (int i = 0; i < NPL; i++)
        ps[wave][row][l * NPL + i] = p[i];
    if (a.scores && row < rows) {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            if (l * NPL + i < a.E)
                a.scores[(t0 + row) * a.E + l * NPL + i] = p[i];
    }
    const bool bad = ((__builtin_amdgcn_ballot_w64(nan) >> (lane & 48)) & 0xFFFF) != 0;
#pragma unroll
    for (int i = 0; i < NPL; i++)
        key[i] = bad ? 0u : key[i];
    bool sure = !infinite;
    if (a.groups > 1)
        sure = sure & keep_groups16<NPL, VALUE>(a, lane, key);

    // each lane's keys as sorted lists of up to 4; a round takes the largest head
    // of the row's lists, the first among equal ones, and moves that list up
    Sorted4 list[LISTS];
#pragma unroll
    for (int c = 0; c < LISTS; c++) {
        uint32_t part[PER];
#pragma unroll
        for (int i = 0; i < PER; i++)
            part[i] = key[c * 4 + i];
        list[c] = sort_lane<PER>(part);
        list[c].at += 0x04040404u * c;
    }
    const int rounds = a.top + (VALUE ? 1 : 0);
    int n = 0;
    for (int j = 0; j < rounds; j++) {
        uint32_t best = list[0].k0;
#pragma unroll
        for (int c = 1; c < LISTS; c++)
            best = max_u32(best, list[c].k0);
        const uint32_t m = row_max(best);
        if (__builtin_amdgcn_ballot_w64(m != 0u) == 0)
            break;
        const uint32_t who = (uint32_t)(__builtin_amdgcn_ballot_w64(best == m) >> (lane & 48));
        const bool mine = m != 0u && (int)__builtin_ctz(who | 0x10000u) == l;
        n += m != 0u ? 1 : 0;
        uint32_t at = 0u;
        bool left = mine;              // the first of its lists that has the key
#pragma unroll
        for (int c = 0; c < LISTS; c++) {
            const bool up = left && list[c].k0 == m;
            left = left && !up;
            at = up ? list[c].at : at;
            list[c].k0 = up ? list[c].k1 : list[c].k0;
            list[c].k1 = up ? list[c].k2 : list[c].k1;
            list[c].k2 = up ? list[c].k3 : list[c].k2;
            list[c].k3 = up ? 0u : list[c].k3;
            list[c].at = up ? list[c].at >> 8 : list[c].at;
        }
        if (mine)
            found[wave][row][j] = make_uint2((uint32_t)(l * NPL) + (at & 0xFFu), m);
    }
    __builtin_amdgcn_wave_barrier();
    if constexpr (VALUE) {
        bool close = false;
        for (int s = l; s < a.top && s < n; s += 16) {
            const uint32_t next = s + 1 < n ? found[wave][row][s + 1].y : 0u;
            close |= found[wave][row][s].y - next < 2u;
        }
        uint64_t again = __builtin_amdgcn_ballot_w64(!bad && (close || !sure) && row < rows);
        while (again) {
            // the wave takes this row's token alone, in 64 bits
            const int r = __builtin_ctzll(again) >> 4;
            again &= ~(0xFFFFull << (16 * r));
            float xw[WIDE], bw[WIDE];
            load_logits<WIDE>(a.logits, t0 + r, 1, 0, lane * WIDE, a.E, a.f32, xw);
            if (a.bias)
                load_floats<WIDE>(make_rsrc(a.bias, 0, 4 * a.E), lane * WIDE, a.E % 4 == 0, bw);
            else
                for (int i = 0; i < WIDE; i++)
                    bw[i] = 0.0f;
            const int e = choose64<WIDE>(a, lane, lds[wave], xw, bw);
            __builtin_amdgcn_wave_barrier();
            if (lane < a.top)
                found[wave][r][lane].x = (uint32_t)e;
            const int count = __builtin_popcountll(__builtin_amdgcn_ballot_w64(e >= 0));
            n = row == r ? count : n;
            __builtin_amdgcn_wave_barrier();
        }
    }
    float sum = 0.0f;
    if (a.renorm) {
        for (int s = l; s < a.top && s < n; s += 16)
            sum += ps[wave][row][found[wave][row][s].x];
        sum = row_sum(sum);
    }
    if (row >= rows)
        return;
    for (int s = l; s < a.top; s += 16) {
        const int64_t o = (t0 + row) * a.top + s;
        const int e = s < n ? (int)found[wave][row][s].x : -1;
        float w = e >= 0 ? ps[wave][row][e] : 0.0f;
        if (a.renorm)
            w = sum > 0.0f ? w / sum : 0.0f;
        a.experts[o] = e;
        a.weights[o] = bad ? __builtin_nanf("") : w * a.scale;
    }
}

// ---- the logits' gradient -------------------------------------------------------

// ROW: four tokens a wave, 16 lanes each; otherwise one.
template <int NPL, bool ROW>
__global__ __launch_bounds__(64 * kRouteWaves) void route_back_kernel(RouteBackArgs a)
{
    constexpr int TOKENS = ROW ? 4 : 1, LANES = 64 / TOKENS;
    __shared__ float ps[kRouteWaves][TOKENS][LANES * NPL];
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int row = ROW ? lane >> 4 : 0, l = lane & (LANES - 1);
    const int64_t t0 = ((int64_t)blockIdx.x * kRouteWaves + wave) * TOKENS;
    if (t0 >= a.T)
        return;
    const int64_t rows = a.T - t0 < TOKENS ? a.T - t0 : TOKENS, t = t0 + row;
    const auto sum_of = [](auto v) { return ROW ? row_sum(v) : wave_sum(v); };
    float x[NPL], p[NPL], q[NPL], dp[NPL];
    load_logits<NPL>(a.logits, t0, rows, row, l * NPL, a.E, a.f32, x);
    if (a.dscores)
        load_floats<NPL>(make_rsrc(a.dscores + t0 * a.E, 0, 4 * rows * a.E), row * a.E + l * NPL,
                         a.E % 4 == 0, dp);
    scores_of<Single, NPL, ROW>(x, a.sigmoid != 0, p, q);
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        ps[wave][row][l * NPL + i] = p[i];
        // (a masked expert's score has no gradient, whatever stands in its place)
        dp[i] = a.dscores && x[i] != -__builtin_inff() ? dp[i] : 0.0f;
    }
    __builtin_amdgcn_wave_barrier();
    // sum over the experts of p times their dp.  With normalised weights the
    // chosen ones' part is 0 (the weights do not change when all p grow alike), so
    // that experts that were not chosen get no gradient from rounding
    float all = 0.0f;
    if (!a.sigmoid && a.dscores) {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            all += p[i] * dp[i];
        all = sum_of(all);
    }
    // slots s0 + l: the chosen p's sum, and that of p times its gradient d = scale dw.
    // d sp - sd cancels, to 0 where one choice is live: 64 bits hold each product
    // exactly, and 1 / sp of any fp32 numbers
    double sp = 0.0, sd = 0.0;
    for (int s = l; s < a.top; s += LANES) {
        const int e = row < rows ? a.experts[t * a.top + s] : -1;
        const bool is = e >= 0 && e < a.E;
        const float pj = is ? ps[wave][row][e] : 0.0f, d = is ? a.scale * a.dweights[t * a.top + s] : 0.0f;
        sp += (double)pj;
        sd = __builtin_fma((double)d, (double)pj, sd);
    }
    sd = sum_of(sd);
    double inv = 0.0;
    if (a.renorm) {
        sp = sum_of(sp);
        inv = sp > 0.0 ? Quick::rcp(sp) : 0.0;
    } else if (!a.sigmoid) {
        all += (float)sd;
    }
    // with normalised weights all gradients are taken times p from here on: the chosen
    // ones' part, which the loop adds, is w (d - sum w d) with w = p / sp
    if (a.renorm) {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            dp[i] = p[i] * (dp[i] - all);
    }
    for (int s0 = 0; s0 < a.top; s0 += LANES) {
        const int s = s0 + l;
        const int e = row < rows && s < a.top ? a.experts[t * a.top + s] : -1;
        const bool is = e >= 0 && e < a.E;
        float d = is ? a.scale * a.dweights[t * a.top + s] : 0.0f;
        if (a.renorm)
            d = (float)((is ? (double)ps[wave][row][e] : 0.0) * inv) *
                (float)(__builtin_fma((double)d, sp, -sd) * inv);
        const int n = a.top - s0 < LANES ? a.top - s0 : LANES;
        for (int j = 0; j < n; j++) {
            const int ej = __shfl(e, (lane & ~(LANES - 1)) + j, 64);
            const float dj = __shfl(d, (lane & ~(LANES - 1)) + j, 64);
#pragma unroll
            for (int i = 0; i < NPL; i++)
                dp[i] += l * NPL + i == ej ? dj : 0.0f;
        }
    }
    if (row >= rows)
        return;
    float o[NPL];
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        if (a.sigmoid)
            o[i] = dp[i] * (a.renorm ? q[i] : p[i] * q[i]);
        else
            o[i] = a.renorm ? dp[i] : p[i] * (dp[i] - all);
    }
    if (NPL % 4 == 0 && a.E % 4 == 0) {
#pragma unroll
        for (int i = 0; i + 3 < NPL; i += 4) {
            const int64_t at = t * a.E + l * NPL + i;
            if (l * NPL + i >= a.E)
                continue;
            if (a.f32)
                *reinterpret_cast<float4 *>(static_cast<float *>(a.dlogits) + at) =
                    make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            else
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.dlogits) + at) =
                    make_uint2(bf16x2_rne(o[i], o[i + 1]), bf16x2_rne(o[i + 2], o[i + 3]));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        const int e = l * NPL + i;
        if (e >= a.E)
            continue;
        if (a.f32)
            static_cast<float *>(a.dlogits)[t * a.E + e] = o[i];
        else
            static_cast<uint16_t *>(a.dlogits)[t * a.E + e] = (uint16_t)(bf16x2_rne(o[i], 0.0f) & 0xFFFFu);
    }
}

template <int NPL>
static void launch_npl(const RouteArgs &a, bool value, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    if (value)
        hipLaunchKernelGGL((route_kernel<NPL, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<NPL, false>), grid, block, 0, s, a);
}

template <int NPL>
static void launch_npl16(const RouteArgs &a, bool value, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + 4 * kRouteWaves - 1) / (4 * kRouteWaves))), block(64 * kRouteWaves);
    if (value)
        hipLaunchKernelGGL((route16_kernel<NPL, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((route16_kernel<NPL, false>), grid, block, 0, s, a);
}

// Tokens up to which a wave takes one alone, for its shorter chain of steps; more fill
// the chip's 1024 SIMDs with four to a wave.  In a graph, one and four to a wave, us:
//                             32 tokens   2048        3000        4096        6000        16384
//   256, sigmoid, bias, groups 4.5  7.8    5.3  8.0    6.1  8.1    7.0  8.2    8.9 10.1   18.2 15.2
//   256, softmax               3.8  5.7    4.3  5.8    4.9  5.9    5.6  6.0    6.8  6.8   13.2  9.9
//   64, softmax                2.8  3.2    3.1  3.5    3.3  3.5    3.6  3.6    4.3  3.7    7.5  4.7
//   8, softmax                 2.5  2.7    2.8  2.9    3.0  3.0    3.2  3.0    3.7  3.1    6.2  3.5
// They cross near 3000 tokens of 8 experts and 8000 of 256 by sigmoid; the one number lies
// below all of that, which costs 256 experts up to 2 us between 2049 and 8000 tokens.  The
// gradient of 64: 32 tokens 3.4 and 3.9, 4096 4.2 and 4.1, 16384 9.4 and 5.6; of 256 with a
// wave to each always (4096 5.5 and 6.9, 16384 13.7 and 13.6, 65536 42.5 and 37.3).
constexpr int64_t kFewTokens = 2048;

hipError_t launch_route(const RouteArgs &a, hipStream_t s)
{
    const bool value = a.bias || (a.pair && a.groups > 1);
    const int npl = a.E <= 16 ? 1 : a.E <= 32 ? 2 : a.E <= 64 ? 4 : a.E <= 128 ? 8 : 16;
    if (a.E <= 256 && a.T > kFewTokens && groups_of_lanes(a.E, a.groups, npl)) {
        switch (npl) {
        case 1: launch_npl16<1>(a, value, s); break;
        case 2: launch_npl16<2>(a, value, s); break;
        case 4: launch_npl16<4>(a, value, s); break;
        case 8: launch_npl16<8>(a, value, s); break;
        default: launch_npl16<16>(a, value, s);
        }
    } else if (a.E <= 64) {
        launch_npl<1>(a, value, s);
    } else if (a.E <= 128) {
        launch_npl<2>(a, value, s);
    } else if (a.E <= 256) {
        launch_npl<4>(a, value, s);
    } else if (a.E <= 512) {
        launch_npl<8>(a, value, s);
    } else {
        launch_npl<16>(a, value, s);
    }
    return hipGetLastError();
}

template <int NPL, bool ROW>
static void launch_back(const RouteBackArgs &a, hipStream_t s)
{
    const int64_t per = kRouteWaves * (ROW ? 4 : 1);
    hipLaunchKernelGGL((route_back_kernel<NPL, ROW>), dim3((unsigned)((a.T + per - 1) / per)),
                       dim3(64 * kRouteWaves), 0, s, a);
}

hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t s)
{
    const bool few = a.T <= kFewTokens;
    if (a.E <= 64 && few)
        launch_back<1, false>(a, s);
    else if (a.E <= 128 && few)
        launch_back<2, false>(a, s);
    else if (a.E <= 16)
        launch_back<1, true>(a, s);
    else if (a.E <= 32)
        launch_back<2, true>(a, s);
    else if (a.E <= 64)
        launch_back<4, true>(a, s);
    else if (a.E <= 128)
        launch_back<8, true>(a, s);
    else if (a.E <= 256)
        launch_back<4, false>(a, s);
    else if (a.E <= 512)
        launch_back<8, false>(a, s);
    else
        launch_back<16, false>(a, s);
    return hipGetLastError();
}

}  // namespace mxk
