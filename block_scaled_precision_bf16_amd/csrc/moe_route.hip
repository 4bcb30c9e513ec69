// moe_route.hip -- a router's choice of experts from its logits, and the logits'
// gradient (gfx950).
//
//   p = softmax(l) or 1 / (1 + e^-l), key = p + bias, the best groups, the `top`
//   best keys among them, w = p / sum p (on request) * scale
//   dl = p (dp - sum p dp) or dp p (1 - p), with
//   dp_j = (scale / s) (dw_j - sum_i dw_i p_i / s) for the chosen ones, plus the
//   scores' own gradient
//
// One wave per token; lane l holds the experts l NPL .. l NPL + NPL - 1, so that
// the lowest lane among equal keys, and there the first, is the lowest index.  The
// bytes (4 an expert) take less time than the instructions: the exponentials and
// `top` maxima over the wave bound it.
#include "device_math.h"
#include "launch_moe.h"
#include "wave.h"

namespace mxk {

constexpr int kRouteWaves = 4;

__device__ __forceinline__ float minus_inf(float) { return -__builtin_inff(); }
__device__ __forceinline__ double minus_inf(double) { return -__builtin_inf(); }

template <int NPL>
__device__ __forceinline__ void load_logits(const void *p, int64_t t, int E, int lane, int f32,
                                            float (&x)[NPL])
{
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        const int e = lane * NPL + i;
        x[i] = -__builtin_inff();
        if (e < E)
            x[i] = f32 ? static_cast<const float *>(p)[t * E + e]
                       : bf16_lo(static_cast<const uint16_t *>(p)[t * E + e]);
    }
}

__device__ __forceinline__ float exp_nonpos(float a) { return exp32_nonpos(a); }
__device__ __forceinline__ double exp_nonpos(double a) { return exp(a); }

// Scores of a token in type F: softmax (those of -Inf logits 0, all of them where
// every logit is) or sigmoid (q: 1 - p); NaN where they have no value.
template <class F, int NPL>
__device__ __forceinline__ void scores_of(const float (&x)[NPL], bool sigmoid, F (&p)[NPL], F (&q)[NPL])
{
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; i++) {
            const F z = (F)x[i], e = exp_nonpos(z < F(0) ? z : -z), r = F(1) / (F(1) + e);
            p[i] = z >= F(0) ? r : e * r;
            q[i] = z >= F(0) ? e * r : r;
            if (x[i] != x[i])
                p[i] = q[i] = (F)x[i];
        }
        return;
    }
    float m = x[0];
#pragma unroll
    for (int i = 1; i < NPL; i++)
        m = __builtin_fmaxf(m, x[i]);
    m = wave_max(m);
    F sum = F(0);
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        p[i] = m == -__builtin_inff() && x[i] == x[i] ? F(0) : exp_nonpos((F)x[i] - (F)m);
        sum += p[i];
    }
    sum = wave_sum(sum);
    const F inv = sum > F(0) ? F(1) / sum : sum;
#pragma unroll
    for (int i = 0; i < NPL; i++)
        p[i] *= inv;
}

// Key: float where the logits themselves give the order, double where scores are
// added to a bias or to each other.
template <int NPL, class Key>
__global__ __launch_bounds__(64 * kRouteWaves) void route_kernel(RouteArgs a)
{
    __shared__ Key keys[kRouteWaves][64 * NPL];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T)
        return;
    const Key low = minus_inf(Key(0));
    float x[NPL], pf[NPL];
    Key key[NPL];
    load_logits<NPL>(a.logits, t, a.E, lane, a.f32, x);
    bool nan = false;
    {
        Key p[NPL], q[NPL];
        scores_of<Key, NPL>(x, a.sigmoid != 0, p, q);
#pragma unroll
        for (int i = 0; i < NPL; i++) {
            const int e = lane * NPL + i;
            pf[i] = (float)p[i];
            key[i] = (Key)x[i];
            float b = 0.0f;
            if constexpr (sizeof(Key) == 8) {
                b = a.bias && e < a.E ? a.bias[e] : 0.0f;
                key[i] = p[i] + (Key)b;
            }
            nan = nan || (e < a.E && (pf[i] != pf[i] || key[i] != key[i]));
            if (x[i] == -__builtin_inff() || b == -__builtin_inff())
                key[i] = low;
            if (a.scores && e < a.E)
                a.scores[t * a.E + e] = pf[i];
        }
    }
    const bool bad = __builtin_amdgcn_ballot_w64(nan) != 0;

    if (a.groups > 1 && !bad) {
        const int S = a.E / a.groups;
#pragma unroll
        for (int i = 0; i < NPL; i++)
            keys[wave][lane * NPL + i] = key[i];
        __builtin_amdgcn_wave_barrier();
        // lane g: group g's score
        Key best = low, second = low;
        if (lane < a.groups)
            for (int j = 0; j < S; j++) {
                const Key k = keys[wave][lane * S + j];
                second = k > best ? best : max_of(second, k);
                best = max_of(best, k);
            }
        if (a.pair && second > low)
            best += second;
        int rank = 0;
        for (int g = 0; g < a.groups; g++) {
            const Key k = from_lane(best, g);
            rank += k > best || (k == best && g < lane) ? 1 : 0;
        }
        const uint64_t kept = __builtin_amdgcn_ballot_w64(lane < a.groups && rank < a.top_groups);
        // e / S for e, S <= 1024, by a reciprocal that is less than 2^-20 too large
        const uint32_t inv = (1u << 20) / (uint32_t)S + 1;
#pragma unroll
        for (int i = 0; i < NPL; i++) {
            const uint32_t g = ((uint32_t)(lane * NPL + i) * inv) >> 20;
            if (!((kept >> (g & 63)) & 1))
                key[i] = low;
        }
    }

    int chosen = -1;
    float w = 0.0f;
    for (int j = 0; j < a.top && !bad; j++) {
        Key best = key[0];
        float bp = pf[0];
        int bi = 0;
#pragma unroll
        for (int i = 1; i < NPL; i++) {
            const bool more = key[i] > best;
            best = more ? key[i] : best;
            bp = more ? pf[i] : bp;
            bi = more ? i : bi;
        }
        const Key m = wave_max(best);
        if (m == low)
            break;
        const int owner = __builtin_ctzll(__builtin_amdgcn_ballot_w64(best == m));
        const int e = __builtin_amdgcn_readlane(lane * NPL + bi, owner);
        const float p = from_lane(bp, owner);
#pragma unroll
        for (int i = 0; i < NPL; i++)
            key[i] = lane == owner && i == bi ? low : key[i];
        chosen = lane == j ? e : chosen;
        w = lane == j ? p : w;
    }
    if (a.renorm) {
        const float s = wave_sum(w);
        w = s > 0.0f ? w / s : 0.0f;
    }
    w *= a.scale;
    if (lane < a.top) {
        a.experts[t * a.top + lane] = chosen;
        a.weights[t * a.top + lane] = bad ? __builtin_nanf("") : w;
    }
}

template <int NPL>
__global__ __launch_bounds__(64 * kRouteWaves) void route_back_kernel(RouteBackArgs a)
{
    __shared__ float ps[kRouteWaves][64 * NPL];
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T)
        return;
    float x[NPL], p[NPL], q[NPL], dp[NPL];
    load_logits<NPL>(a.logits, t, a.E, lane, a.f32, x);
    scores_of<float, NPL>(x, a.sigmoid != 0, p, q);
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        const int e = lane * NPL + i;
        ps[wave][e] = p[i];
        dp[i] = a.dscores && e < a.E ? a.dscores[t * a.E + e] : 0.0f;
    }
    __builtin_amdgcn_wave_barrier();
    // lane j: the gradient of chosen slot j's p
    int e = -1;
    float d = 0.0f, pj = 0.0f;
    if (lane < a.top) {
        e = a.experts[t * a.top + lane];
        if (e >= 0 && e < a.E) {
            pj = ps[wave][e];
            d = a.scale * a.dweights[t * a.top + lane];
        }
    }
    // sum over the experts of p times their dp.  With normalised weights the
    // chosen ones' part is 0 (the weights do not change when all p grow alike), so
    // that experts that were not chosen get no gradient from rounding
    float all = 0.0f;
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NPL; i++)
            all += p[i] * dp[i];
        all = wave_sum(all);
    }
    if (a.renorm) {
        const float s = wave_sum(pj);
        const float c = wave_sum(d * pj);
        d = s > 0.0f ? (d - c / s) / s : 0.0f;
    } else if (!a.sigmoid) {
        all += wave_sum(d * pj);
    }
    for (int j = 0; j < a.top; j++) {
        const int ej = __builtin_amdgcn_readlane(e, j);
        const float dj = from_lane(d, j);
#pragma unroll
        for (int i = 0; i < NPL; i++)
            dp[i] += lane * NPL + i == ej ? dj : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NPL; i++) {
        const int k = lane * NPL + i;
        if (k >= a.E)
            continue;
        const float o = a.sigmoid ? dp[i] * (p[i] * q[i]) : p[i] * (dp[i] - all);
        if (a.f32)
            static_cast<float *>(a.dlogits)[t * a.E + k] = o;
        else
            static_cast<uint16_t *>(a.dlogits)[t * a.E + k] = (uint16_t)(bf16x2_rne(o, 0.0f) & 0xFFFFu);
    }
}

template <int NPL>
static void launch_npl(const RouteArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    if (a.bias || (a.pair && a.groups > 1))
        hipLaunchKernelGGL((route_kernel<NPL, double>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((route_kernel<NPL, float>), grid, block, 0, s, a);
}

hipError_t launch_route(const RouteArgs &a, hipStream_t s)
{
    if (a.E <= 64)
        launch_npl<1>(a, s);
    else if (a.E <= 128)
        launch_npl<2>(a, s);
    else if (a.E <= 256)
        launch_npl<4>(a, s);
    else if (a.E <= 512)
        launch_npl<8>(a, s);
    else
        launch_npl<16>(a, s);
    return hipGetLastError();
}

hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t s)
{
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), block(64 * kRouteWaves);
    if (a.E <= 64)
        hipLaunchKernelGGL(route_back_kernel<1>, grid, block, 0, s, a);
    else if (a.E <= 128)
        hipLaunchKernelGGL(route_back_kernel<2>, grid, block, 0, s, a);
    else if (a.E <= 256)
        hipLaunchKernelGGL(route_back_kernel<4>, grid, block, 0, s, a);
    else if (a.E <= 512)
        hipLaunchKernelGGL(route_back_kernel<8>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(route_back_kernel<16>, grid, block, 0, s, a);
    return hipGetLastError();
}

}  // namespace mxk
