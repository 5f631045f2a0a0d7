// route.cu -- routing to experts: the experts of each token from the router's
// logits, their weights, and the gradient of the logits.
//
//   score p_e = softmax(x)_e over the row, or sigmoid(x_e)
//   choice    the topk largest of x_e (no bias: the order of the scores), or of
//             p_e + bias_e, in falling order, ties to the lowest number; with
//             groups only from the `keep` groups whose two largest sum highest
//   weight    w_j = scale * p_j, or with renorm scale * p_j / sum of the chosen p
//
// A logit of minus infinity is never chosen; choices that nothing is left for
// are -1 and weigh 0.  A NaN or plus infinity is chosen before all else, and makes
// every weight of its row NaN.
//
// The order is that of 64-bit arithmetic.  Without bias and groups it is the
// order of the logits, which is exact.  Otherwise keys are formed in 32 bits and a
// row is done again in 64 where two keys that decide something are closer
// than their errors could reach: neighbours among the topk + 1 first of
// different logit or bias, or the last kept and the first dropped group.  (In
// 64 bits throughout, the exponentials alone cost more than reading the logits.)
// Errors: a sigmoid is off by less than 2^-21, e^(x - top) / sum by less than
// 2^-19 of the row's largest score (the difference, rounded, shifts it by
// |x - top| 2^-24 of itself, and y e^-y < 1), the sum with the bias by 2^-24 of
// itself; a group's sum by twice that.
//
// A warp takes a token.  The row is dealt out so that a group lies in 32 /
// (groups, up to a power of two) neighbouring lanes, V consecutive experts a
// lane: what is found by lane order is in the order of the experts' numbers.
// The chosen sit one in each of the first topk lanes.
#include "host.cuh"
#include "launch.h"
#include "route.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tg {

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kInf = __builtin_huge_valf();

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
    return v;
}

// A 32-bit key in the order of the value: 0 is below all, ~0 above all.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);           // -0 is 0
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}

struct RouteParams {
    int tokens, E, groups, keep, topk, per;      // per: experts to a group
    int lanes;                                   // lanes to a group (a power of two)
    int sigmoid, renorm;
    float scale;
    const void* logits;
    long long ldl;
    const float* bias;
    int* ids;
    float* weights;
    const float* dweights;
    void* dlogits;
    long long ldd;
};

// Two largest of a group's lanes, in all of them.
template <class F>
__device__ __forceinline__ void group_top2(F& a, F& b, int lanes) {
    for (int d = 1; d < lanes; d <<= 1) {
        const F a2 = __shfl_xor_sync(kAll, a, d), b2 = __shfl_xor_sync(kAll, b, d);
        const F lo = a < a2 ? a : a2;
        a = a < a2 ? a2 : a;
        b = b < b2 ? b2 : b;
        b = b < lo ? lo : b;
    }
}

// Score of a group from its two largest: of those that can be chosen.
template <class F>
__device__ __forceinline__ F group_score(F a, F b) {
    return b > static_cast<F>(-kInf) ? a + b : a;
}

// How many groups come before this lane's: higher ones, and equal ones of
// lower number.
template <class F>
__device__ __forceinline__ int group_rank(F score, int group, const RouteParams& p) {
    int before = 0;
    for (int g = 0; g < p.groups; ++g) {
        const F other = __shfl_sync(kAll, score, g * p.lanes);
        before += other > score || (other == score && g < group);
    }
    return before;
}

// A row in 64 bits: choices only.  `x` are the lane's logits, dead ones
// (minus infinity, or past the group's end) as -inf; all are below +inf.
template <int V>
__device__ __noinline__ int choose_exact(const RouteParams& p, const float (&x)[V], int first, int live, float top, int lane) {
    double s[V];
    double sum = 0.0;
    if (!p.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s[i] = x[i] > -kInf ? exp(static_cast<double>(x[i]) - top) : 0.0;
            sum += s[i];
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const double score = p.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(x[i]))) : s[i] / sum;
        s[i] = x[i] > -kInf ? score + (p.bias ? static_cast<double>(__ldg(p.bias + first + i)) : 0.0) : -kInf;
    }
    bool in = true;
    if (p.groups > 1) {
        double a = -kInf, b = -kInf;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const double lo = s[i] < a ? s[i] : a;
            a = s[i] > a ? s[i] : a;
            b = lo > b ? lo : b;
        }
        group_top2(a, b, p.lanes);
        in = group_rank(group_score(a, b), lane / p.lanes, p) < p.keep;
    }
    // without a bias the logits have the scores' order, and keep it where scores saturate
    if (!p.bias) {
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = x[i];
    }
    int mine = -1;
    uint64_t used = in ? 0u : ~0ull;
    for (int j = 0; j < p.topk; ++j) {
        double best = -kInf;
        int at = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!(used >> i & 1) && s[i] > best) { best = s[i]; at = i; }
        double m = best;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const double o = __shfl_xor_sync(kAll, m, d);
            m = o > m ? o : m;
        }
        if (!(m > -kInf)) break;
        const int win = __ffs(__ballot_sync(kAll, best == m)) - 1;
        const int e = __shfl_sync(kAll, first + at, win);
        if (lane == win) used |= 1ull << at;
        if (lane == j) mine = e;
    }
    return mine;
}

template <int V, class T>
__global__ void __launch_bounds__(256)
route_kernel(const RouteParams p) {
    const int lane = threadIdx.x & 31;
    const long long t = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
    const int group = lane / p.lanes, off = (lane % p.lanes) * V;
    const int first = group * p.per + off;                    // this lane's experts: first .. first + live - 1
    const int live = group < p.groups ? min(V, p.per - off) : 0;
    float x[V];
    bool bad = false;
    float top = -kInf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        x[i] = i < live ? to_float(row[first + i]) : -kInf;
        bad |= !(x[i] < kInf);
        top = fmaxf(top, x[i]);
    }
    const bool bad_row = __any_sync(kAll, bad);
    const bool keyed = p.bias != nullptr;                     // keys are scores, not logits
    const bool sums = !p.sigmoid && (keyed || p.groups > 1 || !p.renorm);
    float sum = 1.f;
    top = value_of(__reduce_max_sync(kAll, ordered(top)));
    if (sums) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += x[i] > -kInf ? expf(x[i] - top) : 0.f;
        sum = warp_sum(sum);
    }
    const float inv = 1.f / sum;
    uint32_t key[V];
    bool close = false;
    if (keyed || p.groups > 1) {
        float a = -kInf, b = -kInf, s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float score = bad_row ? 0.f : p.sigmoid ? 1.f / (1.f + expf(-x[i])) : expf(x[i] - top) * inv;
            s[i] = !(x[i] < kInf) ? kInf : x[i] == -kInf ? -kInf : keyed ? score + __ldg(p.bias + first + i) : score;
            const float lo = fminf(s[i], a);
            a = fmaxf(s[i], a);
            b = fmaxf(b, lo);
        }
        bool in = true;
        if (p.groups > 1) {
            group_top2(a, b, p.lanes);
            const float score = group < p.groups ? group_score(a, b) : -kInf;
            const int rank = group_rank(score, group, p);
            in = rank < p.keep;
            // the first of the dropped groups, the last of the kept ones
            const bool head = group < p.groups && lane % p.lanes == 0;
            const unsigned out_at = __ballot_sync(kAll, head && rank == p.keep);
            const unsigned in_at = __ballot_sync(kAll, head && rank == p.keep - 1);
            if (out_at && in_at) {
                const float hi = __shfl_sync(kAll, score, __ffs(in_at) - 1), lo = __shfl_sync(kAll, score, __ffs(out_at) - 1);
                close = lo > -kInf && hi - lo <= 2.f * route_slack(p.sigmoid ? 1.f : inv, fmaxf(fabsf(hi), fabsf(lo)));
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float v = keyed ? s[i] : x[i];
            key[i] = !in || x[i] == -kInf ? 0u : !(x[i] < kInf) ? ~0u : ordered(v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = x[i] == -kInf ? 0u : !(x[i] < kInf) ? ~0u : ordered(x[i]);
    }
    // the topk largest, and with keys that are rounded the next one
    const int picks = min(32, p.topk + (keyed ? 1 : 0));
    uint32_t best = 0;
    int at = 0;
    auto scan = [&] {
        best = 0;
        at = 0;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) { best = key[i]; at = i; }
    };
    scan();
    int mine = -1;                                            // lane j: the j-th choice, its key
    uint32_t mkey = 0;
    for (int j = 0; j < picks; ++j) {
        const uint32_t m = __reduce_max_sync(kAll, best);
        if (m == 0) break;
        const int win = __ffs(__ballot_sync(kAll, best == m)) - 1;
        const int e = __shfl_sync(kAll, first + at, win);
        if (lane == j) { mine = e; mkey = m; }
        if (lane == win) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == at) key[i] = 0;
            scan();
        }
    }
    float mx = mine >= 0 ? to_float(row[mine]) : -kInf;
    if (keyed && !bad_row) {
        // neighbours whose order the keys' rounding could have changed
        const float v = mkey ? value_of(mkey) : -kInf, next = __shfl_down_sync(kAll, v, 1);
        const float bias = mine >= 0 ? __ldg(p.bias + mine) : 0.f;
        const float nx = __shfl_down_sync(kAll, mx, 1), nb = __shfl_down_sync(kAll, bias, 1);
        const bool near = lane < 31 && next > -kInf && (mx != nx || bias != nb) &&
                          v - next <= route_slack(p.sigmoid ? 1.f : inv, fmaxf(fabsf(v), fabsf(next)));
        close = close || __any_sync(kAll, near) || p.topk == 32;
    }
    if (close && !bad_row) {
        mine = choose_exact<V>(p, x, first, live, top, lane);
        mx = mine >= 0 ? to_float(row[mine]) : -kInf;
    }
    if (lane >= p.topk) mine = -1;
    const bool has = mine >= 0;
    float w;
    if (p.renorm) {
        // the chosen scores over their sum, from their logarithms: no sum vanishes
        const float l = !has ? -kInf : p.sigmoid ? fminf(mx, 0.f) - log1pf(expf(-fabsf(mx))) : mx;
        const float lt = value_of(__reduce_max_sync(kAll, ordered(l)));
        w = has ? expf(l - lt) : 0.f;
        w /= warp_sum(w);
    } else {
        w = p.sigmoid ? 1.f / (1.f + expf(-mx)) : expf(mx - top) * inv;
    }
    w = bad_row ? __uint_as_float(0x7fc00000u) : has ? w * p.scale : 0.f;
    if (lane < p.topk) {
        p.ids[t * p.topk + lane] = mine;
        p.weights[t * p.topk + lane] = w;
    }
}

template <class T>
__device__ __forceinline__ T from_float(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (__is_same(T, __half)) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// With renorm, or of sigmoids, only the chosen logits matter; the softmax's
// other ones get -p_i sum_j g_j p_j.
template <class T>
__global__ void __launch_bounds__(256)
route_grad_kernel(const RouteParams p) {
    const int lane = threadIdx.x & 31;
    const long long t = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
    T* out = static_cast<T*>(p.dlogits) + t * p.ldd;
    int e = lane < p.topk ? __ldg(p.ids + t * p.topk + lane) : -1;
    if (e >= p.E) e = -1;
    const bool has = e >= 0;
    const float x = has ? to_float(row[e]) : -kInf;
    const float g = has ? __ldg(p.dweights + t * p.topk + lane) * p.scale : 0.f;
    float d;
    if (!p.sigmoid && !p.renorm) {
        float top = -kInf;
        bool nan = false;
        for (int i = lane; i < p.E; i += 32) {
            const float v = to_float(row[i]);
            top = fmaxf(top, v);
            nan |= v != v;
        }
        top = __any_sync(kAll, nan) ? __uint_as_float(0x7fc00000u) : value_of(__reduce_max_sync(kAll, ordered(top)));
        const float base = top == -kInf ? 0.f : top;
        float sum = 0.f;
        for (int i = lane; i < p.E; i += 32) sum += expf(to_float(row[i]) - base);
        sum = warp_sum(sum);
        const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        const float prob = has ? expf(x - base) * inv : 0.f;
        const float total = warp_sum(has ? g * prob : 0.f);
        for (int i = lane; i < p.E; i += 32) out[i] = from_float<T>(-total * (expf(to_float(row[i]) - base) * inv));
        d = prob * (g - total);
    } else {
        for (int i = lane; i < p.E; i += 32) out[i] = from_float<T>(0.f);
        const float rest = p.sigmoid ? 1.f / (1.f + expf(x)) : 1.f;          // 1 - sigmoid
        if (p.renorm) {
            const float l = !has ? -kInf : p.sigmoid ? fminf(x, 0.f) - log1pf(expf(-fabsf(x))) : x;
            const bool nan = __any_sync(kAll, has && !(x < kInf));
            const float lt = value_of(__reduce_max_sync(kAll, ordered(l)));
            float w = has ? expf(l - lt) : 0.f;
            w /= warp_sum(w);
            const float total = warp_sum(has ? g * w : 0.f);
            d = nan ? __uint_as_float(0x7fc00000u) : w * (g - total) * rest;
        } else {
            d = g * (1.f / (1.f + expf(-x))) * rest;
        }
    }
    __syncwarp();                                             // the row's other values are written
    if (has) out[e] = from_float<T>(d);
}

RouteParams params(const RouteArgs& a) {
    RouteParams p = {};
    p.tokens = static_cast<int>(a.tokens);
    p.E = a.E;
    p.groups = a.groups;
    p.keep = a.keep;
    p.topk = a.topk;
    p.per = a.E / a.groups;
    p.lanes = route_lanes(a.groups);
    p.sigmoid = a.sigmoid;
    p.renorm = a.renorm;
    p.scale = a.scale;
    p.logits = a.logits;
    p.ldl = a.ldl;
    p.bias = a.bias;
    p.ids = a.ids;
    p.weights = a.weights;
    p.dweights = a.dweights;
    p.dlogits = a.dlogits;
    p.ldd = a.ldd;
    return p;
}

template <class T>
void start(const RouteParams& p, cudaStream_t s) {
    const unsigned blocks = static_cast<unsigned>((p.tokens + 7ll) / 8);
    const int v = route_values(p.E, p.groups);
    if (v <= 1) route_kernel<1, T><<<blocks, 256, 0, s>>>(p);
    else if (v <= 2) route_kernel<2, T><<<blocks, 256, 0, s>>>(p);
    else if (v <= 4) route_kernel<4, T><<<blocks, 256, 0, s>>>(p);
    else if (v <= 8) route_kernel<8, T><<<blocks, 256, 0, s>>>(p);
    else if (v <= 16) route_kernel<16, T><<<blocks, 256, 0, s>>>(p);
    else if (v <= 32) route_kernel<32, T><<<blocks, 256, 0, s>>>(p);
    else route_kernel<64, T><<<blocks, 256, 0, s>>>(p);
}

}  // namespace

int launch_route(const RouteArgs& a) {
    if (!current_device(nullptr)) return kNoDevice;
    const RouteParams p = params(a);
    const cudaStream_t s = static_cast<cudaStream_t>(a.stream);
    if (a.type == 2) start<float>(p, s);
    else if (a.type == 1) start<__nv_bfloat16>(p, s);
    else start<__half>(p, s);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

int launch_route_grad(const RouteArgs& a) {
    if (!current_device(nullptr)) return kNoDevice;
    const RouteParams p = params(a);
    const cudaStream_t s = static_cast<cudaStream_t>(a.stream);
    const unsigned blocks = static_cast<unsigned>((p.tokens + 7ll) / 8);
    if (a.type == 2) route_grad_kernel<float><<<blocks, 256, 0, s>>>(p);
    else if (a.type == 1) route_grad_kernel<__nv_bfloat16><<<blocks, 256, 0, s>>>(p);
    else route_grad_kernel<__half><<<blocks, 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? kOk : kCudaError;
}

}  // namespace tg
