// route.cu -- routing to experts: the experts of each token from the router's
// logits, their weights, and the gradient of the logits.
//
//   score p_e = softmax(x)_e over the row, or sigmoid(x_e)
//   choice    the topk largest of x_e (no bias: the order of the scores), or of
//             p_e + bias_e, in falling order, ties to the lowest number; with
//             groups only from the `keep` groups whose two largest sum highest
//   weight    w_j = scale * p_j, or with renorm scale * p_j / sum of the chosen p
//
// A logit or a bias of minus infinity is never chosen; choices that nothing is left
// for are -1 and weigh 0.  A NaN or plus infinity is chosen before all else, and makes
// every weight of its row NaN.
//
// The order is that of 64-bit arithmetic.  Keys are 32-bit: a value in the order of
// its bits, the lowest ones given to the lane's number of the expert, so that one
// comparison moves both.  A row is done again in 64 bits where two keys that decide
// something are closer than their errors could reach: neighbours among the topk +
// 1 first of different logit or bias, where the last two of those are a tie any
// further one of different logit or bias, or the last kept and the first dropped
// group.  (In 64 bits throughout, the exponentials alone cost more than reading
// the logits.)  Errors: a key that is a logit has lost its lowest bits only, so that
// equal ones are in question; 16-bit logits lose nothing.  An exponential is off by
// (2 + 1.5 |v|) 2^-23 of itself; a sigmoid by less than 2^-22 then (s (1 - s) |v| <
// 1/4), e^(x - top) / sum by less than 2^-18 of the row's largest score (y e^-y <
// 1/2, and a sum of E terms), the sum with the bias by 2^-24 of itself; a group's
// sum by twice that.
//
// A warp takes a token.  The row is dealt out so that a group lies in 32 /
// (groups, up to a power of two) neighbouring lanes, V consecutive experts a
// lane: what is found by lane order is in the order of the experts' numbers.
// Each lane sorts its keys (two instructions a comparison), and each choice is the
// largest of the lanes' first, which that lane drops.  The chosen sit one in each
// of the first topk lanes.
//
// Bound by the issue of instructions: 8 of 128 experts take 540 a token, 8192 tokens
// 10 us (floor of the bytes 0.8); 8 of 256 in groups, with a bias, 840, 16383 tokens 25 us
// (2.7).  Rows that are done again cost more: 16383 x 256 saturated sigmoids 44 us.
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

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp2_of(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// A 32-bit key in the order of the value: 0 is below all, ~0 above all.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);           // -0 is 0
    return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}

// Falling order (odd-even merge sort; V a power of two).
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const uint32_t a = k[i + j], b = k[i + j + q];
                        k[i + j] = max(a, b);
                        k[i + j + q] = min(a, b);
                    }
}

struct RouteParams {
    int tokens, E, groups, keep, topk, per;      // per: experts to a group
    int lanes, shift;                            // lanes to a group, 1 << shift
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
        const F other = __shfl_sync(kAll, score, g << p.shift);
        before += other > score || (other == score && g < group);
    }
    return before;
}

// V values of a row for a lane, `none` from the live-th on; as 16-byte vectors
// where `vec`.
template <int V, class T>
__device__ __forceinline__ void load_row(const T* row, int live, bool vec, float none, float (&x)[V]) {
    constexpr int N = 16 / sizeof(T);
    if constexpr (V % N == 0) {
        if (vec) {
#pragma unroll
            for (int i = 0; i < V; i += N) {
                uint4 v = make_uint4(0, 0, 0, 0);
                if (i < live) v = __ldg(reinterpret_cast<const uint4*>(row + i));
                const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
                for (int j = 0; j < N; ++j) x[i + j] = i < live ? to_float(e[j]) : none;
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < live ? to_float(row[i]) : none;
}

// A row in 64 bits: choices only, of logits below plus infinity.  It reads them
// again: an array handed to it would live in memory in every row.
template <int V, class T>
__device__ __noinline__ int choose_exact(const RouteParams& p, const T* row, int first, int live, float top, int lane) {
    float x[V];
    load_row<V>(row + first, live, false, -kInf, x);
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
        in = group_rank(group_score(a, b), lane >> p.shift, p) < p.keep;
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

// vec: the rows, the groups and the bias allow 16-byte loads.
template <int V, class T>
__global__ void __launch_bounds__(256)
route_kernel(const RouteParams p, const bool vec) {
    constexpr uint32_t kLow = V - 1;                          // a key's bits that number the lane's experts
    constexpr uint32_t kNone = 0x007fffffu, kOver = 0xff800000u;    // the infinities, ordered
    const int lane = threadIdx.x & 31;
    const long long t = blockIdx.x * 8ll + (threadIdx.x >> 5);
    if (t >= p.tokens) return;
    const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
    const int group = lane >> p.shift, part = lane & (p.lanes - 1);
    const int first = group * p.per + part * V;               // this lane's experts: first .. first + live - 1
    const int live = group < p.groups ? min(V, p.per - part * V) : 0;
    const bool keyed = p.bias != nullptr;                     // keys are scores, not logits
    float x[V], s[V];
    load_row<V>(row + first, live, vec, -kInf, x);
    if (keyed) load_row<V>(p.bias + first, live, vec, 0.f, s);
    uint32_t key[V];
    uint32_t most = 0, least = ~0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        key[i] = ordered(x[i]);
        most = max(most, key[i]);
        least = min(least, key[i]);
    }
    most = __reduce_max_sync(kAll, most);
    // masked experts, lanes that are not full; NaNs (those with a sign lie below
    // minus infinity) and plus infinity
    const bool odd = __any_sync(kAll, least <= kNone) || most >= kOver;
    bool bad_row = false;
    if (odd) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < V; ++i) bad |= !(x[i] < kInf);
        bad_row = __any_sync(kAll, bad);
    }
    const float top = value_of(most);                         // where it matters the row is not a bad one
    float inv = 1.f;
    if (!p.sigmoid && (keyed || p.groups > 1 || !p.renorm)) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) sum += x[i] > -kInf ? expf(x[i] - top) : 0.f;
        inv = 1.f / warp_sum(sum);
    }
    auto score_of = [&](float v) {
        return p.sigmoid ? reciprocal(1.f + exp2_of(v * -kLog2e)) : exp2_of((v - top) * kLog2e) * inv;
    };
    if (!odd && keyed) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t k = ordered(score_of(x[i]) + s[i]);
            key[i] = k <= kNone ? 0u : (k & ~kLow) | (kLow - i);
        }
    } else if (!odd) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = (key[i] & ~kLow) | (kLow - i);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            uint32_t k = key[i];
            // a NaN or plus infinity takes the other scores of its row with it
            if (keyed) k = ordered((bad_row ? 0.f : score_of(x[i])) + s[i]);
            const bool off = x[i] == -kInf || (keyed && s[i] == -kInf);
            if (!(x[i] < kInf)) k = ~0u;
            key[i] = off ? 0u : (k & ~kLow) | (kLow - i);
        }
    }
    sort_keys(key);
    bool close = false, in = true;
    if (p.groups > 1) {
        float a = -kInf, b = -kInf;                           // this lane's two best
        if (keyed) {
            if (key[0]) a = value_of(key[0] & ~kLow);
            if (V > 1 && key[V > 1 ? 1 : 0]) b = value_of(key[V > 1 ? 1 : 0] & ~kLow);
        } else {
            // Of the logits as they are: a key has lost up to V - 1 of a 32-bit logit's
            // last units, and each is |x| 2^-23 of a softmax's score.
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float v = bad_row && !(x[i] < kInf) ? kInf : x[i];
                b = fmaxf(b, fminf(a, v));
                a = fmaxf(a, v);
            }
            auto scored = [&](float v) { return v == -kInf || v == kInf ? v : bad_row ? 0.f : score_of(v); };
            a = scored(a);
            b = scored(b);
        }
        if (bad_row) {                                        // truncated NaNs
            if (!(a <= kInf)) a = kInf;
            if (!(b <= kInf)) b = kInf;
        }
        group_top2(a, b, p.lanes);
        // the highest groups one by one, a group's number (falling, so that ties go to
        // the lowest) in its key's lowest bits.  Two of the lowest values do not add up
        // to minus infinity, which is a group of none (nor their sizes to infinity).
        constexpr float kMost = 0x1.fffffep127f;
        float score = group < p.groups ? group_score(a, b) : -kInf;
        if (score == -kInf && a > -kInf) score = -kMost;
        uint32_t gkey = score > -kInf ? (ordered(score) & ~31u) | (31 - group) : 0u, last = 0;
        in = false;
        for (int g = 0; g < p.keep; ++g) {
            last = __reduce_max_sync(kAll, gkey);
            if (last == 0) break;
            if (gkey == last) {
                in = true;
                gkey = 0;
            }
        }
        if (__any_sync(kAll, gkey != 0)) {                    // groups that are dropped
            // Of each group its own error: terms may cancel in its sum, and one of very
            // low biases is far off but also far below.
            const float size = fminf(fabsf(a) + (b > -kInf ? fabsf(b) : 0.f), kMost);
            const float off = route_slack(p.sigmoid, inv, size, V);
            const uint32_t low = __reduce_min_sync(kAll, in ? ordered(score - off) : ~0u);
            const uint32_t high = __reduce_max_sync(kAll, gkey ? ordered(score + off) : 0u);
            close = low <= high;
        }
    }
    // the topk largest.  Lanes are compared without the bits that number their
    // experts: of equal values the lowest lane's is the lowest expert.
    // A lane's keys behind its first wait in shared memory (up to 16; more are
    // moved up in registers): one load a choice and not V moves.
    constexpr bool kListed = V > 1 && V <= 16;
    __shared__ uint32_t lists[kListed ? 8 * V * 32 : 1];
    const int base = kListed ? (threadIdx.x >> 5) * V * 32 + lane : 0;
    if constexpr (kListed) {
#pragma unroll
        for (int i = 1; i < V; ++i) lists[base + 32 * (i - 1)] = key[i];
        lists[base + 32 * (V - 1)] = 0;
    }
    int at = base;
    uint32_t best = in && key[0] ? key[0] | kLow : 0u;
    auto drop = [&] {                                         // this lane's first key
        if constexpr (kListed) {
            key[0] = lists[at];
            at += 32;
        } else {
#pragma unroll
            for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
            key[V - 1] = 0;
        }
        best = key[0] ? key[0] | kLow : 0u;
    };
    int mine = -1;                                            // lane j: the j-th choice
    uint32_t mkey = 0;
    for (int j = 0; j < p.topk; ++j) {
        const uint32_t m = __reduce_max_sync(kAll, best);
        if (m == 0) break;
        const int win = __ffs(__ballot_sync(kAll, best == m)) - 1;
        const int e = __shfl_sync(kAll, first + static_cast<int>(kLow - (key[0] & kLow)), win);
        if (lane == j) { mine = e; mkey = m; }
        if (lane == win) drop();
    }
    if (!bad_row && (keyed || (sizeof(T) == 4 && V > 1))) {
        // neighbours whose order the keys could have got wrong, the next key after
        // the choices among them
        const uint32_t lkey = __reduce_max_sync(kAll, best);
        uint32_t nkey = __shfl_down_sync(kAll, mkey, 1);
        if (lane == p.topk - 1) nkey = lkey;
        bool near = lane < p.topk && mkey && nkey && mkey == nkey;
        if (keyed) {
            const float v = value_of(mkey & ~kLow), next = value_of(nkey & ~kLow);
            near = lane < p.topk && mkey && nkey &&
                   v - next <= route_slack(p.sigmoid, inv, fmaxf(fabsf(v), fabsf(next)), V);
        }
        if (__any_sync(kAll, near)) {
            // the same logit and bias are a tie, and ties are in order
            const int win = __ffs(__ballot_sync(kAll, best == lkey)) - 1;
            const int last = __shfl_sync(kAll, first + static_cast<int>(kLow - (key[0] & kLow)), win);
            int next = __shfl_down_sync(kAll, mine, 1);
            if (lane == p.topk - 1) next = last;
            const bool differ = near && (to_float(row[mine]) != to_float(row[next]) ||
                                         (keyed && __ldg(p.bias + mine) != __ldg(p.bias + next)));
            close = close || __any_sync(kAll, differ);
            // behind a tie of the last choice and the next key others may follow that the
            // keys cannot tell from the two: each lane walks its own while they are near
            if (!close && __any_sync(kAll, near && lane == p.topk - 1)) {
                const int e0 = __shfl_sync(kAll, mine, p.topk - 1);
                const uint32_t k0 = __shfl_sync(kAll, mkey, p.topk - 1);
                const float x0 = to_float(row[e0]), b0 = keyed ? __ldg(p.bias + e0) : 0.f;
                bool other = false;
                while (best && !other) {
                    other = best == k0;
                    if (keyed) {
                        const float v = value_of(k0 & ~kLow), w = value_of(best & ~kLow);
                        other = v - w <= route_slack(p.sigmoid, inv, fmaxf(fabsf(v), fabsf(w)), V);
                    }
                    if (!other) break;                        // the lane's further keys are lower still
                    const int e = first + static_cast<int>(kLow - (key[0] & kLow));
                    other = to_float(row[e]) != x0 || (keyed && __ldg(p.bias + e) != b0);
                    drop();
                }
                close = __any_sync(kAll, other);
            }
        }
    }
    if (close && !bad_row) mine = choose_exact<V>(p, row, first, live, top, lane);
    if (lane >= p.topk) mine = -1;
    const bool has = mine >= 0;
    const float mx = has ? to_float(row[mine]) : -kInf;
    float w;
    if (p.renorm) {
        // the chosen scores over their sum; where they could vanish, from their logarithms
        if (p.sigmoid && !__any_sync(kAll, has && !(mx > -60.f))) {
            w = has ? reciprocal(1.f + expf(-mx)) : 0.f;
        } else {
            const float l = !has ? -kInf : p.sigmoid ? fminf(mx, 0.f) - log1pf(expf(-fabsf(mx))) : mx;
            const float lt = value_of(__reduce_max_sync(kAll, ordered(l)));
            w = has ? expf(l - lt) : 0.f;
        }
        w *= reciprocal(warp_sum(w));
    } else {
        w = p.sigmoid ? 1.f / (1.f + expf(-mx)) : expf(mx - top) * inv;
    }
    w = bad_row ? __uint_as_float(0x7fc00000u) : has ? w * p.scale : 0.f;
    if (lane < p.topk) {
        const long long at = t * p.topk + lane;
        p.ids[at] = mine;
        p.weights[at] = w;
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
// A warp takes a token.  Bound by the issue of instructions: 300 a token with renorm
// (16383 x 256 8.7 us, its bytes 2.7), 360 for a softmax without, which reads a row three
// times and forms each exponential twice (8192 x 128 6.3 us, 1.4).
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
        constexpr int N = 16 / sizeof(T);
        if (p.E % N == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0)
            for (int i = lane * N; i < p.E; i += 32 * N) *reinterpret_cast<uint4*>(out + i) = make_uint4(0, 0, 0, 0);
        else
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
    while (1 << p.shift < p.lanes) ++p.shift;
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
    // whole vectors a lane, in every row and group
    constexpr int N = 16 / sizeof(T);
    const bool vec = p.per % N == 0 && (p.tokens == 1 || p.ldl % N == 0) && reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
                     p.per % 4 == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
    if (v <= 1) route_kernel<1, T><<<blocks, 256, 0, s>>>(p, vec);
    else if (v <= 2) route_kernel<2, T><<<blocks, 256, 0, s>>>(p, vec);
    else if (v <= 4) route_kernel<4, T><<<blocks, 256, 0, s>>>(p, vec);
    else if (v <= 8) route_kernel<8, T><<<blocks, 256, 0, s>>>(p, vec);
    else if (v <= 16) route_kernel<16, T><<<blocks, 256, 0, s>>>(p, vec);
    else if (v <= 32) route_kernel<32, T><<<blocks, 256, 0, s>>>(p, vec);
    else route_kernel<64, T><<<blocks, 256, 0, s>>>(p, vec);
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
