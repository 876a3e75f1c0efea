// moe_topk_kernel.cuh -- routing to experts: the expert ids and weights that
// nvfp4_moe_route and nvfp4_moe_combine take, from the router's logits x[T][E].
//
//     s_e  = softmax(x)_e  or  1 / (1 + exp(-x_e))
//     c_e  = s_e + bias_e                       (the bias steers the choice only)
//     with groups of E/G consecutive experts: a group's score is the sum of its
//            `group_top` (1 or 2) largest c; the top_groups best groups are kept
//     ids  = the k largest c of the kept groups, in descending order
//     w    = s[ids], divided by their sum if renormalised (0 if that is 0), times scale
//
// Ties go to the lowest index.  A NaN logit counts as -Inf, +Inf as the largest finite
// value; a NaN choice or group score counts as -Inf.  A row without any logit above -Inf
// has the score 0 for every expert.
//
// The ids are those of the 64-bit values (neighbouring choices can differ by less than an
// FP32 step), at FP32's price: without a bias experts order like their logits, which are
// compared as they are.  Otherwise the choices are computed in FP32 with a proven error
// bound; the list of the best is extended until nothing outside it can belong to the first
// k, and where two neighbours are closer than the bound allows, it is ranked again by
// 64-bit choices, one list entry per lane.  Groups closer than the bound are chosen by
// 64-bit sums; a token with more near-ties than lanes goes through 64 bits as a whole.
// Weights are computed in 64 bits from the k chosen logits and rounded once.  Only the sum
// that softmax weights are divided by when they are not renormalised is one of FP32
// exponentials, added in 64 bits: it is off by at most 2 + ln E units of 2^-24 (see gap), on
// average by less than the rounding.  (All exponentials in 64 bits are the price of the
// whole-token path; tokens whose choices are near each other have them anyway.)
//
// One warp per token; a group's experts sit on `lpg` neighbouring lanes, V per lane, in
// ascending order, so the lowest lane and the lowest slot hold the lowest index.  Few
// bytes, many instructions: bound by their issue.  8192 tokens over 256 experts in 8 groups
// (8.9 MB, 1.4 us of HBM; 936 warp instructions a token) take 10 us, 65536 of them 66 us with
// 81 % of the issue slots and 58 % of the integer pipe's busy (68 and 48 % at 8192 tokens,
// which are 1.7 waves).  3001 tokens over 60 experts (480 instructions a token) take 3.7 us in
// a graph, where 16 tokens over 8 take 1.8: half of it is one token's chain of dependent steps.  Everything in 64 bits took 28.8 us; selection rounds over all of a lane's
// experts instead of the packed list 14.8 against 12.0 us (but for up to 2 experts per lane
// they are the faster form: 64 experts 5.5 against 6.0 us); a whole token in 64 bits where
// only its groups are too close, 11.7 us.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>

#include "moe_kernel.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace topk {

constexpr int MAX_EXPERTS = moe::MAX_EXPERTS;
constexpr int MAX_K = 32;
constexpr int MAX_GROUPS = 32;
constexpr int WARPS = 4;

struct Params {
    int T, E, k;
    int sigmoid;     // scores: 0 softmax, 1 sigmoid
    int groups, top_groups, group_top;
    int renorm;
    float scale;
    int per, lpg;    // experts of a group, lanes of a group
    int lanes;       // lanes that hold at least one expert of the kept groups
};

constexpr float FLT_LARGEST = 3.402823466e38f;

// One token's scores s and choices c by the formulas in 64 bits, by its whole warp; returns
// whether the lane's group is kept.
template <int V, typename X>
__device__ __forceinline__ bool exact_choices(const X* __restrict__ logits, const float* __restrict__ bias,
                                              const Params& p, int t, double (&s)[V], double (&c)[V]) {
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const double NEG = -__longlong_as_double(0x7FF0000000000000ll);
    const int g = lane / p.lpg, i0 = (lane % p.lpg) * V;
    const int e0 = g * p.per + i0;
    const int cnt = g < p.groups ? max(0, min(V, p.per - i0)) : 0;

    double x[V], xmax = NEG;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = NEG;
        if (v < cnt) {
            const float f = (float)logits[(size_t)t * p.E + e0 + v];
            if (f == f) x[v] = (double)fminf(f, FLT_LARGEST);
        }
        xmax = fmax(xmax, x[v]);
    }
    if (!p.sigmoid) {
#pragma unroll
        for (int o = 16; o; o >>= 1) xmax = fmax(xmax, __shfl_xor_sync(FULL, xmax, o));
        double sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            s[v] = x[v] > NEG ? exp(x[v] - xmax) : 0.0;
            sum += s[v];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = sum > 0.0 ? s[v] / sum : 0.0;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = 1.0 / (1.0 + exp(-x[v]));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        c[v] = s[v];
        if (bias && v < cnt) c[v] += (double)__ldg(bias + e0 + v);
        if (!(c[v] == c[v])) c[v] = NEG;
    }

    bool kept = g < p.groups;
    if (p.groups > 1) {
        // the two largest choices of the lane, then of the group's lanes
        double a = NEG, b = NEG;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v < cnt) {
                b = fmax(b, fmin(a, c[v]));
                a = fmax(a, c[v]);
            }
        for (int o = 1; o < p.lpg; o <<= 1) {
            const double a2 = __shfl_xor_sync(FULL, a, o), b2 = __shfl_xor_sync(FULL, b, o);
            b = fmax(fmin(a, a2), fmax(b, b2));
            a = fmax(a, a2);
        }
        double gs = p.group_top == 2 && p.per > 1 ? a + b : a;
        if (!(gs == gs)) gs = NEG;
        int better = 0;
        for (int h = 0; h < p.groups; ++h) {
            const double o = __shfl_sync(FULL, gs, h * p.lpg);
            better += o > gs || (o == gs && h < g);
        }
        kept = kept && better < p.top_groups;
    }
    return kept;
}

// Whether the lane's group is kept, where FP32 sums are too close to tell.
template <int V, typename X>
__device__ __noinline__ bool group_kept_exact(const X* __restrict__ logits, const float* __restrict__ bias,
                                              const Params& p, int t) {
    double s[V], c[V];
    return exact_choices<V, X>(logits, bias, p, t, s, c);
}

// The whole token in 64 bits, chosen with a bias (without one, experts order like their
// logits and no near-tie arises).
template <int V, typename X>
__device__ __noinline__ void topk_exact(const X* __restrict__ logits, const float* __restrict__ bias,
                                        int32_t* __restrict__ ids, float* __restrict__ weights,
                                        const Params& p, int t) {
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    const double NEG = -__longlong_as_double(0x7FF0000000000000ll);
    const int g = lane / p.lpg, i0 = (lane % p.lpg) * V;
    const int e0 = g * p.per + i0;
    const int cnt = g < p.groups ? max(0, min(V, p.per - i0)) : 0;
    double s[V], c[V];
    const bool kept = exact_choices<V, X>(logits, bias, p, t, s, c);

    // k rounds: the best expert left, by (choice, lowest index)
    unsigned left = kept ? (1u << cnt) - 1u : 0u;
    double total = 0.0, mine = 0.0;  // sum of the chosen scores; the score of slot `lane`
    int my_id = 0;
    for (int j = 0; j < p.k; ++j) {
        double best = NEG, sc = 0.0;
        int id = p.E;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if ((left >> v & 1u) && (id == p.E || c[v] > best)) {
                best = c[v];
                sc = s[v];
                id = e0 + v;
            }
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const double ob = __shfl_xor_sync(FULL, best, o), os = __shfl_xor_sync(FULL, sc, o);
            const int oi = __shfl_xor_sync(FULL, id, o);
            if (oi < p.E && (id == p.E || ob > best || (ob == best && oi < id))) {
                best = ob;
                sc = os;
                id = oi;
            }
        }
        if (id >= e0 && id < e0 + cnt) left &= ~(1u << (id - e0));
        total += sc;
        if (lane == j) {
            mine = sc;
            my_id = id;
        }
    }
    if (lane < p.k) {
        double w = mine;
        if (p.renorm) w = total > 0.0 ? w / total : 0.0;
        ids[(size_t)t * p.k + lane] = my_id;
        weights[(size_t)t * p.k + lane] = (float)(w * (double)p.scale);
    }
}

// Order-preserving key of an FP32 value (never 0: that is left for "no expert").
__device__ __forceinline__ uint32_t order_key(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);  // -0 counts as +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// At least twice the error of an FP32 choice whose terms are of size `mag`: two choices
// further apart order as their real values do.  In units of 2^-24, with __expf off by
// 2 + 1.173 |x| steps (4 + 2.35 |x| units) and expf by one step:
//   sigmoid: exp moves s by at most 1.6 (s (1 - s) <= 1/4 and s (1 - s) |x| <= 0.23);
//     1 + exp adds 1, the fast division 4: 6.6 in all.
//   softmax: exp is off by 2 + d relative at d = max - x (its argument's rounding), at
//     most 2.4 of s <= 1 (s d <= 0.37); the sum by 9 (the same, d weighted by the terms
//     at most ln 256, and its rounding); the division and the product add 2: 14 in all.
//   the bias' addition: |c|.
__device__ __forceinline__ float gap(float mag, bool sigmoid) {
    return (sigmoid ? 16.0f : 32.0f) * 0x1p-24f + fabsf(mag) * 0x1p-22f;
}

template <int V, typename X>
__device__ __forceinline__ void load_logits(const X* __restrict__ row, int e0, int cnt, bool vec,
                                            float (&x)[V]) {
    if (vec) {
        if constexpr (sizeof(X) == 4 && V % 4 == 0) {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(row + e0 + v));
                x[v] = f.x, x[v + 1] = f.y, x[v + 2] = f.z, x[v + 3] = f.w;
            }
        } else if constexpr (sizeof(X) == 2 && V % 4 == 0) {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + e0 + v));
                x[v] = __uint_as_float(u.x << 16), x[v + 1] = __uint_as_float(u.x & 0xFFFF0000u);
                x[v + 2] = __uint_as_float(u.y << 16), x[v + 3] = __uint_as_float(u.y & 0xFFFF0000u);
            }
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = v < cnt ? (float)row[e0 + v] : -INFINITY;
    }
    // NaN counts as -Inf (fmaxf drops it), +Inf as the largest finite value
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = fminf(fmaxf(x[v], -INFINITY), FLT_LARGEST);
}

// FULL_LANES: every lane holds exactly V experts, on 16-byte (BF16: 8-byte) boundaries
// (it took 4 us of the 72 that 65536 x 256 in 8 groups took before).
template <int V, typename X, bool FULL_LANES>
__global__ void __launch_bounds__(32 * WARPS, V <= 8 ? 8 : 4)
moe_topk_kernel(const X* __restrict__ logits, const float* __restrict__ bias,
                int32_t* __restrict__ ids, float* __restrict__ weights,
                const __grid_constant__ Params p) {
    const unsigned FULL = 0xffffffffu;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * WARPS + warp;
    grid_dependents_launch();  // the kernel behind may set itself up; it waits for this one's end
    grid_dependency_wait();
    if (t >= p.T) return;
    const int g = lane / p.lpg, i0 = (lane % p.lpg) * V;
    const int e0 = g * p.per + i0;
    const int cnt = FULL_LANES ? V : g < p.groups ? max(0, min(V, p.per - i0)) : 0;
    const X* const row = logits + (size_t)t * p.E;
    const bool group_sum = p.groups > 1 && p.group_top == 2 && p.per > 1;

    float c[V];  // what the experts are ordered by: the choices, or without a bias the logits
    load_logits<V, X>(row, e0, cnt, FULL_LANES, c);
    float xmax = 0.f;
    double sum = 0.0;  // of FP32 exponentials: their errors average out, additions would not
    if (!p.sigmoid) {
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) m = max(m, order_key(c[v]));
        xmax = key_value(__reduce_max_sync(FULL, m));
    }
    float s[V];  // FP32 scores, where something is ordered or summed by them
    const bool scores = bias || group_sum || (!p.sigmoid && !p.renorm);
    if (scores) {
        if (p.sigmoid) {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = __fdividef(1.0f, 1.0f + __expf(-c[v]));
            // __fdividef gives 0 beyond 2^126, as does the formula to within 2^-126
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = c[v] > -INFINITY ? expf(c[v] - xmax) : 0.f;
                sum += (double)s[v];
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
            const float inv = sum > 0.0 ? __fdiv_rn(1.0f, (float)sum) : 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] *= inv;
        }
    }
    if (bias) {
        float b[V];
        if constexpr (FULL_LANES) {
#pragma unroll
            for (int v = 0; v < V; v += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(bias + e0 + v));
                b[v] = f.x, b[v + 1] = f.y, b[v + 2] = f.z, b[v + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) b[v] = v < cnt ? __ldg(bias + e0 + v) : 0.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = fmaxf(s[v] + b[v], -INFINITY);  // a NaN counts as -Inf
    }

    bool kept = FULL_LANES || g < p.groups;
    if (p.groups > 1) {
        float a = -INFINITY, b = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float q = v < cnt ? (group_sum && !bias ? s[v] : c[v]) : -INFINITY;
            b = fmaxf(b, fminf(a, q));
            a = fmaxf(a, q);
        }
        for (int o = 1; o < p.lpg; o <<= 1) {
            const float a2 = __shfl_xor_sync(FULL, a, o), b2 = __shfl_xor_sync(FULL, b, o);
            b = fmaxf(fminf(a, a2), fmaxf(b, b2));
            a = fmaxf(a, a2);
        }
        // half the sum of two choices: that of two finite ones stays finite
        const float gs = fmaxf(group_sum ? fmaf(0.5f, a, 0.5f * b) : a, -INFINITY);
        // groups of lower index with an equal score come first
        int better = 0;
        for (int h = 0; h < p.groups; ++h) {
            const float o = __shfl_sync(FULL, gs, h * p.lpg);
            better += o > gs || (o == gs && h < g);
        }
        const bool exists = kept;
        kept = kept && better < p.top_groups;
        if ((bias || group_sum) && p.top_groups < p.groups) {
            // the worst kept group and the best one left out, too close to call?
            const float lo = key_value(__reduce_min_sync(FULL, kept ? order_key(gs) : 0xFFFFFFFFu));
            const float hi = key_value(__reduce_max_sync(FULL, exists && !kept ? order_key(gs) : 0u));
            // the terms of the largest finite sum bound every sum's error (infinite ones, of an
            // infinite term, are exact; where the terms' magnitudes overflow, 64 bits decide)
            const float mag = key_value(__reduce_max_sync(
                FULL, order_key(exists && fabsf(gs) < INFINITY ? fabsf(a) + (group_sum ? fabsf(b) : 0.f) : 0.f)));
            // (a half sum's error is at most a choice's of the size mag; false for two equal infinities)
            if (lo - hi <= gap(mag, p.sigmoid != 0))
                kept = group_kept_exact<V, X>(logits, bias, p, t);
        }
    }

    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = kept && v < cnt ? order_key(c[v]) : 0u;

    // The list of the best, in descending order: lane j holds the j-th; n entries, and none
    // outside it can belong to the first k (unless n == 32, see below).
    uint32_t my_key = 0;
    int my_id = 0, n = 0;
    bool complete = false;
    __shared__ uint2 list[WARPS][32];
    if (V >= 4 && p.k <= p.lanes) {
        // The k-th largest of the lanes' maxima is no larger than the k-th choice.  What
        // reaches it (with a bias: reaches within the gap below it) is a short list, which
        // is packed in index order and ranked by counting.
        uint32_t m = 0, t0 = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) m = max(m, key[v]);
        for (int j = 0; j < p.k; ++j) {
            t0 = __reduce_max_sync(FULL, m);
            m = m == t0 ? 0u : m;
        }
        if (bias) {
            const float a = key_value(t0);
            t0 = order_key(fmaxf(a - gap(a, p.sigmoid != 0), -INFINITY));
        }
        t0 = max(t0, 1u);
        int mine = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) mine += key[v] >= t0;
        int at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(FULL, at, o);
            if (lane >= o) at += x;
        }
        n = __shfl_sync(FULL, at, 31);
        if (n <= 32) {
            at -= mine;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] >= t0) list[warp][at++] = make_uint2(key[v], (uint32_t)(e0 + v));
            __syncwarp();
            const uint2 e = lane < n ? list[warp][lane] : make_uint2(0u, 0u);
            int r = 0;
            for (int j = 0; j < n; ++j) {
                const uint32_t o = __shfl_sync(FULL, e.x, j);
                r += o > e.x || (o == e.x && j < lane);
            }
            __syncwarp();
            if (lane < n) list[warp][r] = e;
            __syncwarp();
            if (lane < n) {
                my_key = list[warp][lane].x;
                my_id = (int)list[warp][lane].y;
            }
            complete = true;
        }
    }
    if (!complete) {
        // Fewer lanes than k in the kept groups, or many equal choices: each lane's experts
        // in descending order (a stable network: equal keys keep their order), then
        // selection rounds: the best head of all lanes leaves its list; a few more than k
        // rounds while they are too close to the k-th.
        int slot[V];
#pragma unroll
        for (int v = 0; v < V; ++v) slot[v] = e0 + v;
#pragma unroll
        for (int i = 0; i + 1 < V; ++i)
#pragma unroll
            for (int j = V - 1; j > i; --j) {
                const bool swap = key[j] > key[j - 1];
                const uint32_t hi = max(key[j], key[j - 1]), lo = min(key[j], key[j - 1]);
                const int a = swap ? slot[j] : slot[j - 1], b = swap ? slot[j - 1] : slot[j];
                key[j - 1] = hi, key[j] = lo;
                slot[j - 1] = a, slot[j] = b;
            }
        n = 0;
        uint32_t kth = 0;
        auto take = [&](uint32_t top) {
            const int src = __ffs(__ballot_sync(FULL, key[0] == top)) - 1;
            const int id = __shfl_sync(FULL, slot[0], src);
            if (lane == n) {
                my_key = top;
                my_id = id;
            }
            const bool pop = lane == src;
#pragma unroll
            for (int v = 0; v + 1 < V; ++v) {
                key[v] = pop ? key[v + 1] : key[v];
                slot[v] = pop ? slot[v + 1] : slot[v];
            }
            if (pop) key[V - 1] = 0;
            if (n == p.k - 1) kth = top;
            ++n;
        };
        while (n < p.k) take(__reduce_max_sync(FULL, key[0]));  // k experts are kept at least
        complete = true;
        if (bias) {
            // experts out of reach of the k-th end the list; so does one equal to it without
            // rounding (two infinities), where the index has decided already
            const float a = key_value(kth);
            while (true) {
                const uint32_t top = __reduce_max_sync(FULL, key[0]);
                if (top == 0 || !(a - key_value(top) <= gap(a, p.sigmoid != 0))) break;
                if (n == 32) {
                    complete = false;
                    break;
                }
                take(top);
            }
        }
    }
    bool near = false;
    if (bias) {
        const uint32_t next = __shfl_down_sync(FULL, my_key, 1);
        const float a = key_value(my_key);
        near = __any_sync(FULL, lane + 1 < n && a - key_value(next) <= gap(a, p.sigmoid != 0));
        if (!complete) {
            topk_exact<V, X>(logits, bias, ids, weights, p, t);
            return;
        }
    }

    // 64-bit scores of the list, one per lane
    const bool live = lane < n;
    double x = 0.0, sc = 0.0;
    if (live) {
        float f = (float)row[my_id];
        f = fminf(fmaxf(f, -INFINITY), FLT_LARGEST);
        x = (double)f;
        sc = p.sigmoid ? 1.0 / (1.0 + exp(-x)) : f > -INFINITY ? exp(x - (double)xmax) : 0.0;
    }
    double sum64 = sum;
    if (near && !p.sigmoid) {  // the softmax's sum in 64 bits too
        float f[V];
        load_logits<V, X>(row, e0, cnt, FULL_LANES, f);
        sum64 = 0.0;
#pragma unroll 1
        for (int v = 0; v < V; ++v) {
            float q = f[0];
#pragma unroll
            for (int u = 1; u < V; ++u) q = u == v ? f[u] : q;
            if (q > -INFINITY) sum64 += exp((double)q - (double)xmax);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) sum64 += __shfl_xor_sync(FULL, sum64, o);
    }
    int rank = lane;
    if (near) {
        const double NEG = -__longlong_as_double(0x7FF0000000000000ll);
        const double s64 = p.sigmoid ? sc : sum64 > 0.0 ? sc / sum64 : 0.0;
        double ch = live ? s64 + (double)__ldg(bias + my_id) : NEG;
        if (!(ch == ch)) ch = NEG;
        rank = 0;
        for (int i = 0; i < n; ++i) {
            const double o = __shfl_sync(FULL, ch, i);
            const int oi = __shfl_sync(FULL, my_id, i);
            rank += o > ch || (o == ch && oi < my_id);
        }
    }
    const bool chosen = live && rank < p.k;
    double w = sc;
    if (p.renorm) {
        double total = chosen ? sc : 0.0;
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(FULL, total, o);
        w = total > 0.0 ? sc / total : 0.0;
    } else if (!p.sigmoid) {
        w = sum64 > 0.0 ? sc / sum64 : 0.0;
    }
    if (chosen) {
        ids[(size_t)t * p.k + rank] = my_id;
        weights[(size_t)t * p.k + rank] = (float)(w * (double)p.scale);
    }
}

}  // namespace topk
}  // namespace nvfp4
