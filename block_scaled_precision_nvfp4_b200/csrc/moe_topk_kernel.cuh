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
// Choices are compared in 64 bits: without a bias they order like the logits, which are
// compared instead; with one, neighbouring sums can differ by less than an FP32 step.
//
// One warp per token; a group's experts sit on `lpg` neighbouring lanes, V per lane.
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
};

template <int V, typename X>
__global__ void __launch_bounds__(32 * WARPS)
moe_topk_kernel(const X* __restrict__ logits, const float* __restrict__ bias,
                int32_t* __restrict__ ids, float* __restrict__ weights,
                const __grid_constant__ Params p) {
    const unsigned FULL = 0xffffffffu;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * WARPS + warp;
    grid_dependents_launch();  // the kernel behind may set itself up; it waits for this one's end
    grid_dependency_wait();
    if (t >= p.T) return;
    const double NEG = -__longlong_as_double(0x7FF0000000000000ll);
    const int g = lane / p.lpg, i0 = (lane % p.lpg) * V;
    const int e0 = g * p.per + i0;
    const int cnt = g < p.groups ? max(0, min(V, p.per - i0)) : 0;

    double x[V], s[V], c[V];  // logits, scores, choices
    double xmax = NEG;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[v] = NEG;
        if (v < cnt) {
            const float f = (float)logits[(size_t)t * p.E + e0 + v];
            if (f == f) x[v] = (double)fminf(f, 3.402823466e38f);
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

    // k rounds: the best expert left, by (choice, lowest index)
    unsigned left = kept ? (1u << cnt) - 1u : 0u;
    double total = 0.0, mine = 0.0;  // sum of the chosen scores; the score of slot `lane`
    int my_id = 0;
    for (int j = 0; j < p.k; ++j) {
        double best = NEG, sc = 0.0;
        int id = p.E;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double key = bias ? c[v] : x[v];
            if ((left >> v & 1u) && (id == p.E || key > best)) {
                best = key;
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

}  // namespace topk
}  // namespace nvfp4
