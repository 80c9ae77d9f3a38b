// Routing for gfx950: scores, group-limited top-K, weights; and the gradient
// of the weights.
//
//   s = softmax(l) or sigmoid(l);  c = s + bias
//   the groupsPerToken best groups by the sum of their groupTop best c
//   the K best experts of those by c (by l without a bias)
//   w = routedScale * s, or routedScale * s / (sum of the chosen s)
//
// Which expert is chosen may hang on the last bits of two scores, so the
// choice is made on 64-bit values: two programs that compute the same formula
// then agree.
#include "ops_internal.h"

namespace epdc {
namespace {

constexpr float kInf = __builtin_inff();
constexpr double kInf64 = __builtin_inf();

template <bool FP32>
__device__ __forceinline__ float load_logit(const void *p, int64_t i) {
    if (FP32) return static_cast<const float *>(p)[i];
    return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
}

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// One token by one wave, any configuration: lane holds experts lane, lane +
// 64, ...; K rounds of a wave-wide maximum over (choice value, lower index).
// keys: [E] doubles of LDS of this wave, used where groups are limited.
template <int NPL, bool FP32>
__device__ void route_token(const RouteParams &P, int32_t t, double *keys) {
    const int lane = threadIdx.x & 63;
    wave_lds_order();  // the previous token's reads of keys
    const bool biased = P.bias != nullptr;
    float l[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        l[i] = e < P.E ? load_logit<FP32>(P.logits, (int64_t)t * P.E + e) : -kInf;
    }
    // scores in 64 bits; s = 0 and key = -inf for a masked logit
    double s[NPL], key[NPL];
    if (P.softmax) {
        float top = -kInf;
#pragma unroll
        for (int i = 0; i < NPL; ++i) top = fmaxf(top, l[i]);  // fmaxf drops a NaN
        top = wave_max(top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            s[i] = !(l[i] > -kInf) ? 0.0 : l[i] == top ? 1.0 : exp((double)l[i] - (double)top);
            sum += s[i];
        }
        sum = fmax(wave_sum(sum), 1.0);  // 1 or more unless every logit is masked
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] /= sum;
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] = !(l[i] > -kInf) ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
    }
    const bool limited = P.keep < P.G;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        double c = s[i];
        if (biased && e < P.E) c += (double)P.bias[e];
        if (!(l[i] > -kInf) || !(c > -kInf64)) c = -kInf64;
        key[i] = c > -kInf64 && !biased ? (double)l[i] : c;
        // groups go by their best keys (one value), or by sums of choice values
        if (limited && e < P.E) keys[e] = P.groupTop == 1 ? key[i] : c;
    }
    if (limited) {
        wave_lds_order();
        double a = -kInf64, b = -kInf64;  // a group's two best
        if (lane < P.G) {
            for (int j = 0; j < P.perGroup; ++j) {
                const double v = keys[lane * P.perGroup + j];
                b = fmax(b, fmin(a, v));
                a = fmax(a, v);
            }
            if (P.groupTop == 2 && b > -kInf64) a += b;
        }
        int rank = 0;
        for (int g = 0; g < P.G; ++g) {
            const double o = __shfl(a, g);
            rank += (o > a || (o == a && g < lane)) ? 1 : 0;
        }
        const uint64_t kept = __ballot(lane < P.G && rank < P.keep);
        wave_lds_order();
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 64 + lane;
            if (e < P.E && !((kept >> (e / P.perGroup)) & 1)) key[i] = -kInf64;
        }
    }
    int32_t id = -1;    // slot `lane`
    double mine = 0.0;  // its score
    for (int k = 0; k < P.K; ++k) {
        double best = -kInf64;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (key[i] > best) best = key[i], at = i * 64 + lane;
#pragma unroll
        for (int d = 32; d; d >>= 1) {
            const double ob = __shfl_xor(best, d);
            const int oa = __shfl_xor(at, d);
            if (ob > best || (ob == best && oa < at)) best = ob, at = oa;
        }
        at = uniform(at);
        if (at == 0x7fffffff) break;  // nothing left to choose
        double sv = 0.0;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (i == at >> 6) {
                sv = __shfl(s[i], at & 63);
                if (lane == (at & 63)) key[i] = -kInf64;
            }
        if (lane == k) id = at, mine = sv;
    }
    double w = mine;
    if (P.renorm) {
        const double total = wave_sum(mine);
        w = total > 0.0 ? mine / total : 0.0;
    }
    if (lane < P.K) {
        const int64_t o = (int64_t)t * P.K + lane;
        P.expertIds[o] = id;
        P.weights[o] = (float)(w * (double)P.scale);
    }
}

template <int NPL, bool FP32>
__global__ __launch_bounds__(256) void route_kernel(RouteParams P) {
    extern __shared__ double route_keys[];
    const int wave = threadIdx.x >> 6;
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < P.T; t += (int64_t)gridDim.x * 4)
        route_token<NPL, FP32>(P, (int32_t)t, route_keys + wave * P.E);
}

// One wave per token.  Slot k's expert, logit and gradient sit in lane k.
// row: [NPL * 64] floats of LDS of this wave, the token's sums per expert.
template <int NPL, bool FP32>
__device__ void grad_token(const RouteGradParams &P, int64_t t, float *row) {
    const int lane = threadIdx.x & 63;
    const bool dense = P.softmax && !P.renorm;
    int32_t id = -1;
    float g = 0.0f, sel = -kInf;
    if (lane < P.K) {
        id = P.expertIds[t * P.K + lane];
        g = P.dWeights[t * P.K + lane] * P.scale;
        if (id < 0 || id >= P.E)
            id = -1;
        else
            sel = load_logit<FP32>(P.logits, t * P.E + id);
        if (!(sel > -kInf)) id = -1;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) row[i * 64 + lane] = 0.0f;
    float p[NPL];
    float d = 0.0f;  // the slot's contribution to its expert's sum
    if (dense) {
        float top = -kInf;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = i * 64 + lane;
            p[i] = e < P.E ? load_logit<FP32>(P.logits, t * P.E + e) : -kInf;
            top = fmaxf(top, p[i]);
        }
        top = wave_max(top);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            p[i] = !(p[i] > -kInf) ? 0.0f : p[i] == top ? 1.0f : expf(p[i] - top);
            sum += p[i];
        }
        const float inv = 1.0f / fmaxf(wave_sum(sum), 1.0f);
#pragma unroll
        for (int i = 0; i < NPL; ++i) p[i] *= inv;
        d = id >= 0 ? g : 0.0f;
    } else {
        float r, q = 1.0f;
        if (P.softmax) {
            const float top = wave_max(sel);
            r = id < 0 ? 0.0f : sel == top ? 1.0f : expf(sel - top);
        } else {
            // s = e / (1 + e) and 1 - s = 1 / (1 + e) from the exponential of the
            // negative magnitude, which cannot overflow
            const float x = expf(-fabsf(sel)), big = 1.0f / (1.0f + x), small = x * big;
            r = id < 0 ? 0.0f : sel >= 0.0f ? big : small;
            q = sel >= 0.0f ? small : big;
        }
        float dot = 0.0f;
        if (P.renorm) {
            const float total = wave_sum(r);
            r = total > 0.0f ? r / total : 0.0f;
            dot = wave_sum(id >= 0 ? g * r : 0.0f);
        }
        d = id >= 0 ? r * q * (g - dot) : 0.0f;
    }
    // slots of one expert add up in slot order, in the first of them
    float total = 0.0f;
    bool first = id >= 0;
    for (int k = 0; k < P.K; ++k) {
        const int32_t ok = __builtin_amdgcn_readlane(id, k);
        const float od = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(d), k));
        if (ok == id) {
            total += od;
            if (k < lane) first = false;
        }
    }
    wave_lds_order();
    if (first) row[id] = total;
    wave_lds_order();
    float dot = 0.0f;
    if (dense) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) dot += p[i] * row[i * 64 + lane];
        dot = wave_sum(dot);
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        if (e >= P.E) continue;
        const float v = dense ? p[i] * (row[e] - dot) : row[e];
        if (FP32)
            static_cast<float *>(P.dLogits)[t * P.E + e] = v;
        else
            static_cast<uint16_t *>(P.dLogits)[t * P.E + e] = (uint16_t)bf16_rne(v);
    }
}

template <int NPL, bool FP32>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradParams P) {
    __shared__ float rows[4][NPL * 64];
    const int wave = threadIdx.x >> 6;
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < P.T; t += (int64_t)gridDim.x * 4) {
        grad_token<NPL, FP32>(P, t, rows[wave]);
        wave_lds_order();
    }
}

// A wave per token, up to kMaxRouteBlocks blocks of four; more tokens go round.
constexpr int kMaxRouteBlocks = 1 << 20;

dim3 token_grid(int32_t T) {
    const int32_t blocks = ceil_div(T, 4);
    return dim3((uint32_t)(blocks < kMaxRouteBlocks ? blocks : kMaxRouteBlocks));
}

template <int NPL>
hipError_t launch_route_n(const RouteParams &P, bool fp32, hipStream_t stream) {
    const dim3 grid = token_grid(P.T);
    const size_t lds = P.keep < P.G ? (size_t)4 * P.E * sizeof(double) : 0;
    if (fp32)
        hipLaunchKernelGGL((route_kernel<NPL, true>), grid, dim3(256), lds, stream, P);
    else
        hipLaunchKernelGGL((route_kernel<NPL, false>), grid, dim3(256), lds, stream, P);
    return hipGetLastError();
}

template <int NPL>
hipError_t launch_grad_n(const RouteGradParams &P, bool fp32, hipStream_t stream) {
    const dim3 grid = token_grid(P.T);
    if (fp32)
        hipLaunchKernelGGL((route_grad_kernel<NPL, true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((route_grad_kernel<NPL, false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteParams &P, bool fp32, hipStream_t stream) {
    if (P.T == 0) return hipSuccess;
    return P.E <= 64    ? launch_route_n<1>(P, fp32, stream)
           : P.E <= 128 ? launch_route_n<2>(P, fp32, stream)
           : P.E <= 256 ? launch_route_n<4>(P, fp32, stream)
           : P.E <= 512 ? launch_route_n<8>(P, fp32, stream)
                        : launch_route_n<16>(P, fp32, stream);
}

hipError_t launch_route_grad(const RouteGradParams &P, bool fp32, hipStream_t stream) {
    if (P.T == 0) return hipSuccess;
    return P.E <= 64    ? launch_grad_n<1>(P, fp32, stream)
           : P.E <= 128 ? launch_grad_n<2>(P, fp32, stream)
           : P.E <= 256 ? launch_grad_n<4>(P, fp32, stream)
           : P.E <= 512 ? launch_grad_n<8>(P, fp32, stream)
                        : launch_grad_n<16>(P, fp32, stream);
}

}  // namespace epdc
