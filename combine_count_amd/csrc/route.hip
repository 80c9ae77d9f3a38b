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
constexpr float kLargest = 3.40282346638528859812e38f;
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

// A 32-bit value in the order of unsigned integers (no NaN; never 0 for a number).
__device__ __forceinline__ uint32_t order_of(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ (uint32_t)((int32_t)u >> 31 | (int32_t)0x80000000);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}
// Lanes 1 0 3 2, 2 3 0 1, 7 .. 0 of 8 and 15 .. 0 of 16: together an exchange among 16 lanes.
constexpr int kSwap1 = 0xB1, kSwap2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

template <int LPT>
__device__ __forceinline__ uint32_t token_max(uint32_t v) {
    v = max(v, dpp<kSwap1>(v));
    v = max(v, dpp<kSwap2>(v));
    v = max(v, dpp<kMirror8>(v));
    v = max(v, dpp<kMirror16>(v));
    if (LPT == 16) return v;
    const uint32_t a = max((uint32_t)__builtin_amdgcn_readlane((int)v, 0), (uint32_t)__builtin_amdgcn_readlane((int)v, 16));
    const uint32_t b = max((uint32_t)__builtin_amdgcn_readlane((int)v, 32), (uint32_t)__builtin_amdgcn_readlane((int)v, 48));
    return max(a, b);
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
            __builtin_amdgcn_sched_barrier(0);  // one exponential's registers, not all of them
        }
        sum = fmax(wave_sum(sum), 1.0);  // 1 or more unless every logit is masked
#pragma unroll
        for (int i = 0; i < NPL; ++i) s[i] /= sum;
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            s[i] = !(l[i] > -kInf) ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    const bool limited = P.keep < P.G;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = i * 64 + lane;
        double c = s[i];
        if (biased && e < P.E) c += (double)P.bias[e];
        if (!(l[i] > -kInf) || !(c > -kInf64)) c = -kInf64;
        key[i] = (c > -kInf64 && !biased ? (double)l[i] : c) + 0.0;  // -0 as +0
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
        // the largest (value, lower index) of the wave: its upper half, its lower half, its index
        const uint64_t u = (uint64_t)__double_as_longlong(best);
        const uint64_t o = u ^ (uint64_t)((int64_t)u >> 63 | (int64_t)(1ull << 63));
        const uint32_t hi = token_max<64>((uint32_t)(o >> 32));
        const uint32_t lo = token_max<64>((uint32_t)(o >> 32) == hi ? (uint32_t)o : 0u);
        at = (int)~token_max<64>(o == ((uint64_t)hi << 32 | lo) ? ~(uint32_t)at : 0u);
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

// ---- the fast form ----
//
// LPT lanes per token (16: four tokens a wave; 64), EPL experts per lane.  The
// rounds of the selection run on one 32-bit word per expert: the order of a
// 32-bit choice value (sigmoid + bias, or the logit itself without a bias),
// its lowest bits replaced by the expert's complement, so that words differ, a
// tie goes to the lower expert, and the winner of a round names itself.
//
// That is exact for bf16 logits (their 16 low bits are free).  Elsewhere the
// dropped bits and the 32-bit sigmoid can put neighbours the wrong way round;
// so
//   * the rounds go on past the K-th until the next value is out of its reach
//     (nearly always one round more);
//   * the candidates found, one per lane, are valued in 64 bits, and put in order
//     by that where neighbours' words are too close to tell; the same values give
//     the weights.
// A token that has a candidate in every lane, or whose last group kept and
// first group left out are closer than their scores can be off, is done again
// by route_token in 64 bits: one in some ten thousand of random logits, but
// every token of equal logits, or of one expert far above all others with
// groups by their two best, then at 163 and 227 us for 65521 tokens against 31
// and 39.
//
// A lane sorts its experts' words once; a round then compares one word per lane
// and moves the winner's list up by one.
//
// Bound by instructions, not bytes (1050 vector ones per wave of four tokens,
// which keep the vector units busy three quarters of the time): 16 lanes per
// token share each wave-wide maximum among four tokens.  65521 tokens, 256
// experts, top-8, 8 groups, bf16 (38 MB): 39 us, 180 with route_token for every
// token; 4096 tokens fp32 softmax 6.0 us against 13.9.

// The compare-exchanges of the odd-even merge sort (Batcher, "Sorting networks
// and their applications", 1968) of N values, N a power of two.
template <int N>
struct Network {
    int n = 0, a[N * N / 2] = {}, b[N * N / 2] = {};
    constexpr Network() {
        for (int p = 1; p < N; p *= 2)
            for (int k = p; k >= 1; k /= 2)
                for (int j = k % p; j + k < N; j += 2 * k)
                    for (int i = j; i < j + k && i + k < N; ++i)
                        if (i / (2 * p) == (i + k) / (2 * p)) a[n] = i, b[n] = i + k, ++n;
    }
};
template <int N>
__device__ __forceinline__ void sort_down(uint32_t (&v)[N]) {
    constexpr Network<N> net;
    each<net.n>([&](auto i) {
        constexpr int a = net.a[decltype(i)::value], b = net.b[decltype(i)::value];
        const uint32_t hi = max(v[a], v[b]), lo = min(v[a], v[b]);
        v[a] = hi;
        v[b] = lo;
    });
}

template <int LPT>
__device__ __forceinline__ double token_sum(double v) {
#pragma unroll
    for (int d = LPT / 2; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Sum over a token's 16 lanes, the same in all of them.
__device__ __forceinline__ float row_sum(float v) {
    v += __uint_as_float(dpp<kSwap1>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kSwap2>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kMirror8>(__float_as_uint(v)));
    v += __uint_as_float(dpp<kMirror16>(__float_as_uint(v)));
    return v;
}

template <int EPL, bool FP32>
__device__ __forceinline__ void load_logits(const uint8_t *p, float (&x)[EPL]) {
    if constexpr (FP32) {
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) {
            const u32x4 v = load16<true>(p + i * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i * 4 + j] = __uint_as_float(v[j]);
        }
    } else if constexpr (EPL == 4) {
        const u32x2 v = load8<true>(p);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < EPL / 8; ++i) {
            const u32x4 v = load16<true>(p + i * 16);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[i * 8 + j] = __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16);
        }
    }
}

// VEC: E = LPT * EPL and 16-byte aligned logits: a lane's experts are EPL in a
// row (so groups are whole lanes); else experts l, l + LPT, ...
// MODE: the scores (a compile-time choice for its registers: a softmax that is
// not renormalised takes a sum of 64-bit exponentials over all experts).
constexpr int kSigmoid = 0, kSoftmaxRenorm = 1, kSoftmax = 2;

template <int LPT, int EPL, bool VEC, bool FP32, int MODE>
__global__ __launch_bounds__(256) void route_fast_kernel(RouteParams P) {
    extern __shared__ double route_keys[];
    constexpr int kTokens = 64 / LPT;
    constexpr uint32_t kIndex = LPT * EPL - 1;  // the bits that hold the expert
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane & (LPT - 1), row0 = lane - l;
    const bool biased = P.bias != nullptr, limited = P.keep < P.G, sums = P.groupTop == 2;
    const int lanesPerGroup = limited ? P.perGroup / EPL : 1;
    const bool scored = biased || (limited && sums);  // 32-bit scores are needed
    float bias[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) bias[i] = 0.0f;
    if (biased) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) bias[i] = P.bias[VEC ? l * EPL + i : min(i * LPT + l, P.E - 1)];
    }
    for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * kTokens; t0 < P.T; t0 += (int64_t)gridDim.x * 4 * kTokens) {
        const bool live = t0 + lane / LPT < P.T;
        const int64_t t = live ? t0 + lane / LPT : P.T - 1;
        float x[EPL];
        if constexpr (VEC) {
            load_logits<EPL, FP32>(static_cast<const uint8_t *>(P.logits) + (t * P.E + l * EPL) * (FP32 ? 4 : 2), x);
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                x[i] = i * LPT + l < P.E ? load_logit<FP32>(P.logits, t * P.E + i * LPT + l) : -kInf;
        }
        float top = -kInf;  // the token's largest logit (softmax)
        if constexpr (MODE != kSigmoid) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) top = fmaxf(top, x[i]);
            const uint32_t o = token_max<LPT>(order_of(top));
            top = value_of(o);
        }
        // choice values; -inf where masked (NaN compares false)
        float c[EPL];
        if (scored) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                const float v = MODE != kSigmoid ? (x[i] == top ? 1.0f : __expf(x[i] - top)) : __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
                const float u = v + bias[i];
                c[i] = (x[i] > -kInf) & (u > -kInf) ? u : -kInf;
            }
        } else {
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = x[i] > -kInf ? x[i] + 0.0f : -kInf;  // -0 as +0
        }
        bool close = false;  // to be done again in 64 bits
        bool kept = true;    // the lane's group
        if (limited) {
            float a = -kInf, b = -kInf;  // the group's two best
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                b = __builtin_amdgcn_fmed3f(a, b, c[i]);
                a = fmaxf(a, c[i]);
            }
            for (int d = 1; d < lanesPerGroup; d <<= 1) {
                const float oa = __shfl_xor(a, d), ob = __shfl_xor(b, d);
                b = fmaxf(fminf(a, oa), fmaxf(b, ob));
                a = fmaxf(a, oa);
            }
            float size = fabsf(a);  // the largest term of the group's score
            if (sums && b > -kInf) {
                size = fmaxf(size, fabsf(b));
                a = fmaxf(a + b, -kLargest);  // a sum past the range is no masked group (its neighbours are close)
            }
            int better = 0;  // lanes of groups that go before this one
            for (int r = lanesPerGroup; r < LPT; r += lanesPerGroup) {
                const int from = (l + r) & (LPT - 1);
                const float o = __shfl(a, row0 + from);
                better += (o > a || (o == a && from < l)) ? 1 : 0;
            }
            kept = better < P.keep;
            if (scored) {
                // The last group kept and the first left out, each as far off as it can be.  A score: the exponential, the
                // sum and the reciprocal (1 ulp each, and the exponential's argument) under 2^-22 together, the bias'
                // addition half an ulp.  A group's score of two terms: twice that and half an ulp of the sum, which is
                // 2^-21 + 2^-22 times the larger term at most -- of the term, not of the sum: terms of opposite sign
                // cancel and their roundings stay.  Adding `off` rounds once more (2^-23 of the larger term).
                const float off = 0x1.9p-22f * fminf(size, kLargest) + 0x1.1p-21f;
                const float in = value_of(~token_max<LPT>(kept ? ~order_of(a - off) : 0u));
                const float out = value_of(token_max<LPT>(kept ? order_of(-kInf) : order_of(a + off)));
                if (out > -kInf && !(in > out)) close = true;
            }
        }
        uint32_t key[EPL], rest = kIndex - (VEC ? l * EPL : l);  // less i (times LPT): the expert's complement
        asm volatile("" : "+v"(rest));  // not EPL registers kept from token to token
        if (scored && !biased) {  // sums of scores for the groups, but experts go by their logits
#pragma unroll
            for (int i = 0; i < EPL; ++i) c[i] = c[i] > -kInf ? x[i] + 0.0f : -kInf;
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            key[i] = (c[i] > -kInf) & kept ? (order_of(c[i]) & ~kIndex) | (rest - (VEC ? i : i * LPT)) : 0u;
        sort_down(key);  // a lane's best is in front, and a round's winner moves up by one
        // Lane k: the k-th best.  K rounds; where words are not exact, more of them until the token's next one is out of
        // reach of its K-th: dropped bits, kIndex + 1 steps of 2^-23 each, and with a bias the scores' error as above.
        constexpr bool kExact = !FP32;  // of a logit: 16 bits of it, at most 10 of the expert
        const bool exact = kExact && !biased;
        auto off_of = [](float a, float b) { return 3.0f * (kIndex + 1) * 0x1p-23f * fmaxf(fabsf(a), fabsf(b)) + 0x1p-20f; };
        uint32_t win = 0, last = 0;
        int rounds = 0;
#pragma unroll 1
        for (int k = 0; k < LPT; ++k) {
            const uint32_t m = token_max<LPT>(key[0]);
            if (l == k) win = m;
            if (k == P.K - 1) last = m;
            rounds = k + 1;
            if (k >= P.K) {
                const float vi = value_of(last & ~kIndex), vo = value_of(m & ~kIndex);
                const bool open = m != 0 && !(vi - vo > (biased ? off_of(vi, vo) : 0.0f));
                if (!__any(open)) break;
                if (k == LPT - 1) close = close || open;
            } else if (exact && k == P.K - 1) {
                break;
            }
            const uint32_t won = key[0] == m ? ~0u : 0u;
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = ((i + 1 < EPL ? key[i + 1] : 0u) & won) | (key[i] & ~won);
        }
        {  // any lane's doubt is the token's
            const uint64_t doubts = __ballot(close);
            close = LPT == 64 ? doubts != 0 : (doubts >> row0 & 0xffff) != 0;
        }
        // in 64 bits: the candidates' scores, and what they are ordered by
        const bool found = win != 0;
        int32_t id = found ? (int32_t)(kIndex - (win & kIndex)) : -1;
        double s = 0.0, v = -kInf64;
        if (found) {
            const float xe = load_logit<FP32>(P.logits, t * P.E + id);
            if (MODE != kSigmoid)
                s = xe == top ? 1.0 : exp((double)xe - (double)top);
            else
                s = 1.0 / (1.0 + exp(-(double)xe));
            v = biased ? s + (double)P.bias[id] : (double)xe;
        }
        // the words' order is the values' wherever neighbours are further apart than they can be off
        bool doubt = false;
        if (!exact) {
            const uint32_t after = __shfl_down(win, 1, LPT);
            const float vi = value_of(win & ~kIndex), vo = value_of(after & ~kIndex);
            doubt = l + 1 < LPT && after != 0 && !(vi - vo > (biased ? off_of(vi, vo) : 0.0f));
        }
        int rank = l;
        if (__any(doubt)) {
            rank = 0;
            for (int k = 0; k < rounds; ++k) {
                const double o = __shfl(v, row0 + k);
                const int32_t oid = __shfl(id, row0 + k);
                rank += (o > v || (o == v && oid < id)) ? 1 : 0;
            }
            if (!found) rank = l;
        }
        if (rank >= P.K) s = 0.0;  // not among the chosen
        double w = s;
        if (MODE == kSoftmaxRenorm || (MODE == kSigmoid && P.renorm)) {
            const double total = token_sum<LPT>(s);
            w = total > 0.0 ? s / total : 0.0;
        } else if constexpr (MODE == kSoftmax) {
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                sum += !(x[i] > -kInf) ? 0.0 : x[i] == top ? 1.0 : exp((double)x[i] - (double)top);
                __builtin_amdgcn_sched_barrier(0);  // one exponential's registers, not all of them
            }
            w = s / fmax(token_sum<LPT>(sum), 1.0);
        }
        if (live && !close && rank < P.K) {
            const int64_t o = t * P.K + rank;
            P.expertIds[o] = id;
            P.weights[o] = (float)(w * (double)P.scale);
        }
        uint64_t again = __ballot(close && live && l == 0);
        while (again) {
            const int at = __builtin_ctzll(again);
            again &= again - 1;
            // the parameters afresh, opaque: nothing of this is computed ahead for the tokens that do not need it
            const RouteParams *Q = (const RouteParams *)__builtin_amdgcn_kernarg_segment_ptr();
            asm volatile("" : "+s"(Q));
            route_token<LPT * EPL / 64, FP32>(*Q, (int32_t)(t0 + at / LPT), route_keys + wave * Q->E);
        }
    }
}

template <int NPL, bool FP32>
__global__ __launch_bounds__(256) void route_kernel(RouteParams P) {
    extern __shared__ double route_keys[];
    const int wave = threadIdx.x >> 6;
    for (int64_t t = (int64_t)blockIdx.x * 4 + wave; t < P.T; t += (int64_t)gridDim.x * 4)
        route_token<NPL, FP32>(P, (int32_t)t, route_keys + wave * P.E);
}

// A chosen sigmoid as a multiple of one that all of the token's chosen share,
// exp(min(top, 0)), so that scores below the 32-bit range keep their shares of
// the sum; 0 where the score is 0 in 64 bits too (and for a slot without an
// expert, whose logit is -inf here).  big: 1 / (1 + exp(-|logit|)).
__device__ __forceinline__ float share(float logit, float top, float big) {
    return logit <= -709.78271f ? 0.0f : logit >= 0.0f ? big : expf(logit - fminf(top, 0.0f)) * big;
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
        if (!(sel > -kInf)) id = -1, sel = -kInf;  // a NaN too
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
            if (P.renorm) r = share(sel, wave_max(sel), big);
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

// The same for E = 16 EPL experts, at most 16 slots and 16-byte aligned rows:
// 16 lanes per token, four tokens a wave, so that a wave's instructions (what
// bounds the form above) serve four rows.  Slot k in lane k; the token's sums
// per expert in LDS, the slots added one after the other (a wave's LDS
// operations stay in order, so the order of the sum is the slots'); out as
// 16-byte pieces, one contiguous run of the row per store.
template <int EPL, bool FP32>
__global__ __launch_bounds__(256) void route_grad_rows_kernel(RouteGradParams P) {
    constexpr int E = 16 * EPL;
    constexpr int C = EPL < (FP32 ? 4 : 8) ? EPL : (FP32 ? 4 : 8);  // experts of a lane's piece
    constexpr int N = EPL / C;                                     // pieces of a lane: experts (i * 16 + l) * C ..
    __shared__ __attribute__((aligned(16))) float sums[16][E + 4];
    const int lane = threadIdx.x & 63, l = lane & 15, row0 = lane - l;
    float *row = sums[threadIdx.x >> 4];
    const bool dense = P.softmax && !P.renorm;
    for (int64_t t0 = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 6) * 4; t0 < P.T; t0 += (int64_t)gridDim.x * 16) {
        const bool live = t0 + (lane >> 4) < P.T;
        const int64_t t = live ? t0 + (lane >> 4) : P.T - 1;
        int32_t id = -1;
        float g = 0.0f, sel = -kInf;
        if (l < P.K) {
            id = P.expertIds[t * P.K + l];
            g = P.dWeights[t * P.K + l] * P.scale;
        }
        float x[EPL];
        if (dense) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float v[C];
                load_logits<C, FP32>(static_cast<const uint8_t *>(P.logits) + (t * E + (i * 16 + l) * C) * (FP32 ? 4 : 2), v);
#pragma unroll
                for (int j = 0; j < C; ++j) x[i * C + j] = v[j];
            }
        }
        if ((uint32_t)id < (uint32_t)E) sel = load_logit<FP32>(P.logits, t * E + id);
        if (!(sel > -kInf)) id = -1, sel = -kInf;  // a NaN too
#pragma unroll
        for (int i = 0; i < EPL / 4; ++i) *reinterpret_cast<u32x4 *>(row + (i * 16 + l) * 4) = u32x4{0, 0, 0, 0};
        float d, dot = 0.0f;
        if (dense) {
            float top = -kInf;
#pragma unroll
            for (int i = 0; i < EPL; ++i) top = fmaxf(top, x[i]);
            top = value_of(token_max<16>(order_of(top)));
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                x[i] = !(x[i] > -kInf) ? 0.0f : x[i] == top ? 1.0f : expf(x[i] - top);
                sum += x[i];
            }
            const float inv = 1.0f / fmaxf(row_sum(sum), 1.0f);
#pragma unroll
            for (int i = 0; i < EPL; ++i) x[i] *= inv;
            d = id >= 0 ? g : 0.0f;
            dot = row_sum(id < 0 ? 0.0f : g * (sel == top ? 1.0f : expf(sel - top)) * inv);
        } else {
            float r, q = 1.0f;
            if (P.softmax) {
                const float top = value_of(token_max<16>(order_of(sel)));
                r = id < 0 ? 0.0f : sel == top ? 1.0f : expf(sel - top);
            } else {
                const float e = expf(-fabsf(sel)), big = 1.0f / (1.0f + e), small = e * big;
                r = id < 0 ? 0.0f : sel >= 0.0f ? big : small;
                q = sel >= 0.0f ? small : big;
                if (P.renorm) r = share(sel, value_of(token_max<16>(order_of(sel))), big);
            }
            float mean = 0.0f;
            if (P.renorm) {
                const float total = row_sum(r);
                r = total > 0.0f ? r / total : 0.0f;
                mean = row_sum(id >= 0 ? g * r : 0.0f);
            }
            d = id >= 0 ? r * q * (g - mean) : 0.0f;
        }
        wave_lds_order();
        for (int k = 0; k < P.K; ++k)
            if (l == k && id >= 0) __hip_atomic_fetch_add(row + id, d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        wave_lds_order();
        if (live) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                uint32_t w[C];
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    float v = row[(i * 16 + l) * C + j];
                    if (dense) v = x[i * C + j] * (v - dot);
                    w[j] = FP32 ? __float_as_uint(v) : bf16_rne(v);
                }
                uint8_t *out = static_cast<uint8_t *>(P.dLogits) + (t * E + (i * 16 + l) * C) * (FP32 ? 4 : 2);
                if constexpr (FP32)
                    store16<true>(out, u32x4{w[0], w[1], w[2], w[3]});
                else if constexpr (C == 8)
                    store16<true>(out, u32x4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16});
                else
                    store8<true>(out, u32x2{w[0] | w[1] << 16, w[2] | w[3] << 16});
            }
        }
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

template <int LPT, int EPL, bool VEC, int MODE>
hipError_t launch_fast_mode(const RouteParams &P, bool fp32, hipStream_t stream) {
    const dim3 grid = token_grid(ceil_div(P.T, 64 / LPT));
    const size_t lds = P.keep < P.G ? (size_t)4 * P.E * sizeof(double) : 0;
    if (fp32)
        hipLaunchKernelGGL((route_fast_kernel<LPT, EPL, VEC, true, MODE>), grid, dim3(256), lds, stream, P);
    else
        hipLaunchKernelGGL((route_fast_kernel<LPT, EPL, VEC, false, MODE>), grid, dim3(256), lds, stream, P);
    return hipGetLastError();
}

template <int LPT, int EPL, bool VEC>
hipError_t launch_fast(const RouteParams &P, bool fp32, hipStream_t stream) {
    return !P.softmax ? launch_fast_mode<LPT, EPL, VEC, kSigmoid>(P, fp32, stream)
           : P.renorm ? launch_fast_mode<LPT, EPL, VEC, kSoftmaxRenorm>(P, fp32, stream)
                      : launch_fast_mode<LPT, EPL, VEC, kSoftmax>(P, fp32, stream);
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

template <int EPL>
hipError_t launch_grad_rows(const RouteGradParams &P, bool fp32, hipStream_t stream) {
    const dim3 grid = token_grid(ceil_div(P.T, 4));
    if (fp32)
        hipLaunchKernelGGL((route_grad_rows_kernel<EPL, true>), grid, dim3(256), 0, stream, P);
    else
        hipLaunchKernelGGL((route_grad_rows_kernel<EPL, false>), grid, dim3(256), 0, stream, P);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteParams &P, bool fp32, hipStream_t stream) {
    if (P.T == 0) return hipSuccess;
    const RoutePlan pl = plan_route(P.E, P.K, P.G, P.keep, P.T, P.softmax, P.bias != nullptr,
                                    reinterpret_cast<uintptr_t>(P.logits) % 16 == 0);
    if (pl.lanes == 16 && pl.inRow)
        return pl.perLane == 4   ? launch_fast<16, 4, true>(P, fp32, stream)
               : pl.perLane == 8 ? launch_fast<16, 8, true>(P, fp32, stream)
                                 : launch_fast<16, 16, true>(P, fp32, stream);
    if (pl.lanes == 16)
        return pl.perLane == 4   ? launch_fast<16, 4, false>(P, fp32, stream)
               : pl.perLane == 8 ? launch_fast<16, 8, false>(P, fp32, stream)
                                 : launch_fast<16, 16, false>(P, fp32, stream);
    if (pl.lanes == 64 && pl.inRow) return launch_fast<64, 4, true>(P, fp32, stream);
    if (pl.lanes == 64)
        return pl.perLane == 4   ? launch_fast<64, 4, false>(P, fp32, stream)
               : pl.perLane == 8 ? launch_fast<64, 8, false>(P, fp32, stream)
                                 : launch_fast<64, 16, false>(P, fp32, stream);
    return pl.perLane == 1   ? launch_route_n<1>(P, fp32, stream)
           : pl.perLane == 2 ? launch_route_n<2>(P, fp32, stream)
           : pl.perLane == 4 ? launch_route_n<4>(P, fp32, stream)
           : pl.perLane == 8 ? launch_route_n<8>(P, fp32, stream)
                             : launch_route_n<16>(P, fp32, stream);
}

hipError_t launch_route_grad(const RouteGradParams &P, bool fp32, hipStream_t stream) {
    if (P.T == 0) return hipSuccess;
    const RoutePlan pl = plan_route_grad(P.E, P.K, reinterpret_cast<uintptr_t>(P.logits) % 16 == 0 &&
                                                       reinterpret_cast<uintptr_t>(P.dLogits) % 16 == 0);
    if (pl.lanes == 16)
        return pl.perLane == 4   ? launch_grad_rows<4>(P, fp32, stream)
               : pl.perLane == 8 ? launch_grad_rows<8>(P, fp32, stream)
                                 : launch_grad_rows<16>(P, fp32, stream);
    return pl.perLane == 1   ? launch_grad_n<1>(P, fp32, stream)
           : pl.perLane == 2 ? launch_grad_n<2>(P, fp32, stream)
           : pl.perLane == 4 ? launch_grad_n<4>(P, fp32, stream)
           : pl.perLane == 8 ? launch_grad_n<8>(P, fp32, stream)
                             : launch_grad_n<16>(P, fp32, stream);
}

}  // namespace epdc
