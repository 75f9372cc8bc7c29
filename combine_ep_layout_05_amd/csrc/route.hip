// route.hip -- the router: each token's K experts and their weights from its
// E logits, and the gradient with respect to the logits (gfx950).
//
// A token's row lives in the registers of a group of 64 or 16 lanes (4 tokens
// per wave), each lane holding kPer neighbouring logits, so the row is read
// once and never leaves the group.  Selection is K rounds of "largest key
// left, lowest index on ties" over keys that are unsigned integers ordered
// like the values (0 = cannot be chosen): the group's maximum, then the lowest
// index that holds it, both DPP reductions.  The kernels are bound by these
// instructions, not by bytes: 64 lanes keep a single token's chain short, 16
// lanes do a third of the instructions per token (most of a round is the
// reduction) and are taken when there are enough tokens to fill the GPU.
#include <type_traits>

#include "ep_device.h"
#include "ep_launch.h"
#include "ep_numerics.h"

namespace ep {
namespace {

constexpr int kRouteWaves = 4;
constexpr int kRow = 16;                  // lanes of a DPP row
static_assert(kMaxTopK <= kRow, "a token's choices fit the first row of its group");

// Unsigned keys in the order of the values.  -0 counts as +0 (equal values
// have equal keys); -inf and NaN give 0, below every value that can be chosen.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (!(v > -__builtin_inff())) return 0u;
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);      // -0 + 0 = +0
    return (b >> 31) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __builtin_bit_cast(float, (k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ uint64_t order_key(double v)
{
    if (!(v > -__builtin_inf())) return 0ull;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// Maximum over the group, in every lane (butterfly within the 16-lane DPP
// rows; a group of 64 then joins its four rows by lane reads).
template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t v)
{
    v = __builtin_elementwise_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = __builtin_elementwise_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    v = __builtin_elementwise_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
    v = __builtin_elementwise_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    if constexpr (kLanes == kWave) {
        const uint32_t a = (uint32_t)read_lane((int)v, 0), b = (uint32_t)read_lane((int)v, 16);
        const uint32_t c = (uint32_t)read_lane((int)v, 32), d = (uint32_t)read_lane((int)v, 48);
        const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
        v = ab > cd ? ab : cd;
    }
    return v;
}

// Sum over the group in every lane, in a fixed order.
template <int kLanes>
__device__ __forceinline__ float group_sum(float v)
{
    auto moved = [](float x, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x),
                                                                     decltype(ctrl)::value, 0xF, 0xF, false));
    };
    v += moved(v, std::integral_constant<int, 0xB1>());
    v += moved(v, std::integral_constant<int, 0x4E>());
    v += moved(v, std::integral_constant<int, 0x141>());
    v += moved(v, std::integral_constant<int, 0x140>());
    if constexpr (kLanes == kWave) {
        const int b = __builtin_bit_cast(int, v);
        v = (__builtin_bit_cast(float, read_lane(b, 0)) + __builtin_bit_cast(float, read_lane(b, 16))) +
            (__builtin_bit_cast(float, read_lane(b, 32)) + __builtin_bit_cast(float, read_lane(b, 48)));
    }
    return v;
}

// +inf counts as the largest finite value, so that a row's maximum is finite
// and exp(l - max) is never inf - inf.
__device__ __forceinline__ float finite_top(float v)
{
    return v == __builtin_inff() ? 3.4028234663852886e38f : v;
}

template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t i)
{
    if constexpr (kBf16) return finite_top(__builtin_bit_cast(float, (uint32_t)((const uint16_t*)logits)[i] << 16));
    else return finite_top(((const float*)logits)[i]);
}

// kPer neighbouring elements of a lane as one access (4, 8 or 16 bytes, or
// pieces of 16); the launcher says when the rows are aligned for it.
template <int kPer, bool kBf16> struct LanePiece {
    static constexpr int kBytes = kPer * (kBf16 ? 2 : 4);
    static constexpr bool kVector = kBytes >= 4 && (kBytes & (kBytes - 1)) == 0;
    static constexpr int kAlign = kBytes < 16 ? kBytes : 16;
    struct __attribute__((aligned(kVector ? kAlign : 2))) Words {
        uint32_t u[kVector ? kBytes / 4 : 1];
    };
};

// The lane's logits l[j] of experts e0 + j, -inf past E.
template <int kPer, bool kBf16>
__device__ __forceinline__ void load_row(float (&l)[kPer], const void* logits, int64_t row, int E,
                                         int e0, bool vector)
{
    using P = LanePiece<kPer, kBf16>;
    if (P::kVector && vector) {                 // E is a multiple of kPer: all or none of the lane's
        typename P::Words w{};
        if (e0 < E) w = *(const typename P::Words*)((const char*)logits + (row + e0) * (kBf16 ? 2 : 4));
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t u = w.u[P::kVector ? (kBf16 ? j / 2 : j) : 0];
            const float v = kBf16 ? (j % 2 ? bf16_hi(u) : bf16_lo(u)) : __builtin_bit_cast(float, u);
            l[j] = e0 < E ? finite_top(v) : -__builtin_inff();
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            l[j] = e0 + j < E ? load_logit<kBf16>(logits, row + e0 + j) : -__builtin_inff();
    }
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// kLanes lanes per token, kPer logits per lane (E <= kLanes * kPer).  kBias:
// the keys are sigmoid(l) + bias in 64 bits: in 32 bits two scores next to
// each other could round to the same sum, or to sums in the other order.
template <int kLanes, int kPer, bool kBf16, bool kSigmoid, bool kBias>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(
    const void* __restrict__ logits, const float* __restrict__ bias, int T, int E, int K,
    int renorm, float scale, int vector, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w)
{
    constexpr int kTokens = kWave / kLanes;
    const int lane = threadIdx.x % kWave, g = lane % kLanes, e0 = g * kPer;
    const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + wave_uniform(threadIdx.x / kWave);
    for (int64_t first = wave * kTokens; first < T; first += (int64_t)gridDim.x * kRouteWaves * kTokens) {
        const bool mine = first + lane / kLanes < T;         // (the last wave's groups past the end
        const int64_t t = mine ? first + lane / kLanes : T - 1;   // do the last token again, unstored)
        float l[kPer];
        load_row<kPer, kBf16>(l, logits, t * E, E, e0, vector != 0);
        uint32_t hi[kPer], lo[kBias ? kPer : 1];
        bool nan = false;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            nan |= l[j] != l[j];
            hi[j] = order_key(l[j]);
            if constexpr (kBias) {
                const double b = e0 + j < E ? (double)bias[e0 + j] : 0.0;
                const uint64_t k = hi[j] ? order_key(1.0 / (1.0 + exp(-(double)l[j])) + b) : 0ull;
                hi[j] = (uint32_t)(k >> 32);
                lo[j] = (uint32_t)k;
            }
        }
        const uint64_t group_lanes = kLanes == kWave ? ~0ull : 0xFFFFull << (lane & ~(kRow - 1));
        const bool row_nan = (__ballot(nan) & group_lanes) != 0;

        int my_id = -1;                       // lane k of the group: the k-th expert, its logit's key
        uint32_t my_key = 0, first_key = 0;
        for (int k = 0; k < K; ++k) {
            uint32_t best = hi[0];
#pragma unroll
            for (int j = 1; j < kPer; ++j) best = __builtin_elementwise_max(best, hi[j]);
            const uint32_t top = group_max<kLanes>(best);
            if (k == 0) first_key = top;
            if (kLanes == kWave && top == 0) break;          // nothing left to choose
            uint32_t low = 0;
            if constexpr (kBias) {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    low = __builtin_elementwise_max(low, hi[j] == top ? lo[j] : 0u);
                low = group_max<kLanes>(low);
            }
            // the lowest index that holds it: lanes and registers are in index order
            uint32_t e = 0x7FFFFFFFu;
#pragma unroll
            for (int j = kPer - 1; j >= 0; --j)
                if (hi[j] == top && (!kBias || lo[kBias ? j : 0] == low)) e = (uint32_t)(e0 + j);
            e = ~group_max<kLanes>(~e);
            if (g == k && top != 0) { my_id = (int)e; my_key = top; }
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if ((int)e - e0 == j) hi[j] = 0;
        }

        // the choices are lanes 0 .. K - 1 of the group: one DPP row
        float w = 0.0f, total = 1.0f;
        if constexpr (kSigmoid) {
            float my_l = 0.0f;
            if (my_id >= 0) my_l = kBias ? load_logit<kBf16>(logits, t * E + my_id) : key_value(my_key);
            w = my_id >= 0 ? sigmoid(my_l) : 0.0f;
            if (renorm) total = group_sum<kRow>(w);
        } else {
            const float m = first_key != 0 ? key_value(first_key) : 0.0f;   // the row's largest logit
            w = my_id >= 0 ? expf(key_value(my_key) - m) : 0.0f;
            if (renorm) {
                total = group_sum<kRow>(w);
            } else {
                float z = 0.0f;
#pragma unroll
                for (int j = 0; j < kPer; ++j) z += l[j] > -__builtin_inff() ? expf(l[j] - m) : 0.0f;
                total = group_sum<kLanes>(z);
            }
        }
        if (g < K && mine) {
            float v = 0.0f;
            if (my_id >= 0) v = row_nan ? __builtin_nanf("") : scale * (total > 0.0f ? w / total : 0.0f);
            topk_idx[t * K + g] = my_id;
            topk_w[t * K + g] = v;
        }
    }
}

// The gradient: with q the (renormalised) weights before scaling and
// dot = sum_k g_k q_k,
//   softmax            dl_e = scale * q_e * ([e chosen] g_e - dot)
//   softmax, renorm    dl_{i_k} = scale * q_k * (g_k - dot)
//   sigmoid            dl_{i_k} = scale * g_k * p_k * (1 - p_k)
//   sigmoid, renorm    dl_{i_k} = scale * q_k * (1 - p_k) * (g_k - dot)
// and 0 elsewhere.  An expert named twice in a row gets both terms.
template <int kLanes, int kPer, bool kBf16, bool kSigmoid, bool kRenorm>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_backward_kernel(
    const void* __restrict__ logits, int T, int E, int K, float scale, int vector,
    const int32_t* __restrict__ topk_idx, const float* __restrict__ grad_w,
    void* __restrict__ grad_logits)
{
    constexpr int kTokens = kWave / kLanes;
    const int lane = threadIdx.x % kWave, g = lane % kLanes, e0 = g * kPer;
    const int64_t wave = (int64_t)blockIdx.x * kRouteWaves + wave_uniform(threadIdx.x / kWave);
    for (int64_t first = wave * kTokens; first < T; first += (int64_t)gridDim.x * kRouteWaves * kTokens) {
        const bool mine = first + lane / kLanes < T;
        const int64_t t = mine ? first + lane / kLanes : T - 1;
        const int kl = g < K ? g : 0;
        int id = topk_idx[t * K + kl];
        float up = grad_w[t * K + kl];
        if (g >= K || id < 0 || id >= E) { id = -1; up = 0.0f; }
        const float lk = id >= 0 ? load_logit<kBf16>(logits, t * E + id) : -__builtin_inff();

        float out[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) out[j] = 0.0f;
        float d;                                               // lane k: the term of entry k
        if constexpr (kSigmoid) {
            const float p = id >= 0 ? sigmoid(lk) : 0.0f;
            const float r = id >= 0 ? 1.0f / (1.0f + expf(lk)) : 0.0f;      // 1 - p, without cancellation
            if constexpr (kRenorm) {
                const float total = group_sum<kRow>(p);
                const float q = total > 0.0f ? p / total : (total != total ? total : 0.0f);
                d = scale * q * r * (up - group_sum<kRow>(up * q));
            } else {
                d = scale * up * p * r;
            }
        } else if constexpr (kRenorm) {
            // order_key puts NaN lowest: a NaN among the chosen reaches the sum by itself
            const uint32_t mk = group_max<kRow>(order_key(lk));
            const float m = mk == 0 ? 0.0f : key_value(mk);
            const float w = id >= 0 && lk != -__builtin_inff() ? expf(lk - m) : 0.0f;
            const float total = group_sum<kRow>(w);
            const float q = total > 0.0f ? w / total : (total != total ? total : 0.0f);
            d = scale * q * (up - group_sum<kRow>(up * q));
        } else {
            float l[kPer];
            load_row<kPer, kBf16>(l, logits, t * E, E, e0, vector != 0);
            uint32_t mk = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) mk = __builtin_elementwise_max(mk, order_key(l[j]));
            mk = group_max<kLanes>(mk);
            const float m = mk == 0 ? 0.0f : key_value(mk);
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                out[j] = l[j] == -__builtin_inff() ? 0.0f : expf(l[j] - m);
                z += out[j];
            }
            z = group_sum<kLanes>(z);
            const float inv = z > 0.0f ? 1.0f / z : (z != z ? z : 0.0f);
            const float q = id >= 0 && lk != -__builtin_inff() ? expf(lk - m) * inv : 0.0f;
            const float dot = group_sum<kLanes>(up * q);       // 0 past the first row
#pragma unroll
            for (int j = 0; j < kPer; ++j) out[j] = -scale * (out[j] * inv) * dot;
            d = scale * q * up;
        }
        if (id < 0) d = 0.0f;
        for (int k = 0; k < K; ++k) {
            int e;
            float dk;
            if constexpr (kLanes == kWave) {
                e = read_lane(id, k);
                dk = __builtin_bit_cast(float, read_lane(__builtin_bit_cast(int, d), k));
            } else {
                e = __shfl(id, (lane & ~(kRow - 1)) + k);
                dk = __shfl(d, (lane & ~(kRow - 1)) + k);
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (e - e0 == j) out[j] += dk;
        }
        if (!mine) continue;
        using P = LanePiece<kPer, kBf16>;
        char* const o = (char*)grad_logits + (t * E + e0) * (kBf16 ? 2 : 4);
        if (P::kVector && vector) {
            typename P::Words w;
#pragma unroll
            for (int i = 0; i < (P::kVector ? P::kBytes / 4 : 1); ++i)
                w.u[i] = kBf16 ? pack2_bf16(out[(2 * i) % kPer], out[(2 * i + 1) % kPer])
                               : __builtin_bit_cast(uint32_t, out[i % kPer]);
            if (e0 < E) *(typename P::Words*)o = w;
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if (e0 + j >= E) continue;
                if constexpr (kBf16) ((uint16_t*)o)[j] = __builtin_bit_cast(uint16_t, (__bf16)out[j]);
                else ((float*)o)[j] = out[j];
            }
        }
    }
}

// Whether a token gets 16 lanes (four tokens a wave) instead of 64: enough
// tokens to fill the GPU all the same, and few enough logits per lane.
// Measured on MI355X, top-8, graphs of 50 launches, 64 / 16 lanes: choice of
// 1024 tokens x 128 fp32 3.3 / 3.5 us, 4096 x 128 4.7 / 3.6, 4096 x 256 5.3 /
// 4.6, 16384 x 128 bf16 12.5 / 6.4; gradient (stores of 16 bytes per lane,
// one row's lanes side by side) 4096 x 128 fp32 3.4 / 3.4 us, 16384 x 128 bf16
// 8.4 / 5.9, 16384 x 256 fp32 8.8 / 10.0 and bf16 8.3 / 6.1.
bool route_narrow(int T, int E) { return T >= 4096 && E <= 16 * kRow; }
bool route_backward_narrow(int T, int E, bool bf16) { return T >= 8192 && E * (bf16 ? 2 : 4) <= 512; }

// The launch of `kernel` and whether its lanes may load their logits at once.
template <int kLanes, int kPer, bool kBf16>
int route_vector(int E, const void* a, const void* b)
{
    using P = LanePiece<kPer, kBf16>;
    const uintptr_t mask = P::kAlign - 1;
    return P::kVector && E % kPer == 0 && ((uintptr_t)E * (kBf16 ? 2 : 4) & mask) == 0 &&
           ((uintptr_t)a & mask) == 0 && ((uintptr_t)b & mask) == 0;
}

template <int kLanes>
unsigned route_blocks(int T)
{
    constexpr int kTokens = kRouteWaves * (kWave / kLanes);
    const int64_t blocks = ((int64_t)T + kTokens - 1) / kTokens;
    return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
}

template <int kLanes, int kPer, bool kBf16>
void route_launch(const void* logits, int T, int E, int K, bool sigmoid_score, const float* bias,
                  int renorm, float scale, int32_t* topk_idx, float* topk_w, hipStream_t stream)
{
    const int vector = route_vector<kLanes, kPer, kBf16>(E, logits, nullptr);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(route_blocks<kLanes>(T)), dim3(kRouteWaves * kWave), 0,
                           stream, logits, bias, T, E, K, renorm, scale, vector, topk_idx, topk_w);
    };
    if (bias) go(route_kernel<kLanes, kPer, kBf16, true, true>);
    else if (sigmoid_score) go(route_kernel<kLanes, kPer, kBf16, true, false>);
    else go(route_kernel<kLanes, kPer, kBf16, false, false>);
}

template <int kLanes, int kPer, bool kBf16>
void route_backward_launch(const void* logits, int T, int E, int K, bool sigmoid_score, int renorm,
                           float scale, const int32_t* topk_idx, const float* grad_w,
                           void* grad_logits, hipStream_t stream)
{
    const int vector = route_vector<kLanes, kPer, kBf16>(E, logits, grad_logits);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(route_blocks<kLanes>(T)), dim3(kRouteWaves * kWave), 0,
                           stream, logits, T, E, K, scale, vector, topk_idx, grad_w, grad_logits);
    };
    if (sigmoid_score)
        renorm ? go(route_backward_kernel<kLanes, kPer, kBf16, true, true>)
               : go(route_backward_kernel<kLanes, kPer, kBf16, true, false>);
    else
        renorm ? go(route_backward_kernel<kLanes, kPer, kBf16, false, true>)
               : go(route_backward_kernel<kLanes, kPer, kBf16, false, false>);
}

// Calls f(lanes, logits per lane) with the smallest instance that holds E logits.
// Besides the powers of two there is one of 5 (257 to 320 experts with 64 lanes,
// 65 to 80 with 16).  Measured with 5 / 6 / 8 logits per lane, top-8 of 288
// experts in fp32, graphs of 50 launches: 128 tokens 3.8 / 4.0 / 3.9 us, with a
// bias 5.9 / 6.5 / 6.6, 16384 tokens 15.6 / 16.7 / 18.4, with a bias 29 / 33 / 39,
// full softmax gradient 16.1 / 17.8 / 17.0; the renormalised gradient alone is
// slower, 13.1 / 14.7 / 11.4 (its stores are not vectors).  One of 6 for 321 to
// 384 would serve a bias at many tokens (16384 x 384 34 for 39 us) and cost the
// fp32 gradients more (17.4 for 11.8).
template <class F>
void with_shape(bool narrow, int E, F&& f)
{
    auto per = [&](auto lanes, int n) {
        if (n <= 1) f(lanes, std::integral_constant<int, 1>());
        else if (n <= 2) f(lanes, std::integral_constant<int, 2>());
        else if (n <= 4) f(lanes, std::integral_constant<int, 4>());
        else if (n <= 5) f(lanes, std::integral_constant<int, 5>());
        else if (n <= 8) f(lanes, std::integral_constant<int, 8>());
        else f(lanes, std::integral_constant<int, 16>());
    };
    if (narrow) per(std::integral_constant<int, kRow>(), (E + kRow - 1) / kRow);
    else per(std::integral_constant<int, kWave>(), (E + kWave - 1) / kWave);
}

}  // namespace

hipError_t launch_route(const void* logits, bool bf16, int T, int E, int K, bool sigmoid_score,
                        const float* bias, bool renorm, float scale, int32_t* topk_idx,
                        float* topk_w, hipStream_t stream)
{
    with_shape(route_narrow(T, E), E, [&](auto lanes, auto per) {
        constexpr int kL = decltype(lanes)::value, kP = decltype(per)::value;
        bf16 ? route_launch<kL, kP, true>(logits, T, E, K, sigmoid_score, bias, renorm ? 1 : 0,
                                          scale, topk_idx, topk_w, stream)
             : route_launch<kL, kP, false>(logits, T, E, K, sigmoid_score, bias, renorm ? 1 : 0,
                                           scale, topk_idx, topk_w, stream);
    });
    return hipGetLastError();
}

hipError_t launch_route_backward(const void* logits, bool bf16, int T, int E, int K,
                                 bool sigmoid_score, bool renorm, float scale,
                                 const int32_t* topk_idx, const float* grad_w, void* grad_logits,
                                 hipStream_t stream)
{
    with_shape(route_backward_narrow(T, E, bf16), E, [&](auto lanes, auto per) {
        constexpr int kL = decltype(lanes)::value, kP = decltype(per)::value;
        bf16 ? route_backward_launch<kL, kP, true>(logits, T, E, K, sigmoid_score, renorm ? 1 : 0,
                                                   scale, topk_idx, grad_w, grad_logits, stream)
             : route_backward_launch<kL, kP, false>(logits, T, E, K, sigmoid_score, renorm ? 1 : 0,
                                                    scale, topk_idx, grad_w, grad_logits, stream);
    });
    return hipGetLastError();
}

}  // namespace ep
