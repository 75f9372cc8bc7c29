// route.hip -- the router: each token's K experts and their weights from its
// E logits, and the gradient with respect to the logits (gfx950).
//
// One wave per token; lane i holds the logits of experts i, i + 64, ... in
// registers (at most 16), so a token's row is read once, coalesced, and never
// leaves the wave.  Selection is K rounds of "largest key left, lowest index
// on ties" over keys that are unsigned integers ordered like the values
// (0 = cannot be chosen): per round a maximum over the lane's own keys, a DPP
// maximum over the wave, and a ballot for the lane that holds it.
#include "ep_device.h"
#include "ep_launch.h"
#include "ep_numerics.h"

namespace ep {
namespace {

constexpr int kRouteWaves = 4;

// Unsigned keys in the order of the values.  -0 counts as +0 (equal values
// have equal keys); -inf and NaN give 0, below every value that can be chosen.
__device__ __forceinline__ uint32_t order_key(float v)
{
    if (!(v > -__builtin_inff())) return 0u;
    const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);      // -0 + 0 = +0
    return (b >> 31) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint64_t order_key(double v)
{
    if (!(v > -__builtin_inf())) return 0ull;
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// Maximum over the wave, in every lane (butterfly within the 16-lane DPP
// rows, then the row maxima by lane reads).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    v = __builtin_elementwise_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    v = __builtin_elementwise_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
    v = __builtin_elementwise_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
    v = __builtin_elementwise_max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
    const uint32_t a = (uint32_t)read_lane((int)v, 0), b = (uint32_t)read_lane((int)v, 16);
    const uint32_t c = (uint32_t)read_lane((int)v, 32), d = (uint32_t)read_lane((int)v, 48);
    const uint32_t ab = a > b ? a : b, cd = c > d ? c : d;
    return ab > cd ? ab : cd;
}

__device__ __forceinline__ float dpp_add(float v, float moved) { return v + moved; }

__device__ __forceinline__ float wave_sum(float v)
{
#define EP_DPP_F(x, ctrl) __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, 0xF, 0xF, false))
    v = dpp_add(v, EP_DPP_F(v, 0xB1));
    v = dpp_add(v, EP_DPP_F(v, 0x4E));
    v = dpp_add(v, EP_DPP_F(v, 0x141));
    v = dpp_add(v, EP_DPP_F(v, 0x140));
#undef EP_DPP_F
    const int b = __builtin_bit_cast(int, v);
    return (__builtin_bit_cast(float, read_lane(b, 0)) + __builtin_bit_cast(float, read_lane(b, 16))) +
           (__builtin_bit_cast(float, read_lane(b, 32)) + __builtin_bit_cast(float, read_lane(b, 48)));
}

// The maximum of the wave's keys and the lanes that hold it.
__device__ __forceinline__ uint64_t lanes_of_max(uint32_t key, uint32_t& top)
{
    top = wave_max_u32(key);
    return __ballot(key == top);
}

__device__ __forceinline__ uint64_t lanes_of_max(uint64_t key, uint64_t& top)
{
    const uint32_t hi = wave_max_u32((uint32_t)(key >> 32));
    const bool in = (uint32_t)(key >> 32) == hi;
    const uint32_t lo = wave_max_u32(in ? (uint32_t)key : 0u);
    top = ((uint64_t)hi << 32) | lo;
    return __ballot(in && (uint32_t)key == lo);
}

// One logit; +inf counts as the largest finite value, so that a row's maximum
// is finite and exp(l - max) is never inf - inf.
template <bool kBf16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t i)
{
    float v;
    if constexpr (kBf16) v = __builtin_bit_cast(float, (uint32_t)((const uint16_t*)logits)[i] << 16);
    else v = ((const float*)logits)[i];
    return v == __builtin_inff() ? 3.4028234663852886e38f : v;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// kPer: logits per lane (E <= 64 * kPer).  kBias: the keys are
// sigmoid(l) + bias in 64 bits: in 32 bits two scores next to each other
// could round to the same sum, or to sums in the other order.
template <int kPer, bool kBf16, bool kSigmoid, bool kBias>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_kernel(
    const void* __restrict__ logits, const float* __restrict__ bias, int T, int E, int K,
    int renorm, float scale, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w)
{
    using Key = typename std::conditional<kBias, uint64_t, uint32_t>::type;
    const int lane = threadIdx.x % kWave;
    for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave_uniform(threadIdx.x / kWave); t < T;
         t += (int64_t)gridDim.x * kRouteWaves) {
    float l[kPer];
    Key key[kPer];
    bool nan = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = j * kWave + lane;
        l[j] = e < E ? load_logit<kBf16>(logits, t * E + e) : -__builtin_inff();
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = j * kWave + lane;
        nan |= l[j] != l[j];
        if constexpr (kBias) {
            const double s = 1.0 / (1.0 + exp(-(double)l[j])) + (double)(e < E ? bias[e] : 0.0f);
            key[j] = order_key(l[j]) ? order_key(s) : 0ull;
        } else {
            key[j] = order_key(l[j]);
        }
    }
    const bool row_nan = __ballot(nan) != 0;

    int my_id = -1;                       // lane k: the k-th expert and its logit
    float my_l = -__builtin_inff();
    for (int k = 0; k < K; ++k) {
        Key best = key[0];
        int bj = 0;
        float bl = l[0];
#pragma unroll
        for (int j = 1; j < kPer; ++j)
            if (key[j] > best) { best = key[j]; bj = j; bl = l[j]; }
        Key top;
        uint64_t who = lanes_of_max(best, top);
        if (top == 0) break;              // nothing left to choose
        int win = __builtin_ctzll(who);
        if (who & (who - 1)) {            // several lanes: the lowest expert index
            int e = ((who >> lane) & 1ull) ? bj * kWave + lane : 0x7FFFFFFF;
            const uint32_t lowest = ~wave_max_u32(~(uint32_t)e);
            win = (int)lowest % kWave;
        }
        const int sel = read_lane(bj, win) * kWave + win;
        const float sl = __builtin_bit_cast(float, read_lane(__builtin_bit_cast(int, bl), win));
        if (lane == k) { my_id = sel; my_l = sl; }
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j * kWave + lane == sel) key[j] = 0;
    }

    float w = 0.0f, total = 1.0f;
    if constexpr (kSigmoid) {
        w = my_id >= 0 ? sigmoid(my_l) : 0.0f;
        if (renorm) total = wave_sum(w);
    } else {
        // the first choice has the row's largest logit
        const float m = __builtin_bit_cast(float, read_lane(__builtin_bit_cast(int, my_l), 0));
        w = my_id >= 0 ? expf(my_l - m) : 0.0f;
        if (renorm) {
            total = wave_sum(w);
        } else {
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < kPer; ++j) z += l[j] > -__builtin_inff() ? expf(l[j] - m) : 0.0f;
            total = wave_sum(z);
        }
    }
    if (lane < K) {
        float v = 0.0f;
        if (my_id >= 0) v = row_nan ? __builtin_nanf("") : scale * (total > 0.0f ? w / total : 0.0f);
        topk_idx[t * K + lane] = my_id;
        topk_w[t * K + lane] = v;
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
template <int kPer, bool kBf16, bool kSigmoid, bool kRenorm>
__global__ __launch_bounds__(kRouteWaves * kWave) void route_backward_kernel(
    const void* __restrict__ logits, int T, int E, int K, float scale,
    const int32_t* __restrict__ topk_idx, const float* __restrict__ grad_w,
    void* __restrict__ grad_logits)
{
    constexpr bool kFull = !kSigmoid && !kRenorm;          // every expert of the row is involved
    const int lane = threadIdx.x % kWave;
    for (int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave_uniform(threadIdx.x / kWave); t < T;
         t += (int64_t)gridDim.x * kRouteWaves) {
    const int kl = lane < K ? lane : 0;
    int id = topk_idx[t * K + kl];
    float g = grad_w[t * K + kl];
    if (lane >= K || id < 0 || id >= E) { id = -1; g = 0.0f; }
    const float lk = id >= 0 ? load_logit<kBf16>(logits, t * E + id) : -__builtin_inff();

    float out[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) out[j] = 0.0f;
    float d;                                               // lane k: the term of entry k
    if constexpr (kSigmoid) {
        const float p = id >= 0 ? sigmoid(lk) : 0.0f;
        const float r = id >= 0 ? 1.0f / (1.0f + expf(lk)) : 0.0f;      // 1 - p, without cancellation
        if constexpr (kRenorm) {
            const float total = wave_sum(p);
            const float q = total > 0.0f ? p / total : (total != total ? total : 0.0f);
            d = scale * q * r * (g - wave_sum(g * q));
        } else {
            d = scale * g * p * r;
        }
    } else if constexpr (kRenorm) {
        // order_key puts NaN lowest: a NaN among the chosen reaches the sum by itself
        const uint32_t mk = wave_max_u32(order_key(lk));
        const float m = mk == 0 ? 0.0f : __builtin_bit_cast(float, (mk >> 31) ? mk & 0x7FFFFFFFu : ~mk);
        const float w = id >= 0 && lk != -__builtin_inff() ? expf(lk - m) : 0.0f;
        const float total = wave_sum(w);
        const float q = total > 0.0f ? w / total : (total != total ? total : 0.0f);
        d = scale * q * (g - wave_sum(g * q));
    } else {
        float l[kPer];
        uint32_t mk = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = j * kWave + lane;
            l[j] = e < E ? load_logit<kBf16>(logits, t * E + e) : -__builtin_inff();
            mk = __builtin_elementwise_max(mk, order_key(l[j]));
        }
        mk = wave_max_u32(mk);
        const float m = mk == 0 ? 0.0f : __builtin_bit_cast(float, (mk >> 31) ? mk & 0x7FFFFFFFu : ~mk);
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            out[j] = l[j] == -__builtin_inff() ? 0.0f : expf(l[j] - m);
            z += out[j];
        }
        z = wave_sum(z);
        const float inv = z > 0.0f ? 1.0f / z : (z != z ? z : 0.0f);
        const float q = id >= 0 && lk != -__builtin_inff() ? expf(lk - m) * inv : 0.0f;
        const float dot = wave_sum(g * q);
#pragma unroll
        for (int j = 0; j < kPer; ++j) out[j] = -scale * (out[j] * inv) * dot;
        d = scale * q * g;
    }
    (void)kFull;
    if (id < 0) d = 0.0f;
    for (int k = 0; k < K; ++k) {
        const int e = read_lane(id, k);
        const float dk = __builtin_bit_cast(float, read_lane(__builtin_bit_cast(int, d), k));
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (j * kWave + lane == e) out[j] += dk;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = j * kWave + lane;
        if (e >= E) continue;
        if constexpr (kBf16)
            ((uint16_t*)grad_logits)[t * E + e] = __builtin_bit_cast(uint16_t, (__bf16)out[j]);
        else
            ((float*)grad_logits)[t * E + e] = out[j];
    }
    }
}

unsigned route_blocks(int T)
{
    const int64_t blocks = ((int64_t)T + kRouteWaves - 1) / kRouteWaves;
    return (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
}

template <int kPer>
void route_per(const void* logits, bool bf16, int T, int E, int K, bool sigmoid_score,
               const float* bias, int renorm, float scale, int32_t* topk_idx, float* topk_w,
               hipStream_t stream)
{
    const dim3 grid(route_blocks(T)), block(kRouteWaves * kWave);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, logits, bias, T, E, K, renorm, scale,
                           topk_idx, topk_w);
    };
    if (bias) bf16 ? go(route_kernel<kPer, true, true, true>) : go(route_kernel<kPer, false, true, true>);
    else if (sigmoid_score) bf16 ? go(route_kernel<kPer, true, true, false>) : go(route_kernel<kPer, false, true, false>);
    else bf16 ? go(route_kernel<kPer, true, false, false>) : go(route_kernel<kPer, false, false, false>);
}

template <int kPer>
void route_backward_per(const void* logits, bool bf16, int T, int E, int K, bool sigmoid_score,
                        int renorm, float scale, const int32_t* topk_idx, const float* grad_w,
                        void* grad_logits, hipStream_t stream)
{
    const dim3 grid(route_blocks(T)), block(kRouteWaves * kWave);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, 0, stream, logits, T, E, K, scale, topk_idx, grad_w,
                           grad_logits);
    };
    if (sigmoid_score) {
        if (renorm) bf16 ? go(route_backward_kernel<kPer, true, true, true>) : go(route_backward_kernel<kPer, false, true, true>);
        else bf16 ? go(route_backward_kernel<kPer, true, true, false>) : go(route_backward_kernel<kPer, false, true, false>);
    } else {
        if (renorm) bf16 ? go(route_backward_kernel<kPer, true, false, true>) : go(route_backward_kernel<kPer, false, false, true>);
        else bf16 ? go(route_backward_kernel<kPer, true, false, false>) : go(route_backward_kernel<kPer, false, false, false>);
    }
}

// The smallest instance whose lanes hold E logits.
template <class F>
void with_per(int E, F&& f)
{
    const int per = (E + kWave - 1) / kWave;
    if (per <= 1) f(std::integral_constant<int, 1>());
    else if (per <= 2) f(std::integral_constant<int, 2>());
    else if (per <= 4) f(std::integral_constant<int, 4>());
    else if (per <= 6) f(std::integral_constant<int, 6>());
    else if (per <= 8) f(std::integral_constant<int, 8>());
    else f(std::integral_constant<int, 16>());
}

}  // namespace

hipError_t launch_route(const void* logits, bool bf16, int T, int E, int K, bool sigmoid_score,
                        const float* bias, bool renorm, float scale, int32_t* topk_idx,
                        float* topk_w, hipStream_t stream)
{
    with_per(E, [&](auto per) {
        route_per<decltype(per)::value>(logits, bf16, T, E, K, sigmoid_score, bias, renorm ? 1 : 0,
                                        scale, topk_idx, topk_w, stream);
    });
    return hipGetLastError();
}

hipError_t launch_route_backward(const void* logits, bool bf16, int T, int E, int K,
                                 bool sigmoid_score, bool renorm, float scale,
                                 const int32_t* topk_idx, const float* grad_w, void* grad_logits,
                                 hipStream_t stream)
{
    with_per(E, [&](auto per) {
        route_backward_per<decltype(per)::value>(logits, bf16, T, E, K, sigmoid_score,
                                                 renorm ? 1 : 0, scale, topk_idx, grad_w,
                                                 grad_logits, stream);
    });
    return hipGetLastError();
}

}  // namespace ep
