// Row kernels of the expert path's gradients: SiLU(gate) * up with dropout, its backward with the
// router weight, and the gradient of the router's logits.
#include <type_traits>

#include "device_common.h"
#include "launchers.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3",
// SC 2011): a counter and a key to four random words, nothing kept between calls.
__device__ __forceinline__ u32x4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return u32x4{c0, c1, c2, c3};
}

// seed and offset (uniform: scalar loads)
struct Rng {
    uint32_t k0, k1, o0, o1;
    __device__ __forceinline__ explicit Rng(const int64_t* rng) {
        const uint64_t s = static_cast<uint64_t>(rng[0]), o = static_cast<uint64_t>(rng[1]);
        k0 = static_cast<uint32_t>(s); k1 = static_cast<uint32_t>(s >> 32);
        o0 = static_cast<uint32_t>(o); o1 = static_cast<uint32_t>(o >> 32);
    }
};

// dropout factors of eight columns: 16 bits each, so that one counter covers the 16 bytes of bf16 that a lane
// loads (with 32 bits each the ten rounds would be run twice per load)
__device__ __forceinline__ void keep8(const Rng& g, uint32_t chunk, uint32_t pair, uint32_t below, float scale,
                                      float (&f)[8]) {
    const u32x4 w = philox(chunk, pair, g.o0, g.o1, g.k0, g.k1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = (w[i] & 0xffffu) >= below ? scale : 0.f;
        f[2 * i + 1] = (w[i] >> 16) >= below ? scale : 0.f;
    }
}

__device__ __forceinline__ float lo_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// HBM-bound: 6 bytes per value.  The rows' 16-byte chunks are dealt to threads in one flat sequence, so that
// narrow rows leave no lanes idle.  65536 real rows of 768 columns with dropout: 54 us, 5.6 TB/s (302 MB); a copy of
// 1 GiB reaches 4.8.  The ten rounds of the generator, 40 multiplications for 8 values, hide behind the loads.
// 64 tokens x 128: 3 us, the launch itself.
template <bool DROP>
__global__ __launch_bounds__(kThreads) void silu_mul_dropout_kernel(const uint16_t* g, const uint16_t* u, uint16_t* h,
                                                                    const int32_t* __restrict__ sorted_ids, int P,
                                                                    int64_t chunks, uint32_t n8, uint32_t below,
                                                                    float scale, const int64_t* __restrict__ rng) {
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads;
    const int64_t row0 = base / n8;
    const uint32_t at = static_cast<uint32_t>(base - row0 * n8) + threadIdx.x;
    const uint32_t down = at / n8;
    const int64_t row = row0 + down;
    if (base + threadIdx.x >= chunks) return;
    int p = static_cast<int>(row);
    if (sorted_ids) {
        p = sorted_ids[row];
        if (p < 0 || p >= P) return;
    }
    const int64_t off = (base + threadIdx.x) * 8;
    const u32x4 gv = *reinterpret_cast<const u32x4*>(g + off);
    const u32x4 uv = *reinterpret_cast<const u32x4*>(u + off);
    float f[8];
    if constexpr (DROP) keep8(Rng(rng), at - down * n8, p, below, scale, f);
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a = silu_mul(lo_f32(gv[i]), lo_f32(uv[i])), b = silu_mul(hi_f32(gv[i]), hi_f32(uv[i]));
        if constexpr (DROP) {
            a = f[2 * i] != 0.f ? a * f[2 * i] : 0.f;   // a dropped value is 0 whatever the row held
            b = f[2 * i + 1] != 0.f ? b * f[2 * i + 1] : 0.f;
        }
        o[i] = pack_bf16x2(a, b);
    }
    *reinterpret_cast<u32x4*>(h + off) = o;
}

// One value of the backward: the gradients of gate and up, w * h, and d * h.
__device__ __forceinline__ void back1(float g, float u, float d, float w, float f, float& dg, float& du, float& hw,
                                      float& dot) {
    const float sig = __builtin_amdgcn_rcpf(1.f + __expf(-g));
    const float silu = g * sig;
    const float h = silu * u * f;
    const float dh = w * d * f;
    du = dh * silu;
    dg = dh * u * (sig + silu * (1.f - sig));
    hw = w * h;
    dot = fmaf(d, h, dot);
}

// HBM-bound: 12 bytes per value.  TPR threads per row, since d_topk_w is a sum over the row; added in a fixed order.
// Inputs may be outputs: every thread loads all it needs of its columns before it stores any.
// 8192 real rows of 14336 columns: 268 us, 5.3 TB/s (1.41 GB); 11994 of 1408 with dropout: 44 us, 4.6 TB/s (203 MB).
template <bool DROP, int TPR>
__global__ __launch_bounds__(kThreads) void silu_mul_backward_kernel(const uint16_t* g, const uint16_t* u,
                                                                     const uint16_t* d,
                                                                     const float* __restrict__ topk_w,
                                                                     const int32_t* __restrict__ sorted_ids, int P,
                                                                     int64_t rows, int n, uint32_t below, float scale,
                                                                     const int64_t* __restrict__ rng, uint16_t* dg,
                                                                     uint16_t* du, uint16_t* hw,
                                                                     float* __restrict__ dw) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
    if (row >= rows) return;
    int p = static_cast<int>(row);
    if (sorted_ids) p = sorted_ids[row];
    if (p < 0 || p >= P) return;   // (with TPR == kThreads the whole workgroup leaves)
    const float w = topk_w[p];
    const int64_t off = row * n;
    const int t = threadIdx.x % TPR;
    float dot = 0.f;
    const uint32_t cols = n;   // (c0 goes up to 2 * TPR * 8 past n: in signed 32 bits it would wrap in rows next to 2^31)
    for (uint32_t c0 = t * 8; c0 < cols; c0 += 2 * TPR * 8) {
        u32x4 gv[2], uv[2], dv[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t c = c0 + b * TPR * 8;
            if (c < cols) {
                gv[b] = *reinterpret_cast<const u32x4*>(g + off + c);
                uv[b] = *reinterpret_cast<const u32x4*>(u + off + c);
                dv[b] = *reinterpret_cast<const u32x4*>(d + off + c);
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const uint32_t c = c0 + b * TPR * 8;
            if (c >= cols) continue;
            float f[8];
            if constexpr (DROP) keep8(Rng(rng), c >> 3, p, below, scale, f);
            u32x4 og, ou, oh;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[2][3];
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const float gf = s ? hi_f32(gv[b][i]) : lo_f32(gv[b][i]);
                    const float uf = s ? hi_f32(uv[b][i]) : lo_f32(uv[b][i]);
                    const float df = s ? hi_f32(dv[b][i]) : lo_f32(dv[b][i]);
                    const float ff = DROP ? f[2 * i + s] : 1.f;
                    if (DROP && ff == 0.f) x[s][0] = x[s][1] = x[s][2] = 0.f;
                    else back1(gf, uf, df, w, ff, x[s][0], x[s][1], x[s][2], dot);
                }
                og[i] = pack_bf16x2(x[0][0], x[1][0]);
                ou[i] = pack_bf16x2(x[0][1], x[1][1]);
                oh[i] = pack_bf16x2(x[0][2], x[1][2]);
            }
            *reinterpret_cast<u32x4*>(dg + off + c) = og;
            *reinterpret_cast<u32x4*>(du + off + c) = ou;
            *reinterpret_cast<u32x4*>(hw + off + c) = oh;
        }
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) dot += __shfl_xor(dot, o);
    if constexpr (TPR > kWave) {
        __shared__ float s_dot[TPR / kWave];
        if ((t & 63) == 0) s_dot[t >> 6] = dot;
        __syncthreads();
        dot = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / kWave; ++i) dot += s_dot[i];
    }
    if (t == 0) dw[p] = dot;
}

// One wave per token, four tokens per workgroup; lane l holds experts l, l + 64, ...  Sums in fp64: the launch
// is bound by latency and the bytes of d_logits, and w_j * (d_w_j - dot) cancels where one weight is near 1.
// 8192 tokens, 8 of 128 experts: 6.8 us; 64 tokens, 8 of 256, over all experts: 4.9 us (an empty launch: 3).
constexpr int kRouteTokens = kThreads / kWave;

__device__ __forceinline__ double read_lane(double v, int lane) {   // lane uniform
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), lane);
    return __longlong_as_double(static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo));
}

template <bool FULL>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(const int32_t* __restrict__ ids,
                                                                  const float* __restrict__ w,
                                                                  const float* __restrict__ dw,
                                                                  const float* __restrict__ logits, int T, int E, int k,
                                                                  float* __restrict__ out) {
    const int t = blockIdx.x * kRouteTokens + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (t >= T) return;
    const int64_t p0 = static_cast<int64_t>(t) * k, l0 = static_cast<int64_t>(t) * E;
    int id[4];
    double wd[4], wj[4], dot = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = lane + 64 * i;
        id[i] = -1;
        wd[i] = wj[i] = 0.0;
        if (j < k) {   // (three loads at once; what a dropped pair holds is not used)
            const int e = ids[p0 + j];
            const float a = w[p0 + j], d = dw[p0 + j];
            if (e >= 0 && e < E) {
                id[i] = e;
                wj[i] = a;
                wd[i] = d;
            }
        }
        dot += wj[i] * wd[i];
    }
    double pr[4] = {0.0, 0.0, 0.0, 0.0};
    if constexpr (FULL) {
        float top = -__builtin_inff();
        float l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = lane + 64 * i;
            l[i] = e < E ? logits[l0 + e] : -__builtin_inff();
            top = fmaxf(top, l[i]);
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane + 64 * i < E) sum += pr[i] = exp(static_cast<double>(l[i]) - static_cast<double>(top));
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[i] /= sum;
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        if (o < k) dot += __shfl_xor(dot, o);   // (lanes past k hold zeros)
    dot = read_lane(dot, 0);
    // each expert gathers the pairs that name it (an id may come twice)
    double acc[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const double v = FULL ? wd[i] : wj[i] * (wd[i] - dot);
        for (int j = 64 * i; j < min(k, 64 * i + 64); ++j) {   // (scalar reads of lane j: no trip through LDS)
            const int e = __builtin_amdgcn_readlane(id[i], j & 63);
            const double x = lane == (e & 63) ? read_lane(v, j & 63) : 0.0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (e >= 0 && (e >> 6) == q) acc[q] += x;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = lane + 64 * i;
        if (e < E) out[l0 + e] = static_cast<float>(FULL ? pr[i] * (acc[i] - dot) : acc[i]);
    }
}

}  // namespace

hipError_t launch_silu_mul_dropout(const uint16_t* g, const uint16_t* u, uint16_t* h, const int32_t* sorted_ids, int P,
                                   int64_t rows, int N, uint32_t below, const int64_t* rng, hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const int64_t chunks = rows * (N / 8);
    const float scale = 65536.f / static_cast<float>(65536u - below);
    const dim3 grid(static_cast<unsigned>((chunks + kThreads - 1) / kThreads));
    if (below) silu_mul_dropout_kernel<true><<<grid, kThreads, 0, s>>>(g, u, h, sorted_ids, P, chunks, N / 8, below, scale, rng);
    else silu_mul_dropout_kernel<false><<<grid, kThreads, 0, s>>>(g, u, h, sorted_ids, P, chunks, N / 8, below, scale, rng);
    return hipGetLastError();
}

hipError_t launch_silu_mul_backward(const uint16_t* g, const uint16_t* u, const uint16_t* d, const float* w,
                                    const int32_t* sorted_ids, int P, int64_t rows, int N, uint32_t below,
                                    const int64_t* rng, uint16_t* dg, uint16_t* du, uint16_t* hw, float* dw,
                                    hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const float scale = 65536.f / static_cast<float>(65536u - below);
    auto go = [&](auto drop, auto tpr) {
        constexpr int R = kThreads / decltype(tpr)::value;
        silu_mul_backward_kernel<decltype(drop)::value, decltype(tpr)::value>
            <<<static_cast<unsigned>((rows + R - 1) / R), kThreads, 0, s>>>(g, u, d, w, sorted_ids, P, rows, N, below, scale,
                                                                          rng, dg, du, hw, dw);
    };
    using Wave = std::integral_constant<int, kWave>;
    using Block = std::integral_constant<int, kThreads>;
    // A wave per row, or the workgroup for wide rows (us without and with dropout, wave / workgroup: 65536 rows of 256
    // 34, 43 / 53, 83; 65536 of 768 107, 108 / 106, 124; 16384 of 2048 74, 76 / 74, 73; 16384 of 2560 97, 98 / 91, 91;
    // 8192 of 14336 279, 284 / 266, 269).
    const bool wide = N > 2048;
    if (below) wide ? go(std::true_type{}, Block{}) : go(std::true_type{}, Wave{});
    else wide ? go(std::false_type{}, Block{}) : go(std::false_type{}, Wave{});
    return hipGetLastError();
}

hipError_t launch_route_backward(const int32_t* ids, const float* w, const float* dw, const float* logits, int T, int E,
                                 int k, float* out, hipStream_t s) {
    if (T <= 0) return hipSuccess;
    const dim3 grid((T + kRouteTokens - 1) / kRouteTokens);
    if (logits) route_backward_kernel<true><<<grid, kThreads, 0, s>>>(ids, w, dw, logits, T, E, k, out);
    else route_backward_kernel<false><<<grid, kThreads, 0, s>>>(ids, w, dw, logits, T, E, k, out);
    return hipGetLastError();
}

}  // namespace moe
