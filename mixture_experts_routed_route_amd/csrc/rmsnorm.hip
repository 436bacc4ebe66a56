// Residual addition, root-mean-square norm and E4M3 output of bf16 rows:
//   h = bf16(x + r), y = (h * w) * rstd with rstd = 1 / sqrt(mean(h^2) + eps), codes of y.
//
// One pass over the data.  WAVES waves own a row and hold it in registers as the rounded bf16 h
// (16 bytes = 8 columns per chunk, NC chunks per lane); the sum of squares and, for a row scale, the
// largest |h * w| are reduced together, so there is one exchange per row: rstd > 0 is the row's common
// factor and fp32 rounding is monotone, so max |y| = fl(max |h * w| * rstd) exactly.  A block scale
// needs no exchange beyond its 16 lanes (8 columns each).  Rows of at most 2048 columns take one
// wave each, four to a workgroup, with no LDS and no barrier; longer rows take a workgroup.  Rows past
// 16384 columns (NC == 0) are read twice, the second time mostly from L2: the second pass rereads h
// where the first wrote it.
//
// What bounds it: memory.  4096 rows of 4096 with a residual, bf16 and row-scaled codes out (151 MB) take
// 30.5 us, 4.9 TB/s, the rate of a large copy; 5003 rows of 5136 with block-scaled codes only (181 MB) 38 us,
// 4.8 TB/s.  One row is latency: 2.8 us.
//
// Roundings: x + r in fp32 then to bf16 is the correctly rounded sum (24 bits >= 2 * 8 + 2); squares,
// their sum, rstd and y are fp32; y is rounded once, to bf16 and/or to its code.
#include "fp8_quant.h"
#include "launchers.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

enum { kScaleNone = 0, kScaleRow = 1, kScaleBlock = 2 };

struct NormArgs {
    const uint16_t* x;   // x, r and h_out may be one buffer: a lane reads a chunk before it writes it
    const uint16_t* r;
    const uint16_t* w;
    uint16_t* h_out;
    uint16_t* y;
    uint8_t* q;
    float* scale;
    int64_t rows;
    int K;
    float eps;
};

// h of one chunk, packed bf16
__device__ __forceinline__ u32x4 add_chunk(u32x4 x, u32x4 r) {
    u32x4 h;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack_bf16x2(bf_lo(x[i]) + bf_lo(r[i]), bf_hi(x[i]) + bf_hi(r[i]));
    return h;
}

template <int NC, int WAVES, int SCALE>
__global__ __launch_bounds__(kThreads) void rmsnorm_kernel(NormArgs a) {
    constexpr int TPR = 64 * WAVES;              // threads per row
    constexpr int RPW = kThreads / TPR;          // rows per workgroup
    __shared__ float s_sum[2][4], s_max[2][4];   // two sets: a row's exchange may overlap the next row's
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int K = a.K;
    const int chunks = K / 8, blocks = (K + kFp8Block - 1) / kFp8Block;
    int turn = 0;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + sub; row < a.rows;
         row += static_cast<int64_t>(gridDim.x) * RPW, turn ^= 1) {
        const int64_t base = row * K;
        auto ld = [&](const uint16_t* p, int c) { return *reinterpret_cast<const u32x4*>(p + base + 8 * c); };
        auto ldw = [&](int c) { return *reinterpret_cast<const u32x4*>(a.w + 8 * c); };
        auto st = [&](uint16_t* p, int c, u32x4 v) { *reinterpret_cast<u32x4*>(p + base + 8 * c) = v; };
        float sum = 0.f, mx = 0.f;
        auto accumulate = [&](u32x4 h, u32x4 w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float lo = bf_lo(h[i]), hi = bf_hi(h[i]);
                sum = fmaf(lo, lo, sum);
                sum = fmaf(hi, hi, sum);
                if constexpr (SCALE == kScaleRow)
                    mx = fmaxf(mx, fmaxf(fabsf(lo * bf_lo(w[i])), fabsf(hi * bf_hi(w[i]))));
            }
        };
        u32x4 hv[NC > 0 ? NC : 1], wv[NC > 0 ? NC : 1];
        const u32x4 zero = {0u, 0u, 0u, 0u};
        if constexpr (NC > 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int c = t + i * TPR;
                hv[i] = c < chunks ? ld(a.x, c) : zero;
                wv[i] = c < chunks ? ldw(c) : zero;
            }
            if (a.r) {
                u32x4 rv[NC];
#pragma unroll
                for (int i = 0; i < NC; ++i) rv[i] = t + i * TPR < chunks ? ld(a.r, t + i * TPR) : zero;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    hv[i] = add_chunk(hv[i], rv[i]);
                    if (t + i * TPR < chunks) st(a.h_out, t + i * TPR, hv[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) accumulate(hv[i], wv[i]);
        } else {
            for (int c = t; c < chunks; c += TPR) {
                u32x4 h = ld(a.x, c);
                if (a.r) {
                    h = add_chunk(h, ld(a.r, c));
                    st(a.h_out, c, h);
                }
                accumulate(h, ldw(c));
            }
        }
#pragma unroll
        for (int o = 32; o >= 1; o >>= 1) {
            sum += __shfl_xor(sum, o);
            if constexpr (SCALE == kScaleRow) mx = fmaxf(mx, __shfl_xor(mx, o));
        }
        if constexpr (WAVES > 1) {
            if ((t & 63) == 0) {
                s_sum[turn][t >> 6] = sum;
                s_max[turn][t >> 6] = mx;
            }
            __syncthreads();
            sum = (s_sum[turn][0] + s_sum[turn][1]) + (s_sum[turn][2] + s_sum[turn][3]);
            mx = fmaxf(fmaxf(s_max[turn][0], s_max[turn][1]), fmaxf(s_max[turn][2], s_max[turn][3]));
        }
        const float rstd = 1.0f / sqrtf(sum / static_cast<float>(K) + a.eps);
        Fp8Scale rs{1.f, 1.f};
        if constexpr (SCALE == kScaleRow) {
            rs = fp8_scale(mx * rstd);
            if (t == 0) a.scale[row] = rs.scale;
        }
        // one chunk's outputs (`in`: it lies in the row; its 16 lanes share a block's scale)
        auto emit = [&](int c, bool in, u32x4 h, u32x4 w) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[2 * i] = bf_lo(h[i]) * bf_lo(w[i]) * rstd;
                y[2 * i + 1] = bf_hi(h[i]) * bf_hi(w[i]) * rstd;
            }
            if (in && a.y) {
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
                st(a.y, c, o);
            }
            if constexpr (SCALE != kScaleNone) {
                Fp8Scale s = rs;
                if constexpr (SCALE == kScaleBlock) {
                    float m = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
                    s = fp8_scale(row16_max(in ? m : 0.f));
                    if (in && (c & 15) == 0) a.scale[row * blocks + (c >> 4)] = s.scale;
                }
                const float f = s.factor;
                if (in)
                    *reinterpret_cast<uint2*>(a.q + base + 8 * c) =
                        make_uint2(fp8_codes4(y[0] * f, y[1] * f, y[2] * f, y[3] * f),
                                   fp8_codes4(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
            }
        };
        if constexpr (NC > 0) {
#pragma unroll
            for (int i = 0; i < NC; ++i) emit(t + i * TPR, t + i * TPR < chunks, hv[i], wv[i]);
        } else {
            // whole 16-lane groups, so that a block's lanes stay together; every lane rereads only
            // chunks that it wrote itself
            const uint16_t* src = a.r ? a.h_out : a.x;
            for (int c = t; c < blocks * 16; c += TPR) {
                const bool in = c < chunks;
                emit(c, in, in ? ld(src, c) : zero, in ? ldw(c) : zero);
            }
        }
    }
}

template <int SCALE>
void launch_scale(const NormArgs& a, hipStream_t s) {
    const int chunks = a.K / 8;
    // rows are strided over the grid: its size stays under the 2^32 work-items of one dimension
    auto grid = [&](int rpw) {
        const int64_t need = (a.rows + rpw - 1) / rpw;
        return static_cast<unsigned>(need < (1 << 20) ? need : (1 << 20));
    };
    if (chunks <= 64) rmsnorm_kernel<1, 1, SCALE><<<grid(4), kThreads, 0, s>>>(a);
    else if (chunks <= 128) rmsnorm_kernel<2, 1, SCALE><<<grid(4), kThreads, 0, s>>>(a);
    else if (chunks <= 256) rmsnorm_kernel<4, 1, SCALE><<<grid(4), kThreads, 0, s>>>(a);
    else if (chunks <= 512) rmsnorm_kernel<2, 4, SCALE><<<grid(1), kThreads, 0, s>>>(a);
    else if (chunks <= 1024) rmsnorm_kernel<4, 4, SCALE><<<grid(1), kThreads, 0, s>>>(a);
    else if (chunks <= 2048) rmsnorm_kernel<8, 4, SCALE><<<grid(1), kThreads, 0, s>>>(a);
    else rmsnorm_kernel<0, 4, SCALE><<<grid(1), kThreads, 0, s>>>(a);
}

// ------------------------------------------------------------------ block quantisation
// Codes of bf16 rows with one scale per 128 columns: 16 lanes of 8 columns make a block, so a row needs
// no exchange beyond DPP.  TPR lanes walk a row, U chunks each in flight together.  Rows of up to 2048
// columns take one wave and one round of loads: 12288 real rows of 1408 among 16320 sorted ones (52 MB) 11.4
// us, 4.6 TB/s, against 14.9 with a workgroup per row, most of whose lanes had one chunk or none.  Longer rows
// take a workgroup, so that one row alone is one round up to 4096 columns: 8191 rows of 4096 (102 MB) 17.3 us
// either way, 5.9 TB/s of reads and writes.
template <int TPR, int U>
__global__ __launch_bounds__(kThreads) void quantize_block_kernel(const uint16_t* __restrict__ x,
                                                                  uint8_t* __restrict__ q,
                                                                  float* __restrict__ scale,
                                                                  const int32_t* __restrict__ sorted_ids, int P,
                                                                  int64_t rows, int K) {
    constexpr int RPW = kThreads / TPR;
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int chunks = K / 8, blocks = (K + kFp8Block - 1) / kFp8Block;
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + sub; row < rows;
         row += static_cast<int64_t>(gridDim.x) * RPW) {
        if (sorted_ids) {
            const int p = sorted_ids[row];
            if (p < 0 || p >= P) continue;  // the same for the row's 16-lane groups
        }
        const uint16_t* xr = x + row * K;
        auto load = [&](int c) {
            return c < chunks ? *reinterpret_cast<const u32x4*>(xr + 8 * c) : u32x4{0u, 0u, 0u, 0u};
        };
        auto emit = [&](int c, u32x4 v) {
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(bf_lo(v[i])), fabsf(bf_hi(v[i]))));
            const Fp8Scale s = fp8_scale(row16_max(m));
            if (c >= chunks) return;
            if ((c & 15) == 0) scale[row * blocks + (c >> 4)] = s.scale;
            const float f = s.factor;
            *reinterpret_cast<uint2*>(q + row * K + 8 * c) =
                make_uint2(fp8_codes4(bf_lo(v[0]) * f, bf_hi(v[0]) * f, bf_lo(v[1]) * f, bf_hi(v[1]) * f),
                           fp8_codes4(bf_lo(v[2]) * f, bf_hi(v[2]) * f, bf_lo(v[3]) * f, bf_hi(v[3]) * f));
        };
        for (int c = t; c < blocks * 16; c += U * TPR) {
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = load(c + u * TPR);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * TPR < blocks * 16) emit(c + u * TPR, v[u]);
        }
    }
}

}  // namespace

hipError_t launch_rmsnorm(const uint16_t* x, const uint16_t* r, const uint16_t* w, float eps, int64_t rows, int K,
                          uint16_t* h_out, uint16_t* y, uint8_t* q, float* scale, int scale_block, hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const NormArgs a{x, r, w, h_out, y, q, scale, rows, K, eps};
    if (!q) launch_scale<kScaleNone>(a, s);
    else if (scale_block == 0) launch_scale<kScaleRow>(a, s);
    else launch_scale<kScaleBlock>(a, s);
    return hipGetLastError();
}

hipError_t launch_quantize_fp8_block(const uint16_t* x, int64_t rows, int K, const int32_t* sorted_ids, int P,
                                     uint8_t* q, float* scale, hipStream_t s) {
    if (rows <= 0) return hipSuccess;
    const int slots = (K + kFp8Block - 1) / kFp8Block * 16;  // lanes of 8 columns, whole blocks
    auto grid = [&](int rpw) {
        const int64_t need = (rows + rpw - 1) / rpw;
        return static_cast<unsigned>(need < (1 << 20) ? need : (1 << 20));
    };
    if (slots <= 16) quantize_block_kernel<16, 1><<<grid(16), kThreads, 0, s>>>(x, q, scale, sorted_ids, P, rows, K);
    else if (slots <= 256) quantize_block_kernel<64, 4><<<grid(4), kThreads, 0, s>>>(x, q, scale, sorted_ids, P, rows, K);
    else quantize_block_kernel<256, 2><<<grid(1), kThreads, 0, s>>>(x, q, scale, sorted_ids, P, rows, K);
    return hipGetLastError();
}

}  // namespace moe
