// The whole routed layer for at most 32 tokens in two launches:
//
//   few_gate_up   top-k softmax routing, then h[p] = bf16(SiLU(x Wg^T) * (x Wu^T)) of every (token,
//                 slot) pair p = t * top_k + j
//   few_down      out[t] = bf16(sum_j w[t, j] * (h[p] Wd^T)), fp32 sums over k and over the experts
//
// What bounds it: reading the active experts' weights once.  A few tokens leave the matrix units idle
// (16 tokens use 1/20 of their rate at the streaming rate of HBM), so each weight value goes from memory
// to one MFMA through registers, with no LDS in between, and the tokens are the other operand: a
// 16x16x32 bf16 MFMA takes 16 tokens x 16 output columns (TF = 2 fragments above 16 tokens; a token not
// routed to the expert is a row of zeros there, or a row whose result nobody stores).  There is no
// sorted layout: a 32-bit mask of tokens per expert is the whole routing, and the experts with a
// non-empty mask, ascending, are the work list.
//
// Routing.  Every workgroup of few_gate_up selects all tokens' experts itself from the logits (at most
// 32 KB, from L2): a launch less, and cheaper than waiting for one workgroup's result.  Workgroup 0
// alone computes the weights (in fp64, route_tokens: ids and weights bit for bit those of moe_route)
// and stores them; few_down reads them back.
//
// Work split.  A workgroup takes one panel of 16 * CPL output columns of one expert; its waves split the
// projections (gate, up) and the contraction, and their partial sums meet in LDS.  In few_down a
// workgroup keeps one column panel and adds up the experts i = s, s + splits, ... of the work list in
// registers, weighted per token; with splits > 1 (fewer panels than the GPU has room for) the partial
// panels meet in the workspace, the last workgroup to arrive adding them in the order of s, so the
// result does not depend on who arrives last.
//
// Roundings: h to bf16 (the operand type of the second product, as between the grouped GEMMs); the
// expert outputs are not rounded before the weighted sum; out once to bf16.  fp8 weights convert to
// bf16 exactly, their scales multiply fp32 sums; int4 words enter as 128 + q (int4_dequant.h).
//
// Rows past N or T, k past K and tokens that are not the expert's are read through bounds-checked
// buffer loads with an offset past the end: zeros, and no memory traffic.
#include "few_tokens.h"
#include "fp8_quant.h"
#include "int4_dequant.h"
#include "launchers.h"
#include "route_common.h"

namespace moe {
namespace {

constexpr int kMaxE = 256;
constexpr int kPast = static_cast<int>(0x80000000u);  // a buffer offset past every buffer (all are < 2 GiB)

enum { kBf16 = 0, kInt4 = 1, kFp8Row = 2, kFp8Blk = 3 };

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), 0x00020000);
}

__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t b, int off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0));
}

// ------------------------------------------------------------------ routing state in LDS
struct Routed {
    uint32_t tok[kMaxE];              // tokens routed to the expert, one bit each
    uint8_t slot[kFewTokens][kMaxE];  // the token's slot j for the expert (where its bit is set)
    int act[kMaxE];                   // experts with tokens, ascending
    int scan[16];
    int n_act;
};

// act and n_act from tok; every thread of the workgroup, at least kMaxE threads
template <int NW>
__device__ __forceinline__ void list_active(Routed& r, int E) {
    const int tid = threadIdx.x;
    const int f = tid < E && r.tok[tid] != 0 ? 1 : 0;
    const int incl = block_inclusive_scan<NW>(f, r.scan, (E + 63) / 64);
    if (f) r.act[incl - 1] = tid;
    if (tid == E - 1) r.n_act = incl;
    __syncthreads();
}

// Expert selection of tokens t0, t0 + dt, .. (NTOK of them, interleaved to hide each other's latency),
// one wave: top_k rounds of a wave maximum over the order-preserving images of the logits, the lowest
// expert of those that hold it (route_tokens' selection, without the weights).
template <int EPL, int NTOK>
__device__ __forceinline__ void select_experts(const float* __restrict__ logits, int t0, int dt, int T, int E,
                                               int top_k, Routed& r, int lane) {
    uint32_t key[NTOK][EPL];
#pragma unroll
    for (int n = 0; n < NTOK; ++n) {
        const int t = t0 + n * dt;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            key[n][i] = t < T && e < E ? order_bits(logits[t * E + e]) : 0u;
        }
    }
    for (int j = 0; j < top_k; ++j) {
        uint32_t best[NTOK];
#pragma unroll
        for (int n = 0; n < NTOK; ++n) {
            best[n] = key[n][0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) best[n] = max(best[n], key[n][i]);
        }
#pragma unroll
        for (int n = 0; n < NTOK; ++n) best[n] = wave_max_u32(best[n]);
#pragma unroll
        for (int n = 0; n < NTOK; ++n) {
            int e = 0;
#pragma unroll
            for (int i = EPL - 1; i >= 0; --i) {
                const uint64_t hit = __ballot(key[n][i] == best[n]);
                if (hit) e = 64 * i + __ffsll(static_cast<unsigned long long>(hit)) - 1;
            }
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (lane + 64 * i == e) key[n][i] = 0;
            const int t = t0 + n * dt;
            if (lane == 0 && t < T && e < E) {
                r.slot[t][e] = static_cast<uint8_t>(j);
                atomicOr(&r.tok[e], 1u << t);
            }
        }
    }
}

template <int NW>
__device__ __forceinline__ void select_all(const FewArgs& a, Routed& r, int wave, int lane) {
    auto go = [&](auto epl) {
        constexpr int EPL = decltype(epl)::value;
        if (a.T <= NW) {
            if (wave < a.T) select_experts<EPL, 1>(a.logits, wave, NW, a.T, a.E, a.top_k, r, lane);
        } else {
            for (int t = wave; t < a.T; t += 4 * NW)
                select_experts<EPL, 4>(a.logits, t, NW, a.T, a.E, a.top_k, r, lane);
        }
    };
    switch ((a.E + 63) / 64) {
        case 1: go(std::integral_constant<int, 1>{}); break;
        case 2: go(std::integral_constant<int, 2>{}); break;
        case 3: go(std::integral_constant<int, 3>{}); break;
        default: go(std::integral_constant<int, 4>{}); break;
    }
}

// ------------------------------------------------------------------ one wave's share of a panel
// out[j][f] += sum over the wave's part of K of A(token, k) * W(column, k) for columns n0 + CPL * m + j
// (m = lane % 16) and tokens 16 f + 4 (lane / 16) + v.  `arow[f]`: byte offset of the row of token
// 16 f + m in `abuf` (kPast: none).
struct Panel {
    const FewWeight* w;
    int e, n0, N, K;
    int part, parts;  // the wave's share of K
    int group;        // int4: k under one scale
    __amdgpu_buffer_rsrc_t abuf;
};

// [E, N, K] weights, K contiguous.  A load instruction takes 16 bytes of 4 consecutive k chunks of 16
// rows; U of them per column set are in flight before the first is used.
template <int KIND, int CPL, int TF, int U>
__device__ __forceinline__ void panel_rows(const Panel& p, const int (&arow)[TF], f32x4 (&out)[CPL][TF]) {
    constexpr int ES = KIND == kBf16 ? 2 : 1;
    constexpr int FR = KIND == kBf16 ? 1 : 2;  // MFMA k-steps (32 k) per 16-byte chunk set
    constexpr int KS = 32 * FR;                // k per load
    const int lane = threadIdx.x & 63, m = lane & 15, kq = lane >> 4;
    const int N = p.N, K = p.K;
    const int64_t mat = static_cast<int64_t>(N) * K * ES;
    const __amdgpu_buffer_rsrc_t wbuf = buffer(static_cast<const char*>(p.w->data) + p.e * mat, mat);
    int woff[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
        const int n = p.n0 + CPL * m + j;
        woff[j] = n < N ? n * K * ES + kq * 16 : kPast;
    }
    int aoff[TF];
#pragma unroll
    for (int f = 0; f < TF; ++f) aoff[f] = arow[f] + kq * (8 * FR * 2);
    const int steps = (K + KS - 1) / KS;
    const int s0 = __builtin_amdgcn_readfirstlane(p.part * steps / p.parts);
    const int s1 = __builtin_amdgcn_readfirstlane((p.part + 1) * steps / p.parts);
    const int kb_n = (K + 127) / 128, nb_n = (N + 127) / 128;
    const float* bscale = nullptr;  // block scales of this panel's 128 rows
    if constexpr (KIND == kFp8Blk)
        bscale = static_cast<const float*>(p.w->scales) + (static_cast<int64_t>(p.e) * nb_n + p.n0 / 128) * kb_n;
    for (int s = s0; s < s1; s += U) {
        u32x4 b[U][CPL], x[U][TF][FR];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = s + u < s1 && (s + u) * KS + kq * (16 / ES) < K;
#pragma unroll
            for (int j = 0; j < CPL; ++j) b[u][j] = load16(wbuf, in ? woff[j] + (s + u) * (KS * ES) : kPast);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = s + u < s1 && (s + u) * KS + kq * (16 / ES) < K;
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int c = 0; c < FR; ++c)
                    x[u][f][c] = load16(p.abuf, in && arow[f] != kPast ? aoff[f] + (s + u) * (KS * 2) + c * 16 : kPast);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float sc = 1.f;
            if constexpr (KIND == kFp8Blk) sc = bscale[min((s + u) * KS / 128, kb_n - 1)];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                bf16x8 w[FR];
                if constexpr (KIND == kBf16) {
                    w[0] = as_bf16x8(b[u][j]);
                } else {
                    w[0] = fp8_to_bf16(b[u][j][0], b[u][j][1]);
                    w[FR - 1] = fp8_to_bf16(b[u][j][2], b[u][j][3]);
                }
#pragma unroll
                for (int f = 0; f < TF; ++f) {
                    f32x4 d = KIND == kFp8Blk ? f32x4{0.f, 0.f, 0.f, 0.f} : out[j][f];
#pragma unroll
                    for (int c = 0; c < FR; ++c)
                        d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x[u][f][c]), w[c], d, 0, 0, 0);
                    if constexpr (KIND == kFp8Blk) {
#pragma unroll
                        for (int v = 0; v < 4; ++v) out[j][f][v] = fmaf(sc, d[v], out[j][f][v]);
                    } else {
                        out[j][f] = d;
                    }
                }
            }
        }
    }
    if constexpr (KIND == kFp8Row) {
        const float* sc = static_cast<const float*>(p.w->scales) + static_cast<int64_t>(p.e) * N;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const float s = sc[min(p.n0 + CPL * m + j, N - 1)];
#pragma unroll
            for (int f = 0; f < TF; ++f) out[j][f] *= s;
        }
    }
}

// GPTQ words [E, K/8, N]: a lane reads 4 consecutive columns of a k-octet, one column per MFMA.  Each
// unit of 32 * STEPS k of one quantisation group (the whole group up to 128 k, half of one of 256, so that
// two units fit the registers) contributes s * (acc - (128 + z) * sum_k x), the sum from one more MFMA
// against ones.  Two register sets take turns, so a unit's loads are in flight during the other's products.
template <int STEPS, int TF>
struct Int4Set {
    u32x4 q[STEPS], x[STEPS][TF];
    uint2 s;
    uint32_t z;
};

template <int STEPS, int TF>
__device__ __forceinline__ void panel_int4(const Panel& p, const int (&arow)[TF], f32x4 (&out)[4][TF]) {
    constexpr int UK = STEPS * 32;
    const int lane = threadIdx.x & 63, m = lane & 15, kq = lane >> 4;
    const int N = p.N, K = p.K;
    const int units = K / UK, per = p.group / UK;  // units per group: 1 or 2
    const int64_t words = static_cast<int64_t>(K / 8) * N, cells = static_cast<int64_t>(K / p.group) * N;
    const __amdgpu_buffer_rsrc_t wbuf = buffer(static_cast<const int32_t*>(p.w->data) + p.e * words, words * 4);
    const __amdgpu_buffer_rsrc_t sbuf = buffer(static_cast<const uint16_t*>(p.w->scales) + p.e * cells, cells * 2);
    const __amdgpu_buffer_rsrc_t zbuf = buffer(p.w->qzeros + p.e * (cells / 8), cells / 2);
    const int ncol = p.n0 + 4 * m, zshift = 16 * (m & 1);
    const int g0 = __builtin_amdgcn_readfirstlane(p.part * units / p.parts);
    const int g1 = __builtin_amdgcn_readfirstlane((p.part + 1) * units / p.parts);
    auto load = [&](Int4Set<STEPS, TF>& R, int g) __attribute__((always_inline)) {
        const bool in = g < g1;
        const int sg = per == 1 ? g : g >> 1;
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
            R.q[st] = load16(wbuf, in ? ((g * (UK / 8) + st * 4 + kq) * N + ncol) * 4 : kPast);
        R.s = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(sbuf, in ? (sg * N + ncol) * 2 : kPast, 0, 0));
        R.z = __builtin_amdgcn_raw_buffer_load_b32(zbuf, in ? (sg * (N / 8) + ncol / 8) * 4 : kPast, 0, 0);
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
#pragma unroll
            for (int f = 0; f < TF; ++f)
                R.x[st][f] = load16(p.abuf, in && arow[f] != kPast ? arow[f] + (g * UK + st * 32 + kq * 8) * 2 : kPast);
    };
    const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
    uint32_t nib_mask, bf16_128;
    asm volatile("v_mov_b32 %0, 0x000f000f" : "=v"(nib_mask));
    asm volatile("v_mov_b32 %0, 0x43004300" : "=v"(bf16_128));
    auto compute = [&](const Int4Set<STEPS, TF>& R) __attribute__((always_inline)) {
        f32x4 acc[4][TF], accx[TF];
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            accx[f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            bf16x8 xf[TF];
#pragma unroll
            for (int f = 0; f < TF; ++f) {
                xf[f] = as_bf16x8(permute_k(R.x[st][f]));
                accx[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[f], as_bf16x8(ones), accx[f], 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 w = as_bf16x8(dequant_word(R.q[st][j], nib_mask, bf16_128));
#pragma unroll
                for (int f = 0; f < TF; ++f)
                    acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[f], w, acc[j][f], 0, 0, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t sbits = (j < 2 ? R.s.x : R.s.y) >> (16 * (j & 1));
            const float sc = f16_to_f32(static_cast<uint16_t>(sbits & 0xffffu));
            const float zz = 128.0f + static_cast<float>((R.z >> (zshift + 4 * j)) & 0xfu);
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int v = 0; v < 4; ++v) out[j][f][v] = fmaf(sc, fmaf(-zz, accx[f][v], acc[j][f][v]), out[j][f][v]);
        }
    };
    // (a unit past the wave's last loads zeros: its scale is 0, so it adds nothing)
    Int4Set<STEPS, TF> ra, rb;
    load(ra, g0);
    for (int g = g0; g < g1; g += 2) {
        load(rb, g + 1);
        __builtin_amdgcn_sched_barrier(0);
        compute(ra);
        __builtin_amdgcn_sched_barrier(0);
        load(ra, g + 2);
        __builtin_amdgcn_sched_barrier(0);
        compute(rb);
        __builtin_amdgcn_sched_barrier(0);
    }
}

// the weight types: columns per lane and the panel routine
template <int KIND, int STEPS, int TF>
struct Kind {
    static constexpr int CPL = KIND == kInt4 ? 4 : 1;
    static constexpr int NCOL = 16 * CPL;
    __device__ static __forceinline__ void panel(const Panel& p, const int (&arow)[TF], f32x4 (&out)[CPL][TF]) {
        if constexpr (KIND == kInt4) panel_int4<STEPS, TF>(p, arow, out);
        else panel_rows<KIND, CPL, TF, 8>(p, arow, out);
    }
};

// ------------------------------------------------------------------ launch 1: routing, gate/up, SiLU
template <int KIND, int STEPS, int TF, int NW>
__global__ __launch_bounds__(64 * NW, 2) void few_gate_up_kernel(FewArgs a) {
    using W = Kind<KIND, STEPS, TF>;
    constexpr int CPL = W::CPL, NCOL = W::NCOL, NT = 64 * NW;
    constexpr int PARTS = NW / 2;  // waves of one projection
    __shared__ Routed r;
    __shared__ f32x4 red[2][NW][CPL][TF][64];  // two sets: an item's sums are read while the next one's form
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

    if (blockIdx.x == 0) {  // ids and weights for few_down and the caller
        for (int t = wave; t < a.T; t += NW) {
            switch ((a.E + 63) / 64) {
                case 1: route_tokens<1, 1>(a.logits, t, 0, a.T, a.E, a.top_k, a.renorm, a.ids, a.w, lane); break;
                case 2: route_tokens<2, 1>(a.logits, t, 0, a.T, a.E, a.top_k, a.renorm, a.ids, a.w, lane); break;
                case 3: route_tokens<3, 1>(a.logits, t, 0, a.T, a.E, a.top_k, a.renorm, a.ids, a.w, lane); break;
                default: route_tokens<4, 1>(a.logits, t, 0, a.T, a.E, a.top_k, a.renorm, a.ids, a.w, lane); break;
            }
        }
        return;
    }
    if (tid < kMaxE) r.tok[tid] = 0;
    __syncthreads();
    select_all<NW>(a, r, wave, lane);
    __syncthreads();
    list_active<NW>(r, a.E);

    const int panels = (a.I + NCOL - 1) / NCOL;
    const int items = __builtin_amdgcn_readfirstlane(r.n_act) * panels;
    const int proj = wave / PARTS;
    Panel p;
    p.w = proj ? &a.up : &a.gate;
    p.N = a.I;
    p.K = a.H;
    p.group = a.group;
    p.part = wave % PARTS;
    p.parts = PARTS;
    p.abuf = buffer(a.x, static_cast<int64_t>(a.T) * a.H * 2);
    int arow[TF];
#pragma unroll
    for (int f = 0; f < TF; ++f) {
        const int t = 16 * f + (lane & 15);
        arow[f] = t < a.T ? t * a.H * 2 : kPast;
    }
    int set = 0;
    for (int it = blockIdx.x - 1; it < items; it += gridDim.x - 1, set ^= 1) {
        const int i = it / panels;
        p.e = __builtin_amdgcn_readfirstlane(r.act[i]);
        p.n0 = (it - i * panels) * NCOL;
        f32x4 out[CPL][TF];
#pragma unroll
        for (int j = 0; j < CPL; ++j)
#pragma unroll
            for (int f = 0; f < TF; ++f) out[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        W::panel(p, arow, out);
#pragma unroll
        for (int j = 0; j < CPL; ++j)
#pragma unroll
            for (int f = 0; f < TF; ++f) red[set][wave][j][f][lane] = out[j][f];
        __syncthreads();
        // one (lane, v) of the panel per thread: token 16 f + 4 (sl / 16) + v, columns CPL * (sl % 16) ..
        const uint32_t mask = r.tok[p.e];
        for (int c = tid; c < 256 * TF; c += NT) {
            const int f = c >> 8, v = (c >> 6) & 3, sl = c & 63;
            const int t = 16 * f + 4 * (sl >> 4) + v;
            const int col = p.n0 + CPL * (sl & 15);
            if (!((mask >> t) & 1u) || col >= a.I) continue;
            float h[CPL];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                float g = 0.f, u = 0.f;
#pragma unroll
                for (int w = 0; w < PARTS; ++w) {
                    g += red[set][w][j][f][sl][v];
                    u += red[set][PARTS + w][j][f][sl][v];
                }
                h[j] = silu_mul(g, u);
            }
            uint16_t* dst = a.hs + static_cast<int64_t>(t * a.top_k + r.slot[t][p.e]) * a.I + col;
            if constexpr (CPL == 4)
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
            else
                *dst = f32_to_bf16(h[0]);
        }
    }
}

// ------------------------------------------------------------------ launch 2: down, weighted sum
template <int KIND, int STEPS, int TF, int NW>
__global__ __launch_bounds__(64 * NW, 2) void few_down_kernel(FewArgs a) {
    using W = Kind<KIND, STEPS, TF>;
    constexpr int CPL = W::CPL, NCOL = W::NCOL, NT = 64 * NW;
    __shared__ Routed r;
    __shared__ float s_w[kFewTokens * kFewTopK];
    __shared__ f32x4 red[NW][CPL][TF][64];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int panel = blockIdx.x / a.splits, s = blockIdx.x - panel * a.splits;

    if (tid < kMaxE) r.tok[tid] = 0;
    __syncthreads();
    for (int q = tid; q < a.T * a.top_k; q += NT) {
        const int e = a.ids[q], t = q / a.top_k;
        s_w[q] = a.w[q];
        if (e >= 0 && e < a.E) {
            r.slot[t][e] = static_cast<uint8_t>(q - t * a.top_k);
            atomicOr(&r.tok[e], 1u << t);
        }
    }
    __syncthreads();
    list_active<NW>(r, a.E);
    const int n_act = __builtin_amdgcn_readfirstlane(r.n_act);
    const int splits = max(1, min(a.splits, n_act));
    if (s >= splits) return;  // the whole workgroup

    Panel p;
    p.w = &a.down;
    p.N = a.H;
    p.K = a.I;
    p.group = a.group;
    p.part = wave;
    p.parts = NW;
    p.n0 = panel * NCOL;
    p.abuf = buffer(a.hs, static_cast<int64_t>(a.T) * a.top_k * a.I * 2);
    f32x4 sum[CPL][TF];
#pragma unroll
    for (int j = 0; j < CPL; ++j)
#pragma unroll
        for (int f = 0; f < TF; ++f) sum[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int i = s; i < n_act; i += splits) {
        p.e = __builtin_amdgcn_readfirstlane(r.act[i]);
        const uint32_t mask = r.tok[p.e];
        int arow[TF];
        f32x4 out[CPL][TF];
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            const int t = 16 * f + (lane & 15);
            arow[f] = (mask >> t) & 1u ? (t * a.top_k + r.slot[t][p.e]) * a.I * 2 : kPast;
#pragma unroll
            for (int j = 0; j < CPL; ++j) out[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        W::panel(p, arow, out);
#pragma unroll
        for (int f = 0; f < TF; ++f)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int t = 16 * f + 4 * (lane >> 4) + v;
                if (!((mask >> t) & 1u)) continue;
                const float w = s_w[t * a.top_k + r.slot[t][p.e]];
#pragma unroll
                for (int j = 0; j < CPL; ++j) sum[j][f][v] = fmaf(w, out[j][f][v], sum[j][f][v]);
            }
    }
#pragma unroll
    for (int j = 0; j < CPL; ++j)
#pragma unroll
        for (int f = 0; f < TF; ++f) red[wave][j][f][lane] = sum[j][f];
    __syncthreads();
    constexpr int CELLS = 256 * TF;  // (lane, v) cells of CPL columns each
    constexpr int PER = (CELLS + NT - 1) / NT;
    float res[PER][CPL];
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int c = tid + q * NT;
        if (c >= CELLS) break;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < NW; ++w) v += red[w][j][c >> 8][c & 63][(c >> 6) & 3];
            res[q][j] = v;
        }
    }
    if (splits > 1) {
        // partial panels [panel][s][j][cell], written and read device-coherently (relaxed agent-scope
        // accesses); complete (vmcnt 0) before the workgroup counts itself
        float* part = a.part + static_cast<int64_t>(panel) * a.splits * (CPL * CELLS);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int c = tid + q * NT;
            if (c >= CELLS) break;
#pragma unroll
            for (int j = 0; j < CPL; ++j)
                __hip_atomic_store(part + (s * CPL + j) * CELLS + c, res[q][j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0)
            s_last = __hip_atomic_fetch_add(&a.cnt[panel], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
        __syncthreads();
        if (!s_last) return;
        if (tid == 0) __hip_atomic_store(&a.cnt[panel], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int c = tid + q * NT;
            if (c >= CELLS) break;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                float v = 0.f;
                for (int o = 0; o < splits; ++o)
                    v += __hip_atomic_load(part + (o * CPL + j) * CELLS + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                res[q][j] = v;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int c = tid + q * NT;
        if (c >= CELLS) break;
        const int t = 16 * (c >> 8) + 4 * ((c & 63) >> 4) + ((c >> 6) & 3);
        const int col = p.n0 + CPL * (c & 15);
        if (t >= a.T || col >= a.H) continue;
        uint16_t* dst = a.out + static_cast<int64_t>(t) * a.H + col;
        if constexpr (CPL == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(res[q][0], res[q][1]), pack_bf16x2(res[q][2], res[q][3]));
        else
            *dst = f32_to_bf16(res[q][0]);
    }
}

constexpr int kWaves = 8;

template <int KIND, int STEPS, int TF>
hipError_t launch_kind(const FewArgs& a, hipStream_t s) {
    using W = Kind<KIND, STEPS, TF>;
    const int most = a.T * a.top_k < a.E ? a.T * a.top_k : a.E;  // active experts at most
    const int64_t items = static_cast<int64_t>(most) * ((a.I + W::NCOL - 1) / W::NCOL);
    const int grid = static_cast<int>(items < kFewGrid ? items : kFewGrid);
    few_gate_up_kernel<KIND, STEPS, TF, kWaves><<<grid + 1, 64 * kWaves, 0, s>>>(a);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int panels = (a.H + W::NCOL - 1) / W::NCOL;
    few_down_kernel<KIND, STEPS, TF, kWaves><<<panels * a.splits, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
}

template <int TF>
hipError_t launch_tf(int kind, const FewArgs& a, hipStream_t s) {
    switch (kind) {
        case kBf16: return launch_kind<kBf16, 1, TF>(a, s);
        case kFp8Row: return launch_kind<kFp8Row, 1, TF>(a, s);
        case kFp8Blk: return launch_kind<kFp8Blk, 1, TF>(a, s);
        default: break;
    }
    if (kind != kInt4) return hipErrorInvalidValue;
    switch (a.group) {
        case 32: return launch_kind<kInt4, 1, TF>(a, s);
        case 64: return launch_kind<kInt4, 2, TF>(a, s);
        case 128:
        case 256: return launch_kind<kInt4, 4, TF>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_few_tokens(int kind, const FewArgs& a, hipStream_t s) {
    return a.T <= 16 ? launch_tf<1>(kind, a, s) : launch_tf<2>(kind, a, s);
}

}  // namespace moe
