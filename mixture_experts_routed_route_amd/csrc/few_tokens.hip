// The whole routed layer for at most 32 tokens in two launches:
//
//   few_gate_up   top-k softmax routing, then h[p] = SiLU(x Wg^T) * (x Wu^T) of every (token,
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
// Roundings: h is kept as the sum of two bf16 values (16 bits of it: the operand type of the second
// product, whose spare MFMA rate makes the second part free, where one bf16 value alone would put as much
// error into out as out's own rounding); the expert outputs are not rounded before the weighted sum; out
// once to bf16.  fp8 weights convert to
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

typedef float f32x2 __attribute__((ext_vector_type(2)));

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

// ------------------------------------------------------------------ streaming a panel's weights
// A wave walks a list of granules: UK consecutive k of one column panel (16 * CPL columns n0 + CPL * m + j,
// m = lane % 16) of one expert.  Granules of one segment (an expert's panel) add up in `out`:
//   out[j][f] += sum_k A(token, k) * W(column, k), tokens 16 f + 4 (lane / 16) + v
// The next granule's loads (weights and token rows, of the next segment too) are always in flight while
// one is multiplied: two register sets take turns.
struct Seg {
    int e, n0;                     // expert, first column
    __amdgpu_buffer_rsrc_t w;      // its matrix
    __amdgpu_buffer_rsrc_t s, z;   // int4: its scales and zeros
    const float* bscale;           // block scales of the panel's 128 rows
    int woff[4];                   // byte offset of the lane's chunk of column j at k 0
};

struct Matrix {
    const FewWeight* w;
    int N, K, group;
};

// Where a stream's token rows come from: LDS (kTile: the rows of x, the same for every expert, laid out as
// MFMA operands by stage_x), memory, row by row (kRow: x where LDS cannot hold it), or memory as pairs of
// bf16 values whose sum is the operand (kPair: the rows of h, which differ from expert to expert).
enum { kTile, kRow, kPair };

template <int TF>
struct TokenRows {
    __amdgpu_buffer_rsrc_t buf;
    int lo;  // kPair: byte offset of the low parts
};

template <int TF>
struct TokenTile {
    const uint16_t* at[TF];  // this lane's part of fragment 0 of tokens 16 f ..
    int step[TF];            // elements from one fragment (32 k) to the next
};

// [E, N, K] weights, K contiguous: a load takes 16 bytes of 4 consecutive k chunks of 16 rows.  A granule
// is US loads per column set.
template <int KIND, int CPL_, int TF, int US, int SRC>
struct Rows {
    static constexpr int CPL = CPL_;
    static constexpr int ES = KIND == kBf16 ? 2 : 1;
    static constexpr int FR = KIND == kBf16 ? 1 : 2;  // MFMA k-steps (32 k) per load
    static constexpr int KS = 32 * FR;                // k per load
    static constexpr int UK = KS * US;
    static constexpr int NB = UK > 128 ? UK / 128 : 1;  // block scales of a granule
    static_assert(KIND != kFp8Blk || 128 % UK == 0 || UK % 128 == 0, "granules and blocks of k nest");
    using X = std::conditional_t<SRC == kTile, TokenTile<TF>, TokenRows<TF>>;
    static constexpr int NP = SRC == kPair ? 2 : 1;  // bf16 parts of a token operand
    struct Set {
        u32x4 b[US][CPL], x[SRC == kTile ? 1 : US][TF][FR][NP];
        float sc[NB];
    };
    // the 8 k of chunk c of a row: which 32-k fragment, and which quarter wave of it
    __device__ static __forceinline__ void place(int c, int& frag, int& kq) {
        frag = FR == 1 ? c >> 2 : (c >> 3) * 2 + (c & 1);
        kq = FR == 1 ? c & 3 : (c >> 1) & 3;
    }
    __device__ static __forceinline__ u32x4 prepare(u32x4 v) { return v; }
    __device__ static __forceinline__ int granules(const Matrix& m) { return (m.K + UK - 1) / UK; }
    __device__ static __forceinline__ void open(const Matrix& m, int e, int n0, Seg& g) {
        const int lane = threadIdx.x & 63, kq = lane >> 4;
        const int64_t mat = static_cast<int64_t>(m.N) * m.K * ES;
        g.e = e;
        g.n0 = n0;
        g.w = buffer(static_cast<const char*>(m.w->data) + e * mat, mat);
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const int n = n0 + CPL * (lane & 15) + j;
            g.woff[j] = n < m.N ? n * m.K * ES + kq * 16 : kPast;
        }
        if constexpr (KIND == kFp8Blk)
            g.bscale = static_cast<const float*>(m.w->scales) +
                       (static_cast<int64_t>(e) * ((m.N + 127) / 128) + n0 / 128) * ((m.K + 127) / 128);
    }
    // granule i (of none: zeros)
    __device__ static __forceinline__ void load(Set& r, const Matrix& m, const Seg& g, const X& x,
                                                const int (&arow)[TF], int i, bool some) {
        const int kq = (threadIdx.x & 63) >> 4;
#pragma unroll
        for (int u = 0; u < US; ++u) {
            const int k = (i * US + u) * KS;
            const bool in = some && k + kq * (16 / ES) < m.K;
#pragma unroll
            for (int j = 0; j < CPL; ++j) r.b[u][j] = load16(g.w, in ? g.woff[j] + k * ES : kPast);
        }
        if constexpr (SRC != kTile)
#pragma unroll
        for (int u = 0; u < US; ++u) {
            const int k = (i * US + u) * KS;
            const bool in = some && k + kq * (16 / ES) < m.K;
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int c = 0; c < FR; ++c)
#pragma unroll
                    for (int h = 0; h < NP; ++h)
                        r.x[u][f][c][h] =
                            load16(x.buf, in && arow[f] != kPast ? arow[f] + (k + kq * (8 * FR) + c * 8) * 2 + h * x.lo : kPast);
        }
        if constexpr (KIND == kFp8Blk)
#pragma unroll
            for (int b = 0; b < NB; ++b) r.sc[b] = some ? g.bscale[min(i * UK / 128 + b, (m.K + 127) / 128 - 1)] : 0.f;
    }
    __device__ static __forceinline__ void multiply(const Set& r, const X& x, int i, f32x4 (&out)[CPL][TF]) {
        bf16x8 xf[US][TF][FR][NP];
#pragma unroll
        for (int u = 0; u < US; ++u)
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int c = 0; c < FR; ++c) {
                    if constexpr (SRC == kTile)
                        xf[u][f][c][0] = *reinterpret_cast<const bf16x8*>(x.at[f] + ((i * US + u) * FR + c) * x.step[f]);
                    else
#pragma unroll
                        for (int h = 0; h < NP; ++h) xf[u][f][c][h] = as_bf16x8(r.x[u][f][c][h]);
                }
        constexpr int UB = KIND == kFp8Blk ? US / NB : US;  // loads under one scale
#pragma unroll
        for (int j = 0; j < CPL; ++j)
#pragma unroll
            for (int b = 0; b < US / UB; ++b) {
                f32x4 d[TF];
#pragma unroll
                for (int f = 0; f < TF; ++f) d[f] = KIND == kFp8Blk ? f32x4{0.f, 0.f, 0.f, 0.f} : out[j][f];
#pragma unroll
                for (int u = b * UB; u < (b + 1) * UB; ++u)
#pragma unroll
                    for (int c = 0; c < FR; ++c) {
                        const bf16x8 w = KIND == kBf16 ? as_bf16x8(r.b[u][j]) : fp8_to_bf16(r.b[u][j][2 * c], r.b[u][j][2 * c + 1]);
#pragma unroll
                        for (int f = 0; f < TF; ++f)
#pragma unroll
                            for (int h = 0; h < NP; ++h)
                                d[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[u][f][c][h], w, d[f], 0, 0, 0);
                    }
#pragma unroll
                for (int f = 0; f < TF; ++f)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        out[j][f][v] = KIND == kFp8Blk ? fmaf(r.sc[b], d[f][v], out[j][f][v]) : d[f][v];
            }
    }
    // channel scales, once per segment
    __device__ static __forceinline__ void close(const Matrix& m, int e, int n0, f32x4 (&out)[CPL][TF]) {
        if constexpr (KIND == kFp8Row) {
            const float* sc = static_cast<const float*>(m.w->scales) + static_cast<int64_t>(e) * m.N;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const float s = sc[min(n0 + CPL * static_cast<int>(threadIdx.x & 15) + j, m.N - 1)];
#pragma unroll
                for (int f = 0; f < TF; ++f) out[j][f] *= s;
            }
        }
    }
};

// GPTQ words [E, K/8, N]: a lane reads 4 consecutive columns of a k-octet, one column per MFMA.  A granule
// of 32 * STEPS k lies in one quantisation group and contributes s * (acc - (128 + z) * sum_k x), the sum from one more MFMA against ones.
template <int STEPS, int TF, int SRC>
struct Words {
    static constexpr int CPL = 4;
    static constexpr int UK = STEPS * 32;
    using X = std::conditional_t<SRC == kTile, TokenTile<TF>, TokenRows<TF>>;
    static constexpr int NP = SRC == kPair ? 2 : 1;  // bf16 parts of a token operand
    struct Set {
        u32x4 q[STEPS], x[SRC == kTile ? 1 : STEPS][TF][NP];
        uint2 s;
        uint32_t z;
    };
    __device__ static __forceinline__ void place(int c, int& frag, int& kq) {
        frag = c >> 2;
        kq = c & 3;
    }
    __device__ static __forceinline__ u32x4 prepare(u32x4 v) { return permute_k(v); }
    __device__ static __forceinline__ int granules(const Matrix& m) { return m.K / UK; }
    __device__ static __forceinline__ void open(const Matrix& m, int e, int n0, Seg& g) {
        const int64_t words = static_cast<int64_t>(m.K / 8) * m.N, cells = static_cast<int64_t>(m.K / m.group) * m.N;
        g.e = e;
        g.n0 = n0;
        g.w = buffer(static_cast<const int32_t*>(m.w->data) + e * words, words * 4);
        g.s = buffer(static_cast<const uint16_t*>(m.w->scales) + e * cells, cells * 2);
        g.z = buffer(m.w->qzeros + e * (cells / 8), cells / 2);
    }
    __device__ static __forceinline__ void load(Set& r, const Matrix& m, const Seg& g, const X& x,
                                                const int (&arow)[TF], int i, bool some) {
        const int lane = threadIdx.x & 63, kq = lane >> 4;
        const int ncol = g.n0 + 4 * (lane & 15);
        const int sg = i * UK / m.group;
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
            r.q[st] = load16(g.w, some ? ((i * (UK / 8) + st * 4 + kq) * m.N + ncol) * 4 : kPast);
        r.s = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(g.s, some ? (sg * m.N + ncol) * 2 : kPast, 0, 0));
        r.z = __builtin_amdgcn_raw_buffer_load_b32(g.z, some ? (sg * (m.N / 8) + ncol / 8) * 4 : kPast, 0, 0);
        if constexpr (SRC != kTile)
#pragma unroll
        for (int st = 0; st < STEPS; ++st)
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int h = 0; h < NP; ++h)
                    r.x[st][f][h] =
                        load16(x.buf, some && arow[f] != kPast ? arow[f] + (i * UK + st * 32 + kq * 8) * 2 + h * x.lo : kPast);
    }
    __device__ static __forceinline__ void multiply(const Set& r, const X& x, int i, f32x4 (&out)[4][TF]) {
        const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        const int zshift = 16 * (threadIdx.x & 1);
        uint32_t nib_mask, bf16_128;
        asm("v_mov_b32 %0, 0x000f000f" : "=v"(nib_mask));
        asm("v_mov_b32 %0, 0x43004300" : "=v"(bf16_128));
        f32x4 acc[4][TF], accx[TF];
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            accx[f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            bf16x8 xf[TF][NP];
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int h = 0; h < NP; ++h) {
                    if constexpr (SRC == kTile) xf[f][h] = *reinterpret_cast<const bf16x8*>(x.at[f] + (i * STEPS + st) * x.step[f]);
                    else xf[f][h] = as_bf16x8(permute_k(r.x[st][f][h]));
                    accx[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[f][h], as_bf16x8(ones), accx[f], 0, 0, 0);
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 w = as_bf16x8(dequant_word(r.q[st][j], nib_mask, bf16_128));
#pragma unroll
                for (int f = 0; f < TF; ++f)
#pragma unroll
                    for (int h = 0; h < NP; ++h)
                        acc[j][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[f][h], w, acc[j][f], 0, 0, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t sbits = (j < 2 ? r.s.x : r.s.y) >> (16 * (j & 1));
            const float sc = f16_to_f32(static_cast<uint16_t>(sbits & 0xffffu));
            const float zz = 128.0f + static_cast<float>((r.z >> (zshift + 4 * j)) & 0xfu);
#pragma unroll
            for (int f = 0; f < TF; ++f)
#pragma unroll
                for (int v = 0; v < 4; ++v) out[j][f][v] = fmaf(sc, fmaf(-zz, accx[f][v], acc[j][f][v]), out[j][f][v]);
        }
    }
    __device__ static __forceinline__ void close(const Matrix&, int, int, f32x4 (&)[4][TF]) {}
};

// The weight types' streams.  The granule is what two register sets, the sums and the addresses leave room
// for, given the waves that are to share a compute unit: sixteen (128 registers) with x in LDS or in memory,
// twelve with pairs, eight for int4 with two token fragments from memory.  2 to 8 KB of weights a wave are
// in flight.
template <int KIND, int STEPS, int TF, int SRC>
using Stream = std::conditional_t<
    KIND == kInt4, Words<STEPS, TF, SRC>,
    Rows<KIND, 2, TF, SRC == kTile ? (KIND == kBf16 ? (TF == 1 ? 4 : 3) : (TF == 1 ? 4 : 2)) : KIND == kBf16 ? (TF == 1 ? 3 : 2) : (TF == 1 ? 2 : 1), SRC>>;
constexpr int min_waves(int kind, int tf, int src) {
    return kind == kInt4 && tf == 2 && src != kTile ? 2 : src == kPair ? 3 : 4;
}

// The wave's granules: `n` of them from granule g of segment `seg`, the segments' granules being [gb, ge) and
// their numbers `stride` apart.  open_at(seg, Seg&, arow) opens a segment; flush(seg, out) takes its sums
// (before the next granule is multiplied, with the loads after it in flight).
template <class S, int TF, class Open, class Flush>
__device__ __forceinline__ void walk(const Matrix& m, const typename S::X& x, int n, int seg, int g, int gb, int ge,
                                     int stride, Open open_at, Flush flush) {
    typename S::Set ra, rb;
    Seg cur;
    int arow[TF];
    f32x4 out[S::CPL][TF];
    auto zero = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < S::CPL; ++j)
#pragma unroll
            for (int f = 0; f < TF; ++f) out[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    int lseg = seg, lg = g;  // the granule that the last loads took
    auto fetch = [&](typename S::Set& r, bool some) __attribute__((always_inline)) {
        if (some && ++lg == ge) {
            lg = gb;
            lseg += stride;
            open_at(lseg, cur, arow);
        }
        S::load(r, m, cur, x, arow, lg, some);
        __builtin_amdgcn_sched_barrier(0);
    };
    int left = n;
    auto take = [&](const typename S::Set& r) __attribute__((always_inline)) {
        S::multiply(r, x, g, out);
        __builtin_amdgcn_sched_barrier(0);
        --left;
        if (++g == ge || left == 0) {
            flush(seg, out);
            zero();
            g = gb;
            seg += stride;
        }
    };
    zero();
    if (n <= 0) return;
    open_at(lseg, cur, arow);
    S::load(ra, m, cur, x, arow, lg, true);
    while (true) {
        fetch(rb, left > 1);
        take(ra);
        if (left == 0) break;
        fetch(ra, left > 1);
        take(rb);
        if (left == 0) break;
    }
}

// barrier that orders LDS only: loads from memory stay in flight
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ------------------------------------------------------------------ launch 1: routing, gate/up, SiLU
// LDS for the rows of x: what the panel sums and the routing state leave of 160 KB
constexpr int x_bytes(int cpl, int nw) { return 163840 - 256 - static_cast<int>(sizeof(Routed)) - nw * cpl * 1024; }

// token rows kept for fragment f: a power of two, so that lanes past it read rows again (never stored)
__host__ __device__ inline int x_rows(int T, int f) {
    int r = 1;
    while (r < 16 && r < T - 16 * f) r *= 2;
    return r;
}

// x in LDS as MFMA operands: fragment by fragment (32 k), quarter wave by quarter wave (8 k), row by row.
// Chunks past K are zeros (the weights' zeros there must not meet stale bits); rows past T are left as
// they are (an MFMA row only reaches its own results).
template <class S, int TF, int NT>
__device__ __forceinline__ void stage_x(const FewArgs& a, uint16_t* lds, int kpad, typename S::X& x) {
    const __amdgpu_buffer_rsrc_t buf = buffer(a.x, static_cast<int64_t>(a.T) * a.H * 2);
    const int chunks = kpad / 8, lane = threadIdx.x & 63;
    int base = 0;
#pragma unroll
    for (int f = 0; f < TF; ++f) {
        const int rows = x_rows(a.T, f), t0 = 16 * f, n = min(a.T - t0, 16);
        x.step[f] = rows * 32;
        x.at[f] = lds + base + ((lane >> 4) * rows + (lane & (rows - 1))) * 8;
        // four chunks a thread in flight
        for (int c0 = threadIdx.x; c0 < n * chunks; c0 += 4 * NT) {
            u32x4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int c = c0 + u * NT, t = c / chunks, k = (c - t * chunks) * 8;
                v[u] = load16(buf, c < n * chunks && k < a.H ? ((t0 + t) * a.H + k) * 2 : kPast);
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int c = c0 + u * NT, t = c / chunks;
                if (c >= n * chunks) break;
                int frag, kq;
                S::place(c - t * chunks, frag, kq);
                *reinterpret_cast<u32x4*>(lds + base + (frag * 4 * rows + kq * rows + t) * 8) = S::prepare(v[u]);
            }
        }
        base += rows * kpad;
    }
}

template <int KIND, int STEPS, int TF, int NW, int SRC>
__global__ __launch_bounds__(64 * NW, min_waves(KIND, TF, SRC)) void few_gate_up_kernel(FewArgs a) {
    using S = Stream<KIND, STEPS, TF, SRC>;
    constexpr int CPL = S::CPL, NCOL = 16 * CPL, NT = 64 * NW;
    constexpr int PARTS = NW / 2;  // waves of one projection
    __shared__ Routed r;
    __shared__ f32x4 red[NW][CPL][64];
    __shared__ __attribute__((aligned(16))) uint16_t xl[SRC == kTile ? x_bytes(CPL, NW) / 2 : 8];
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
    const int proj = wave / PARTS, part = wave % PARTS;
    const Matrix m{proj ? &a.up : &a.gate, a.I, a.H, a.group};
    const int grans = S::granules(m);
    typename S::X x;
    if (tid < kMaxE) r.tok[tid] = 0;
    if constexpr (SRC == kTile) stage_x<S, TF, NT>(a, xl, grans * S::UK, x);
    else x.buf = buffer(a.x, static_cast<int64_t>(a.T) * a.H * 2);
    lds_barrier();
    select_all<NW>(a, r, wave, lane);
    lds_barrier();
    list_active<NW>(r, a.E);

    const int panels = (a.I + NCOL - 1) / NCOL;
    const int items = __builtin_amdgcn_readfirstlane(r.n_act) * panels;
    const int stride = gridDim.x - 1, first = blockIdx.x - 1;
    const int mine = first < items ? (items - first + stride - 1) / stride : 0;
    const int gb = __builtin_amdgcn_readfirstlane(part * grans / PARTS);
    const int ge = __builtin_amdgcn_readfirstlane((part + 1) * grans / PARTS);
    auto open_at = [&](int it, Seg& g, int (&arow)[TF]) __attribute__((always_inline)) {
        const int i = it / panels;
        S::open(m, __builtin_amdgcn_readfirstlane(r.act[i]), (it - i * panels) * NCOL, g);
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            const int t = 16 * f + (lane & 15);
            arow[f] = t < a.T ? t * a.H * 2 : kPast;
        }
    };
    // the item's sums over the waves, one token fragment at a time; every wave flushes every item
    auto flush = [&](int it, f32x4 (&out)[CPL][TF]) __attribute__((always_inline)) {
        const int i = it / panels;
        const int e = __builtin_amdgcn_readfirstlane(r.act[i]), n0 = (it - i * panels) * NCOL;
        S::close(m, e, n0, out);
        const uint32_t mask = r.tok[e];
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            lds_barrier();  // the sums before these have been read
#pragma unroll
            for (int j = 0; j < CPL; ++j) red[wave][j][lane] = out[j][f];
            lds_barrier();
            // one (lane, v) of the panel per thread: token 16 f + 4 (sl / 16) + v, columns CPL * (sl % 16) ..
            const int v = (tid >> 6) & 3, sl = tid & 63;
            const int t = 16 * f + 4 * (sl >> 4) + v;
            const int col = n0 + CPL * (sl & 15);
            if (tid >= 256 || !((mask >> t) & 1u) || col >= a.I) continue;
            float h[CPL];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                float g = 0.f, u = 0.f;
#pragma unroll
                for (int w = 0; w < PARTS; ++w) {
                    g += red[w][j][sl][v];
                    u += red[PARTS + w][j][sl][v];
                }
                h[j] = silu_mul(g, u);
            }
            // the value and what its rounding to bf16 left, in two planes
            uint16_t* dst = a.hs + static_cast<int64_t>(t * a.top_k + r.slot[t][e]) * a.I + col;
            uint16_t* rest = dst + static_cast<int64_t>(a.T) * a.top_k * a.I;
            uint32_t hi[CPL / 2], lo[CPL / 2];
#pragma unroll
            for (int j = 0; j < CPL / 2; ++j) {
                hi[j] = pack_bf16x2(h[2 * j], h[2 * j + 1]);
                // (an infinite value has no rest: inf - inf would be NaN)
                const float h0 = bf_lo(hi[j]), h1 = bf_hi(hi[j]);
                lo[j] = pack_bf16x2(fabsf(h0) < INFINITY ? h[2 * j] - h0 : 0.f, fabsf(h1) < INFINITY ? h[2 * j + 1] - h1 : 0.f);
            }
            if constexpr (CPL == 4) {
                *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(rest) = make_uint2(lo[0], lo[1]);
            } else {
                *reinterpret_cast<uint32_t*>(dst) = hi[0];
                *reinterpret_cast<uint32_t*>(rest) = lo[0];
            }
        }
    };
    if (ge > gb) {
        walk<S, TF>(m, x, mine * (ge - gb), first, gb, gb, ge, stride, open_at, flush);
    } else {  // fewer granules than waves: this one only adds zeros
        f32x4 out[CPL][TF];
#pragma unroll
        for (int j = 0; j < CPL; ++j)
#pragma unroll
            for (int f = 0; f < TF; ++f) out[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < mine; ++i) flush(first + i * stride, out);
    }
}

// ------------------------------------------------------------------ launch 2: down, weighted sum
// The granules of a column panel, expert by expert of the work list, are one sequence; the waves of the
// panel's workgroups take equal consecutive shares of it, whatever the number of active experts.
template <int KIND, int STEPS, int TF, int NW>
__global__ __launch_bounds__(64 * NW, min_waves(KIND, TF, kPair)) void few_down_kernel(FewArgs a) {
    using S = Stream<KIND, STEPS, TF, kPair>;
    constexpr int CPL = S::CPL, NCOL = 16 * CPL, NT = 64 * NW;
    __shared__ Routed r;
    __shared__ float s_w[kFewTokens * kFewTopK];
    __shared__ f32x4 red[NW][CPL][TF][64];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int panel = blockIdx.x / a.splits, s = blockIdx.x - panel * a.splits;

    if (tid < kMaxE) r.tok[tid] = 0;
    lds_barrier();
    for (int q = tid; q < a.T * a.top_k; q += NT) {
        const int e = a.ids[q], t = q / a.top_k;
        s_w[q] = a.w[q];
        if (e >= 0 && e < a.E) {
            r.slot[t][e] = static_cast<uint8_t>(q - t * a.top_k);
            atomicOr(&r.tok[e], 1u << t);
        }
    }
    lds_barrier();
    list_active<NW>(r, a.E);
    const int n_act = __builtin_amdgcn_readfirstlane(r.n_act);

    const Matrix m{&a.down, a.H, a.I, a.group};
    const int grans = S::granules(m);
    const int total = n_act * grans, waves = a.splits * NW;
    const int who = s * NW + wave;
    const int q0 = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<int64_t>(total) * who / waves));
    const int q1 = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<int64_t>(total) * (who + 1) / waves));
    const int n0 = panel * NCOL;
    typename S::X x;
    x.lo = a.T * a.top_k * a.I * 2;
    x.buf = buffer(a.hs, 2 * static_cast<int64_t>(x.lo));
    f32x4 sum[CPL][TF];
#pragma unroll
    for (int j = 0; j < CPL; ++j)
#pragma unroll
        for (int f = 0; f < TF; ++f) sum[j][f] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto open_at = [&](int i, Seg& g, int (&arow)[TF]) __attribute__((always_inline)) {
        const int e = __builtin_amdgcn_readfirstlane(r.act[i]);
        S::open(m, e, n0, g);
        const uint32_t mask = r.tok[e];
#pragma unroll
        for (int f = 0; f < TF; ++f) {
            const int t = 16 * f + (lane & 15);
            arow[f] = (mask >> t) & 1u ? (t * a.top_k + r.slot[t][e]) * a.I * 2 : kPast;
        }
    };
    auto flush = [&](int i, f32x4 (&out)[CPL][TF]) __attribute__((always_inline)) {
        const int e = __builtin_amdgcn_readfirstlane(r.act[i]);
        S::close(m, e, n0, out);
        const uint32_t mask = r.tok[e];
#pragma unroll
        for (int f = 0; f < TF; ++f)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int t = 16 * f + 4 * (lane >> 4) + v;
                if (!((mask >> t) & 1u)) continue;  // not the expert's: its row is no result
                const float w = s_w[t * a.top_k + r.slot[t][e]];
#pragma unroll
                for (int j = 0; j < CPL; ++j) sum[j][f][v] = fmaf(w, out[j][f][v], sum[j][f][v]);
            }
    };
    walk<S, TF>(m, x, q1 - q0, q0 / grans, q0 % grans, 0, grans, 1, open_at, flush);
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
    if (a.splits > 1) {
        // Partial panels [panel][s][cell][j] meet in the workspace, written and read device-coherently
        // (sc1, what agent-scope atomic accesses use: no cache has to be written back or invalidated);
        // a workgroup's are complete (vmcnt 0) before it counts itself.  The last to arrive reads
        // kBatch of them at a time (a read takes about a microsecond) and adds them in the order of s.
        constexpr int kSc1 = 16, kBatch = 8, CB = CPL * 4;  // bytes per cell
        const __amdgpu_buffer_rsrc_t part = buffer(a.part + static_cast<int64_t>(panel) * a.splits * (CPL * CELLS),
                                                   static_cast<int64_t>(a.splits) * CELLS * CB);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int c = tid + q * NT;
            if (c >= CELLS) break;
            const int off = (s * CELLS + c) * CB;
            if constexpr (CPL == 4)
                __builtin_amdgcn_raw_buffer_store_b128(f32x4{res[q][0], res[q][1], res[q][2], res[q][3]}, part, off, 0, kSc1);
            else
                __builtin_amdgcn_raw_buffer_store_b64(f32x2{res[q][0], res[q][1]}, part, off, 0, kSc1);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0)
            s_last = __hip_atomic_fetch_add(&a.cnt[panel], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.splits - 1;
        __syncthreads();
        if (!s_last) return;
        if (tid == 0) __hip_atomic_store(&a.cnt[panel], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int q = 0; q < PER; ++q) {
            const int c = tid + q * NT;
            if (c >= CELLS) break;
#pragma unroll
            for (int j = 0; j < CPL; ++j) res[q][j] = 0.f;
            for (int o = 0; o < a.splits; o += kBatch) {
                std::conditional_t<CPL == 4, f32x4, f32x2> v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    const int off = o + i < a.splits ? ((o + i) * CELLS + c) * CB : kPast;
                    if constexpr (CPL == 4)
                        v[i] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(part, off, 0, kSc1));
                    else
                        v[i] = __builtin_bit_cast(f32x2, __builtin_amdgcn_raw_buffer_load_b64(part, off, 0, kSc1));
                }
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
#pragma unroll
                    for (int j = 0; j < CPL; ++j) res[q][j] += v[i][j];
            }
        }
    }
#pragma unroll
    for (int q = 0; q < PER; ++q) {
        const int c = tid + q * NT;
        if (c >= CELLS) break;
        const int t = 16 * (c >> 8) + 4 * ((c & 63) >> 4) + ((c >> 6) & 3);
        const int col = n0 + CPL * (c & 15);
        if (t >= a.T || col >= a.H) continue;
        uint16_t* dst = a.out + static_cast<int64_t>(t) * a.H + col;
        if constexpr (CPL == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(res[q][0], res[q][1]), pack_bf16x2(res[q][2], res[q][3]));
        else
            *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(res[q][0], res[q][1]);
    }
}

template <int KIND, int STEPS, int TF, int SRC>
hipError_t launch_gate_up(const FewArgs& a, hipStream_t s) {
    constexpr int NCOL = 16 * Stream<KIND, STEPS, TF, SRC>::CPL, NW = 4 * min_waves(KIND, TF, SRC);
    const int most = a.T * a.top_k < a.E ? a.T * a.top_k : a.E;  // active experts at most
    const int64_t items = static_cast<int64_t>(most) * ((a.I + NCOL - 1) / NCOL);
    const int grid = static_cast<int>(items < kFewGrid ? items : kFewGrid);
    few_gate_up_kernel<KIND, STEPS, TF, NW, SRC><<<grid + 1, 64 * NW, 0, s>>>(a);
    return hipGetLastError();
}

// LSTEPS: the int4 granule with x in LDS
template <int KIND, int LSTEPS, int STEPS, int TF>
hipError_t launch_kind(const FewArgs& a, hipStream_t s) {
    using L = Stream<KIND, LSTEPS, TF, kTile>;
    const int64_t kpad = (a.H + L::UK - 1) / L::UK * L::UK;
    int64_t rows = 0;
    for (int f = 0; f < TF; ++f) rows += x_rows(a.T, f);
    const bool lds = rows * kpad * 2 <= x_bytes(L::CPL, 16);
    const hipError_t err = lds ? launch_gate_up<KIND, LSTEPS, TF, kTile>(a, s) : launch_gate_up<KIND, STEPS, TF, kRow>(a, s);
    if (err != hipSuccess) return err;
    constexpr int NCOL = 16 * L::CPL, NW = 4 * min_waves(KIND, TF, kPair);
    few_down_kernel<KIND, STEPS, TF, NW><<<(a.H + NCOL - 1) / NCOL * a.splits, 64 * NW, 0, s>>>(a);
    return hipGetLastError();
}

template <int TF>
hipError_t launch_tf(int kind, const FewArgs& a, hipStream_t s) {
    switch (kind) {
        case kBf16: return launch_kind<kBf16, 1, 1, TF>(a, s);
        case kFp8Row: return launch_kind<kFp8Row, 1, 1, TF>(a, s);
        case kFp8Blk: return launch_kind<kFp8Blk, 1, 1, TF>(a, s);
        default: break;
    }
    if (kind != kInt4) return hipErrorInvalidValue;
    switch (a.group) {
        case 32: return launch_kind<kInt4, 1, 1, TF>(a, s);
        case 64: return launch_kind<kInt4, 2, 2, TF>(a, s);
        case 128:
        case 256: return launch_kind<kInt4, TF == 1 ? 4 : 2, 2, TF>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_few_tokens(int kind, const FewArgs& a, hipStream_t s) {
    return a.T <= 16 ? launch_tf<1>(kind, a, s) : launch_tf<2>(kind, a, s);
}

}  // namespace moe
