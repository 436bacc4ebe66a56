// The whole routed layer for at most 32 tokens in two launches:
//
//   few_gate_up   top-k softmax routing, then h[p] = SiLU(x Wg^T) * (x Wu^T) of every (token,
//                 slot) pair p = t * top_k + j
//   few_down      out[t] = bf16(sum_j w[t, j] * (h[p] Wd^T)), fp32 sums over k and over the experts
//
// What bounds it: reading the active experts' weights once.  A few tokens leave the matrix units idle
// (16 tokens use 1/20 of their rate at the streaming rate of HBM), so each weight value goes from memory
// to one MFMA through registers, with no LDS in between, and the tokens are the other operand: a
// 16x16x32 bf16 MFMA takes 16 tokens x 16 output columns.  The operand's rows are the tokens that chose the
// expert, packed: an expert of a batch of 32 has few, so that its weights meet one MFMA each, and one with
// more than 16 is walked once more for the rest (its weights come from the caches then).  With rows by token
// instead, two operands from 17 tokens on, 32 tokens of 8 of 64 experts of 1408 x 2048 took 289 us in bf16
// (233 packed), 203 in fp8 (136) and 111 in int4 (79).  There is no sorted layout: the list of those groups
// of at most 16 tokens, with the rows' tokens and slots, is the whole routing and the work list.
//
// Routing.  Every workgroup of few_gate_up selects all tokens' experts itself from the logits (at most
// 32 KB, from L2): a launch less, and cheaper than waiting for one workgroup's result.  Workgroup 0
// alone computes the weights (in fp64, route_tokens: ids and weights bit for bit those of moe_route)
// and stores them; few_down reads them back.
//
// Work split.  A workgroup takes one panel of 16 * CPL output columns of one expert; its waves split the
// projections (gate, up) and the contraction, and their partial sums meet in LDS.  In few_down a
// workgroup keeps one column panel; its waves take equal shares of the experts' granules and each adds its
// experts up per token, weighted, in a panel of its own in LDS; the panels are added in the order of the
// waves.  With splits > 1 (fewer panels than the GPU has room for) the workgroups' panels meet in the
// workspace, the last workgroup to arrive adding them in the order of s, so the result does not depend on
// who arrives last.
//
// Roundings: h is kept as the sum of two bf16 values (16 bits of it: the operand type of the second
// product, whose spare MFMA rate makes the second part free, where one bf16 value alone would put as much
// error into out as out's own rounding); the expert outputs are not rounded before the weighted sum; out
// once to bf16.  fp8 weights convert to bf16 exactly, their scales multiply fp32 sums; int4 words enter as
// 128 + q (int4_dequant.h).
//
// Rows past N, k past K and rows past a group's tokens are read through bounds-checked buffer loads with an
// offset past the end: zeros, and no memory traffic.
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
// The work list: groups of at most 16 tokens of one expert, the experts ascending, an expert's tokens
// ascending.  An expert has two groups where more than 16 of the 32 tokens chose it, which takes 17 of
// the 32 * 32 pairs: at most 60 experts.
constexpr int kGroups = kMaxE + 64;
constexpr uint16_t kNoToken = 0x8000;  // a row past its group; its token bits name token 0
constexpr uint16_t kNoExpert = 0xffff;

struct Routed {
    uint32_t tok[kMaxE];                  // tokens routed to the expert, one bit each
    uint16_t of[kFewTokens][kFewTopK];    // the expert of a token's slot
    uint16_t base[kMaxE];                 // the expert's first group
    uint16_t act[kGroups];                // expert + 256 * tokens of the group
    uint16_t pair[kGroups][16];           // row of the group: token + 32 * slot, or kNoToken
    int scan[16];
    int n_act;
};

struct Group {
    int e, rows;
    __device__ __forceinline__ Group(const Routed& r, int i) {
        const int a = __builtin_amdgcn_readfirstlane(static_cast<int>(r.act[i]));
        e = a % kMaxE;
        rows = a / kMaxE;
    }
};

template <int NT>
__device__ __forceinline__ void clear_routing(Routed& r, int pairs) {
    const int tid = threadIdx.x;
    if (tid < kMaxE) r.tok[tid] = 0;
    for (int c = tid; c < min(pairs, kGroups) * 8; c += NT) reinterpret_cast<uint32_t*>(&r.pair)[c] = kNoToken * 0x10001u;
}

// the work list from tok and of; every thread of the workgroup, at least kMaxE threads
template <int NW>
__device__ __forceinline__ void list_active(Routed& r, int T, int E, int top_k) {
    const int tid = threadIdx.x;
    const int n = tid < E ? __popc(r.tok[tid]) : 0, f = (n + 15) / 16;
    const int incl = block_inclusive_scan<NW>(f, r.scan, (E + 63) / 64);
    if (f > 0) {
        r.base[tid] = static_cast<uint16_t>(incl - f);
        r.act[incl - f] = static_cast<uint16_t>(tid + kMaxE * min(n, 16));
        if (f > 1) r.act[incl - 1] = static_cast<uint16_t>(tid + kMaxE * (n - 16));
    }
    if (tid == E - 1) r.n_act = incl;
    __syncthreads();
    for (int q = tid; q < T * kFewTopK; q += 64 * NW) {
        const int t = q / kFewTopK, j = q % kFewTopK, e = r.of[t][j];
        if (j >= top_k || e >= E) continue;
        const int rank = __popc(r.tok[e] & ((1u << t) - 1));
        r.pair[r.base[e] + rank / 16][rank % 16] = static_cast<uint16_t>(t + 32 * j);
    }
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
            if (lane == 0 && t < T) {
                r.of[t][j] = e < E ? static_cast<uint16_t>(e) : kNoExpert;
                if (e < E) atomicOr(&r.tok[e], 1u << t);
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
//   out[j][v] += sum_k A(row, k) * W(column, k), rows 4 (lane / 16) + v of the segment's group of tokens
// The next granule's loads (weights and token rows, of the next segment too) are issued before one is
// multiplied: two register sets take turns.  In eight of the seventeen kernels (few_gate_up: fp8 of both
// kinds with x in LDS, int4 in groups of 64 and more with x in memory; few_down: bf16, int4 and block fp8) the
// compiler waits with vmcnt(0) at the loop's head, where an edge of the control flow leaves the idle set
// loading: there every second granule is multiplied with its successor's loads issued only after its own
// have landed.
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

struct TokenRows {
    __amdgpu_buffer_rsrc_t buf;
    int lo;  // kPair: byte offset of the low parts
};

struct TokenTile {
    const uint16_t* base;
    int step;  // elements from one fragment (32 k) to the next
};

// [E, N, K] weights, K contiguous: a load takes 16 bytes of 4 consecutive k chunks of 16 rows.  A granule
// is US loads per column set.
template <int KIND, int CPL_, int US, int SRC>
struct Rows {
    static constexpr int CPL = CPL_;
    static constexpr int ES = KIND == kBf16 ? 2 : 1;
    static constexpr int FR = KIND == kBf16 ? 1 : 2;  // MFMA k-steps (32 k) per load
    static constexpr int KS = 32 * FR;                // k per load
    static constexpr int UK = KS * US;
    static constexpr int NB = UK > 128 ? UK / 128 : 1;  // block scales of a granule
    static_assert(KIND != kFp8Blk || 128 % UK == 0 || UK % 128 == 0, "granules and blocks of k nest");
    using X = std::conditional_t<SRC == kTile, TokenTile, TokenRows>;
    static constexpr int NP = SRC == kPair ? 2 : 1;  // bf16 parts of a token operand
    static constexpr bool kLds = SRC == kTile;
    struct Set {
        u32x4 b[US][CPL], x[SRC == kTile ? 1 : US][FR][NP];
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
                                                int row, int i, bool some) {
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
            for (int c = 0; c < FR; ++c)
#pragma unroll
                for (int h = 0; h < NP; ++h)
                    r.x[u][c][h] = load16(x.buf, in && row != kPast ? row + (k + kq * (8 * FR) + c * 8) * 2 + h * x.lo : kPast);
        }
        if constexpr (KIND == kFp8Blk)
#pragma unroll
            for (int b = 0; b < NB; ++b) r.sc[b] = some ? g.bscale[min(i * UK / 128 + b, (m.K + 127) / 128 - 1)] : 0.f;
    }
    __device__ static __forceinline__ void multiply(const Set& r, const X& x, int row, int i, f32x4 (&out)[CPL]) {
        bf16x8 xf[US][FR][NP];
#pragma unroll
        for (int u = 0; u < US; ++u)
#pragma unroll
            for (int c = 0; c < FR; ++c) {
                if constexpr (SRC == kTile)
                    xf[u][c][0] = *reinterpret_cast<const bf16x8*>(x.base + row + ((i * US + u) * FR + c) * x.step);
                else
#pragma unroll
                    for (int h = 0; h < NP; ++h) xf[u][c][h] = as_bf16x8(r.x[u][c][h]);
            }
        constexpr int UB = KIND == kFp8Blk ? US / NB : US;  // loads under one scale
#pragma unroll
        for (int j = 0; j < CPL; ++j)
#pragma unroll
            for (int b = 0; b < US / UB; ++b) {
                f32x4 d = KIND == kFp8Blk ? f32x4{0.f, 0.f, 0.f, 0.f} : out[j];
#pragma unroll
                for (int u = b * UB; u < (b + 1) * UB; ++u)
#pragma unroll
                    for (int c = 0; c < FR; ++c) {
                        const bf16x8 w = KIND == kBf16 ? as_bf16x8(r.b[u][j]) : fp8_to_bf16(r.b[u][j][2 * c], r.b[u][j][2 * c + 1]);
#pragma unroll
                        for (int h = 0; h < NP; ++h) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[u][c][h], w, d, 0, 0, 0);
                    }
#pragma unroll
                for (int v = 0; v < 4; ++v) out[j][v] = KIND == kFp8Blk ? fmaf(r.sc[b], d[v], out[j][v]) : d[v];
            }
    }
    // channel scales, once per segment
    __device__ static __forceinline__ void close(const Matrix& m, int e, int n0, f32x4 (&out)[CPL]) {
        if constexpr (KIND == kFp8Row) {
            const float* sc = static_cast<const float*>(m.w->scales) + static_cast<int64_t>(e) * m.N;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                out[j] *= sc[min(n0 + CPL * static_cast<int>(threadIdx.x & 15) + j, m.N - 1)];
            }
        }
    }
};

// GPTQ words [E, K/8, N]: a lane reads 4 consecutive columns of a k-octet, one column per MFMA.  A granule
// of 32 * STEPS k lies in one quantisation group and contributes s * (acc - (128 + z) * sum_k x), the sum from one more MFMA against ones.
template <int STEPS, int SRC>
struct Words {
    static constexpr int CPL = 4;
    static constexpr int UK = STEPS * 32;
    using X = std::conditional_t<SRC == kTile, TokenTile, TokenRows>;
    static constexpr int NP = SRC == kPair ? 2 : 1;  // bf16 parts of a token operand
    static constexpr bool kLds = SRC == kTile;
    struct Set {
        u32x4 q[STEPS], x[SRC == kTile ? 1 : STEPS][NP];
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
                                                int row, int i, bool some) {
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
            for (int h = 0; h < NP; ++h)
                r.x[st][h] = load16(x.buf, some && row != kPast ? row + (i * UK + st * 32 + kq * 8) * 2 + h * x.lo : kPast);
    }
    __device__ static __forceinline__ void multiply(const Set& r, const X& x, int row, int i, f32x4 (&out)[4]) {
        const u32x4 ones = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
        const int zshift = 16 * (threadIdx.x & 1);
        uint32_t nib_mask, bf16_128;
        asm("v_mov_b32 %0, 0x000f000f" : "=v"(nib_mask));
        asm("v_mov_b32 %0, 0x43004300" : "=v"(bf16_128));
        const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
        f32x4 acc[4] = {zero, zero, zero, zero}, accx = zero;
#pragma unroll
        for (int st = 0; st < STEPS; ++st) {
            bf16x8 xf[NP];
#pragma unroll
            for (int h = 0; h < NP; ++h) {
                if constexpr (SRC == kTile) xf[h] = *reinterpret_cast<const bf16x8*>(x.base + row + (i * STEPS + st) * x.step);
                else xf[h] = as_bf16x8(permute_k(r.x[st][h]));
                accx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[h], as_bf16x8(ones), accx, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 w = as_bf16x8(dequant_word(r.q[st][j], nib_mask, bf16_128));
#pragma unroll
                for (int h = 0; h < NP; ++h) acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xf[h], w, acc[j], 0, 0, 0);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t sbits = (j < 2 ? r.s.x : r.s.y) >> (16 * (j & 1));
            const float sc = f16_to_f32(static_cast<uint16_t>(sbits & 0xffffu));
            const float zz = 128.0f + static_cast<float>((r.z >> (zshift + 4 * j)) & 0xfu);
#pragma unroll
            for (int v = 0; v < 4; ++v) out[j][v] = fmaf(sc, fmaf(-zz, accx[v], acc[j][v]), out[j][v]);
        }
    }
    __device__ static __forceinline__ void close(const Matrix&, int, int, f32x4 (&)[4]) {}
};

// The weight types' streams.  The granule is what two register sets, the sums and the addresses leave room
// for, given the waves that are to share a compute unit: sixteen (128 registers) with x in LDS or in memory,
// twelve with pairs, or eight with the larger granule that int4 groups of 128 allow (16 tokens of 8 of 64
// experts of 1408 x 2048: 23.7 us for few_down against 25.1 with granules of 64 k and twelve waves).  2 to
// 8 KB of weights a wave are in flight.
template <int KIND, int STEPS, int SRC>
using Stream = std::conditional_t<KIND == kInt4, Words<STEPS, SRC>,
                                  Rows<KIND, 2, KIND != kBf16 ? 2 : SRC == kTile ? 4 : 3, SRC>>;
constexpr int min_waves(int steps, int src) { return src != kPair ? 4 : steps == 4 ? 2 : 3; }

// The wave's granules: `n` of them from granule g of segment `seg`, the segments' granules being [gb, ge) and
// their numbers `stride` apart.  open_at(seg, Seg&) opens a segment, rows_at(seg) is this lane's token row in
// it (an offset into x's source, which kTile reads as it multiplies and the others as they load); flush(seg,
// out) takes its sums
// (before the next granule is multiplied, with the loads after it in flight).
template <class S, class Open, class RowsAt, class Flush>
__device__ __forceinline__ void walk(const Matrix& m, const typename S::X& x, int n, int seg, int g, int gb, int ge,
                                     int stride, Open open_at, RowsAt rows_at, Flush flush) {
    typename S::Set ra, rb;
    Seg cur;
    int row;
    f32x4 out[S::CPL];
    auto zero = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < S::CPL; ++j) out[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    int lseg = seg, lg = g;  // the granule that the last loads took
    auto fetch = [&](typename S::Set& r, bool some) __attribute__((always_inline)) {
        if (some && ++lg == ge) {
            lg = gb;
            lseg += stride;
            open_at(lseg, cur);
            if constexpr (!S::kLds) row = rows_at(lseg);
        }
        S::load(r, m, cur, x, row, lg, some);
        __builtin_amdgcn_sched_barrier(0);
    };
    int left = n;
    auto take = [&](const typename S::Set& r) __attribute__((always_inline)) {
        S::multiply(r, x, row, g, out);
        __builtin_amdgcn_sched_barrier(0);
        --left;
        if (++g == ge || left == 0) {
            flush(seg, out);
            zero();
            g = gb;
            seg += stride;
            if constexpr (S::kLds)
                if (left) row = rows_at(seg);
        }
    };
    zero();
    if (n <= 0) return;
    open_at(lseg, cur);
    row = rows_at(lseg);
    S::load(ra, m, cur, x, row, lg, true);
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

// x in LDS as MFMA operands: fragment by fragment (32 k), quarter wave by quarter wave (8 k), row by row.
// Chunks past K are zeros (the weights' zeros there must not meet stale bits).
template <class S, int NT>
__device__ __forceinline__ void stage_x(const FewArgs& a, uint16_t* lds, int kpad, typename S::X& x) {
    const __amdgpu_buffer_rsrc_t buf = buffer(a.x, static_cast<int64_t>(a.T) * a.H * 2);
    const int chunks = kpad / 8;
    x.base = lds;
    x.step = a.T * 32;
    // four chunks a thread in flight
    for (int c0 = threadIdx.x; c0 < a.T * chunks; c0 += 4 * NT) {
        u32x4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int c = c0 + u * NT, t = c / chunks, k = (c - t * chunks) * 8;
            v[u] = load16(buf, c < a.T * chunks && k < a.H ? (t * a.H + k) * 2 : kPast);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int c = c0 + u * NT, t = c / chunks;
            if (c >= a.T * chunks) break;
            int frag, kq;
            S::place(c - t * chunks, frag, kq);
            *reinterpret_cast<u32x4*>(lds + ((frag * 4 + kq) * a.T + t) * 8) = S::prepare(v[u]);
        }
    }
}

template <int KIND, int STEPS, int NW, int SRC>
__global__ __launch_bounds__(64 * NW, min_waves(STEPS, SRC)) void few_gate_up_kernel(FewArgs a) {
    using S = Stream<KIND, STEPS, SRC>;
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
    clear_routing<NT>(r, a.T * a.top_k);
    if constexpr (SRC == kTile) stage_x<S, NT>(a, xl, grans * S::UK, x);
    else x.buf = buffer(a.x, static_cast<int64_t>(a.T) * a.H * 2);
    lds_barrier();
    select_all<NW>(a, r, wave, lane);
    lds_barrier();
    list_active<NW>(r, a.T, a.E, a.top_k);

    const int panels = (a.I + NCOL - 1) / NCOL;
    const int items = __builtin_amdgcn_readfirstlane(r.n_act) * panels;
    const int stride = gridDim.x - 1, first = blockIdx.x - 1;
    const int mine = first < items ? (items - first + stride - 1) / stride : 0;
    const int gb = __builtin_amdgcn_readfirstlane(part * grans / PARTS);
    const int ge = __builtin_amdgcn_readfirstlane((part + 1) * grans / PARTS);
    auto open_at = [&](int it, Seg& g) __attribute__((always_inline)) {
        const int i = it / panels;
        S::open(m, Group(r, i).e, (it - i * panels) * NCOL, g);
    };
    // rows past the group: token 0's (LDS), or none (their results are not stored)
    auto rows_at = [&](int it) __attribute__((always_inline)) {
        const int p = r.pair[it / panels][lane & 15], t = p % kFewTokens;
        if constexpr (SRC == kTile) return ((lane >> 4) * a.T + t) * 8;
        else return p != kNoToken ? t * a.H * 2 : kPast;
    };
    // the item's sums over the waves; every wave flushes every item
    auto flush = [&](int it, f32x4 (&out)[CPL]) __attribute__((always_inline)) {
        const int i = it / panels;
        const Group q(r, i);
        const int n0 = (it - i * panels) * NCOL;
        S::close(m, q.e, n0, out);
        lds_barrier();  // the sums before these have been read
#pragma unroll
        for (int j = 0; j < CPL; ++j) red[wave][j][lane] = out[j];
        lds_barrier();
        // one (lane, v) of the panel per thread: row 4 (sl / 16) + v, columns CPL * (sl % 16) ..
        const int v = (tid >> 6) & 3, sl = tid & 63;
        const int row = 4 * (sl >> 4) + v, col = n0 + CPL * (sl & 15);
        if (tid < 256 && row < q.rows && col < a.I) {
            const int p = r.pair[i][row];
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
            uint16_t* dst = a.hs + static_cast<int64_t>(p % kFewTokens * a.top_k + p / kFewTokens) * a.I + col;
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
        walk<S>(m, x, mine * (ge - gb), first, gb, gb, ge, stride, open_at, rows_at, flush);
    } else {  // fewer granules than waves: this one only adds zeros
        f32x4 out[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) out[j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < mine; ++i) flush(first + i * stride, out);
    }
}

// ------------------------------------------------------------------ launch 2: down, weighted sum
// The granules of a column panel, expert by expert of the work list, are one sequence; the waves of the
// panel's workgroups take equal consecutive shares of it, whatever the number of active experts.
template <int KIND, int STEPS, int NW>
__global__ __launch_bounds__(64 * NW, min_waves(STEPS, kPair)) void few_down_kernel(FewArgs a) {
    using S = Stream<KIND, STEPS, kPair>;
    constexpr int CPL = S::CPL, NCOL = 16 * CPL, NT = 64 * NW;
    using Cell = std::conditional_t<CPL == 4, f32x4, f32x2>;  // CPL columns of a token
    static_assert(NT >= kFewTokens * 16, "a thread per cell");
    __shared__ Routed r;
    __shared__ float s_w[kFewTokens * kFewTopK];
    __shared__ Cell sum[NW][kFewTokens][16];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int panel = blockIdx.x / a.splits, s = blockIdx.x - panel * a.splits;

    clear_routing<NT>(r, a.T * a.top_k);
    lds_barrier();
    for (int q = tid; q < a.T * a.top_k; q += NT) {
        const int e = a.ids[q], t = q / a.top_k;
        s_w[q] = a.w[q];
        const bool known = e >= 0 && e < a.E;
        r.of[t][q - t * a.top_k] = known ? static_cast<uint16_t>(e) : kNoExpert;
        if (known) atomicOr(&r.tok[e], 1u << t);
    }
    lds_barrier();
    list_active<NW>(r, a.T, a.E, a.top_k);
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
    for (int c = lane; c < a.T * 16; c += 64) sum[wave][c >> 4][c & 15] = Cell{};  // this wave's own
    auto open_at = [&](int i, Seg& g) __attribute__((always_inline)) { S::open(m, Group(r, i).e, n0, g); };
    auto rows_at = [&](int i) __attribute__((always_inline)) {
        const int p = r.pair[i][lane & 15];
        return p != kNoToken ? (p % kFewTokens * a.top_k + p / kFewTokens) * a.I * 2 : kPast;
    };
    auto flush = [&](int i, f32x4 (&out)[CPL]) __attribute__((always_inline)) {
        const Group q(r, i);
        S::close(m, q.e, n0, out);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int row = 4 * (lane >> 4) + v;
            if (row >= q.rows) continue;
            const int p = r.pair[i][row], t = p % kFewTokens;
            const float w = s_w[t * a.top_k + p / kFewTokens];
            Cell c = sum[wave][t][lane & 15];
#pragma unroll
            for (int j = 0; j < CPL; ++j) c[j] = fmaf(w, out[j][v], c[j]);
            sum[wave][t][lane & 15] = c;
        }
    };
    walk<S>(m, x, q1 - q0, q0 / grans, q0 % grans, 0, grans, 1, open_at, rows_at, flush);
    __syncthreads();
    const int cells = a.T * 16;  // one per thread: token tid / 16, columns n0 + CPL * (tid % 16) ..
    Cell res = {};
    if (tid < cells) {
#pragma unroll
        for (int w = 0; w < NW; ++w) res += sum[w][tid >> 4][tid & 15];
    }
    if (a.splits > 1) {
        // Partial panels [panel][s][cell] meet in the workspace, written and read device-coherently
        // (sc1, what agent-scope atomic accesses use: no cache has to be written back or invalidated);
        // a workgroup's are complete (vmcnt 0) before it counts itself.  The last to arrive reads
        // kBatch of them at a time (a read takes about a microsecond) and adds them in the order of s.
        constexpr int kSc1 = 16, kBatch = 8, CB = CPL * 4;  // bytes per cell
        const __amdgpu_buffer_rsrc_t part = buffer(a.part + static_cast<int64_t>(panel) * a.splits * cells * CPL,
                                                   static_cast<int64_t>(a.splits) * cells * CB);
        const int off = tid < cells ? (s * cells + tid) * CB : kPast;  // (a store past the end is dropped)
        if constexpr (CPL == 4) __builtin_amdgcn_raw_buffer_store_b128(res, part, off, 0, kSc1);
        else __builtin_amdgcn_raw_buffer_store_b64(res, part, off, 0, kSc1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (tid == 0)
            s_last = __hip_atomic_fetch_add(&a.cnt[panel], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == a.splits - 1;
        __syncthreads();
        if (!s_last) return;
        if (tid == 0) __hip_atomic_store(&a.cnt[panel], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        res = Cell{};
        for (int o = 0; o < a.splits; o += kBatch) {
            Cell v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = tid < cells && o + i < a.splits ? ((o + i) * cells + tid) * CB : kPast;
                if constexpr (CPL == 4) v[i] = __builtin_bit_cast(Cell, __builtin_amdgcn_raw_buffer_load_b128(part, at, 0, kSc1));
                else v[i] = __builtin_bit_cast(Cell, __builtin_amdgcn_raw_buffer_load_b64(part, at, 0, kSc1));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) res += v[i];
        }
    }
    const int col = n0 + CPL * (tid & 15);
    if (tid >= cells || col >= a.H) return;
    uint16_t* dst = a.out + static_cast<int64_t>(tid >> 4) * a.H + col;
    if constexpr (CPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(res[0], res[1]), pack_bf16x2(res[2], res[3]));
    else *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(res[0], res[1]);
}

template <int KIND, int STEPS, int SRC>
hipError_t launch_gate_up(const FewArgs& a, hipStream_t s) {
    constexpr int NCOL = 16 * Stream<KIND, STEPS, SRC>::CPL, NW = 4 * min_waves(STEPS, SRC);
    const int most = a.T * a.top_k < a.E ? a.T * a.top_k : a.E;  // active experts at most
    const int64_t items = static_cast<int64_t>(most) * ((a.I + NCOL - 1) / NCOL);
    const int grid = static_cast<int>(items < kFewGrid ? items : kFewGrid);
    few_gate_up_kernel<KIND, STEPS, NW, SRC><<<grid + 1, 64 * NW, 0, s>>>(a);
    return hipGetLastError();
}

// ROW_STEPS: the int4 granule where the registers have to hold x of sixteen waves
template <int KIND, int STEPS, int ROW_STEPS>
hipError_t launch_kind(const FewArgs& a, hipStream_t s) {
    using L = Stream<KIND, STEPS, kTile>;
    const int64_t kpad = (a.H + L::UK - 1) / L::UK * L::UK;
    const bool lds = a.T * kpad * 2 <= x_bytes(L::CPL, 16);
    const hipError_t err = lds ? launch_gate_up<KIND, STEPS, kTile>(a, s) : launch_gate_up<KIND, ROW_STEPS, kRow>(a, s);
    if (err != hipSuccess) return err;
    constexpr int NCOL = 16 * L::CPL, NW = 4 * min_waves(STEPS, kPair);
    few_down_kernel<KIND, STEPS, NW><<<(a.H + NCOL - 1) / NCOL * a.splits, 64 * NW, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few_tokens(int kind, const FewArgs& a, hipStream_t s) {
    switch (kind) {
        case kBf16: return launch_kind<kBf16, 1, 1>(a, s);
        case kFp8Row: return launch_kind<kFp8Row, 1, 1>(a, s);
        case kFp8Blk: return launch_kind<kFp8Blk, 1, 1>(a, s);
        default: break;
    }
    if (kind != kInt4) return hipErrorInvalidValue;
    switch (a.group) {
        case 32: return launch_kind<kInt4, 1, 1>(a, s);
        case 64: return launch_kind<kInt4, 2, 2>(a, s);
        case 128:
        case 256: return launch_kind<kInt4, 4, 2>(a, s);
        default: return hipErrorInvalidValue;
    }
}

}  // namespace moe
