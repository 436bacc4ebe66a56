// Grouped products for the gradients of the expert path, one launch for all experts.
//
//   dgrad   dx[r, k]   = sum over n of dy(r, n) W_e[n, k]  (+ a second pair)   rows r of expert e
//   wgrad   dw_e[n, k] = sum over rows r of e of dy(r, n) x(r, k)  (+ base)
//
// The forward products contract over the dimension in which both operands are contiguous.  Here the
// contraction runs across the memory rows of W (dgrad) and of both operands (wgrad): such an operand
// comes into LDS row by row as it lies in memory, 64 contraction rows of 256 columns a stage, and the
// MFMA fragments, which want eight consecutive contraction indices per lane, are read with the
// transposing LDS read (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 columns, lane i gets column i
// of the 4 rows).  No operand is transposed in memory.
//
// Tile: 256 output rows x 256 output columns on 8 waves (4 x 2, each 64 x 128 of 32x32x16 MFMA blocks),
// contraction 64 at a time through two LDS stages filled by direct global -> LDS loads.  The column
// operand is the MFMA's first one, so that a lane's 16 results of a block lie in one output row:
// two half-wave swaps give it 8 adjacent columns, 16 bytes of bf16.
//
// LDS layout.  Column-major-read operands: row of 512 bytes, 16-byte chunk c of contraction row q at
// chunk c ^ ((q & 3) << 2 | (q >> 3 & 1) << 1): the 4 rows (and the 2 x 16 columns, or the 2 x 8 rows)
// that one transposing read touches together lie in different banks.  dy of dgrad: rows of 128 bytes,
// chunk c of row q at c ^ (q / 2 & 7), as in the forward kernel.
//
// Rows without a pair (sentinels inside an expert's padded span) load a valid row and are not stored
// (dgrad), or load zeros from both operands (wgrad: they would enter every sum, and may hold anything).
#include <type_traits>

#include "device_common.h"
#include "launchers.h"

namespace moe {
namespace {

constexpr int kTile = 256;     // output rows and columns of a tile
constexpr int kBK = 64;        // contraction per stage
constexpr int kNT = 512;
constexpr int kPart = kTile * kBK;      // elements of one operand's stage
constexpr int kStage = 2 * kPart;
constexpr int kMaxE = 256;
constexpr int kBand = 8;       // row tiles per band of the tile order

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// division by a launch constant d >= 1 of numbers below 2^31 (round-up reciprocal: exact there)
struct FastDiv {
    uint32_t m;
    int sh;   // < 0: d == 1
};
__device__ __forceinline__ int fast_div(int x, FastDiv d) {
    return d.sh < 0 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), d.m) >> d.sh);
}

struct GradArgs {
    const uint16_t* r0;   // operand of the output rows: dy
    const uint16_t* r1;   // dgrad: the second pair's (NULL: none)
    const uint16_t* c0;   // operand of the output columns: W, or x
    const uint16_t* c1;
    void* out;
    const void* base;     // wgrad, or NULL
    const int32_t* sorted_ids;
    const int32_t* offsets;
    FastDiv top_k;
    int P, E, N, K, max_pad;
    int r_tok, c_tok;     // operand rows by token
};

// DGRAD: bf16 out; else wgrad with bf16 (F32 false) or fp32 results
template <bool DGRAD, bool F32>
__global__ __launch_bounds__(kNT, 1) void grad_gemm_kernel(GradArgs g) {
    __shared__ __attribute__((aligned(1024))) uint16_t smem[2 * kStage];
    __shared__ int s_lo[kMaxE], s_hi[kMaxE], s_tb[kMaxE + 1], s_order[kMaxE];
    __shared__ int s_scan[kNT / 64];
    __shared__ __attribute__((aligned(16))) int s_id[2][kTile];    // dgrad: sorted ids of the tile's rows; wgrad: of its first two stages
    __shared__ __attribute__((aligned(16))) int s_ring[2][kBK];    // wgrad: sorted ids of stages 2, 3, ...

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int N = g.N, K = g.K, E = g.E;

    // ---- expert spans; dgrad: row tiles before each expert; wgrad: experts by falling span
    {
        int lo = 0, hi = 0;
        if (tid < E && g.P > 0) {
            lo = min(max(g.offsets[tid], 0), g.max_pad);
            hi = min(max(g.offsets[tid + 1], lo), g.max_pad);
        }
        if (tid < E) { s_lo[tid] = lo; s_hi[tid] = hi; }
        if constexpr (DGRAD) {
            const int incl = block_inclusive_scan<kNT / 64>((hi - lo + kTile - 1) / kTile, s_scan, (E + 63) / 64);
            if (tid < E) s_tb[tid + 1] = incl;
            if (tid == 0) s_tb[0] = 0;
        }
        __syncthreads();
        if constexpr (!DGRAD) {
            if (tid < E) {
                int rank = 0;
                for (int i = 0; i < E; ++i) {
                    const int n = s_hi[i] - s_lo[i];
                    rank += n > hi - lo || (n == hi - lo && i < tid);
                }
                s_order[rank] = tid;
            }
            __syncthreads();
        }
    }
    const int n_tiles = (K + kTile - 1) / kTile;     // column tiles
    const int r_tiles = (N + kTile - 1) / kTile;     // wgrad: row tiles of an expert's matrix
    const int per_xcd = gridDim.x >> 3;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;

    // ---- this XCD's list of tiles, entries i = slot, slot + per_xcd, ...
    // dgrad: an eighth of the tiles.  wgrad: units of up to 32 tiles of one expert, dealt to the XCDs in turn by
    // falling length.
    const int m_real = DGRAD ? __builtin_amdgcn_readfirstlane(s_tb[E]) : 0;
    const long long T = DGRAD ? static_cast<long long>(m_real) * n_tiles : 0;
    const int l_lo = DGRAD ? static_cast<int>(T * xcd / 8) : 0;
    const int tiles_e = r_tiles * n_tiles;
    int unit = 1, units_e = 1;
    if constexpr (!DGRAD) {
        const int most = static_cast<int>(min<long long>(32, max<long long>(1, static_cast<long long>(E) * tiles_e / 64)));
        units_e = (tiles_e + most - 1) / most;
        unit = (tiles_e + units_e - 1) / units_e;
    }
    const int units = E * units_e;
    const int l_n = DGRAD ? static_cast<int>(T * (xcd + 1) / 8) - l_lo : (units + 7) / 8 * unit;

    struct Seg {
        int e, r0, r_end;   // dgrad: expert, first sorted row, end of rows; wgrad: expert, its span
        int row0, col0;     // first output row (wgrad: of N) and column
        int nst;            // stages
    };
    const int nk = (N + kBK - 1) / kBK;              // dgrad: stages of one pair
    // the next entry at or after i that is a tile; false: none
    auto locate = [&](int& i, Seg& s) __attribute__((always_inline)) -> bool {
        for (;; i += per_xcd) {
            if (i >= l_n) return false;
            int idx, m_lim, m_t, n_t;
            if constexpr (DGRAD) {
                idx = l_lo + i;
                m_lim = m_real;
            } else {
                const int v = i / unit;
                const int u = v * 8 + ((v & 1) ? 7 - xcd : xcd);
                if (u >= units) continue;
                idx = (u % units_e) * unit + i % unit;
                if (idx >= tiles_e) continue;
                m_lim = r_tiles;
                s.e = __builtin_amdgcn_readfirstlane(s_order[u / units_e]);
            }
            // bands of kBand row tiles, row tiles fastest: tiles that run together share operands in L2
            const int band = idx / (kBand * n_tiles);
            const int in = idx - band * kBand * n_tiles;
            const int rows = min(kBand, m_lim - band * kBand);
            n_t = in / rows;
            m_t = band * kBand + in - n_t * rows;
            s.col0 = n_t * kTile;
            if constexpr (DGRAD) {
                int a = 0, b = E - 1;  // largest expert whose first row tile is <= m_t
                while (a < b) {
                    const int mid = (a + b + 1) >> 1;
                    if (s_tb[mid] <= m_t) a = mid; else b = mid - 1;
                }
                s.e = __builtin_amdgcn_readfirstlane(a);
                s.r0 = __builtin_amdgcn_readfirstlane(s_lo[s.e] + (m_t - s_tb[s.e]) * kTile);
                s.r_end = __builtin_amdgcn_readfirstlane(min(s.r0 + kTile, s_hi[s.e]));
                s.row0 = 0;
                s.nst = g.r1 ? 2 * nk : nk;
            } else {
                s.row0 = m_t * kTile;
                s.r0 = __builtin_amdgcn_readfirstlane(s_lo[s.e]);
                s.r_end = __builtin_amdgcn_readfirstlane(s_hi[s.e]);
                s.nst = (s.r_end - s.r0 + kBK - 1) / kBK;
            }
            return true;
        }
    };

    int L = slot;
    Seg cur;
    if (!locate(L, cur)) return;

    const uint32_t lds0 = lds_u32(smem);
    // sorted ids of 64 rows from r into LDS (rows past max_pad read the last one; checked where used)
    auto load_ids = [&](int r, const int* dst) __attribute__((always_inline)) {
        dma4(g.sorted_ids + min(r + lane, g.max_pad - 1), lds_u32(dst));
    };
    // those a segment needs before its first stage's loads: by the waves that hold them
    auto first_ids = [&](const Seg& s, int b) __attribute__((always_inline)) {
        constexpr int W = DGRAD ? kTile / 64 : 2;
        if (wave < W) load_ids(s.r0 + wave * 64, s_id[b] + wave * 64);
    };
    // row of an operand for sorted row r with id p; < 0: no pair
    auto source = [&](int p, int r, int r_end, int tok) __attribute__((always_inline)) {
        return r < r_end && p >= 0 && p < g.P ? (tok ? fast_div(p, g.top_k) : r) : -1;
    };

    // ---- loads of stage t of a segment into LDS buffer b: 8 waves x 8 instructions of 1 KB
    auto issue = [&](const Seg& s, int sbuf, int t, int b) __attribute__((always_inline)) {
        const uint32_t dst_r = lds0 + b * (kStage * 2) + wave * 4096, dst_c = dst_r + kPart * 2;
        const int half = lane >> 5;
        const char* zero = reinterpret_cast<const char*>(kZero16);
        if constexpr (DGRAD) {
            const bool second = t >= nk;
            const int k0 = (second ? t - nk : t) * kBK;
            const uint16_t* R = second ? g.r1 : g.r0;
            const uint16_t* C = (second ? g.c1 : g.c0) + static_cast<size_t>(s.e) * N * K;
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // dy: 8 tile rows of 128 bytes
                const int row = wave * 32 + q * 8 + (lane >> 3);
                const int src = source(s_id[sbuf][row], s.r0 + row, s.r_end, g.r_tok);
                const size_t at = src >= 0 ? src : (g.r_tok ? 0 : s.r0);
                const int n = k0 + (((lane & 7) ^ ((row >> 1) & 7)) << 3);
                dma16(n < N ? reinterpret_cast<const char*>(R + at * N + n) : zero, dst_r + q * 1024);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {   // W: 2 contraction rows of 512 bytes
                const int row = wave * 8 + q * 2 + half;
                const int chunk = (lane & 31) ^ (((row & 3) << 2) | (((row >> 3) & 1) << 1));
                const int col = min(s.col0 + chunk * 8, K - 8);  // columns past K are never stored
                const int n = k0 + row;
                dma16(n < N ? reinterpret_cast<const char*>(C + static_cast<size_t>(n) * K + col) : zero, dst_c + q * 1024);
            }
        } else {
            const int* ids = t < 2 ? s_id[sbuf] + t * kBK : s_ring[t & 1];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = wave * 8 + q * 2 + half;
                const int chunk = (lane & 31) ^ (((row & 3) << 2) | (((row >> 3) & 1) << 1));
                const int r = s.r0 + t * kBK + row, p = ids[row];
                const int ry = source(p, r, s.r_end, g.r_tok), rx = source(p, r, s.r_end, g.c_tok);
                const int n = min(s.row0 + chunk * 8, N - 8), k = min(s.col0 + chunk * 8, K - 8);
                dma16(ry >= 0 ? reinterpret_cast<const char*>(g.r0 + static_cast<size_t>(ry) * N + n) : zero, dst_r + q * 1024);
                dma16(rx >= 0 ? reinterpret_cast<const char*>(g.c0 + static_cast<size_t>(rx) * K + k) : zero, dst_c + q * 1024);
            }
        }
    };

    const int wm = wave >> 1, wn = wave & 1;   // the wave's 64 rows and 128 columns
    const int fr = lane & 31, fc = lane >> 5;
    // fragment offsets in bytes within a stage.  Transposed reads: lane i of group gr of 16 lanes reads 8 bytes
    // of contraction row (gr / 2) * 8 + i / 4 (+ 4 in the second read), columns (gr % 2) * 16 + (i % 4) * 4.
    const int i16 = lane & 15, gr = lane >> 4;
    auto tr_off = [&](int block) __attribute__((always_inline)) {   // 32 columns from block * 32
        const int row = (gr >> 1) * 8 + (i16 >> 2);
        const int chunk = ((block ^ (i16 >> 2)) << 2) + ((((gr & 1) ^ (gr >> 1)) << 1) | ((i16 & 3) >> 1));
        return row * 512 + chunk * 16 + (i16 & 1) * 8;
    };
    int c_off[4], r_off[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) c_off[j] = kPart * 2 + tr_off(wn * 4 + j);
#pragma unroll
    for (int i = 0; i < 2; ++i) r_off[i] = DGRAD ? (wm * 64 + i * 32 + fr) * 128 : tr_off(wm * 2 + i);
    const int fswz = (fr >> 1) & 7;

    f32x16 acc[2][4];
    bf16x8 fa[2][2], fb[2][4];
    auto tr_read = [&](const char* p) __attribute__((always_inline)) {
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * 512));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto read = [&](int b, int kk, int set) __attribute__((always_inline)) {
        const char* st = reinterpret_cast<const char*>(smem + b * kStage);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (DGRAD)
                fa[set][i] = *reinterpret_cast<const bf16x8*>(st + r_off[i] + (((kk * 2 + fc) ^ fswz) << 4));
            else
                fa[set][i] = tr_read(st + r_off[i] + kk * (16 * 512));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) fb[set][j] = tr_read(st + c_off[j] + kk * (16 * 512));
    };
    auto mfma = [&](int set) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
    };

    int sbuf = 0;   // LDS id buffer of the current segment
    int b = 0;      // LDS buffer of its stage 0
    first_ids(cur, 0);
    wait_vmcnt<0>();
    __syncthreads();
    if (cur.nst > 0) issue(cur, 0, 0, 0);

    while (true) {
        int L2 = L + per_xcd;
        Seg nxt;
        const bool more = locate(L2, nxt);
        // Stage t becomes readable: every wave waits for its own loads, then the barrier makes the stage
        // visible and frees the other buffer for stage t + 1.
        auto ready = [&](int t) __attribute__((always_inline)) {
            wait_vmcnt<0>();
            __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
            __builtin_amdgcn_s_barrier();
            if (t + 1 < cur.nst) issue(cur, sbuf, t + 1, (b + t + 1) & 1);
            if constexpr (!DGRAD)
                if (t + 2 < cur.nst && wave == 7) load_ids(cur.r0 + (t + 2) * kBK, s_ring[t & 1]);
            if (t == 0 && more && cur.nst >= 2) first_ids(nxt, sbuf ^ 1);
        };
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;
        if (cur.nst > 0) {
            ready(0);
            read(b, 0, 0);
            for (int t = 0; t < cur.nst; ++t) {
                const int bt = (b + t) & 1;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    if (kk < 3) {
                        read(bt, kk + 1, (kk + 1) & 1);
                    } else if (t + 1 < cur.nst) {
                        ready(t + 1);
                        read(bt ^ 1, 0, 0);
                    }
                    mfma(kk & 1);
                }
            }
        }
        // ---- the next segment's first stage, before this one's epilogue
        if (more) {
            if (cur.nst < 2) {      // its ids were not loaded on the way
                __syncthreads();
                first_ids(nxt, sbuf ^ 1);
                wait_vmcnt<0>();
                __syncthreads();
            }
            if (nxt.nst > 0) issue(nxt, sbuf ^ 1, 0, (b + cur.nst) & 1);
        }

        // ---- epilogue: value v of block [i][j] is output row i * 32 + fr, column j * 32 + (v / 4) * 8 + fc * 4 +
        // v % 4 of the wave's tile; the half waves swap quads, so that a lane gets 8 adjacent columns
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rl = wm * 64 + i * 32 + fr;
            bool ok;
            size_t at;
            if constexpr (DGRAD) {
                ok = source(s_id[sbuf][rl], cur.r0 + rl, cur.r_end, 0) >= 0;
                at = static_cast<size_t>(cur.r0 + rl) * K;
            } else {
                ok = cur.row0 + rl < N;
                at = (static_cast<size_t>(cur.e) * N + cur.row0 + rl) * K;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float o[8];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i][j][8 * p + x]),
                                                                        __float_as_uint(acc[i][j][8 * p + 4 + x]), false, false);
                        o[x] = __uint_as_float(r[0]);
                        o[4 + x] = __uint_as_float(r[1]);
                    }
                    const int col = cur.col0 + wn * 128 + j * 32 + p * 16 + fc * 8;
                    if (!ok || col >= K) continue;
                    if constexpr (F32) {
                        float* c = static_cast<float*>(g.out) + at + col;
                        f32x4 a{o[0], o[1], o[2], o[3]}, d{o[4], o[5], o[6], o[7]};
                        if (g.base) {
                            const float* s = static_cast<const float*>(g.base) + at + col;
                            a += *reinterpret_cast<const f32x4*>(s);
                            d += *reinterpret_cast<const f32x4*>(s + 4);
                        }
                        *reinterpret_cast<f32x4*>(c) = a;
                        *reinterpret_cast<f32x4*>(c + 4) = d;
                    } else {
                        if (!DGRAD && g.base) {
                            const u32x4 s = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(g.base) + at + col);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                o[2 * x] += __uint_as_float(s[x] << 16);
                                o[2 * x + 1] += __uint_as_float(s[x] & 0xffff0000u);
                            }
                        }
                        *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + at + col) =
                            u32x4{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7])};
                    }
                }
        }
        if (!more) break;
        b = (b + cur.nst) & 1;
        sbuf ^= 1;
        L = L2;
        cur = nxt;
    }
}

FastDiv make_div(uint32_t d) {
    if (d == 1) return {0, -1};
    int l = 0;
    while ((1u << l) < d) ++l;      // 2^(l-1) < d <= 2^l
    return {static_cast<uint32_t>(((1ull << (31 + l)) + d - 1) / d), l - 1};
}

hipError_t device_cus(int& cus) {
    static int known[kMaxDevices] = {0};
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
    if (known[dev] == 0) {
        int n = 0;
        err = hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev);
        if (err != hipSuccess) return err;
        known[dev] = n;
    }
    cus = known[dev];
    return hipSuccess;
}

// one workgroup per compute unit (128 KB of LDS each), in whole rounds over the 8 XCDs, or one per tile
hipError_t grid_for(int64_t tiles, int& grid) {
    int cus = 0;
    const hipError_t err = device_cus(cus);
    if (err != hipSuccess) return err;
    const int64_t most = cus / 8 * 8 > 8 ? cus / 8 * 8 : 8, want = (tiles + 7) / 8 * 8;
    grid = static_cast<int>(want < most ? want : most);
    return hipSuccess;
}

}  // namespace

hipError_t launch_dgrad(const uint16_t* dy0, const uint16_t* w0, const uint16_t* dy1, const uint16_t* w1, uint16_t* dx,
                        const int32_t* sorted_ids, const int32_t* offsets, int P, int top_k, int E, int N, int K,
                        int max_pad, int by_token, void* ws, int64_t ws_bytes, hipStream_t s) {
    GradArgs g{dy0, dy1, w0, w1, dx, nullptr, sorted_ids, offsets, make_div(top_k), P, E, N, K, max_pad, by_token, 0};
    const int64_t m = static_cast<int64_t>(max_pad) / kTile + (P < E ? P : E), n = (K + kTile - 1) / kTile;
    int grid = 0;
    const hipError_t err = grid_for(m * n, grid);
    if (err != hipSuccess) return err;
    grad_gemm_kernel<true, false><<<grid, kNT, 0, s>>>(g);
    return hipGetLastError();
}

hipError_t launch_wgrad(const uint16_t* dy, const uint16_t* x, void* dw, const void* base, bool f32,
                        const int32_t* sorted_ids, const int32_t* offsets, int P, int top_k, int E, int N, int K,
                        int max_pad, int dy_by_token, int x_by_token, void* ws, int64_t ws_bytes, hipStream_t s) {
    GradArgs g{dy, nullptr, x, nullptr, dw, base, sorted_ids, offsets, make_div(top_k), P, E, N, K, max_pad, dy_by_token, x_by_token};
    int grid = 0;
    const hipError_t err = grid_for(static_cast<int64_t>(E) * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile), grid);
    if (err != hipSuccess) return err;
    if (f32) grad_gemm_kernel<false, true><<<grid, kNT, 0, s>>>(g);
    else grad_gemm_kernel<false, false><<<grid, kNT, 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace moe
