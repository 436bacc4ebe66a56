// Grouped products for the gradients of the expert path, one launch for all experts.
//
//   dgrad   dx[r, k]   = sum over n of dy(r, n) W_e[n, k]  (+ a second pair)   rows r of expert e
//   wgrad   dw_e[n, k] = sum over rows r of e of dy(r, n) x(r, k)  (+ base)
//
// The forward products contract over the dimension in which both operands are contiguous.  Here the
// contraction runs across the memory rows of W (dgrad) and of both operands (wgrad): such an operand
// comes into LDS row by row as it lies in memory, and the MFMA fragments, which want eight consecutive
// contraction indices per lane, are read with the transposing LDS read (ds_read_b64_tr_b16: 16 lanes
// read 4 rows of 16 columns, lane i gets column i of the 4 rows).  No operand is transposed in memory.
//
// A workgroup of 8 waves computes tiles of 256 x 256 results, one after the other, 32 contraction
// indices (a half) at a time through a ring of four LDS slots that direct global -> LDS loads fill 3 to
// 4 halves ahead, across the ends of tiles.  A half costs a CU 1024 cycles of its matrix cores and
// 1024 of LDS (96 KB of fragments, 32 KB of loads at 128 bytes a cycle), so the two must run side by
// side: the two waves of a SIMD are in different groups, and while one group reads its fragments the
// other computes (two groups, a barrier per phase: 14336 x 4096 by 8 experts of 1024 rows, wgrad 1117 ->
// 923 us, dgrad 1138 -> 1000 us against both in step on 64-deep stages).  The column operand is the MFMA's first
// one, so that a lane's 4 results of a block lie in one output row.  16x16x32 MFMAs, not 32x32x16: on
// random data the card's power limit sets the clock, and a loop of the former alone reaches 2060 TFLOP/s
// against 1812.
//
// What bounds it: at 8 x (1024 x 4096 x 14336), 0.96 TFLOP, dgrad takes 887 us (1.08 PFLOP/s) and
// wgrad 868 us (1.11); eight library products of these layouts take 798 to 849 and 1020 us.  Matrix
// cores are busy for 60 and 56% of the cycles at a clock that falls to 1.6 to 1.9 GHz under the load; bank conflicts take
// 8 and 2% of the cycles.  The loads' path is what the rest waits for: without the loads in the
// main loop the same products take 618 and 820 us.  Their average latency is 400 cycles, far less than
// they are issued ahead; the address unit is busy for 77 and 57% of the cycles, since dgrad's rows of dy come in pieces
// of 64 bytes, half a line each.  A tile of few rows is loaded as a whole one (copies of a row that is there), so what
// counts of skewed experts' row tiles is how full they are: 73% (128 of them, 768 x 2048, two pairs: 456 us).
// Tiles of few halves are bound by that and by their ends (wgrad of 64 experts of 192 rows, 1408 x 4096: 263 us, 3.0
// TB/s): of 19 to 20 thousand cycles a tile its 7 halves take 14, 1400 to 1500 each where nothing waits and 1000 to 2000
// more in three of them, which wait for loads queued behind the stores of the last tile; an epilogue takes 4200 to 5400,
// and the way to the next tile's first half 700 to 950.  With sums to add to (2048 x 768 fp32, 501 us) an epilogue takes
// 27 to 42 thousand, and workgroups end 105 us before the last one on average: the busiest expert's tiles are as long as
// 250 halves.
//
// Tried and slower: two workgroups of 4 waves per CU with tiles of 128 x 256 and three slots, so that one's
// epilogue runs beside the other's products (dgrad 1000 to 1085 us, wgrad 1030, ragged 277; half as many
// bytes more through L2), the same with fragments read one half ahead (1057, 1069, 285).
//
// LDS layout.  Operands read by columns: row of 512 bytes, 16-byte chunk c of contraction row q at
// chunk c ^ ((q & 3) << 2 | ((q >> 3 ^ q >> 4) & 1) << 1): the 4 rows of each 16 lanes that one transposing read
// touches together lie in different banks.  dy of dgrad: rows of 64 bytes, chunk c of row q at c ^ (q >> 2 & 3).
//
// Rows without a pair (sentinels inside an expert's padded span) load a valid row and are not stored
// (dgrad), or load zeros from both operands (wgrad: they would enter every sum, and may hold anything).
#include <type_traits>

#include "device_common.h"
#include "launchers.h"

namespace moe {
namespace {

constexpr int kTile = 256;     // output rows and columns of a tile
constexpr int kBK = 32;        // contraction per LDS slot (a "half")
constexpr int kSlots = 4;
constexpr int kNT = 512;
constexpr int kPartB = kTile * kBK * 2;  // bytes of one operand in a slot
constexpr int kSlotB = 2 * kPartB;
constexpr int kMaxE = 256;
constexpr int kBand = 4;       // row tiles per band of the tile order (dgrad of 8 experts of 1024 rows, 4096 x 14336, and of
                               // 128 skewed ones, 768 x 2048: 2 948 and 469 us, 4 896 and 474 us, 8 898 and 482 us)
constexpr int kTab = 128;      // tiles of a workgroup
constexpr int kMaxPieces = 256;  // workgroups of a launch whose tiles are cut along the contraction
constexpr int kMaxSplit = 8;     // pieces of a tile
constexpr int kMinPiece = 16;    // halves of a piece
constexpr int kSegs = 8;       // dgrad: tiles whose row ids are held

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float lo_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

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
    int32_t* cnt;         // workspace, or NULL: counters [kMaxPieces], zero between calls
    float* part;          // and partial tiles [kMaxPieces][kTile * kTile]
};

// a tile of a workgroup's list
struct __attribute__((aligned(16))) Tile {
    int r0, r_end;   // dgrad: first sorted row, end of rows; wgrad: the expert's span
    int at;          // dgrad: first half (a piece's); wgrad: first output row, of N
    int en;          // expert | column tile << 8; < 0: no more tiles
};

// ---- Lists of tiles and addresses in LDS: whole numbers alone, so that a test compiles these for the CPU as they stand.

// wgrad: the tiles of an expert that go to one XCD together, and how many such units it has
__host__ __device__ __forceinline__ void units_of(int tiles_e, int tiles, int& unit, int& units_e) {
    units_e = (tiles_e + 31) / 32;
    if (tiles < 2048) {
        // Few tiles: an expert's go to all XCDs, so that a busy expert's long tiles do not stay in one (us with and without:
        // 8 skewed experts of 4096 x 1024 180 and 198, of 1408 x 4096 165 and 172, 16 of 2048 x 1024 145 and 150; 40, 64 and
        // 128 skewed ones level; equal ones 67 and 66, 50 and 50, 128 and 126).  It costs where short last units add a round:
        // 2 skewed experts of 4096 x 4096 215 and 209, 3 of 8192 x 2048 443 and 332.
        const int per = tiles < 128 ? 1 : tiles / 64;
        units_e = tiles_e / per > units_e ? tiles_e / per : units_e;
        units_e = units_e < tiles_e ? units_e : tiles_e;
    }
    unit = (tiles_e + units_e - 1) / units_e;
}

// the expert's unit that XCD xcd gets in round v: back and forth over the XCDs
__host__ __device__ __forceinline__ int unit_of_round(int v, int xcd) { return v * 8 + ((v & 1) ? 7 - xcd : xcd); }

// row and column tile of tile idx: bands of kBand row tiles, row tiles fastest, so that tiles that run together share
// operands in L2
__host__ __device__ __forceinline__ void tile_of(int idx, int row_tiles, int n_tiles, int& m_t, int& n_t) {
    const int band = idx / (kBand * n_tiles);
    const int at = idx - band * kBand * n_tiles;
    const int left = row_tiles - band * kBand, rows = left < kBand ? left : kBand;
    n_t = at / rows;
    m_t = band * kBand + at - n_t * rows;
}

// pieces of a tile where a launch of `grid` workgroups with a workspace has T of them, the longest of `most` halves
__host__ __device__ __forceinline__ int pieces_of(int T, int grid, int most) {
    if (T <= 0 || 2 * T > grid) return 1;
    int n = (grid < kMaxPieces ? grid : kMaxPieces) / T;
    n = n < kMaxSplit ? n : kMaxSplit;
    n = n < most / kMinPiece ? n : most / kMinPiece;
    return n > 1 ? n : 1;
}

// workgroups per XCD for `tiles` tiles, of which an XCD's list has at most `entries`
__host__ __device__ __forceinline__ int64_t per_xcd_for(int64_t tiles, int64_t entries, bool ws, int cus) {
    const int64_t most = cus / 8 > 1 ? cus / 8 : 1, want = (tiles + 7) / 8;
    const int64_t n = ws || want > most ? most : want;
    return entries > n * kTab ? (entries + kTab - 1) / kTab : n;
}

// Operands read by columns.  First of the eight columns that load q of `wave` puts where its lane's 16 bytes go; and the
// bytes from a slot's start to what `lane` reads of 16 columns from block * 16 (block < 8; 8 further on: + 256 bytes).
__host__ __device__ __forceinline__ int column_loaded(int wave, int lane, int q) {
    return ((lane & 31) ^ (((q * 2 + (lane >> 5)) << 2) | ((((wave >> 1) ^ (wave >> 2)) & 1) << 1))) * 8;
}
__host__ __device__ __forceinline__ int column_read(int lane, int block) {
    const int i16 = lane & 15, gr = lane >> 4, row = gr * 8 + (i16 >> 2), bit = (gr ^ (gr >> 1)) & 1;
    return row * 512 + (((((block >> 1) ^ (i16 >> 2)) << 2) | (((block & 1) ^ bit) << 1) | ((i16 & 3) >> 1)) << 4) + (i16 & 1) * 8;
}
// dy of dgrad: first contraction index of the lane's 16 bytes of a row, and where it reads row wm * 16 + lane % 16
__host__ __device__ __forceinline__ int row_loaded(int lane) { return ((lane & 3) ^ ((lane >> 4) & 3)) * 8; }
__host__ __device__ __forceinline__ int row_read(int lane, int wm) {
    const int i16 = lane & 15, gr = lane >> 4;
    return (wm * 16 + i16) * 64 + ((gr ^ (i16 >> 2)) << 4);
}
// results on their way out: 16-byte chunk `chunk` of row `row` in the wave's 1 KB
__host__ __device__ __forceinline__ int staged(int row, int chunk) { return row * 64 + (chunk ^ (row >> 2 & 3)) * 16; }

// ---- (end)

// DGRAD: bf16 out; else wgrad with bf16 (F32 false) or fp32 results
template <bool DGRAD, bool F32>
__global__ __launch_bounds__(kNT, 1) void grad_gemm_kernel(GradArgs g) {
    __shared__ __attribute__((aligned(1024))) char smem[kSlots * kSlotB];
    __shared__ int s_lo[kMaxE], s_hi[kMaxE], s_tb[kMaxE + 1], s_order[kMaxE];
    __shared__ int s_scan[kNT / 64];
    __shared__ Tile s_tab[kTab];
    __shared__ int s_n;           // entries in it
    __shared__ int s_arrived;
    __shared__ __attribute__((aligned(1024))) char s_stage[kNT / 64 * 1024];   // a wave's results on their way out
    // sorted ids.  dgrad: of the rows of the last kSegs tiles.  wgrad: per wave, of its rows (4 per half) of 16 halves, twice
    __shared__ __attribute__((aligned(16))) int s_id[DGRAD ? kSegs * kTile : kNT / 64 * 2 * 64];
    // wgrad: per wave, the rows' addresses in the two operands (the zeros' where a row holds no pair)
    __shared__ ulonglong2 s_ptr[DGRAD ? 1 : kNT];

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
    const int nkh = (N + kBK - 1) / kBK;             // dgrad: halves of one pair
    const int per_xcd = gridDim.x >> 3;
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int m_real = DGRAD ? __builtin_amdgcn_readfirstlane(s_tb[E]) : 0;
    const int tiles_e = r_tiles * n_tiles;
    const int T = DGRAD ? m_real * n_tiles : E * tiles_e;
    auto halves_of = [&](int e) __attribute__((always_inline)) { return (s_hi[e] - s_lo[e] + kBK - 1) / kBK; };

    // ---- Few tiles (and a workspace): each is cut along the contraction into `pieces`, one per workgroup, which meet
    // through fp32 partial tiles in the workspace (dgrad of 64 rows, 14336 x 4096: 160 -> 54 us; wgrad of 8192 rows,
    // 1024 x 1024: 167 -> 56 us).  Meeting costs 5 to 20 us, so pieces have 16 halves or more (300 rows, 520 x 264: whole
    // 16 us, in pieces of 8 halves 21).  All tiles of a launch count, those of experts without rows among them.
    int pieces = 1;
    if (g.part && T > 0 && 2 * T <= static_cast<int>(gridDim.x)) {
        const int most = DGRAD ? (g.r1 ? 2 * nkh : nkh) : halves_of(s_order[0]);
        pieces = __builtin_amdgcn_readfirstlane(pieces_of(T, gridDim.x, most));
    }

    // ---- this workgroup's list of tiles.  An XCD's tiles are dealt to its workgroups in turn, entries slot,
    // slot + per_xcd, ...; dgrad: an eighth of the tiles each.  wgrad: units of up to 32 tiles of one expert, dealt to
    // the XCDs by falling length, back and forth.
    const int l_lo = DGRAD ? static_cast<int>(static_cast<long long>(T) * xcd / 8) : 0;
    int unit = 1, units_e = 1;
    if constexpr (!DGRAD) units_of(tiles_e, T, unit, units_e);
    const int units = E * units_e, xcd_units = (units + 7) / 8;
    const int l_n = DGRAD ? static_cast<int>(static_cast<long long>(T) * (xcd + 1) / 8) - l_lo : xcd_units * unit;
    // tile idx (dgrad: of all; wgrad: of expert e)
    auto tile_at = [&](int idx, int e) __attribute__((always_inline)) {
        int m_t, n_t;
        tile_of(idx, DGRAD ? m_real : r_tiles, n_tiles, m_t, n_t);
        Tile s;
        if constexpr (DGRAD) {
            int hi = E - 1;  // e: the largest expert whose first row tile is <= m_t
            e = 0;
            while (e < hi) {
                const int mid = (e + hi + 1) >> 1;
                if (s_tb[mid] <= m_t) e = mid; else hi = mid - 1;
            }
            s.r0 = s_lo[e] + (m_t - s_tb[e]) * kTile;
            s.r_end = min(s.r0 + kTile, s_hi[e]);
            s.at = 0;
        } else {
            s.at = m_t * kTile;
            s.r0 = s_lo[e];
            s.r_end = s_hi[e];
        }
        s.en = e | n_t << 8;
        return s;
    };
    // entry number n of this workgroup, if it is a tile
    const int all_nh = g.r1 ? 2 * nkh : nkh;
    const int piece = pieces > 1 ? blockIdx.x / T : 0;       // of tile blockIdx % T
    auto locate = [&](int n, Tile& s) __attribute__((always_inline)) {
        if (pieces > 1) {
            const int t = blockIdx.x % T;
            if (n > 0 || piece >= pieces) return false;
            s = tile_at(DGRAD ? t : t % tiles_e, DGRAD ? 0 : t / tiles_e);
            const int nh = DGRAD ? all_nh : (s.r_end - s.r0 + kBK - 1) / kBK;
            const int h0 = nh * piece / pieces, h1 = nh * (piece + 1) / pieces;
            if constexpr (DGRAD) {
                s.at = h0;
            } else {
                s.r0 += h0 * kBK;
                s.r_end = min(s.r_end, s.r0 + (h1 - h0) * kBK);
            }
            return true;
        }
        const int i = slot + n * per_xcd;
        if (i >= l_n) return false;
        if constexpr (DGRAD) {
            s = tile_at(l_lo + i, 0);
        } else {
            const int u = unit_of_round(i / unit, xcd), idx = (u % units_e) * unit + i % unit;
            if (u >= units || idx >= tiles_e) return false;
            s = tile_at(idx, s_order[u / units_e]);
        }
        return true;
    };
    // located once, by a thread each (a dependent chain of divisions and searches; in the main loop it cost
    // 5% where tiles have few halves); the launcher sees to it that the table holds all
    {
        Tile t = {};
        const bool is_tile = tid < kTab && locate(tid, t);
        const int at = block_inclusive_scan<kNT / 64>(is_tile ? 1 : 0, s_scan, kTab / 64) - 1;
        if (is_tile) s_tab[at] = t;
        if (tid == kTab - 1) s_n = at + 1;
        __syncthreads();
    }
    const int tab_n = __builtin_amdgcn_readfirstlane(s_n);
    auto tile = [&](int n) __attribute__((always_inline)) {
        Tile t = {0, 0, 0, -1};
        if (n < tab_n) {
            t = s_tab[n];
            t.r0 = __builtin_amdgcn_readfirstlane(t.r0);
            t.r_end = __builtin_amdgcn_readfirstlane(t.r_end);
            t.at = __builtin_amdgcn_readfirstlane(t.at);
            t.en = __builtin_amdgcn_readfirstlane(t.en);
        }
        return t;
    };
    const int piece_nh = all_nh * (piece + 1) / pieces - all_nh * piece / pieces;   // dgrad
    auto halves = [&](const Tile& t) __attribute__((always_inline)) {
        return DGRAD ? piece_nh : static_cast<int>(static_cast<uint32_t>(t.r_end - t.r0 + kBK - 1) / kBK);
    };
    auto expert = [](const Tile& t) __attribute__((always_inline)) { return t.en & 255; };
    auto column = [](const Tile& t) __attribute__((always_inline)) { return (t.en >> 8) * kTile; };

    // address of row `row` of an operand of `width` columns (one 32 x 32 bit product)
    auto row_address = [](const void* p, int row, int width) __attribute__((always_inline)) {
        uint32_t bytes = static_cast<uint32_t>(width) * 2;
        asm volatile("" : "+s"(bytes));   // (keeps the compiler from widening it first)
        return reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(static_cast<uint32_t>(row)) * bytes;
    };
    const uint32_t lds0 = lds_u32(smem), lds_id = lds_u32(s_id);
    const char* zero = reinterpret_cast<const char*>(kZero16);
    const int half = lane >> 5;
    // row of an operand for sorted row r with id p; < 0: no pair
    auto source = [&](int p, int r, int r_end, int tok) __attribute__((always_inline)) {
        return r < r_end && p >= 0 && p < g.P ? (tok ? fast_div(p, g.top_k) : r) : -1;
    };

    // ---- the issuing cursor, 3 or 4 halves ahead of the one that is computed.  i_left halves can be issued before
    // the cursor has to be moved (move()): to the half that ends past N and to the second pair (dgrad), to the next 16
    // ids (wgrad), to the next segment, and behind the last one to halves of zeros that nobody reads, so that the main
    // loop needs no tests.
    int i_n = 1, i_seq = 0, i_h = 0, i_left = 0, i_since = 0, i_slot = 0, id_par = 1;
    Tile is = tile(0), in = {};      // the tile whose halves are loaded, and the next one
    int is_nh = is.en < 0 ? 0 : halves(is);
    bool i_next = false;
    // Ids that this wave's loads need, straight into LDS (rows past max_pad read the last id; checked where
    // used).  dgrad: the wave's 32 rows of tile number seq.  wgrad: its 4 rows of each of 16 halves.
    auto load_ids = [&](int r0, int batch, int seq, int par) __attribute__((always_inline)) {
        if constexpr (DGRAD) {
            if (lane < 32)
                dma4(g.sorted_ids + min(r0 + wave * 32 + lane, g.max_pad - 1),
                     lds_id + ((seq & (kSegs - 1)) * kTile + wave * 32) * 4);
        } else {
            const int r = r0 + (batch * 16 + (lane >> 2)) * kBK + wave * 4 + (lane & 3);
            dma4(g.sorted_ids + min(r, g.max_pad - 1), lds_id + (wave * 2 + par) * 256);
        }
    };
    // this lane's sources, loads q of each operand.  dgrad: of the coming half, and how far to the next.  wgrad: the
    // bytes from a row's start.
    const char* rp[2];
    const char* cp[2];
    uint32_t step_r = 0;
    uint64_t step_c = 0;
    int at[2], chunk_c[2], col_r[2], col_c[2];
    uint32_t lane_c[2];         // dgrad: bytes from a half's first row of W to this lane's
#pragma unroll
    for (int q = 0; q < 2; ++q) chunk_c[q] = column_loaded(wave, lane, q);
#pragma unroll
    for (int q = 0; q < 2; ++q) lane_c[q] = static_cast<uint32_t>(wave * 4 + q * 2 + half) * (static_cast<uint32_t>(K) * 2);
    const int k_r = row_loaded(lane);   // dgrad: first n of this lane's chunk of a row of dy
    const ulonglong2* row_p = s_ptr;   // wgrad: the row addresses of the coming half
    // what can be issued from half i_h of the segment on
    auto move = [&](bool first) __attribute__((always_inline)) {
        if constexpr (DGRAD) {
            const int at_h = is.at + i_h;            // of both pairs' halves
            const bool second = at_h >= nkh;
            const int h = second ? at_h - nkh : at_h;
            if (first || h == 0) {                   // the tile or a pair begins
                const char* R = reinterpret_cast<const char*>((second ? g.r1 : g.r0) + h * kBK);
                const char* C = reinterpret_cast<const char*>((second ? g.c1 : g.c0) + (static_cast<uint64_t>(expert(is)) * N + h * kBK) * K);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    rp[q] = reinterpret_cast<const char*>(row_address(R, at[q], N)) + k_r * 2;
                    cp[q] = C + lane_c[q] + min(column(is) + chunk_c[q], K - 8) * 2;  // columns past K are never stored
                }
                step_r = kBK * 2;
                step_c = static_cast<uint64_t>(kBK * 2) * K;
            }
            i_left = min(N / kBK - h, is_nh - i_h);  // whole halves
            if (i_left <= 0) {                       // the one that ends past N: zeros there, of both operands
                i_left = 1;
                const int rest = N - h * kBK;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (k_r >= rest) rp[q] = zero;
                    if (wave * 4 + q * 2 + half >= rest) cp[q] = zero;
                }
            }
        } else {
            // the row addresses of 16 halves, a row per lane
            id_par ^= 1;
            const int p = s_id[(wave * 2 + id_par) * 64 + lane];
            const int r = is.r0 + (i_h + (lane >> 2)) * kBK + wave * 4 + (lane & 3);
            const bool real = r < is.r_end && p >= 0 && p < g.P;
            const int tok = fast_div(p, g.top_k);
            s_ptr[wave * 64 + lane] = real ? ulonglong2{row_address(g.r0, g.r_tok ? tok : r, N), row_address(g.c0, g.c_tok ? tok : r, K)}
                                           : ulonglong2{reinterpret_cast<uint64_t>(zero), reinterpret_cast<uint64_t>(zero)};
            row_p = s_ptr + wave * 64 + half;
            const int b = i_h / 16 + 1;
            const bool same = b * 16 < is_nh;
            const int this_r0 = is.r0, next_r0 = in.r0;   // (a choice between the members would put both in memory)
            if (same || i_next) load_ids(same ? this_r0 : next_r0, same ? b : 0, 0, id_par ^ 1);
            i_left = min(16, is_nh - i_h);
        }
        i_h += i_left;
    };
    // the cursor moves: within the segment (i_h: the first half not yet given out), or to the next
    auto next = [&](bool start) __attribute__((always_inline)) {
        const bool first = start || i_h >= is_nh;
        if (first) {
            if (!start) {
                if (!i_next) {
                    if constexpr (DGRAD) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) rp[q] = cp[q] = zero;
                        step_r = 0;
                        step_c = 0;
                    } else {
                        s_ptr[wave * 64 + lane] = ulonglong2{reinterpret_cast<uint64_t>(zero), reinterpret_cast<uint64_t>(zero)};
                        row_p = s_ptr + wave * 64 + half;
                    }
                    i_left = 0x7fffffff;   // (at most 4 are computed and issued from here on)
                    return;
                }
                is = in;
                is_nh = halves(is);
                ++i_seq;
            }
            in = tile(i_n++);                  // (tiles without halves come last)
            i_next = in.en >= 0 && halves(in) > 0;
            i_h = 0;
        }
        // the ids: this wave's own loads of them, at least 3 halves ago (then the waits of the main loop cover them)
        if (!DGRAD || first) {
            if (i_since < 3) wait_vmcnt<0>();
            i_since = 0;
        }
        if (first) {
            if constexpr (DGRAD) {
                const int* ids = s_id + (i_seq & (kSegs - 1)) * kTile;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int row = wave * 32 + q * 16 + (lane >> 2);
                    const int src = source(ids[row], is.r0 + row, is.r_end, g.r_tok);
                    at[q] = src >= 0 ? src : (g.r_tok ? 0 : is.r0);   // a row that is always there; not stored
                }
                if (i_next) load_ids(in.r0, 0, i_seq + 1, 0);
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    col_r[q] = min(is.at + chunk_c[q], N - 8) * 2;   // (columns past the ends are never stored)
                    col_c[q] = min(column(is) + chunk_c[q], K - 8) * 2;
                }
            }
        }
        move(first);
    };

    // Sources of the coming half (in the shadow of the MFMAs); then a load of each operand per q.
    // wgrad: rows[q] are the addresses of the row of load q, read from LDS beforehand.
    const char* src_r[2];
    const char* src_c[2];
    ulonglong2 rows[2];
    uint32_t dst_r;
    auto read_rows = [&]() __attribute__((always_inline)) {
        if constexpr (!DGRAD) {
            rows[0] = row_p[0];
            rows[1] = row_p[2];
        }
    };
    auto sources = [&](int q) __attribute__((always_inline)) {
        if constexpr (DGRAD) {
            src_r[q] = rp[q];
            src_c[q] = cp[q];
            rp[q] += step_r;
            cp[q] += step_c;
        } else {
            const bool real = rows[q].x != reinterpret_cast<uint64_t>(zero);
            src_r[q] = reinterpret_cast<const char*>(rows[q].x) + static_cast<uint32_t>(real ? col_r[q] : 0);
            src_c[q] = reinterpret_cast<const char*>(rows[q].y) + static_cast<uint32_t>(real ? col_c[q] : 0);
            if (q == 1) row_p += 4;
        }
        if (q == 1) {
            dst_r = lds0 + i_slot + wave * 2048;
            i_slot = (i_slot + kSlotB) & (kSlots * kSlotB - 1);
        }
    };
    auto load_r = [&](int q) __attribute__((always_inline)) { dma16(src_r[q], dst_r + q * 1024); };
    auto load_c = [&](int q) __attribute__((always_inline)) { dma16(src_c[q], dst_r + kPartB + q * 1024); };

    int c_slot = 0, c_seq = 0;               // slot of the half that is computed; tiles done
    // A wave's rows are i * 64 + wm * 16 (i < 4), its columns (j / 2) * 64 + wn * 32 + (j % 2) * 16 (j < 8), 16 each:
    // tiles of few rows or columns then leave the same share of blocks to every wave.
    constexpr int kStores = F32 ? 32 : 16;   // store instructions of an epilogue, whatever is masked
    const int wm = wave >> 1, wn = wave & 1;
    const int group = wave >> 2;               // the two waves of a SIMD (w and w + 4) are in different groups
    // Fragment offsets in bytes within a slot.  A lane of the 16x16x32 MFMA holds 8 contraction indices from
    // 8 * (lane / 16) of row or column lane % 16.  Transposed reads: lane i16 of group gr of 16 lanes reads 8 bytes of
    // contraction row gr * 8 + i16 / 4 (+ 4 in the second read), columns (i16 % 4) * 4.
    int c_off[4], r_off[2];      // blocks 8 further on lie 256 bytes further on
#pragma unroll
    for (int j = 0; j < 4; ++j) c_off[j] = kPartB + column_read(lane, (j >> 1) * 4 + wn * 2 + (j & 1));
#pragma unroll
    for (int i = 0; i < 2; ++i) r_off[i] = DGRAD ? row_read(lane, wm) : column_read(lane, i * 4 + wm);

    f32x4 acc[4][8];
    bf16x8 fa[4], fb[8];
    auto tr_read = [&](const char* p) __attribute__((always_inline)) {
        typedef __attribute__((address_space(3))) s16x4 lds4;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)(p + 4 * 512));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    };
    auto read = [&](auto rf_c, auto cf_c) __attribute__((always_inline)) {
        const char* st = smem + c_slot;
#pragma unroll
        for (int i = 0; i < decltype(rf_c)::value; ++i) {
            if constexpr (DGRAD) fa[i] = *reinterpret_cast<const bf16x8*>(st + r_off[0] + i * 4096);
            else fa[i] = tr_read(st + r_off[i & 1] + (i >> 1) * 256);
        }
#pragma unroll
        for (int j = 0; j < decltype(cf_c)::value; ++j) fb[j] = tr_read(st + c_off[j & 3] + (j >> 2) * 256);
    };
    auto barrier = [&]() __attribute__((always_inline)) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    // The MFMAs of a half, RF x CF blocks, with the loads of a later half spread among them; FIRST: from zero.
    auto compute = [&](auto rf_c, auto cf_c, auto first_c) __attribute__((always_inline)) {
        constexpr int CF = decltype(cf_c)::value, M = decltype(rf_c)::value * CF;
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int n = 0; n < M; ++n) {
            const int i = n / CF, j = n % CF;
            const f32x4 z = {};
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], decltype(first_c)::value ? z : acc[i][j], 0, 0, 0);
            if (n == 0) sources(0);
            if (n == M / 8) sources(1);
            if (n == M / 4 - 1) { __builtin_amdgcn_sched_barrier(0); load_r(0); }
            if (n == M / 2 - 1) { __builtin_amdgcn_sched_barrier(0); load_c(0); }
            if (n == M * 11 / 16 - 1) { __builtin_amdgcn_sched_barrier(0); load_r(1); }
            if (n == M * 7 / 8 - 1) { __builtin_amdgcn_sched_barrier(0); load_c(1); }
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(0);
    };
    // One half, in two phases with a barrier at the end of each; the first group computes while the second reads.  At the
    // barriers this wave's loads of the next half have landed: vmcnt counts in order, and what may be in flight are the
    // loads of two later halves (4 each) and, in the two halves that follow an epilogue (after), its stores.  (The first
    // group needs the wait at the second barrier only, the second group at the first; at the other one it asks for what
    // has landed before, or for what the next half will need.)
    auto one_half = [&](auto rf_c, auto cf_c, auto first_c, bool after, bool close) __attribute__((always_inline)) {
        auto landed = [&]() __attribute__((always_inline)) {
            if (after) wait_vmcnt<8 + kStores>();
            else wait_vmcnt<8>();
        };
        read(rf_c, cf_c);
        read_rows();
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): the slot is read
        landed();
        barrier();
        compute(rf_c, cf_c, first_c);
        if (close) {
            landed();
            barrier();
        }
        c_slot = (c_slot + kSlotB) & (kSlots * kSlotB - 1);
        ++i_since;
    };
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I4 = std::integral_constant<int, 4>;
    using I8 = std::integral_constant<int, 8>;

    // ---- Epilogue of tile cs.  Value v of block [i][j] is output row i16 of the block's rows and column gr * 4 + v of its
    // columns.  Four neighbouring lanes, four rows, would store to four places, which the address unit takes one by one
    // (16 rows of 64 bytes an instruction: 280 cycles each, and 1.4 x the time of the whole product where tiles are short);
    // so 16 rows of 64 bytes at a time go through 1 KB of LDS of the wave's own, from which lane l reads 16 bytes
    // of row l / 4 (110 cycles).  The 16-byte chunk c of row r is at c ^ (r / 4 & 3): no bank conflicts either way.
    // Masked lanes store past the buffer's end, which the hardware drops: the number of stores is always the same.
    // base: the loads of two steps are in flight while the one before is added and stored (fp32 sums of 128 skewed experts,
    // 2048 x 768: 511 -> 501 us against one step; three spill).
    Tile cs = {};
    auto finish = [&]() __attribute__((always_inline)) {
        constexpr int ES = F32 ? 4 : 2, PW = F32 ? 8 : 4;   // bytes of a value, 64-byte pieces of a wave's row
        const uint64_t first = (DGRAD ? static_cast<uint64_t>(cs.r0) : static_cast<uint64_t>(expert(cs)) * N + cs.at) * K + column(cs);
        auto resource = [&](const void* p) __attribute__((always_inline)) {
            return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(uniform_ptr(static_cast<const char*>(p) + first * ES)), 0,
                                                     0x7fffffff, 0x00020000);
        };
        const __amdgpu_buffer_rsrc_t out = resource(g.out);
        // (opaque to the compiler, which would else keep the offsets below in registers through the main loop)
        int ln = lane, wv = wave;
        asm volatile("" : "+v"(ln), "+s"(wv));
        const int em = wv >> 1, en = wv & 1, sr = ln >> 2;   // the row of this lane's pieces
        char* const stage = s_stage + wv * 1024;
        char* const mine = stage + staged(sr, ln & 3);
        const int br = ln & 15, bg = ln >> 4;                // row and columns of its values of a block
        auto of_block = [&](int chunk) __attribute__((always_inline)) { return stage + staged(br, chunk); };
        uint32_t ok = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rl = i * 64 + em * 16 + sr;
            bool in;
            if constexpr (DGRAD) in = source(s_id[(c_seq & (kSegs - 1)) * kTile + rl], cs.r0 + rl, cs.r_end, 0) >= 0;
            else in = cs.at + rl < N;
            ok |= in ? 1u << i : 0u;
        }
        const int col0 = F32 ? en * 32 + (ln & 3) * 4 : en * 32 + (ln & 3) * 8;
        const uint32_t off0 = (static_cast<uint32_t>(em * 16 + sr) * K + col0) * ES, row64 = static_cast<uint32_t>(K) * (64 * ES);
        auto offset = [&](int i, int q) __attribute__((always_inline)) -> uint32_t {   // of piece q of row i
            const int col = F32 ? (q >> 1) * 64 + (q & 1) * 16 : q * 64;
            const uint32_t at = off0 + i * row64 + col * ES;
            const bool in = static_cast<bool>(ok >> i & 1) & (column(cs) + col0 + col < K);
            return in ? at : 0x80000000u;
        };
        auto store = [&](auto base_c) __attribute__((always_inline)) {
            constexpr bool BASE = decltype(base_c)::value;
            constexpr int STEPS = PW;   // 4 rows of PW pieces, 4 pieces a step
            __amdgpu_buffer_rsrc_t in = out;
            u32x4 old[3][4], w[2][4];
            auto of_step = [&](int n, int q) __attribute__((always_inline)) { return F32 ? offset(n >> 1, (n & 1) * 4 + q) : offset(n, q); };
            auto fetch = [&](int n) __attribute__((always_inline)) {
#pragma unroll
                for (int q = 0; q < 4; ++q) old[n % 3][q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(in, of_step(n, q), 0, 0));
            };
            auto through_lds = [&](int n) __attribute__((always_inline)) {
                const int i = F32 ? n >> 1 : n;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if constexpr (F32) {
                        *reinterpret_cast<f32x4*>(of_block(bg)) = acc[i][(n & 1) * 4 + q];
                    } else {
                        f32x4 a = acc[i][2 * q], b = acc[i][2 * q + 1];
                        char* const lo = of_block(bg >> 1) + (bg & 1) * 8;
                        char* const hi = of_block(2 + (bg >> 1)) + (bg & 1) * 8;
                        if constexpr (BASE) {   // added before the rounding, in the blocks' layout
                            *reinterpret_cast<u32x4*>(mine) = old[n % 3][q];
                            const u32x2 x = *reinterpret_cast<const u32x2*>(lo), y = *reinterpret_cast<const u32x2*>(hi);
                            a += f32x4{lo_f32(x[0]), hi_f32(x[0]), lo_f32(x[1]), hi_f32(x[1])};
                            b += f32x4{lo_f32(y[0]), hi_f32(y[0]), lo_f32(y[1]), hi_f32(y[1])};
                        }
                        *reinterpret_cast<u32x2*>(lo) = u32x2{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])};
                        *reinterpret_cast<u32x2*>(hi) = u32x2{pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])};
                    }
                    w[n & 1][q] = *reinterpret_cast<const u32x4*>(mine);
                }
            };
            if constexpr (BASE) {
                in = resource(g.base);
                fetch(0);
                fetch(1);
            }
            through_lds(0);
#pragma unroll
            for (int n = 0; n < STEPS; ++n) {   // a step's results leave while the next one's come from LDS
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (BASE)
                    if (n + 2 < STEPS) fetch(n + 2);
                u32x4 sum[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    sum[q] = w[n & 1][q];
                    if constexpr (F32 && BASE) sum[q] = __builtin_bit_cast(u32x4, __builtin_bit_cast(f32x4, sum[q]) + __builtin_bit_cast(f32x4, old[n % 3][q]));
                }
                if (n + 1 < STEPS) through_lds(n + 1);
#pragma unroll
                for (int q = 0; q < 4; ++q) __builtin_amdgcn_raw_buffer_store_b128(sum[q], out, of_step(n, q), 0, 0);
            }
        };
        if (!DGRAD && g.base) store(std::true_type{});
        else store(std::false_type{});
        ++c_seq;
    };

    // ---- main loop
    const bool any = is_nh > 0;
    if (any) {
        load_ids(is.r0, 0, 0, 0);
        next(true);
#pragma nounroll
        for (int q = 0; q < 3 + group; ++q) {
            read_rows();
            sources(0);
            sources(1);
            load_r(0); load_r(1); load_c(0); load_c(1);
            if (--i_left == 0) next(false);   // (i_since stays 0: nothing has been waited for)
        }
        wait_vmcnt<8>();
        barrier();
        if (group) barrier();
    }
    for (int n = 0;; ++n) {
        cs = tile(n);
        if (cs.en < 0) break;
        const int nh = halves(cs);
        const int n_rows = DGRAD ? cs.r_end - cs.r0 : N - cs.at, n_cols = K - column(cs);
        const bool again = n > 0;
        const bool whole = nh > 0 && n_rows > 128 && n_cols > 128;
        // The second group's last barrier of a whole tile comes after its epilogue, which so runs beside the first group's
        // instead of after it (wgrad of 8 experts of 1024 rows, 14336 x 4096: 874 -> 864 us; 64 experts of 192 rows,
        // 1408 x 4096: 270 -> 263 us; not for parts of tiles, where the test in every half costs 2%).
        const bool open = whole && group && pieces == 1;
        if (whole) {
            one_half(I4{}, I8{}, std::true_type{}, again, nh > 1 || !open);
            if (--i_left == 0) next(false);
            int left = nh - 1;
            if (left > 0) {
                one_half(I4{}, I8{}, std::false_type{}, again, left > 1 || !open);
                if (--i_left == 0) next(false);
                --left;
            }
            while (left > 0) {
                const int run = min(left, i_left);
                for (int r = 1; r <= run; ++r) one_half(I4{}, I8{}, std::false_type{}, false, r < left || !open);
                left -= run;
                i_left -= run;
                if (i_left == 0) next(false);
            }
        } else {
            // Fewer blocks hold rows or columns (or the expert has no rows): a half then costs a wave less (dgrad of 16 tokens
            // over 64 experts 103 us, else 139; of 128 skewed experts 474, else 498).
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
            auto some = [&](auto rf_c, auto cf_c) __attribute__((always_inline)) {
                for (int h = 0; h < nh; ++h) {
                    one_half(rf_c, cf_c, std::false_type{}, again && h < 2, true);
                    if (--i_left == 0) next(false);
                }
            };
            if (n_rows > 128) some(I4{}, I4{});
            else if (n_rows > 64) some(I2{}, I8{});
            else some(I1{}, I8{});
        }
        if (pieces > 1) break;      // a piece is not a tile yet
        finish();
        if (open) barrier();
    }
    if (any && !group) barrier();   // the other group's last
    wait_vmcnt<0>();                // the halves of zeros: nothing may land in LDS after the end

    // ---- A piece of a tile: its partial sums through the workspace.  They are written and read with device-coherent
    // accesses (sc1), complete (vmcnt) before the piece is counted on the tile's counter.  The last piece to arrive adds
    // all of them in the pieces' order, so that the result does not depend on which it is, stores the tile and resets the
    // counter.  Nobody waits for anybody.
    if (pieces > 1 && static_cast<int>(blockIdx.x) < pieces * T) {
        constexpr int kSc1 = 16;
        const int t = blockIdx.x % T;
        const __amdgpu_buffer_rsrc_t part = __builtin_amdgcn_make_buffer_rsrc(g.part, 0, kMaxPieces * kTile * kTile * 4, 0x00020000);
        auto at_part = [&](int piece) __attribute__((always_inline)) {   // [piece][16-byte chunk][thread]
            return (static_cast<uint32_t>(piece) * T + t) * (kTile * kTile * 4) + tid * 16;
        };
        uint32_t o = at_part(blockIdx.x / T);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), part, o + (i * 8 + j) * (kNT * 16), 0, kSc1);
        wait_vmcnt<0>();
        __syncthreads();
        if (tid == 0) s_arrived = __hip_atomic_fetch_add(&g.cnt[t], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (s_arrived != pieces - 1) return;
        if (tid == 0) __hip_atomic_store(&g.cnt[t], 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma nounroll
        for (int piece = 0; piece < pieces; ++piece) {
            o = at_part(piece);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u32x4 v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(part, o + (i * 8 + j) * (kNT * 16), 0, kSc1));
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i][j] += __builtin_bit_cast(f32x4, v[j]);
            }
        }
        finish();
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

// One workgroup per compute unit (160 KB of LDS), in whole rounds over the 8 XCDs; one per tile where there are fewer and
// no workspace to cut them in; more where an XCD's list of `entries` would not fit its workgroups' tables.
hipError_t grid_for(int64_t tiles, int64_t entries, bool ws, int& grid) {
    int cus = 0;
    const hipError_t err = device_cus(cus);
    if (err != hipSuccess) return err;
    grid = static_cast<int>(per_xcd_for(tiles, entries, ws, cus) * 8);
    return hipSuccess;
}

// the workspace of the grouped GEMMs: counters, then partial tiles (the entry points check its size)
constexpr int64_t kCounterBytes = 4096;
int32_t* counters(void* ws) { return static_cast<int32_t*>(ws); }
float* partials(void* ws) { return ws ? reinterpret_cast<float*>(static_cast<char*>(ws) + kCounterBytes) : nullptr; }

}  // namespace

int64_t grad_gemm_workspace_bytes() { return kCounterBytes + static_cast<int64_t>(kMaxPieces) * kTile * kTile * 4; }

hipError_t launch_dgrad(const uint16_t* dy0, const uint16_t* w0, const uint16_t* dy1, const uint16_t* w1, uint16_t* dx,
                        const int32_t* sorted_ids, const int32_t* offsets, int P, int top_k, int E, int N, int K,
                        int max_pad, int by_token, void* ws, hipStream_t s) {
    GradArgs g{dy0, dy1, w0, w1, dx, nullptr, sorted_ids, offsets, make_div(top_k), P, E, N, K, max_pad, by_token, 0, counters(ws), partials(ws)};
    const int64_t m = static_cast<int64_t>(max_pad) / kTile + (P < E ? P : E), n = (K + kTile - 1) / kTile;
    int grid = 0;
    const hipError_t err = grid_for(m * n, (m * n + 7) / 8, ws != nullptr, grid);
    if (err != hipSuccess) return err;
    grad_gemm_kernel<true, false><<<grid, kNT, 0, s>>>(g);
    return hipGetLastError();
}

hipError_t launch_wgrad(const uint16_t* dy, const uint16_t* x, void* dw, const void* base, bool f32,
                        const int32_t* sorted_ids, const int32_t* offsets, int P, int top_k, int E, int N, int K,
                        int max_pad, int dy_by_token, int x_by_token, void* ws, hipStream_t s) {
    GradArgs g{dy, nullptr, x, nullptr, dw, base, sorted_ids, offsets, make_div(top_k), P, E, N, K, max_pad, dy_by_token, x_by_token, counters(ws), partials(ws)};
    int grid = 0;
    const int tiles_e = ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile), tiles = E * tiles_e;
    int unit = 1, units_e = 1;
    units_of(tiles_e, tiles, unit, units_e);
    const hipError_t err = grid_for(tiles, (static_cast<int64_t>(E) * units_e + 7) / 8 * unit, ws != nullptr, grid);
    if (err != hipSuccess) return err;
    if (f32) grad_gemm_kernel<false, true><<<grid, kNT, 0, s>>>(g);
    else grad_gemm_kernel<false, false><<<grid, kNT, 0, s>>>(g);
    return hipGetLastError();
}

}  // namespace moe
