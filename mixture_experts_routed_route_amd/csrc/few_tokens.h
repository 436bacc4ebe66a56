// Host-side description of the few-token layer (few_tokens.hip): limits, workspace layout, arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kFewTokens = 32;  // tokens: one bit each of an expert's mask
constexpr int kFewTopK = 32;    // slots per token
constexpr int kFewGrid = 256;   // workgroups of the first launch: one per compute unit
constexpr int kFewDownGrid = 256;  // workgroups the second launch aims at, by splitting the experts
constexpr int kFewMaxSplits = 16;
constexpr int kFewMaxHidden = 65536;
constexpr int kFewCounterBytes = kFewMaxHidden / 32 * 4;  // one counter per output panel (32 columns or more)

struct FewWeight {
    const void* data;
    const void* scales;
    const int32_t* qzeros;
};

struct FewArgs {
    const float* logits;
    const uint16_t* x;
    FewWeight gate, up, down;
    int32_t* ids;
    float* w;
    uint16_t* out;
    uint16_t* hs;   // workspace: bf16 [2, T * top_k, I], high and low parts
    float* part;    // workspace: partial output panels
    int32_t* cnt;   // workspace: one counter per output panel, zero between calls
    int T, E, top_k, H, I, renorm, splits, group;
};

// Workspace: counters | partial panels | hs.  The counters' place and size are the same for every call,
// so that no call's partial sums land where another layer's counters have to be zero; the size grows
// with the number of tokens, so a workspace made for more tokens serves fewer.
struct FewLayout {
    int splits;
    int64_t part_at, hs_at, bytes;
};

inline FewLayout few_layout(int T, int E, int top_k, int H, int I, bool int4) {
    auto up = [](int64_t v) { return (v + 255) / 256 * 256; };
    const int ncol = int4 ? 64 : 32;  // columns of a panel
    const int panels = (H + ncol - 1) / ncol;
    const int most = T * top_k < E ? T * top_k : E;
    int splits = (kFewDownGrid + panels - 1) / panels;
    splits = splits < most ? splits : most;
    splits = splits < kFewMaxSplits ? splits : kFewMaxSplits;
    FewLayout l;
    l.splits = splits < 1 ? 1 : splits;
    l.part_at = kFewCounterBytes;
    l.hs_at = l.part_at + up(l.splits > 1 ? static_cast<int64_t>(panels) * l.splits * T * ncol * 4 : 0);
    l.bytes = l.hs_at + up(static_cast<int64_t>(T) * top_k * I * 4);
    return l;
}

// kind: the moe_wtype of the weights; group: int4 only
hipError_t launch_few_tokens(int kind, const FewArgs& a, hipStream_t s);

}  // namespace moe
