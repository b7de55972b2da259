// How attention calls are cut into workgroups and what their workspaces hold:
// host code, and the sizes that it shares with the kernels.
#pragma once

#include "qmv_kv.h"

namespace qmv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kBias = 11.f, kSlack = 4.f;  // the kernels' probabilities (qmv_attn.h)

constexpr int kBM = 128, kBK = 64;  // prompts: rows a workgroup takes, positions a chunk
// Decode: positions a wave takes at a time (16 KB at 128 columns).
constexpr int decode_chunk(int type) { return type == kKvI8 ? 64 : 32; }
constexpr int kMaxPieces = 512;  // pieces of an output row that the join takes

// Workgroups of four waves and 16-row tiles that the registers of a compute
// unit hold at once (256 columns take more than half of them).
constexpr int resident(int type, int hd) { return hd == 256 ? 1 : hd == 64 && type != kKvI8 ? 3 : 2; }

// Whether the 256 registers that eight waves leave each lane hold the kernel's
// operands; four waves have 512.
constexpr bool eight_fit(int type, int hd, int rt) {
    return rt == 1 ? hd <= 128 : hd == 64 || (hd == 96 && type == kKvF16);
}

// How a call is cut: 16-row operand tiles per wave, row tiles per key-value
// head, pieces of the cache's length (as in AttnArgs), slots for the pieces of
// a decode call, waves per workgroup; workspace offsets in bytes.
struct AttnPlan {
    int rt, tiles, splits, parts, slots, waves;
    int64_t part_rows;
    int64_t ld_logits;
    size_t ml_off, o_off, share_off, logits_off, bytes;
};
AttnPlan attn_decode_plan(int type, int hd, int64_t n_seq, int n_kv, int group, int n,
                          int64_t max_len, int window, int sinks, bool with_acc);
AttnPlan attn_prefill_plan(int type, int hd, int64_t n_seq, int n_kv, int group, int64_t rows,
                           int64_t max_len, int window, int sinks);

}  // namespace qmv
