// paged_internal.h -- layout contract between the planner (paged_plan.cpp) and
// the kernels (paged_attn.cu) of the paged attention.  Not part of the public ABI.
#pragma once
#include <stdint.h>

#include "sarathi_internal.h"

namespace sarathi {
namespace paged {

constexpr int block_keys(int d) { return d == 128 ? 80 : 128; }  // keys of one K/V block of a tile item
constexpr int kItemWords = 8;      // int32 words of a work item
constexpr int kTokenWords = 4;     // per token: lo, hi, position, first page entry of its row
constexpr int kMergeWords = 8;
constexpr int kStreamWarps = 8;    // warps of a CTA that stream pages, each its own items
constexpr int kStreamMinPages = 4; // pages of a stream item that is cut off a longer one, at least, in a full plan
// Large stream items, of a warp's share (the sizes to choose from); the next ones.
constexpr double kStreamFirst[] = {0.7, 0.35, 0.42, 0.5, 0.6};
constexpr double kStreamRest = 0.3;
constexpr double kStreamUneven = 0.3;  // how much later than equal the last SM is with a large piece
constexpr int kStreamItemPages = 4;   // what an item costs beside its pages, in pages
constexpr double kStreamTaper = 0.3;  // a later one, of what is left of its row
constexpr int kTileMinBlocks = 2;  // blocks of a piece of a tile, at least
// Keys of a piece of a tile, at most: the rows of a piece that are done again one by
// one (32 a warp, 8 keys in 1.2 us with all SMs at it: 0.65 s) end within the kernel's
// waits.
constexpr int kTileMaxKeys = 1 << 17;

// A tile holds up to 128 query rows (token-major, q head of the group minor);
// a tile item up to two tiles of consecutive tokens.
inline int tile_tokens(int group) { return kTileRows / group; }

enum ItemKind : int32_t { kTile = 0, kStream = 1 };

// Work item, kItemWords int32 (32 bytes):
//   [0] kind
//   [1] g      kv head
//   [2] t0     first token
//   [3] nt     tokens (tile: up to 2 tile_tokens; stream: 1)
//   [4] kvp0   entry of the packed page list where the row's pages start
//   [5] kb     first key, a multiple of 16
//   [6] ke     end of the keys (kb = ke: no key; the outputs are zeros)
//   [7] part   first partial row, -1: the item writes out itself
enum ItemField { kKind = 0, kG, kT0, kNt, kKvp0, kKb, kKe, kPart };

// Merge record of a token whose work is split, kMergeWords int32: token, then
// for its two sources (the group's shared pages; its own pages) the pieces n, the
// first partial row base and the rows per (piece, kv head) step: q head c of kv
// head h has its partial of piece k in row base + (k H_kv + h) step + c.
enum MergeField { kMTok = 0, kMN0, kMBase0, kMStep0, kMN1, kMBase1, kMStep1 };

// Workspace: kHdrWords int32 -- [0], [1] the queues' heads, [2] error word, [3]
// its detail, [4] CTAs out -- then {max, sum} of each partial row (base-2
// logits), then the rows' fp32 sums [n_partials][d], from 256-byte boundaries.
constexpr int kHdrWords = 64;
enum HdrField { kHead0 = 0, kHead1 = 1, kError = 2, kDetail = 3, kOut = 4 };
inline int64_t ml_offset() { return kHdrWords * 4; }
inline int64_t o_offset(int64_t n_partials) { return ml_offset() + (n_partials * 8 + 255) / 256 * 256; }
inline int64_t workspace_size(int64_t n_partials, int d) { return o_offset(n_partials) + n_partials * d * 4; }

}  // namespace paged
}  // namespace sarathi
