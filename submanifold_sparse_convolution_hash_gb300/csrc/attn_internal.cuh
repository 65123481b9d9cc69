// Declarations shared by the attention kernels (attn.cu, attn_fwd.cu,
// attn_bwd.cu).
//
// Packed rows.  The G = heads_q / heads_kv query heads that read one key head
// are rows of one matrix: row r of a sequence is query r / G, head r % G of the
// group.  A 128-row tile holds P = 128 / G queries (P * G rows, the rest is
// padding), so a group shares every key and value it reads, and a sum over the
// rows is already the sum over the heads.
#pragma once

#include "sc_internal.cuh"
#include "tma_map.cuh"

namespace sc {

constexpr int kKeyTile = 128;

// One piece of work, for every key head.
struct __align__(16) AttnItem {
  int q_row;   // first query of the item (its row in q); gk, gv: of the sequence
  int n_pos;   // queries of the item; gk, gv: of the sequence
  int lim0;    // with a causal mask the item's query i sees keys j <= lim0 + i
  int k_row;   // the sequence's first key row
  int lk;      // its keys
  int kt0, kt1;  // key tiles [kt0, kt1); gk, gv: kt0 is the item's key tile
  int slot;    // first of its partial results, or -1: it writes the result itself
  int split, nsplit;  // which of how many parts of the keys
  int dual;    // one row tile: both halves of the block work on it, on every other key tile
  int seq;     // the item's sequence
};
static_assert(sizeof(AttnItem) == 48, "read as three 16-byte words");

// Written by k_attn_plan: [0] items, [1] next work unit, [2] joins, [3] rows of
// a partial result.
constexpr int kPlanHeader = 16;  // ints

enum PlanMode { kPlanRows = 0, kPlanKeys = 1 };

struct PlanArgs {
  const int *q_off, *k_off, *k_len;
  int n_seq;
  int64_t t_q, t_k;
  int pos_per_item;  // queries of an item (kPlanRows), of a row tile (kPlanKeys)
  int g;
  int causal;
  int packed_keys;   // the key lists have to cover every key row
  int heads_kv;
  int mode;
  int sms;
  int over;           // parts an SM that a short list is cut into
  int64_t part_rows;  // rows of partial results that fit; 0: the keys are never cut
  int min_tiles;      // least key tiles of a part
  int dual;           // items of one row tile may be worked on by both halves
  int cap, join_cap;  // items and joins that fit
  int* header;
  AttnItem* items;
  AttnItem* joins;    // per item that has parts: where its rows and parts are
  int* status;
};
// Two plans in one launch where b is given; `after`: it may overlap the kernel
// before it, which it then outlasts.
sc_status attn_plan(const PlanArgs& a, const PlanArgs* b, bool after, cudaStream_t s);
int* attn_status_word();

// Workspace pieces, 256-byte aligned.
struct Arena {
  size_t bytes = 0;
  size_t take(size_t n) {
    const size_t at = bytes;
    bytes += (n + 255) & ~size_t(255);
    return at;
  }
};

sc_status attn_map(CUtensorMap* m, const void* data, sc_dtype dt, int d, int heads, int64_t tokens, int64_t ts,
                   int64_t hs, int box_heads, int box_tokens);

}  // namespace sc
