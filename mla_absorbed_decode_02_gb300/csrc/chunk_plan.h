// Planner of the chunk attention: ragged new tokens -> blocks of rows -> stretches of work for
// the units (CTA pairs).
//
// A block is up to 128 rows of the flattened [token][head] order of one sequence: 128 / H whole
// tokens, so with few heads several tokens share every key tile.  A block's tiles are 256 keys
// each, up to what its last token sees; a block that sees nothing keeps one (fully masked) tile,
// which writes its zero rows.  Blocks lie one after another on a line of cost positions
// (kChunkPieceCost, then kChunkTileCost per tile) and unit u owns the tiles in [u * budget, (u + 1) * budget):
// long sequences are split over units ("MLA inference: two computation paths and FlashMLA",
// section "Decode attention becomes a compute problem") and merged by their LSE.  Where there are
// no more blocks than units, a unit can take one share of one block instead -- a whole block, which
// needs no merging, or at most m tiles of one, m the least that the units suffice for -- and the
// plan is the one of the three whose longest unit costs least.
//
// Where there are more blocks than units they can be dealt instead, whole, in rounds of one for each unit: the
// sequences' blocks in order of their length, the longest first, and in a round the longest to the unit
// that has least.  Nothing is split or merged, and the blocks of a sequence, side by side in a round, read the same
// keys at the same time: in stretches they start at any of its tiles, and where the keys are more than L2 holds
// HBM brings them once for each.  So dealing is taken up to 5/4 of the stretches' cost (tiles and pieces):
// 50 sequences of 5 tokens x 128 heads over 8192 keys 370 against 441 us at 1.19 of the cost, 57 of 1..10
// over 400 to 8100 112 against 132 at 1.08, 39 of 6 over 8192 364 against 366 at 1.26, 16 of 10 266 against
// 251 at 1.37.  Keys that L2 holds anyway leave the pieces and the merge: 11/10.  Prompt pieces on 16 heads
// 124 against 130 us at 1.04, 12 of 10 over 2048 51 against 57 at 1.06; over 4096 101 against 97 at 1.15.
//
// The per-item functions are shared by the scheduler kernel (which runs the prefix sums in
// parallel) and the host twin.
#pragma once
#include <cstdint>
#include <vector>

#include "plan.h"

namespace mla {

constexpr int32_t kChunkMagic = 0x4D4C4143;  // "MLAC"
constexpr int kChunkHeader = 16;              // int32 header words
constexpr int kChunkBlockInts = 8;            // int32 words per block record
constexpr int kChunkUnitInts = 16;            // int32 words per unit record
constexpr int kChunkRows = 128;               // rows of a block (MMA M of a CTA pair)
constexpr int kChunkTile = 256;               // keys of a tile (four pages)
// Cost positions of a tile, and of a piece beyond its tiles (the query load, the epilogue, the
// pipeline's refill).
#ifndef MLA_CHUNK_TILE_COST
#define MLA_CHUNK_TILE_COST 4
#endif
#ifndef MLA_CHUNK_PIECE_COST
#define MLA_CHUNK_PIECE_COST 3
#endif
constexpr int kChunkTileCost = MLA_CHUNK_TILE_COST, kChunkPieceCost = MLA_CHUNK_PIECE_COST;
MLA_HD inline int32_t chunk_cost(int32_t nt) { return kChunkPieceCost + kChunkTileCost * nt; }
// What writing and merging the partial results of split blocks costs, in tiles.
#ifndef MLA_CHUNK_MERGE_COST
#define MLA_CHUNK_MERGE_COST 2
#endif
constexpr int kChunkMergeCost = MLA_CHUNK_MERGE_COST;
// Tiles of a share (of whole blocks: `longest`), or 0 for stretches of `budget` positions.  The walk
// over stretches needs a budget of at least a tile's cost.
MLA_HD inline int32_t chunk_share_tiles(int32_t longest, int32_t least, int64_t budget) {
  const int64_t merge = (int64_t)kChunkTileCost * kChunkMergeCost;
  const int64_t whole = chunk_cost(longest), share = chunk_cost(least) + merge;
  const int64_t stretch = budget >= kChunkTileCost ? budget + kChunkPieceCost + merge : INT64_MAX;
  if (whole <= share && whole <= stretch) return longest;
  return share <= stretch ? least : 0;
}

// The order of the blocks: by sequence, the longest first (with more blocks than units and no more sequences
// than this; each counts those before it).
constexpr int kChunkSortSeqs = 1024, kChunkDealUnits = 1024;
MLA_HD inline int32_t chunk_sort_key(int32_t n, int32_t len) { return n > 0 ? (len + kChunkTile - 1) / kChunkTile : -1; }
MLA_HD inline bool chunk_sorts_before(int32_t key_a, int a, int32_t key_b, int b) {
  return key_a > key_b || (key_a == key_b && a < b);
}
constexpr int kChunkNearPages = 896;  // 64 MB of rows: what either half of the L2 holds of its own
MLA_HD inline bool chunk_is_dealt(int64_t most, int64_t budget, int64_t pages) {
  const int64_t stretch = budget + kChunkPieceCost + (int64_t)kChunkTileCost * kChunkMergeCost;
  return most <= stretch + stretch / (pages > kChunkNearPages ? 4 : 10);
}

// header words
enum {
  kChMagic = 0, kChUnits, kChCapacity, kChBlocks, kChSlots, kChBudget, kChTokens, kChNumSplit, kChPages, kChShares, kChBatch,
  kChCausal, kChMaxTokens, kChHeads, kChMaxPages, kChKvPages
};

// What a plan was made for.  The kernels that use it compare all of it: every index they form is
// bounded by the plan's own limits, not by the lengths.
struct ChunkKey {
  int32_t units, capacity, batch, causal, max_tokens, heads, max_pages, kv_pages;
};
MLA_HD inline void chunk_write_key(int32_t* sched, const ChunkKey& k) {
  sched[kChUnits] = k.units;
  sched[kChCapacity] = k.capacity;
  sched[kChBatch] = k.batch;
  sched[kChCausal] = k.causal;
  sched[kChMaxTokens] = k.max_tokens;
  sched[kChHeads] = k.heads;
  sched[kChMaxPages] = k.max_pages;
  sched[kChKvPages] = k.kv_pages;
}

// Block record.
struct ChunkBlock {
  int32_t tok0;    // first token (row of q / H)
  int32_t ntok;    // tokens of this block
  int32_t seq;
  int32_t base;    // keys the first token sees under the causal rule, before clipping to [0, L]
  int32_t len;     // L of the sequence
  int32_t nt;      // tiles
  int32_t splits;  // units its tiles span
  int32_t offset;  // first partial slot (splits > 1)
};

struct ChunkLayout {
  int64_t units, blocks, split_list, page_off, blk_off, pos, total;  // int32 offsets into sched
};

MLA_HD inline int chunk_tokens_per_block(int H) { return H >= kChunkRows ? 1 : kChunkRows / H; }

// Blocks that max_tokens tokens in at most `batch` sequences can make.
MLA_HD inline int64_t chunk_block_capacity(int64_t max_tokens, int batch, int H) {
  const int tb = chunk_tokens_per_block(H);
  const int64_t partial = tb == 1 ? 0 : (batch < max_tokens ? batch : max_tokens);
  const int64_t cap = max_tokens / tb + partial;
  return cap < 1 ? 1 : cap;
}

MLA_HD inline ChunkLayout chunk_layout(int U, int64_t cap, int batch) {
  ChunkLayout l;
  l.units = kChunkHeader;
  l.blocks = l.units + (int64_t)kChunkUnitInts * U;
  l.split_list = l.blocks + kChunkBlockInts * cap;
  l.page_off = l.split_list + (int64_t)kChunkBlockInts * U;
  l.blk_off = l.page_off + batch + 1;
  l.pos = l.blk_off + batch + 1;
  l.total = l.pos + cap;
  return l;
}

// Keys token j of a block sees.
MLA_HD inline int32_t chunk_visible(const ChunkBlock& b, int j, int causal) {
  int32_t v = causal ? b.base + j : b.len;
  if (v > b.len) v = b.len;
  return v < 0 ? 0 : v;
}

// Lengths a plan accepts: new tokens in order within the buffer, rows within the block table.
MLA_HD inline bool chunk_sequence_ok(int32_t lo, int32_t hi, int32_t L, int64_t max_tokens, int max_pages) {
  return lo >= 0 && hi >= lo && hi <= max_tokens && L >= 0 && (int64_t)L <= (int64_t)max_pages * 64;
}

MLA_HD inline int32_t chunk_seq_blocks(int32_t n, int tb) { return (n + tb - 1) / tb; }

// Block `blk` of sequence `b`, whose blocks start at first_blk.
MLA_HD inline ChunkBlock chunk_make_block(const int32_t* cu, const int32_t* lens, int b, int blk, int first_blk, int tb,
                                          int causal) {
  ChunkBlock k;
  const int32_t n = cu[b + 1] - cu[b], i0 = (blk - first_blk) * tb;
  k.tok0 = cu[b] + i0;
  k.ntok = n - i0 < tb ? n - i0 : tb;
  k.seq = b;
  k.len = lens[b];
  k.base = k.len - n + i0 + 1;  // token i of n sees keys 0 .. L - n + i
  const int32_t nt = (chunk_visible(k, k.ntok - 1, causal) + kChunkTile - 1) / kChunkTile;
  k.nt = nt > 0 ? nt : 1;
  k.splits = k.offset = 0;
  return k;
}

// The sequence that holds block blk: the last b with blk_off[b] <= blk (sequences without new
// tokens hold none).
MLA_HD inline int chunk_find(const int32_t* off, int n, int32_t v) {
  int a = 0, b = n;
  while (b - a > 1) {
    const int m = (a + b) / 2;
    if (off[m] <= v) a = m; else b = m;
  }
  return a;
}

// Unit u's record {first block, first tile, last block, end tile, split index of the first piece, 0, 0, 0,
// the first block's record} (the kernels read what they need of the plan in one memory latency).
MLA_HD inline void chunk_unit(const ChunkBlock* blocks, const int32_t* pos, int NB, int64_t total, int64_t budget, int u,
                              int32_t* rec) {
  rec[0] = -1;
  for (int i = 1; i < kChunkUnitInts; ++i) rec[i] = 0;
  const int64_t lo = (int64_t)u * budget, hi = lo + budget;
  if (lo >= total || NB == 0) return;
  int a = 0, b = NB;  // first block whose last tile lies at or past lo
  while (a < b) {
    const int m = (a + b) / 2;
    if ((int64_t)pos[m] + chunk_cost(blocks[m].nt - 1) >= lo) b = m; else a = m + 1;
  }
  if (a >= NB) return;
  const int64_t first0 = (int64_t)pos[a] + kChunkPieceCost;
  if (first0 >= hi) return;  // the stretch holds overhead positions only
  int c = a, d = NB;  // last block whose first tile lies before hi
  while (d - c > 1) {
    const int m = (c + d) / 2;
    if ((int64_t)pos[m] + kChunkPieceCost < hi) c = m; else d = m;
  }
  int64_t end = (hi - ((int64_t)pos[c] + kChunkPieceCost) + kChunkTileCost - 1) / kChunkTileCost;
  if (end > blocks[c].nt) end = blocks[c].nt;
  rec[0] = a;
  rec[1] = (int32_t)(lo > first0 ? (lo - first0 + kChunkTileCost - 1) / kChunkTileCost : 0);
  rec[2] = c;
  rec[3] = (int32_t)end;
  rec[4] = (int32_t)(u - first0 / budget);
  *reinterpret_cast<ChunkBlock*>(rec + kUnitInts) = blocks[a];
}

// (The budget is at least a tile's cost -- with more blocks than units it always is -- so every unit between
// a block's first and its last holds some of its tiles.)
MLA_HD inline int32_t chunk_splits(int32_t pos, int32_t nt, int64_t budget) {
  const int64_t first = (int64_t)pos + kChunkPieceCost;
  return (int32_t)((first + kChunkTileCost * (int64_t)(nt - 1)) / budget - first / budget + 1);
}

// Shares of a block of nt tiles in shares of at most m tiles, made equal.
MLA_HD inline int32_t chunk_shares(int32_t nt, int32_t m) {
  const int32_t s = (nt + m - 1) / m, even = (nt + s - 1) / s;
  return (nt + even - 1) / even;
}

// Unit u's share: pos[k] = the shares before block k.
MLA_HD inline void chunk_share_unit(const ChunkBlock* blocks, const int32_t* pos, int NB, int64_t total, int u,
                                    int32_t* rec) {
  rec[0] = -1;
  for (int i = 1; i < kChunkUnitInts; ++i) rec[i] = 0;
  if (u >= total) return;
  const int k = chunk_find(pos, NB, u), i = u - pos[k];
  const int32_t nt = blocks[k].nt, s = blocks[k].splits, even = (nt + s - 1) / s;
  rec[0] = rec[2] = k;
  rec[1] = i * even;
  rec[3] = nt < (i + 1) * even ? nt : (i + 1) * even;
  rec[4] = i;
  *reinterpret_cast<ChunkBlock*>(rec + kUnitInts) = blocks[k];
}

// The record of a unit that was dealt the blocks [first, end).
MLA_HD inline void chunk_deal_unit(const ChunkBlock* blocks, int first, int end, int32_t* rec) {
  for (int i = 0; i < kChunkUnitInts; ++i) rec[i] = 0;
  rec[0] = first;
  rec[2] = end - 1;
  rec[3] = blocks[end - 1].nt;
  *reinterpret_cast<ChunkBlock*>(rec + kUnitInts) = blocks[first];
}

// Host twin: writes sched as the scheduler kernel does; false (and a header without the magic
// word) where the lengths are refused.
inline bool chunk_plan_host(const int32_t* cu, const int32_t* lens, int B, int64_t max_tokens, int H, int causal,
                            int max_pages, int64_t max_kv_pages, int U, int32_t* sched) {
  const int tb = chunk_tokens_per_block(H);
  const int64_t cap = chunk_block_capacity(max_tokens, B, H);
  const ChunkLayout l = chunk_layout(U, cap, B);
  for (int i = 0; i < kChunkHeader; ++i) sched[i] = 0;
  ChunkBlock* blocks = reinterpret_cast<ChunkBlock*>(sched + l.blocks);
  int32_t *page_off = sched + l.page_off, *blk_off = sched + l.blk_off, *pos = sched + l.pos;
  int64_t pages = 0, nb = 0;
  bool ok = cu[0] == 0;
  for (int b = 0; b < B && ok; ++b) {
    ok = chunk_sequence_ok(cu[b], cu[b + 1], lens[b], max_tokens, max_pages);
    page_off[b] = (int32_t)pages;
    blk_off[b] = (int32_t)nb;
    if (!ok) break;
    const int32_t n = cu[b + 1] - cu[b];
    nb += chunk_seq_blocks(n, tb);
    if (n > 0) pages += num_tiles(lens[b]);
    ok = pages <= max_kv_pages;
  }
  if (!ok) return false;
  page_off[B] = (int32_t)pages;
  blk_off[B] = (int32_t)nb;
  const bool sorted = nb > U && B <= kChunkSortSeqs;
  for (int b = 0; b < B; ++b) {
    const int32_t n = cu[b + 1] - cu[b], key = chunk_sort_key(n, lens[b]);
    int at = sorted ? 0 : blk_off[b];
    for (int o = 0; sorted && o < B; ++o)
      if (chunk_sorts_before(chunk_sort_key(cu[o + 1] - cu[o], lens[o]), o, key, b)) at += chunk_seq_blocks(cu[o + 1] - cu[o], tb);
    for (int i = 0; i < chunk_seq_blocks(n, tb); ++i) blocks[at + i] = chunk_make_block(cu, lens, b, i, 0, tb, causal);
  }
  int64_t total = 0;
  int32_t longest = 1;
  for (int k = 0; k < nb; ++k) {
    if (blocks[k].nt > longest) longest = blocks[k].nt;
    pos[k] = (int32_t)total;
    total += chunk_cost(blocks[k].nt);
  }
  if (total > kMaxPlanPositions) return false;
  bool shares = nb <= U;
  int64_t budget = plan_budget(total, U);
  if (shares) {
    int32_t lo = 1, hi = longest;  // the least m that U units suffice for
    while (lo < hi) {
      const int32_t m = (lo + hi) / 2;
      int64_t need = 0;
      for (int k = 0; k < nb; ++k) need += chunk_shares(blocks[k].nt, m);
      if (need <= U) hi = m; else lo = m + 1;
    }
    const int32_t m = chunk_share_tiles(longest, lo, budget);
    shares = m > 0;
    if (shares) budget = m;
  }
  bool dealt = false;
  std::vector<std::vector<ChunkBlock>> hand(sorted && U <= kChunkDealUnits ? U : 0);
  if (!hand.empty()) {
    std::vector<int64_t> load(U, 0);
    for (int64_t k0 = 0; k0 < nb; k0 += U) {
      const std::vector<int64_t> had = load;
      for (int u = 0; u < U; ++u) {
        int64_t k = k0;
        for (int v = 0; v < U; ++v) k += had[v] < had[u] || (had[v] == had[u] && v < u);
        if (k >= nb) continue;
        hand[u].push_back(blocks[k]);
        load[u] += chunk_cost(blocks[k].nt);
      }
    }
    int64_t most = 0;
    for (int64_t c : load) most = c > most ? c : most;
    dealt = chunk_is_dealt(most, budget, pages);
    if (dealt) {
      budget = most;
      int64_t k = 0;
      for (const auto& h : hand)
        for (const ChunkBlock& b : h) {
          pos[k] = k ? pos[k - 1] + chunk_cost(blocks[k - 1].nt) : 0;
          blocks[k++] = b;
        }
    }
  }
  int64_t at = 0;
  int32_t slots = 0, ns = 0;
  for (int k = 0; k < nb; ++k) {
    blocks[k].splits = dealt ? 1 : shares ? chunk_shares(blocks[k].nt, (int32_t)budget) : chunk_splits(pos[k], blocks[k].nt, budget);
    blocks[k].offset = slots;
    if (shares) pos[k] = (int32_t)at;
    at += blocks[k].splits;
    if (blocks[k].splits > 1) {
      slots += blocks[k].splits;
      reinterpret_cast<ChunkBlock*>(sched + l.split_list)[ns++] = blocks[k];
    }
  }
  int dealt_at = 0;
  for (int u = 0; u < U; ++u) {
    int32_t* rec = sched + l.units + kChunkUnitInts * u;
    if (dealt) {
      chunk_deal_unit(blocks, dealt_at, dealt_at + (int)hand[u].size(), rec);
      dealt_at += (int)hand[u].size();
    } else if (shares)
      chunk_share_unit(blocks, pos, (int)nb, at, u, rec);
    else
      chunk_unit(blocks, pos, (int)nb, total, budget, u, rec);
  }
  sched[kChMagic] = kChunkMagic;
  chunk_write_key(sched, {U, (int32_t)cap, B, causal, (int32_t)max_tokens, H, max_pages, (int32_t)max_kv_pages});
  sched[kChBlocks] = (int32_t)nb;
  sched[kChSlots] = slots;
  sched[kChBudget] = (int32_t)budget;
  sched[kChTokens] = tb;
  sched[kChNumSplit] = ns;
  sched[kChPages] = (int32_t)pages;
  sched[kChShares] = dealt ? 2 : shares;
  return true;
}

}  // namespace mla
