// workspace.cuh -- where the parts of a call's workspace lie.
//
// A workspace serves calls of any entry point and any sizes in turn and is never cleared. What must outlast a call in
// it is the epoch word alone: a graph replays its captured call tag, and the word, which every captured call
// of split counters advances, tells the replays apart. So every layout keeps the first kWsHead bytes for it and
// puts nothing else there; no call's partials or plan can put an older word back.
#pragma once
#include <algorithm>
#include <cstddef>

#include "common.cuh"
#include "plan.cuh"

namespace pgqa {

constexpr size_t kWsEpochOff = 0;  // the epoch word, in every layout
constexpr size_t kWsHead = 256;    // the parts begin here

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct ClassSizes {
  int num_ctas, max_blocks, max_items, max_slots, slot_rows;
};

// The paged calls (dense, 4-bit, tree).
struct WsLayout {
  ClassSizes cls[kNumClasses];
  size_t off[kNumClasses][8];
  size_t q_amax_off;  // per-CTA maxima of |q| (calls that quantise Q)
  size_t total;
};

inline WsLayout make_layout(int num_seqs, int T, int Hq, int Hkv, int sms) {
  WsLayout L{};
  const long long G = Hq / Hkv;
  const long long rows_all = (long long)T * G;
  // verify blocks: one per (sequence, kv head); prefill blocks: 128-row blocks
  const long long vb = (long long)num_seqs * Hkv;
  // a prefill block needs some sequence with q_len*G > 64, so none exist if T*G <= 64
  const long long pb =
      rows_all > kVerifyRows ? (long long)Hkv * ((rows_all + kPrefillRows - 1) / kPrefillRows + num_seqs) : 0;
  const long long nb[2] = {vb, pb};
  const int rows[2] = {kVerifyRows, kPrefillRows};
  size_t at = kWsHead;
  for (int c = 0; c < kNumClasses; ++c) {
    ClassSizes& s = L.cls[c];
    s.num_ctas = sms;
    s.max_blocks = (int)std::max<long long>(1, nb[c]);
    s.max_items = s.max_blocks + s.num_ctas;
    // Split pieces take slots by split_slot_base: below 2 per CTA.
    s.max_slots = nb[c] == 0 ? 0 : 2 * s.num_ctas;
    s.slot_rows = rows[c];
    size_t sz[8] = {
        256,                                                          // n_blocks, n_items, total_tiles
        sizeof(int) * (size_t)(s.num_ctas + 1),                       // cta_item_begin
        sizeof(RowBlock) * (size_t)s.max_blocks,                      // blocks
        sizeof(WorkItem) * (size_t)s.max_items,                       // items
        sizeof(unsigned long long) * (size_t)s.max_blocks,            // counters
        sizeof(uint16_t) * (size_t)s.max_slots * s.slot_rows * kHeadDim, // part_o (f16)
        sizeof(float) * (size_t)s.max_slots * s.slot_rows,            // part_lse
        0};
    for (int i = 0; i < 8; ++i) {
      L.off[c][i] = at;
      at += align256(sz[i]);
    }
  }
  L.q_amax_off = at;
  at += align256(sizeof(float) * (size_t)q_amax_parts(sms));
  L.total = at;
  return L;
}

// The prompt attention on `clusters` pairs of CTAs (PromptScratch).
struct PromptLayout {
  size_t part_o, part_lse, counters, total;
};

inline PromptLayout prompt_layout(int clusters) {
  const size_t slots = 4 * (size_t)clusters;
  PromptLayout L;
  L.part_o = kWsHead;
  L.part_lse = L.part_o + align256(slots * kSlotRows * kHeadDim * sizeof(float));
  L.counters = L.part_lse + align256(slots * kSlotRows * sizeof(float));
  L.total = L.counters + align256(slots * sizeof(unsigned long long));
  return L;
}

}  // namespace pgqa
