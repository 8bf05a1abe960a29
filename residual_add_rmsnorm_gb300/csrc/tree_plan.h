// tree_plan.h -- which kernel an attention call gets and the workspace it
// needs: host arithmetic on sizes alone (lengths live on the device).
#pragma once

#include <stdint.h>

namespace rarn {
namespace tree {

constexpr int kBoxSlots = 8;  // pages of whole groups of these are copied by k_tree_tile

// Whether k_tree_rows copies by TMA where pages and scales allow it
// (Params::whole_steps): rows of 64 or 128 bytes.
constexpr bool rows_by_tma(int64_t D) { return D == 64 || D % 128 == 0; }

struct Plan {
    int rows;          // rows (drafted token x query head of the group) of a segment
    bool tiles;        // the tensor-memory kernel (tree_tile.cuh)
    int64_t segments;  // at most
    int64_t expected;  // segments where all sequences draft alike
    int64_t joins_off, ml_off, part_off, bytes;
};

inline bool dim_ok(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

// tokens drafted tokens in all, of B sequences; boxes: the pages are made of
// whole groups of kBoxSlots slots.
//
// k_tree_rows reads a segment's keys once for each 16 rows, k_tree_tile once for
// all, but spends about 10 us where a CTA's segment begins and ends.  With few
// segments, each CTA has a part of one, and the tiles win as soon as rows fill
// more than a block of 16; where CTAs have ends of several, from about 33 rows
// on (us, rows against tiles; 8 key heads of 128, bfloat16 queries, average
// rows and keys):
//   1 sequence of 32768    16 rows  34 / 44      24 rows   50 / 45
//   1 sequence of 65536    32 rows  86 / 67      48 rows  121 / 68
//   16 sequences of 2100   24 rows  55 / 58      28 rows   59 / 58     36 rows  68 / 58
//   64 sequences of 590    32 rows  86 / 105     36 rows   95 / 106    44 rows 113 / 106
//   (binary16 queries, e5m2, 16 of 2100: 28 rows 66 / 65, 36 rows 74 / 65; heads
//   of 64: 24 rows 39 / 50, 36 rows 51 / 50, 48 rows 62 / 51)
// Tiles of 256 rows against two blocks of 128: 16 sequences of 2100, 140 rows,
// 74 / 115.  Blocks of 16 rows against two of 8, with half the CTAs on an SM: 16
// sequences of 2100, 12 rows, 37 / 35; 1 of 65536, 32 rows, 85 / 103; 64 of
// 590, 24 rows, 74 / 70.  Heads of 192, whose 16 rows fill the registers: 16
// sequences of 2100, 24 rows, 73 / 72, 36 rows 90 / 97, 96 rows 198 / 231; 1 of
// 32768, 24 rows, 64 / 60, 48 rows 88 / 105.  Heads of 256 leave no room.
inline Plan plan(int64_t tokens, int64_t B, int64_t Hq, int64_t Hk, int64_t D, bool boxes) {
    Plan p{};
    const int64_t G = Hq / Hk;
    const int64_t per = ((tokens + B - 1) / B) * G;  // rows of an average sequence
    p.tiles = boxes && (D == 64 || D == 128) && per > (2 * B * Hk >= 160 ? 32 : 16);
    const bool sixteen = D <= 128 ? per > 8 : D <= 192 && per > 32;
    p.rows = p.tiles ? (per > 128 ? 256 : 128) : sixteen ? 16 : 8;
    const int64_t ctas = p.tiles ? 160 : 608;
    // every sequence ends in at most one block that is not full
    p.segments = Hk * (tokens * G / p.rows + B);
    p.expected = Hk * B * ((per + p.rows - 1) / p.rows);
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    p.joins_off = 256;
    p.ml_off = p.joins_off + up(32 * p.segments);
    p.part_off = p.ml_off + up(2 * ctas * p.rows * 8);
    p.bytes = p.part_off + 2 * ctas * p.rows * D * 4;
    return p;
}

}  // namespace tree
}  // namespace rarn
