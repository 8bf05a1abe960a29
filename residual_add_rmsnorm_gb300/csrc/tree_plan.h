// tree_plan.h -- which kernel an attention call gets and the workspace it
// needs: host arithmetic on sizes alone (lengths live on the device).
#pragma once

#include <stdint.h>

namespace rarn {
namespace tree {

constexpr int kBoxSlots = 8;

struct Plan {
    int rows;          // rows (drafted token x query head of the group) of a segment
    bool tiles;        // the tensor-memory kernel (tree_tile.cuh)
    int64_t segments;  // at most
    int64_t expected;  // segments where all sequences draft alike
    int64_t joins_off, ml_off, part_off, bytes;
};

inline bool dim_ok(int64_t D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

// tokens drafted tokens in all, of B sequences; boxes: the pages are made of
// whole groups of eight slots, which the tensor-memory kernel copies.
inline Plan plan(int64_t tokens, int64_t B, int64_t Hq, int64_t Hk, int64_t D, bool boxes) {
    Plan p{};
    const int64_t G = Hq / Hk;
    const int64_t per = ((tokens + B - 1) / B) * G;  // rows of an average sequence
    p.tiles = boxes && (D == 64 || D == 128) && per > 16;
    p.rows = p.tiles ? (per > 128 ? 256 : 128) : per > 8 && D <= 128 ? 16 : 8;
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
