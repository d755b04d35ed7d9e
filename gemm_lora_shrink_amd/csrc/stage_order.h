// The order in which the attention kernels over a quantized cache find, bring and
// read stages of keys.  Between two barriers waves run in any order, so what one
// writes in such a phase must not be what another reads in it.
//
// The kernel with turns: step t of the first group of waves is the phases 2 t
// (products) and 2 t + 1 (softmax of stage t), of the second group one phase later.
// Every wave looks up its own rows of stages 4 k + 4 .. 4 k + 7 in step 4 k + kTurnsFind
// and settles their factors in step 4 k + kTurnsSettle, in the phase of the products
// (short heads) or of the softmax.  With short heads the first group thus finds those
// stages in phase 8 k, in which the second one is at the softmax of stage 4 k - 1: as
// many stages before 4 k + 7 as a ring of 8 holds, hence 16 places for what find()
// writes.  What settle() writes comes two phases later, and 8 places do.
//
// The wide kernel: one phase a tile of 32 keys.
#pragma once

namespace lora {

constexpr int kValidRing = 16;   // stages of which it is held which rows are keys
constexpr int kFactorRing = 8;   // stages whose factors are held
constexpr int kTurnsRing = 4;    // stages in LDS, kernel with turns
constexpr int kTurnsFind = 0, kTurnsSettle = 1, kTurnsAsk = 2;  // of four steps
constexpr int kWideRing = 2;     // stages in LDS, wide kernel
constexpr int kWideFind = 1, kWideSettle = 2, kWideAsk = 3;

}  // namespace lora
