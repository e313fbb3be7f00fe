// dg_few_plan.h — how a launch of the few-token products' stream kernel (dg_few.cu) is laid out. Host code without CUDA.
#pragma once

#include <cstddef>

namespace dg {

// An SM's shared memory, of which each CTA takes 1 KB for itself, and the SMs of the whole GPU that these kernels are for (the layout,
// and with it the order of every sum, is that of the whole GPU whatever dg_set_num_sms says).
constexpr size_t kFewSmem = (size_t)227 << 10, kFewSmemOfCta = 1 << 10;
constexpr int kFewSms = 152;

constexpr int kUnitBytes = 128;   // of a unit's rows
// A stage of the ring holds a unit of R tiles of 16 rows: codes, then scales (E2M1: 16 bytes a row; E4M3: one or two words).
constexpr int stage_bytes(int R) { return 16 * R * (kUnitBytes + 16); }
// The tables of a pass with so many (token, choice) pairs (Routing in dg_few.cu).
constexpr size_t routing_bytes(int E, int pairs) { return ((size_t)E * 8 + (size_t)pairs * 14 + 31) / 16 * 16; }
// Tiles of eight columns that a call's passes have.
constexpr int few_tiles(int T) { return T <= 8 ? 1 : T <= 16 ? 2 : 4; }

// Warps a CTA, CTAs an SM, stages of a warp's ring.
struct FewPlan {
  int warps, ctas, stages;
  size_t smem;
  double cost;
};
constexpr int few_most_warps(int R) { return R == 2 ? 12 : 16; }
inline size_t few_smem(int warps, int stages, int NT, int R, size_t routing) {
  return (size_t)warps * (stages * stage_bytes(R) + 2 * R * NT * 128 * sizeof(float)) + routing;
}
// The most stages that so many CTAs leave room for: at least three, or two where there is one CTA; 0 where they do not fit.
inline int few_stages(int warps, int ctas, int NT, int R, size_t routing) {
  for (int s = 4; s >= (ctas == 1 ? 2 : 3); --s)
    if (ctas * (few_smem(warps, s, NT, R, routing) + kFewSmemOfCta) <= kFewSmem) return s;
  return 0;
}

// Sixteen warps fill an SM, twelve on units of two tiles (whose stages are twice as large; 16 x 2 stages, 14 x 3 and 8 x 4 take 5% longer
// than 12 x 3 for one token through 8 of 32 experts of 7168x2048, E4M3). Fewer warps do not take their steps faster, so the layout is the
// one with the least rounds of items x turns of a warp, and 0.3 for the item's own steps (without: 63.4 us for 61 there, 162 for 153 with 4
// tokens), of those that fit: with CTAs taken off afterwards instead, SMs ran on half of their warps with 17 tokens and more (32 tokens
// through 8 of 64 experts of 7168x2048 677 us for 551, 24 through 8 of 32 424 for 343). At least four warps a CTA: 16 tokens through 64
// experts take 415 us with two and 325 with four. Of one CTA with two stages some number of warps always fits.
inline FewPlan few_plan(long long items, int units, int NT, int R, size_t routing, bool capped) {
  const int most = few_most_warps(R);
  FewPlan p{};
  p.cost = 1e300;
  for (int w = most; w >= 4; --w) {
    for (int c = 1; c * w <= most; ++c) {
      if (few_stages(w, c, NT, R, routing) == 0) continue;
      const double rounds = (double)((items + (long long)kFewSms * c - 1) / ((long long)kFewSms * c));
      const double cost = rounds * ((units + w - 1) / w + 0.3) * most;
      if (cost < p.cost * (1.0 - 1e-9)) p.cost = cost, p.warps = w, p.ctas = c;
    }
  }
  if (capped) p.ctas = 1;
  p.stages = few_stages(p.warps, p.ctas, NT, R, routing);
  p.smem = few_smem(p.warps, p.stages, NT, R, routing);
  return p;
}

// The unit's tiles of rows and the layout of a call's product.
// rows: of weights, over all experts that can be active (kStreamDown: of one); units: of an item along its contraction.
// Units of two tiles (32 rows) share the tokens' operands and the steps between them and cost about 1.5 of one tile (us, two and one: one
// token through 8 of 32 experts of 7168x2048 59 and 65, 16 tokens through 8 of 64 320 and 399, 32 such 551 and 638; where rows are too few
// for it, 32 tokens through 8 of 256 of 2048x512 148 and 125; four-bit weights, 2 tokens through 8 of 32 experts of 7168x2048 68 and 82, 16
// tokens 212 and 234; of 26 sizes the rule's side is the faster one or within 2% of it in 24, 3% of 3 us and of 23 in the others). Not E2M1
// weights whose rows are no whole units (5 tokens through 16 experts of 2080x1408 25.5 and 24.3) or with four column tiles, which leave no
// registers for them (404 and 311).
struct FewChoice {
  int R;
  FewPlan plan;
};
constexpr bool few_two_tiles(int NT, bool four) { return NT <= 2 || !four; }   // whether there are such kernels
inline FewChoice few_choice(int T, int k, int E, int rows, int units, bool four, bool whole, bool capped) {
  const int NT = few_tiles(T);
  const size_t routing = routing_bytes(E, (T < 8 * NT ? T : 8 * NT) * k);
  const FewPlan one = few_plan((rows + 15) / 16, units, NT, 1, routing, capped);
  if (few_two_tiles(NT, four) && (!four || whole)) {
    const FewPlan two = few_plan((rows + 31) / 32, units, NT, 2, routing, capped);
    if (1.5 * two.cost <= 1.1 * one.cost) return {2, two};
  }
  return {1, one};
}

}  // namespace dg
