// Calls with few token slots, one workgroup column per slot: a slot's expert picked
// from the router's logits where it is needed.
#pragma once

#include "device_common.h"
#include "launch.h"
#include "route_key.h"
#include "wave_reduce.h"

namespace moe {
namespace {

// The decision of a call in slots: logits in; ids, weights and the identity
// permutation out (gate_up), ids in (down).
struct Slots {
  const double* logits;   // [T][E]
  int32_t* ids;           // [T][k]
  float* w;               // [T][k]
  int32_t* pos;           // [T k]
  int k;
};

// The picks of one token, best first (float32 logit descending, index
// ascending), up to and with pick `last`; wl takes their float64 logits.
__device__ __forceinline__ void pick_experts(const double* __restrict__ logits, int E, int last, int lane,
                                             int (&sel)[MOE_MAX_K_DEV], double (&wl)[MOE_MAX_K_DEV]) {
  constexpr int kPer = MOE_MAX_E_DEV / kWave;
  double l[kPer];
  uint64_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + kWave * i;
    l[i] = e < E ? logits[e] : 0.0;
    key[i] = e < E ? make_key((float)l[i], e) : 0;
  }
#pragma unroll
  for (int j = 0; j < MOE_MAX_K_DEV; ++j) {
    if (j > last) break;
    uint64_t best = key[0];
#pragma unroll
    for (int i = 1; i < kPer; ++i) best = key[i] > best ? key[i] : best;
    sel[j] = key_expert(wave_max(best));
    double mine = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + kWave * i == sel[j]) {
        key[i] = 0;
        mine = l[i];
      }
    wl[j] = lane_f64(mine, __builtin_amdgcn_readfirstlane(sel[j] % kWave));
  }
}

// The expert of pick j of token t (every lane of the wave gets it).
__device__ __forceinline__ int slot_expert(const Slots& slots, int t, int j, int E, int lane) {
  int sel[MOE_MAX_K_DEV], e = 0;
  double wl[MOE_MAX_K_DEV];
  pick_experts(slots.logits + (size_t)t * E, E, j, lane, sel, wl);
#pragma unroll
  for (int i = 0; i < MOE_MAX_K_DEV; ++i)
    if (i == j) e = __builtin_amdgcn_readfirstlane(sel[i]);
  return e;
}

// One wave writes token t's picks, their weights and the identity permutation: lane
// i < k takes pick i; softmax over the picks in float64, summed in order.
__device__ __forceinline__ void write_decision(const Slots& slots, int t, int E, int lane) {
  int sel[MOE_MAX_K_DEV];
  double wl[MOE_MAX_K_DEV];
  pick_experts(slots.logits + (size_t)t * E, E, slots.k - 1, lane, sel, wl);
  int my = sel[0];
  double myl = wl[0];
#pragma unroll
  for (int i = 1; i < MOE_MAX_K_DEV; ++i)
    if (i < slots.k && lane == i) my = sel[i], myl = wl[i];
  const double z = lane < slots.k ? exp(myl - wl[0]) : 0.0;
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < MOE_MAX_K_DEV; ++i) sum += lane_f64(z, i);
  if (lane < slots.k) {
    const int slot = t * slots.k + lane;
    slots.ids[slot] = my;
    slots.w[slot] = (float)(z / sum);
    slots.pos[slot] = slot;
  }
}

}  // namespace
}  // namespace moe
