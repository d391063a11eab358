// Shared memory of the few tokens' down kernel (few.hip), in host code by itself,
// so that every size can be walked without a GPU.
#pragma once
#include <stddef.h>

namespace nvfp4 {

constexpr int kDownWaves = 8, kDownPitch = 36, kDownStages = 5;
constexpr size_t kLdsBytes = 160 * 1024;                  // of a CU
constexpr size_t kFoundBytes = 1040;                      // the experts found: 1028, and the dynamic part starts on 16
constexpr size_t kRingBytes = (size_t)kDownWaves * 2048;  // a stage's tokens, eight for each wave

// Whether up to eight tokens of an expert go through LDS, and the bytes asked for
// at the launch: sums [waves][T][pitch] and weights [T][k] of float, ids [T][k] of
// int16, in whole runs of 16.
struct FewDownLds {
  bool ring;
  size_t bytes;
};
constexpr FewDownLds few_down_lds(int T, int k) {
  const size_t bytes = ((size_t)kDownWaves * T * kDownPitch * 4 + (size_t)T * k * 6 + 15) / 16 * 16;
  return {bytes + kDownStages * kRingBytes + kFoundBytes <= kLdsBytes, bytes};
}

}  // namespace nvfp4
