// Which scale groups of a weight row a run of its k touches (host and device).
#pragma once

namespace nvfp4 {

struct I4Groups {
  int first, count;
};

// Groups of k0, ..., k0 + span - 1, as far as they lie below K; 0 <= k0 < K.  K and
// group go to 2^30, so no sum here may pass K: k0 + span + group would not fit an int.
constexpr I4Groups i4_groups(int k0, int span, int K, int group) {
  const int k1 = span < K - k0 ? k0 + span : K;
  return I4Groups{k0 / group, (k1 - 1) / group + 1 - k0 / group};
}

}  // namespace nvfp4
