// Arguments of the caches' reordering (kv_reorder.cu).
#pragma once

#include "common.cuh"

namespace tfl {

struct ReorderArgs {
    int n, n_kv, layers;
    int lo, hi;                // all ranges lie in [lo, hi)
    int run;                   // positions of a CTA, set by the launch
    const int* parents;        // device, n
    int first;                 // the number that parents have for cache 0
    int begin[kMaxStreams], end[kMaxStreams];
    KvView kv[kMaxStreams];
};
cudaError_t launch_kv_reorder(ReorderArgs a, int sms, cudaStream_t st, bool pdl);

}  // namespace tfl
