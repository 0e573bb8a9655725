// The vocabulary's loss and its gradients for few tokens (vocab_few.cu), behind the
// entry points of vocab_loss.cu.
#pragma once
#include "ssm_common.cuh"

namespace gdn {

struct FewArgs {
    const void* h; int64_t ldh;
    const void* w; int64_t ldw;
    gdn_dtype dtype;
    const void* targets; int wide;
    int T, V, W;
    float scale;
};

// Whether a call is taken by these kernels: by its sizes and type alone, so that a forward and its
// backward agree
bool few_takes(int T, int V, int W, gdn_dtype dtype);

// Maxima and sums of exponentials of all words but the target, [few_blocks()][T], and the
// targets' logits [T]
int few_blocks(int T, int V);
gdn_status few_logits(const FewArgs& a, float2* stat, float* at, cudaStream_t s);

// Gradients: P [V][T] and dh's parts [few_parts()][T][W], both fp32, in the workspace; loss may be
// null
int few_parts(int T, int V, int W, gdn_dtype dtype);
gdn_status few_grads(const FewArgs& a, const float* dloss, const float* loss, const float* lse, float* P, float* parts,
                     void* dh, int64_t lddh, void* dw, int64_t lddw, cudaStream_t s);

}  // namespace gdn
