// The device image of a list of tensors for the multi-tensor AdamW step.
#pragma once

#include <stdint.h>

namespace qlin {

// Elements that one scale of an 8-bit moment covers, and elements of a chunk
// (the work of one workgroup).
constexpr int kStateBlock = 256;
constexpr int kTensorChunk = 4096;

constexpr uint32_t kParamBf16 = 1, kGradBf16 = 2, kState8 = 4;

// One tensor of the image; the image is `count` of these, then one int32 per
// chunk: the tensor that the chunk belongs to.
struct TensorEntry {
    void *p;
    const void *g;
    void *m, *v;
    float *ms, *vs;
    int64_t numel;
    int64_t index0;         // index of the first element for the rounding's uniforms
    int64_t chunk0;         // first chunk of the tensor
    float weight_decay;
    uint32_t flags;
};
static_assert(sizeof(TensorEntry) == 80, "layout of the tensor image");

} // namespace qlin
