// AdamW over a list of tensors: chunk records and launchers (adamw.cu).
#pragma once

#include "tensor_list.cuh"

namespace dash {

// One chunk of one tensor, all pointers at its first element.  Chunks start
// at multiples of kQBlock elements, so no block of 8-bit moments is split.
struct AdamwChunk {
  void* param;
  const void* grad;
  void* copy;        // fp32 parameters may have a 16-bit copy written beside them, or null
  void* m;           // fp32 moments, or 8-bit codes
  void* v;
  uint8_t* m_scale;  // 8-bit: one scale for each block
  uint8_t* v_scale;
  long long elem;    // first element's index in its tensor
  long long flat;    // and in the flat moments of the read and load calls
  int count;         // elements
  int flags;
  int tensor;        // index in the list
  float lr_scale, decay;
  int pad;
};
static_assert(sizeof(AdamwChunk) == 96, "six 16-byte words");

constexpr int kParamShift = 0, kGradShift = 4, kCopyShift = 8;  // element types in AdamwChunk::flags
constexpr int kFlagEight = 1 << 12;                             // 8-bit moments
constexpr int kFlagVec = 1 << 13;                               // every pointer allows eight-element accesses

// Start of the workspace: the status word, the blocks' arrival count, and the
// step counter with what the next step's bias corrections need.
struct AdamwHeader {
  unsigned status;
  unsigned ticket;
  unsigned bad;          // a non-finite value was met in the running step
  int t;                 // last step taken
  double pow1, pow2;     // beta1^t, beta2^t
  float c1, c2;          // for step t + 1: 1 / (1 - beta1^(t+1)), sqrt(1 / (1 - beta2^(t+1)))
};

struct AdamwArgs {
  float beta1, beta2, eps;
  unsigned seed_lo, seed_hi;
  int step;              // > 0: take this step number and the values below; 0: the header's next
  float c1, c2;
  double pow1, pow2;
  float lr;
  const float* lr_device;  // null: lr
  const float* coef;       // null: 1
};

int adamw_blocks(int which);  // resident blocks of the 0: 32-bit, 1: 8-bit, 2: mixed step, 3: load, 4: read kernel
void launch_adamw(const AdamwChunk* chunks, int n, int which, int grid, AdamwHeader* hdr, const AdamwArgs& a,
                  cudaStream_t st);
void launch_load_moments(const AdamwChunk* chunks, int n, int grid, AdamwHeader* hdr, const float* m, const float* v,
                         cudaStream_t st);
void launch_read_moments(const AdamwChunk* chunks, int n, int grid, void* m, void* v, int dtype, cudaStream_t st);

}  // namespace dash
