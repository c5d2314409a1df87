// AdamW over a list of tensors: table records and launchers (adamw.cu).
#pragma once

#include "tensor_list.cuh"

namespace dash {

// One tensor of the list (tensors without elements are left out).
struct AdamwTensorDev {
  void* param;
  const void* grad;
  void* m;           // fp32 moments, or 8-bit codes
  void* v;
  uint8_t* m_scale;  // 8-bit: one scale for each block
  uint8_t* v_scale;
  void* copy;        // fp32 parameters may have a 16-bit copy written beside them, or null
  long long n;
  int first;         // first block, counted over the list; kQBlock times it is its place in the flat moments
  int first_tile;    // first tile of kTile elements, likewise counted
  int flags;
  int index;         // in the caller's list
  float lr_scale, decay;
  int pad[2];
};
static_assert(sizeof(AdamwTensorDev) == 96, "six 16-byte words");

constexpr int kParamShift = 0, kGradShift = 4, kCopyShift = 8;  // element types in AdamwTensorDev::flags
constexpr int kFlagEight = 1 << 12;                             // 8-bit moments
constexpr int kFlagVec = 1 << 13;                               // every array but the scales is on a 16-byte boundary
constexpr int kFlagWide = 1 << 14;  // and written fp32 on a 32-byte one, scales on a 4-byte one: tiles can be staged

// Elements that the step takes at a time: 16 blocks, a scale of m and of v for
// each lane of a warp.
constexpr int kTileBlocks = 16;
constexpr int kTile = kTileBlocks * kQBlock;

// The list on the device: 'first_tile' of each tensor; the records.
struct AdamwTable {
  const int* first_tile;
  const AdamwTensorDev* tensors;
  int n_tensors, n_tiles;
};

// Start of the workspace: the status word, the blocks' arrival count, and the
// step counter with what the next step's bias corrections need.
struct AdamwHeader {
  unsigned status;
  unsigned ticket;
  unsigned bad;          // status bits of the running step
  unsigned next;         // shares taken in the running step, beyond the first of each block
  int t;                 // last step taken
  double pow1, pow2;     // beta1^t, beta2^t
  float d1, d0;          // for step t + 1, see AdamwArgs
};

struct AdamwArgs {
  // beta, and 1 - beta, as pairs of one value: operands of the packed products, read from the constant bank
  float2 beta1, om1, beta2, om2;
  float2 one;            // 1, not known as such when the kernel is compiled
  float eps;
  unsigned seed_lo, seed_hi;
  int withhold;          // test hook: tiles are announced and not copied, so that the waits for them run out
  int step;              // > 0: take this step number and the values below; 0: the header's next
  // m_hat / (sqrt(v_hat) + eps) = m / (d1 sqrt(v) + d0): d1 = (1 - beta1^t) / sqrt(1 - beta2^t),
  // d0 = eps (1 - beta1^t)
  float d1, d0;
  double pow1, pow2;
  float lr;
  const float* lr_device;  // null: lr
  const float* coef;       // null: 1
};

// How the step is launched on the current device: blocks that fill it, and
// their shared memory.
struct AdamwLaunch {
  int step;
  int direct;                // lists of up to so many tiles go without the ring
  int bits;                  // 32, 8, or 0 for both
  int stages, stride, smem;
};
int adamw_stage_bytes(bool eight, int param_dtype, int grad_dtype);
// stage_bytes: the largest adamw_stage_bytes of the list.  Returns a SHAMPOO_* code.
int adamw_prepare(int bits, int stage_bytes, AdamwLaunch* out);
void launch_adamw(const AdamwTable& t, const AdamwLaunch& l, int grid, AdamwHeader* hdr, const AdamwArgs& a,
                  cudaStream_t st);
void launch_load_moments(const AdamwTable& t, AdamwHeader* hdr, const float* m, const float* v, cudaStream_t st);
void launch_read_moments(const AdamwTable& t, void* m, void* v, int dtype, cudaStream_t st);

}  // namespace dash
