// What a clipping plan holds (clip_grad.cu, capi.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

namespace swin {

// Consecutive elements of one tensor, for one block.
struct alignas(32) ClipPiece {
  const void* in;
  void* out;
  int len, bf16, pad0, pad1;
};
struct ClipShape {
  uint32_t pieces, keep_from;  // pieces from keep_from on are left in L2 for the second launch
  bool in_place;               // all of them
};

void clip_pieces(const void* const* in, void* const* out, const int64_t* sizes, const int* dtypes, int count,
                 std::vector<ClipPiece>* list, ClipShape* shape);
size_t clip_piece_count(const int64_t* sizes, int count);
size_t clip_workspace_bytes();
int clip_launches(const ClipShape& s);
cudaError_t clip_launch(const ClipPiece* list, const ClipShape& s, float max_norm, float scale, float eps, float* norm,
                        void* workspace, cudaStream_t st);

}  // namespace swin
