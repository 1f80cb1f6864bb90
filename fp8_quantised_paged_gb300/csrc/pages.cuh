// pages.cuh -- what the page operators (pages.cu) share with their host side.
#pragma once

#include "internal.h"

namespace fp8pa {

// The arrays of a cache that a launch copies in, by value: more arrays take more
// launches.
constexpr int kMaxArrays = 128;
struct PageArrays {
  int n;
  uint8_t* ptr[kMaxArrays];
  uint32_t page_bytes[kMaxArrays];  // multiples of 16
  uint32_t first[kMaxArrays + 1];   // chunks of a page before an array's (prefix sum)
};

// Rows of block tables and their pages.
struct PageRows {
  int32_t* tables;
  int32_t* lens;
  int32_t* refs;
  int max_blocks, rows, num_blocks, bs;
  uint32_t* err;
};

cudaError_t launch_keep_accepted(const int32_t* accepted, int max_accepted,
                                 const int32_t* q_offsets, const PageRows& r, void* const* pages,
                                 const long long* page_bytes, int arrays, int hkv,
                                 int32_t* new_lens, cudaStream_t stream);
cudaError_t launch_fork(const int32_t* src, const int32_t* dst, int forks, const PageRows& r,
                        void* const* pages, const long long* page_bytes, int arrays,
                        int32_t* workspace, cudaStream_t stream);
cudaError_t launch_resize(const int32_t* new_lens, const PageRows& r, int32_t* workspace,
                          cudaStream_t stream);
cudaError_t launch_compact(const PageRows& r, void* const* pages, const long long* page_bytes,
                           int arrays, int32_t* page_map, int32_t* workspace,
                           cudaStream_t stream);
// Words of workspace for any of them.
inline size_t pages_workspace_words(int rows, int num_blocks) {
  return 3 * static_cast<size_t>(rows) + static_cast<size_t>(num_blocks) + 8;
}

}  // namespace fp8pa
