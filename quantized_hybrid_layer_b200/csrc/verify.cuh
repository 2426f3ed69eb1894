// Types shared by the operators that verify trees of drafted tokens over a
// paged KV cache (norm_rope.cu, tree_attention.cu, deltanet_tree.cu, pages.cu),
// and their host-side argument checks.
//
// A batch of trees is ragged: the tokens of entry b are rows q_start[b] ..
// q_start[b + 1] - 1 of every per-token tensor.  parent[row] is the index of a
// token's parent within its own tree, smaller than its own index; -1 continues
// the cached sequence; -2 marks a padded token.  A token sees the cached rows,
// its ancestors and itself; a padded token, and every descendant of one, sees
// nothing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <string>

#include "../../include/qhl_stage.h"
#include "common.cuh"

namespace qhl {

// Bit of the device error word: an index read on the device (page, parent,
// row offset, state) was out of its range and was not followed.
constexpr unsigned ERR_BAD_INDEX = 4u;

constexpr int kMaxNodes = 128;      // drafted tokens of one tree
constexpr int kMaxBatch = 2048;     // trees of one call
constexpr int kMaxRequests = 1024;  // sequences of one qhl_pages_* call

void set_last_error(const std::string& s);   // kernel_abi.cu

// Device error word of the verify operators on the current device (a static
// device word: no call allocates), and the value qhl_sync takes from it.
cudaError_t verify_error_word(unsigned** word);
unsigned verify_take_error(int dev);

inline int verify_err(const char* call, int code, const std::string& msg) {
  set_last_error(std::string(call) + ": " + msg);
  return code;
}
inline int verify_cuda_err(const char* call, cudaError_t e) {
  return verify_err(call, STAGE_E_CUDA, std::string(cudaGetErrorName(e)) + " (" + cudaGetErrorString(e) + ")");
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// 0, or the status of a KV cache description that the kernels cannot use.
int check_pages(const char* call, const qhl_kv_pages* kv);

// Rows [first, first + n) of tree b, or n = 0 (and the error bit) where q_start
// does not fit the call's n_rows and max_nodes.
QHL_DEV void tree_rows(const int* q_start, int b, int n_rows, int max_nodes, int& first, int& n, unsigned* err) {
  const int a = q_start[b], e = q_start[b + 1];
  first = a;
  n = e - a;
  if (a < 0 || e < a || e > n_rows || n > max_nodes) {
    atomicOr(err, ERR_BAD_INDEX);
    first = 0;
    n = 0;
  }
}

}  // namespace qhl
