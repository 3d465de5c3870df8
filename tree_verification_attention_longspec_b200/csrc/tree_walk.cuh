// The walk down a verified draft tree, given the target's token at every node (its argmax, or
// the token drawn there): the one rule of both acceptance calls.
#pragma once
#include "ls_device.cuh"

namespace ls {

// The smallest child of every node whose draft token is that node's token, then the walk
// from the root: path[0..len] (root first) and its length. All threads of the CTA (one
// per node slot, kMaxTree of them) call it; `token`, `parent` and `draft` are the tree's in
// shared memory, `first_match` is scratch, filled with INT32_MAX before a barrier that
// precedes the call. Thread 0 writes path and returns len; the others return 0.
__device__ __forceinline__ int walk_tree(const int32_t* token, const int32_t* parent, const int32_t* draft,
                                         int32_t* first_match, int n, int32_t* path) {
  const int tid = threadIdx.x;
  if (tid > 0 && tid < n && draft[tid] == token[parent[tid]]) atomicMin(&first_match[parent[tid]], tid);
  __syncthreads();
  int len = 0;
  if (tid == 0) {
    int cur = 0;
    path[0] = 0;
    while (first_match[cur] < n) {  // children lie above their parent: the walk ends
      cur = first_match[cur];
      path[++len] = cur;
    }
  }
  return len;
}

}  // namespace ls
