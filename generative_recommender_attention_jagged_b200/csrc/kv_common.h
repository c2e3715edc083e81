// What the append kernels of the paged cache share: the arguments of a call and
// the plan launch (page allocation, new lengths), the same for every element
// type of the pool.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "hstu_internal.h"

namespace hstu {

struct KvArgs {
  int32_t B, H, d, P, num_pages, max_pages, esize, total_new;
  long long kv_stride;  // elements between tokens of k_new / v_new
  const uint8_t* k_new;
  const uint8_t* v_new;
  const int32_t* new_offsets;
  const int32_t* num_append;
  uint8_t* k_pool;
  uint8_t* v_pool;
  int32_t* page_table;
  int32_t* cached_lens;
  int32_t* free_pages;
  int32_t* free_count;
  WsHeader* hdr;     // status word; pad[0] = 1 once the plan was applied
  int32_t* l_old;    // [B] lengths before the append
  int32_t* n_app;    // [B] tokens appended
};

// Validates an append and, if all of it fits, takes its pages, writes the new
// lengths and leaves hdr->pad[0] = 1, l_old and n_app for the copy (hdr zeroed before).
cudaError_t launch_kv_append_plan(const KvArgs& a, cudaStream_t s);

}  // namespace hstu
