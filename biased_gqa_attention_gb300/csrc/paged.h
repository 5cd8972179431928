// paged.h -- arguments and launchers of the packed and paged entry points
// (host side).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "extkv.h"
#include "internal.h"

namespace extkv {

// Rows to rotate and / or to write into pages.  Row t of batch b (BNSH: t < S)
// or of the packed axis (B = 1, S = T) starts at b * sb + t * ss + h * sh.
struct RowTensor {
  const void* src;
  void* dst;
  int64_t sb, ss, sh;  // source strides in elements: batch, row, head
  int64_t db, ds, dh;  // destination strides; for pages dh alone (head)
  int heads;           // 0: absent
};

struct RotaryArgs {
  RowTensor q, k, v;
  int64_t B, S, D;  // S rows in each of B batches
  const extkv_rotary* rotary;  // nullptr: copies
  // pages (append): k.dst / v.dst are pools
  int paged;
  const int64_t* page_table;
  const int64_t* write_idx;
  const int64_t* cu_seqlens;  // nullptr: one row per sequence
  int64_t n_seqs, num_pages, page_size, max_pages;
  int dtype;
  int32_t* status;
  cudaStream_t stream;
};
cudaError_t launch_rotary(const RotaryArgs& a);

struct PagedDecodeArgs {
  void* y;
  const void* q;
  const void* k_pages;
  const void* v_pages;
  const int64_t* page_table;
  const int64_t* nonpad;
  float scale;
  int32_t window;
  int64_t B, Hq, Hkv, D, num_pages, page_size, max_pages, q_stride;
  int dtype;
  void* workspace;
  int32_t* status;
  cudaStream_t stream;
  uint32_t wait_limit_plus1;  // as AttnArgs
  int variant;                // kDecodeAuto, kDecodeStreamK (the axis of tiles) or kDecodeCluster
};
size_t paged_decode_workspace_bytes(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int dtype);
// cudaErrorNotSupported: the cluster kernel was asked for and cannot take the call.
cudaError_t launch_paged_decode(const PagedDecodeArgs& a, const char** name);

struct PackedArgs {
  void* y;
  const void* q;
  const void* k;
  const void* v;
  const int64_t* cu_seqlens;
  float scale;
  int32_t causal, window;
  int64_t T, B, Hq, Hkv, D, q_stride, k_stride, v_stride;
  int dtype;
  void* workspace;
  int32_t* status;
  cudaStream_t stream;
  uint32_t wait_limit_plus1;  // as AttnArgs
};
size_t packed_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int dtype);
cudaError_t launch_packed(const PackedArgs& a, const char** name);

// Launch configuration with programmatic dependent launch: the kernel may be
// scheduled while its predecessor in the stream drains, and waits
// (griddepcontrol.wait) before it touches global memory.
struct PdlLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  PdlLaunch(dim3 grid, int threads, size_t smem, cudaStream_t stream) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

}  // namespace extkv
