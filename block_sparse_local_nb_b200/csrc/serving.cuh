// What the kernels of the windowed attention with sinks and of the 4-bit cache share:
// their arguments and launchers, and a few device helpers.
#pragma once

#include "nb_internal.h"
#include "sm100.cuh"

namespace nb {

// Arguments of an attention call with a window and sinks, validated on the host.
struct SinkArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* o;      // forward: output; backward: input
  const void* dout;   // backward only
  float* lse;         // forward: output (may be null); backward: input
  const int32_t* lengths;  // may be null = all full
  void* dq;
  void* dk;
  void* dv;
  void* workspace;
  int* err;
  int batch, heads, kv_heads, n, d, window, sinks;
  float scale;        // 1/sqrt(d)
};

// Arguments of a write to or a read from the 4-bit cache.
struct Kv4Args {
  void* k;  // write: input; read: output
  void* v;
  void* cache;
  const int32_t* table;
  const int32_t* starts;  // may be null = 0
  const int32_t* counts;  // may be null = n
  int* skip;  // first token that was not mapped
  int batch, kv_heads, n, d, max_pages, num_pages;
  bool f32;
};

struct Kv4DecodeArgs {
  const void* q;
  const void* cache;
  const int32_t* table;
  const int32_t* lengths;
  void* o;
  float* lse;
  void* workspace;
  int* err;   // first wait that ran out
  int* skip;  // first page that was not mapped
  int batch, heads, kv_heads, d, max_pages, num_pages, window, sinks;
};

// What nb_kernel_error makes of the two device words, the site of a wait that ran out and
// a NB_KERR_KV4_* code: the first of them that is set, and which.
struct KernelReport {
  int code, word;
};
inline KernelReport kernel_report(const int (&words)[2]) {
  if (words[0] != 0) return {NB_KERR_WAIT | words[0], 0};
  return {words[1], 1};
}

// launch_pdl with the grid's blocks in clusters of `cluster` along x (1: none).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                               cudaStream_t stream, int cluster, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// make_tmap_bf16_rows whose loads read 0 from row `first` (at least 1) of every head on.
bool make_tmap_first_rows(CUtensorMap* m, const void* base, int d, int64_t n, int64_t heads_total,
                          int first, int box_rows);
cudaError_t launch_attn_sink_fwd(const SinkArgs& a, cudaStream_t stream);
size_t sink_bwd_workspace_bytes(const SinkArgs& a);
cudaError_t launch_attn_sink_bwd(const SinkArgs& a, cudaStream_t stream);
int kv4_page_bytes(int d);  // d = 64 or 128
cudaError_t launch_kv4(const Kv4Args& a, bool write, cudaStream_t stream);
size_t kv4_decode_workspace_bytes(const Kv4DecodeArgs& a);
cudaError_t launch_kv4_decode(const Kv4DecodeArgs& a, cudaStream_t stream);

namespace sm100 {

// Position in a ring of N barriers and the parity of its current pass.
template <int N>
struct Ring {
  int i = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int step = 1) {  // step <= N
    i += step;
    if (i >= N) {
      i -= N;
      ph ^= 1;
    }
  }
};

// A ring of N stages, each with a barrier that completes a phase when its copy has landed,
// and nothing else: i and ph are where the next copy would go and its phase's parity.  Calls
// wait(stage, parity) for the last copy of each; it returns at once where none is in flight.
template <int N, class Wait>
__host__ __device__ __forceinline__ void drain_ring(int i, uint32_t ph, Wait&& wait) {
#pragma unroll 1
  for (int s = 0; s < N; ++s) wait(s, s < i ? ph : ph ^ 1u);
}

// d = a b + c (a row-major 16 x 16, b 16 x 8, bf16 in, fp32 out).
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]),
        "f"(c[2]), "f"(c[3]));
}

}  // namespace sm100
}  // namespace nb
