// C ABI of the library (declared in include/nb.h): host-side argument
// validation, device check and dispatch to the kernel launchers.  Everything
// here runs on the host before any launch, so an invalid call launches nothing.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <mutex>

#include "../../include/nb.h"
#include "nb_internal.h"
#include "serving.cuh"

namespace {

constexpr int kMaxDevices = 64;
// Per-device cache: 0 = unknown, 1 = sm_100 (supported), -1 = other.
int g_device_ok[kMaxDevices];

// Device word where kernels record the first wait-timeout code (0 = none),
// and its device address per device (looked up once).
// the site of the first wait that ran out, and the first NB_KERR_KV4_* code
__device__ int g_kernel_error[2];
std::mutex g_err_mutex;
int* g_err_addr[kMaxDevices];

int* error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lock(g_err_mutex);
  if (g_err_addr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_kernel_error) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    g_err_addr[dev] = static_cast<int*>(p);
  }
  return g_err_addr[dev];
}
int* skip_word() {
  int* w = error_word();
  return w ? w + 1 : nullptr;
}

nb_status check_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return NB_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return NB_ERR_DEVICE;
  int state = __atomic_load_n(&g_device_ok[dev], __ATOMIC_RELAXED);
  if (state == 0) {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return NB_ERR_CUDA;
    state = (major == 10 && minor == 0) ? 1 : -1;
    __atomic_store_n(&g_device_ok[dev], state, __ATOMIC_RELAXED);
  }
  return state == 1 ? NB_OK : NB_ERR_DEVICE;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shape checks shared by forward and backward.
nb_status check_shape(int batch, int heads, int n, int d, int R, int dtype) {
  if (batch < 0 || heads < 0 || n < 0 || R < 0) return NB_ERR_INVALID_ARG;
  if (n % nb::kBlock != 0) return NB_ERR_INVALID_ARG;
  if (dtype != NB_F32 && dtype != NB_BF16) return NB_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return NB_ERR_UNSUPPORTED;
  if (heads > 65535 || batch > 65535) return NB_ERR_UNSUPPORTED;  // grid y / z limits
  // element count must fit comfortably in int64 and rows*d*4 in size_t
  const double elems = static_cast<double>(batch) * heads * n * d;
  if (elems > 9.0e15) return NB_ERR_INVALID_ARG;
  return NB_OK;
}

nb::AttnArgs make_args(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, const int32_t* lengths, void* dq,
                       void* dk, void* dv, void* ws, int batch, int heads, int n, int d, int R,
                       bool causal) {
  nb::AttnArgs a;
  a.q = q; a.k = k; a.v = v; a.o = o; a.dout = dout;
  a.lse = const_cast<float*>(lse);
  a.lengths = lengths;
  a.dq = dq; a.dk = dk; a.dv = dv; a.workspace = ws;
  a.batch = batch; a.heads = heads; a.n = n; a.d = d; a.R = R;
  a.scale = static_cast<float>(1.0 / sqrt(static_cast<double>(d)));
  a.causal = causal;
  a.err = error_word();
  return a;
}

nb_status attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                   const int32_t* lengths, int batch, int heads, int n, int d, int R, int dtype,
                   void* stream, bool causal) {
  nb_status st = check_shape(batch, heads, n, d, R, dtype);
  if (st != NB_OK) return st;
  if (static_cast<int64_t>(batch) * heads * n == 0) return NB_OK;
  if (!q || !k || !v || !o) return NB_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      (lse && !aligned16(lse)) || (lengths && (reinterpret_cast<uintptr_t>(lengths) & 3u)))
    return NB_ERR_MISALIGNED;
  st = check_device();
  if (st != NB_OK) return st;
  nb::AttnArgs a = make_args(q, k, v, o, nullptr, lse, lengths, nullptr, nullptr, nullptr,
                             nullptr, batch, heads, n, d, R, causal);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e =
      dtype == NB_F32 ? nb::launch_attn_fwd_f32(a, s) : nb::launch_attn_fwd_bf16_tc(a, s);
  return e == cudaSuccess ? NB_OK : NB_ERR_CUDA;
}

// Pointer checks of the backward (null -> invalid, alignment).
nb_status bwd_pointers(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, const int32_t* lengths, void* dq,
                       void* dk, void* dv) {
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv) return NB_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
      !aligned16(lse) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) ||
      (lengths && (reinterpret_cast<uintptr_t>(lengths) & 3u)))
    return NB_ERR_MISALIGNED;
  return NB_OK;
}

nb_status attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                   const float* lse, const int32_t* lengths, void* dq, void* dk, void* dv,
                   void* workspace, size_t workspace_bytes, int batch, int heads, int n, int d,
                   int R, int dtype, void* stream, bool causal) {
  nb_status st = check_shape(batch, heads, n, d, R, dtype);
  if (st != NB_OK) return st;
  if (static_cast<int64_t>(batch) * heads * n == 0) return NB_OK;
  if (dtype != NB_BF16) return NB_ERR_UNSUPPORTED;
  st = bwd_pointers(q, k, v, o, dout, lse, lengths, dq, dk, dv);
  if (st != NB_OK) return st;
  const int64_t rows = static_cast<int64_t>(batch) * heads * n;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < nb::bwd_workspace_bytes(rows, d))
    return NB_ERR_WORKSPACE;
  st = check_device();
  if (st != NB_OK) return st;
  nb::AttnArgs a = make_args(q, k, v, o, dout, lse, lengths, dq, dk, dv, workspace, batch, heads,
                             n, d, R, causal);
  cudaError_t e = nb::launch_attn_bwd_bf16(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NB_OK : NB_ERR_CUDA;
}

// Shape checks of the attention with a window and sinks.
nb_status check_sink(int batch, int heads, int kv_heads, int n, int d, int window, int sinks,
                     int dtype) {
  if (batch < 0 || heads < 0 || kv_heads < 1 || n < 0 || window < 1 || sinks < 0)
    return NB_ERR_INVALID_ARG;
  if (heads % kv_heads != 0) return NB_ERR_INVALID_ARG;
  if (dtype != NB_F32 && dtype != NB_BF16) return NB_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || dtype != NB_BF16 || sinks > NB_MAX_SINKS) return NB_ERR_UNSUPPORTED;
  if (heads > 65535 || batch > 65535) return NB_ERR_UNSUPPORTED;
  // the row statistics take a block for 64 rows, and where all rows see few keys one more
  // for 16: they fit 31 bits, and so do the work items
  const double rows = static_cast<double>(batch) * heads * (static_cast<double>(n) + 127);
  if (rows > 2.7e10 || n > INT32_MAX - 512) return NB_ERR_UNSUPPORTED;
  return NB_OK;
}

nb::SinkArgs make_sink(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, const int32_t* lengths, void* dq,
                       void* dk, void* dv, void* ws, int batch, int heads, int kv_heads, int n,
                       int d, int window, int sinks) {
  nb::SinkArgs a = {q, k, v, o, dout, const_cast<float*>(lse), lengths, dq, dk, dv, ws, nullptr,
                    batch, heads, kv_heads, n, d, window, sinks,
                    static_cast<float>(1.0 / sqrt(static_cast<double>(d)))};
  return a;
}

// Shape checks of the 4-bit cache calls.  Positions, rows and grid sizes fit 31 bits.
nb_status check_kv4(int batch, int kv_heads, int d, int max_pages, int num_pages) {
  if (batch < 0 || kv_heads < 1 || max_pages < 0 || num_pages < 0) return NB_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return NB_ERR_UNSUPPORTED;
  if (max_pages >= INT32_MAX / NB_KV4_PAGE) return NB_ERR_UNSUPPORTED;
  return NB_OK;
}

nb_status kv4_rows(const void* k, const void* v, const void* cache, const int32_t* table,
                   const int32_t* starts, const int32_t* counts, int batch, int kv_heads, int n,
                   int d, int max_pages, int num_pages, int dtype, void* stream, bool write) {
  nb_status st = check_kv4(batch, kv_heads, d, max_pages, num_pages);
  if (st != NB_OK) return st;
  if (n < 0 || (dtype != NB_F32 && dtype != NB_BF16)) return NB_ERR_INVALID_ARG;
  if (kv_heads > 65535 || batch > 65535) return NB_ERR_UNSUPPORTED;  // grid y / z limits
  if (n > INT32_MAX - 64) return NB_ERR_UNSUPPORTED;
  if (batch == 0 || n == 0) return NB_OK;
  // a table without pages maps nothing, so it and the pool may then be null
  if (!k || !v || (max_pages > 0 && !table) || (max_pages > 0 && num_pages > 0 && !cache))
    return NB_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || !aligned4(table) ||
      !aligned4(starts) || !aligned4(counts))
    return NB_ERR_MISALIGNED;
  st = check_device();
  if (st != NB_OK) return st;
  nb::Kv4Args a = {const_cast<void*>(k), const_cast<void*>(v), const_cast<void*>(cache), table,
                   starts, counts, skip_word(), batch, kv_heads, n, d, max_pages, num_pages,
                   dtype == NB_F32};
  const cudaError_t e = nb::launch_kv4(a, write, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NB_OK : NB_ERR_CUDA;
}

// Shape checks of the single-token attention over the 4-bit cache.
nb_status check_decode(int batch, int heads, int kv_heads, int d, int max_pages, int num_pages,
                       int window, int sinks, int dtype) {
  nb_status st = check_kv4(batch, kv_heads, d, max_pages, num_pages);
  if (st != NB_OK) return st;
  if (heads < 0 || heads % kv_heads != 0 || window < 1 || sinks < 0) return NB_ERR_INVALID_ARG;
  if (dtype != NB_F32 && dtype != NB_BF16) return NB_ERR_INVALID_ARG;
  if (dtype != NB_BF16 || sinks > NB_MAX_SINKS) return NB_ERR_UNSUPPORTED;
  // rows, and blocks (few shares a row when there are many rows), fit 31 bits
  if (static_cast<double>(batch) * heads > INT32_MAX / 4) return NB_ERR_UNSUPPORTED;
  return NB_OK;
}

}  // namespace

namespace nb {

nb_status bwd_host_checks(int batch, int heads, int n, int d, int R, int dtype) {
  const nb_status st = check_shape(batch, heads, n, d, R, dtype);
  if (st != NB_OK) return st;
  if (static_cast<int64_t>(batch) * heads * n == 0) return NB_OK;
  return dtype == NB_BF16 ? NB_OK : NB_ERR_UNSUPPORTED;
}

nb_status bwd_pointer_checks(const void* q, const void* k, const void* v, const void* o,
                             const void* dout, const float* lse, const int32_t* lengths,
                             void* dq, void* dk, void* dv) {
  return bwd_pointers(q, k, v, o, dout, lse, lengths, dq, dk, dv);
}

nb_status device_check() { return check_device(); }

}  // namespace nb

extern "C" {

const char* nb_status_string(int status) {
  switch (status) {
    case NB_OK: return "NB_OK";
    case NB_ERR_INVALID_ARG: return "NB_ERR_INVALID_ARG: invalid argument";
    case NB_ERR_UNSUPPORTED: return "NB_ERR_UNSUPPORTED: unsupported configuration";
    case NB_ERR_MISALIGNED: return "NB_ERR_MISALIGNED: pointer not 16-byte aligned";
    case NB_ERR_CUDA: return "NB_ERR_CUDA: CUDA runtime error";
    case NB_ERR_WORKSPACE: return "NB_ERR_WORKSPACE: workspace missing, misaligned or too small";
    case NB_ERR_DEVICE: return "NB_ERR_DEVICE: current device is not sm_100";
    default: return "unknown nb_status";
  }
}

int nb_abi_version(void) { return NB_ABI_VERSION; }

nb_status nb_kernel_error(int* code, int clear) {
  if (!code) return NB_ERR_INVALID_ARG;
  *code = 0;
  int* w = error_word();
  if (!w) return NB_ERR_CUDA;
  if (cudaDeviceSynchronize() != cudaSuccess) return NB_ERR_CUDA;
  int words[2];
  if (cudaMemcpy(words, w, sizeof(words), cudaMemcpyDeviceToHost) != cudaSuccess) return NB_ERR_CUDA;
  const nb::KernelReport r = nb::kernel_report(words);
  *code = r.code;
  if (clear && r.code != 0 && cudaMemset(w + r.word, 0, sizeof(int)) != cudaSuccess)
    return NB_ERR_CUDA;
  return NB_OK;
}

nb_status nb_attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                      const int32_t* lengths, int batch, int heads, int n, int d, int R,
                      int dtype, void* stream) {
  return attn_fwd(q, k, v, o, lse, lengths, batch, heads, n, d, R, dtype, stream, false);
}

nb_status nb_attn_fwd_causal(const void* q, const void* k, const void* v, void* o, float* lse,
                             const int32_t* lengths, int batch, int heads, int n, int d, int R,
                             int dtype, void* stream) {
  return attn_fwd(q, k, v, o, lse, lengths, batch, heads, n, d, R, dtype, stream, true);
}

size_t nb_attn_bwd_workspace_size(int batch, int heads, int n, int d, int dtype) {
  if (check_shape(batch, heads, n, d, 0, dtype) != NB_OK) return 0;
  const int64_t rows = static_cast<int64_t>(batch) * heads * n;
  if (rows == 0) return 0;
  return nb::bwd_workspace_bytes(rows, d);
}

nb_status nb_attn_bwd(const void* q, const void* k, const void* v, const void* o,
                      const void* dout, const float* lse, const int32_t* lengths, void* dq,
                      void* dk, void* dv, void* workspace, size_t workspace_bytes, int batch,
                      int heads, int n, int d, int R, int dtype, void* stream) {
  return attn_bwd(q, k, v, o, dout, lse, lengths, dq, dk, dv, workspace, workspace_bytes, batch,
                  heads, n, d, R, dtype, stream, false);
}

nb_status nb_attn_bwd_causal(const void* q, const void* k, const void* v, const void* o,
                             const void* dout, const float* lse, const int32_t* lengths, void* dq,
                             void* dk, void* dv, void* workspace, size_t workspace_bytes,
                             int batch, int heads, int n, int d, int R, int dtype, void* stream) {
  return attn_bwd(q, k, v, o, dout, lse, lengths, dq, dk, dv, workspace, workspace_bytes, batch,
                  heads, n, d, R, dtype, stream, true);
}

nb_status nb_tokenize_kmer(const uint8_t* seq, int64_t len, uint16_t* ids, uint8_t* packed,
                           int k, void* stream) {
  if (len < 0) return NB_ERR_INVALID_ARG;
  if (k < 1 || k > 7) return NB_ERR_UNSUPPORTED;
  if (ids && (reinterpret_cast<uintptr_t>(ids) & 1u)) return NB_ERR_MISALIGNED;
  if (len == 0 || (!ids && !packed)) return NB_OK;
  if (!seq) return NB_ERR_INVALID_ARG;
  if (len < k) ids = nullptr;  // no complete window: only the packed stream is written
  if (!ids && !packed) return NB_OK;
  nb_status st = check_device();
  if (st != NB_OK) return st;
  cudaError_t e =
      nb::launch_tokenize_kmer(seq, len, ids, packed, k, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NB_OK : NB_ERR_CUDA;
}

nb_status nb_tokenize_batch(const uint8_t* seqs, const int64_t* offsets, int batch, int k,
                            int64_t* input_ids, int32_t* lengths, int n_pad, void* stream) {
  if (batch < 0 || n_pad < 0 || n_pad % NB_BLOCK != 0) return NB_ERR_INVALID_ARG;
  if (k < 1 || k > 7 || batch > 65535) return NB_ERR_UNSUPPORTED;
  if (batch == 0) return NB_OK;
  if (!seqs || !offsets || (n_pad > 0 && !input_ids)) return NB_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(input_ids) & 15u) || (reinterpret_cast<uintptr_t>(offsets) & 7u) ||
      (reinterpret_cast<uintptr_t>(lengths) & 3u))
    return NB_ERR_MISALIGNED;
  if (n_pad == 0 && !lengths) return NB_OK;
  nb_status st = check_device();
  if (st != NB_OK) return st;
  cudaError_t e = nb::launch_tokenize_batch(seqs, offsets, batch, k, input_ids, lengths, n_pad,
                                            static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NB_OK : NB_ERR_CUDA;
}

nb_status nb_batch_ceiling(const int64_t* offsets, int batch, int k, int32_t* n_pad) {
  if (!n_pad || batch < 0 || (batch > 0 && !offsets)) return NB_ERR_INVALID_ARG;
  if (k < 1 || k > 7) return NB_ERR_UNSUPPORTED;
  int64_t windows = 0;
  for (int b = 0; b < batch; ++b) {
    const int64_t bases = offsets[b + 1] - offsets[b];
    const int64_t w = bases >= k ? bases - k + 1 : 0;
    if (w > windows) windows = w;
  }
  const int64_t ceil32 = (windows + NB_BLOCK - 1) / NB_BLOCK * NB_BLOCK;
  if (ceil32 > INT32_MAX) return NB_ERR_INVALID_ARG;
  *n_pad = static_cast<int32_t>(ceil32);
  return NB_OK;
}

nb_status nb_attn_sink_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                           const int32_t* lengths, int batch, int heads, int kv_heads, int n, int d,
                           int window, int sinks, int dtype, void* stream) {
  nb_status st = check_sink(batch, heads, kv_heads, n, d, window, sinks, dtype);
  if (st != NB_OK) return st;
  if (batch == 0 || heads == 0 || n == 0) return NB_OK;
  if (!q || !k || !v || !o) return NB_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      !aligned4(lengths))
    return NB_ERR_MISALIGNED;
  st = check_device();
  if (st != NB_OK) return st;
  nb::SinkArgs a = make_sink(q, k, v, o, nullptr, lse, lengths, nullptr, nullptr, nullptr, nullptr,
                             batch, heads, kv_heads, n, d, window, sinks);
  a.err = error_word();
  const cudaError_t e = nb::launch_attn_sink_fwd(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NB_OK : NB_ERR_CUDA;
}

size_t nb_attn_sink_bwd_workspace_size(int batch, int heads, int kv_heads, int n, int d, int window,
                                       int sinks, int dtype) {
  if (check_sink(batch, heads, kv_heads, n, d, window, sinks, dtype) != NB_OK) return 0;
  if (batch == 0 || heads == 0 || n == 0) return 0;
  return nb::sink_bwd_workspace_bytes(make_sink(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                                nullptr, nullptr, nullptr, nullptr, nullptr, batch,
                                                heads, kv_heads, n, d, window, sinks));
}

nb_status nb_attn_sink_bwd(const void* q, const void* k, const void* v, const void* o,
                           const void* dout, const float* lse, const int32_t* lengths, void* dq,
                           void* dk, void* dv, void* workspace, size_t workspace_bytes, int batch,
                           int heads, int kv_heads, int n, int d, int window, int sinks, int dtype,
                           void* stream) {
  nb_status st = check_sink(batch, heads, kv_heads, n, d, window, sinks, dtype);
  if (st != NB_OK) return st;
  if (batch == 0 || heads == 0 || n == 0) return NB_OK;
  st = bwd_pointers(q, k, v, o, dout, lse, lengths, dq, dk, dv);
  if (st != NB_OK) return st;
  nb::SinkArgs a = make_sink(q, k, v, o, dout, lse, lengths, dq, dk, dv, workspace, batch, heads,
                             kv_heads, n, d, window, sinks);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
      workspace_bytes < nb::sink_bwd_workspace_bytes(a))
    return NB_ERR_WORKSPACE;
  st = check_device();
  if (st != NB_OK) return st;
  a.err = error_word();
  const cudaError_t e = nb::launch_attn_sink_bwd(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NB_OK : NB_ERR_CUDA;
}

size_t nb_kv4_page_bytes(int d) {
  return d == 64 || d == 128 ? static_cast<size_t>(nb::kv4_page_bytes(d)) : 0;
}

nb_status nb_kv4_write(const void* k, const void* v, void* cache, const int32_t* block_table,
                       const int32_t* starts, const int32_t* counts, int batch, int kv_heads, int n,
                       int d, int max_pages, int num_pages, int dtype, void* stream) {
  return kv4_rows(k, v, cache, block_table, starts, counts, batch, kv_heads, n, d, max_pages,
                  num_pages, dtype, stream, true);
}

nb_status nb_kv4_read(const void* cache, const int32_t* block_table, const int32_t* starts,
                      const int32_t* counts, void* k, void* v, int batch, int kv_heads, int n,
                      int d, int max_pages, int num_pages, int dtype, void* stream) {
  return kv4_rows(k, v, cache, block_table, starts, counts, batch, kv_heads, n, d, max_pages,
                  num_pages, dtype, stream, false);
}

size_t nb_attn_kv4_decode_workspace_size(int batch, int heads, int kv_heads, int d, int max_pages,
                                         int window, int sinks, int dtype) {
  if (check_decode(batch, heads, kv_heads, d, max_pages, 0, window, sinks, dtype) != NB_OK) return 0;
  if (batch == 0 || heads == 0) return 0;
  nb::Kv4DecodeArgs a = {};
  a.batch = batch; a.heads = heads; a.kv_heads = kv_heads; a.d = d;
  a.max_pages = max_pages; a.window = window; a.sinks = sinks;
  return nb::kv4_decode_workspace_bytes(a);
}

nb_status nb_attn_kv4_decode(const void* q, const void* cache, const int32_t* block_table,
                             const int32_t* lengths, void* o, float* lse, void* workspace,
                             size_t workspace_bytes, int batch, int heads, int kv_heads, int d,
                             int max_pages, int num_pages, int window, int sinks, int dtype,
                             void* stream) {
  nb_status st =
      check_decode(batch, heads, kv_heads, d, max_pages, num_pages, window, sinks, dtype);
  if (st != NB_OK) return st;
  if (batch == 0 || heads == 0) return NB_OK;
  if (!q || !o || (max_pages > 0 && !block_table) || (max_pages > 0 && num_pages > 0 && !cache))
    return NB_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(o) || !aligned16(cache) || !aligned4(block_table) ||
      !aligned4(lengths) || !aligned4(lse))
    return NB_ERR_MISALIGNED;
  nb::Kv4DecodeArgs a = {q, cache, block_table, lengths, o, lse, workspace, nullptr, nullptr, batch,
                         heads, kv_heads, d, max_pages, num_pages, window, sinks};
  const size_t need = nb::kv4_decode_workspace_bytes(a);
  if (need > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                   workspace_bytes < need))
    return NB_ERR_WORKSPACE;
  st = check_device();
  if (st != NB_OK) return st;
  a.err = error_word();
  a.skip = skip_word();
  const cudaError_t e = nb::launch_kv4_decode(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? NB_OK : NB_ERR_CUDA;
}

}  // extern "C"
