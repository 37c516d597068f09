// C ABI of the windowed attention and of the 4-bit key/value cache: argument checks and launches.
#include <climits>
#include <string>

#include "cache4.cuh"
#include "launch.h"
#include "rmt.h"

namespace rmt {
void set_last_error(const std::string& msg);
rmt_status device_error_word(int** err);
}  // namespace rmt

namespace {

using namespace rmt;

rmt_status fail(rmt_status st, const std::string& msg) {
  set_last_error(msg);
  return st;
}

// Device memory (or managed); its device becomes the current one for the rest of the call.
struct OnDeviceOf {
  int prev = -1;
  rmt_status st = RMT_OK;
  explicit OnDeviceOf(const void* p) {
    cudaPointerAttributes attr;
    cudaError_t e = cudaPointerGetAttributes(&attr, p);
    if (e != cudaSuccess) {
      cudaGetLastError();
      st = fail(RMT_ECUDA, std::string("cudaPointerGetAttributes: ") + cudaGetErrorString(e));
      return;
    }
    if (attr.type != cudaMemoryTypeDevice && attr.type != cudaMemoryTypeManaged) {
      st = fail(RMT_EINVAL, "a device pointer is needed");
      return;
    }
    int cur = -1;
    e = cudaGetDevice(&cur);
    if (e == cudaSuccess && attr.device >= 0 && cur != attr.device) {
      e = cudaSetDevice(attr.device);
      if (e == cudaSuccess) prev = cur;
    }
    if (e != cudaSuccess) st = fail(RMT_ECUDA, std::string("the tensors' device: ") + cudaGetErrorString(e));
  }
  ~OnDeviceOf() {
    if (prev >= 0) cudaSetDevice(prev);
  }
};

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Window length as the kernels take it: 0 means every earlier key. Positions stay below 2^30.
constexpr int kNoWindow = 1 << 30;
int window_length(int32_t w) { return w == 0 || w > kNoWindow ? kNoWindow : w; }

const char* cache_problem(const rmt_cache* c) {
  if (!c || !c->pages || !c->page_table || !c->lens) return "null pointer";
  if (c->n_pages <= 0 || c->n_seqs <= 0 || c->max_pages <= 0 || c->n_kv_heads <= 0) return "sizes must be positive";
  if (c->max_pages > kNoWindow / RMT_CACHE_PAGE) return "a sequence holds at most 2^30 tokens";
  if (c->n_kv_heads > 4096) return "n_kv_heads must be at most 4096";
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 128) return "head_dim must be 32, 64 or 128";
  if (!aligned(c->pages, 16)) return "pages must be 16-byte aligned";
  if (!aligned(c->page_table, 4) || !aligned(c->lens, 4)) return "page_table and lens must be 4-byte aligned";
  return nullptr;
}

cache4::CacheArgs cache_args(const rmt_cache* c, int* err) {
  return {static_cast<unsigned char*>(c->pages), c->page_table, c->lens, c->n_pages, c->n_seqs, c->max_pages,
          c->n_kv_heads, err};
}

rmt_status cache_rows(const rmt_cache* c, const void* k, const void* v, int64_t ld, int32_t M, const int32_t* n_new,
                      rmt_dtype dtype, bool write, void* stream) {
  if (const char* why = cache_problem(c)) return fail(RMT_EINVAL, why);
  if (!k || !v) return fail(RMT_EINVAL, "null pointer");
  if (M <= 0 || int64_t(c->n_seqs) * M > INT_MAX) return fail(RMT_EINVAL, "M must be positive, n_seqs * M below 2^31");
  // 8 channels a thread: no more than 2^30 warps, and their heads rounded up
  if (int64_t(c->n_seqs) * M * (int64_t(c->n_kv_heads) * c->head_dim) > (int64_t(1) << 37))
    return fail(RMT_EINVAL, "n_seqs * M * n_kv_heads * head_dim must be at most 2^37");
  if (dtype != RMT_F32 && dtype != RMT_BF16) return fail(RMT_EINVAL, "dtype must be RMT_F32 or RMT_BF16");
  const int64_t es = dtype == RMT_BF16 ? 2 : 4;
  if (ld < int64_t(c->n_kv_heads) * c->head_dim) return fail(RMT_EINVAL, "ld is below n_kv_heads * head_dim");
  if (!aligned(k, 16) || !aligned(v, 16) || (ld * es) % 16)
    return fail(RMT_EINVAL, "k, v and their rows must be 16-byte aligned");
  if (n_new && !aligned(n_new, 4)) return fail(RMT_EINVAL, "n_new must be 4-byte aligned");
  OnDeviceOf dev(c->pages);
  if (dev.st != RMT_OK) return dev.st;
  int* err = nullptr;
  if (rmt_status st = device_error_word(&err); st != RMT_OK) return st;
  CacheRowsArgs a{cache_args(c, err), const_cast<void*>(k), const_cast<void*>(v), ld, M, n_new};
  const cudaError_t e =
      write ? launch_cache_write(a, c->head_dim, dtype == RMT_BF16, static_cast<cudaStream_t>(stream))
            : launch_cache_read(a, c->head_dim, dtype == RMT_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RMT_OK : fail(RMT_ECUDA, std::string("launch failed: ") + cudaGetErrorString(e));
}

const char* attention_problem(const rmt_cache* c, int32_t n_q, int32_t H, int32_t window, int32_t sinks) {
  if (const char* why = cache_problem(c)) return why;
  if (n_q <= 0 || n_q > 64) return "n_q must be in 1 .. 64";
  if (H <= 0 || H % c->n_kv_heads || H > 65536) return "H must be a positive multiple of n_kv_heads, at most 65536";
  if (window < 0 || sinks < 0) return "window and sinks must not be negative";
  if (int64_t(c->n_seqs) * n_q * H > INT_MAX) return "n_seqs * n_q * H must be below 2^31";
  return nullptr;
}

}  // namespace

extern "C" {

size_t rmt_cache_page_bytes(int32_t n_kv_heads, int32_t head_dim) {
  if (n_kv_heads <= 0 || (head_dim != 32 && head_dim != 64 && head_dim != 128)) return 0;
  return size_t(n_kv_heads) * 72 * head_dim;
}

rmt_status rmt_cache_write(const rmt_cache* c, const void* k, const void* v, int64_t ld, int32_t M,
                           const int32_t* n_new, rmt_dtype dtype, void* stream) {
  return cache_rows(c, k, v, ld, M, n_new, dtype, true, stream);
}

rmt_status rmt_cache_read(const rmt_cache* c, void* k, void* v, int64_t ld, int32_t M, const int32_t* n_new,
                          rmt_dtype dtype, void* stream) {
  return cache_rows(c, k, v, ld, M, n_new, dtype, false, stream);
}

size_t rmt_attention_cache_workspace(const rmt_cache* c, int32_t n_q, int32_t H, int32_t window, int32_t sinks) {
  const char* why = attention_problem(c, n_q, H, window, sinks);
  const size_t n = why ? 0
                       : cache_attention_workspace(c->n_seqs, c->max_pages, n_q, H, c->n_kv_heads, c->head_dim,
                                                   window_length(window), sinks);
  if (n == 0) fail(RMT_EINVAL, why ? why : "the sequences hold too many pages for one call");
  return n;
}

rmt_status rmt_attention_cache(const rmt_cache* c, const void* q, int64_t ldq, void* out, int32_t n_q, int32_t H,
                               int32_t window, int32_t sinks, void* workspace, size_t workspace_bytes,
                               rmt_dtype dtype, void* stream) {
  if (const char* why = attention_problem(c, n_q, H, window, sinks)) return fail(RMT_EINVAL, why);
  if (!q || !out || !workspace) return fail(RMT_EINVAL, "null pointer");
  if (dtype != RMT_F32 && dtype != RMT_BF16) return fail(RMT_EINVAL, "dtype must be RMT_F32 or RMT_BF16");
  const int64_t es = dtype == RMT_BF16 ? 2 : 4;
  if (ldq < int64_t(H) * c->head_dim) return fail(RMT_EINVAL, "ldq is below H * head_dim");
  if (!aligned(q, 16) || !aligned(out, 16) || (ldq * es) % 16 || !aligned(workspace, 16))
    return fail(RMT_EINVAL, "q, its rows, out and workspace must be 16-byte aligned");
  const size_t need = rmt_attention_cache_workspace(c, n_q, H, window, sinks);
  if (need == 0) return RMT_EINVAL;
  if (workspace_bytes < need)
    return fail(RMT_EINVAL, "the workspace is smaller than rmt_attention_cache_workspace asks for");
  OnDeviceOf dev(c->pages);
  if (dev.st != RMT_OK) return dev.st;
  int* err = nullptr;
  if (rmt_status st = device_error_word(&err); st != RMT_OK) return st;
  CacheAttnArgs a{cache_args(c, err), q, ldq, out, n_q, H, window_length(window), sinks, workspace};
  const cudaError_t e = launch_cache_attention(a, c->head_dim, dtype == RMT_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RMT_OK : fail(RMT_ECUDA, std::string("launch failed: ") + cudaGetErrorString(e));
}

rmt_status rmt_attention_window(const void* qkv, void* out, int32_t G, int32_t M, int32_t H, int32_t Hkv, int32_t dh,
                                int32_t window, int32_t sinks, const int32_t* lens, rmt_dtype dtype, void* stream) {
  if (!qkv || !out) return fail(RMT_EINVAL, "null pointer");
  if (G <= 0 || M <= 0 || H <= 0 || Hkv <= 0 || H % Hkv) return fail(RMT_EINVAL, "bad sizes");
  if (G > 65535 || H > 65535 || M > kNoWindow) return fail(RMT_EINVAL, "G and H at most 65535, M at most 2^30");
  if (dh != 32 && dh != 64 && dh != 128) return fail(RMT_EINVAL, "dh must be 32, 64 or 128");
  if (window < 0 || sinks < 0) return fail(RMT_EINVAL, "window and sinks must not be negative");
  if (dtype != RMT_F32 && dtype != RMT_BF16) return fail(RMT_EINVAL, "dtype must be RMT_F32 or RMT_BF16");
  if (!aligned(qkv, 16) || !aligned(out, 16)) return fail(RMT_EINVAL, "qkv and out must be 16-byte aligned");
  if (lens && !aligned(lens, 4)) return fail(RMT_EINVAL, "lens must be 4-byte aligned");
  OnDeviceOf dev(qkv);
  if (dev.st != RMT_OK) return dev.st;
  int* err = nullptr;
  if (rmt_status st = device_error_word(&err); st != RMT_OK) return st;
  WindowAttnArgs a{qkv, out, G, M, H, Hkv, window_length(window), sinks, lens, err};
  const cudaError_t e = launch_window_attention(a, dh, dtype == RMT_BF16, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? RMT_OK : fail(RMT_ECUDA, std::string("launch failed: ") + cudaGetErrorString(e));
}

}  // extern "C"
