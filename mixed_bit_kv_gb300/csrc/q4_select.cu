// Page selection of the 4-bit paged cache (rdkv_q4_select).
#include "q4.cuh"

namespace rdkv {
namespace q4 {

struct SelectArgs {
  View c;
  const void* q;
  int32_t* sel;
  double* score;  // [rows][page_stride]
  int64_t q_stride;
  int dtype, n_q, G, D, keep, first, last;
};

// One block per (sequence, query token, KV head): the scores in 64 bits, then the best page again and
// again until enough are kept.
__global__ void __launch_bounds__(256) select_kernel(SelectArgs a) {
  __shared__ double best_s[8];
  __shared__ int arg_s[8], got_s;
  const int h = blockIdx.x % a.c.h_kv, bt = blockIdx.x / a.c.h_kv, t = bt % a.n_q, b = bt / a.n_q, tid = threadIdx.x;
  const int warp = tid / 32, lane = tid % 32;
  const int seen = held_tokens(a.c, b) - a.n_q + t + 1, P = seen > 0 ? ceil_div(seen, kPage) : 0;
  int32_t* sel = a.sel + (int64_t)blockIdx.x * a.keep;
  if (P <= a.keep) {
    for (int i = tid; i < a.keep; i += 256) sel[i] = i < P ? i : -1;
    return;
  }
  double* score = a.score + (int64_t)blockIdx.x * a.c.page_stride;
  const int64_t qrow = ((int64_t)b * a.n_q + t) * a.q_stride + (int64_t)h * a.G * a.D;
  for (int p = warp; p < P; p += 8) {
    const int phys = a.c.page_table[(int64_t)b * a.c.page_stride + p];
    double best = -INFINITY;
    if (phys < 0 || phys >= a.c.n_pages) {
      if (lane == 0) raise(a.c, RDKV_ERR_INVALID_ARG);
    } else {
      const __half* e = a.c.bounds + ((int64_t)phys * a.c.h_kv + h) * 2 * a.D;
      for (int g = 0; g < a.G; ++g) {
        double s = 0;
        for (int c = lane; c < a.D; c += 32) {
          const double x = load_q(a.q, qrow + g * a.D + c, a.dtype);
          s += x * (double)__half2float(e[x > 0 ? a.D + c : c]);
        }
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        best = fmax(best, s);
      }
    }
    if (p < a.first || p >= P - a.last) best = INFINITY;
    if (lane == 0) score[p] = best;
  }
  __syncthreads();
  // the kept pages are marked by NaN, then listed in order
  for (int n = 0; n < a.keep; ++n) {
    double best = -INFINITY;
    int arg = INT32_MAX;
    for (int p = tid; p < P; p += 256) {
      const double s = score[p];
      if (s > best || (s == best && p < arg)) best = s, arg = p;
    }
    for (int o = 16; o; o >>= 1) {
      const double s = __shfl_xor_sync(0xffffffffu, best, o);
      const int p = __shfl_xor_sync(0xffffffffu, arg, o);
      if (s > best || (s == best && p < arg)) best = s, arg = p;
    }
    if (lane == 0) best_s[warp] = best, arg_s[warp] = arg;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < 8; ++w)
        if (best_s[w] > best || (best_s[w] == best && arg_s[w] < arg)) best = best_s[w], arg = arg_s[w];
      if (arg < P) score[arg] = NAN;
    }
    __syncthreads();
  }
  if (tid == 0) {
    int n = 0;
    for (int p = 0; p < P && n < a.keep; ++p)
      if (isnan(score[p])) sel[n++] = p;
    got_s = n;
  }
  __syncthreads();
  for (int i = got_s + tid; i < a.keep; i += 256) sel[i] = -1;
}

}  // namespace q4
}  // namespace rdkv

using namespace rdkv;
using namespace rdkv::q4;

extern "C" size_t rdkv_q4_select_workspace_bytes(const rdkv_q4_cache* cache, int32_t h_q, int32_t n_q) {
  if (check_queries(cache, h_q, n_q) != RDKV_OK) return 0;
  return (size_t)align_up((int64_t)cache->batch * n_q * cache->h_kv * cache->page_stride * 8, 256);
}

extern "C" rdkv_status rdkv_q4_select(const rdkv_q4_cache* cache, int32_t dtype, const void* q, int64_t q_stride,
                                      int32_t h_q, int32_t n_q, int32_t n_keep, int32_t n_first, int32_t n_last, int32_t* sel,
                                      void* ws, size_t ws_bytes, void* stream) {
  rdkv_status st = check_q(cache, dtype, q, q_stride, h_q, n_q);
  if (st != RDKV_OK) return st;
  RDKV_REQUIRE(cache->bounds && sel, RDKV_ERR_INVALID_ARG, "NULL bounds or selection");
  RDKV_REQUIRE(n_keep >= 1 && n_first >= 0 && n_last >= 0 && (int64_t)n_first + n_last <= n_keep, RDKV_ERR_INVALID_ARG,
               "n_keep=%d n_first=%d n_last=%d", n_keep, n_first, n_last);
  const size_t need = rdkv_q4_select_workspace_bytes(cache, h_q, n_q);
  RDKV_REQUIRE(ws && (uintptr_t)ws % 16 == 0 && ws_bytes >= need, RDKV_ERR_WORKSPACE,
               "selection workspace too small (%zu < %zu) or unaligned", ws_bytes, need);
  SelectArgs a{view_of(cache), q, sel, static_cast<double*>(ws), q_stride, dtype, n_q, h_q / cache->h_kv, cache->head_dim,
               n_keep, n_first, n_last};
  select_kernel<<<(unsigned)((int64_t)cache->batch * n_q * cache->h_kv), 256, 0, (cudaStream_t)stream>>>(a);
  RDKV_CHECK_LAUNCH("4-bit cache selection");
  return RDKV_OK;
}
