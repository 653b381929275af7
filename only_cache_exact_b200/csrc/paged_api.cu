// C ABI of the paged K+V cache (slim_mha_paged_*, declared in include/slim.h):
// argument checks; the kernels are in paged_append.cu, paged_decode.cu and
// paged_prefill.cu.
#include <cuda_runtime.h>

#include <algorithm>

#include "paged.cuh"

namespace slim {

void set_last_launch_count(int n);

namespace {

constexpr int64_t kInt32Max = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxCap = int64_t(1) << 30;   // a position and the tile behind it fit in int32
constexpr int64_t kMaxRows = int64_t(1) << 35;  // the 16-row tiles of all sequences are counted in 32 bits

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_cache(const slim_paged_cache* c) {
  if (!c || !c->kpages || !c->vpages || !c->table) return SLIM_EINVAL;
  if (!aligned(c->kpages, 16) || !aligned(c->vpages, 16) || !aligned(c->table, 4)) return SLIM_EINVAL;
  if (c->dtype != SLIM_F32 && c->dtype != SLIM_BF16 && c->dtype != SLIM_E4M3) return SLIM_EINVAL;
  if (c->B < 1 || c->Hkv < 1 || c->Hkv > 1024 || c->dh < 1 || c->page < 1 || c->max_pages < 1 || c->num_pages < 1)
    return SLIM_EINVAL;
  if (c->dtype == SLIM_F32 || (c->dh != 64 && c->dh != 128) || c->B > kPagedMaxB ||
      (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128))
    return SLIM_EUNSUPPORTED;
  const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page;
  if (c->num_pages > kInt32Max / (static_cast<int64_t>(c->Hkv) * c->page) || cap > kMaxCap || cap * c->B > kMaxRows)
    return SLIM_EINVAL;
  if (c->dtype == SLIM_E4M3 && (!c->kscale || !c->vscale || !aligned(c->kscale, 4) || !aligned(c->vscale, 4)))
    return SLIM_EINVAL;
  return SLIM_OK;
}

bool check_rows(const void* p, int64_t stride, int64_t heads, int dh) {
  return p && aligned(p, 16) && stride % 8 == 0 && stride >= heads * dh;
}

// max_new as the launches use it; false where the sizes are out of range.
bool check_packed(const int32_t* starts, const int32_t* other, int64_t rows, int64_t& max_new, int64_t heads) {
  if (!starts || !other || !aligned(starts, 4) || !aligned(other, 4) || rows < 1 || max_new < 0) return false;
  if (rows > kInt32Max || rows > kInt32Max * 64 / std::max<int64_t>(heads, 1)) return false;
  max_new = max_new == 0 ? rows : std::min(max_new, rows);
  return true;
}

int finish(cudaError_t e, int launches) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return e == cudaErrorNotSupported ? SLIM_EUNSUPPORTED : SLIM_ECUDA;
  }
  set_last_launch_count(launches);
  return SLIM_OK;
}

}  // namespace
}  // namespace slim

using namespace slim;

extern "C" {

int slim_mha_paged_append(const slim_paged_cache* cache, const void* q, int64_t q_stride, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, const float* cosines,
                          const float* sines, int rot, int interleaved, int64_t n_pos, const int32_t* starts,
                          const int32_t* lens, int64_t rows, int64_t max_new, int Hq, void* q_out,
                          int32_t* dev_status, void* stream) {
  const int rc = check_cache(cache);
  if (rc != SLIM_OK) return rc;
  if (rows == 0) return finish(cudaSuccess, 0);
  if (!dev_status || (!q != !q_out) || (interleaved != 0 && interleaved != 1)) return SLIM_EINVAL;
  if (q && (Hq < 1 || Hq > 8192 || Hq % cache->Hkv)) return SLIM_EINVAL;
  if (!check_packed(starts, lens, rows, max_new, std::max(cache->Hkv, q ? Hq : 0))) return SLIM_EINVAL;
  if (!check_rows(k, k_stride, cache->Hkv, cache->dh) || !check_rows(v, v_stride, cache->Hkv, cache->dh) ||
      (q && (!check_rows(q, q_stride, Hq, cache->dh) || !aligned(q_out, 16))))
    return SLIM_EINVAL;
  if (q && q == q_out && q_stride != static_cast<int64_t>(Hq) * cache->dh) return SLIM_EINVAL;
  if (rot < 0 || rot > cache->dh || rot % 16 || (rot > 0) != (cosines != nullptr) || !cosines != !sines)
    return SLIM_EINVAL;
  if (rot > 0 && (n_pos < 1 || !aligned(cosines, 16) || !aligned(sines, 16))) return SLIM_EINVAL;
  PagedAppendArgs a{cache, q, q_stride, k, k_stride, v, v_stride, cosines, sines, rot, interleaved, n_pos,
                    starts, lens, rows, max_new, Hq, q_out, dev_status};
  int launches = 0;
  const cudaError_t e = launch_paged_append(a, static_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

int slim_mha_paged_gather(const slim_paged_cache* cache, const int32_t* starts, const int32_t* first, int64_t rows,
                          int64_t max_new, void* k_out, void* v_out, int32_t* dev_status, void* stream) {
  const int rc = check_cache(cache);
  if (rc != SLIM_OK) return rc;
  if (rows == 0) return finish(cudaSuccess, 0);
  if (!k_out || !v_out || !dev_status || !aligned(k_out, 16) || !aligned(v_out, 16)) return SLIM_EINVAL;
  if (!check_packed(starts, first, rows, max_new, cache->Hkv)) return SLIM_EINVAL;
  int launches = 0;
  const cudaError_t e = launch_paged_gather(*cache, starts, first, rows, max_new, k_out, v_out, dev_status,
                                            static_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

size_t slim_mha_paged_decode_workspace_bytes(const slim_paged_cache* cache, int Hq) {
  if (check_cache(cache) != SLIM_OK || Hq < 1 || Hq > 8192 || Hq % cache->Hkv) return 0;
  return paged_rows_ws_bytes(*cache, Hq / cache->Hkv);
}

int slim_mha_paged_decode(const slim_paged_cache* cache, const void* q, int64_t q_stride, const int32_t* lens,
                          int rows_extra, int Hq, int64_t t_hint, void* out, void* workspace, size_t ws_bytes,
                          int32_t* dev_status, void* stream) {
  const int rc = check_cache(cache);
  if (rc != SLIM_OK) return rc;
  if (!lens || !aligned(lens, 4) || !out || !aligned(out, 16) || !dev_status) return SLIM_EINVAL;
  if (rows_extra != 0 && rows_extra != 1) return SLIM_EINVAL;
  if (Hq < 1 || Hq > 8192 || Hq % cache->Hkv || !check_rows(q, q_stride, Hq, cache->dh)) return SLIM_EINVAL;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < paged_rows_ws_bytes(*cache, Hq / cache->Hkv))
    return SLIM_EWORKSPACE;
  int launches = 0;
  const cudaError_t e = launch_paged_rows(*cache, q, q_stride, nullptr, lens, cache->B, 1, rows_extra, Hq, t_hint, out,
                                          workspace, dev_status, static_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

size_t slim_mha_paged_prefill_workspace_bytes(const slim_paged_cache* cache, int Hq, int64_t rows, int64_t max_new,
                                              int64_t t_hint) {
  if (check_cache(cache) != SLIM_OK || Hq < 1 || Hq > 8192 || Hq % cache->Hkv || Hq / cache->Hkv > 128 || rows < 1 ||
      rows > kInt32Max || max_new < 0)
    return 0;
  return paged_prefill_ws_bytes(*cache, Hq, rows, max_new == 0 ? rows : std::min(max_new, rows), t_hint);
}

int slim_mha_paged_prefill(const slim_paged_cache* cache, const void* q, int64_t q_stride, const int32_t* starts,
                           const int32_t* lens, int64_t rows, int64_t max_new, int Hq, int64_t t_hint, void* out,
                           void* workspace, size_t ws_bytes, int32_t* dev_status, void* stream) {
  const int rc = check_cache(cache);
  if (rc != SLIM_OK) return rc;
  if (rows == 0) return finish(cudaSuccess, 0);
  if (!out || !aligned(out, 16) || !dev_status) return SLIM_EINVAL;
  if (Hq < 1 || Hq > 8192 || Hq % cache->Hkv || !check_rows(q, q_stride, Hq, cache->dh)) return SLIM_EINVAL;
  if (!check_packed(starts, lens, rows, max_new, Hq)) return SLIM_EINVAL;
  if (Hq / cache->Hkv > 128) return SLIM_EUNSUPPORTED;
  if (!paged_prefill_fits(*cache, Hq, rows, max_new, t_hint)) return SLIM_EINVAL;
  const size_t need = paged_prefill_ws_bytes(*cache, Hq, rows, max_new, t_hint);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || ws_bytes < need)) return SLIM_EWORKSPACE;
  int launches = 0;
  const cudaError_t e =
      launch_paged_prefill(*cache, q, q_stride, starts, lens, rows, max_new, Hq, t_hint, out, workspace, dev_status,
                           static_cast<cudaStream_t>(stream), &launches);
  return finish(e, launches);
}

}  // extern "C"
