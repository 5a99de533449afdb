// Row offsets of the items of a batch, from the batch column of sorted sites.
#include "dense_common.h"
#include "items.h"

namespace submconv {
namespace {

// Row i writes the offsets between its item's and the previous row's; row n the
// last ones. status: 1 for an item outside 0 .. items - 1, 2 for rows that are
// not in the items' order (any row may write it, always the same bits' union).
__global__ __launch_bounds__(256) void k_item_offsets(const int32_t* __restrict__ coords, int64_t ld, int64_t n,
                                                      int32_t items, int32_t* __restrict__ offsets,
                                                      int32_t* __restrict__ status) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i > n) return;
  const int32_t before = i > 0 ? coords[(i - 1) * ld] : -1, here = i < n ? coords[i * ld] : items;
  int bad = 0;
  if (i < n && (here < 0 || here >= items)) bad |= 1;
  if (i > 0 && i < n && here < before) bad |= 2;
  if (bad) atomicOr(status, bad);
  if (before >= items) return;  // (refused; before + 1 may pass 32 bits)
  const int32_t last = here < items ? here : items;
  for (int32_t b = before < -1 ? 0 : before + 1; b <= last; ++b) offsets[b] = static_cast<int32_t>(i);
}
__global__ void k_clear_status(int32_t* status) { *status = 0; }

}  // namespace
}  // namespace submconv

using namespace submconv;

extern "C" int submconv_item_offsets(const int32_t* coords, int64_t ld, int64_t n, int32_t items, int32_t* offsets,
                                     int32_t* status, hipStream_t stream) {
  clear_error();
  if (n < 0 || n > INT32_MAX) return set_error(SUBMCONV_ERR_INVALID_ARG, "n = %lld", (long long)n);
  if (items < 1 || items > 65535)
    return set_error(SUBMCONV_ERR_INVALID_ARG, "%d items, 1 to 65535 are supported", items);
  if (!offsets || !status || (n > 0 && !coords))
    return set_error(SUBMCONV_ERR_INVALID_ARG, "coords, offsets or status is NULL");
  if (n > 1 && ld < 1) return set_error(SUBMCONV_ERR_INVALID_ARG, "row stride %lld", (long long)ld);
  k_clear_status<<<1, 1, 0, stream>>>(status);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  k_item_offsets<<<static_cast<unsigned>(n / 256 + 1), 256, 0, stream>>>(coords, ld, n, items, offsets, status);
  SUBMCONV_HIP_CHECK(hipGetLastError());
  return SUBMCONV_OK;
}
