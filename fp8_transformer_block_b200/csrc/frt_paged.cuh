// frt_paged.cuh -- the paged KV cache's addresses (include/frt.h,
// frt_kv_record_bytes), shared by the kernels that write and read it.
#pragma once

#include "frt_common.cuh"

namespace frt {

struct PagePool {
  uint8_t* base;
  long record_bytes;  // one head's page_size tokens
  int n_pages, hkv;
  int page_size, shift;  // page_size = 1 << shift

  __host__ __device__ long slots() const { return long(n_pages) << shift; }
  __device__ __forceinline__ uint8_t* record(long slot, int head) const {
    return base + ((slot >> shift) * hkv + head) * record_bytes;
  }
  __device__ __forceinline__ int row(long slot) const { return int(slot) & (page_size - 1); }
};

inline PagePool make_page_pool(void* base, int format, int page_size, int n_pages, int hkv, int hd) {
  PagePool p{};
  p.base = static_cast<uint8_t*>(base);
  p.record_bytes = long(frt_kv_record_bytes(format, page_size, hd));
  p.n_pages = n_pages;
  p.hkv = hkv;
  p.page_size = page_size;
  while ((1 << p.shift) < page_size) ++p.shift;
  return p;
}

}  // namespace frt
