// paged.cuh -- what the paged cache's calls share (append, decode).
//
// Layout.  A page holds one complete 64-token chunk of every kv-head: its
// keys and values as 8-bit codes with a float32 scale for each 8-token group
// and kv-head, and the float32 chunk and group summaries of the keys.  The
// chunk that a sequence is filling lives outside the pages, in the
// sequence's open rows: rotated keys in float32, values in their own type.
// So a code is rounded once, from the exact key, and never again while its
// chunk fills; and a token reads its own chunk exactly.
#pragma once

#include "check.cuh"
#include "hga_internal.cuh"

namespace hga {
namespace paged {

// Sequence lengths, token offsets and page numbers live on the device, so
// they are checked there, in every build: what is out of range is skipped
// and recorded in the translation unit's check word (hga_device_check).
__device__ __forceinline__ void flag(int site) { atomicCAS(&chk::g_check, 0, site); }

// Page number of a table entry, or -1 (recorded) outside the pool.
__device__ __forceinline__ int64_t page_or_none(int32_t page, int64_t n_pages, int site)
{
    if (page >= 0 && page < n_pages) return page;
    flag(site);
    return -1;
}

}  // namespace paged
}  // namespace hga
