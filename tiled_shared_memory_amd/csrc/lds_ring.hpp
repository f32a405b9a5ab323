// K-contiguous operand slabs on their way from global memory into LDS: the
// copies, swizzles and buffer resources of the large-tile kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tsm {

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) char lds_char;

// A per-lane offset past every buffer resource (which the host keeps below
// 1 GiB): such a load returns zeros.  Slice offsets added to it stay below 2^32.
constexpr uint32_t kOutside = 0x80000000u;

// Buffer resource over `bytes` bytes starting at `base` (raw addressing,
// dword 3 = the gfx9 default data format).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void *base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}

// LDS position of 16-byte chunk c of row r of a K-contiguous slab, KB = slab
// depth / 32.  The fragment reads take rows (lane % 16) + 16i at chunk
// 4U + lane / 16 (16x16x32 operands).  Both swizzles were chosen by measuring
// the LDS bank-conflict counter on that read pattern, over every swizzle of
// the form c ^ (XOR-linear function of row bits 0..3) and random ones: with
// these, the reads are conflict-free (4 LDS cycles per 64-lane 16-byte read);
// unswizzled rows cost 2x (64-byte rows) and 4x (128-byte rows).
//  KB = 1 (64-byte rows): c ^ (3 * bit 3 of r).
//  KB = 2 (128-byte rows): c ^ ((r / 2) % 8).
template <int KB>
__device__ __forceinline__ int swz(int r, int c) {
  if constexpr (KB == 1) {
    return c ^ (((r >> 3) & 1) * 3);
  } else {
    return c ^ ((r >> 1) & 7);
  }
}

// Per-lane byte offsets, relative to the slab origin, of the chunks a lane
// fetches for one 256 x 32KB K-contiguous operand slab (rows ld elements
// apart).  One wave-wide load fills 1 KiB = 16 / KB whole rows: lane l writes
// LDS slot l, i.e. row l / (4 KB) of its group at position l % (4 KB), so it
// fetches the chunk whose swizzled position that is (swz is an involution in
// its chunk argument).
template <int LOADS, int KB>
__device__ __forceinline__ void slice_offsets(uint32_t (&off)[LOADS], int64_t ld, int wave, int lane) {
  constexpr int CPR = 4 * KB;  // chunks per row
#pragma unroll
  for (int g = 0; g < LOADS; ++g) {
    const int r = (wave * LOADS + g) * (64 / CPR) + lane / CPR;
    off[g] = (uint32_t)(r * ld + swz<KB>(r, lane % CPR) * 8) * 2u;
  }
}

// Asynchronous copy of one operand slice into LDS: 16 buffer loads shared by
// the waves, each writing 1 KiB of LDS; kbytes is the slice's K offset in bytes.
template <int LOADS>
__device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t rsrc, const uint32_t *off, uint32_t kbytes, char *lds,
                                      int wave) {
#pragma unroll
  for (int g = 0; g < LOADS; ++g)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void *)(lds + (wave * LOADS + g) * 1024), 16, off[g],
                                             kbytes, 0, 0);
}

// Scheduling classes of __builtin_amdgcn_sched_group_barrier.
constexpr int SG_MFMA = 0x008, SG_VMEM_READ = 0x020, SG_DS_READ = 0x100;

}  // namespace tsm
