// Raw buffers: a load's or store's address is a lane's 32-bit byte offset plus a
// wave-uniform one from a wave-uniform base, so streams need no vector arithmetic
// for their addresses; what lies past the buffer's size reads as zeros and is not
// written, so a lane without work needs no branch.
#pragma once

#include "common.hpp"

namespace moe {

// [base, base + bytes); base and bytes wave-uniform (word 3 as for every raw
// buffer on gfx9 parts).  A wave-uniform offset has to stay within `bytes`: the
// range check compares each 4-byte word's lane offset with what is left after it,
// so the words of a load that lie before the end are read and the others are zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t raw_buffer(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t lane_off, uint32_t off = 0) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off, off, 0));
}
// 2: nontemporal (read once)
__device__ __forceinline__ u32x4 buffer_load16_nt(__amdgpu_buffer_rsrc_t r, uint32_t lane_off, uint32_t off = 0) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_off, off, 2));
}
__device__ __forceinline__ void buffer_store16(__amdgpu_buffer_rsrc_t r, uint32_t lane_off, const u32x4 &v) {
    __builtin_amdgcn_raw_buffer_store_b128(v, r, lane_off, 0, 0);
}

}  // namespace moe
