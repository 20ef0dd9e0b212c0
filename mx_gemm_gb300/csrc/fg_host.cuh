// Host helpers of the C ABI that its translation units share (defined in
// fg_api.cu): error reporting, argument checks and tensor-map set-up.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/fg.h"

namespace fg {

// Record the message of fg_last_error_message and return the status.
fg_status fail(fg_status s, const char* fmt, ...);
fg_status cuda_fail(cudaError_t e, const char* what);

bool aligned(const void* p, uintptr_t a);
bool mode_ok(int mode);
const char* mode_name(int mode);
fg_status check_nk(int mode, int64_t N, int64_t K);
fg_status check_arch();
fg_status check_desc(const fg_bshuf* d);

// Device address of the error word of the current device, the limit of every
// wait inside a kernel, and a tag no other call of this process gets.
uint32_t* dev_error_ptr();
uint64_t wait_timeout_ns();
uint64_t next_epoch();

// Byte-typed 2-D map of [rows][row bytes], boxes of box_rows x 128 bytes in
// the 128-byte swizzle; a plain map of whole rows (at most 2048 bytes) in
// 8-byte elements; and the 3-D map of an fp4 weight image.
fg_status make_tmap(CUtensorMap* map, const void* base, int64_t rows, int64_t rbytes, uint32_t box_rows);
fg_status make_tmap_rows(CUtensorMap* map, const void* base, int64_t rows, uint32_t rbytes, uint32_t box_rows);
fg_status make_tmap_fp4w(CUtensorMap* map, const void* base, int64_t N, int64_t K);

}  // namespace fg
