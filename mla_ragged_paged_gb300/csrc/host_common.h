// Host-side helpers shared by the entry points: per-thread error text, the
// device capability check and the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdint>

#include "../../include/mla_prefill.h"

namespace mla {

// Record a failure for mla_last_error_string() and return `status`.
mla_status_t fail(mla_status_t status, const char* fmt, ...);
mla_status_t ok();

// Current device must be compute capability 10.3.  Fills the SM count.
mla_status_t check_device(int* device_out, int* num_sms_out);

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against libcuda).  Returns MLA_ERR_CUDA when the encoder rejects the map.
mla_status_t encode_tiled(CUtensorMap* map, CUtensorMapDataType dtype, uint32_t rank, void* base,
                          const uint64_t* dims, const uint64_t* strides_bytes,
                          const uint32_t* box, CUtensorMapSwizzle swizzle, const char* what);

bool aligned16(const void* ptr);
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Descriptor checks: non-NULL data, rank, dtype, shapes in [0, 2^31),
// non-negative strides, innermost stride 1.  empty_ok: a tensor without
// elements may have NULL data.
mla_status_t check_tensor(const mla_tensor_t* t, const char* name, int ndim, mla_dtype_t dtype,
                          bool empty_ok = false);

// Allow `bytes` of dynamic shared memory for `func` on `device`, cached per
// (device, slot), the same `bytes` in every call of a slot (calls of several threads are
// not ordered): each kernel needs a slot of its own (0 plan, 1 scheduler,
// 2 / 3 / 4 attention bf16 / fp8 / fp8 with per-token K scales, 6 / 7 the last
// two with two-term precision, 5 up-projection, 8 / 12 fp8 product, 9 .. 11 its
// form for few tokens, 13 / 14 latent decode, 15 / 18 / 20 / 21
// norm and rotation, 16 / 17 / 19 latent decode over 4-bit rows).
constexpr int kSmemSlots = 22;
mla_status_t set_max_dynamic_smem(const void* func, int bytes, int device, int slot);

// A kernel that moves registers between its warps (setmaxnreg) may only run as
// built with exactly `regs` registers per thread; cached per (device, slot).
mla_status_t check_registers(const void* func, int regs, int device, int slot);

// What a 4-bit cache [num_pages, P, row bytes] has to keep: alignment, and rows apart.
mla_status_t check_fp4_cache(const mla_tensor_t* cache);

// What mla_decode_latent and mla_decode_latent_fp4 ask of everything but their caches.
mla_status_t check_decode_operands(const mla_tensor_t* out, const mla_tensor_t* lse, const mla_tensor_t* q,
                                   const mla_tensor_t* page_table, const uint32_t* row_offsets, const uint32_t* cache_lens,
                                   float scale, mla_mask_t mask, const uint32_t* status, const void* workspace,
                                   size_t workspace_bytes);

// What the test hooks mla_test_inject_stall and mla_test_delay_softmax ask of launches.
uint32_t test_stall();
uint32_t test_delay_ns();

}  // namespace mla
