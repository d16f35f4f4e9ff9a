// Internal (not part of the C ABI): what the operators' host sides share.
#pragma once
#include "fwd_ws.h"
#include "moe.h"
#include "spans.h"

constexpr int64_t I32_MAX = 0x7fffffff;
constexpr long MAX_BLOCKS = (1L << 24) - 1;     // of 256 threads: a launch holds fewer than 2^32

inline int bad(int code, const char* msg) {
  moe_set_thread_error(msg);
  return code;
}

inline int launched() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? MOE_OK : bad(MOE_E_HIP, hipGetErrorString(e));
}

inline int shared() { return bad(MOE_E_INVAL, "an output shares memory with an input or another output"); }

inline int elem_bytes(int dt) { return dt == MOE_T_F32 ? 4 : (dt == MOE_T_BF16 || dt == MOE_T_F16 ? 2 : 0); }
