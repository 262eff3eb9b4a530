// api_checks.h -- argument checks of the C ABI's head-wise calls (one per
// translation unit: everything has internal linkage).
#pragma once

#include <cstdarg>
#include <cstdio>

#include <nvtx3/nvToolsExt.h>

#include "kernels.h"
#include "varlen_ssm.h"

namespace {

using namespace vssm;

struct Range {
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
};

int bad(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return record_error(code, buf);
}

int check(cudaError_t e, const char* what) {
  return e == cudaSuccess ? VSSM_OK : bad(VSSM_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define TRY(expr)                   \
  do {                              \
    const int rc_ = (expr);         \
    if (rc_ != VSSM_OK) return rc_; \
  } while (0)

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_dtype(vssm_dtype dt, IO* io) {
  if (dt != VSSM_F32 && dt != VSSM_BF16) return bad(VSSM_ERR_DTYPE, "dtype %d is neither VSSM_F32 nor VSSM_BF16", (int)dt);
  *io = dt == VSSM_F32 ? IO::F32 : IO::BF16;
  return VSSM_OK;
}

// A tensor that has to be there when the call has rows.
int check_ptr(const void* p, const char* name, bool needed) {
  if (!p) return needed ? bad(VSSM_ERR_ARG, "%s is NULL", name) : VSSM_OK;
  return al16(p) ? VSSM_OK : bad(VSSM_ERR_ALIGN, "%s is not 16-byte aligned", name);
}

int check_stride(int64_t stride, int64_t row, IO io, const char* name) {
  if (stride < row) return bad(VSSM_ERR_ARG, "%s %lld is below the row's %lld values", name, (long long)stride, (long long)row);
  if (stride % (16 / io_bytes(io))) return bad(VSSM_ERR_ALIGN, "%s %lld is not a multiple of 16 bytes", name, (long long)stride);
  return VSSM_OK;
}

int check_room(const void* p, size_t have, size_t need, const char* name) {
  if (have < need) return bad(VSSM_ERR_WORKSPACE, "%s has %zu bytes, needs %zu", name, have, need);
  if (!p) return bad(VSSM_ERR_WORKSPACE, "%s is NULL", name);
  return al16(p) ? VSSM_OK : bad(VSSM_ERR_ALIGN, "%s is not 16-byte aligned", name);
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace
