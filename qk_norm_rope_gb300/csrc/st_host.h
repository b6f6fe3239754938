// Host-side helpers shared by the C-ABI layers (argument checks, error
// reporting, launch accounting, tensor-map encoding).
#pragma once
#include <cstdint>

#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "st_aux.h"
#include "st_common.cuh"
#include "st_rope_attn.h"

namespace st {

// Records the calling thread's error message and returns `s`.
st_status fail(st_status s, const char* fmt, ...);
void clear_error();
st_status cuda_check(cudaError_t e, const char* what);

int elem_bytes(int dt);
bool aligned16(const void* p);
long long wait_budget();

struct Dev {
  unsigned* status = nullptr;
  unsigned long long* counters = nullptr;
};
st_status device_globals(Dev* d);

// Launch accounting: a launch is counted and, when timing is on, bracketed
// with events on its stream.
struct LaunchMark {
  cudaEvent_t a = nullptr, b = nullptr;
};
LaunchMark launch_begin(cudaStream_t stream);
void launch_end(const LaunchMark& m, int kind, cudaStream_t stream, cudaError_t e);

// Launches one kernel through `fn`, counting it and, when timing is on,
// bracketing it with events on its stream.
template <class F>
cudaError_t launch_counted(int kind, cudaStream_t stream, F&& fn) {
  const LaunchMark m = launch_begin(stream);
  const cudaError_t e = fn();
  launch_end(m, kind, stream, e);
  return e;
}

constexpr unsigned bit(int dt) { return 1u << dt; }

// A [B, S, H, D] tensor whose dtype is one of `dts` (a set of bit(st_dtype)).
st_status check_bshd(const st_tensor* t, const char* name, int B, int S, int H, int D, unsigned dts, RowTensor* out);
// An fp32 [D] vector, contiguous.
st_status check_vec(const st_tensor* t, const char* name, int D);

// The rotation source of q or of k: position ids (t), or in the table form
// the caller's cos (t) and sin tables.
struct Ids {
  const st_tensor* t;
  int Bt, S;
  const st_tensor* sin = nullptr;
  bool table = false;
};
st_status check_ids(const st_tensor* t, const char* name, int B, int S, int n_axes, Ids* out);
st_status check_tables(const st_tensor* c, const st_tensor* sn, const char* name, int B, int S, Ids* out);
// Axis widths and theta of the position-id form (widths must sum to D).
st_status check_axes(const st_rope* rope, int D);
void fill_ids(const Ids& ids, TableParams* t);  // the position-id form's tensor
void fill_table(const Ids& ids, const st_rope* rope, float2* out, __half2* out16, unsigned* ctrl, TableParams* t);

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
st_status encode_rows_map(const st_tensor* t, CUtensorMap* map, int* s_first, int box_rows = kTile);

}  // namespace st
