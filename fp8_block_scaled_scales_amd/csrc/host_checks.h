// Argument checks shared by the host sides of the calls (dg_host.hip,
// route_host.hip). No HIP call but device_ready's.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/dg.h"

namespace dg {

// The last HIP call's result on this thread, for dg_strerror.
extern thread_local hipError_t t_last_hip;

// One-time per-device check; DG_OK, DG_EUNSUPPORTED or DG_ELAUNCH.
int device_ready(int* dev_out = nullptr);

// DG_LOG=1 in the environment.
bool log_enabled();

// DG_FORCE_TILE, read at every call; -1 without it.
int forced_tile();

// Whether the byte ranges [p, p + n) and [q, q + m) share a byte (empty
// ranges share none).
inline bool overlaps(const void* p, uint64_t n, const void* q, uint64_t m) {
  const uintptr_t x = (uintptr_t)p, y = (uintptr_t)q;
  return n && m && x < y + m && y < x + n;
}

// Bytes from the first element of a [rows][cols] matrix of row pitch ld to the
// end of its last.
inline uint64_t extent(int64_t rows, int64_t cols, int64_t ld, uint64_t esize) {
  return esize * ((uint64_t)(rows - 1) * (uint64_t)ld + (uint64_t)cols);
}

inline bool known_kind(int type) { return type == DG_IN_F32 || type == DG_IN_BF16 || type == DG_IN_F16; }
inline uint64_t kind_size(int type) { return type == DG_IN_F32 ? 4 : 2; }

// A row pitch of an input: at least the row, at most DG_MAX_DIM.
inline bool good_pitch(int64_t ld, int64_t cols) { return ld >= cols && ld <= DG_MAX_DIM; }

// A range of device memory an argument takes; none when p is null.
struct Range {
  const void* p;
  uint64_t n;
};

// Whether any output overlaps an input or another output, but for the one pair
// (output `o`, input `i`) that may be the same memory (o < 0: no pair).
template <int NO, int NI>
bool clash(const Range (&outs)[NO], const Range (&ins)[NI], int o = -1, int i = -1) {
  for (int x = 0; x < NO; ++x) {
    if (!outs[x].p) continue;
    for (int y = 0; y < NI; ++y)
      if (ins[y].p && !(x == o && y == i) && overlaps(outs[x].p, outs[x].n, ins[y].p, ins[y].n)) return true;
    for (int y = 0; y < x; ++y)
      if (outs[y].p && overlaps(outs[x].p, outs[x].n, outs[y].p, outs[y].n)) return true;
  }
  return false;
}

inline bool good_dims(int64_t rows, int64_t cols) { return rows > 0 && cols > 0 && rows <= DG_MAX_DIM && cols <= DG_MAX_DIM; }
inline bool good_gran(int gran, int64_t cols) { return (gran == 64 || gran == 128 || gran == 256) && cols % gran == 0; }
inline bool misaligned(const void* p, uint64_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
// rows of 16-byte pieces: the base and the row pitch
inline bool misaligned_rows(const void* p, int64_t ld, uint64_t esize) { return p && (misaligned(p, 16) || (ld * esize) % 16); }

}  // namespace dg
