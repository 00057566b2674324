// Host helpers shared by the files of the C-ABI layer: the per-thread error
// message and the pointer checks of every entry point.  Host code only.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "gdn.h"

namespace gdn {

// Sets gdn_last_error() of this host thread and returns s (defined in gdn_api.cpp).
gdn_status fail(gdn_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears gdn_last_error() and returns GDN_OK.
gdn_status ok();
// GDN_OK for a launch the runtime took (err 0), else GDN_ERR_LAUNCH naming `what`.
gdn_status launched(int err, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace gdn

#define GDN_NEED_PTR(p, name)                                                          \
  do {                                                                                 \
    if (!(p)) return gdn::fail(GDN_ERR_NULL, "%s: NULL, required: a device pointer", name); \
    if (!gdn::aligned16(p))                                                            \
      return gdn::fail(GDN_ERR_ALIGN, "%s: address %p, required: 16-byte aligned", name, \
                       static_cast<const void*>(p));                                   \
  } while (0)

#define GDN_NEED_PTR4(p, name)                                                         \
  do {                                                                                 \
    if (!(p)) return gdn::fail(GDN_ERR_NULL, "%s: NULL, required: a device pointer", name); \
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0)                                    \
      return gdn::fail(GDN_ERR_ALIGN, "%s: address %p, required: 4-byte aligned", name, \
                       static_cast<const void*>(p));                                   \
  } while (0)

// Debug builds check that a call's slot ids are distinct before its kernels
// (uses the enclosing entry point's dev_err and stream).
#ifdef GDN_DEBUG_CHECKS
#define GDN_DEBUG_DISTINCT(name, a, na, b, nb, kb, k_row)                                               \
  do {                                                                                                 \
    const int e_ = gdn::launch_check_distinct(a, na, b, nb, kb, k_row, dev_err, stream);               \
    if (e_ != 0)                                                                                       \
      return gdn::fail(GDN_ERR_LAUNCH, "%s: HIP launch of the slot check failed with error %d", name, e_); \
  } while (0)
#else
#define GDN_DEBUG_DISTINCT(name, a, na, b, nb, kb, k_row) \
  do {                                                  \
  } while (0)
#endif
