// What the entry points' argument checks share.
#pragma once

#include <cstdint>
#include <initializer_list>

#include "la_internal.h"

namespace la {

inline bool at(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// An output that is one of the inputs, or another output. (Tensors that overlap in part are not looked for.)
inline bool same(std::initializer_list<const void *> outs, std::initializer_list<const void *> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    for (const void *i : ins)
      if (*o == i) return true;
    for (auto u = outs.begin(); u != o; ++u)
      if (*o == *u) return true;
  }
  return false;
}

inline int bad(const char *fn, const char *what) {
  set_error("%s: %s", fn, what);
  return LA_ERR_INVALID_ARG;
}

}  // namespace la
