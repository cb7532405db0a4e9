// One-line error reasons of the entry points; no CUDA headers, so that
// host-only units can include it.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "bsa.h"

namespace bsa {

// Records the reason bsa_last_error() reports on this thread.
void set_last_error(const char *msg);

inline bsa_status fail(bsa_status code, const char *fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return code;
}

inline bsa_status ok() {
    set_last_error("");
    return BSA_OK;
}

}  // namespace bsa
