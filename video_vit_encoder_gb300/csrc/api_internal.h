// What the translation units that hold C entry points share.
#pragma once
#include "jepa_gb300.h"

namespace jepa {

// Records the message that jepa_last_error() returns to this thread; returns st.
jepa_status api_fail(jepa_status st, const char* fmt, ...);
// The current device's status word of the single operations.
jepa_status api_ops_status(int** out);

}  // namespace jepa
