// qg_error.h -- the thread's last error message (qg_last_error), shared by the
// translation units that implement the C ABI.
#pragma once
#include "../../include/qgemv.h"

namespace qg {
// set the message and return st
qg_status fail(qg_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_error();
// QG_OK and the current device, or QG_ERR_UNSUPPORTED where it is no gfx950
qg_status check_device(int* dev);
}  // namespace qg
