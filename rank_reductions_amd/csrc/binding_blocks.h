// The block operators' part of the Python module _rows.
#pragma once

#include "binding.h"

namespace rows_binding {
extern PyMethodDef block_methods[];  // ends with a null entry
}
