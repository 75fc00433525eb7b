// Shared by the stubs and the driver of the sanitizer build of the operators that close a training step.
#pragma once
#include "hostcheck.h"

namespace hostcheck {
long step_launches();   // launches of these operators so far
}
