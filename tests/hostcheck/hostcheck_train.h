// Shared by the stubs and the driver of the training operators' sanitizer build.
#pragma once
#include "hostcheck.h"

namespace hostcheck {
long train_launches();   // launches of the training operators so far
}
