// fp16 on the host (host_quant.cpp).
#pragma once

#include <stdint.h>

namespace qmoe {

// Nearest fp16 to a double (one rounding, ties to even; infinity beyond its range), and an fp16's value.
uint16_t f64_to_f16_rne(double x);
double f16_value(uint16_t h);

}  // namespace qmoe
