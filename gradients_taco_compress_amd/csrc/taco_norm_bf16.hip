// Layer norm row kernels for bf16 activations (one translation unit per type
// keeps each compilation small; see taco_norm_rows.hpp for the kernels).
#include "taco_norm_rows.hpp"

template struct taco_norm::Rows<taco_norm::BF16>;
