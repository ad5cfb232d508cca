// Root-mean-square norm's row kernels for bf16 activations (one translation unit per
// type keeps each compilation small; see taco_rms_rows.hpp for the kernels).
#include "taco_rms_rows.hpp"

template struct taco_norm::Rms<taco_norm::BF16>;
