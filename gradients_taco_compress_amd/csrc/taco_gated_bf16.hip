// Matrix products of the gated block for bf16 operands (one translation unit
// per type keeps each compilation small; see taco_gated_product.hpp).
#include "taco_gated_product.hpp"
#include "taco_gated_few.hpp"

template struct taco_gated::Products<taco_gated::BF16>;
