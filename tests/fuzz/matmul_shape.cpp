// The product's choice of kernel, for tests without a GPU.
#include "matmul_shape.hpp"

extern "C" int matmul_shape(const rs_fp8_matmul* mm, int gathered) { return int(rs::matmul_shape(*mm, gathered != 0)); }
