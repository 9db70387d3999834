// gemm_epilogue.hip -- gemm.hip's products followed by bias, activation,
// multiplier and residual (namespace fp4::epi).
#define FP4_EPILOGUE_FORM 1
#include "gemm.hip"
