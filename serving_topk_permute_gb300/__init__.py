"""GB300-native (sm_103a) routed-expert MoE layer forward, and the operators around it: a C-ABI
library (libmoe.so, include/moe.h) of hand-written CUDA kernels and this thin binding."""
from .block import (LinearConfig, LinearPlan, LinearWeight, Quantized, Router, RouterConfig,  # noqa: F401
                    RouterOutput, add_rmsnorm, linear_validate, quantize, sf_size)
from .moe import (FORMATS, LayerConfig, MoeError, Plan, config_workspace_size, error_string,  # noqa: F401
                  lib, library_path, permute_noalloc, validate)
