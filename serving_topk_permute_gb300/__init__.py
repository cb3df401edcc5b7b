"""GB300-native (sm_103a) routed-expert MoE layer forward, and the operators around it: a C-ABI
library (libmoe.so, include/moe.h) of hand-written CUDA kernels and this thin binding."""
from .block import (LinearConfig, LinearPlan, LinearWeight, Quantized, Router, RouterConfig,  # noqa: F401
                    RouterOutput, add_rmsnorm, linear_validate, quantize, sf_size)
from .moe import (FORMATS, LayerConfig, MoeError, Plan, config_workspace_size, error_string,  # noqa: F401
                  lib, library_path, permute_noalloc, validate)
from .score_router import ScoreRouter, ScoreRouterConfig  # noqa: F401
from .sandwich import (SandwichGrads, sandwich_norm, sandwich_norm_backward,  # noqa: F401
                       sandwich_norm_workspace_size)
from .int4 import Int4LinearConfig, Int4LinearPlan, Int4LinearWeight, int4_validate  # noqa: F401
