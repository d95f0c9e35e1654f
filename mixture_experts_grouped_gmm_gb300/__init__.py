"""GB300-native Mixture-of-Experts grouped GEMM (sm_103a).

The compute path is libmgemm.so (hand-written CUDA for sm_103a, C ABI in
include/mgemm.h); ``binding`` marshals torch tensors into it and ``gmm``
wraps forward/backward as an autograd op; ``fp4`` holds the 4-bit
block-scaled tensors and their grouped product, ``moe`` the routers and the
routed layers.  ``workloads`` draws the seeded synthetic inputs.
"""

from . import binding, moe  # noqa: F401
from .fp4 import Fp4Tensor, dequantize_fp4, gmm_fp4, quantize_fp4  # noqa: F401
from .gmm import gmm, gmm_fp8  # noqa: F401
