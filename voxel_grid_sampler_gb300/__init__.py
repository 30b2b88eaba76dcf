"""GB300-native fused registration objective of FFDP (single GPU, sm_103a), and
the operators of a network over volume tokens that is trained through it.

The compute lives in libffdp (CUDA, C ABI in include/ffdp.h); ``ffdp`` is its
ctypes binding, ``synth`` makes the seeded synthetic volume pairs and
``build`` compiles the library and ``learned`` is a small registration network
on the token operators.
"""
from . import ffdp  # noqa: F401
from .ffdp import (FfdpError, ffdp_attention_bwd, ffdp_attention_fwd, ffdp_grid_sample_bwd,  # noqa: F401
                   ffdp_grid_sample_fwd, ffdp_linear_bwd, ffdp_linear_fwd, ffdp_lncc_fwd_bwd, ffdp_mi_fwd_bwd,
                   ffdp_objective, ffdp_rope_bwd, ffdp_rope_fwd, ffdp_workspace_bytes)
