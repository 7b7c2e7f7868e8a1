"""GB300-native DFlash draft attention: a C-ABI CUDA library for sm_103a
(include/dflash_attn.h) and its thin Python binding."""
from .dflash_attn import (DFlashAttention, DFlashError, DraftCache,  # noqa: F401
                          DecoderMLP, KVGroup, PagedCache, Q8Cache, clip_grad_norm,
                          declared_functions, grad_norm, lib, linear_cross_entropy,
                          linear_cross_entropy_grad, verify_draft)
