"""RMSNorm (and LayerNorm) forward and backward for one GB300 (sm_103a).

The compute path is the C-ABI library ``librmsnorm.so`` built from ``csrc/``
(declared in ``include/rmsnorm.h``, ``include/layernorm.h``,
``include/rmsnorm_double_backward.h`` and ``include/rmsnorm_fused.h``); ``binding`` is its thin Python front end
and ``autograd`` its PyTorch integration (``rms_norm`` / ``RMSNorm`` with
second-order gradients, ``layer_norm`` / ``LayerNorm``). ``fused`` holds the
operators around the norm: ``rms_norm_add`` (residual addition with dropout),
``rms_norm_quant`` (8-bit output) and ``rms_norm_rope`` (head norms with rotary
positions). Importing the package
loads nothing; the library is loaded on first use and a missing library is an
error.
"""
