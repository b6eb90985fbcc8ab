"""bit_tensor_gemm_gb300 -- low-bit integer GEMM (8-, 4- and 1-bit) for GB300.

The compute path is the CUDA library ``lib/liblbgemm.so`` (C ABI in
``include/lbgemm.h``), built in-tree by ``build.build()``; ``lbgemm`` is its
Python binding, ``synth`` draws seeded synthetic operands and
``attention_layer`` runs the attention operators between two linear layers.
"""
__all__ = ["attention_layer", "build", "lbgemm", "synth"]
