"""Fused FP16 MLP inference on MI355X (gfx950): a C-ABI HIP library, its thin Python binding
(``binding``) and the torch form of its single operators (``ops``, and ``ops_fp8`` for 8-bit operands)."""
