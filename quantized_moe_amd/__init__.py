"""MI355X-native W4A16 mixture-of-experts layer (HIP for gfx950), with the
router in front of it, its 8-bit floating point form, and the norms and 16-bit
products of the block around it.

``quantized_moe_amd.chord`` binds the C ABI of ``libchord.so``
(``include/chord.h``); ``quantized_moe_amd.build`` compiles it in-tree.
"""

__all__ = ["chord", "build"]
