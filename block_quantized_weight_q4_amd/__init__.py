"""Block-quantized weight products on MI355X: ggml Q4_0 / Q4_K / Q5_K / Q6_K, and
e4m3 with a scale for each 128 x 128 block (``gq_f8_*``), and 4 bits with a scale
for each group of inputs (``gq_g4_*``); routing, and tokens sorted by expert
(``gq_expert_*``).

The compute lives in ``libgq.so`` (HIP kernels for gfx950 behind the C ABI of
``include/gq.h``, ``gq_f8.h``, ``gq_g4.h`` and ``gq_expert.h``); :mod:`._binding` is a thin ctypes layer with the
same entry point names that marshals torch tensors (device memory, streams) into it.

The binding is loaded on first use, so ``block_quantized_weight_q4_amd.synth``
(the seeded input generator) can be imported without the library.
"""
import importlib
import sys
import types

__all__ = [
    "gq_abi_version", "gq_block_info", "gq_dequant", "gq_matvec", "gq_matvec_id",
    "gq_matvec_id_workspace", "gq_matvec_id_check", "gq_matmul", "gq_route_topk", "gq_matvec_glu",
    "gq_matvec_id_glu", "gq_matvec_id_noalloc", "gq_route_topk_plan", "gq_route_matvec_id_glu",
    "gq_f8_quant", "gq_f8_glu_quant", "gq_f8_matvec", "gq_f8_matmul", "gq_f8_matmul_id", "gq_f8_matmul_id_workspace",
    "gq_f8_matmul_id_check", "gq_route_scored", "gq_g4_matvec", "gq_g4_matmul", "gq_g4_matmul_dx", "gq_expert_sort",
    "gq_expert_gather", "gq_expert_combine", "gq_expert_combine_grad", "GqError", "TYPES", "lib_path",
]


class _Package(types.ModuleType):
    pass


class _FromBinding:
    """An entry point, looked up in the binding at every use (0.15 us; a module's
    __getattr__ takes 0.5), so that a replaced one is found."""

    def __init__(self, name):
        self.name = name

    def __get__(self, package, _):
        module = package.__dict__.get("_binding")
        if module is None:
            module = importlib.import_module(package.__name__ + "._binding")  # (sets package._binding)
        return getattr(module, self.name)


for _name in __all__:
    setattr(_Package, _name, _FromBinding(_name))
sys.modules[__name__].__class__ = _Package
