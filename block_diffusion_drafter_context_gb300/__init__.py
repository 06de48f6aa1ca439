"""GB300-native (sm_103a) DFlash block-diffusion drafting step.

The hot path lives in libdflash.so (hand-written CUDA behind the C ABI of
include/dflash.h); ``binding`` exposes those calls under their C names and
``drafter`` adds weight packing, the paged KV cache and a small object
wrapper; ``target`` does the same for the operators of the target model's
pass (append to the paged cache, attention over it, token log probabilities).  Nothing here computes the method on the host.
"""
from . import binding  # noqa: F401
from .binding import DflashError, load  # noqa: F401

__all__ = ["binding", "drafter", "target", "DflashError", "load"]


def __getattr__(name):
    # ``drafter`` and ``target`` on first use; importing them by their full
    # name keeps ``from block_diffusion_drafter_context_gb300 import drafter``
    # from re-entering this hook
    if name in ("drafter", "target"):
        import importlib
        return importlib.import_module(__name__ + "." + name)
    raise AttributeError(name)
