"""GB300 training-update megakernel for a top-K-of-E mixture-of-experts
transformer: one persistent CUDA kernel per microbatch runs the forward pass,
next-token cross-entropy, backward pass, global-norm clipping and AdamW.

The compute path is the CUDA library built from ``csrc/`` (C ABI in
``include/moe_train.h``); :mod:`.binding` marshals arguments to it and
:mod:`.trainer` allocates device buffers through torch.  :mod:`.expert_ops` and
:mod:`.experts8` offer the expert layer's steps as stand-alone operators, with
8-bit products; :mod:`.block_ops` what a training step needs around them:
block norms with gate and residual, the router's choice with its balance loss,
and the gradient norm with clipping.
"""
from . import binding  # noqa: F401

__all__ = ["binding", "build", "MoETrainer", "ExpertLayer8", "expert_ops", "block_ops"]


def build(force: bool = False) -> str:
    from . import _build
    return _build.build(force=force)


def __getattr__(name):
    if name == "MoETrainer":
        from .trainer import MoETrainer
        return MoETrainer
    if name == "ExpertLayer8":
        from .experts8 import ExpertLayer8
        return ExpertLayer8
    if name in ("expert_ops", "block_ops"):
        import importlib
        return importlib.import_module("." + name, __name__)
    raise AttributeError(name)
