"""GB300-native Periodic Row-wise Muon (PR-Muon) and MuonBP optimizer step.

Next to the optimizer, the operators of a transformer block whose parameters
it updates, forward and backward: the gated feed-forward block, the norms
around a block and the token embedding.

The compute lives in libprm.so (CUDA kernels for sm_103a behind a C ABI,
declared in include/prm.h and include/prm_blocks.h); this package only binds it. Build the library
with `python -m matrix_aware_optimizer_gb300.build`.
"""
from . import native  # noqa: F401
from .native import PrmError, prm_branch  # noqa: F401


_BLOCKS = ("gated_ffn", "gated_ffn_backward", "block_norm", "block_norm_backward", "embedding",
           "embedding_backward", "blocks_sync_status")


def __getattr__(name):
    # torch is only needed by the tensor-level API; keep `import` cheap.
    if name in ("PeriodicRowMuon", "newton_schulz", "adamw_step"):
        from . import optimizer as module
    elif name in _BLOCKS:
        from . import blocks as module
    else:
        raise AttributeError(name)
    value = globals()[name] = getattr(module, name)
    return value
