"""B200-native fused sigmoid-gating Gated DeltaNet decode update.

The product is the C-ABI library ``libgdn_decode.so`` (declared in
``include/gdn_decode.h``), whose sm_100a kernel performs the whole decode /
speculative-decode state update, and beside it ``libgdn_spec.so``
(``include/gdn_spec.h``) with the other operators of a speculative step:
index arrays, probabilities, verification of drafts, commit of states.
``binding`` and ``speculative`` are thin ctypes layers that marshal torch
tensors into those ABIs; ``workloads`` draws seeded synthetic inputs.  The
bindings load their library on first use and raise if it is missing: there is
no CPU or library fallback.
"""
from __future__ import annotations

__all__ = ["decode_update", "recurrent_update", "gating", "token_probs", "verify_drafts", "commit_states",
           "step_maps", "binding", "speculative", "workloads"]


def __getattr__(name):
    # Lazy: importing the package (e.g. for ``workloads``) must not need the
    # CUDA library; calling into it must.
    if name in ("decode_update", "decode_update_host", "recurrent_update", "gating", "PreparedCall",
                "HostStagedDecode", "GdnError", "L2NORM_QK", "WRITE_INTERMEDIATE", "NO_FINAL_WRITEBACK",
                "CHECK_INDICES", "LAUNCH_PDL"):
        from . import binding
        return getattr(binding, name)
    if name in ("token_probs", "verify_drafts", "commit_states", "step_maps", "PreparedTokenProbs",
                "PreparedVerifyDrafts", "PreparedCommitStates", "PreparedStepMaps"):
        from . import speculative
        return getattr(speculative, name)
    if name in ("binding", "speculative", "workloads", "build"):
        import importlib
        return importlib.import_module(f"{__name__}.{name}")
    raise AttributeError(name)
