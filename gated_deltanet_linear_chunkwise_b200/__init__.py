"""B200-native (sm_100a) chunkwise gated delta rule.

The computation lives in ``libgdn_b200.so`` (C ABI declared in
``include/gdn.h``); this package re-exports a thin ctypes binding of it and
the named synthetic workloads.  Importing the package does not load the
library; the first call does, and fails loudly if it has not been built.
"""
from .binding import (GdnError, bidirectional, gdn_bwd, gdn_decode, gdn_fwd, gdn_fwd_host, gdn_packed,
                      gdn_step, last_error, load_library, seq_workspace_bytes, workspace_bytes)

__all__ = ["GdnError", "bidirectional", "gated_delta_rule", "gdn_bwd", "gdn_decode", "gdn_fwd", "gdn_fwd_host",
           "gdn_packed", "gdn_step", "last_error", "load_library", "seq_workspace_bytes", "workspace_bytes"]


def __getattr__(name):
    # the differentiable form needs torch at import time; the rest of the package does not
    if name == "gated_delta_rule":
        from .autograd import gated_delta_rule
        return gated_delta_rule
    raise AttributeError("module %r has no attribute %r" % (__name__, name))
