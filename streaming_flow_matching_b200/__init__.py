"""Performer next-unit flow-matching denoise step on B200: Python binding of libsfm.

Importing this package loads libsfm.so (built in-tree by
``python streaming_flow_matching_b200/build.py``) and fails if it is missing.
"""
from . import _lib
from ._lib import SfmError, lib  # noqa: F401
from .performer import Performer, attention, attention_workspace_bytes, euler_update, linear  # noqa: F401
from .paged import (attention_bounds, attention_masked, paged_append, paged_attention,  # noqa: F401
                    paged_evict)

__all__ = ["Performer", "attention", "attention_workspace_bytes", "euler_update", "linear", "SfmError",
           "lib", "attention_bounds", "attention_masked", "paged_append", "paged_attention", "paged_evict"]
