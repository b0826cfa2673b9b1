"""MI355X (gfx950) fast-weight prefill of In-Place Test-Time Training.

The compute path is libipttt.so (hand-written HIP kernels behind a C ABI,
include/ipttt.h); `ipttt` is its ctypes binding. Importing the binding does not
load the library; the first call does, and fails loudly if it is not built. `block` holds
the operators around the layer (norm, recurrence, feed-forward block;
include/ipttt_block.h), `attention` those of the attention beside it
(include/ipttt_attention.h).
"""
from . import attention, block, ipttt  # noqa: F401
from .ipttt import Layer, IptttError  # noqa: F401
