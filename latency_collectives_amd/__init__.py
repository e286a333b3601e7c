"""Barrier-free small/medium-message AllReduce (sum) for N ranks emulated on one MI355X.

The compute path is the HIP library ``libar.so`` (sources in ``csrc/``, C ABI in
``include/ar.h``); :mod:`latency_collectives_amd._ar` is its ctypes binding. Nothing in this
package computes an AllReduce on the CPU. What a tensor-parallel rank computes between two
AllReduces of a decode step over its own heads (page tables, norm and rotation of q and k, a
4-bit paged cache and the attention over it) is in ``include/ar_decode.h`` and
:mod:`latency_collectives_amd._decode`; an 8-bit cache with its attention, sharing, freeing and moving
pages, and attention over packed prompts are in ``include/ar_serving.h`` and
:mod:`latency_collectives_amd._serving`.
"""

from ._ar import *  # noqa: F401,F403
from ._ar import ArError, lib  # noqa: F401
from . import _decode
from ._decode import *  # noqa: F401,F403
from . import _serving
from ._serving import *  # noqa: F401,F403


def __getattr__(name):
    # the compiled calls load with their first use
    for module, names in ((_decode, _decode.DECODE_EXPORTS), (_serving, _serving.SERVING_EXPORTS)):
        if name in names:
            globals()[name] = getattr(module, name)
            return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
