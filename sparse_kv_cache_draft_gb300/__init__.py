"""okv: lookahead sparse KV staging and sparse decode attention on one GB300 (sm_103a).

The compute path is the CUDA library ``libokv.so`` (C ABI in ``include/okv.h``); this
package is its Python binding (argument marshalling only). There is no CPU fallback: if the
library is missing, :func:`load_library` (called by every :class:`Context`) raises ImportError.
"""
from . import binding
from .binding import BF16, F32, Config, Context, HostBuffer, OkvError, library_path, load_library  # noqa: F401


def __getattr__(name: str):
    """Rotary, norm_rope, append_qkv_static and attend_tree_static, which load torch."""
    if name.startswith("_") or name not in binding._CALLS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    value = getattr(binding, name)
    globals()[name] = value
    return value
