"""Float64 CPU oracle of the KronQ layer-quantization path (test infrastructure only)."""
from . import kronq as _kronq
from . import microscale as _microscale
from .kronq import *  # noqa: F401,F403
from .microscale import *  # noqa: F401,F403

__all__ = list(_kronq.__all__) + list(_microscale.__all__)
