"""fp64 CPU oracle (test infrastructure only; see ``oracle.zebra`` and ``oracle.serving``)."""
from .zebra import *  # noqa: F401,F403
from . import zebra as _zebra
from .serving import *  # noqa: F401,F403
from . import serving as _serving

__all__ = list(_zebra.__all__) + list(_serving.__all__)
