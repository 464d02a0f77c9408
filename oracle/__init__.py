"""fp64 CPU oracle of the retention operator, its gated layer and the operators around it -- test infrastructure only.

Only ``tests/``, ``__graft_entry__.smoke()`` and ``bench.py``'s CPU-baseline leg may
import this package.  It shares no code with the HIP library and imports nothing from
it.  Pins: every public function is checked in ``tests/test_oracle.py`` against exact
rational arithmetic, closed forms, textbook special cases and hand-worked fixtures
(``tests/golden/``), in ``tests/test_oracle_msr.py`` and ``tests/test_oracle_block.py``; no function here is "parity unpinned".
"""
from .retention_oracle import *  # noqa: F401,F403
from .retention_oracle import __all__ as _ops_all
from .msr_oracle import *  # noqa: F401,F403
from .msr_oracle import __all__ as _msr_all
from .block_oracle import *  # noqa: F401,F403
from .block_oracle import __all__ as _block_all

__all__ = list(_ops_all) + list(_msr_all) + list(_block_all)
