"""GB300 (sm_103a) tensor-parallel transformer MLP block: a C-ABI CUDA library
(libmlpb) and its thin ctypes binding."""
from .mlpb import *  # noqa: F401,F403
from .mlpb import (ActCheckpoint8, Join, MLPBlock, MLPBError, MLPBranch, MoEDecode,  # noqa: F401
                   load_library)
