"""B200-native (sm_100a) chunked write-and-read of the Titans neural memory.

The compute lives in libtitansmem.so (CUDA, C ABI in include/titansmem.h);
this package is its thin Python binding.
"""
from .memory import NeuralMemory, prologue  # noqa: F401
from ._native import TitansMemError  # noqa: F401
from .mixer import (group_norm, group_norm_backward, selective_scan, selective_scan_backward,  # noqa: F401
                    selective_scan_step, short_conv, short_conv_backward, short_conv_step)
