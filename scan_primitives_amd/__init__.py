"""MI355X-native scan primitives: element-scan, matrix-scan, linear-scan and table-scan on gfx950,
the operators of a linear-attention layer (decay attention, head norm and rotation), and those of a layer on a
selective state space (causal convolution, selective scan, group norm).

The computation lives in ``libsx_scan.so`` (hand-written HIP kernels behind
the C ABI in ``include/sx_scan.h``); this package is its Python binding.
PyTorch provides device memory and streams.
"""

from ._binding import (BODIES, SxError, causal_conv, causal_conv_backward, causal_conv_step, cumsum, decay_attention,
                       decay_attention_backward, decay_attention_step, element_scan, element_scan_backward, group_norm,
                       group_norm_backward, head_norm_rotate, head_norm_rotate_backward, linear_scan, load_library,
                       matrix_scan, matrix_scan_backward, matrix_scan_status, rotation_turns, selective_scan,
                       selective_scan_backward, selective_scan_step, set_lookback_spin_limit, table_scan)

__all__ = ["BODIES", "SxError", "element_scan", "element_scan_backward", "matrix_scan", "matrix_scan_backward",
           "linear_scan", "cumsum", "table_scan", "decay_attention", "decay_attention_backward", "decay_attention_step",
           "head_norm_rotate", "head_norm_rotate_backward", "rotation_turns", "causal_conv", "causal_conv_backward",
           "causal_conv_step", "selective_scan", "selective_scan_backward", "selective_scan_step", "group_norm",
           "group_norm_backward", "load_library", "matrix_scan_status", "set_lookback_spin_limit"]
__version__ = "0.1.0"
