"""GB300-native W8A8 block-FP8 linear layer (1x128 activation / 128x128 weight scales).

The compute lives in ``libfp8act.so`` (hand-written CUDA for sm_103a behind a
C ABI, declared in ``include/fp8act.h``): the linear layer, and the operators
between linear layers of a decoder (norm, gated activation, paged E4M3 cache and
attention over it, verification of drafted tokens).
``block_scaled_fp8_act_gb300.fp8act`` is the thin binding (ctypes, and a small
extension module for the operators); importing this package does not load the
library.
"""
