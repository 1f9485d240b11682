"""GB300-native Gaussian Mixture Attention (GMA) forward pass.

The compute lives in ``libgma.so`` (hand-written sm_103a CUDA behind a C ABI, declared in
``include/gma.h``); ``linear_latent_routing_gb300.gma`` is the thin ctypes binding over it.
``ssm`` and ``norm`` bind the operators that stand next to the mixer in a block (the selective state
space scan with its short convolution, and the norms around a block; ``include/gma_block.h``).
The bindings are imported on demand so that host-only code (input generation) works without a
built library; they raise if the library is missing.
"""
__all__ = ["gma", "inputs", "norm", "ssm"]
