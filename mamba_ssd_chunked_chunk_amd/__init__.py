"""libssd: Mamba-2 SSD varlen chunked scan (forward prefill) for AMD MI355X,
linear attention with a fixed decay per head (forward, backward, single
tokens; ``linear_attention`` is the differentiable function), parking of
either's states in 8 bits, and what stands around a mixer: the norm, the short
convolution and the selective scan with a decay per channel and state (forward,
backward, single tokens; ``mixer`` has the differentiable functions).

The compute path is the HIP library ``libssd.so`` (built for gfx950) behind
the C ABI declared in ``include/ssd.h``; ``binding`` marshals torch tensors
into that ABI.  Importing this package does not load the library; the first
call does, and raises if it is missing (there is no CPU fallback).
"""

__all__ = ["workloads"]
