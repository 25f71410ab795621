"""MI355X-native ZeRO-1 shard optimizer step.

The work is done by ``libz1.so`` (HIP for gfx950, C ABI in ``include/z1.h``
and ``include/z1_ops.h``); ``binding`` and ``ops`` marshal torch tensors into
it, ``shard`` and ``muon`` wire one rank's buffers together, ``workloads``
defines the synthetic parameter lists.
"""
__all__ = ["binding", "ops", "shard", "muon", "workloads", "build"]
