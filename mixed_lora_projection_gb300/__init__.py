"""Shared-base, per-request LoRA projection on one GB300 (sm_103a).

    Y[t,:] = X[t,:] W^T + s_a (X[t,:] A_a^T) B_a^T   for rows of requests naming adapter a
    Y[t,:] = X[t,:] W^T                              for rows of requests naming none

The compute runs in the C-ABI library ``liblora_linear.so`` (hand-written sm_103a
kernels); this package is a thin ctypes binding around it. Importing the package does
not load the library; ``LoraLinear`` and ``plan`` do, and raise if it is missing.

Between the projections of an adapted layer: ``add_rms_norm`` and ``add_rms_norm_fp8`` (the
residual's addition with the norm), ``kv_append`` (new keys and values into a paged cache, with
the rotary turn), ``PagedAttention`` (the batch's new rows over that cache) and ``silu_mul`` (the gated
activation). ``LoraLinear.forward_fp8`` takes 8-bit activations, which ``add_rms_norm_fp8``,
``silu_mul_fp8`` and ``fp8_rows`` write, and a weight from ``fp8_blocks``; behind the last projection
``token_logprobs`` scores given tokens.
"""
from .synth import WORKLOADS, Workload, make_inputs  # noqa: F401


def __getattr__(name):
    # (once a name: a call of a decode step takes a few microseconds, a look-up through here more than one)
    if name in ("LoraLinear", "plan", "LoraError", "validate", "w4_repack", "launch_shape", "host_chunks", "k_split"):
        from . import lora_linear as module
    elif name in ("add_rms_norm", "add_rms_norm_fp8", "kv_append", "PagedAttention", "silu_mul", "silu_mul_fp8", "fp8_rows",
                  "fp8_blocks", "token_logprobs", "TokenLogprobs"):
        from . import layer as module
    else:
        raise AttributeError(name)
    globals()[name] = value = getattr(module, name)
    return value
