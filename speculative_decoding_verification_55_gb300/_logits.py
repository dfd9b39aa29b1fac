"""ctypes binding of the calls of include/spec_verify.h that shape a round's logits, under the same names.

Argument marshalling only, as in _binding: torch tensors supply device memory and the stream.
"""
from __future__ import annotations

from ._binding import SV_OK, SpecVerifyError, _dtype_code, _on, lib
from ._cache import _raw_stream, _small


def _launch(f, dev, stream, *args):
    import torch
    if dev.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, got {dev}")
    if torch._C._cuda_getDevice() == dev.index:
        st = f(*args, _raw_stream(stream, dev))
    else:
        with _on(dev):
            st = f(*args, _raw_stream(stream, dev))
    if st != SV_OK:
        raise SpecVerifyError(st, f.__name__)


def spec_verify_shape_logits(logits, num_positions=None, tokens=None, tree_parents=None, counts=None,
                             repetition=None, frequency=None, presence=None, bias_tokens=None, bias=None, mask=None,
                             stream=None) -> None:
    """Calls the C ABI spec_verify_shape_logits on torch tensors: penalties, biases and masks applied in place to
    logits [B, N, V] before they are verified. tokens [B, T] (T >= N - 1; a tree: T >= N) are the round's, counts
    [B, V] int16 the text's (spec_verify_count_tokens), repetition, frequency and presence [B], bias_tokens and bias
    [B, K], mask [B, N, (V + 31) // 32] or [B, 1, ...] int32. Raises SpecVerifyError on a nonzero status."""
    import torch
    if logits.dim() != 3 or not logits.is_contiguous():
        raise ValueError(f"logits must be contiguous and [B, N, V], got {tuple(logits.shape)}")
    B, N, V = logits.shape
    dev, i32, f32 = logits.device, torch.int32, torch.float32
    T = K = P = 0
    if tokens is not None:
        if tokens.dim() != 2:
            raise ValueError(f"tokens must be [{B}, T], got {tuple(tokens.shape)}")
        T = tokens.shape[1]
    if (bias_tokens is None) != (bias is None):
        raise ValueError("bias_tokens and bias go together")
    if bias is not None:
        if bias.dim() != 2:
            raise ValueError(f"bias must be [{B}, K], got {tuple(bias.shape)}")
        K = bias.shape[1]
    if mask is not None:
        if mask.dim() != 3 or mask.shape[1] not in (1, N):
            raise ValueError(f"mask must be [{B}, {N} or 1, {(V + 31) // 32}], got {tuple(mask.shape)}")
        P = mask.shape[1]
    _launch(lib().spec_verify_shape_logits, dev, stream, logits.data_ptr(),
            _small(num_positions, "num_positions", i32, (B,), dev), _small(tokens, "tokens", i32, (B, T), dev), T,
            _small(tree_parents, "tree_parents", i32, (B, N), dev), _small(counts, "counts", torch.int16, (B, V), dev),
            _small(repetition, "repetition", f32, (B,), dev), _small(frequency, "frequency", f32, (B,), dev),
            _small(presence, "presence", f32, (B,), dev), _small(bias_tokens, "bias_tokens", i32, (B, K), dev),
            _small(bias, "bias", f32, (B, K), dev), K, _small(mask, "mask", i32, (B, P, (V + 31) // 32), dev), P,
            B, N, V, _dtype_code(logits))


def spec_verify_count_tokens(tokens, num, counts, prompt=False, stream=None) -> None:
    """Calls the C ABI spec_verify_count_tokens on torch tensors: the first num[b] (None: all) of tokens [B, M] go
    into counts [B, V] int16, as the row's output or as its prompt. Raises SpecVerifyError on a nonzero status."""
    import torch
    if tokens.dim() != 2 or counts.dim() != 2:
        raise ValueError(f"tokens must be [B, M] and counts [B, V], got {tuple(tokens.shape)} and {tuple(counts.shape)}")
    B, M = tokens.shape
    dev, V = counts.device, counts.shape[1]
    _launch(lib().spec_verify_count_tokens, dev, stream, _small(tokens, "tokens", torch.int32, (B, M), dev),
            _small(num, "num", torch.int32, (B,), dev), _small(counts, "counts", torch.int16, (B, V), dev),
            1 if prompt else 0, B, M, V)
