"""fp64 definitions of the linear, rotary and dropout operators for their tests:
plain torch in float64, gradients by autograd, and the generator's words in
numpy's 64-bit integers."""

import numpy as np
import torch

from block_reference import act


def philox_words(index, seed, offset):
    """Four 32-bit words (..., 4) of Philox4x32-10's blocks with counters
    (index, offset) and key seed, index an array of 64-bit numbers."""
    low = np.uint64(0xFFFFFFFF)
    index = np.asarray(index, dtype=np.uint64)
    c = [index & low, index >> np.uint64(32), np.full_like(index, offset & 0xFFFFFFFF), np.full_like(index, offset >> 32)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=-1)


def kept(shape, p, rng, device="cuda", first=0):
    """Which of the elements from number `first` (a multiple of four) on stay."""
    n = int(np.prod(shape))
    words = philox_words(np.arange(first // 4, first // 4 + (n + 3) // 4, dtype=np.uint64), *rng).reshape(-1)[:n]
    return torch.from_numpy(words >= round(p * 2 ** 32)).view(shape).to(device)


def drop(x, p, rng):
    if p == 0.0:
        return x
    if p == 1.0:
        return torch.zeros_like(x)
    return torch.where(kept(tuple(x.shape), p, rng, x.device), x / (1.0 - p), 0.0)


def acted(z, kind):
    return z if kind == "none" else act(z, kind)


def linear(x, w, bias, residual, kind, p, rng):
    """(y, z) in float64; dropout by the number of an element in y."""
    z = x @ w.T
    if bias is not None:
        z = z + bias
    y = drop(acted(z, kind), p, rng)
    return (y if residual is None else residual + y), z


def rotary(x, freqs, positions, interleaved=False, scale=1.0, inverse=False):
    """x (batch, len, heads, dim) turned; positions (batch or 1, len, axes)."""
    pairs = freqs.shape[1]
    t = positions.double() @ freqs.double()
    t = (-t if inverse else t)[:, :, None]
    cos, sin = torch.cos(t) * scale, torch.sin(t) * scale
    y = x.clone()
    a, b = (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)) if interleaved else (slice(0, pairs), slice(pairs, 2 * pairs))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y
