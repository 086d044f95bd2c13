"""Comparison of the serving operators' outputs with fp64 references, and the references themselves.

Tolerances, from the arithmetic (u = 2^-24, the fp32 unit roundoff):
  * rounding to bf16 (8 significant bits, nearest) is at most 2^-8 of the value, to e4m3 at most 2^-4 of a normal value and half a
    step of 2^-9 below 2^-6 (times the scale);
  * the recurrence in fp32: a token's update of an element takes about 24 roundings (16 products in
    sequence, 3 shuffles, the update itself), statistically 5 u of the state's size; the updates are
    contractions, so over 100 tokens the errors add up to at most 100 x 5 u, as independent ones to
    10 x 5 u = 3e-6.  Bound: 1e-5 of the tensor's largest magnitude;
  * the convolution, norms and gates in fp32: at most 20 roundings and hardware exponentials of a few
    parts in 10^7.  Bound: 4e-6 of the value, or of the head's (row's) largest for what is summed there.
"""
from __future__ import annotations

import numpy as np
import torch

FP32_STATE = 1e-5
FP32_VALUE = 4e-6


def check_rounded(got: torch.Tensor, ref: np.ndarray, fp32: float, what: str):
    """Each value within ``fp32`` of its neighbourhood's largest magnitude, plus its own rounding to the
    output's type.  Neighbourhood: the last dimension's vector."""
    x = got.detach().to("cpu", torch.float64).numpy()
    assert x.shape == ref.shape, f"{what}: shape {x.shape} for {ref.shape}"
    if ref.size == 0:
        return 0.0
    assert not np.isnan(x).any(), f"{what}: NaN"
    top = np.abs(ref).max(axis=-1, keepdims=True) if ref.ndim else np.abs(ref)
    unit = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    lim = fp32 * top + unit * np.abs(ref) + 1e-30
    worst = float((np.abs(x - ref) / lim).max())
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"
    return worst


def check_e4m3(y: torch.Tensor, scales: np.ndarray, ref: np.ndarray, what: str):
    """y * scales (broadcast to ref) against ref: half a step of the 8-bit type plus the fp32 bound."""
    v = y.float().cpu().double().numpy()
    assert not np.isnan(v).any(), f"{what}: NaN"
    q = np.abs(ref) / scales
    step = np.exp2(np.floor(np.log2(np.maximum(q, 2.0 ** -6))) - 3)
    lim = (0.5 * step + FP32_VALUE * 448) * scales
    worst = float((np.abs(v * scales - ref) / lim).max()) if ref.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} times the bound"


def to64(t):
    return None if t is None else t.detach().to("cpu", torch.float64).numpy()


def spans(shape, cu):
    """[(first, last)] of each sequence on the flat token axis."""
    if cu is None:
        return [(n * shape[1], (n + 1) * shape[1]) for n in range(shape[0])]
    return list(zip(cu[:-1], cu[1:]))


def prep_ref(x, weight, bias, a, b, A_log, dt_bias, conv_state, Hk, Hv, d, slots, cu, expand, eps=1e-6):
    """gdn_prep_fwd in fp64, a token and a tap at a time.  Returns q, k, v, g, beta and the new pool."""
    shape = x.shape[:2]
    D, taps = weight.shape
    xf = x.reshape(-1, D)
    y = np.zeros_like(xf)
    pool = conv_state.copy()
    for n, (s, e) in enumerate(spans(shape, cu)):
        slot = n if slots is None else int(slots[n])
        before = conv_state[slot] if slot >= 0 else np.zeros((taps - 1, D))
        line = np.concatenate([before, xf[s:e]])
        for t in range(e - s):
            acc = np.zeros(D) if bias is None else bias.copy()
            for j in range(taps):
                acc = acc + weight[:, j] * line[t + j]
            y[s + t] = acc / (1 + np.exp(-acc))
        if slot >= 0:
            pool[slot] = line[len(line) - (taps - 1):]
    heads = y.reshape(*shape, 2 * Hk + Hv, d)
    q, k, v = heads[:, :, :Hk], heads[:, :, Hk:2 * Hk], heads[:, :, 2 * Hk:]
    q = q / np.sqrt((q ** 2).sum(-1, keepdims=True) + eps)
    k = k / np.sqrt((k ** 2).sum(-1, keepdims=True) + eps)
    if expand:
        q, k = np.repeat(q, Hv // Hk, 2), np.repeat(k, Hv // Hk, 2)
    g = -np.exp(A_log) * np.logaddexp(0, a + dt_bias)
    return q, k, v, g, 1 / (1 + np.exp(-b)), pool


def norm_ref(h, weight, eps=1e-6):
    return h / np.sqrt((h ** 2).mean(-1, keepdims=True) + eps) * weight


def silu_ref(z):
    return z / (1 + np.exp(-z))
