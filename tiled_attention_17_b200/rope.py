"""Frequencies of rotary positions, with the usual scalings for long contexts.

`frequencies` returns what `binding.rope` and `binding.paged_append` take: the
radians each pair turns per position, in fp64, and the factor on the rotated
elements.  Everything here is host arithmetic on a few dozen numbers, done once
when a model is set up.

Pair i of rotary_dim / 2 turns by base^(-2 i / rotary_dim) radians per position.
Scalings (a context `factor` times the trained one):
  linear       every frequency divided by the factor (position interpolation,
               Chen et al. 2023)
  ntk          a larger base, base * factor^(r / (r - 2)), which leaves the
               fastest pair as it is and divides the slowest by the factor
  yarn         pairs that turn more than beta_fast times over the trained
               length are kept, those that turn less than beta_slow times are
               divided by the factor, a linear ramp over the pair index
               between; amplitude 0.1 ln(factor) + 1 (Peng et al. 2023)
  wavelength   the same with the ramp over the number of turns itself: a pair
               of t turns over the trained length (the length divided by the
               pair's wavelength) keeps (t - low_turns) / (high_turns -
               low_turns) of its frequency, within [0, 1], the rest is divided
               by the factor; amplitude 1 ("by parts" in Peng et al. 2023)
"""
from __future__ import annotations

import math

SCALINGS = {"linear": (), "ntk": (), "yarn": ("trained_length", "beta_fast", "beta_slow", "amplitude"),
            "wavelength": ("trained_length", "low_turns", "high_turns")}


def frequency_list(rotary_dim: int, base: float = 10000.0, scaling: dict | None = None):
    """(list of rotary_dim / 2 radians per position, amplitude)."""
    r = rotary_dim
    if r <= 0 or r % 2:
        raise ValueError(f"rotary_dim must be positive and even, got {r}")
    if not (math.isfinite(base) and base > 1.0):
        raise ValueError(f"base must be finite and above 1, got {base}")
    if scaling is None:
        return [base ** (-2.0 * i / r) for i in range(r // 2)], 1.0
    opts = dict(scaling)
    kind = opts.pop("type", None)
    factor = opts.pop("factor", None)
    if kind not in SCALINGS:
        raise ValueError(f"scaling type must be one of {sorted(SCALINGS)}, got {kind!r}")
    if factor is None or not (math.isfinite(factor) and factor >= 1.0):
        raise ValueError(f"scaling factor must be finite and at least 1, got {factor}")
    unknown = set(opts) - set(SCALINGS[kind])
    if unknown:
        raise ValueError(f"unknown options for {kind} scaling: {sorted(unknown)}")
    if kind == "ntk":
        if r == 2:
            raise ValueError("ntk scaling needs rotary_dim above 2")
        base = base * factor ** (r / (r - 2))
    plain = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "ntk":
        return plain, 1.0
    if kind == "linear":
        return [f / factor for f in plain], 1.0
    trained = opts.get("trained_length")
    if trained is None or not trained > 0:
        raise ValueError(f"{kind} scaling needs a positive trained_length, got {trained}")
    if kind == "yarn":
        fast, slow = opts.get("beta_fast", 32.0), opts.get("beta_slow", 1.0)
        if not fast > slow > 0:
            raise ValueError(f"yarn scaling needs beta_fast > beta_slow > 0, got {fast}, {slow}")

        def pair_with(turns):   # the (real) index of the pair that makes this many turns
            return r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))

        lo, hi = max(math.floor(pair_with(fast)), 0), min(math.ceil(pair_with(slow)), r - 1)
        keep = [1.0 - min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(r // 2)]
        amplitude = opts.get("amplitude", 0.1 * math.log(factor) + 1.0)
    else:
        low, high = opts.get("low_turns", 1.0), opts.get("high_turns", 4.0)
        if not high > low > 0:
            raise ValueError(f"wavelength scaling needs high_turns > low_turns > 0, got {low}, {high}")
        keep = [min(max((trained * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for f in plain]
        amplitude = 1.0
    return [f * k + f / factor * (1.0 - k) for f, k in zip(plain, keep)], amplitude


def frequencies(rotary_dim: int, base: float = 10000.0, scaling: dict | None = None, device="cuda"):
    """(inv_freq, amplitude): the fp64 tensor [rotary_dim / 2] on `device` and
    the factor, as `binding.rope` and `binding.paged_append` take them.
    scaling: None or a dict, e.g. {"type": "yarn", "factor": 8.0,
    "trained_length": 8192}."""
    import torch
    values, amplitude = frequency_list(rotary_dim, base, scaling)
    return torch.tensor(values, dtype=torch.float64, device=device), amplitude
