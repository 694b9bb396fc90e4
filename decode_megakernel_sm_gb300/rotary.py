"""Rotary: how positions turn queries and keys, for KVCache.append."""
from __future__ import annotations

import ctypes as C
import math
import struct

_ROTARY = struct.Struct("=iiQd")  # mk_rotary


class Rotary:
    """The first ``dims`` dims of a head (default: all of them; a multiple of 16) turn as
    pairs, (t, t + dims / 2) or, ``interleaved``, (2t, 2t + 1), pair t by the angle
    position * frequencies[t]; the other dims stay.  Turned dims are multiplied by
    ``magnitude``.

    frequencies[t] = theta^(-2t / dims), stretched for contexts longer than a model was
    trained on by ``factor``: without ``trained`` all alike (positions / factor); with
    ``trained``, the length in positions it was trained on, by the turns that a pair makes
    over it: pairs of at least ``high`` turns stay as they are, pairs of at most ``low``
    are divided by factor, those between in proportion:
        f' = (w + (1 - w) / factor) f,   w = (turns - low) / (high - low) cut to [0, 1].
    ``frequencies`` given: these instead, dims / 2 radians per position; so for every other
    rule (a w that is linear in the pair's index t is not the one above)."""

    __slots__ = ("head_dim", "dims", "interleaved", "magnitude", "frequencies", "_held", "_packed")

    def __init__(self, head_dim, theta=None, *, dims=None, interleaved=False, factor=1.0,
                 trained=None, low=1.0, high=4.0, magnitude=1.0, frequencies=None):
        dims = head_dim if dims is None else dims
        if dims < 0 or dims > head_dim or dims % 16:
            raise ValueError(f"dims: expected a multiple of 16 of at most {head_dim}, got {dims}")
        if not math.isfinite(magnitude):
            raise ValueError("magnitude: expected a finite number")
        if (theta is None) == (frequencies is None):
            raise ValueError("expected theta or frequencies")
        if frequencies is None:
            theta = float(theta)
            if not (1.0 <= theta <= 1e30):
                raise ValueError("theta: expected a number from 1 to 1e30")
            if not (1.0 <= factor < math.inf):
                raise ValueError("factor: expected a number of at least 1")
            frequencies = [theta ** (-2.0 * t / dims) for t in range(dims // 2)]
            if trained is None:
                frequencies = [f / factor for f in frequencies]
            else:
                if not (0 < trained < math.inf and -math.inf < low < high < math.inf):
                    raise ValueError("expected a trained length above 0 and low below high")
                frequencies = [f * (w + (1 - w) / factor) for f, w in (
                    (f, min(max((trained * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0))
                    for f in frequencies)]
        else:
            frequencies = [float(f) for f in frequencies]
            if factor != 1.0 or trained is not None:
                raise ValueError("factor and trained go with theta")
            if len(frequencies) != dims // 2 or not all(abs(f) <= math.pi for f in frequencies):
                raise ValueError(f"frequencies: expected {dims // 2} numbers within [-pi, pi]")
        magnitude, frequencies = float(magnitude), tuple(float(f) for f in frequencies)
        held = (C.c_double * (dims // 2))(*frequencies)  # what the calls read
        packed = _ROTARY.pack(dims, bool(interleaved), C.addressof(held) if dims else 0, magnitude)
        for name, value in zip(self.__slots__, (head_dim, dims, bool(interleaved), magnitude, frequencies,
                                                held, packed)):
            object.__setattr__(self, name, value)

    def __setattr__(self, name, value):
        raise AttributeError("Rotary: cannot be changed, make another one")

    def __delattr__(self, name):
        raise AttributeError("Rotary: cannot be changed, make another one")

    def __reduce__(self):  # copies pack the address of their own numbers
        return _again, (self.head_dim, self.dims, self.interleaved, self.magnitude, self.frequencies)


def _again(head_dim, dims, interleaved, magnitude, frequencies):
    return Rotary(head_dim, dims=dims, interleaved=interleaved, magnitude=magnitude, frequencies=frequencies)
