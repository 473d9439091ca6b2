"""fp64 oracle of the rotary calls (plain numpy): rows of heads in, rows of heads out. It shares no code with the GPU path.

x: [rows][heads][d]; positions: [rows] whole numbers; freq: [rot / 2] radians a token. An angle is the exact product of
position and frequency, reduced to one turn with 60 digits of 2 pi, so that far positions lose nothing."""

from fractions import Fraction

import numpy as np

TWO_PI = Fraction(6283185307179586476925286766559005768394338798750211641949889, 10 ** 60)


def angles(positions, freq):
    """[rows][rot / 2] in [0, 2 pi]."""
    turns = [Fraction(float(f)) / TWO_PI for f in freq]
    return np.array([[float((int(p) * t % 1) * TWO_PI) for t in turns] for p in positions]).reshape(len(positions), len(turns))


def pairs(rot, interleaved):
    """Indexes of the two sides of each pair."""
    e = np.arange(rot // 2)
    return (2 * e, 2 * e + 1) if interleaved else (e, e + rot // 2)


def turn(x, theta, interleaved, amplitude):
    """Each row's pairs turned by theta [rows][rot / 2]."""
    rot = 2 * theta.shape[1]
    a, b = pairs(rot, interleaved)
    c, s = amplitude * np.cos(theta)[:, None], amplitude * np.sin(theta)[:, None]
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def reach(x, rot, interleaved, amplitude):
    """What bounds the fp32 errors of a turned element: |A| (|a| + |b|) of its pair, |x| of an element that passes."""
    a, b = pairs(rot, interleaved)
    y = np.abs(x)
    y[..., a] = y[..., b] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y


def forward(x, theta, interleaved, amplitude=1.0, w=None, eps=0.0):
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return turn(x, theta, interleaved, amplitude)


def backward(dy, theta, interleaved, amplitude=1.0, x=None, w=None, eps=0.0):
    """(dx, dw), dw None without weights."""
    dz = turn(dy, -theta, interleaved, amplitude)
    if w is None:
        return dz, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = x * r
    g = dz * w
    return r * (g - h * (g * h).mean(-1, keepdims=True)), (dz * h).sum((0, 1))


def shard_positions(P, B, Lp, head_sharded, pos0=0):
    """Positions of the rows of [P][B][Lp] token shards, or of [P][B][P * Lp] head groups, flattened."""
    if head_sharded:
        return np.tile(pos0 + np.arange(P * Lp), P * B)
    return np.concatenate([np.tile(pos0 + r * Lp + np.arange(Lp), B) for r in range(P)])
