"""Oracle: token vectors from a table and the table's gradient, float64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).
"""
from __future__ import annotations

import numpy as np


def fwd(table, tokens, scale=1.0):
    """[N, C]; a token outside [0, V) has a vector of zeros."""
    table, tokens = np.asarray(table, np.float64), np.asarray(tokens)
    out = np.zeros((len(tokens), table.shape[1]))
    on = (tokens >= 0) & (tokens < len(table))
    out[on] = scale * table[tokens[on]]
    return out


def bwd(d_out, tokens, vocab, scale=1.0):
    """(gradient [V, C], sums of magnitudes [V, C], occurrences [V])."""
    d_out, tokens = np.asarray(d_out, np.float64), np.asarray(tokens)
    grad, size, count = np.zeros((vocab, d_out.shape[1])), np.zeros((vocab, d_out.shape[1])), np.zeros(vocab, np.int64)
    on = (tokens >= 0) & (tokens < vocab)
    np.add.at(grad, tokens[on], scale * d_out[on])
    np.add.at(size, tokens[on], abs(scale) * np.abs(d_out[on]))
    np.add.at(count, tokens[on], 1)
    return grad, size, count
