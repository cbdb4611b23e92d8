"""Outputs of a selective scan of up to 2048 tokens compared in norm, for the tests on a
CPU and on a GPU.

In units of U = 2^-24, errors without a pattern: a state or a gradient that went through n
tokens is off by sqrt(4 n / 3) U, 53 U for 2048; a gradient of the parameters, of B, C or a
step is a product of two such, with the step's own 8 U and sums in two levels that lose 30
U at most: 150 U < 2^-16.5 in norm, whichever part of the outputs has the most of it.  An
output of 16 bits is rounded once more: off by at most u of itself (u = 2^-8 for bf16, 2^-11
for fp16), in norm by less than 0.6 u (u / sqrt(3) for evenly spread values).
"""
import numpy as np
import torch

from oracle import state_space as orc

WITHIN = 2.0 ** -16.5
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}
PER_RANK = ("y", "hT", "du", "ddt", "dz", "dB", "dC", "dh0")
PARAMS = ("dA", "dD", "ddt_bias")


def in_norm(got, want, dtype):
    """Whether `got`, an output of that type, is `want` up to its roundings."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    limit = WITHIN + 0.6 * HALF_STEP[dtype]
    return np.isfinite(got).all() and np.linalg.norm(got - want) <= limit * np.linalg.norm(want)


def cpu64(x):
    return None if x is None else x.double().cpu().numpy()


def oracle(i, r, lens, soft=True):
    """The oracle's outputs for rank r of a call's inputs, by name."""
    cu = None if lens is None else np.concatenate(([0], np.cumsum(lens)))
    c = i["u"][0].shape[2]
    rank = lambda k: None if i[k] is None else cpu64(i[k][r])
    par = lambda k: None if i[k] is None else cpu64(i[k][r * c:(r + 1) * c])
    w = orc.selective_scan(rank("u"), rank("dt"), par("A"), rank("B"), rank("C"), par("D"), rank("z"),
                           par("dt_bias"), soft, rank("h0"), cu, rank("dy"), rank("dhT"))
    return {k: w[k] for k in PER_RANK + PARAMS if k in w}


def off_in_norm(outputs, i, r, lens, soft=True):
    """Names of rank r's outputs that are not the oracle's."""
    c = i["u"][0].shape[2]
    bad = []
    for k, want in oracle(i, r, lens, soft).items():
        x = outputs.get(k)
        if x is None:
            continue
        x = x[r * c:(r + 1) * c] if k in PARAMS else x[r]
        if not in_norm(cpu64(x), want, x.dtype):
            bad.append(k)
    return bad
