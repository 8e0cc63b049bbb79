"""The example's decoder beside its plain definition (oracle/decoder.py), for the tests of both."""
from __future__ import annotations

import importlib.util
import math
import os

import numpy as np

from oracle.decoder import Decoder

VOCAB, LAYERS, MAX_POS = 512, 2, 256

# How far the logits of the two (of size 1, root mean square over the vocabulary) may be apart.  Values
# are rounded to bfloat16 about ten times a layer and once before the head, 21 times in two layers, by at
# most half of a step of 2^-7 to 2^-8 of the value: 2^-7 / sqrt 12 in the mean square at most.  The
# roundings are independent, and on both sides: sqrt(2 * 21) of that; twice it for gains above one.
TOL = 2 * math.sqrt(2 * 21) * 2.0 ** -7 / math.sqrt(12)
# An 8-bit cache rounds K and V to steps of 2^-3 on both sides, of values that may differ by a bfloat16
# step: as if none of the four roundings (K and V, two layers) were the same, in a branch that is half of
# the sum at most.
TOL_E4M3 = math.hypot(TOL, 0.5 * math.sqrt(4) * 2.0 ** -3 / math.sqrt(12))


def load_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def models(example, monkeypatch, device, pack=None):
    """The example's decoder, and its plain definition for a bfloat16 and an 8-bit cache.  pack: what stands in
    for pack_weights (None: itself)."""
    weights, real = [], pack or example.tl.pack_weights

    def keep(codes, scales):
        weights.append((codes.cpu().numpy(), scales.cpu().numpy()))
        return real(codes, scales)
    with monkeypatch.context() as m:
        m.setattr(example.tl, "pack_weights", keep)
        model = example.Decoder(layers=LAYERS, vocab=VOCAB, max_pos=MAX_POS, device=device)
    plain = [Decoder(model.embed.cpu().numpy(), [weights[4 * i:4 * i + 4] for i in range(LAYERS)], weights[-1],
                     model.cos_sin.cpu().numpy(), example.HEADS, example.KV_HEADS, example.D, e4m3)
             for e4m3 in (False, True)]
    return model, plain


def apart(a, b):
    """Root mean square of the difference of rows of logits."""
    return np.sqrt(((a - b) ** 2).mean(-1))
