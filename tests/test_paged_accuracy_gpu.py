"""How exact the packed and paged calls are, held more tightly than the
library's bar, so that a rounding more than the documented ones shows.

A rounding to bf16 is off by up to 2^-8 of a value with mantissa 1 and half of
that just below 2: uniform over +-2^-8 / m, with mantissas m spread over their
logarithm, its root mean square is 2^-8 / sqrt(3) * sqrt(E[1 / m^2]) =
2^-8 * 0.577 * 0.736 = 1.66e-3 (E[1 / m^2] = (1 - 1/4) / (2 ln 2)).

With independent normal q, k and v, relative to the output's norm:
  - the output's rounding                                  u = 1.66e-3
  - probabilities as one bf16 term: sum p d v against
    sum p v, both with independent signs                   u
  - rotated queries: a score's error is sum d q k / 16
    over r rotated dims of 256, rms u sqrt(r / 256), and
    changes its probability by as much                     u sqrt(r / 256)
  - rotated keys (here the reference does not round them)  u sqrt(r / 256)
Independent, so their squares add.  The bound allows a quarter more for what
the estimate leaves out (scores are not quite independent of |q| and |k|); a
second rounding of the probabilities, or scores in bf16, are past it."""
from __future__ import annotations

import math

import pytest

import full_gqa_attention_gb300 as fga
from parity import check_close
from test_paged_gpu import blank, layer_of, run_packed, run_paged
from test_split_tiles_gpu import Prompts

pytestmark = pytest.mark.gpu

U = 2.0 ** -8 / math.sqrt(3) * math.sqrt(0.75 / (2 * math.log(2)))


def bound(layer, p_terms):
    """p_terms: 1 where probabilities are one bf16 term, 2 where they are two."""
    return 1.25 * U * math.sqrt(1 + (p_terms == 1) + 2 * layer.rot_dim / 256)


@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_packed(cuda, kind):
    layer = layer_of(kind, window=512)
    s = Prompts([1400, 600, 64], H=8, Hkv=2, seed=31)
    check_close(run_packed(s, layer), s.expected(layer)[0], "packed", rel_l2=bound(layer, 1))


@pytest.mark.parametrize("kind", ["full", "sliding"])
@pytest.mark.parametrize("page", [16, 64])
def test_paged(cuda, kind, page):
    layer = layer_of(kind, window=512)
    s = Prompts([300, 50, 700], [1000, 4000, 0], H=8, Hkv=2, page=page, seed=32)
    check_close(run_paged(s, layer)[0], s.expected(layer)[0], "paged", rel_l2=bound(layer, 1))


@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_decode(cuda, kind):
    layer = layer_of(kind, window=512)
    old = [300 + 53 * i for i in range(60)]
    s = Prompts([1] * len(old), old, H=8, Hkv=2, page=32, seed=33)
    qkv, gate, pos, k, v, table = s.cuda("qkv", "gate", "pos", "k", "v", "table")
    out = fga.spark_attn_decode_paged(qkv, gate, pos, k, v, table, layer, out=blank(s))
    check_close(out, s.expected(layer)[0], "decode", rel_l2=bound(layer, 2))
