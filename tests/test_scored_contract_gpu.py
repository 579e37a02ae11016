"""What the scored operators promise beside their formulas: precision without asking for it, and nothing from masked memory."""
import math

import numpy as np
import pytest
import torch

import exact_tiled_attention_46_b200 as fa

import scored as S
from parity import need_gpu
from scored import BF, f64
from test_scored_gpu import CASES, cuda, forward, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


@pytest.fixture(autouse=True)
def _clean_status():
    yield
    assert fa.device_status(reset=True) == (0, 0)


# -------------------------------------------------------------- precision --
# Without changes the call is the plain forward, bit for bit, whose P is bf16.
CHANGED = [n for n in CASES if n != "plain"]


@pytest.mark.parametrize("name", CHANGED)
def test_forward_keeps_sixteen_bits_of_p(name):
    """O in fp32 against the bound of P in two bf16 parts (half steps of half steps), 2^8 below that of one part."""
    p = problem(name, seed=6)
    o, lse = forward(p, o_dtype=torch.float32)
    for b, h, g, P, l, d, ok, Q, K, V, dO, err in p.heads():
        O, lim = S.o_bound(P, V, err, fine=True)
        S.check(f64(o)[b, :, h], O, lim, f"O[{b},:,{h}]", 2.0 ** -23)
    assert torch.equal(forward(p)[0], o.to(torch.bfloat16))
