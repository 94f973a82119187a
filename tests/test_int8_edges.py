"""The 8-bit prefix operators where they are easily wrong: values of zero, long
tails of small weights, queries of wide range, scales at the end of fp32, wide
rows, products of several tiles per SM, errors that were left pending.

Tolerances count roundings: one to a type t is off by at most eps(t) / 2 relative
to the value (bf16 2^-8, fp16 2^-11, fp32 2^-24).
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import flow_matching_action_pi0_b200 as fm
from flow_matching_action_pi0_b200 import build as fbuild
from tests.test_int8_ops import DT, HALF_ULP, assert_attention, attention_ref, quant_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _put(c, k_codes, k_scale, v_codes, v_scale):
    """Fill a cache with codes [slots, heads, cap, d] and scales; the values it stands for, float64."""
    for t, x in ((c.k, k_codes), (c.v, v_codes), (c.k_scale, k_scale), (c.v_scale, v_scale)):
        t.copy_(x)
    return [(q.double() * s.double().unsqueeze(-1)).cpu() for q, s in ((c.k, c.k_scale), (c.v, c.v_scale))]


def _lens(*n):
    return torch.tensor(n, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ values of zero
@pytest.mark.gpu
@pytest.mark.parametrize("nq,cap,zeros,causal", [
    (1, 100, 100, False), (1, 3000, 3000, False), (600, 100, 100, False), (600, 100, 100, True),  # row groups; tiles, one part
    (200, 600, 600, False), (200, 600, 600, True),                                                # tiles, several parts
    (200, 600, 75, False), (200, 600, 525, False), (1, 3000, 640, False),                         # a part of zeros beside others
    (40, 100, 70, True), (600, 700, 150, True)])                                                  # the first queries see zeros alone
def test_values_of_zero_under_low_scores(nq, cap, zeros, causal):
    """All scores near -163 in log2: keys whose values are zero contribute zero,
    however small the row's weight is in absolute terms."""
    d, group = 128, 4
    g = torch.Generator().manual_seed(nq + cap + zeros)
    c = fm.KvCacheInt8(1, 1, cap, d)
    vs = torch.rand(1, 1, cap, generator=g) * 0.01 + 0.01
    vs[..., :zeros] = 0.0
    vc = torch.randint(-127, 128, (1, 1, cap, d), generator=g, dtype=torch.int8)
    vc[..., :zeros, :] = 0
    kc = torch.randint(90, 110, (1, 1, cap, d), generator=g, dtype=torch.int8)
    k, v = _put(c, kc, torch.full((1, 1, cap), 0.1), vc, vs)
    q = -torch.ones(1, nq, group, d, dtype=torch.bfloat16)
    o, a = attention_ref(q.double(), k, v, [cap], causal, None, None, d ** -0.5)
    got = c.attend(q.cuda(), _lens(cap), causal=causal)
    assert bool(torch.isfinite(got).all())
    assert_attention(got, o, a)
    assert bool((got.cpu()[a == 0] == 0).all())
    # a NaN value scale still shows
    c.v_scale[0, 0, 0] = math.nan
    sees = slice(max(0, nq - cap) if causal else 0, nq)
    assert bool(torch.isnan(c.attend(q.cuda(), _lens(cap), causal=causal)[:, sees]).all())
