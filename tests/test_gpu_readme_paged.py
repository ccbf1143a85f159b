"""The README's step of drafted tokens, run as it stands: the drafts' keys and
queries are turned to the positions behind the request's rows."""
import os

import numpy as np
import pytest
import torch

import oracle
from tests.test_gpu_paged import make_tree, sca  # noqa: F401

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_drafts_lie_behind_the_rows_that_are_there(sca):
    text = open(README).read()
    code = text[text.index("angles = sca.RotaryAngles"):]
    code = code[:code.index("```")]
    B, H, Hkv, T, D, page, pages = 2, 16, 8, 5, 64, 64, 20
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    q, k, v = rnd(B, H, T, D), rnd(B, Hkv, T, D), rnd(B, Hkv, T, D)
    words, parents = make_tree(B, T, seed=3)
    depths = torch.zeros(B, T, dtype=torch.int32)
    for b in range(B):
        for t, p in enumerate(parents[b]):
            depths[b, t] = depths[b, p] + 1 if p >= 0 else 0
    lengths = torch.tensor([130, 61], dtype=torch.int32)
    table = torch.randperm(pages, generator=g)[:8].to(torch.int32).reshape(2, 4)
    names = dict(sca=sca, B=B, H=H, T=T, D=D, pages=pages, q=q.cuda(), k=k.cuda(), v=v.cuda(), table=table.cuda(),
                 lengths=lengths.cuda(), depths=depths.cuda(), ancestors=words.cuda(),
                 path=torch.arange(T, dtype=torch.int32).expand(B, T).contiguous().cuda(),
                 accepted=torch.ones(B, dtype=torch.int32, device="cuda"))
    exec(code, names)
    assert names["step"].read_status() == 0 and torch.equal(names["lengths"].cpu(), lengths + 1)
    angles = names["angles"]
    cos, sin = oracle.rotary_cos_sin((lengths[:, None] + depths).numpy(), angles.frequencies)
    ref = oracle.rotary(q, cos[:, None], sin[:, None], "half", angles.amplitude)
    mag = np.abs(q.double().numpy())
    mag = angles.amplitude * (mag + np.roll(mag, D // 2, -1))
    # the rotation's bound and half a step of bf16 (tests/test_gpu_rotary.py)
    err = np.abs(names["q1"].double().cpu().numpy() - ref)
    assert (err <= 6 * 2.0 ** -24 * mag + 1.01 * 2.0 ** -8 * np.abs(ref)).all()
