"""What attention to another sequence loses to roundings, against its definition in 64
bits: single tokens hold their weights in two bf16 parts."""

import pytest
import torch

from _mixer_ref import f64
from test_gpu_mixers import BF, DEV, gen, normal

pytestmark = pytest.mark.gpu


def own_rounding(ref):
    """How far, in the 2-norm, rounding to bf16 alone takes the values."""
    return float((ref.to(BF).double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("Hq,Hk,D,Tk", [(16, 16, 128, 1500), (16, 4, 128, 700), (20, 1, 64, 300), (12, 12, 96, 77)])
def test_step_weights(lib, Hq, Hk, D, Tk):
    """The weights' second part is off by 2^-8 of what the first left, 2^-16 of a weight: an
    output is as far off as its own rounding takes it. Of more than 10^4 roundings the sum of
    squares strays by 1 % (its standard deviation is sqrt(0.8 / N) of it), 32-bit sums of
    1500 terms add (1500 2^-24)^2 of it, below 1e-3: five hundredths are left. Weights of one
    part, each off by 2^-9.2 as the output is, would make it more by a quarter."""
    g = gen(Tk)
    B = 12
    q = normal(g, B, Hq, D, dtype=BF)
    kc, vc = (normal(g, B, Tk, Hk, D, dtype=BF) for _ in range(2))
    lens = [Tk - Tk // 3 * b // B for b in range(B)]
    o = f64(lib.cross_attn_step(q, kc, vc, torch.tensor(lens, dtype=torch.int32, device=DEV)))
    want = torch.empty_like(o)
    for b, n in enumerate(lens):
        k, v = (f64(x[b, :n]).repeat_interleave(Hq // Hk, 1) for x in (kc, vc))
        want[b] = torch.einsum("hn,nhd->hd", torch.softmax(torch.einsum("hd,nhd->hn", f64(q[b]), k) * D ** -0.5, -1), v)
    assert float((o - want).norm() / want.norm()) <= 1.05 * own_rounding(want)
