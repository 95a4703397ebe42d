"""What attention to another sequence loses to roundings, against its definition in 64
bits: single tokens hold their weights in two bf16 parts, the backward the gradients of the
scores of a sequence of few keys, whatever batch it comes in."""

import pytest
import torch

import _block_ref as ref
from _mixer_ref import f64
from test_gpu_cross import inputs, ints
from test_gpu_mixers import BF, DEV, gen, normal, offsets

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


@pytest.mark.parametrize("D,Hq,Hk", [(64, 4, 2), (128, 3, 1), (96, 2, 2)])
@pytest.mark.parametrize("Tk", [300, 513, 2048])
def test_short_rows_of_a_padded_batch(lib, D, Hq, Hk, Tk):
    """Rows of 130 to 300 keys, padded to 300 and to more: dq and dk are as far off as their
    own rounding takes them. Besides that there is the delta of rows of more than 128 keys, from the
    output as it was rounded: some 2^-9.2 of it, an output being some sqrt(e / 130) = 0.15 of a
    value (weights of normal scores), so 0.02 of their own rounding in the squares; the sums
    of squares stray by 1 %. A tenth is left; ds in one part would make it more by two
    fifths."""
    q, k, v, do = inputs(4, 400, Tk, Hq, Hk, D, BF, 31)
    lens = ints(130, 300, 257, 191)
    o, lse = lib.cross_attn_fwd(q, k, v, lens)
    got = lib.cross_attn_bwd(q, k, v, o, lse, do, lens)
    want, _ = ref.cross_grads(f64(q), f64(k), f64(v), f64(do), D ** -0.5, ref.spans(4, 400, Tk, lens))
    for a, b, name in list(zip(got, want, ("dq", "dk")))[:2]:
        rel = float((f64(a) - b).norm() / b.norm())
        assert rel <= 1.1 * own_rounding(b), (name, rel, own_rounding(b))


@pytest.mark.parametrize("D,Hq,Hk", [(64, 4, 2), (128, 3, 1)])
def test_a_sequence_does_not_feel_its_neighbours(lib, D, Hq, Hk):
    """Outputs and dq of a sequence are the same bits alone, beside longer and shorter ones and
    padded; its dk and dv, sums over queries that blocks share in other places, are as near to
    them as 32-bit sums make them, so equal but for a few elements' last bit."""
    lq, lk = [200, 333, 140], [130, 1700, 600]
    q, k, v, do = inputs(1, sum(lq), sum(lk), Hq, Hk, D, BF, 32)
    cu = offsets(lq), offsets(lk)

    def both(q, k, v, do, *seqs):
        o, lse = lib.cross_attn_fwd(q, k, v, *seqs)
        return (o, *lib.cross_attn_bwd(q, k, v, o, lse, do, *seqs))

    packed = both(q, k, v, do, None, *cu)
    a = c = 0
    for i, (nq, nk) in enumerate(zip(lq, lk)):
        part = [t[:, b:b + n].contiguous() for t, b, n in ((q, a, nq), (k, c, nk), (v, c, nk), (do, a, nq))]
        alone = both(*part)
        long = [part[0], *(torch.cat([t, normal(gen(5), 1, 2000 - nk, Hk, D, dtype=BF)], 1) for t in part[1:3]), part[3]]
        padded = both(*long, ints(nk))
        for other in ([t[:, b:b + n] for t, b, n in zip(packed, (a, a, c, c), (nq, nq, nk, nk))],
                      [t[:, :n] for t, n in zip(padded, (nq, nq, nk, nk))]):
            assert torch.equal(other[0], alone[0]) and torch.equal(other[1], alone[1]), i
            for x, y in zip(other[2:], alone[2:]):
                assert float((x != y).float().mean()) <= 0.01, i
        a, c = a + nq, c + nk
