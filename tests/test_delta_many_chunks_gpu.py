"""Batches with more chunks of 64 tokens than the GPU has multiprocessors, so
that a block of the chunk gradients walks several chunks: full ones, part ones,
and ones behind a sequence's end between them.  One sequence at a time against
64 bits; tolerances as in test_delta_gpu.py."""
import pytest
import torch

from tests._delta_ref import delta_inputs
from tests.test_delta_gpu import _bwd, _check_bwd, _check_fwd, _fwd

pytestmark = pytest.mark.gpu

# batch, tokens, heads, groups, headdim
CASES = [(24, 200, 4, 4, 64), (24, 200, 4, 2, 64), (12, 250, 4, 4, 128), (12, 250, 4, 1, 128)]


@pytest.mark.parametrize("case", CASES, ids=["b%d_t%d_h%d_g%d_p%d" % c for c in CASES])
def test_prefill_and_gradient(case):
    b, t, h, g, p = case
    x = delta_inputs(b, t, h, g, p, 128, torch.bfloat16, seed=31)
    some = [t, 0, 64, 65, 1, 128, t - 1, 192, 130, 0, 63, t]
    lengths = torch.tensor([some[i % 12] for i in range(b)])
    for i, n in enumerate(lengths.tolist()):
        for k in ("q", "k", "v", "dy"):
            x[k][i, n:] = float("nan")
    y, hn = _fwd(x, 0.2, lengths)
    grads = _bwd(x, 0.2, lengths)
    for i, n in enumerate(lengths.tolist()):
        one = {k: torch.nan_to_num(v[i:i + 1], nan=0.0) for k, v in x.items()}
        _check_fwd(one, y[i:i + 1], hn[i:i + 1], 0.2, lengths[i:i + 1])
        got = {k: v[i:i + 1] for k, v in grads.items()}
        if n:
            _check_bwd(one, got, 0.2, lengths[i:i + 1])
        for k in ("dq", "dk", "dv", "dg", "dbeta"):
            assert float(got[k][:, n:].float().abs().sum()) == 0.0, k
        if not n:
            assert torch.equal(got["dh0"].cpu(), x["dh"][i:i + 1])


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_a_gate_that_is_no_number_stays_in_its_sequence(sign):
    """NaN of either sign in one head's gate: that head's results are NaN from
    there on, all others are the numbers they were."""
    x = delta_inputs(3, 200, 2, 1, 64, 128, torch.bfloat16, seed=32)
    y0, h0 = _fwd(x, 0.2)
    g0 = _bwd(x, 0.2)
    bad = {k: v.clone() for k, v in x.items()}
    bad["g"][1, 70, 0] = torch.copysign(torch.tensor(float("nan")), torch.tensor(sign))
    y1, h1 = _fwd(bad, 0.2)
    g1 = _bwd(bad, 0.2)
    assert bool(torch.isnan(h1[1, 0]).all()) and bool(torch.isnan(y1[1, 128:, 0]).all())
    for b, h in ((0, 0), (0, 1), (1, 1), (2, 0), (2, 1)):
        assert torch.equal(h1[b, h], h0[b, h]) and torch.equal(y1[b, :, h], y0[b, :, h])
        for k in ("dv", "dg", "dbeta"):
            assert torch.equal(g1[k][b, :, h], g0[k][b, :, h]), k
        assert torch.equal(g1["dh0"][b, h], g0["dh0"][b, h])
    for b in (0, 2):
        assert torch.equal(g1["dq"][b], g0["dq"][b]) and torch.equal(g1["dk"][b], g0["dk"][b])
    assert torch.equal(y1[1, :64, 0], y0[1, :64, 0])


# batch, tokens, heads, headdim: chains that are cut between blocks, of 64 and of 32 columns a block
CUT = [(40, 200, 4, 64), (60, 130, 5, 64), (21, 330, 5, 64), (19, 70, 2, 256), (300, 65, 1, 64)]


@pytest.mark.parametrize("init", [False, True])
@pytest.mark.parametrize("case", CUT, ids=["b%d_t%d_h%d_p%d" % c for c in CUT])
def test_chains_cut_between_blocks(case, init):
    """More chains than multiprocessors: a chain's first and last part are made
    by different blocks, whatever the sequences' lengths."""
    b, t, h, p = case
    x = delta_inputs(b, t, h, 1, p, 128, torch.bfloat16, seed=33)
    for lengths in (None, torch.tensor([(37 * i) % (t + 40) for i in range(b)])):
        y, hn = _fwd(x, 0.2, lengths, init=init)
        again, hn2 = _fwd(x, 0.2, lengths, init=init)
        assert torch.equal(hn, hn2) and torch.equal(torch.nan_to_num(y), torch.nan_to_num(again))
        _check_fwd(x, y, hn, 0.2, lengths, init=init)


@pytest.mark.parametrize("shape", [(2, 1, 12, 1, 128), (3, 70, 2, 2, 64), (160, 2, 4, 1, 64)])
def test_the_first_gate_has_no_gradient_without_a_state(shape):
    """dg_0 = a_0 <dS, S before the first token>: exactly zero where that state is."""
    b, t, h, g, p = shape
    x = delta_inputs(b, t, h, g, p, 128, torch.bfloat16, seed=34)
    x["h0"] = torch.zeros_like(x["h0"])
    got = _bwd(x, 0.2, init=False)
    assert float(got["dg"][:, 0].float().abs().sum()) == 0.0
    _check_bwd(x, got, 0.2, init=False)
