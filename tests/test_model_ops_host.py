"""Group norm and the router without a GPU: refusals before any device work, scratch
sizes, and the tests' 64-bit forms against differences."""

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import model_ops_ref as ref

FAKE = 0x10000  # never dereferenced: every case fails validation

GN = dict(x=FAKE, n=2, s=10, c=8, ldx=8, sx=80, kind=2, groups=2, weight=FAKE, bias=FAKE, pkind=0,
          eps=1e-5, act=2, y=FAKE, ldy=8, sy=80, mean=FAKE, rstd=FAKE, ws=FAKE, nbytes=1 << 20)


def _gn_forward(L, **change):
    k = {**GN, **change}
    return L.fc_groupnorm_forward(k["x"], k["n"], k["s"], k["c"], k["ldx"], k["sx"], k["kind"],
                                  k["groups"], k["weight"], k["bias"], k["pkind"], k["eps"],
                                  k["act"], k["y"], k["ldy"], k["sy"], k["mean"], k["rstd"],
                                  k["ws"], k["nbytes"], None)


GB = dict(GN, dy=FAKE, lddy=8, sdy=80, dx=FAKE, lddx=8, sdx=80, dw=FAKE, db=FAKE, gkind=1)


def _gn_backward(L, **change):
    k = {**GB, **change}
    return L.fc_groupnorm_backward(k["dy"], k["lddy"], k["sdy"], k["x"], k["ldx"], k["sx"],
                                   k["kind"], k["n"], k["s"], k["c"], k["groups"], k["weight"],
                                   k["bias"], k["pkind"], k["act"], k["mean"], k["rstd"], k["dx"],
                                   k["lddx"], k["sdx"], k["dw"], k["db"], k["gkind"], k["ws"],
                                   k["nbytes"], None)


SHARED = [dict(kind=3), dict(kind=-1), dict(pkind=1), dict(act=-1), dict(act=3), dict(n=-1),
          dict(n=(1 << 24) + 1), dict(s=0), dict(s=-1), dict(s=1 << 41), dict(c=0),
          dict(c=(1 << 20) + 1, groups=1), dict(groups=0), dict(groups=-2), dict(groups=3),
          dict(groups=16), dict(n=1 << 24, s=1 << 20, sx=8 << 20, sy=8 << 20), dict(x=None),
          dict(ldx=7), dict(ldx=-8), dict(sx=79), dict(sx=-80), dict(sx=0), dict(ldx=0),
          dict(sx=1 << 41), dict(ldx=8, sx=8), dict(ldx=15, sx=8)]


@pytest.mark.parametrize("call", [_gn_forward, _gn_backward])
def test_groupnorm_shared_refusals(fc_lib, call):
    for change in SHARED:
        assert call(fc_lib, **change) == fc.FC_ERR_INVALID_ARG, change
        assert fc_lib.fc_last_error()
    for change in (dict(x=FAKE + 1), dict(weight=FAKE + 2), dict(bias=FAKE + 2),
                   dict(mean=FAKE + 2), dict(rstd=FAKE + 1), dict(ws=FAKE + 64)):
        assert call(fc_lib, **change) == fc.FC_ERR_ALIGNMENT, change
    need = fc.fc_groupnorm_workspace_size(2, 10, 8, 2)
    for change in (dict(ws=None), dict(nbytes=need - 1), dict(nbytes=0)):
        assert call(fc_lib, **change) == fc.FC_ERR_WORKSPACE, change


def test_groupnorm_forward_refusals(fc_lib):
    for change in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None),
                   dict(mean=None), dict(rstd=None), dict(ldy=7), dict(sy=79)):
        assert _gn_forward(fc_lib, **change) == fc.FC_ERR_INVALID_ARG, change
    assert _gn_forward(fc_lib, y=FAKE + 1) == fc.FC_ERR_ALIGNMENT
    # no samples: nothing to do, whatever the pointers
    assert _gn_forward(fc_lib, n=0, x=None, y=None) == fc.FC_OK


def test_groupnorm_backward_refusals(fc_lib):
    for change in (dict(gkind=3), dict(dy=None), dict(dx=None), dict(lddy=7), dict(sdx=79),
                   dict(mean=None), dict(rstd=None)):
        assert _gn_backward(fc_lib, **change) == fc.FC_ERR_INVALID_ARG, change
    for change in (dict(dy=FAKE + 1), dict(dx=FAKE + 1), dict(dw=FAKE + 1), dict(db=FAKE + 1)):
        assert _gn_backward(fc_lib, **change) == fc.FC_ERR_ALIGNMENT, change
    assert _gn_backward(fc_lib, n=0, dw=None, db=None) == fc.FC_OK


def test_groupnorm_workspace_sizes(fc_lib):
    size = fc.fc_groupnorm_workspace_size
    assert size(-1, 4, 8, 2) == size(2, 0, 8, 2) == size(2, 4, 0, 1) == size(2, 4, 8, 3) == 0
    assert size(0, 4, 8, 2) > 0 and size(2, 4, 8, 2) % 256 == 0
    # a small share of maps of some size: at bf16 these hold 64 x 4096 x 512 x 2 bytes
    assert size(64, 4096, 512, 32) < 64 * 4096 * 512 * 2 // 10


@pytest.mark.parametrize("n,s,c,groups", [
    (65536, 1, 4096, 1), (4096, 1, 1024, 2), (1 << 24, 1, 512, 1), (70000, 3, 520, 1),
    (2000, 16, 1 << 20, 1), (1 << 20, 40, 300, 1), (1 << 24, 1, 8, 1), (513, 1, 1 << 20, 2),
    (600, 5000, 8192, 8), (1024, 1, 1 << 20, 1 << 18)])
def test_groupnorm_scratch_of_many_samples(fc_lib, n, s, c, groups):
    """Not a share of the images, however few positions they have: 2^23 pairs of sums at a
    time (or those of one sample), a set for each chunk, two values a group and sample."""
    chunks = -(-n // min(8192, max(1, (1 << 23) // c)))
    most = 8 * (max(c, 1 << 23) + chunks * c + n * groups) + 768
    assert fc.fc_groupnorm_workspace_size(n, s, c, groups) <= most


def test_groupnorm_scratch_without_samples(fc_lib):
    assert fc.fc_groupnorm_workspace_size(0, 1 << 16, 1 << 20, 1) <= 768


RT = dict(x=FAKE, seq=3, tok=4, e=8, ld=8, kind=2, lengths=FAKE, k=2, norm=1, per=1, chosen=FAKE,
          weights=FAKE, lse=FAKE, counts=FAKE, routed=FAKE, probs=FAKE, loss=FAKE, ws=FAKE,
          nbytes=1 << 20)


def _router(L, **change):
    k = {**RT, **change}
    return L.fc_router_forward(k["x"], k["seq"], k["tok"], k["e"], k["ld"], k["kind"],
                               k["lengths"], k["k"], k["norm"], k["per"], k["chosen"],
                               k["weights"], k["lse"], k["counts"], k["routed"], k["probs"],
                               k["loss"], k["ws"], k["nbytes"], None)


RB = dict(RT, dw=FAKE, dl=FAKE, dx=FAKE, lddx=8)


def _router_bwd(L, **change):
    k = {**RB, **change}
    return L.fc_router_backward(k["x"], k["seq"], k["tok"], k["e"], k["ld"], k["kind"], k["k"],
                                k["norm"], k["per"], k["chosen"], k["weights"], k["lse"],
                                k["counts"], k["routed"], k["dw"], k["dl"], k["dx"], k["lddx"],
                                None)


@pytest.mark.parametrize("call", [_router, _router_bwd])
def test_router_shared_refusals(fc_lib, call):
    for change in (dict(kind=3), dict(seq=-1), dict(tok=-1), dict(seq=1 << 20, tok=1 << 20),
                   dict(seq=1 << 40), dict(e=0, ld=8), dict(k=0), dict(k=-1), dict(k=9),
                   dict(ld=7), dict(ld=1 << 41), dict(x=None), dict(chosen=None),
                   dict(weights=None), dict(lse=None), dict(counts=None), dict(routed=None)):
        assert call(fc_lib, **change) == fc.FC_ERR_INVALID_ARG, change
        assert fc_lib.fc_last_error()
    for change in (dict(e=1025, ld=1025), dict(e=64, ld=64, k=33)):
        assert call(fc_lib, **change) == fc.FC_ERR_LIMIT, change
    for change in (dict(x=FAKE + 1), dict(chosen=FAKE + 2), dict(weights=FAKE + 2),
                   dict(lse=FAKE + 2), dict(counts=FAKE + 1), dict(routed=FAKE + 2)):
        assert call(fc_lib, **change) == fc.FC_ERR_ALIGNMENT, change


def test_router_forward_refusals(fc_lib):
    for change in (dict(probs=None), dict(loss=None)):
        assert _router(fc_lib, **change) == fc.FC_ERR_INVALID_ARG, change
    for change in (dict(lengths=FAKE + 2), dict(loss=FAKE + 2), dict(ws=FAKE + 64)):
        assert _router(fc_lib, **change) == fc.FC_ERR_ALIGNMENT, change
    need = fc.fc_router_workspace_size(3, 4, 8, True)
    for change in (dict(ws=None), dict(nbytes=need - 1)):
        assert _router(fc_lib, **change) == fc.FC_ERR_WORKSPACE, change


def test_router_backward_refusals(fc_lib):
    for change in (dict(dx=None), dict(lddx=7)):
        assert _router_bwd(fc_lib, **change) == fc.FC_ERR_INVALID_ARG, change
    for change in (dict(dx=FAKE + 1), dict(dw=FAKE + 2), dict(dl=FAKE + 2)):
        assert _router_bwd(fc_lib, **change) == fc.FC_ERR_ALIGNMENT, change
    # no rows: nothing to do, whatever the pointers
    assert _router_bwd(fc_lib, seq=0, x=None, dx=None, lse=None, chosen=None) == fc.FC_OK


def test_router_workspace_sizes(fc_lib):
    size = fc.fc_router_workspace_size
    assert size(-1, 4, 8) == size(4, -1, 8) == size(1, 4, 0) == size(1, 4, 1025) == 0
    assert size(0, 0, 8, True) > 0 and size(1, 1 << 30, 1024) < 32 << 20


def test_router_takes_many_sequences_that_are_balanced_together(fc_lib):
    """Fewer than 2^31 rows, whatever their sequences: the shape is not what is refused."""
    many = dict(seq=(1 << 24) + 5, tok=2, e=1024, ld=1024, lddx=1024)
    size = fc.fc_router_workspace_size
    assert size(many["seq"], 2, 1024) > 0 and size(many["seq"], 2, 1024, True) == 0
    assert _router(fc_lib, **many, per=0, ws=None) == fc.FC_ERR_WORKSPACE
    assert _router_bwd(fc_lib, **many, per=0, lse=FAKE + 2) == fc.FC_ERR_ALIGNMENT
    for call in (_router, _router_bwd):
        assert call(fc_lib, **many, per=1, lse=FAKE + 2) == fc.FC_ERR_INVALID_ARG


def test_binding_refuses_tensors_off_the_gpu(fc_lib):
    x, w = torch.zeros(2, 5, 8), torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fc.fc_groupnorm_forward(x, 2, None, None, 1e-5, fc.FC_ACT_SILU, x.clone(), None, None, w)
    i = torch.zeros(10, 2, dtype=torch.int32)
    f = torch.zeros(10, 2)
    with pytest.raises(ValueError):
        fc.fc_router_forward(x[0], 1, None, True, False, i, f, f, i, i, f, f, w)


def _differences(loss, pairs, scale):
    e = 1e-6
    for t, grad in pairs:
        flat, want = t.view(-1), grad.reshape(-1)
        for i in range(flat.numel()):
            keep = float(flat[i])
            flat[i] = keep + e
            up = loss()
            flat[i] = keep - e
            down = loss()
            flat[i] = keep
            # central differences: e^2 times a third derivative, and 1e-16 of the
            # loss over e
            assert abs((up - down) / (2 * e) - float(want[i])) < 1e-6 * scale


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("n,s,c,groups", [(1, 3, 4, 2), (2, 5, 6, 3), (2, 1, 8, 1)])
def test_groupnorm_formula_against_differences(n, s, c, groups, kind):
    g = torch.Generator().manual_seed(3)
    rnd = lambda *sh: torch.randn(*sh, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, b, dy = rnd(n, s, c), rnd(c), rnd(c), rnd(n, s, c)
    (_, mean, rstd), _ = ref.groupnorm(x, groups, w, b, 0.1, kind)
    (dx, dw, db), _ = ref.groupnorm_backward(dy, x, groups, w, b, kind, mean, rstd)

    def loss():
        return float((ref.groupnorm(x, groups, w, b, 0.1, kind)[0][0] * dy).sum())
    _differences(loss, ((x, dx), (w, dw), (b, db)), 1 + float(rstd.max()) ** 3 * n * s * c)


@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("per_sequence", [False, True])
def test_router_formula_against_differences(per_sequence, normalise):
    g = torch.Generator().manual_seed(4)
    rows, experts, k, sequences = 8, 5, 2, 2
    x = torch.randn(rows, experts, generator=g, dtype=torch.float64)
    x[2, 3] = -float("inf")
    lengths = torch.tensor([4, 3], dtype=torch.int32)
    dw = torch.randn(rows, k, generator=g, dtype=torch.float64)
    dl = torch.tensor([0.8, 0.6], dtype=torch.float64)
    o, _ = ref.router(x, sequences, lengths, k, normalise, per_sequence)
    dx, _ = ref.router_backward(x, sequences, k, normalise, per_sequence, o["chosen"],
                                o["weights"], o["lse"], o["counts"], o["routed"], dw, dl)

    def loss():
        p, _ = ref.router(x, sequences, lengths, k, normalise, per_sequence)
        assert torch.equal(p["chosen"], o["chosen"])  # no step crosses a choice
        return float((p["weights"] * dw).sum() + (p["loss"] * dl).sum())
    e = 1e-6
    for r in range(rows):
        for q in range(experts):
            keep = float(x[r, q])
            if keep == -float("inf"):
                assert float(dx[r, q]) == 0
                continue
            x[r, q] = keep + e
            up = loss()
            x[r, q] = keep - e
            down = loss()
            x[r, q] = keep
            assert abs((up - down) / (2 * e) - float(dx[r, q])) < 1e-6
