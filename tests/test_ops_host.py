"""The training-step operators without a GPU: refusals of the C entry points and
of the binding, and the 64-bit forms of the tests against differences."""

import ctypes

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import ops_ref

P = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced: every call below fails its checks first


def _table(ptrs, sizes):
    a = (ctypes.c_void_p * len(ptrs))(*ptrs)
    s = (ctypes.c_int64 * len(sizes))(*sizes)
    return a, s, ctypes.cast(a, P), ctypes.cast(s, P)


def _norm(L, ptrs=(FAKE,), sizes=(8,), kind=0, count=None, loss_scale=1.0, max_norm=1.0,
          norm=FAKE, scale=FAKE, ws=FAKE, nbytes=1 << 20):
    keep = _table(ptrs, sizes)
    return L.fc_grad_norm(keep[2], kind, len(sizes) if count is None else count, keep[3],
                          loss_scale, max_norm, norm, scale, ws, nbytes, None)


def test_grad_norm_refusals(fc_lib):
    L = fc_lib
    assert _norm(L, kind=3) == fc.FC_ERR_INVALID_ARG and b"grad_type" in L.fc_last_error()
    assert _norm(L, kind=-1) == fc.FC_ERR_INVALID_ARG
    assert _norm(L, count=0) == fc.FC_ERR_INVALID_ARG
    assert _norm(L, sizes=(0,)) == fc.FC_ERR_INVALID_ARG
    assert _norm(L, sizes=(-1,)) == fc.FC_ERR_INVALID_ARG
    assert _norm(L, sizes=(1 << 43,)) == fc.FC_ERR_INVALID_ARG
    assert _norm(L, ptrs=(None,)) == fc.FC_ERR_INVALID_ARG
    assert _norm(L, ptrs=(FAKE + 2,)) == fc.FC_ERR_ALIGNMENT
    assert _norm(L, ptrs=(FAKE + 1,), kind=1) == fc.FC_ERR_ALIGNMENT
    many = fc.FC_MAX_OPT_LAYERS + 1
    assert _norm(L, ptrs=(FAKE,) * many, sizes=(8,) * many) == fc.FC_ERR_LIMIT
    assert b"FC_MAX_OPT_LAYERS" in L.fc_last_error()
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert _norm(L, loss_scale=bad) == fc.FC_ERR_INVALID_ARG
    for bad in (-1.0, float("inf"), float("nan")):
        assert _norm(L, max_norm=bad) == fc.FC_ERR_INVALID_ARG
    assert _norm(L, norm=None) == fc.FC_ERR_INVALID_ARG
    assert _norm(L, scale=FAKE + 2) == fc.FC_ERR_ALIGNMENT
    assert _norm(L, ws=None) == fc.FC_ERR_WORKSPACE
    assert _norm(L, nbytes=fc.fc_grad_norm_workspace_size() - 1) == fc.FC_ERR_WORKSPACE
    assert _norm(L, ws=FAKE + 128) == fc.FC_ERR_ALIGNMENT


ADAM = dict(ptrs=(FAKE,), sizes=(8,), kind=0, decay=None, grad_scale=FAKE, lr=1e-3, b1=0.9,
            b2=0.999, eps=1e-8, wd=0.1, weights=FAKE, low=None, low_type=1, a=FAKE, b=FAKE,
            c=FAKE, d=FAKE, steps=FAKE)


def _adam(L, bits, **change):
    k = {**ADAM, **change}
    keep = _table(k["ptrs"], k["sizes"])
    decay = None if k["decay"] is None else (ctypes.c_float * len(k["decay"]))(*k["decay"])
    head = (keep[2], k["kind"], len(k["sizes"]), keep[3],
            None if decay is None else ctypes.cast(decay, P), k["grad_scale"], k["lr"], k["b1"],
            k["b2"], k["eps"], k["wd"], k["weights"], k["low"], k["low_type"])
    if bits == 32:
        return L.fc_adamw_step(*head, k["a"], k["b"], k["steps"], None)
    return L.fc_adamw8_step(*head, k["a"], k["c"], k["b"], k["d"], k["steps"], 7, None)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_refusals(fc_lib, bits):
    L = fc_lib
    nan, inf = float("nan"), float("inf")
    wrong = [dict(kind=5), dict(sizes=(0,)), dict(ptrs=(None,)), dict(decay=(-1.0,)),
             dict(decay=(nan,)), dict(lr=-1.0), dict(lr=nan), dict(lr=inf), dict(b1=1.0),
             dict(b1=-0.1), dict(b1=nan), dict(b2=1.0), dict(b2=1 - 1e-12), dict(eps=0.0),
             dict(eps=1e-60), dict(eps=nan), dict(eps=inf), dict(wd=-0.1), dict(wd=inf),
             dict(weights=None), dict(low=FAKE, low_type=0), dict(low=FAKE, low_type=9),
             dict(a=None), dict(b=None), dict(steps=None)]
    if bits == 8:
        wrong += [dict(c=None), dict(d=None)]
    for change in wrong:
        assert _adam(L, bits, **change) == fc.FC_ERR_INVALID_ARG, change
        assert L.fc_last_error()
    shifted = [dict(ptrs=(FAKE + 2,)), dict(weights=FAKE + 4), dict(low=FAKE + 8),
               dict(a=FAKE + 4), dict(b=FAKE + 8), dict(steps=FAKE + 4),
               dict(grad_scale=FAKE + 2)]
    for change in shifted:
        assert _adam(L, bits, **change) == fc.FC_ERR_ALIGNMENT, change
    many = fc.FC_MAX_OPT_LAYERS + 1
    assert _adam(L, bits, ptrs=(FAKE,) * many, sizes=(4,) * many) == fc.FC_ERR_LIMIT


LN = dict(x=FAKE, rows=4, cols=8, ldx=8, kind=2, weight=FAKE, bias=FAKE, pkind=0, eps=1e-5,
          y=FAKE, ldy=8, mean=FAKE, rstd=FAKE)


def _forward(L, **change):
    k = {**LN, **change}
    return L.fc_layernorm_forward(k["x"], k["rows"], k["cols"], k["ldx"], k["kind"], k["weight"],
                                  k["bias"], k["pkind"], k["eps"], k["y"], k["ldy"], k["mean"],
                                  k["rstd"], None)


def test_layernorm_forward_refusals(fc_lib):
    L = fc_lib
    wrong = [dict(kind=3), dict(pkind=1), dict(pkind=7), dict(rows=-1), dict(cols=0),
             dict(cols=(1 << 31) + 1, ldx=1 << 32, ldy=1 << 32), dict(ldx=7), dict(ldy=7),
             dict(ldx=1 << 41), dict(rows=1 << 50, ldx=1 << 20), dict(x=None), dict(y=None),
             dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(mean=None),
             dict(rstd=None)]
    for change in wrong:
        assert _forward(L, **change) == fc.FC_ERR_INVALID_ARG, change
    for change in (dict(x=FAKE + 1), dict(y=FAKE + 1), dict(weight=FAKE + 2),
                   dict(bias=FAKE + 2), dict(mean=FAKE + 2), dict(rstd=FAKE + 1)):
        assert _forward(L, **change) == fc.FC_ERR_ALIGNMENT, change
    # no rows: nothing to do, whatever the pointers
    assert _forward(L, rows=0, x=None, y=None) == fc.FC_OK


BWD = dict(dy=FAKE, lddy=8, x=FAKE, ldx=8, kind=2, weight=FAKE, pkind=0, mean=FAKE, rstd=FAKE,
           rows=4, cols=8, dx=FAKE, lddx=8, dw=FAKE, db=FAKE, gkind=1, ws=FAKE, nbytes=1 << 20)


def _backward(L, **change):
    k = {**BWD, **change}
    return L.fc_layernorm_backward(k["dy"], k["lddy"], k["x"], k["ldx"], k["kind"], k["weight"],
                                   k["pkind"], k["mean"], k["rstd"], k["rows"], k["cols"],
                                   k["dx"], k["lddx"], k["dw"], k["db"], k["gkind"], k["ws"],
                                   k["nbytes"], None)


def test_layernorm_backward_refusals(fc_lib):
    L = fc_lib
    wrong = [dict(kind=4), dict(pkind=1), dict(gkind=3), dict(rows=-1), dict(cols=0),
             dict(lddy=7), dict(ldx=7), dict(lddx=7), dict(dy=None), dict(x=None), dict(dx=None),
             dict(mean=None), dict(rstd=None)]
    for change in wrong:
        assert _backward(L, **change) == fc.FC_ERR_INVALID_ARG, change
    for change in (dict(dy=FAKE + 1), dict(dx=FAKE + 1), dict(weight=FAKE + 2),
                   dict(dw=FAKE + 1), dict(db=FAKE + 1), dict(mean=FAKE + 2),
                   dict(ws=FAKE + 64)):
        assert _backward(L, **change) == fc.FC_ERR_ALIGNMENT, change
    assert _backward(L, ws=None) == fc.FC_ERR_WORKSPACE
    need = fc.fc_layernorm_backward_workspace_size(4, 8)
    assert _backward(L, nbytes=need - 1) == fc.FC_ERR_WORKSPACE
    assert _backward(L, rows=0, dw=None, db=None, ws=None) == fc.FC_OK


def test_workspace_sizes(fc_lib):
    size = fc.fc_layernorm_backward_workspace_size
    assert size(-1, 8) == 0 and size(4, 0) == 0 and size(4, (1 << 31) + 1) == 0
    assert size(0, 8) > 0
    assert size(1 << 20, 4096) >= size(100, 4096) >= size(1, 4096) > 0
    assert fc.fc_grad_norm_workspace_size() > 0


def test_binding_refuses_what_a_kernel_could_not_check(fc_lib):
    """Tensors off the GPU never reach the library."""
    with pytest.raises(ValueError):
        fc.LayerGrads([])
    with pytest.raises(ValueError):
        fc.LayerGrads([torch.zeros(4)])
    with pytest.raises(ValueError):
        fc.LayerGrads([torch.zeros(4, dtype=torch.float64)])
    with pytest.raises(ValueError):
        fc.fc_layernorm_forward(torch.zeros(2, 4), None, None, 1e-5, torch.zeros(2, 4))
    with pytest.raises(ValueError):
        fc.fc_layernorm_forward(torch.zeros(4, 2).t(), None, None, 1e-5, torch.zeros(2, 4))


def test_layernorm_formula_against_differences():
    """The 64-bit backward form of the tests is the derivative of the forward one."""
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    for rows, cols in ((1, 2), (3, 5), (4, 33)):
        x, w, b, dy = rnd(rows, cols), rnd(cols), rnd(cols), rnd(rows, cols)
        loss = lambda x, w, b: float((ops_ref.layernorm(x, w, b, 1e-5)[0][0] * dy).sum())  # noqa
        (_, mean, rstd), _ = ops_ref.layernorm(x, w, b, 1e-5)
        (dx, dw, db), _ = ops_ref.layernorm_backward(dy, x, w, mean, rstd)
        e = 1e-6
        for t, grad in ((x, dx), (w, dw), (b, db)):
            flat, gflat = t.view(-1), grad.reshape(-1)
            for i in range(flat.numel()):
                keep = float(flat[i])
                flat[i] = keep + e
                up = loss(x, w, b)
                flat[i] = keep - e
                down = loss(x, w, b)
                flat[i] = keep
                # central differences: e^2 times a third derivative, and
                # 1e-16 of a loss of order cols over e
                assert abs((up - down) / (2 * e) - float(gflat[i])) < 1e-5 * (
                    1 + float(rstd.max()) ** 3 * cols)
