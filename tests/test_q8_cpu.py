"""Refusals of the 8-bit activation calls that need no GPU: every bad argument
is turned away before anything touches a device."""
import pytest


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import quantized_weight_quant_gb300 as q
    return q


X, R, H, W, C, SC = (0x100000 * k for k in range(1, 7))


def _quant(q, x=X, kind=0, ldx=64, c=C, ld8=64, sc=SC, S=4, D=64):
    return q.lib.b200q_quantize_q8(x, kind, ldx, c, ld8, sc, S, D, None)


def _norm(q, x=X, r=R, h=H, kind=0, ldx=64, ldr=64, ldh=64, w=W, c=C, ld8=64, sc=SC, S=4, D=64, eps=1e-6):
    return q.lib.b200q_rmsnorm_q8(x, r, h, kind, ldx, ldr, ldh, w, c, ld8, sc, S, D, eps, None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(c=None), dict(sc=None), dict(kind=3), dict(kind=-1), dict(S=-1), dict(D=0), dict(D=65),
    dict(ldx=63), dict(ld8=48), dict(ld8=72), dict(c=C + 8), dict(x=X + 2), dict(x=X + 1, kind=1), dict(sc=SC + 2),
    dict(x=C), dict(x=C + 16), dict(sc=X + 16), dict(sc=C + 16), dict(ldx=1 << 60), dict(ld8=1 << 60),
], ids=str)
def test_quantize_refusals(q, bad):
    assert _quant(q, **bad) == q.EINVAL
    assert "b200q_quantize_q8" in q.last_error()


@pytest.mark.parametrize("bad", [
    dict(w=None), dict(w=W + 1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(r=R + 2),
    dict(h=H + 1), dict(ldr=10), dict(ldh=10), dict(h=X + 4), dict(h=X, ldh=80), dict(h=R + 8), dict(h=R, ldh=128),
    dict(c=H), dict(c=R), dict(c=W), dict(h=W), dict(sc=W), dict(sc=H), dict(sc=R), dict(h=X + 16, ldx=80, ldh=80),
], ids=str)
def test_rmsnorm_refusals(q, bad):
    assert _norm(q, **bad) == q.EINVAL
    assert "b200q_rmsnorm_q8" in q.last_error()


def test_no_rows_is_a_no_op(q):
    assert _quant(q, S=0, x=None, c=None, sc=None) == q.OK
    assert _norm(q, S=0, x=None, r=None, h=None, w=None, c=None, sc=None) == q.OK


def test_products_without_a_tensor(q):
    L = q.lib
    assert L.b200q_matmul_q8(None, C, 64, SC, None, 0, None, 0, X, 0, 64, 1, None) == q.EINVAL
    assert "tensor is NULL" in q.last_error()
    assert L.b200q_glu_q8(None, None, C, 64, SC, None, None, 4, X, 0, 64, 1, None) == q.EINVAL


def test_binding_refusals(q):
    import torch
    a = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        q.quantize_q8(a, None, 4, 64)                 # a CPU tensor
    with pytest.raises(TypeError):
        q.quantize_q8([1.0], None, 1, 1)
    rows = q.Q8Rows(3, 50, device="cpu")
    assert rows.codes.shape == (3, 64) and rows.values().shape == (3, 50)


def test_rows_changed_in_place(q):
    """codes and scales are the caller's to resize or to point elsewhere: nothing goes by an earlier address."""
    import torch
    rows = q.Q8Rows(3, 50, device="cpu")
    old = rows.codes.data_ptr()
    new = torch.full((5, 80), 0x38, dtype=torch.uint8)
    rows.codes.set_(new)
    assert rows.values().data_ptr() == new.data_ptr() != old
    assert rows.values().shape == (5, 50) and (rows.values().float() == 1).all()
    rows._look()
    assert rows._cp == new.data_ptr() and rows._ld == 80
    scales = torch.ones(7)
    rows.scales.set_(scales)
    rows._look()
    assert rows._sp == scales.data_ptr()
    rows.codes.resize_(2, 40)
    with pytest.raises(ValueError):
        rows.values()                                 # 40 columns for 50
    rows = q.Q8Rows(3, 50, device="cpu")
    rows.scales.set_(torch.ones(6)[::2])
    with pytest.raises(ValueError):
        rows._look()                                  # not contiguous
