"""Refusals of the mixture-of-experts calls that need no GPU: every bad argument
is turned away before anything touches a device."""
import pytest


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import quantized_weight_quant_gb300 as q
    return q


X, B, IDS, WTS, M, H, G, O, Y, W, W2 = (0x100000 * k for k in range(1, 12))


def _route(q, l=X, kind=0, ld=64, bias=B, S=4, E=64, k=8, score=1, n=8, keep=4, top=2, norm=1, scale=2.5, ids=IDS, w=WTS):
    return q.lib.b200q_moe_route(l, kind, ld, bias, S, E, k, score, n, keep, top, norm, scale, ids, w, None)


@pytest.mark.parametrize("bad", [
    dict(l=None), dict(ids=None), dict(w=None), dict(kind=3), dict(kind=-1), dict(S=-1), dict(E=0), dict(E=1025, ld=1025, n=1, keep=1),
    dict(k=0), dict(k=33), dict(E=4, k=5, n=1, keep=1), dict(score=2), dict(score=-1), dict(n=0), dict(n=7), dict(n=33),
    dict(n=64), dict(keep=0), dict(keep=9), dict(top=0), dict(top=3), dict(n=8, E=8, k=2), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(ld=63), dict(ld=1 << 60), dict(l=X + 2), dict(l=X + 1, kind=2), dict(ids=IDS + 2),
    dict(w=WTS + 1), dict(bias=B + 2), dict(ids=X), dict(w=X + 4), dict(w=IDS), dict(w=IDS + 4), dict(ids=B), dict(w=B + 16),
    dict(ids=X + 256, ld=80),
], ids=str)
def test_route_refusals(q, bad):
    assert _route(q, **bad) == q.EINVAL
    assert "b200q_moe_route" in q.last_error()


def test_experts_refusals(q):
    L = q.lib
    assert not L.b200q_experts_create(None, None, None, 1)
    assert "NULL" in q.last_error()
    for E in (0, -1, 1025):
        assert not L.b200q_experts_create(None, None, None, E)
        assert "E must be" in q.last_error()
    none = q._ptr_array([0], lambda v: v)
    assert not L.b200q_experts_create(none, none, none, 1)
    assert "tensor is NULL" in q.last_error()
    L.b200q_experts_free(None)               # a no-op
    q.experts_free(None)
    with pytest.raises(ValueError):
        q.experts_create([1], [1, 2], [1])
    with pytest.raises(q.B200QError):
        q.Experts([], [], [])
    assert L.b200q_moe_experts(None, X, 0, 64, IDS, WTS, 2, 4, None, 0, Y, 64, 1, None) == q.EINVAL
    assert "handle is NULL" in q.last_error()


def _norm(q, m=M, kind=0, ldm=64, h=H, ldh=64, g=G, ldg=64, gc=64, wp=W2, rs=1.0, os=1.0, o=O, ldo=64, w=W, y=Y, yk=0, ldy=64, S=4,
          D=64, eps=1e-6):
    return q.lib.b200q_block_norm(m, kind, ldm, h, ldh, g, ldg, gc, wp, rs, os, o, ldo, w, y, yk, ldy, S, D, eps, None)


@pytest.mark.parametrize("bad", [
    dict(m=None), dict(o=None, y=None), dict(w=None), dict(kind=3), dict(yk=3), dict(yk=-1), dict(S=-1), dict(D=0), dict(D=65),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rs=float("nan")), dict(os=float("inf")), dict(gc=2),
    dict(gc=0), dict(ldm=63), dict(ldh=63), dict(ldg=63), dict(ldo=63), dict(ldy=63), dict(ldm=-64), dict(ldg=-64), dict(m=M + 2),
    dict(h=H + 2), dict(g=G + 1), dict(o=O + 2), dict(y=Y + 2), dict(y=Y + 1, yk=1), dict(w=W + 2), dict(wp=W2 + 1),
    dict(y=M), dict(y=H), dict(y=G), dict(y=O), dict(y=W), dict(y=W2), dict(y=M + 64), dict(o=M + 4), dict(o=H + 16),
    dict(o=M, ldo=128), dict(o=H, ldo=65), dict(o=G), dict(o=W), dict(o=W2), dict(g=Y, ldg=0), dict(g=O + 60, ldg=0, gc=1),
    dict(ldm=1 << 60), dict(ldy=1 << 60),
], ids=str)
def test_norm_refusals(q, bad):
    assert _norm(q, **bad) == q.EINVAL
    assert "b200q_block_norm" in q.last_error()


def test_no_rows_is_a_no_op(q):
    assert _route(q, S=0, l=None, ids=None, w=None, bias=None) == q.OK
    assert _norm(q, S=0, m=None, h=None, g=None, o=None, y=None, w=None, wp=None) == q.OK


def test_binding_refusals(q):
    import torch
    a = torch.zeros(4, 64)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):                              # no CUDA tensors
        q.moe_route(a, ids, torch.zeros(4, 2), 4, 64, 2)
    with pytest.raises(ValueError):
        q.block_norm(a, 4, 64, 1e-6, y=a, w=a[0])
    with pytest.raises(TypeError):
        q.moe_experts(7, a, ids, a, a, 4, 2)


def test_self_test_refusals(q):
    for bad in ((-2, False), (2 * 10 ** 9 + 1, False), (-1, True), (10 ** 8 + 1, True)):
        with pytest.raises(q.B200QError):
            q.selftest_moe(*bad)
    q.selftest_moe(5, True)
    q.selftest_moe()


def test_experts_create_tells_a_failed_call_from_a_bad_argument(q, monkeypatch):
    class Failing:
        def b200q_experts_create(self, *a):
            return None
    monkeypatch.setattr(q, "lib", Failing())
    for msg, status in (("b200q_experts_create: out of host memory", q.ENOMEM), ("b200q_experts_create: out of memory (cudaErrorMemoryAllocation)", q.ENOMEM),
                        ("b200q_experts_create: encoding a tensor map failed", q.ECUDA),
                        ("b200q_experts_create: unspecified launch failure (cudaErrorLaunchFailure)", q.ECUDA),
                        ("b200q_experts_create: a message on memory (cudaErrorInvalidValue)", q.ECUDA),
                        ("b200q_experts_create: gate 0 is not [8, 8] in the first tensor's format", q.EINVAL)):
        monkeypatch.setattr(q, "last_error", lambda: msg)
        with pytest.raises(q.B200QError) as e:
            q.experts_create([1], [2], [3])
        assert e.value.status == status
