"""The mixture-of-experts calls against plain 64-bit references.

Tolerances (half a step of a type t: finfo(t).eps / 2):
  moe_route    ids are equal; weights: a softmax or sigmoid of f32 logits is a handful of f32 roundings
               (exponential, sum of at most 1024 terms over a warp, division, product): 2e-6 relative
  moe_experts  g, u within 1e-5 of B = scale * sum |deq x| (the bar of the f32 products); the
               activations' slopes are at most 1.13 and their f32 evaluation within 4e-6; h = act(g) u in f32,
               rounded to f16's 11 bits (half a step 2^-11) where the rows are bf16; the down product within
               1e-5 of scale * sum |deq h| again; one rounding to the output type
  block_norm   a dozen f32 roundings and two sums of squares: 1e-5 of the formula with magnitudes added, then
               one rounding to the output type
"""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

FMTS = {"i8": 1, "i4": 2, "i2": 3}
BITS = {"i8": 8, "i4": 4, "i2": 2}
ZERO = {"i8": 0, "i4": 8, "i2": 2}
TYPES = ["f32", "f16", "bf16"]


@pytest.fixture(scope="module")
def q():
    import torch
    torch.cuda.set_device(0)
    import quantized_weight_quant_gb300 as q
    return q


def _type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _half_step(name):
    return {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[name]


def _tiny(name):
    """Half the smallest step of the type (its subnormal grid)."""
    return {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[name]


def _dev(a, name="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(_type(name))


def _np64(t):
    return t.double().cpu().numpy()


def _near(got, want, tol, kind, what=""):
    got = _np64(got)
    assert np.isfinite(got).all(), what
    err, room = np.abs(got - want), tol + _half_step(kind) * (np.abs(want) + tol) + _tiny(kind)
    assert (err <= room).all(), "%s: %g of the tolerance" % (what, (err / room).max())


# ---------------------------------------------------------------- routing
def _route_ref(l, k, score, bias, n, keep, top, norm, scale):
    """ids and weights of the formula in 64 bits; -infinity masks, NaN poisons the weights."""
    S, E = l.shape
    ids, wts = np.full((S, k), -1, np.int32), np.zeros((S, k))
    for r in range(S):
        row = l[r].astype(np.float64)
        bad = np.isnan(row).any() or (bias is not None and np.isnan(bias).any()) or (score == 0 and np.isposinf(row).any())
        ok = ~np.isnan(row)
        with np.errstate(all="ignore"):
            if score == 0:
                m = row[ok].max() if ok.any() else 0.0
                e = np.where(ok & np.isfinite(row), np.exp(np.where(np.isfinite(row), row, 0) - (m if np.isfinite(m) else 0)), 0.0)
                s = e / e.sum() if e.sum() > 0 else e
            else:
                s = np.where(ok, 1 / (1 + np.exp(-np.where(ok, row, 0))), 0.0)
            c = s + bias.astype(np.float64) if bias is not None else row.copy()
            c[~ok | np.isneginf(row) | np.isnan(c)] = -np.inf
            if n > 1:
                by = np.where(np.isneginf(c), -np.inf, s) if bias is None and top > 1 else c
                value = []
                for g in by.reshape(n, -1):
                    v = np.sort(g[~np.isneginf(g)])[::-1][:top]
                    value.append(v.sum() if len(v) else -np.inf)
                stay = sorted(range(n), key=lambda g: (-value[g], g))[:keep]
                for g in range(n):
                    if g not in stay:
                        c[g * (E // n):(g + 1) * (E // n)] = -np.inf
        best = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if not np.isneginf(c[e])][:k]
        ids[r, :len(best)] = best
        with np.errstate(all="ignore"):
            if score == 0:
                t = np.exp(row[best] - (row[best].max() if norm and best else (m if np.isfinite(m) else 0)))
                w = t / t.sum() if norm else t / e.sum()
            elif norm and len(best):
                lo = min(row[best].max(), 0.0)
                t = np.exp(np.minimum(row[best], 0) - lo) / (1 + np.exp(-np.abs(row[best])))
                w = t / t.sum()
            else:
                w = s[best]
        wts[r, :len(best)] = w * scale
        if bad:
            wts[r] = np.nan
    return ids, wts


def _route(q, l, k, score=1, bias=None, n=1, keep=1, top=1, norm=True, scale=1.0, ld=None):
    import torch
    S, E = l.shape
    ids = torch.full((S, k), -7, dtype=torch.int32, device="cuda")
    wts = torch.full((S, k), float("nan"), device="cuda")
    b = None if bias is None else torch.from_numpy(np.ascontiguousarray(bias, np.float32)).cuda()
    q.moe_route(l, ids, wts, S, E, k, score=score, bias=b, n_group=n, topk_group=keep, group_top=top, norm=norm, scale=scale)
    torch.cuda.synchronize()
    got = ids.cpu().numpy(), wts.double().cpu().numpy()
    want = _route_ref(l.float().cpu().numpy(), k, score, bias, n, keep, top, norm, scale)
    assert np.array_equal(got[0], want[0])
    assert np.array_equal(np.isnan(got[1]), np.isnan(want[1]))
    f = ~np.isnan(want[1])
    assert (np.abs(got[1][f] - want[1][f]) <= 2e-6 * np.abs(want[1][f]) + 1e-37).all()
    return got


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("S,E,k,n,keep,top", [(1, 1, 1, 1, 1, 1), (3, 2, 2, 1, 1, 1), (5, 31, 4, 1, 1, 1), (7, 64, 6, 8, 3, 2), (2, 33, 5, 3, 2, 1),
                                              (4, 256, 8, 8, 4, 2), (1, 1024, 32, 32, 7, 2), (3, 513, 9, 27, 5, 2), (400, 160, 6, 8, 3, 1),
                                              (2, 8, 3, 8, 8, 1), (2, 64, 32, 32, 16, 2)])
def test_route(q, S, E, k, n, keep, top, score, kind):
    l = _dev(1.5 * synth.normal_f32((S, E), S + E, 1), kind)
    bias = (0.1 * synth.normal_f32((E,), S + E, 2)).astype(np.float32)
    _route(q, l, k, score, None, n, keep, top, False)
    _route(q, l, k, score, None, n, keep, top, True, 2.5)
    _route(q, l, k, score, bias, n, keep, top, True, 2.5)
    _route(q, l, k, score, bias, n, keep, top, False)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("n,keep,top", [(1, 1, 1), (8, 3, 2), (8, 3, 1)])
def test_route_ties_go_to_the_lowest_index(q, n, keep, top, score):
    """Equal values, values one f32 step apart, and values that f32 scores cannot tell but 64 bits can."""
    E, k = 64, 12
    bias = np.zeros(E, np.float32)
    rows = [np.zeros(E), np.repeat([1.0, 2.0], 32), np.tile([1.0, 1.0, 2.0, 0.5], 16), np.where(np.arange(E) % 3, -0.0, 0.0)]
    near = np.full(E, 9.0, np.float32) + np.float32(2.0 ** -20) * ((np.arange(E) * 37) % 64)
    rows += [near, 4 + near, np.full(E, 0.25, np.float32) + np.float32(2.0 ** -25) * ((np.arange(E) * 29) % 64)]
    l = _dev(np.stack([np.asarray(r, np.float32) for r in rows]))
    for b in (None, bias, (1e-8 * ((np.arange(E) * 11) % 64)).astype(np.float32), np.full(E, 1e3, np.float32)):
        for norm in (False, True):
            _route(q, l, k, score, b, n, keep, top, norm)


@pytest.mark.parametrize("score", [0, 1])
def test_route_masks_and_values_that_are_not_finite(q, score):
    E, k = 40, 6
    l = synth.normal_f32((12, E), 3, 1)
    l[1, ::2] = -np.inf
    l[2, 3:] = -np.inf                       # fewer than k left
    l[3] = -np.inf                           # none
    l[4, 7] = np.nan
    l[5] = np.nan
    l[6, 9] = np.inf
    l[7, [2, 5]] = np.inf
    l[8] = np.finfo(np.float32).min          # the type's lowest value is a value
    l[9] = -95.0 - np.arange(E)              # scores below f32's range; their ratios are not
    l[10, :5] = 80.0
    l[11, 8:16] = -np.inf                    # a whole group
    bias = (0.1 * synth.normal_f32((E,), 3, 2)).astype(np.float32)
    masked, poisoned = bias.copy(), bias.copy()
    masked[4] = -np.inf
    poisoned[4] = np.nan
    for n, keep, top in ((1, 1, 1), (5, 2, 2), (5, 5, 1)):
        for b in (None, masked, poisoned):
            for norm in (False, True):
                _route(q, _dev(l), k, score, b, n, keep, top, norm)


def test_route_strides_stream_and_rows_behind(q):
    import torch
    S, E, k = 5, 48, 4
    wide = _dev(synth.normal_f32((S, 64), 5, 1), "bf16")
    _route(q, wide[:, 3:3 + E], k, 0)
    ids, wts = torch.full((S + 2, k), -9, dtype=torch.int32, device="cuda"), torch.full((S + 2, k), 5.0, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    q.moe_route(wide[:, :E], ids, wts, S, E, k, stream=st)
    st.synchronize()
    assert (ids[S:] == -9).all() and (wts[S:] == 5).all() and (ids[:S] >= 0).all()


# ---------------------------------------------------------------- experts
def _values(codes, fmt, I):
    c = codes.astype(np.int64)
    if fmt == "i8":
        return np.where(c > 127, c - 256, c).astype(np.float64)
    b = BITS[fmt]
    f = np.stack([(c >> (b * j)) & (2 ** b - 1) for j in range(8 // b)], -1).reshape(c.shape[0], -1)
    return f[:, :I].astype(np.float64) - ZERO[fmt]


class Layer:
    """E random experts: the resident handle and their 64-bit values."""

    def __init__(self, q, fmt, E, D, F, seed=0):
        self.E, self.D, self.F = E, D, F
        self.t, self.v = [[], [], []], [[], [], []]
        for m, (O, I) in enumerate([(F, D), (F, D), (D, F)]):
            for e in range(E):
                codes, scales = synth.quant_tensor(FMTS[fmt], O, I, seed, 10 + 3 * e + m, 0.5, 1.5)
                scales = (scales / (2.0 ** BITS[fmt] / 12 ** 0.5 * I ** 0.5)).astype(np.float32)
                self.t[m].append(q.tensor_upload(FMTS[fmt], O, I, codes, scales))
                self.v[m].append(_values(np.asarray(codes).reshape(O, -1), fmt, I) * scales.astype(np.float64)[:, None])
        self.ex = q.Experts(*self.t)

    def free(self):
        self.ex.free()
        for ts in self.t:
            for t in ts:
                t.free()

    def ref(self, x, ids, wts, act, res, kind):
        """y and its tolerance before the last rounding."""
        y = res.copy() if res is not None else np.zeros_like(x)
        tol = np.zeros_like(x)
        for s in range(x.shape[0]):
            for e, w in zip(ids[s], wts[s]):
                if e < 0:
                    continue
                wg, wu, wd = (self.v[m][e] for m in range(3))
                g, u = wg @ x[s], wu @ x[s]
                dg, du = 1e-5 * (np.abs(wg) @ np.abs(x[s])), 1e-5 * (np.abs(wu) @ np.abs(x[s]))
                a = _act(act, g)
                h = a * u
                dh = (1.13 * dg + 4e-6 * np.abs(g)) * (np.abs(u) + du) + np.abs(a) * du
                h16 = 2.0 ** -11 if kind == "bf16" else 0.0
                y[s] += w * (wd @ h)
                tol[s] += abs(w) * (np.abs(wd) @ (dh + (1e-5 + h16) * (np.abs(h) + dh)))
        return y, tol + 1e-6 * np.abs(y)


def _act(name, v):
    import math
    if name == "relu":
        return np.maximum(v, 0)
    if name == "gelu":
        return 0.5 * v * (1 + np.vectorize(math.erf)(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "none":
        return v
    return v / (1 + np.exp(-v))


def _pick(S, k, E, seed, empty=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(S)]).astype(np.int32)
    ids[rng.random((S, k)) < empty] = -1
    return ids, rng.uniform(0.05, 0.6, (S, k)).astype(np.float32)


def _moe(q, layer, x, ids, wts, kind, act="silu", res=None, y=None):
    import torch
    S, k = ids.shape
    if y is None:
        y = torch.full((S, layer.D), float("nan"), dtype=_type(kind), device="cuda")
    q.moe_experts(layer.ex, x, torch.from_numpy(ids).cuda(), torch.from_numpy(wts).cuda(), y, S, k, act=q.ACTS[act], res=res)
    torch.cuda.synchronize()
    return y


def _check(q, layer, S, k, kind, act="silu", res=True, empty=0.0, seed=0):
    x = _dev(synth.normal_f32((S, layer.D), seed, 1) * np.exp2(np.arange(S) % 5 - 2).astype(np.float32)[:, None], kind)
    r = _dev(synth.normal_f32((S, layer.D), seed, 2), kind) if res else None
    ids, wts = _pick(S, k, layer.E, seed, empty)
    y = _moe(q, layer, x, ids, wts, kind, act, r)
    want, tol = layer.ref(_np64(x), ids, wts.astype(np.float64), act, None if r is None else _np64(r), kind)
    _near(y, want, tol, kind, "S=%d k=%d %s" % (S, k, kind))
    again = _moe(q, layer, x, ids, wts, kind, act, r)
    assert (y.view(dtype=again.dtype) == again).all()
    assert q.device_status() == q.OK
    return x, r, ids, wts, y


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("E,D,F", [(1, 1, 1), (2, 7, 5), (5, 64, 48), (3, 129, 257), (4, 512, 96), (7, 333, 130)])
def test_experts(q, fmt, E, D, F):
    layer = Layer(q, fmt, E, D, F, seed=D)
    for n, (S, k) in enumerate([(1, 1), (1, 8), (2, 3), (5, 2), (8, 1), (9, 4), (17, 3), (33, 2)]):
        _check(q, layer, S, k, TYPES[n % 3], list(q.ACTS)[(n + E) % 5], n % 2 == 0, 0.25 * (n % 3 == 2), seed=n)
    layer.free()


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("fmt", list(FMTS))
def test_experts_ordinary_sizes(q, fmt, kind):
    layer = Layer(q, fmt, 6, 1024, 640, seed=3)
    for S, k in [(1, 4), (8, 2), (40, 3)]:
        _check(q, layer, S, k, kind, seed=S)
    layer.free()


@pytest.mark.parametrize("fmt,D,F", [("i4", 8192, 40), ("i4", 40, 8192), ("i8", 9001, 33), ("i2", 33, 9001), ("i2", 20000, 24), ("i8", 24, 20000)])
def test_experts_long_rows(q, fmt, D, F):
    layer = Layer(q, fmt, 3, D, F, seed=1)
    for S, k, kind in [(1, 2, "f32"), (6, 2, "bf16"), (20, 2, "f16")]:
        _check(q, layer, S, k, kind, seed=S)
    layer.free()


@pytest.mark.parametrize("fmt,D", [("i2", 65536), ("i4", 65536), ("i8", 32768)])
@pytest.mark.parametrize("S", [1, 6, 20])
def test_experts_long_rows_of_one_sign(q, S, fmt, D):
    """The sums grow all along the row, and with them what a truncating accumulator drops.  f16 out and one h: its rounding,
    2^-11 of y, is below the products' 1e-5 of sum |x w|, over 100 times a sum of random signs at these lengths."""
    layer = Layer(q, fmt, 2, D, 1, seed=8)
    x = _dev(0.25 + np.abs(synth.normal_f32((S, D), S, 1)), "f16")
    ids, wts = _pick(S, 1, 2, S)
    y = _moe(q, layer, x, ids, wts, "f16", "none")
    want, tol = layer.ref(_np64(x), ids, wts.astype(np.float64), "none", None, "f16")
    _near(y, want, tol, "f16", "S=%d" % S)
    layer.free()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_experts_long_rows_of_one_sign_many_tiles(q, kind):
    """As above where there are enough rows for every SM; down takes h[0] alone, so that the other rows' errors do not hide its."""
    import torch
    S, D, F = 64, 8192, 2432
    codes = np.random.default_rng(9).integers(0, 256, (2, F, D)).astype(np.uint8)
    down = np.zeros((D, F), np.uint8)
    down[:, 0] = 64
    one = np.ones(F, np.float32)
    ts = [[q.tensor_upload(FMTS["i8"], *c.shape, c, v)] for c, v in
          [(codes[0], one / 4096), (codes[1], one / 4096), (down, np.full(D, 1 / 64, np.float32))]]
    ex = q.Experts(*ts)
    x = _dev(0.25 + np.abs(synth.normal_f32((S, D), 9, 1)), kind)
    y = torch.empty_like(x)
    q.moe_experts(ex, x, torch.zeros(S, 1, dtype=torch.int32, device="cuda"), torch.ones(S, 1, device="cuda"), y, S, 1, act=q.ACTS["none"])
    x = _np64(x)
    wg, wu = (_values(c[:1], "i8", D)[0] / 4096 for c in codes)
    g, u, dg, du = x @ wg, x @ wu, 1e-5 * (x @ np.abs(wg)), 1e-5 * (x @ np.abs(wu))
    h, dh = g * u, dg * (np.abs(u) + du) + np.abs(g) * du
    tol = dh + (1e-5 + (2.0 ** -11 if kind == "bf16" else 0.0)) * (np.abs(h) + dh) + 1e-6 * np.abs(h)
    _near(y, np.repeat(h[:, None], D, 1), np.repeat(tol[:, None], D, 1), kind)
    ex.free()
    for t in ts:
        t[0].free()


@pytest.mark.parametrize("fmt,E,D,F", [("i8", 2, 2048, 64), ("i8", 3, 9001, 40), ("i4", 2, 4097, 77), ("i2", 1, 100, 9001)])
def test_experts_many_tokens_of_few_tiles(q, fmt, E, D, F):
    layer = Layer(q, fmt, E, D, F, seed=D)
    for S, k, kind in [(24, 1, "f32"), (64, E, "bf16"), (33, E, "f16"), (40, E, "f32")]:
        _check(q, layer, S, k, kind, empty=0.1, seed=S)
    layer.free()


def test_experts_many_tokens_and_slots(q):
    """More tokens than one launch plans at once, 32 slots a token, one expert for all of them."""
    layer = Layer(q, "i4", 5, 96, 80, seed=2)
    for S, k in [(64, 8), (65, 1), (130, 2), (300, 1), (3, 32), (70, 32)]:
        _check(q, layer, S, k, "f32", seed=S)
    layer.free()
    one = Layer(q, "i8", 1, 64, 48, seed=4)
    _check(q, one, 100, 1, "bf16", seed=5)
    one.free()


def test_experts_empty_slots_twice_and_in_place(q):
    import torch
    layer = Layer(q, "i4", 4, 160, 96, seed=6)
    x = _dev(synth.normal_f32((5, 160), 1, 1), "bf16")
    ids = np.array([[-1, -1, -1], [2, 2, -1], [0, 3, 0], [-1, 1, -1], [3, 3, 3]], np.int32)
    wts = np.array([[9, 9, 9], [.5, .25, np.nan], [0, 1, 0], [np.inf, 1, 7], [-1, .5, .5]], np.float32)
    want, tol = layer.ref(_np64(x), ids, wts.astype(np.float64), "silu", None, "bf16")
    y = _moe(q, layer, x, ids, wts, "bf16")
    _near(y, want, tol, "bf16")
    assert (y[0] == 0).all()
    # the residual stream updated in place, rows of a wider buffer, rows behind the last left alone
    buf = _dev(synth.normal_f32((7, 200), 1, 2), "bf16")
    was = buf.clone()
    r = buf[:5, 16:176]
    want, tol = layer.ref(_np64(x), ids, wts.astype(np.float64), "silu", _np64(r), "bf16")
    _moe(q, layer, x, ids, wts, "bf16", res=r, y=r)
    _near(r, want, tol, "bf16")
    assert torch.equal(r[0], was[0, 16:176])
    assert torch.equal(buf[5:], was[5:]) and torch.equal(buf[:, :16], was[:, :16]) and torch.equal(buf[:, 176:], was[:, 176:])
    layer.free()


@pytest.mark.parametrize("kind", TYPES)
def test_experts_strides_and_alignment(q, kind):
    import torch
    D, F, S = 121, 77, 6
    layer = Layer(q, "i4", 3, D, F, seed=7)
    xb = _dev(synth.normal_f32((S, 140), 2, 1), kind)
    rb = _dev(synth.normal_f32((S, 133), 2, 2), kind)
    yb = torch.full((S, 129), 3.0, dtype=_type(kind), device="cuda")
    ids, wts = _pick(S, 2, 3, 1)
    x, r, y = xb[:, 5:5 + D], rb[:, 1:1 + D], yb[:, 3:3 + D]
    _moe(q, layer, x, ids, wts, kind, res=r, y=y)
    want, tol = layer.ref(_np64(x), ids, wts.astype(np.float64), "silu", _np64(r), kind)
    _near(y, want, tol, kind)
    assert (yb[:, :3] == 3).all() and (yb[:, 3 + D:] == 3).all()
    layer.free()


def test_experts_rows_do_not_depend_on_each_other(q):
    """A token among others gives the same bits where one of them is NaN and one infinite."""
    import torch
    layer = Layer(q, "i4", 6, 256, 160, seed=8)
    x = _dev(synth.normal_f32((9, 256), 3, 1), "bf16")
    ids, wts = _pick(9, 3, 6, 2)
    y = _moe(q, layer, x, ids, wts, "bf16")
    bad = x.clone()
    bad[2, 100] = float("nan")
    bad[5, 3] = float("inf")
    z = _moe(q, layer, bad, ids, wts, "bf16")
    for s in range(9):
        if s == 2:
            assert torch.isnan(z[s]).all()
        elif s == 5:
            assert (~torch.isfinite(z[s])).any()
        else:
            assert torch.equal(z[s], y[s])
    layer.free()


@pytest.mark.parametrize("top", [2.0 ** -120, 2.0 ** -60, 2.0 ** 60])
def test_experts_small_and_large_values(q, top):
    """Rows far from 1 keep f32's relative accuracy (no activation: the result is quadratic in x)."""
    layer = Layer(q, "i4", 2, 96, 64, seed=9)
    S = 3
    x = (synth.normal_f32((S, 96), 4, 1) * np.float32(top)).astype(np.float32)
    ids, wts = _pick(S, 2, 2, 3)
    import torch
    xd = torch.from_numpy(x).cuda()
    y = _np64(_moe(q, layer, xd, ids, wts, "f32", "none"))
    want, tol = layer.ref(x.astype(np.float64), ids, wts.astype(np.float64), "none", None, "f32")
    assert (np.abs(y - want) <= tol + 2.0 ** -24 * np.abs(want) + 96 * 64 * 2.0 ** -149).all()
    layer.free()


def test_experts_outside_numbers_are_reported(q):
    import torch
    layer = Layer(q, "i4", 3, 64, 32, seed=10)
    x = _dev(synth.normal_f32((2, 64), 5, 1))
    for outside in (3, -2, 2 ** 31 - 1, -2 ** 31):
        ids, wts = np.array([[0, outside], [1, 2]], np.int32), np.full((2, 2), 0.5, np.float32)
        y = _moe(q, layer, x, ids, wts, "f32")
        with pytest.raises(q.B200QError) as e:
            q.device_status()
        assert e.value.status == q.EINVAL and "expert number" in str(e.value)
        assert q.device_status() == q.OK
        want, tol = layer.ref(_np64(x), np.array([[0, -1], [1, 2]]), wts.astype(np.float64), "silu", None, "f32")
        _near(y, want, tol, "f32")
    layer.free()


def test_experts_refusals(q):
    import torch
    layer = Layer(q, "i4", 2, 64, 32, seed=11)
    L, h = q.lib, layer.ex.handle
    x, y, r = (torch.zeros(4, 64, device="cuda") for _ in range(3))
    ids, w = torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(4, 2, device="cuda")
    good = dict(x=x.data_ptr(), t=0, ldx=64, ids=ids.data_ptr(), w=w.data_ptr(), k=2, act=4, r=r.data_ptr(), ldr=64, y=y.data_ptr(), ldy=64, S=4)
    call = lambda **b: L.b200q_moe_experts(h, *(dict(good, **b)[n] for n in ("x", "t", "ldx", "ids", "w", "k", "act", "r", "ldr", "y", "ldy", "S")), None)  # noqa: E731
    assert call() == q.OK and call(S=0, x=None, y=None, ids=None, w=None) == q.OK and call(r=None) == q.OK
    for bad in (dict(x=None), dict(y=None), dict(ids=None), dict(w=None), dict(t=3), dict(ldx=63), dict(ldy=10), dict(ldr=0), dict(k=0),
                dict(k=33), dict(act=5), dict(act=-1), dict(S=-1), dict(x=good["x"] + 2), dict(ids=good["ids"] + 2), dict(w=good["w"] + 1),
                dict(y=good["x"]), dict(y=good["x"] + 256), dict(y=good["ids"]), dict(y=good["w"]), dict(r=good["y"] + 16), dict(r=good["y"], ldr=65)):
        assert call(**bad) == q.EINVAL, bad
        assert "b200q_moe_experts" in q.last_error()
    other = q.tensor_upload(q.I8, 32, 64, np.zeros((32, 64), np.uint8), np.ones(32, np.float32))
    f32 = q.tensor_upload(q.F32, 32, 64, np.zeros((32, 64), np.float32), None)
    grouped = q.tensor_upload(q.I4, 32, 64, np.zeros((32, 32), np.uint8), np.ones((32, 2), np.float32), gs=32)
    g, u, d = (layer.t[m] for m in range(3))
    for bad in (([g[0], other], u, d), ([f32], [f32], d[:1]), ([grouped], [grouped], d[:1]), (g, u, [d[0], g[1]]), (g, [u[0], d[1]], d)):
        with pytest.raises(q.B200QError) as e:
            q.Experts(*bad)
        assert e.value.status == q.EINVAL
    for t in (other, f32, grouped):
        t.free()
    for bad in ((x, ids.long(), w), (x, ids, w.double()), (x[:, :32], ids, w), (x, ids[:, :1], w), (x, ids.t().contiguous().t(), w)):
        with pytest.raises(ValueError):
            q.moe_experts(layer.ex, *bad, y, 4, 2)
    with pytest.raises(ValueError):
        q.moe_experts(layer.ex, x, ids, w, y.half(), 4, 2)
    layer.ex.free()
    layer.ex.free()
    with pytest.raises(q.B200QError):
        q.moe_experts(layer.ex, x, ids, w, y, 4, 2)
    layer.free()


# ---------------------------------------------------------------- norm
def _norm_ref(m, h, gate, wp, w, rs, os, eps):
    p = m * (wp / np.sqrt((m * m).mean(1, keepdims=True) + eps)) if wp is not None else m
    if gate is not None:
        p = p * gate
    a = rs * h if h is not None else 0.0
    n = a + os * p
    mag = np.abs(a) + np.abs(os * p)
    y = n * (w / np.sqrt((n * n).mean(1, keepdims=True) + eps)) if w is not None else None
    ty = 1e-5 * mag * np.abs(w) / np.sqrt((n * n).mean(1, keepdims=True) + eps) if w is not None else None
    return n, 1e-5 * mag, y, ty


def _norm(q, m, h=None, gate=None, wp=None, w=None, rs=1.0, os=1.0, kind="f32", ykind="f32", out=True, eps=1e-6):
    import torch
    S, D = m.shape
    o = torch.full((S, D), float("nan"), dtype=_type(kind), device="cuda") if out else None
    y = torch.full((S, D), float("nan"), dtype=_type(ykind), device="cuda") if w is not None else None
    q.block_norm(m, S, D, eps, h=h, h_out=o, w_post=wp, gate=gate, res_scale=rs, out_scale=os, w=w, y=y)
    torch.cuda.synchronize()
    g = None if gate is None else _np64(gate if gate.dim() == 2 else gate[None])
    n, tn, yr, ty = _norm_ref(_np64(m), None if h is None else _np64(h), g, None if wp is None else _np64(wp),
                              None if w is None else _np64(w), rs, os, eps)
    if out:
        _near(o, n, tn, kind, "h' %dx%d" % (S, D))
    if w is not None:
        _near(y, yr, ty, ykind, "y %dx%d" % (S, D))
    return o, y


NORM_SIZES = [(1, 1), (2, 7), (3, 8), (5, 33), (1, 255), (2, 1024), (7, 2049), (1, 6144), (3, 5003), (2, 16384), (2, 16385), (1, 40000),
              (400, 64), (310, 96), (320, 1000), (311, 1003)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("S,D", NORM_SIZES)
def test_norm(q, S, D, kind):
    m, h = (_dev(synth.normal_f32((S, D), D, j) * np.exp2(np.arange(S) % 7 - 3).astype(np.float32)[:, None], kind) for j in (1, 2))
    wp, w = (_dev(0.5 + np.abs(synth.normal_f32((D,), D, j))) for j in (3, 4))
    gates = [None] + [_dev(synth.normal_f32(s, D, 5), kind) for s in ((S, D), (1, D), (D,), (S, 1))]
    for n, gate in enumerate(gates):
        yk = TYPES[(n + D) % 3]
        _norm(q, m, h, gate, wp, w, 0.7, 0.25, kind, yk)
        _norm(q, m, h if n % 2 else None, gate, None if n % 2 else wp, w, 1.0, -1.5, kind, yk, out=n % 2 == 0)
    _norm(q, m, h, None, wp, None, kind=kind)


@pytest.mark.parametrize("kind", TYPES)
def test_norm_in_place_strides_and_rows_behind(q, kind):
    import torch
    for D, off, wide in ((64, 0, 80), (64, 8, 80), (61, 3, 77), (1000, 5, 1011)):
        S = 4
        hb, mb = (_dev(synth.normal_f32((S + 1, wide), D, j), kind) for j in (1, 2))
        gb = _dev(synth.normal_f32((S, wide), D, 3), kind)
        yb = torch.full((S + 1, wide), 3.0, dtype=_type("f16"), device="cuda")
        wp, w = (_dev(0.5 + np.abs(synth.normal_f32((D + 1,), D, j)))[1:] for j in (4, 5))
        for inplace in ("h", "m"):
            h, m, g, y = (b[:S, off:off + D] for b in (hb.clone(), mb.clone(), gb, yb))
            before = h._base.clone() if inplace == "h" else m._base.clone()
            n, tn, yr, ty = _norm_ref(_np64(m), _np64(h), _np64(g), _np64(wp), _np64(w), 0.5, 2.0, 1e-6)
            o = h if inplace == "h" else m
            q.block_norm(m, S, D, 1e-6, h=h, h_out=o, w_post=wp, gate=g, res_scale=0.5, out_scale=2.0, w=w, y=y)
            torch.cuda.synchronize()
            _near(o, n, tn, kind)
            _near(y, yr, ty, "f16")
            after = o._base
            assert torch.equal(after[S:], before[S:]) and torch.equal(after[:, :off], before[:, :off]) and torch.equal(after[:, off + D:], before[:, off + D:])
            assert (yb[S:] == 3).all() and (yb[:, :off] == 3).all() and (yb[:, off + D:] == 3).all()


def test_norm_y_comes_from_the_unrounded_sum(q):
    """bf16 streams, f32 y: a y from the stored h' would be off by up to 2^-8."""
    m, h = (_dev(synth.normal_f32((3, 512), 1, j), "bf16") for j in (1, 2))
    w = _dev(np.ones(512))
    _norm(q, m, h, None, w, w, kind="bf16", ykind="f32")


def test_norm_zero_rows_nan_and_one_row_for_all(q):
    import torch
    S, D = 4, 96
    m, h = (_dev(synth.normal_f32((S, D), 2, j)) for j in (1, 2))
    m[0] = 0
    h[0] = 0
    w = _dev(np.ones(D))
    _norm(q, m, h, None, w, w)
    m[1, 5], h[2, 7] = float("nan"), float("inf")
    o, y = torch.empty_like(m), torch.empty_like(m)
    q.block_norm(m, S, D, 1e-6, h=h, h_out=o, w_post=w, w=w, y=y)
    assert (y[0] == 0).all() and torch.isnan(y[1]).all() and (~torch.isfinite(y[2])).any() and torch.isfinite(y[3]).all()
    gate = _dev(synth.normal_f32((D,), 2, 3))
    a, b = _norm(q, m[3:], h[3:], gate[None].expand(1, D), w, w), _norm(q, m[3:], h[3:], gate, w, w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    many = torch.empty_like(m)
    q.block_norm(m, S, D, 1e-6, h=h, h_out=many, gate=gate[None].expand(S, D))     # a row stride of 0
    torch.cuda.synchronize()
    assert torch.allclose(many[3], h[3] + gate * m[3], rtol=1e-6, atol=1e-6)


# ---------------------------------------------------------------- together
class Block:
    """Norm -> router -> experts -> norm after, gate, residual, norm before the next block."""

    def __init__(self, q, D=256, F=160, E=12, k=3, S=6, kind="bf16"):
        import torch
        self.q, self.D, self.E, self.k, self.S, self.kind = q, D, E, k, S, kind
        self.layer = Layer(q, "i4", E, D, F, seed=20)
        self.wr = (synth.normal_f32((E, D), 21, 1) / D ** 0.5).astype(np.float32)
        self.router = q.tensor_upload(q.F32, E, D, self.wr, None)
        self.w = [_dev(0.5 + np.abs(synth.normal_f32((D,), 21, j))) for j in (2, 3, 4)]
        self.bias = _dev(0.05 * synth.normal_f32((E,), 21, 5))
        t = _type(kind)
        new = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        self.m, self.h, self.h1, self.h2, self.a = (new(S, D, d=t) for _ in range(5))
        self.n1, self.n2 = new(S, D), new(S, D, d=t)
        self.logits, self.ids, self.wts = new(S, E), new(S, k, d=torch.int32), new(S, k)

    def step(self):
        q, S, D = self.q, self.S, self.D
        q.block_norm(self.m, S, D, 1e-6, h=self.h, h_out=self.h1, w=self.w[0], y=self.n1)
        q.matmul(self.router, self.n1, self.logits, S)
        q.moe_route(self.logits, self.ids, self.wts, S, self.E, self.k, score=q.SCORE_SIGMOID, bias=self.bias, n_group=4, topk_group=2,
                    group_top=2, norm=True, scale=2.5)
        self.x = self.n1 if self.kind == "f32" else self.n1.to(_type(self.kind))
        q.moe_experts(self.layer.ex, self.x, self.ids, self.wts, self.a, S, self.k)
        q.block_norm(self.a, S, D, 1e-6, h=self.h1, h_out=self.h2, w_post=self.w[1], w=self.w[2], y=self.n2, out_scale=0.5)

    def check(self):
        """Each call against its own inputs as the device has them: what one rounds does not blur the next."""
        f = _np64
        n, tn, y, ty = _norm_ref(f(self.m), f(self.h), None, None, f(self.w[0]), 1.0, 1.0, 1e-6)
        _near(self.h1, n, tn, self.kind)
        _near(self.n1, y, ty, "f32")
        lr = f(self.n1) @ self.wr.T.astype(np.float64)
        assert (np.abs(f(self.logits) - lr) <= 1e-5 * (np.abs(f(self.n1)) @ np.abs(self.wr.T))).all()
        ids, wts = _route_ref(self.logits.cpu().numpy(), self.k, 1, self.bias.cpu().numpy(), 4, 2, 2, True, 2.5)
        assert np.array_equal(ids, self.ids.cpu().numpy())
        assert (np.abs(f(self.wts) - wts) <= 2e-6 * wts).all()
        a, ta = self.layer.ref(f(self.x), ids, f(self.wts), "silu", None, self.kind)
        _near(self.a, a, ta, self.kind)
        n, tn, y, ty = _norm_ref(f(self.a), f(self.h1), None, f(self.w[1]), f(self.w[2]), 1.0, 0.5, 1e-6)
        _near(self.h2, n, tn, self.kind)
        _near(self.n2, y, ty, self.kind)

    def fill(self, seed):
        self.m.copy_(_dev(synth.normal_f32((self.S, self.D), seed, 1)))
        self.h.copy_(_dev(synth.normal_f32((self.S, self.D), seed, 2)))


@pytest.mark.parametrize("kind", TYPES)
def test_block(q, kind):
    import torch
    b = Block(q, kind=kind)
    for seed in (1, 2):
        b.fill(seed)
        b.step()
        torch.cuda.synchronize()
        b.check()
    assert q.device_status() == q.OK
    b.layer.free()
    b.router.free()


def test_block_captured_and_replayed_with_other_routing(q):
    """Two captured graphs replayed in turn, on inputs that route differently, beside eager calls on another stream."""
    import torch
    blocks = [Block(q, S=s) for s in (1, 6)]
    graphs = []
    for b in blocks:
        b.fill(1)
        b.step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.step()
        graphs.append(g)
    seen = set()
    side, eager = torch.cuda.Stream(), Block(q, S=9)
    eager.fill(7)
    torch.cuda.synchronize()
    for seed in range(2, 6):
        for b in blocks:
            b.fill(seed)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            eager.step()
        for _ in range(3):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for b in blocks + [eager]:
            b.check()
        seen.add(tuple(blocks[1].ids.flatten().tolist()))
    assert len(seen) > 1
    assert q.device_status() == q.OK
    for b in blocks + [eager]:
        b.layer.free()
        b.router.free()


def test_two_streams_at_once(q):
    import torch
    layer = Layer(q, "i4", 6, 512, 320, seed=30)
    xs = [_dev(synth.normal_f32((S, 512), S, 1), "bf16") for S in (4, 11)]
    picks = [_pick(S, 3, 6, S) for S in (4, 11)]
    alone = [_moe(q, layer, x, *p, "bf16").clone() for x, p in zip(xs, picks)]
    streams = [torch.cuda.Stream() for _ in xs]
    args = [(x, torch.from_numpy(i).cuda(), torch.from_numpy(w).cuda(), torch.zeros_like(x)) for x, (i, w) in zip(xs, picks)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (x, i, w, y) in zip(streams, args):
            q.moe_experts(layer.ex, x, i, w, y, x.shape[0], 3, stream=st)
    torch.cuda.synchronize()
    for a, (_, _, _, y) in zip(alone, args):
        assert torch.equal(a, y)
    layer.free()


def test_layers_made_where_freed_ones_were(q):
    """A layer's table often lies where a freed layer's did: its tensor maps are those of the new one, of another shape and
    other codes, for few and for many columns, eager and when a graph of the new layer is replayed."""
    import torch
    for n in range(12):
        D, F = ((1024, 640), (256, 520), (640, 1024))[n % 3]
        layer = Layer(q, list(FMTS)[n // 2 % 3], 8, D, F, seed=n)
        for S, k in ((1, 3), (6, 2), (64, 4)):
            x, r, ids, wts, y = _check(q, layer, S, k, TYPES[n % 3], seed=n)
            if n % 4 == 0:
                args = torch.from_numpy(ids).cuda(), torch.from_numpy(wts).cuda(), torch.zeros_like(y)
                torch.cuda.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    q.moe_experts(layer.ex, x, *args, S, k, res=r)
                g.replay()
                torch.cuda.synchronize()
                assert torch.equal(args[2], y)
        layer.free()


@pytest.mark.parametrize("S,k", [(5, 2), (64, 4)])
def test_experts_that_give_up_report_it(q, S, k):
    """Prepared rows that never come whole, for few and for many columns: the call ends, says so, and the next one is right."""
    layer = Layer(q, "i4", 8, 1024, 640, seed=31)
    _check(q, layer, S, k, "bf16")
    x = _dev(synth.normal_f32((S, 1024), 3, 1), "bf16")
    ids, wts = _pick(S, k, 8, 3)
    q.selftest_moe(1000000, True)
    try:
        _moe(q, layer, x, ids, wts, "bf16")
        with pytest.raises(q.B200QError) as e:
            q.device_status()
        assert e.value.status == q.ETIMEOUT
    finally:
        q.selftest_moe()
    assert q.device_status() == q.OK
    _check(q, layer, S, k, "bf16")
    layer.free()


# ---------------------------------------------------------------- accuracy of the products
def _pack(v, fmt):
    """Host codes of whole numbers [O, I]."""
    b = BITS[fmt]
    c = (v + ZERO[fmt]).astype(np.uint8) if fmt != "i8" else v.astype(np.int8).view(np.uint8)
    n = 8 // b
    c = np.pad(c, ((0, 0), (0, -c.shape[1] % n)), constant_values=ZERO[fmt]).reshape(c.shape[0], -1, n).astype(np.uint32)
    return (c << (b * np.arange(n, dtype=np.uint32))).sum(-1).astype(np.uint8)


class Given:
    """One expert of given whole numbers: gate and up [F, D], down [D, F], with one scale per row."""

    def __init__(self, q, fmt, mats):
        self.F, self.D = mats[0][0].shape
        self.t = [q.tensor_upload(FMTS[fmt], *v.shape, _pack(v, fmt), np.asarray(s, np.float32)) for v, s in mats]
        self.ex = q.Experts(*([t] for t in self.t))

    def free(self):
        self.ex.free()
        for t in self.t:
            t.free()


def _given(q, layer, x, kind):
    import torch
    S = x.shape[0]
    xd = torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(_type(kind))
    y = torch.full((S, layer.D), float("nan"), dtype=_type(kind), device="cuda")
    q.moe_experts(layer.ex, xd, torch.zeros(S, 1, dtype=torch.int32, device="cuda"), torch.ones(S, 1, device="cuda"), y, S, 1, act=q.ACT_NONE)
    torch.cuda.synchronize()
    return _np64(xd), _np64(y)


def _opposite(O, I, fmt, rng, zeros=0.0):
    """Random whole numbers whose second half is the first's with the other sign: a row that repeats its first half in the second has product 0."""
    top = {"i8": 127, "i4": 7, "i2": 1}[fmt]
    half = rng.integers(-top, top + 1, (O, I // 2))
    half[rng.random(half.shape) < zeros] = 0
    return np.concatenate([half, -half], 1)


def _one_of(O, I, of):
    """[O, I] with a 1 in column of(o) of row o."""
    v = np.zeros((O, I), np.int64)
    v[np.arange(O), of(np.arange(O))] = 1
    return v


# tokens and sizes: one token, few columns, many columns (rows enough for all SMs)
PRODUCTS = [(1, 2048, 48), (8, 2048, 48), (64, 8192, 2432)]


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("S,D,F", PRODUCTS)
def test_experts_a_large_value_on_a_weight_of_zero(q, S, D, F, fmt):
    """gate's product is 0 by opposite halves and a row's largest values meet codes of 0, so that sum |deq x| is that of the others alone; u = 1 and
    y[d] = h[d % F] are exact.  The error has to stay within 1e-5 of that sum however large those values are."""
    rng = np.random.default_rng(D + S)
    gate, large = _opposite(F, D, fmt, rng, 0.3), rng.permutation(np.arange(1, D))[:3]
    large[2] = D - 1                                             # in the last piece of the row
    gate[:, 0] = gate[:, D // 2] = 0
    gate[:, large] = gate[:, (large + D // 2) % D] = 0
    layer = Given(q, fmt, [(gate, np.ones(F)), (_one_of(F, D, lambda o: 0 * o), np.ones(F)), (_one_of(D, F, lambda o: o % F), np.ones(D))])
    for kind in TYPES:
        for ratio in (1e3, 1e4, 2.0 ** 30):
            x = synth.normal_f32((S, D), D, 1)
            x[:, D // 2:] = x[:, :D // 2]
            if kind == "f16":                                    # the largest of the type's values is 65504
                x *= np.float32(min(1.0, 2.0 ** 15 / ratio))
            x[:, large] = np.array([1, -1, 0.75]) * ratio * (min(1.0, 2.0 ** 15 / ratio) if kind == "f16" else 1.0)
            x[:, 0] = 1
            x, y = _given(q, layer, x, kind)
            x[:, large] = 0
            tol = 1e-5 * (np.abs(x) @ np.abs(gate).T.astype(np.float64))
            worst = (np.abs(y) / tol[:, np.arange(D) % F]).max()
            assert worst <= 1.01, "%s, largest %g times the rest: %g of the tolerance" % (kind, ratio, worst)
    layer.free()


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("zeros", [0.5, 0.9, 0.999])
@pytest.mark.parametrize("S,D,F", PRODUCTS)
def test_experts_weights_near_zero(q, S, D, F, zeros, fmt):
    """Rows of one sign on codes most of which are 0: the products' error goes by sum |deq x|, not by sum |x|."""
    rng = np.random.default_rng(D + S)
    gate = np.sign(_opposite(F, D, fmt, rng, zeros))
    gate[:, 0] = gate[:, D // 2] = 0
    layer = Given(q, fmt, [(gate, np.ones(F)), (_one_of(F, D, lambda o: 0 * o), np.ones(F)), (_one_of(D, F, lambda o: o % F), np.ones(D))])
    for kind in TYPES:
        x = 0.25 + np.abs(synth.normal_f32((S, D), D, 1))
        x[:, D // 2:] = x[:, :D // 2]
        x[:, 0] = 1
        x, y = _given(q, layer, x, kind)
        tol = 1e-5 * (np.abs(x) @ np.abs(gate).T.astype(np.float64))[:, np.arange(D) % F]
        assert (np.abs(y) <= 1.01 * tol).all(), "%s: %g" % (kind, (np.abs(y) / np.maximum(tol, 1e-30)).max())
    layer.free()


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("S,D,F", PRODUCTS)
def test_experts_down_of_a_large_h_on_a_weight_of_zero(q, S, D, F, fmt):
    """As above for down: h repeats its first half, two of its values are 2^10, 2^14 or 2^30 times the rest and meet codes of 0."""
    rng = np.random.default_rng(D + S + 1)
    down, large = _opposite(D, F, fmt, rng, 0.3), np.array([3, F - 2])
    down[:, large] = down[:, (large + F // 2) % F] = 0
    for log in (10, 14, 30):
        scale = np.ones(F)
        scale[large] = 2.0 ** (log // 2)
        layer = Given(q, fmt, [(_one_of(F, D, lambda o: 1 + o % (F // 2)), scale), (_one_of(F, D, lambda o: 0 * o), scale), (down, np.ones(D))])
        for kind in TYPES:
            x = np.abs(synth.normal_f32((S, D), D, 1)) + 0.25
            x[:, 0] = 1
            x, y = _given(q, layer, x, kind)
            h = x[:, 1 + np.arange(F) % (F // 2)]
            tol = 1e-5 * (np.abs(h) @ np.abs(down).T.astype(np.float64))
            worst = (np.abs(y) / tol).max()
            assert worst <= 1.01, "%s, largest 2^%d times the rest: %g of the tolerance" % (kind, log, worst)
        layer.free()


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("S,D,F", PRODUCTS)
def test_experts_matrix_of_zeros(q, S, D, F, fmt):
    """A matrix of zeros with scales that are not: y is 0."""
    rng = np.random.default_rng(5)
    some = lambda O, I: _opposite(O, I, fmt, rng)  # noqa: E731
    zero = lambda O, I: np.zeros((O, I), np.int64)  # noqa: E731
    for m in range(3):
        mats = [(zero if m == j else some)(*s) for j, s in enumerate([(F, D), (F, D), (D, F)])]
        layer = Given(q, fmt, [(v, np.full(v.shape[0], 0.37)) for v in mats])
        for kind in TYPES:
            x, y = _given(q, layer, synth.normal_f32((S, D), D, 1) + 0.5, kind)
            assert (y == 0).all(), "%s: %g" % (kind, np.abs(y).max())
        layer.free()


# ---------------------------------------------------------------- decisions and sums where f32 alone is not enough
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("size", [0.5, 32.0, 100.0, 1000.0])
@pytest.mark.parametrize("n,per,keep", [(2, 2, 1), (8, 8, 3), (4, 33, 2), (32, 32, 5), (16, 3, 4)])
def test_route_groups_whose_biases_cancel(q, n, per, keep, size, score):
    """Every group has one large positive bias and for the rest the same negative one: its value is a small sum of two large c, and neighbouring
    groups' values are nearer than the roundings of those."""
    E, S = n * per, 24
    bias = np.full(E, -size, np.float32)
    bias[np.arange(n) * per + (np.arange(n) * 7) % per] = size
    l = synth.normal_f32((S, E), E, 1)
    l[1::3] = 0.01 * l[1::3]
    l[2::3] = np.float32(1e-4) * l[2::3] + 0.5
    for norm in (False, True):
        _route(q, _dev(l), min(2, per), score, bias, n, keep, 2, norm)


def test_route_two_groups_that_f32_takes_for_the_wrong_order(q):
    l = np.array([[-0.81081446, 0.75224382, 0.25344652, -0.30490190]], np.float32)
    got = _route(q, _dev(l), 2, 1, np.array([32, -32, 32, -32], np.float32), 2, 1, 2)
    assert got[0].tolist() == [[0, 1]]


@pytest.mark.parametrize("big", [3.0e38, 2.0e38])
def test_route_group_values_past_f32(q, big):
    """Sums of two biases that f32 does not hold, of either sign."""
    l = synth.normal_f32((6, 16), 1, 1)
    for signs in ((1, 1, -1, -1), (-1, -1, -1, -1), (1, 1, 1, 1), (-1, 1, -1, 1)):
        bias = np.repeat(np.array(signs, np.float32) * np.float32(big), 4) * (1 - np.float32(1e-6) * (np.arange(16, dtype=np.float32) % 5))
        for keep in (1, 2, 3):
            _route(q, _dev(l), 4, 1, bias.astype(np.float32), 4, keep, 2)


RANGES = [(1, 6144), (5, 8), (400, 64), (310, 96), (311, 1003), (400, 6144), (2, 16385), (1, 40000)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("S,D", RANGES)
def test_norm_rows_of_any_finite_size(q, S, D, kind):
    """Squares that f32 does not hold, too large and (eps = 0, or as small) too small; rows of ordinary size among them; zeros stay zeros."""
    a, b = (synth.normal_f32((S, D), D, j) for j in (1, 2))
    wp, w = (_dev(0.5 + np.abs(synth.normal_f32((D,), D, j))) for j in (3, 4))
    for log, eps in ((62, 1e-6), (62, 0.0), (120, 1e-6), (-63, 1e-38), (-80, 0.0), (-80, 1e-35), (-80, 1e-6), (-100, 0.0)):
        size = np.exp2(np.where(np.arange(S) % 3 == 1, 0, log)).astype(np.float32)[:, None]
        m, h = _dev(a * size, kind), _dev(b * size, kind)
        _norm(q, m, h, None, wp, w, 1.0, 0.5, kind, "f32", eps=eps)              # p of ordinary size beside h
        _norm(q, m, h, None, None, w, 1.0, 0.5, kind, kind, eps=eps)
        _norm(q, m, None, None, wp, w, kind=kind, ykind="f32", eps=eps)
        _norm(q, m, None, _dev(synth.normal_f32((S, 1), D, 5), kind), None, w, kind=kind, ykind="f32", eps=eps, out=False)


def test_norm_one_large_value_and_subnormal_rows(q):
    S, D = 3, 1024
    m = 0.1 * synth.normal_f32((S, D), 1, 1)
    m[0, 77] = 3.0e38
    m[1] *= np.float32(2.0 ** -140)
    m[2, 0] = -2.0 ** 70
    w = _dev(np.ones(D))
    for eps in (0.0, 1e-6):
        _norm(q, _dev(m), None, None, w, w, eps=eps)
        _norm(q, _dev(m), None, None, None, w, eps=eps)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("D", [4069, 4073, 4081, 4087, 4093, 4095])
def test_norm_odd_rows_whose_weights_fill_48_kb(q, D, kind):
    """Rows of an odd stride keep their weights in shared memory: about what a kernel may have without asking for more."""
    m, h = (_dev(synth.normal_f32((3, D), D, j), kind) for j in (1, 2))
    wp, w = (_dev(0.5 + np.abs(synth.normal_f32((D,), D, j))) for j in (3, 4))
    _norm(q, m, h, _dev(synth.normal_f32((1, D), D, 5), kind), wp, w, 0.7, 0.25, kind, kind)


def test_norm_gates_that_are_refused(q):
    import torch
    m, o, one = _dev(np.ones((3, 8))), _dev(np.ones((3, 8))), torch.ones
    for gate, what in ((2.0, TypeError), (np.ones(8, np.float32), TypeError), (one((), device="cuda"), ValueError), (one(3, 8, 1, device="cuda"), ValueError),
                       (one(7, device="cuda"), ValueError), (one(2, 8, device="cuda"), ValueError), (one(2, 1, device="cuda"), ValueError),
                       (one(3, 8), ValueError), (one(3, 8, device="cuda").half(), ValueError), (one(8, 3, device="cuda").t(), ValueError)):
        with pytest.raises(what):
            q.block_norm(m, 3, 8, 1e-6, h_out=o, gate=gate)


@pytest.mark.parametrize("n,keep", [(1, 1), (32, 5), (8, 8)])
def test_route_many_tokens_of_many_experts(q, n, keep):
    """1024 experts for more tokens than one to a block: the most shared memory that routing takes."""
    l = _dev(synth.normal_f32((400, 1024), n, 1))
    bias = (0.1 * synth.normal_f32((1024,), n, 2)).astype(np.float32)
    _route(q, l, 8, 1, bias, n, keep, 2)
    _route(q, l, 8, 0, bias, n, keep, 1)


FIRST = """
import sys
sys.path.insert(0, %r)
import numpy as np, torch
import quantized_weight_quant_gb300 as q
S, E, D, F, k = %d, 4, 320, 192, 2
g, u, d = ([q.tensor_upload(q.I4, O, I, np.full((O, I // 2), 0x99, np.uint8), np.full(O, 1 / 64, np.float32)) for _ in range(E)]
           for O, I in ((F, D), (F, D), (D, F)))
ex = q.Experts(g, u, d)
x, h, y = torch.ones(S, D, device="cuda"), torch.empty(S, D, device="cuda"), torch.empty(S, D, device="cuda")
l, ids, wts = torch.zeros(S, E, device="cuda"), torch.zeros(S, k, dtype=torch.int32, device="cuda"), torch.zeros(S, k, device="cuda")
w = torch.ones(D, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    q.moe_route(l, ids, wts, S, E, k)
    q.moe_experts(ex, x, ids, wts, h, S, k, act=q.ACT_NONE)
    q.block_norm(h, S, D, 0.0, w=w, y=y)
graph.replay()
torch.cuda.synchronize()
assert (h == 25.0 * F / 64).all() and (y - 1).abs().max() < 1e-5, (h, y)
"""


@pytest.mark.parametrize("S", [1, 5, 64])
def test_first_calls_of_a_process_may_be_captured(S):
    """1 * 320 / 64 = 5 for gate and for up, h = 25, y = 25 * 192 / 64 with weights that add up to 1."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % (root, S)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("S,D,F", PRODUCTS)
def test_experts_small_values_beside_a_large_one(q, S, D, F, fmt):
    """Products that do not cancel, of rows whose largest value, 2^30 times the rest, meets a code of 0: what f32 rows have beside it is held
    to 2^-50 of it, what bf16 rows have to 2^-40."""
    rng = np.random.default_rng(D + S + 2)
    top = {"i8": 127, "i4": 7, "i2": 1}[fmt]
    gate, large = rng.integers(-top, top + 1, (F, D)), D // 3
    gate[:, 0] = gate[:, large] = 0
    layer = Given(q, fmt, [(gate, np.ones(F)), (_one_of(F, D, lambda o: 0 * o), np.ones(F)), (_one_of(D, F, lambda o: o % F), np.ones(D))])
    for kind, part in (("f32", 2.0 ** -50), ("bf16", 2.0 ** -40)):
        x = synth.normal_f32((S, D), D, 1)
        x[:, 0], x[:, large] = 1, 2.0 ** 30
        x, y = _given(q, layer, x, kind)
        g = (x @ gate.T.astype(np.float64))
        x[:, large] = 0
        tol = 1e-5 * (np.abs(x) @ np.abs(gate).T.astype(np.float64)) + part * 2.0 ** 30 * np.abs(gate).sum(1)
        tol = tol + (2.0 ** -11 if kind == "bf16" else 2.0 ** -22) * (np.abs(g) + tol)          # h
        g, tol = (v[:, np.arange(D) % F] for v in (g, tol))
        assert (np.abs(y - g) <= tol + _half_step(kind) * (np.abs(g) + tol)).all(), "%s: %g" % (kind, (np.abs(y - g) / tol).max())
    layer.free()
