"""The 8-bit activation calls against plain 64-bit references.

Tolerances, from the formats (half a step of a type t: finfo(t).eps / 2):
  quantize_q8   one f32 division by a f32 scale on both sides: bytes and scales are equal
  rmsnorm_q8    f32 arithmetic within 1e-5 of y (the bar of b200q_rmsnorm), then an E4M3
                rounding: half a step of its grid at y / scale
  matmul / glu  1e-5 * B before the activation, B = scale * xs * sum |deq * x8| (+ |bias|); the
                activations' slopes are at most 1.13 in magnitude and their f32 evaluation is within 4e-6 |v|
                (a dozen roundings and the error bounds of expf, tanhf and erff); then one rounding to
                the output type
"""
import numpy as np
import pytest

import synth

pytestmark = pytest.mark.gpu

FMTS = {"i8": 1, "i4": 2, "i2": 3}
BITS = {"i8": 8, "i4": 4, "i2": 2}
ACT_SLOPE = 1.13


@pytest.fixture(scope="module")
def q():
    import torch
    torch.cuda.set_device(0)
    import quantized_weight_quant_gb300 as q
    return q


def _torch_type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _half_step(name):
    return {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[name]


def _tiny(name):
    """Half the smallest step of the type (its subnormal grid)."""
    return {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[name]


# ---------------------------------------------------------------- E4M3 in numpy
def _e4m3_table():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if c & 127 == 127:
            a = np.nan
        v[c] = -a if c & 128 else a
    return v


E4M3 = _e4m3_table()


def _e4m3_round(v):
    """Nearest E4M3 value, ties to even, |v| up to 464."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(np.abs(v))
    step = 2.0 ** (np.maximum(e - 1, -6) - 3.0)
    return np.clip(np.rint(v / step) * step, -448, 448)


def _rows(S, D, seed, spread=True):
    x = synth.normal_f32((S, D), seed, 1)
    if spread:
        x *= np.exp2(np.arange(S) % 7 - 3).astype(np.float32)[:, None]
    return x


def _dev(a, name="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(_torch_type(name))


def _np64(t):
    return t.double().cpu().numpy()


def _fresh(q, S, D):
    out = q.Q8Rows(S, D)
    out.codes.fill_(0x5A)
    out.scales.fill_(float("nan"))
    return out


def _quantised(q, out, D):
    c = out.codes.cpu().numpy()
    assert (c[:, D:] == 0x5A).all(), "bytes past D were written"
    return E4M3[c[:, :D]], out.scales.double().cpu().numpy()


# ---------------------------------------------------------------- rows
SIZES = [(1, 1), (2, 7), (3, 8), (5, 15), (1, 16), (4, 33), (3, 255), (2, 1024), (7, 2049), (1, 6144), (3, 5003),
         (2, 12288), (2, 16384), (1, 16385), (2, 40000), (300, 64), (65, 96)]


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S,D", SIZES)
def test_quantize(q, S, D, kind):
    import torch
    x = _dev(_rows(S, D, D + S), kind)
    out = _fresh(q, S, D)
    q.quantize_q8(x, out, S, D)
    torch.cuda.synchronize()
    v, s = _quantised(q, out, D)
    xf = x.float().cpu().numpy()
    s_ref = np.maximum(np.abs(xf).max(1) / np.float32(448), np.float32(2.0 ** -126))
    assert np.array_equal(s.astype(np.float32), s_ref)
    assert np.array_equal(v, _e4m3_round(xf / s_ref[:, None]))


def _norm_ref(x, r, w, eps):
    h = x + r if r is not None else x
    return h, h * w / np.sqrt((h * h).mean(1, keepdims=True) + eps)


def _check_rows(v, s, y):
    assert np.all(np.abs(s - np.maximum(np.abs(y).max(1) / 448, 2.0 ** -126)) <= 1e-5 * s)
    # the nearest E4M3 value of y / s: within half the grid's step there, and the f32 error of y and s
    # (which decides between two values only where y / s is a tie to within that error)
    t = np.clip(y / s[:, None], -448, 448)
    _, e = np.frexp(np.abs(t))
    half = 2.0 ** (np.maximum(e - 1, -6) - 4.0)
    assert np.all(np.abs(v - t) <= half + 2e-5 * np.abs(t))


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("res", [False, True], ids=["x", "x+r"])
@pytest.mark.parametrize("S,D", SIZES)
def test_rmsnorm(q, S, D, kind, res):
    import torch
    x, w = _dev(_rows(S, D, D), kind), _dev(synth.uniform_f32((D,), -1.5, 1.5, D, 3))
    r = _dev(synth.normal_f32((S, D), D, 2), kind) if res else None
    out, h = _fresh(q, S, D), torch.full_like(x, float("nan"))
    q.rmsnorm_q8(x, w, out, S, D, 1e-6, r=r, h=h)
    torch.cuda.synchronize()
    h_ref, y = _norm_ref(_np64(x), _np64(r) if res else None, _np64(w), 1e-6)
    h_f32 = x.float() + r.float() if res else x.float()
    assert torch.equal(h, h_f32.to(h.dtype))
    _check_rows(*_quantised(q, out, D), y)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("alias", ["x", "r"])
@pytest.mark.parametrize("D", [6144, 5003, 20000])
def test_rmsnorm_in_place(q, D, alias, kind):
    import torch
    S = 3
    x, r, w = _dev(_rows(S, D, 1), kind), _dev(synth.normal_f32((S, D), 1, 2), kind), _dev(np.ones(D))
    _, y = _norm_ref(_np64(x), _np64(r), _np64(w), 1e-5)
    want = (x.float() + r.float()).to(x.dtype)
    out = _fresh(q, S, D)
    h = x if alias == "x" else r
    q.rmsnorm_q8(x, w, out, S, D, 1e-5, r=r, h=h)
    torch.cuda.synchronize()
    assert torch.equal(h, want)
    _check_rows(*_quantised(q, out, D), y)


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_rows_strided_and_shifted(q, kind, shift):
    """Columns of wider buffers: row strides of their own, starts off a vector's boundary, h next to x in one buffer."""
    import torch
    S, D, wide = 5, 1000, 2311
    buf = _dev(_rows(S, wide, 4), kind)
    x, h = buf[:, shift:shift + D], buf[:, 1200 + shift:1200 + shift + D]
    r = _dev(_rows(S, 1500, 5), kind)[:, 7:7 + D]
    w = _dev(synth.uniform_f32((D + 3,), 0.5, 1.5, 6, 1))[shift:shift + D]
    store = torch.full((S, 1200), 0x5A, dtype=torch.uint8, device="cuda")
    out = q.Q8Rows(S, D)
    out.codes = store[:, 16:16 + 1008]
    keep = buf.clone()
    _, y = _norm_ref(_np64(x), _np64(r), _np64(w), 1e-6)
    want = (x.float() + r.float()).to(x.dtype)
    q.rmsnorm_q8(x, w, out, S, D, 1e-6, r=r, h=h)
    torch.cuda.synchronize()
    assert torch.equal(h, want)
    keep[:, 1200 + shift:1200 + shift + D] = want
    assert torch.equal(buf, keep)
    _check_rows(E4M3[store[:, 16:16 + D].cpu().numpy()], out.scales.double().cpu().numpy(), y)
    assert (store[:, :16] == 0x5A).all() and (store[:, 16 + D:] == 0x5A).all()


def test_rows_zero_tiny_and_not_finite(q):
    """A zero row has the least scale and zero codes; tiny rows use the least scale; a row with a NaN or an
    infinity gets a scale or codes that are not finite, and only that row."""
    import torch
    D = 500
    x = np.ones((6, D), np.float32)
    x[0] = 0
    x[1] *= 1e-40
    x[2, 499] = np.nan
    x[3, 3] = -np.inf
    x[4] *= 3e38
    xd, out = _dev(x), _fresh(q, 6, D)
    q.quantize_q8(xd, out, 6, D)
    torch.cuda.synchronize()
    v, s = _quantised(q, out, D)
    assert s[0] == 2.0 ** -126 and (v[0] == 0).all()
    assert s[1] == 2.0 ** -126 and (v[1] == 2.0 ** -7).all()   # 1e-40 / 2^-126 = 0.0085, in steps of 2^-9: 4
    assert not np.isfinite(v[2] * s[2]).all() and not np.isfinite(s[2])
    assert not np.isfinite(s[3]) and np.isnan(v[3, 3])
    assert (v[4] == 448).all() and (v[5] == 448).all()
    w = _dev(np.ones(D))
    out = _fresh(q, 6, D)
    q.rmsnorm_q8(xd, w, out, 6, D, 1e-6)
    torch.cuda.synchronize()
    v, s = _quantised(q, out, D)
    assert s[0] == 2.0 ** -126 and (v[0] == 0).all() and (v[5] == 448).all()
    assert not np.isfinite(s[2]) and not np.isfinite(s[3])


# ---------------------------------------------------------------- products
def _codes(fmt, O, I, seed):
    return synth.codes(FMTS[fmt], O, I, seed, 7, int8_lo=-128)


def _decoded(codes, fmt, I):
    c = codes.astype(np.int64)
    if fmt == "i8":
        return codes.view(np.int8).astype(np.float64)
    n = 8 // BITS[fmt]
    f = [(c >> (BITS[fmt] * k)) & (2 ** BITS[fmt] - 1) for k in range(n)]
    return np.stack(f, 2).reshape(c.shape[0], -1)[:, :I] - 2.0 ** (BITS[fmt] - 1)


def _input8(q, S, I, seed):
    """Random E4M3 bytes (every code but the NaNs), scales of different sizes; the bytes past I are NaN codes."""
    import torch
    rng = synth.rng(seed, 9)
    c = rng.integers(0, 256, (S, I), dtype=np.uint8)
    c[c & 127 == 127] = 0x7E
    keep = rng.random((S, I)) < 0.5
    c = np.where(keep, c & 0xBF, c).astype(np.uint8)          # half of them below 2 in magnitude
    xs = np.exp2(rng.uniform(-12, -6, S)).astype(np.float32)
    xq = q.Q8Rows(S, I)
    xq.codes.fill_(0x7F)
    xq.codes[:, :I] = torch.from_numpy(c).cuda()
    xq.scales.copy_(torch.from_numpy(xs))
    return xq, E4M3[c], xs.astype(np.float64)


def _act(name, v):
    from scipy.special import erf
    if name == "relu":
        return np.maximum(v, 0)
    if name == "gelu":
        return 0.5 * v * (1 + erf(v / np.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v * 0.5 * (1 + np.tanh(v / 2))
    return v


class _Pair:
    """One weight set on the device and its exact product with 8-bit rows."""

    def __init__(self, q, fmt, O, I, seed, bias):
        codes = _codes(fmt, O, I, seed)
        self.scale = synth.uniform_f32((O,), 1e-3, 2e-2, seed, 8)
        self.t = q.tensor_upload(FMTS[fmt], O, I, codes, self.scale)
        self.w = _decoded(codes, fmt, I)
        self.bias = synth.normal_f32((O,), seed, 11) if bias else None
        self.bias_d = _dev(self.bias) if bias else None

    def exact(self, x, xs):
        sc = self.scale.astype(np.float64)[None, :] * xs[:, None]
        v, b = (x @ self.w.T) * sc, (np.abs(x) @ np.abs(self.w).T) * sc
        if self.bias is not None:
            v, b = v + self.bias, b + np.abs(self.bias)
        return v, 1e-5 * b


def _check(y, want, tol, kind, what):
    got = _np64(y)
    assert np.all(np.isfinite(got)), what
    tol = tol + _half_step(kind) * (np.abs(want) + tol) + _tiny(kind)
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance at %s" % (
        what, bad.sum(), bad.size, np.max(np.abs(got - want) / np.maximum(tol, 1e-300)), np.argwhere(bad)[:4].tolist())


def _mm(q, fmt, O, I, S, kind, act="none", bias=False, res=False, seed=0, ldy=None):
    import torch
    p = _Pair(q, fmt, O, I, seed + O + I, bias)
    xq, x, xs = _input8(q, S, I, seed + S)
    wide = torch.full((S, ldy or O), 7.0, dtype=_torch_type(kind), device="cuda")
    y = wide[:, :O]
    r = _dev(synth.normal_f32((S, O), seed, 12), kind) if res else None
    with p.t:
        q.matmul_q8(p.t, xq, y, S, bias=p.bias_d, act=q.ACTS[act], res=r)
        torch.cuda.synchronize()
    v, e = p.exact(x, xs)
    want = _act(act, v) + (_np64(r) if res else 0)
    tol = ACT_SLOPE * e + 4e-6 * np.abs(v) + 2.0 ** -23 * np.abs(want)
    _check(y, want, tol, kind, "mm %s %dx%d S=%d" % (fmt, O, I, S))
    assert (wide[:, O:] == 7.0).all()
    assert q.device_status() == q.OK
    return y


def _glu(q, fmt, O, I, S, kind, act="silu", bg=False, bu=False, seed=0, ldy=None):
    import torch
    g, u = _Pair(q, fmt, O, I, seed + O + I, bg), _Pair(q, fmt, O, I, seed + O + I + 1, bu)
    xq, x, xs = _input8(q, S, I, seed + S)
    wide = torch.full((S, ldy or O), 7.0, dtype=_torch_type(kind), device="cuda")
    y = wide[:, :O]
    with g.t, u.t:
        q.glu_q8(g.t, u.t, xq, y, S, act=q.ACTS[act], bias_g=g.bias_d, bias_u=u.bias_d)
        torch.cuda.synchronize()
    (vg, eg), (vu, eu) = g.exact(x, xs), u.exact(x, xs)
    a = _act(act, vg)
    ea = ACT_SLOPE * eg + 4e-6 * np.abs(vg)
    _check(y, a * vu, ea * np.abs(vu) + np.abs(a) * eu + ea * eu, kind, "glu %s %dx%d S=%d" % (fmt, O, I, S))
    assert (wide[:, O:] == 7.0).all()
    assert q.device_status() == q.OK
    return y


SHAPES = [(1, 1, 1), (1, 40, 3), (7, 3, 2), (16, 64, 1), (33, 31, 5), (64, 129, 8), (65, 512, 9), (127, 1000, 16),
          (128, 256, 17), (129, 257, 33), (200, 2049, 64), (384, 640, 100), (1000, 300, 129), (130, 1153, 200),
          (513, 128, 300)]


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("O,I,S", SHAPES)
def test_matmul(q, fmt, O, I, S):
    _mm(q, fmt, O, I, S, "f32")


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("O,I,S", SHAPES)
def test_glu(q, fmt, O, I, S):
    _glu(q, fmt, O, I, S, "f32")


@pytest.mark.parametrize("S", list(range(1, 40)) + [47, 48, 49, 63, 64, 65, 95, 96, 97, 127, 128, 130, 159, 161, 255, 257])
def test_every_row_count(q, S):
    _mm(q, "i4", 272, 416, S, "f32", bias=True, seed=3)
    _glu(q, "i8", 144, 352, S, "f32", bg=True, seed=4)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("S", [1, 6, 20, 70])
def test_epilogue(q, kind, act, S):
    _mm(q, "i4", 150, 384, S, kind, act, bias=S != 6, res=S != 20, seed=1, ldy=163)
    _glu(q, "i2", 150, 384, S, kind, act, bg=S != 6, bu=S != 20, seed=2, ldy=175)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("S", [1, 4, 12, 40, 180])
def test_long_rows(q, fmt, S):
    """Long sums: many k-blocks, K split over blocks; sizes off every tile."""
    _mm(q, fmt, 257, 12000 + 77, S, "f32", seed=5)
    _glu(q, fmt, 130, 9001, S, "f32", seed=6)


@pytest.mark.parametrize("S", [1, 8, 30, 150])
def test_many_tiles(q, S):
    """More output tiles than multiprocessors."""
    _mm(q, "i4", 21000, 260, S, "bf16", bias=True, res=True, seed=7)
    _glu(q, "i8", 10100, 130, S, "f16", seed=8)


@pytest.mark.parametrize("S", [1, 40])
def test_residual_in_place(q, S):
    import torch
    O, I = 300, 500
    p = _Pair(q, "i8", O, I, 1, True)
    xq, x, xs = _input8(q, S, I, 2)
    y = _dev(synth.normal_f32((S, O), 1, 12), "bf16")
    before = _np64(y)
    with p.t:
        q.matmul_q8(p.t, xq, y, S, bias=p.bias_d, res=y)
        torch.cuda.synchronize()
    v, e = p.exact(x, xs)
    _check(y, v + before, e + 2.0 ** -23 * np.abs(v + before), "bf16", "in place")


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("S", [1, 24])
def test_every_code_exact(q, fmt, S):
    """One-hot rows read single weights back: every code, in every position of a byte, bit for bit."""
    import torch
    I, O = 64, 256
    codes = np.zeros((O, I * BITS[fmt] // 8), np.uint8)
    codes[:] = (np.arange(O)[:, None] * 5 + np.arange(codes.shape[1])[None, :] * 3) % 256
    w = _decoded(codes, fmt, I)
    with q.tensor_upload(FMTS[fmt], O, I, codes, np.ones(O, np.float32)) as t:
        for i0 in range(0, I, S):
            n = min(S, I - i0)
            xq = q.Q8Rows(n, I)
            xq.codes.zero_()
            for k in range(n):
                xq.codes[k, i0 + k] = 0x38                    # 1.0
            xq.scales.fill_(1.0)
            y = torch.empty(n, O, device="cuda")
            q.matmul_q8(t, xq, y, n)
            torch.cuda.synchronize()
            assert np.array_equal(_np64(y), w[:, i0:i0 + n].T)


@pytest.mark.parametrize("S", [3, 20, 140])
def test_bad_row_stays_alone(q, S):
    """A row whose scale or codes are not finite spoils its own outputs only."""
    import torch
    O, I = 140, 300
    p = _Pair(q, "i4", O, I, 3, False)
    xq, x, xs = _input8(q, S, I, 4)
    xq.codes[1, 17] = 0x7F
    xq.scales[S - 1] = float("nan")
    y = torch.zeros(S, O, device="cuda")
    with p.t:
        q.matmul_q8(p.t, xq, y, S)
        torch.cuda.synchronize()
    got = _np64(y)
    assert np.isnan(got[1]).all() and np.isnan(got[S - 1]).all()
    v, e = p.exact(x, xs)
    ok = [s for s in range(S) if s not in (1, S - 1)]
    assert np.all(np.abs(got[ok] - v[ok]) <= e[ok] + 2.0 ** -24 * np.abs(v[ok]))


@pytest.mark.parametrize("S", [1, 5, 16, 33, 200])
def test_same_bits_each_time(q, S):
    import torch
    p = _Pair(q, "i4", 700, 4500, 5, False)
    xq, _, _ = _input8(q, S, 4500, 6)
    ys = [torch.empty(S, 700, device="cuda") for _ in range(4)]
    with p.t:
        for y in ys:
            q.matmul_q8(p.t, xq, y, S)
        torch.cuda.synchronize()
    assert all(torch.equal(ys[0], y) for y in ys[1:])


@pytest.mark.parametrize("S", [1, 7, 18, 130])
def test_streams_and_graphs(q, S):
    """The chain norm -> pair -> rows -> product on a stream of its own, captured and replayed on new inputs."""
    import torch
    D, F = 320, 200
    g, u, d = (_Pair(q, "i4", *sh, 9 + k, False) for k, sh in enumerate([(F, D), (F, D), (D, F)]))
    x, w = _dev(_rows(S, D, 1), "bf16"), _dev(np.ones(D))
    a, b = q.Q8Rows(S, D), q.Q8Rows(S, F)
    mid, y = torch.empty(S, F, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)

    def chain(stream):
        q.rmsnorm_q8(x, w, a, S, D, 1e-6, stream=stream)
        q.glu_q8(g.t, u.t, a, mid, S, stream=stream)
        q.quantize_q8(mid, b, S, F, stream=stream)
        q.matmul_q8(d.t, b, y, S, res=x, stream=stream)

    with g.t, u.t, d.t:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        chain(st)
        st.synchronize()
        first = y.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            chain(st)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, y)
        x.copy_(_dev(_rows(S, D, 2), "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        second = y.clone()
        chain(None)
        torch.cuda.synchronize()
        assert torch.equal(second, y) and not torch.equal(first, y)
    assert q.device_status() == q.OK


def test_two_streams_at_once(q):
    """Calls that share tensors on two streams without ordering do not disturb each other."""
    import torch
    p = _Pair(q, "i4", 512, 6000, 2, False)
    for S in (2, 40, 150):
        xa, _, _ = _input8(q, S, 6000, 1)
        xb, _, _ = _input8(q, S, 6000, 2)
        want = []
        for xq in (xa, xb):
            y = torch.empty(S, 512, device="cuda")
            q.matmul_q8(p.t, xq, y, S)
            torch.cuda.synchronize()
            want.append(y)
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        ya, yb = ([torch.empty(S, 512, device="cuda") for _ in range(8)] for _ in range(2))
        torch.cuda.synchronize()
        for k in range(8):
            q.matmul_q8(p.t, xa, ya[k], S, stream=s1)
            q.matmul_q8(p.t, xb, yb[k], S, stream=s2)
        torch.cuda.synchronize()
        assert all(torch.equal(v, want[0]) for v in ya) and all(torch.equal(v, want[1]) for v in yb)
    p.t.free()


def test_refusals(q):
    import torch
    O, I, S = 64, 96, 4
    p, p2 = _Pair(q, "i4", O, I, 1, False), _Pair(q, "i4", O, 128, 1, False)
    f32 = q.tensor_upload(q.F32, O, I, np.zeros((O, I), np.float32), None)
    gs = q.tensor_upload(q.I4, O, I, _codes("i4", O, I, 1), np.ones((O, 3), np.float32), gs=32)
    xq, _, _ = _input8(q, S, I, 1)
    y = torch.empty(S, O, device="cuda")
    L, c, sc, yp = q.lib, xq.codes.data_ptr(), xq.scales.data_ptr(), y.data_ptr()

    def mm(t=None, c=c, ld8=96, sc=sc, bias=None, act=0, res=None, ldr=O, y=yp, kind=0, ldy=O, S=S):
        return L.b200q_matmul_q8((t or p.t).handle, c, ld8, sc, bias, act, res, ldr, y, kind, ldy, S, None)

    assert mm(t=f32) == q.EINVAL and "int8, int4 and int2" in q.last_error()
    assert mm(t=gs) == q.EINVAL and "per-row" in q.last_error()
    for bad in (dict(c=None), dict(sc=None), dict(y=None), dict(c=c + 8), dict(ld8=100), dict(ld8=80), dict(sc=sc + 2),
                dict(y=yp + 2), dict(ldy=O - 1), dict(act=5), dict(act=-1), dict(kind=3), dict(S=-1), dict(bias=sc + 1),
                dict(res=yp + 4), dict(res=yp, ldr=O - 1), dict(y=c), dict(bias=yp), dict(sc=yp), dict(ldy=1 << 61),
                dict(res=yp, ldr=O + 4)):
        assert mm(**bad) == q.EINVAL, bad
    assert mm(S=0, c=None, y=None) == q.OK
    assert L.b200q_glu_q8(p.t.handle, None, c, 96, sc, None, None, 4, yp, 0, O, S, None) == q.EINVAL
    assert L.b200q_glu_q8(p.t.handle, p2.t.handle, c, 96, sc, None, None, 4, yp, 0, O, S, None) == q.EINVAL
    assert "differ" in q.last_error()
    with pytest.raises(ValueError):
        q.matmul_q8(p2.t, xq, y, S)                                     # 96 columns for 128
    with pytest.raises(ValueError):
        q.matmul_q8(p.t, xq, y, S + 1)                                  # more rows than there are
    with pytest.raises(ValueError):
        q.matmul_q8(p.t, xq, y.t(), S)
    with pytest.raises(ValueError):
        q.matmul_q8(p.t, xq, y, S, res=y.half())
    with pytest.raises(ValueError):
        q.matmul_q8(p.t, xq, y, S, bias=torch.zeros(O - 1, device="cuda"))
    with pytest.raises(ValueError):
        q.matmul_q8(p.t, xq, y.int(), S)
    with pytest.raises(ValueError):
        q.quantize_q8(y.cpu(), xq, S, O)
    for t in (f32, gs, p.t, p2.t):
        t.free()
    assert q.device_status() == q.OK


def test_example_block(q):
    """The example's block.  Each of its two quantisations rounds by at most 2^-4 of a value, 2^-5 / sqrt(3) in the
    root mean square of a uniform error over a binade's steps (about 0.025); the three products see the first one
    in gate and up and the second in down: below 0.025 * (1.5 + 1 + 1) with independent roundings, and the bf16
    roundings (h, m, y) are far smaller (y - h: 2^-8 of |h| ~ 1.4 against values near 0.5)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "dense_block_q8.py")
    spec = importlib.util.spec_from_file_location("dense_block_q8", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for e in mod.run(512, 1024, [1, 7, 40], time_it=False):
        assert 1e-3 < e < 0.0875


def test_long_batch_in_parts(q):
    """More rows than one launch of the tensor-core kernel numbers: the last part's rows and the first's."""
    import torch
    O, I, S = 40, 64, (1 << 16) + 9
    p = _Pair(q, "i4", O, I, 2, True)
    xq, x, xs = _input8(q, S, I, 3)
    y, r = torch.zeros(S, O, device="cuda"), _dev(synth.normal_f32((S, O), 5, 6))
    with p.t:
        q.matmul_q8(p.t, xq, y, S, bias=p.bias_d, res=r)
        torch.cuda.synchronize()
    v, e = p.exact(x, xs)
    want = v + _np64(r)
    _check(y, want, e + 2.0 ** -23 * np.abs(want), "f32", "long batch")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S,D", SIZES)
def test_rmsnorm_alone(q, S, D, kind):
    """Neither residual nor h; w off a vector's boundary for odd D."""
    import torch
    x = _dev(_rows(S, D, D + 1), kind)
    w = _dev(synth.uniform_f32((D + 1,), -1.5, 1.5, D, 4))[D % 2:][:D]
    out = _fresh(q, S, D)
    q.rmsnorm_q8(x, w, out, S, D, 1e-6)
    torch.cuda.synchronize()
    _check_rows(*_quantised(q, out, D), _norm_ref(_np64(x), None, _np64(w), 1e-6)[1])


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [1, 2, 9, 31, 257, 263, 511, 1025, 2049, 4099])
@pytest.mark.parametrize("S", [2, 700])
def test_rmsnorm_odd_rows_in_place(q, S, D, kind):
    """Rows of D values one after the other, from an odd value on: h over x, every value its own, nothing beside it."""
    import torch
    buf = _dev(_rows(1, S * D + 40, D)[0], kind)
    keep = buf.clone()
    x, r = buf[3:3 + S * D].view(S, D), _dev(_rows(S, D, D + 2), kind)
    want = (x.float() + r.float()).to(x.dtype)
    w = _dev(synth.uniform_f32((D,), 0.5, 1.5, D, 5))
    _, y = _norm_ref(_np64(x), _np64(r), _np64(w), 1e-6)
    out = _fresh(q, S, D)
    q.rmsnorm_q8(x, w, out, S, D, 1e-6, r=r, h=x)
    torch.cuda.synchronize()
    keep[3:3 + S * D] = want.view(-1)
    assert torch.equal(buf, keep)
    _check_rows(*_quantised(q, out, D), y)


def test_longest_row_to_8_bits(q):
    """2^31 - 1 columns: column numbers pass 31 bits in the last step of the walk."""
    import torch
    D = 2 ** 31 - 1
    x = torch.zeros(1, D, dtype=torch.float16, device="cuda")
    for d, v in ((0, -224.0), (2 ** 30 + 5, 3.0), (D - 1, 448.0)):
        x[0, d] = v
    out = q.Q8Rows(1, D)
    out.codes.fill_(0x5A)
    q.quantize_q8(x, out, 1, D)
    torch.cuda.synchronize()
    assert float(out.scales[0]) == 1.0
    got = [int(out.codes[0, d]) for d in (0, 2 ** 30 + 5, D - 1, D)]
    assert got == [0xF6, 0x44, 0x7E, 0x5A]                  # -224, 3, 448, not written
    assert sum(int(torch.count_nonzero(c)) for c in out.codes[0].split(2 ** 28)) == 4


def _long_call(q):
    """Rows so long that every block of the tensor-core kernel walks for more than 0.1 ms, in one tile that all share."""
    import torch
    O, I, S = 40, 10_000_000, 9
    codes = synth.rng(1, 2).integers(0, 256, (O, I // 4), dtype=np.uint8)
    t = q.tensor_upload(q.I2, O, I, codes, np.ones(O, np.float32))
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    xq = q.Q8Rows(S, I)
    xq.codes.copy_(torch.randint(0, 0x50, xq.codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    xq.scales.fill_(0.5)
    return t, xq, O, S


def test_giving_up_is_reported(q):
    """A wait that runs out ends the kernel with a status; the next call is whole again."""
    import torch
    t, xq, O, S = _long_call(q)
    want, y = torch.empty(S, O, device="cuda"), torch.empty(S, O, device="cuda")
    with t:
        q.matmul_q8(t, xq, want, S)
        assert q.device_status() == q.OK
        try:
            q.selftest_q8(0)
            q.matmul_q8(t, xq, y, S)
            with pytest.raises(q.B200QError) as e:
                q.device_status()
            assert e.value.status == q.ETIMEOUT
        finally:
            q.selftest_q8(-1)
        q.matmul_q8(t, xq, y, S)
        assert q.device_status() == q.OK
        assert torch.equal(y, want)
    for bad in ((-2, 0), (1 << 40, 0), (-1, 1), (-1, -9)):
        with pytest.raises(q.B200QError):
            q.selftest_q8(*bad)


def test_replay_after_giving_up(q):
    """A captured call whose blocks partly gave up leaves nothing behind that its next replay takes for its own."""
    import torch
    t, xq, O, S = _long_call(q)
    inputs = [xq.codes.clone(), xq.codes.flip(0).clone()]
    want, y = [torch.empty(S, O, device="cuda") for _ in inputs], torch.empty(S, O, device="cuda")
    with t:
        for c, w in zip(inputs, want):
            xq.codes.copy_(c)
            q.matmul_q8(t, xq, w, S)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            q.matmul_q8(t, xq, y, S, stream=st)
        gave_up = 0
        for k in range(40):
            xq.codes.copy_(inputs[k % 2])
            q.selftest_q8(5000 * k)
            graph.replay()
            try:
                q.device_status()
            except q.B200QError as e:
                assert e.status == q.ETIMEOUT
                gave_up += 1
            finally:
                q.selftest_q8(-1)
            xq.codes.copy_(inputs[1 - k % 2])
            y.fill_(float("nan"))
            graph.replay()
            assert q.device_status() == q.OK
            assert torch.equal(y, want[1 - k % 2]), "after a limit of %d ns" % (5000 * k)
        assert gave_up


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("res", [False, True], ids=["x", "x+r"])
@pytest.mark.parametrize("S,D", [(3, 5), (400, 96), (2, 501), (2, 6144), (3, 5003), (2, 20000)])
def test_rmsnorm_with_a_bad_weight(q, S, D, kind, res):
    """The scale is the largest |y| / 448: where a weight is NaN or infinite it is not finite in any row."""
    import torch
    x, r = _dev(_rows(S, D, D), kind), _dev(synth.normal_f32((S, D), D, 2), kind) if res else None
    for bad in (float("nan"), float("inf")):
        w = _dev(synth.uniform_f32((D,), 0.5, 1.5, D, 3))
        w[D // 2] = bad
        out = _fresh(q, S, D)
        q.rmsnorm_q8(x, w, out, S, D, 1e-6, r=r)
        torch.cuda.synchronize()
        assert not torch.isfinite(out.scales).any()


def test_rows_changed_in_place(q):
    """A call reads and writes the tensors that a Q8Rows holds now, and counts their rows now."""
    import torch
    S, D = 4, 96
    x, out = _dev(_rows(S, D, 1)), q.Q8Rows(S, D)
    q.quantize_q8(x, out, S, D)
    codes, scales = out.codes, out.scales
    before = codes.clone(), scales.clone()
    kept = codes.view(codes.shape), scales.view(scales.shape)      # the old memory stays allocated
    codes.set_(torch.zeros(S, 112, dtype=torch.uint8, device="cuda"))
    scales.set_(torch.zeros(S, device="cuda"))
    q.quantize_q8(2 * x, out, S, D)
    torch.cuda.synchronize()
    assert torch.equal(codes[:, :D], before[0][:, :D]) and torch.equal(scales, 2 * before[1])
    assert torch.equal(kept[0], before[0]) and torch.equal(kept[1], before[1])
    codes.resize_(S - 1, 112)
    with pytest.raises(ValueError):
        q.quantize_q8(x, out, S, D)
    q.quantize_q8(x, out, S - 1, D)
    torch.cuda.synchronize()
    assert torch.equal(scales[:S - 1], before[1][:S - 1])


def test_status_codes(q):
    """What the tensor-core kernel records is reported as what it is, once."""
    for status, words in ((q.ECUDA, "tensor memory"), (q.ETIMEOUT, "bounded wait")):
        q.selftest_q8(-1, status)
        with pytest.raises(q.B200QError, match=words) as e:
            q.device_status()
        assert e.value.status == status
        assert q.device_status() == q.OK


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("op", ["mm", "glu"])
def test_runs_of_several_tiles(q, op, fmt, kind):
    """Runs that begin and end inside a tile and hold whole tiles between: what large pairs and prompts take.  Seen from
    the plan, so that the case stays one: blocks whose last tile is shared and the third of their run, and the fourth."""
    import torch
    O, I, S = (2560 if op == "glu" else 5120) + 20, 5121, 1408
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    p = q.selftest_q8_plan(FMTS[fmt], op == "glu", O, I, S, sms)
    starts = [c * p["items"] // p["grid"] for c in range(p["grid"] + 1)]
    last = {(b - 1) // p["nk"] - a // p["nk"] for a, b in zip(starts, starts[1:]) if a % p["nk"] and b % p["nk"]}
    assert p["cut"] and p["grain"] == 1 and {2, 3} <= last, p
    if op == "mm":
        _mm(q, fmt, O, I, S, kind, "silu", bias=True, res=True, seed=21)
    else:
        _glu(q, fmt, O, I, S, kind, "gelu", bg=True, bu=True, seed=22)


def _one_sign(q, fmt, O, I, S, seed, sign, head, top):
    """Codes of one sign, bytes of one sign below `top`, and `head` columns of the largest of both first."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    most = {"i8": (127, -128), "i4": (7, -8), "i2": (1, -2)}[fmt][sign < 0]
    w = torch.randint(min(sign, most), max(sign, most) + 1, (O, I), generator=g, device="cuda", dtype=torch.int16)
    c = torch.randint(1, top, (S, I), generator=g, device="cuda", dtype=torch.uint8)
    w[:, :head], c[:, :head] = most, 0x7E
    if fmt == "i8":
        codes = w.to(torch.int8).view(torch.uint8)
    else:
        n, bits = 8 // BITS[fmt], BITS[fmt]
        u = (w + 2 ** (bits - 1)).to(torch.uint8).view(O, I // n, n)
        codes = sum(u[:, :, k] << (bits * k) for k in range(n)).to(torch.uint8)
    xq = q.Q8Rows(S, I)
    xq.codes[:, :I] = c
    xq.scales.fill_(1.0)
    return q.tensor_upload(FMTS[fmt], O, I, codes.cpu().numpy(), np.ones(O, np.float32)), w, xq


@pytest.mark.parametrize("S", [2, 1408])
@pytest.mark.parametrize("I", [12288, 32768])
@pytest.mark.parametrize("fmt", list(FMTS))
def test_long_rows_of_one_sign(q, fmt, I, S):
    """The error bound where the running sum is as large as the sum of the magnitudes all along: what each step of the
    tensor cores drops adds up.  Tolerance, per sum |deq x8|: 1e-5, and 4 units in the last place of f32 (2^-23 each) per
    32 columns, twice for int8, whose codes are two operands."""
    import torch
    O = 2432
    tol = 1e-5 + I * 2.0 ** -26 * (2 if fmt == "i8" else 1)
    if S > 8:
        sms = torch.cuda.get_device_properties(0).multi_processor_count
        p = q.selftest_q8_plan(FMTS[fmt], False, O, I, S, sms)
        assert sms != 152 or not p["cut"], p                           # one accumulator holds a whole row's sum
    y = torch.empty(S, O, device="cuda")
    pick = [s for s in (0, 1, S // 2, S - 1)]
    for sign, head, top in ((1, 0, 0x7F), (-1, 0, 0x7F), (1, 512, 0x28), (-1, 64, 0x28), (1, 64, 0x40)):
        t, w, xq = _one_sign(q, fmt, O, I, S, 7, sign, head, top)
        with t:
            q.matmul_q8(t, xq, y, S)
            torch.cuda.synchronize()
        want = xq.values()[pick].double() @ w.double().t()             # |want| = sum |deq x8|: one sign
        off = float(((y[pick].double() - want).abs() / want.abs()).max())
        assert off <= tol, (sign, head, top, off, tol)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S,D", [(1, 6144), (700, 5003), (3, 20000), (2000, 96)])
def test_rows_same_bits_each_time(q, S, D, kind):
    """Sums and maxima in a fixed order: rows, scales and h repeat bit for bit."""
    import torch
    x, r, w = _dev(_rows(S, D, 1), kind), _dev(synth.normal_f32((S, D), 1, 2), kind), _dev(synth.uniform_f32((D,), 0.5, 1.5, 1, 3))
    first = None
    for _ in range(5):
        a, b, h = _fresh(q, S, D), _fresh(q, S, D), torch.empty_like(x)
        q.rmsnorm_q8(x, w, a, S, D, 1e-6, r=r, h=h)
        q.quantize_q8(x, b, S, D)
        got = a.codes, a.scales, b.codes, b.scales, h
        first = first or got
        assert all(torch.equal(u, v) for u, v in zip(first, got))


def test_norm_codes_are_the_nearest(q):
    """Codes of 448 h w / max |h w| in 64 bits.  f32 has three roundings there (h w, the factor, their product, 2^-24 each):
    a code may differ only where the exact quotient is that close to the middle between two codes."""
    import torch
    S, D = 900, 6144
    x, w = _dev(_rows(S, D, 8), "bf16"), _dev(synth.uniform_f32((D,), 0.5, 1.5, 8, 3))
    out = _fresh(q, S, D)
    q.rmsnorm_q8(x, w, out, S, D, 1e-6)
    torch.cuda.synchronize()
    hw = _np64(x) * _np64(w)
    t = hw * (448 / np.abs(hw).max(1, keepdims=True))
    v, _ = _quantised(q, out, D)
    off = v != _e4m3_round(t)
    _, e = np.frexp(np.abs(t))
    half = 2.0 ** (np.maximum(e - 1, -6) - 4.0)
    assert np.all(np.abs(v - t)[off] <= half[off] + 3 * 2.0 ** -24 * np.abs(t)[off])
    assert off.sum() <= S * D * 1e-5
