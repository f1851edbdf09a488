"""How the 8-bit products are launched: host arithmetic on sizes, checked without a GPU."""
import random

import pytest

SMS = 152


@pytest.fixture(scope="module")
def q():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import quantized_weight_quant_gb300 as q
    return q


def _draws(n, seed):
    rng = random.Random(seed)
    for _ in range(n):
        yield (rng.choice([1, 2, 3]), rng.random() < 0.5, int(2 ** rng.uniform(0, 15)), int(2 ** rng.uniform(0, 15)),
               int(2 ** rng.uniform(0, 12)))


def test_refusals(q):
    for bad in ((0, 0, 8, 8, 1, SMS), (4, 0, 8, 8, 1, SMS), (1, 0, 0, 8, 1, SMS), (1, 0, 8, 0, 1, SMS),
                (1, 0, 8, 8, 0, SMS), (1, 0, 8, 8, 1, 0)):
        with pytest.raises(q.B200QError):
            q.selftest_q8_plan(*bad)
    assert q.lib.b200q_selftest_q8_plan(1, 0, 8, 8, 1, SMS, None) == q.EINVAL


def test_plans_are_whole(q):
    """Every plan fits the GPU, and its runs cover every (tile, k-block) item once."""
    for fmt, pair, O, I, S in _draws(3000, 1):
        p = q.selftest_q8_plan(fmt, pair, O, I, S)
        what = (fmt, pair, O, I, S, p)
        assert p["few"] == 0 or (S <= 8 and p["few_smem"] <= 227 * 1024 and p["few_warps"] <= 32), what
        assert p["ok"] and S <= p["part"], what
        assert p["N"] % 16 == 0 and 16 <= p["N"] <= 192 and p["N"] * p["n_tiles"] >= S > p["N"] * (p["n_tiles"] - 1), what
        assert p["tiles"] == -(-O // (64 if pair else 128)) * p["n_tiles"], what
        assert p["nk"] == -(-I // 128) and p["items"] == p["tiles"] * p["nk"], what
        assert 1 <= p["grid"] <= SMS and p["grain"] in (1, p["nk"]), what
        units = p["items"] // p["grain"]
        starts = [c * units // p["grid"] * p["grain"] for c in range(p["grid"] + 1)]
        assert starts[0] == 0 and starts[-1] == p["items"] and all(a < b for a, b in zip(starts, starts[1:])), what
        shared = any(s % p["nk"] for s in starts)
        assert shared == bool(p["cut"]), what


INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("pair", [0, 1])
@pytest.mark.parametrize("fmt", [1, 2, 3])
@pytest.mark.parametrize("I", [2 ** 30 - 1, 2 ** 30, 2 ** 30 + 77, INT_MAX - 75000, INT_MAX - 200, INT_MAX - 64, INT_MAX])
def test_longest_rows(q, fmt, pair, I):
    """Rows of up to 2^31 - 1 codes: x never fits in the few-row kernel's shared memory, and the k-blocks are counted."""
    for S in range(1, 9):
        p = q.selftest_q8_plan(fmt, pair, 40, I, S)
        assert p["few"] == 0, (S, p)
        assert p["ok"] and p["nk"] == (I + 127) // 128 and p["items"] == p["tiles"] * p["nk"], (S, p)


def test_most_rows(q):
    """Batches of up to 2^31 - 1 rows are cut into launches that end."""
    for S in (1, 2 ** 16, 2 ** 16 + 1, INT_MAX - 2 ** 16, INT_MAX - 1, INT_MAX):
        p = q.selftest_q8_plan(2, 0, 40, 64, S)
        assert p["part"] == 2 ** 16 and p["launches"] == -(-S // 2 ** 16), (S, p)
    p = q.selftest_q8_plan(1, 0, INT_MAX, 64, 9)
    assert p["tiles"] == -(-INT_MAX // 128)


def _form(p):
    """whole tiles, equal parts of a tile, or even runs"""
    if not p["cut"]:
        return "whole"
    return "parts" if p["grid"] % p["tiles"] == 0 else "runs"


# Calls whose forms were timed against one another: the fastest, us of all three
# (None: that form is not to be had or is another one).
TIMED = [
    (2, 0, 10240, 12288, 16, "runs", 34.7, None, 26.5),
    (2, 0, 10240, 12288, 96, "runs", 37.6, None, 29.9),
    (2, 0, 10240, 12288, 192, "runs", 44.8, None, 37.3),
    (2, 0, 5120, 12288, 300, "runs", 40.9, None, 33.0),
    (1, 0, 12288, 8192, 16, "runs", 41.3, None, 34.2),
    (1, 0, 5120, 8192, 300, "runs", 45.4, None, 37.0),
    (1, 0, 8192, 8192, 32, "runs", None, 29.5, 27.8),
    (1, 1, 5120, 6144, 16, "runs", 32.5, None, 26.0),
    (1, 1, 5120, 6144, 48, "runs", 33.5, None, 27.0),
    (2, 0, 11008, 4096, 32, "whole", 16.5, None, 19.1),
    (2, 1, 4096, 2048, 16, "whole", 10.4, 12.9, None),
    (2, 1, 4096, 2048, 144, "whole", 13.5, 16.6, None),
    (2, 0, 6144, 12288, 1571, "whole", 113, None, 120),
    (2, 0, 12288, 256, 176, "whole", 11.7, None, 33.0),
    (2, 0, 512, 512, 300, "whole", 11.5, None, 17.5),
    (2, 1, 5120, 6144, 192, "whole", 26.5, None, 31.8),
    (2, 1, 5120, 6144, 96, "whole", 22.4, None, 25.4),
    (1, 0, 5120, 8192, 192, "parts", 47.4, 31.6, 33.7),
    (3, 0, 5001, 4097, 77, "parts", None, 16.9, 20.8),
    (3, 0, 5001, 4097, 16, "parts", None, 13.7, 16.2),
]


@pytest.mark.parametrize("fmt,pair,O,I,S,form,whole,parts,runs", TIMED)
def test_the_faster_form_is_taken(q, fmt, pair, O, I, S, form, whole, parts, runs):
    times = {k: v for k, v in (("whole", whole), ("parts", parts), ("runs", runs)) if v}
    assert min(times, key=times.get) == form
    p = q.selftest_q8_plan(fmt, pair, O, I, S)
    assert _form(p) == form, p
    if form == "whole":
        assert p["grid"] == min(p["tiles"], SMS), p                # no SM idle while tiles wait


def test_shared_tiles_and_their_planes(q):
    """What the kernel derives from a plan by itself: which block owns an item, which blocks share a tile, and in which of
    its two planes a block holds its part."""
    cut = 0
    for fmt, pair, O, I, S in _draws(3000, 2):
        p = q.selftest_q8_plan(fmt, pair, O, I, S)
        if not p["cut"]:
            continue
        cut += 1
        n, nk, what = p["items"], p["nk"], (fmt, pair, O, I, S, p)
        starts = [c * n // p["grid"] for c in range(p["grid"] + 1)]
        owner = lambda i: ((i + 1) * p["grid"] - 1) // n
        for c in range(p["grid"]):
            assert owner(starts[c]) == c == owner(starts[c + 1] - 1), what
            for tile in range(starts[c] // nk + 1, (starts[c + 1] - 1) // nk):
                assert owner(tile * nk) == owner(tile * nk + nk - 1) == c, what      # between its ends a block has whole tiles
        for tile in {s // nk for s in starts[1:-1] if s % nk}:
            first, last = owner(tile * nk), owner(tile * nk + nk - 1)
            assert 0 <= first < last < p["grid"] and last - first + 1 < 1024, what
            assert all(starts[c] // nk == tile for c in range(first + 1, last + 1)), what   # first plane, but for the first block
    assert cut > 500
