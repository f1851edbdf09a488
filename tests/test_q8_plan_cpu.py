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
