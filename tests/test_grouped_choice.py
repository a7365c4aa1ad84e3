"""Which kernel a grouped product runs on, by its sizes: whatever is chosen can be launched, and what the header allows
is refused only where no kernel can.  The rule is host code, run here in a program of its own."""
import math
import os
import random
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
MOST = 2 ** 31 - 1  # threads of a launch


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path_factory.mktemp("choice") / "grouped_choice")
    made = subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", os.path.join(HERE, "native", "grouped_choice.cpp"),
                           "-o", exe], capture_output=True, text=True, timeout=120)
    assert made.returncode == 0, made.stderr[-3000:]

    def f(problems):
        run = subprocess.run([exe], input="".join("%s %d %d %d %d\n" % p for p in problems), capture_output=True, text=True,
                             timeout=120)
        assert run.returncode == 0
        out = [tuple(map(int, line.split())) for line in run.stdout.splitlines()]
        assert len(out) == len(problems)
        return out
    return f


def up(a, b):
    return -(-a // b)


def workgroups(op, R, K, M, E, tile):
    """Tiles that a launch must have for any sizes of the groups, a multiple of eight."""
    if op in ("dw", "acc"):
        n = up(M, tile) * up(K, tile) * E
    else:
        rows, cols = (16, 32) if tile == 16 else (tile, tile)
        n = (R // rows + min(E, R)) * up(M if op == "fwd" else K, cols)
    return up(n, 8) * 8


# problems whose quickest kernel would be a launch of more threads than a launch can have
TOO_MANY = [("dw", 768, 8, 131072, 4096), ("fwd", 4096, 8, 131072, 4096), ("fwd", 1 << 29, 8, 8, 1), ("dx", 1 << 29, 8, 8, 1),
            ("fwd", 1 << 30, 8, 8, 1), ("dx", 1 << 30, 8, 8, 4096), ("dx", 4096, 131072, 8, 4096)]


def test_a_larger_tile_where_the_quickest_is_too_many(choose):
    for p, (tile, grid, threads) in zip(TOO_MANY, choose(TOO_MANY)):
        assert tile in (128, 256), (p, tile)
        assert grid == workgroups(*p, tile) and grid * threads <= MOST, (p, tile, grid)
        assert workgroups(*p, tile // 2) * 256 > MOST, p


def test_refused_only_where_no_tile_can(choose):
    rng = random.Random(5)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    problems = [(op, log(1, 1 << 30), 8 * log(1, 1 << 17), 8 * log(1, 1 << 17), log(1, 4096))
                for op in ("fwd", "dx", "dw", "acc") for _ in range(3000)]
    refused = 0
    for p, (tile, grid, threads) in zip(problems, choose(problems)):
        if tile == 0:
            assert workgroups(*p, 256) * 256 > MOST, p
            refused += 1
            continue
        assert tile in ((256,) if p[0] == "acc" else (64, 128, 256) if p[0] == "dw" else (16, 64, 128, 256)), (p, tile)
        assert grid == workgroups(*p, tile) and 0 < grid * threads <= MOST, (p, tile, grid)
    assert 0 < refused < len(problems) // 2


def test_the_choice_of_ordinary_sizes(choose):
    """The kernels whose times the rule was made from."""
    want = [(("fwd", 32, 2048, 1408, 64), 16), (("fwd", 32768, 8192, 32768, 8), 256), (("fwd", 8000, 4096, 1024, 60), 128),
            (("dx", 14211, 5000, 2048, 24), 256), (("dx", 21, 160, 22488, 2), 16), (("dx", 500, 512, 8192, 4), 64),
            (("dw", 32768, 2048, 8192, 16), 256), (("acc", 100, 64, 64, 2), 256), (("dw", 0, 64, 64, 2), 64)]
    got = choose([p for p, _ in want])
    for (p, tile), (chosen, _, _) in zip(want, got):
        if tile == 64:
            assert chosen in (64, 128), (p, chosen)
        else:
            assert chosen == tile, (p, chosen)


@pytest.mark.parametrize("op,R,K,M,E", [("fwd", 1 << 20, 8, 1 << 20, 4096), ("dx", 1 << 30, 1 << 20, 8, 1), ("dw", 8, 1 << 20, 1 << 20, 1),
                                        ("acc", 8, 8, 1 << 20, 4096)])
def test_refused_before_anything_is_enqueued(op, R, K, M, E):
    """As a shape, with addresses that nothing reads."""
    from offload_memory_centric_amd import zi
    at = 1 << 20
    g = zi.zi_grouped(R, K, M, 0, 0, 0, 0, 0, E, zi.ZI_BF16, zi.ZI_F32 if op == "acc" else zi.ZI_BF16, 0, op == "acc")
    with pytest.raises(zi.ZiError) as e:
        if op == "fwd":
            zi.zi_grouped_fwd(g, at, at, at, at, None)
        elif op == "dx":
            zi.zi_grouped_dx(g, at, at, at, None, at)
        else:
            zi.zi_grouped_dw(g, at, at, at, at)
    assert e.value.status == zi.ZI_ERR_SHAPE, str(e.value)
    g.R = 0
    zi.zi_grouped_fwd(g, None, None, None, None, None)  # nothing to do, whatever the sizes
    assert zi.zi_last_error() == ""
