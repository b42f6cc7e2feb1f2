"""The cuts of the shared FFN's products into tiles, clusters and shares (host
arithmetic only, no GPU needed)."""
import ctypes
import random

import pytest

from ffn_plans import EXACT_SIZES, GUARD_SIZES, KINDS, PAIRS, PRODUCTS, kind, plan
from mixture_experts_layer_59_b200 import binding as B


def test_refusals():
    out = (ctypes.c_int * 7)()
    call = B.lib().moe_debug_shared_ffn_plan
    assert call(4, 256, 128, 5, out) == -1 and call(4, 256, 128, -1, out) == -1
    assert call(0, 256, 128, 0, out) == -1 and call(4, 256, 128, 0, None) == -1
    assert call(4, 12, 128, 0, out) == -2 and call(1 << 30, 1 << 20, 8, 0, out) == -2


@pytest.mark.parametrize("T", [1 << 20, 200_000_000, 392_000_000, 500_000_000, 700_000_001, 1 << 30])
def test_costs_of_many_k_blocks_stay_in_range(T):
    """The weights' gradients of narrow matrices over very many rows: three tiles, so
    24 pairs can share each.  A part costs 2000 clocks and saves 700 per k-block,
    so at these lengths the most parts that fit are the cheapest."""
    p = plan(T, 8, 8, PRODUCTS.index("DW"))
    assert p.kbs == -(-T // 64) and p.tiles == 3 and p.whole == 0
    assert p.share == -(-p.kbs // (PAIRS // 3))


def walk(p):
    """Per pair the (tile, first, last + 1 k-block) of its share, as the kernel's
    walk goes (whole tiles left out)."""
    for pair in range(PAIRS):
        pos = pair * p.share
        end = min(pos + p.share, (p.tiles - p.whole) * p.span)
        while pos < end:
            t = pos // p.span
            k0, k1 = pos - t * p.span, min(p.span, end - t * p.span)
            pos = t * p.span + k1
            yield pair, t, k0, min(k1, p.kbs)


def check_shares(p):
    shared = p.tiles - p.whole
    assert 0 < shared < PAIRS and p.share <= p.span and p.span >= p.kbs and p.whole % PAIRS == 0
    cover, slots = {t: [] for t in range(shared)}, set()
    for pair, t, k0, k1 in walk(p):
        assert k1 > k0
        cover[t].append((k0, k1, pair))
        seg = 1 if pair * p.share < t * p.span else 0       # its share began in the tile before
        assert (pair, seg) not in slots                     # one place per partial
        slots.add((pair, seg))
    for t, parts in cover.items():
        parts.sort()
        assert parts[0][0] == 0 and parts[-1][1] == p.kbs
        assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
        first = t * p.span // p.share
        n = (t * p.span + p.kbs - 1) // p.share - first + 1
        assert [q for _, _, q in parts] == list(range(first, first + n))   # what the last arrival sums


def test_every_k_block_is_in_one_share():
    rng = random.Random(11)
    seen = {}
    for _ in range(40000):
        T, d, f = (int(2 ** rng.uniform(0, 14.3)), 8 * int(2 ** rng.uniform(0, 10)), 8 * int(2 ** rng.uniform(0, 9)))
        i = rng.randrange(5)
        p = plan(T, d, f, i)
        k = (PRODUCTS[i], kind(p))
        seen[k] = seen.get(k, 0) + 1
        if p.bn:
            assert 1 <= p.cluster <= 8 and p.cluster <= p.kbs and p.tiles * p.cluster <= 148
        elif p.share == 0:
            assert p.whole == p.tiles
        elif seen[k] <= 60:
            check_shares(p)
    # the planner does choose each of them for each product
    assert set(seen) == {(a, b) for a in PRODUCTS for b in KINDS}


def test_gpu_tests_cover_every_cut():
    everything = {(a, b) for a in PRODUCTS for b in KINDS}
    covered = {(a, kind(plan(*s, i))) for s in EXACT_SIZES for i, a in enumerate(PRODUCTS)}
    assert covered == everything, everything - covered
    guarded = {(a, kind(plan(*s, i))) for s in GUARD_SIZES for i, a in enumerate(PRODUCTS)}
    pairs = {(a, b) for a in PRODUCTS for b in KINDS if b.startswith("shared")}
    assert len(guarded & pairs) >= 8 and {a for a, _ in guarded & pairs} >= {"UP", "DOWN", "DAP", "DX"}, guarded
    assert {a for a, b in guarded if b == "split 128 cluster"} >= {"UP", "DAP", "DX"}, guarded
