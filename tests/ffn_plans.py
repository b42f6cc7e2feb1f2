"""How the shared FFN cuts its products, asked of the library (no GPU needed)."""
import ctypes
from collections import namedtuple

from mixture_experts_layer_59_b200 import binding as B

PRODUCTS = ("UP", "DOWN", "DAP", "DX", "DW")
PAIRS = 74
Plan = namedtuple("Plan", "bn cluster tiles whole share span kbs")


def plan(T, d, f, product):
    out = (ctypes.c_int * 7)()
    rc = B.lib().moe_debug_shared_ffn_plan(T, d, f, product, out)
    assert rc == 0, (T, d, f, rc)
    return Plan(*out)


def kind(p):
    """split tiles of 128 or 256 columns, one CTA each or several; pairs: whole
    tiles only, or the last ones shared, cut alike or anywhere."""
    if p.bn:
        return f"split {p.bn}" + (" cluster" if p.cluster > 1 else "")
    return "whole" if p.share == 0 else ("shared alike" if p.span % p.share == 0 else "shared anywhere")


KINDS = ("split 128", "split 128 cluster", "split 256", "split 256 cluster", "whole", "shared alike", "shared anywhere")

# Sizes of the GPU tests: between them every kind of cut for every product, with
# widths and row counts that tiles and boxes do not divide.
EXACT_SIZES = [(1, 72, 72), (200, 4096, 2048), (259, 6864, 72), (300, 4096, 2048), (700, 7168, 2048), (1493, 4104, 2056),
               (1500, 4096, 2048), (2500, 1024, 2048), (2511, 1032, 2056), (2971, 136, 3272), (4630, 176, 1016),
               (6207, 544, 272)]
# The same for outputs and workspaces with guard bands: pairs with shared tiles and
# clipped edges, clusters.
GUARD_SIZES = [(300, 1000, 680), (259, 6864, 72), (1493, 4104, 2056), (2511, 1032, 2056), (2971, 136, 3272),
               (4321, 1992, 1352), (5000, 2048, 520), (10000, 2048, 648)]
