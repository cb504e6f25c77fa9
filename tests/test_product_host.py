"""Host side of how the 8-bit product is dispatched (CPU only)."""
import ctypes
from pathlib import Path

import pytest

import product_cases

SM_SMEM, CTA_SMEM = 228 * 1024, 1024          # an SM's shared memory, and what a CTA takes beside its own
OWNER_SMEM = 120 * 1024                       # the least of a kernel that takes an SM's whole tensor memory


class Plan(ctypes.Structure):
    """MatmulPlan (csrc/dsv_launch.h)."""
    _fields_ = [(n, ctypes.c_int) for n in ("pair", "swap", "bn", "split", "dual", "smem")]


@pytest.fixture(scope="module")
def plan():
    from dynamic_block_sparse_projection_gb300.build import LIB, build
    build()
    from dynamic_block_sparse_projection_gb300 import binding
    f = ctypes.CDLL(str(LIB))["_ZN3dsv11matmul_planERK10dsv_matmul"]
    f.restype, f.argtypes = Plan, [ctypes.POINTER(binding.Matmul)]
    return lambda *p: f(ctypes.byref(binding.Matmul(*p)))


# M, N, K, a_rows, b_rows of every kind of tile
TILES = [(1, 24576, 2048, 1, 128), (30000, 32, 2048, 1, 128), (1, 128, 128, 1, 128), (33, 2048, 512, 1, 128),
         (1000, 50, 300, 1, 128), (300, 500, 3000, 1, 1), (2300, 2208, 2500, 1, 128)]


def test_products_share_no_sm_with_a_kernel_that_takes_all_tensor_memory(plan):
    """A product that is launched early holds its tensor memory while it waits for the kernel in front of it: that one
    must have its own by then, so the two may not be able to meet on an SM."""
    kinds = set()
    for p in TILES:
        t = plan(*p, 0)
        kinds.add((t.pair, t.bn, t.dual))
        assert t.smem + OWNER_SMEM + 2 * CTA_SMEM > SM_SMEM, p
        assert (2 if t.dual else 1) * (t.smem + CTA_SMEM) <= SM_SMEM, p
    assert kinds == {(0, 32, 0), (0, 32, 1), (0, 64, 0), (0, 128, 0), (1, 128, 0)}
    src = Path(__file__).resolve().parent.parent / "dynamic_block_sparse_projection_gb300" / "csrc"
    for f in src.glob("*.cu"):                # whoever allots tensor memory is one or the other
        if "tmem_alloc(" in f.read_text():
            assert "kTmemOwnerSmem" in f.read_text() or "fits_beside_owner(" in f.read_text(), f.name


def test_arrivals_at_another_cta_are_of_the_clusters_scope():
    """An arrival on a barrier in another CTA's shared memory orders nothing between the two where its scope is the
    CTA's, which it is where none is named."""
    import re
    csrc = Path(__file__).resolve().parent.parent / "dynamic_block_sparse_projection_gb300" / "csrc"
    found = 0
    for f in sorted(csrc.glob("*.cu*")):
        for op in re.findall(r"mbarrier\.arrive[a-z0-9_.:]*\.shared::cluster[a-z0-9_.:]*", f.read_text()):
            found += 1
            assert re.match(r"mbarrier\.arrive(\.expect_tx)?\.(release|relaxed)\.cluster\.", op), f"{f.name}: {op}"
    assert found


def test_the_listed_sizes_take_every_way(plan):
    """Columns of a tile, their side, scales, splits of K and CTAs of an SM: each that a sweep of sizes meets."""
    def kind(m, n, k, ar, br):
        t = plan(m, n, k, ar, br, 0)
        return t.pair, t.bn, t.dual, t.swap, (ar if t.swap else br), 0 if t.pair else t.split

    listed = {kind(*p, *r) for p in product_cases.SMALL + product_cases.PAIRS for r in product_cases.LAYOUTS}
    sizes = [1, 2, 9, 31, 33, 60, 64, 65, 100, 129, 250, 600, 1300, 2500, 5000, 6200, 9900, 15000, 19500, 25000]
    met = {kind(m, n, k, *r) for m in sizes for n in sizes for r in product_cases.LAYOUTS
           for k in (1, 130, 300, 500, 700, 900, 1030, 1300, 1458, 2050, 3000, 6100, 8100, 10000, 11600, 13300, 20000, 40000)}
    assert met <= listed, sorted(met - listed)
    for s in range(1, 9):
        for bn in (32, 64):
            assert {(0, bn, 0, swap, r, s) for swap in (0, 1) for r in (1, 128)} <= listed, (bn, s)
        assert {(0, 128, 0, 0, r, s) for r in (1, 128)} <= listed, s
    groups = [(-(-n // 256), product_cases.columns_of_a_group(k)) for _, n, k in product_cases.PAIRS]
    assert any(tn <= g for tn, g in groups) and sum(tn > g and tn % g for tn, g in groups) >= 2
    assert all(plan(*p, *r, 0).pair for p in product_cases.PAIRS for r in product_cases.LAYOUTS)


def test_a_product_lets_the_next_kernel_come_with_its_tensor_memory_in_hand():
    """What comes early, a kernel of another library too, may take the rest of an SM's tensor memory until the product
    in front of it is done: that one must not still want some."""
    text = (Path(__file__).resolve().parent.parent / "dynamic_block_sparse_projection_gb300" / "csrc" / "matmul_fp8.cu").read_text()
    lines = [line.strip() for line in text.splitlines()]
    at = [i for i, line in enumerate(lines) if line == "cudaTriggerProgrammaticLaunchCompletion();"]
    assert len(at) == 3                                      # the small tile's, and each CTA's of a pair
    for i in at:
        assert any("_alloc(&tmem_slot" in line for line in lines[i - 2:i]), lines[i - 2:i]
