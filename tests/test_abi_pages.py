"""Refusals of the page and beam entry points, checked without a GPU: argument errors come before any launch."""

import ctypes

import pytest
import torch

mxa = pytest.importorskip("mx_block_scaled_quantize_amd",
                          reason="libmx.so not built (run __graft_entry__.build())")
if torch.cuda.is_available():
    pytest.skip("argument-validation tests use fake device addresses; CPU only", allow_module_level=True)
lib = mxa.lib

OK, NULL, SHAPE, ALIGN, UNSUP, LAUNCH, ARG = range(7)
FAKE = 0x10000
BIG = 1 << 40


def caches(*changes):
    a = dict(k=FAKE, k_scales=FAKE, v=FAKE, v_scales=FAKE, pages=4, kv_heads=2, page=16, dim=64)
    return (mxa._KVCacheArgs * max(1, len(changes)))(*(mxa._KVCacheArgs(**{**a, **c}) for c in changes or ({},)))


def caller(f, names, values):
    base = dict(zip(names.split(), values))

    def call(**kw):
        assert set(kw) <= set(base), kw
        return f(*{**base, **kw}.values())
    return call


LAYERS = [(SHAPE, [{"dim": 80}]), (SHAPE, [{"page": 8}]), (SHAPE, [{"kv_heads": 0}]), (SHAPE, [{"pages": -1}]),
          (SHAPE, [{}, {"pages": 5}]), (SHAPE, [{}, {"dim": 128}]), (SHAPE, [{}, {"page": 32}]), (SHAPE, [{}, {"kv_heads": 1}]),
          (NULL, [{"k": None}]), (NULL, [{}, {"v_scales": None}]), (ALIGN, [{"v": FAKE + 8}]), (ALIGN, [{}, {"k_scales": FAKE + 4}]),
          (SHAPE, [{"pages": 1, "kv_heads": 65536, "page": 4096}])]

copy = caller(lib.mx_kv_copy, "src dst layers src_pages dst_pages count stream",
              [caches(), caches(), 1, FAKE, FAKE, 2, None])


@pytest.mark.parametrize("status,layers", LAYERS)
def test_copy_layers(status, layers):
    plain = caches(*[{}] * len(layers))
    assert copy(src=caches(*layers), dst=plain, layers=len(layers)) == status
    assert copy(src=plain, dst=caches(*layers), layers=len(layers)) == status


@pytest.mark.parametrize("status,kw", [
    (NULL, {"src": None}), (NULL, {"dst": None}), (SHAPE, {"layers": 0}), (SHAPE, {"layers": -1}), (SHAPE, {"layers": 65537}),
    (SHAPE, {"count": -1}), (SHAPE, {"count": 1 << 31}), (NULL, {"src_pages": None}), (NULL, {"dst_pages": None}),
    (ALIGN, {"src_pages": FAKE + 2}), (ALIGN, {"dst_pages": FAKE + 1}), (OK, {"count": 0, "src_pages": None}),
    (SHAPE, {"dst": caches({"dim": 128})}), (OK, {"dst": caches({"pages": 0, "k": None})})])
def test_copy(status, kw):
    assert copy(**kw) == status


fork = caller(lib.mx_kv_fork, "caches layers refs table stride cols lens rows parents children cu tokens release refs_out table_out "
              "out_cols lens_out slots space bytes stream",
              [caches(), 1, FAKE, FAKE, 3, 3, FAKE, 2, FAKE, 2, FAKE, 2, 1, FAKE, FAKE + 4096, 3, FAKE + 8192, FAKE, FAKE, 1 << 20,
               None])


@pytest.mark.parametrize("status,layers", LAYERS)
def test_fork_layers(status, layers):
    assert fork(caches=caches(*layers), layers=len(layers)) == status


@pytest.mark.parametrize("status,kw", [
    (NULL, {"caches": None}), (SHAPE, {"layers": 0}), (SHAPE, {"rows": -1}), (SHAPE, {"rows": (1 << 20) + 1}),
    (SHAPE, {"children": -1}), (SHAPE, {"children": (1 << 20) + 1}), (SHAPE, {"tokens": -1}), (SHAPE, {"tokens": 1 << 31}),
    (SHAPE, {"cols": -1}), (SHAPE, {"out_cols": 2}), (SHAPE, {"out_cols": 1 << 28}), (SHAPE, {"stride": 2}),
    (SHAPE, {"parents": None, "children": 3}), (NULL, {"cu": None}), (NULL, {"refs": None}), (NULL, {"refs_out": None}),
    (NULL, {"lens": None}), (NULL, {"table": None}), (NULL, {"table_out": None}), (NULL, {"lens_out": None}),
    (NULL, {"slots": None}), (NULL, {"space": None}), (SHAPE, {"bytes": 0}), (ALIGN, {"space": FAKE + 8}),
    (ALIGN, {"refs": FAKE + 2}), (ALIGN, {"slots": FAKE + 4}), (ALIGN, {"cu": FAKE + 1}), (ALIGN, {"parents": FAKE + 2}),
    (ARG, {"table_out": FAKE}), (ARG, {"lens_out": FAKE})])
def test_fork(status, kw):
    assert fork(**kw) == status


free = caller(lib.mx_kv_free, "refs pages page table stride cols lens rows keep refs_out lens_out space bytes stream",
              [FAKE, 4, 16, FAKE, 3, 3, FAKE, 2, None, FAKE, FAKE, None, 0, None])
MANY = {"pages": 1 << 17, "rows": 1 << 10, "cols": 1 << 9, "stride": 1 << 9}


@pytest.mark.parametrize("status,kw", [
    (SHAPE, {"pages": -1}), (SHAPE, {"pages": 1 << 31}), (SHAPE, {"page": 8}), (SHAPE, {"page": 24}), (SHAPE, {"page": 1 << 17}),
    (SHAPE, {"rows": -1}), (SHAPE, {"rows": (1 << 20) + 1}), (SHAPE, {"cols": -1}), (SHAPE, {"cols": 1 << 28, "stride": 1 << 28}),
    (SHAPE, {"stride": 2}), (NULL, {"refs": None}), (NULL, {"refs_out": None}), (NULL, {"table": None}), (NULL, {"lens": None}),
    (NULL, {"lens_out": None}), (ALIGN, {"refs": FAKE + 1}), (ALIGN, {"table": FAKE + 2}), (ALIGN, {"keep": FAKE + 2}),
    (ARG, {"keep": FAKE}), (SHAPE, MANY), (SHAPE, {**MANY, "space": FAKE, "bytes": 1 << 20}),
    (NULL, {**MANY, "bytes": 1 << 30}), (ALIGN, {**MANY, "space": FAKE + 4, "bytes": 1 << 30}),
    (OK, {"rows": 0, "lens": None, "table": None})])
def test_free(status, kw):
    assert free(**kw) == status


compact = caller(lib.mx_kv_compact, "caches layers refs table stride cols lens rows refs_out table_out used space bytes stream",
                 [caches(), 1, FAKE, FAKE, 3, 3, FAKE, 2, FAKE, FAKE, FAKE, FAKE, 1 << 20, None])


@pytest.mark.parametrize("status,layers", LAYERS)
def test_compact_layers(status, layers):
    assert compact(caches=caches(*layers), layers=len(layers)) == status


@pytest.mark.parametrize("status,kw", [
    (NULL, {"caches": None}), (SHAPE, {"layers": 0}), (SHAPE, {"rows": -1}), (SHAPE, {"cols": -1}), (SHAPE, {"stride": 2}),
    (NULL, {"refs": None}), (NULL, {"refs_out": None}), (NULL, {"table": None}), (NULL, {"table_out": None}),
    (NULL, {"lens": None}), (NULL, {"used": None}), (NULL, {"space": None}), (SHAPE, {"bytes": 16}), (ALIGN, {"space": FAKE + 4}),
    (ALIGN, {"used": FAKE + 1}), (ARG, {"stride": 4})])
def test_compact(status, kw):
    assert compact(**kw) == status


select = caller(lib.mx_beam_select, "x dt requests beams vocab rs bs scores finished width eos pad history lens cols scores_out parents "
                "tokens finished_out history_out lens_out space bytes stream",
                [FAKE, 1, 2, 3, 100, 300, 100, FAKE, None, 4, -1, 0, None, None, 0, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, 1 << 20,
                 None])


@pytest.mark.parametrize("status,kw", [
    (UNSUP, {"dt": 3}), (UNSUP, {"dt": -1}), (SHAPE, {"requests": -1}), (SHAPE, {"requests": BIG}), (SHAPE, {"beams": 0}),
    (SHAPE, {"beams": 65}), (SHAPE, {"vocab": 0}), (SHAPE, {"vocab": BIG}), (SHAPE, {"width": 0}), (SHAPE, {"width": 65}),
    (SHAPE, {"cols": -1}), (SHAPE, {"cols": 1 << 31}), (ARG, {"eos": 1 << 31}), (ARG, {"pad": -(1 << 31) - 1}),
    (NULL, {"x": None}), (NULL, {"scores": None}), (NULL, {"scores_out": None}), (NULL, {"parents": None}),
    (NULL, {"tokens": None}), (NULL, {"finished_out": None}), (NULL, {"history": FAKE}), (NULL, {"lens": FAKE, "cols": 0}),
    (NULL, {"lens": FAKE, "lens_out": FAKE, "cols": 4}), (ALIGN, {"x": FAKE + 1}), (ALIGN, {"dt": 0, "x": FAKE + 2}),
    (ALIGN, {"scores": FAKE + 2}), (SHAPE, {"bytes": 16}), (NULL, {"space": None}), (ALIGN, {"space": FAKE + 8}),
    (OK, {"requests": 0, "x": None})])
def test_select(status, kw):
    assert select(**kw) == status


def test_frees_of_fewer_than_2_19_entries_need_no_workspace():
    n = ctypes.c_int64(-1)
    for rows, cols, none in ((1, (1 << 19) - 1, True), ((1 << 19) - 1, 1, True), (1 << 10, (1 << 9) - 1, True),
                             (1 << 19, 1, False), (1, 1 << 19, False)):
        assert lib.mx_kv_free_workspace(1 << 20, rows, cols, 16, ctypes.byref(n)) == OK and (n.value == 0) == none


def test_workspaces():
    n = ctypes.c_int64(-1)
    at = ctypes.byref(n)
    assert lib.mx_kv_fork_workspace(100, 4, 8, 9, 16, at) == OK and n.value % 16 == 0 and n.value > 0
    assert lib.mx_kv_fork_workspace(100, 4, 8, 9, 15, at) == SHAPE
    assert lib.mx_kv_fork_workspace(100, 4, 8, 9, 16, None) == NULL
    assert lib.mx_kv_fork_workspace((1 << 31) - 1, 1 << 20, 1 << 20, (1 << 31) - 1, 16, at) == OK and n.value < 1 << 30
    assert lib.mx_kv_free_workspace(1 << 17, 1 << 10, 1 << 9, 16, at) == OK and n.value >= 4 << 19
    assert lib.mx_kv_free_workspace(1 << 17, 1 << 10, 1 << 8, 16, at) == OK and n.value == 0
    assert lib.mx_kv_free_workspace(1 << 17, 1 << 10, 1 << 9, 15, at) == SHAPE
    assert lib.mx_kv_compact_workspace(0, at) == OK and n.value > 0
    assert lib.mx_kv_compact_workspace((1 << 31) - 1, at) == OK and n.value < 1 << 35
    assert lib.mx_kv_compact_workspace(-1, at) == SHAPE
    assert lib.mx_beam_select_workspace(2, 3, 1000, 4, at) == OK and n.value >= 6 * (16 + 32)
    assert lib.mx_beam_select_workspace(2, 3, 1000, 0, at) == SHAPE
    # a grid has fewer than 2^32 threads
    assert lib.mx_beam_select_workspace(1 << 20, 64, 1, 64, at) == OK
    assert lib.mx_beam_select_workspace((1 << 20) + 1, 1, 1, 1, at) == SHAPE
