"""Refusals of the rotary and cache entry points, checked without a GPU: argument
errors come before any launch."""

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
INF = float("inf")


def cache(**kw):
    a = dict(k=FAKE, k_scales=FAKE, v=FAKE, v_scales=FAKE, pages=4, kv_heads=2, page=16, dim=64)
    return mxa._KVCacheArgs(**{**a, **kw})


def caller(f, names, values):
    base = dict(zip(names, values))

    def call(**kw):
        assert set(kw) <= set(base), kw
        return f(*{**base, **kw}.values())
    return call


table = caller(lib.mx_rope_table, "rows rot base scaling factor orig out stream".split(),
               [8, 64, 1e4, 0, 1.0, 0, FAKE, None])


@pytest.mark.parametrize("status,kw", [
    (UNSUP, {"scaling": 5}), (UNSUP, {"scaling": -1}), (SHAPE, {"rows": -1}), (SHAPE, {"rows": (1 << 31) + 1}),
    (SHAPE, {"rot": 0}), (SHAPE, {"rot": 7}), (SHAPE, {"rot": 1026}), (SHAPE, {"rot": 2, "scaling": 2, "factor": 2.0}),
    (ARG, {"base": 1.0}), (ARG, {"base": INF}), (ARG, {"base": float("nan")}), (ARG, {"scaling": 1, "factor": 0.5}),
    (ARG, {"scaling": 3, "factor": 2.0}), (ARG, {"scaling": 4, "factor": INF, "orig": 8}), (NULL, {"out": None}),
    (ARG, {"scaling": 2, "factor": 1e300, "base": 1e300}), (ALIGN, {"out": FAKE + 4}), (OK, {"rows": 0, "out": None})])
def test_rope_table(status, kw):
    assert table(**kw) == status


rope = caller(lib.mx_rope, "x dt tokens heads dim xt xh pos table rows rot layout inv y yt yh stream".split(),
              [FAKE, 1, 4, 2, 64, 128, 64, FAKE, FAKE, 8, 64, 0, 0, FAKE, 128, 64, None])


@pytest.mark.parametrize("status,kw", [
    (UNSUP, {"dt": 3}), (UNSUP, {"layout": 2}), (SHAPE, {"tokens": -1}), (SHAPE, {"rot": 66}), (SHAPE, {"rot": 5}),
    (SHAPE, {"dim": 1}), (SHAPE, {"heads": -1}), (SHAPE, {"rows": -1}), (NULL, {"x": None}), (NULL, {"pos": None}),
    (NULL, {"table": None}), (NULL, {"y": None}), (ALIGN, {"x": FAKE + 1}), (ALIGN, {"dt": 0, "x": FAKE + 2}),
    (ALIGN, {"table": FAKE + 8}), (ALIGN, {"pos": FAKE + 2}), (OK, {"tokens": 0, "x": None}), (OK, {"heads": 0})])
def test_rope(status, kw):
    assert rope(**kw) == status


append = caller(lib.mx_kv_append,
                "k v dt tokens kt kh vt vh cache slots pos table rows rot layout q heads qt qh q_out stream".split(),
                [FAKE, FAKE, 1, 4, 128, 64, 128, 64, cache(), FAKE, FAKE, FAKE, 8, 64, 0, FAKE, 8, 512, 64, FAKE, None])


@pytest.mark.parametrize("status,kw", [
    (NULL, {"cache": None}), (SHAPE, {"cache": cache(dim=80)}), (SHAPE, {"cache": cache(page=24)}),
    (SHAPE, {"cache": cache(page=0)}), (SHAPE, {"cache": cache(kv_heads=0)}), (SHAPE, {"cache": cache(pages=-1)}),
    (SHAPE, {"cache": cache(pages=1 << 40)}), (NULL, {"cache": cache(v_scales=None)}), (ALIGN, {"cache": cache(k=FAKE + 8)}),
    (UNSUP, {"dt": 7}), (UNSUP, {"layout": -1}), (SHAPE, {"rot": 128}), (SHAPE, {"tokens": -4}), (SHAPE, {"heads": 0}),
    (NULL, {"k": None}), (NULL, {"v": None}), (NULL, {"slots": None}), (NULL, {"pos": None}), (NULL, {"table": None}),
    (NULL, {"q_out": None}), (ALIGN, {"k": FAKE + 1}), (ALIGN, {"slots": FAKE + 4}), (ALIGN, {"q": FAKE + 1}),
    (ALIGN, {"table": FAKE + 8}), (OK, {"tokens": 0})])
def test_append(status, kw):
    assert append(**kw) == status


attention = caller(lib.mx_paged_attention,
                   "q dt tokens heads qt qh cache table stride cols cu lens requests max_q max_kv window scale out lse "
                   "space bytes stream".split(),
                   [FAKE, 1, 4, 8, 512, 64, cache(), FAKE, 4, 4, FAKE, FAKE, 4, 1, 64, 0, 0.1, FAKE, FAKE, FAKE, 1 << 40, None])


@pytest.mark.parametrize("status,kw", [
    (NULL, {"cache": None}), (UNSUP, {"dt": 0}), (SHAPE, {"cache": cache(dim=32)}), (SHAPE, {"heads": 7}),
    (SHAPE, {"heads": 0}), (SHAPE, {"tokens": -1}), (SHAPE, {"requests": -1}), (SHAPE, {"stride": -1}),
    (ARG, {"max_q": -1}), (ARG, {"max_kv": -1}), (ARG, {"window": -1}), (ARG, {"scale": 0.0}), (ARG, {"scale": INF}),
    (ARG, {"scale": float("nan")}), (ARG, {"scale": -1.0}), (NULL, {"q": None}), (NULL, {"cu": None}), (NULL, {"lens": None}),
    (NULL, {"out": None}), (NULL, {"table": None}), (NULL, {"cache": cache(k=None)}), (ALIGN, {"q": FAKE + 8}),
    (ALIGN, {"qt": 516}), (ALIGN, {"out": FAKE + 8}), (ALIGN, {"lens": FAKE + 2}), (ALIGN, {"space": FAKE + 4}),
    (ALIGN, {"cache": cache(v=FAKE + 8)}), (SHAPE, {"max_kv": 1 << 40}), (OK, {"tokens": 0}), (OK, {"requests": 0})])
def test_attention(status, kw):
    assert attention(**kw) == status


@pytest.mark.parametrize("status,args", [
    (SHAPE, (4, 7, 2, 64, 4, 1, 64, 0)), (SHAPE, (4, 8, 2, 80, 4, 1, 64, 0)), (ARG, (4, 8, 2, 64, 4, -1, 64, 0)),
    (SHAPE, (-1, 8, 2, 64, 4, 1, 64, 0))])
def test_workspace(status, args):
    assert lib.mx_paged_attention_workspace(*args, ctypes.c_int64(0)) == status
    assert lib.mx_paged_attention_workspace(*args, None) == NULL


def test_binding_refuses():
    x, pos, t = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32), torch.zeros(8, 32, 2)
    c = mxa.KVCache(*(torch.zeros((2, 2, 16, n), dtype=torch.uint8) for n in (64, 2, 64, 2)))
    slots, cu, lens, table_ = torch.zeros(4, dtype=torch.int64), torch.zeros(3, dtype=torch.int32), pos[:2], pos.view(2, 2)
    half = x.bfloat16()
    good = dict(q=half, cache=c, page_table=table_, cu=cu, lens=lens, max_q=1, max_kv=1)
    for f in (lambda: mxa.mx_rope(x, pos, t), lambda: mxa.mx_kv_append(x, x, c, slots, pos, t),
              lambda: mxa.mx_paged_attention(**good), lambda: mxa.mx_rope_table(8, 64, device="cpu")):
        with pytest.raises(ValueError, match="device tensors only"):
            f()
    for f in (lambda: mxa.mx_rope(x, pos.long(), t), lambda: mxa.mx_rope(x, pos[:3], t), lambda: mxa.mx_rope(x, pos, t.double()),
              lambda: mxa.mx_rope(x.transpose(1, 2), pos, t), lambda: mxa.mx_rope(x, pos, t, "other"),
              lambda: mxa.mx_rope(x.int(), pos, t), lambda: mxa.mx_rope(x, pos, t, out=half),
              lambda: mxa.mx_rope_table(8, 63, device="cpu"), lambda: mxa.mx_rope_table(8, 64, scaling="more", device="cpu"),
              lambda: mxa.mx_kv_append(x[:, :1], x, c, slots, pos, t), lambda: mxa.mx_kv_append(x, half, c, slots, pos, t),
              lambda: mxa.mx_kv_append(x, x, c, slots.int(), pos, t), lambda: mxa.mx_kv_append(x, x, c, slots, None, t),
              lambda: mxa.mx_kv_append(x, x, c, slots, q=x), lambda: mxa.mx_kv_append(x, x, c, slots, pos, t, q=half),
              lambda: mxa.mx_kv_append(x, x, c._replace(v=c.v[:1]), slots, pos, t),
              lambda: mxa.mx_kv_append(x, x, c._replace(k_scales=c.k_scales.transpose(0, 1)), slots, pos, t),
              lambda: mxa.mx_paged_attention(**{**good, "q": half[..., :32]}),
              lambda: mxa.mx_paged_attention(**{**good, "q": half[:, :1]}),
              lambda: mxa.mx_paged_attention(**{**good, "cu": cu[:2]}),
              lambda: mxa.mx_paged_attention(**{**good, "lens": lens.long()}),
              lambda: mxa.mx_paged_attention(**{**good, "page_table": table_[:1]}),
              lambda: mxa.mx_paged_attention(**{**good, "page_table": table_.t()}),
              lambda: mxa.mx_paged_attention(**{**good, "out": x})):
        with pytest.raises(ValueError):
            f()
