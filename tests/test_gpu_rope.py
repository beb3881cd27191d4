"""Rotary tables, rotation and the append to a paged MXFP8 cache on the GPU.

Rotation is exact to the bit: FP32 products and sums rounded one by one, then one
rounding to the storage type, which numpy and torch do alike.  Codes and scales
are those of the quantizer's oracle on the FP32 values."""

import numpy as np
import pytest
import torch

from oracle import attention as oa
from tests.gpu_util import assert_bytes_equal, assert_float_equal, dev, import_library

pytestmark = pytest.mark.gpu

mxa = import_library()

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def data(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * torch.exp2(torch.randn(shape[-1], generator=g))).to(DT[dtype]).to(dev())


def table_of(rows, rot, seed=0):
    g = np.random.default_rng(seed)
    return torch.from_numpy(oa.rope_table(rows, rot, 1e4 * (1 + g.random())).astype(np.float32)).to(dev())


def rotated_f32(x, pos, table, layout, inverse=False):
    return oa.rotate(x.float().cpu().numpy(), pos.cpu().numpy(), table.cpu().numpy(), layout, inverse)


def bits(t):
    return t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16).cpu().numpy()


@pytest.mark.parametrize("rows,rot", [(1, 2), (7, 34), (513, 128), (8192, 128), (70001, 62), (131072, 128)])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn", "bands"])
def test_table(rows, rot, scaling):
    if scaling == "ntk" and rot == 2:
        pytest.skip("no such table")
    got = mxa.mx_rope_table(rows, rot, 5e5, scaling, 16.0, 8192).cpu().numpy().astype(np.float64)
    want = oa.rope_table(rows, rot, 5e5, scaling, 16.0, 8192)
    f, m = oa.frequencies(rot, 5e5, scaling, 16.0, 8192)
    # one rounding to FP32; frequency, angle and product errors of a few 2^-53 of the angle on either
    # side, and of 2^-52 for each of at most 32 steps
    angle = np.arange(rows)[:, None, None] * f[None, :, None]
    tol = 2.0 ** -24 * np.abs(want) + m * 2.0 ** -52 * (8 * angle + 64)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 64, 64), (5, 3, 96, 20), (33, 8, 128, 128), (700, 7, 128, 64),
                                                  (1021, 32, 128, 128), (2, 4, 6, 6), (3, 5, 10, 2), (64, 9, 256, 130)])
def test_rotation_and_its_inverse(tokens, heads, dim, rot, dtype, layout):
    x = data((tokens, heads, dim), dtype, tokens + dim)
    t = table_of(2048, rot)
    pos = torch.randint(0, 2048, (tokens,), generator=torch.Generator().manual_seed(3)).int().to(dev())
    for inverse in (False, True):
        got = mxa.mx_rope(x, pos, t, layout, inverse)
        want = torch.from_numpy(rotated_f32(x, pos, t, layout, inverse)).to(DT[dtype])
        assert_bytes_equal(bits(got), bits(want), f"inverse {inverse}")


@pytest.mark.parametrize("shift", [0, 1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rotation_of_slices_and_in_place(dtype, shift):
    """Heads of a fused projection, at addresses that allow 16-byte, 4-byte and single accesses."""
    flat = data((50, 12 * 64 + 8), dtype, 5)
    x = flat[:, shift:shift + 12 * 64].unflatten(1, (12, 64))[:, 2:9]
    pos = torch.arange(50, dtype=torch.int32, device=dev())
    t = table_of(64, 64)
    want = torch.from_numpy(rotated_f32(x, pos, t, "half")).to(DT[dtype])
    rest = flat.clone()
    assert_bytes_equal(bits(mxa.mx_rope(x, pos, t)), bits(want), "slice")
    got = mxa.mx_rope(x, pos, t, out=x)
    assert got is x
    assert_bytes_equal(bits(x), bits(want), "in place")
    rest[:, shift:shift + 12 * 64].unflatten(1, (12, 64))[:, 2:9] = want.to(dev())
    assert_bytes_equal(bits(flat), bits(rest), "what lies around it")


def test_gradient_against_differences():
    """w . rope(x) is linear in x: its difference along any direction is the inverse rotation of w there."""
    x, w, d = (data((40, 4, 96), "f32", s).double() for s in (1, 2, 3))
    t, pos = table_of(64, 48), torch.arange(40, dtype=torch.int32, device=dev())
    grad = mxa.mx_rope(w.float(), pos, t, "interleaved", inverse=True).double()
    up, down = (mxa.mx_rope((x + s * d).float(), pos, t, "interleaved").double() for s in (1, -1))
    num, got = ((up - down) * w).sum() / 2, (grad * d).sum()
    # inputs, products, sums and the gradient are each rounded by 2^-24 of magnitudes below |x| + |d|
    tol = 2.0 ** -24 * 8 * ((x.abs() + d.abs()) * 2 * w.abs()).sum()
    assert abs(num - got) <= tol


def test_positions_without_a_row_give_nan():
    x = data((3, 2, 64), "bf16", 1)
    pos = torch.tensor([-1, 5, 64], dtype=torch.int32, device=dev())
    y = mxa.mx_rope(x, pos, table_of(64, 32)).float()
    assert y[0, :, :32].isnan().all() and y[2, :, :32].isnan().all() and y[1].isfinite().all()
    assert torch.equal(y[:, :, 32:], x[:, :, 32:].float())


# ---------------------------------------------------------------- append
def check_append(tokens, heads, hk, dim, page, rot, layout, dtype, slots, pages, with_q=True, with_table=True, spoil=None,
                 shift=0):
    width = (heads + 2 * hk) * dim
    qkv = data((tokens, width + 8), dtype, tokens + dim)[:, shift:shift + width].unflatten(1, (-1, dim))
    if spoil is not None:
        spoil(qkv)
    q, k, v = qkv[:, :heads], qkv[:, heads:heads + hk], qkv[:, heads + hk:]
    pos = torch.randint(0, 512, (tokens,), generator=torch.Generator().manual_seed(3)).int().to(dev())
    t = table_of(512, rot)
    cache = mxa.new_kv_cache(pages, hk, page, dim)
    for c in cache:
        c.fill_(0xA5)                 # what is not appended keeps its bytes
    want = [c.cpu().numpy().copy() for c in cache]
    got_q = mxa.mx_kv_append(k, v, cache, torch.tensor(slots, device=dev()), pos if with_table else None,
                             t if with_table else None, layout, q=q if with_q else None)
    kr = rotated_f32(k, pos, t, layout) if with_table else k.float().cpu().numpy()
    oa.append(want, kr, v.float().cpu().numpy(), slots)
    for name, g, w in zip(mxa.KVCache._fields, cache, want):
        assert_bytes_equal(g.cpu().numpy(), w, name)
    if with_q:
        assert_float_equal(got_q.float().cpu().numpy(),
                           torch.from_numpy(rotated_f32(q, pos, t, layout)).to(DT[dtype]).float().numpy(), "q")
    else:
        assert got_q is None


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("heads,hk,dim,page,rot", [(32, 8, 128, 64, 128), (4, 4, 64, 16, 32), (7, 1, 96, 32, 96),
                                                   (6, 2, 96, 48, 48), (2, 2, 192, 128, 20), (8, 2, 256, 16, 256)])
def test_append_of_scattered_tokens(heads, hk, dim, page, rot, dtype, layout):
    pages = 300 // page + 2
    slots = np.random.default_rng(dim).permutation(pages * page)[:37].astype(np.int64)
    check_append(37, heads, hk, dim, page, rot, layout, dtype, slots, pages)


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 400])
def test_append_of_a_run(tokens):
    check_append(tokens, 8, 4, 128, 64, 128, "half", "bf16", np.arange(tokens, dtype=np.int64) + 29, 8)


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_append_of_unaligned_rows(shift, layout):
    check_append(20, 3, 2, 64, 16, 64, layout, "bf16", np.arange(20, dtype=np.int64)[::-1].copy(), 2, shift=shift)


def test_append_skips_slots_outside_the_cache():
    check_append(6, 2, 2, 64, 16, 64, "half", "bf16", np.array([-1, 5, 32, 31, 1 << 40, -(1 << 40)], dtype=np.int64), 2)


def test_append_without_queries_or_rotation():
    slots = np.arange(9, dtype=np.int64)
    check_append(9, 2, 2, 64, 16, 64, "half", "f16", slots, 1, with_q=False)
    check_append(9, 2, 2, 64, 16, 64, "half", "f32", slots, 1, with_q=False, with_table=False)


def test_append_of_zeros_and_tiny_and_nonfinite_values():
    def spoil(x):
        x[0] = 0.0
        x[1] *= 1e-38
        x[2, :, 5] = float("inf")
        x[3, :, 70] = float("nan")
        x[4] = 1e-45
    g = mxa.new_kv_cache(1, 2, 16, 128)
    check_append(5, 2, 2, 128, 16, 2, "half", "f32", np.arange(5, dtype=np.int64), 1, with_q=False, with_table=False,
                 spoil=spoil)
    del g


def test_empty_calls():
    t = table_of(8, 64)
    e = torch.empty((0, 4, 64), device=dev())
    none = torch.empty(0, dtype=torch.int32, device=dev())
    assert mxa.mx_rope(e, none, t).shape == (0, 4, 64)
    cache = mxa.new_kv_cache(2, 4, 16, 64)
    assert mxa.mx_kv_append(e, e, cache, none.long(), none, t, q=e).shape == (0, 4, 64)
    assert mxa.mx_rope_table(0, 64).shape == (0, 32, 2)
