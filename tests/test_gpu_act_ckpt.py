"""8-bit activation checkpoints on the GPU against the fp64 oracle.

encode and decode are specified to the bit (the scale is the smallest power of two that holds the block, q rounds to
nearest even, q 2^E is exact in both types), so they are compared for equality.  The weight gradient multiplies exact
bf16 values and adds in fp32: a sum over T tokens rounds at most once every 16 of them on the tensor cores and a few
times more where parts are joined, each time by 2^-23 of at most S = sum |dy x^|, so |error| <= (T/16 + 16) 2^-23 S, and
2^-8 of the result more where it is stored as bf16.
"""

import numpy as np
import pytest
import torch

from oracle import train_ops as O
from zero_sharded_gb300 import cz

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _values(rows, cols, seed, corners=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 12, (rows, 1)))
    x[:, rng.random(cols) < 0.02] *= 30
    if corners and rows * cols > 40:
        f = x.reshape(-1)
        f[::37] = np.rint(f[::37] * 2) / 2            # ties
        if rows > 6:
            x[0] = 0
            x[1, -1] = np.nan
            x[2, 0] = -np.inf
            x[3] *= 2.0 ** -130                        # below the smallest scale
            x[4, :: 3] = 127.0 * 2.0 ** 3              # the largest value of a scale, and one step more
            x[5, cols // 2] = 128.0 * 2.0 ** 10
            x[6, 0] = 3.38e38
    return torch.from_numpy(x.astype(np.float32))


def _strided(t, pad):
    wide = torch.full((t.shape[0], t.shape[1] + pad), 77.0, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _ckpt(rows, cols):
    return torch.full((cz.cz_act_size(rows, cols),), 0xA5, dtype=torch.uint8, device="cuda")


def _bits(t):
    return t.contiguous().cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32).numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 31, 0), (3, 32, 0), (9, 33, 0), (17, 64, 8), (130, 200, 0), (7, 257, 3),
                                           (64, 520, 1), (33, 2048, 0), (515, 1000, 24), (2, 16385, 0)])
def test_encode_decode_bits(rows, cols, pad, dtype):
    x = _strided(_values(rows, cols, rows + cols).to(TYPES[dtype]).cuda(), pad)
    ck = _ckpt(rows, cols)
    cz.cz_act_encode(x, ck)
    out = _strided(torch.zeros(rows, cols, dtype=TYPES[dtype]).cuda(), pad)
    cz.cz_act_decode(ck, out)
    torch.cuda.synchronize()
    q, b = O.ckpt_encode(x.float().cpu().numpy())
    gq, gb = O.ckpt_split(ck.cpu().numpy(), rows, cols)
    assert np.array_equal(gb, b)
    assert np.array_equal(gq, q)
    want = torch.from_numpy(O.ckpt_decode(q, b, cols).astype(np.float32)).to(TYPES[dtype])
    got = out.cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert np.array_equal(_bits(torch.where(nan, 0.0, got.float())), _bits(torch.where(nan, 0.0, want.float())))
    if pad:
        assert bool((out.as_strided((rows, pad), (cols + pad, 1), cols) == 77.0).all()), "written past the row"


def test_encode_of_an_offset_view_and_a_side_stream():
    base = torch.randn(40, 300, device="cuda").to(torch.bfloat16)
    x = base[3:20, 5:261]                               # 2-byte aligned rows
    ck, out = _ckpt(17, 256), torch.empty(17, 256, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cz.cz_act_encode(x, ck, stream=s)
    cz.cz_act_decode(ck, out, stream=s)
    s.synchronize()
    q, b = O.ckpt_encode(x.float().cpu().numpy())
    assert np.array_equal(O.ckpt_decode(q, b, 256), out.double().cpu().numpy())


def _wgrad_case(rows, n_out, n_in, out, add, pad=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, n_in, generator=gen)
    dy = _strided((0.01 * torch.randn(rows, n_out, generator=gen)).to(torch.bfloat16).cuda(), pad)
    ck = torch.zeros(max(1, cz.cz_act_size(rows, n_in)), dtype=torch.uint8, device="cuda")
    cz.cz_act_encode(x.cuda(), ck)
    # the gradient lies inside a flat buffer, between sentinels
    flat = torch.full((n_out * n_in + 12,), 5.0, dtype=TYPES[out], device="cuda")
    off = 4
    g = flat[off:off + n_out * n_in].view(n_out, n_in)
    a = None
    if add == "other":
        a = torch.randn(n_out, n_in, generator=gen).to(TYPES[out]).cuda()
    elif add == "inplace":
        g.copy_(torch.randn(n_out, n_in, generator=gen))
        a = g
    a0 = None if a is None else a.double().cpu().numpy()
    ws = torch.zeros(cz.cz_act_wgrad_workspace(dy, n_in), dtype=torch.uint8, device="cuda")
    cz.cz_act_wgrad(dy, ck, g, add=a, workspace=ws)
    assert cz.cz_device_status(None, ws) == cz.CZ_OK
    xh = torch.empty(rows, n_in, dtype=torch.float32, device="cuda")
    cz.cz_act_decode(ck, xh)
    xh, d = xh.double().cpu().numpy(), dy.double().cpu().numpy()
    want = O.wgrad(d, xh, a0)
    err = np.abs(g.double().cpu().numpy() - want)
    tol = (rows / 16 + 16) * 2.0 ** -23 * (np.abs(d).T @ np.abs(xh) + (0 if a0 is None else np.abs(a0))) + 1e-30
    if out == "bf16":
        tol += 2.0 ** -8 * np.abs(want)
    assert (err <= tol).all(), float((err / tol).max())
    assert bool((flat[:off] == 5.0).all()) and bool((flat[off + n_out * n_in:] == 5.0).all()), "written outside the tensor"
    return flat


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("rows,n_out,n_in,add,pad", [
    (1, 1, 1, None, 0), (1, 8, 32, None, 0), (5, 40, 24, "other", 0), (64, 256, 256, None, 0), (63, 257, 255, "inplace", 0),
    (65, 128, 512, "other", 8), (200, 300, 100, None, 4), (129, 77, 1001, "inplace", 1), (1000, 192, 96, None, 0),
    (2050, 520, 264, "other", 0), (4097, 64, 48, None, 0), (300, 2056, 1032, None, 0), (640, 1024, 2048, "inplace", 0)])
def test_wgrad_against_oracle(rows, n_out, n_in, add, pad, out):
    _wgrad_case(rows, n_out, n_in, out, add, pad, seed=rows)


def test_wgrad_many_tiles_and_a_long_sum():
    _wgrad_case(520, 6144, 2048, "f32", "inplace", seed=3)
    _wgrad_case(16384, 256, 264, "f32", None, seed=4)


def test_wgrad_with_little_workspace_takes_panels():
    """The smallest workspace (64 columns at a time), one for a panel and a half of tiles, and the recommended one: all right."""
    rows, n_out, n_in = 700, 300, 1000
    x, dy = torch.randn(rows, n_in, device="cuda"), torch.randn(rows, n_out, device="cuda").to(torch.bfloat16)
    ck = _ckpt(rows, n_in)
    cz.cz_act_encode(x, ck)
    add = torch.randn(n_out, n_in, device="cuda")
    xh = torch.empty_like(x)
    cz.cz_act_decode(ck, xh)
    d, xn = dy.double().cpu().numpy(), xh.double().cpu().numpy()
    want = O.wgrad(d, xn, add.double().cpu().numpy())
    tol = (rows / 16 + 16) * 2.0 ** -23 * (np.abs(d).T @ np.abs(xn) + np.abs(add.double().cpu().numpy()))
    copy = -(-2 * rows * 304 // 256) * 256               # dy's rows are 600 bytes: not on 16-byte boundaries
    least = 256 + copy + 128 * rows
    for size in (least, least + 1000, 256 + copy + 2 * rows * 400, cz.cz_act_wgrad_workspace(dy, n_in)):
        g = torch.empty(n_out, n_in, device="cuda")
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        cz.cz_act_wgrad(dy, ck, g, add=add, workspace=ws)
        assert cz.cz_device_status(None, ws) == cz.CZ_OK
        assert (np.abs(g.double().cpu().numpy() - want) <= tol).all()
    with pytest.raises(cz.CzError):
        cz.cz_act_wgrad(dy, ck, g, workspace=ws[:least - 1])


def test_wgrad_of_no_rows_is_the_added_gradient():
    for add in (None, "other"):
        flat = _wgrad_case(0, 40, 72, "f32", add)
        if add is None:
            assert bool((flat[4:4 + 40 * 72] == 0).all())


def test_wgrad_is_the_same_every_time_and_nan_blocks_show():
    a = _wgrad_case(3000, 320, 200, "f32", None, seed=9)
    b = _wgrad_case(3000, 320, 200, "f32", None, seed=9)
    assert torch.equal(a, b)
    x = torch.randn(50, 96, device="cuda")
    x[7, 40] = float("nan")                              # block 32..63 of token 7
    ck, dy = _ckpt(50, 96), torch.ones(50, 32, device="cuda", dtype=torch.bfloat16)
    cz.cz_act_encode(x, ck)
    g = torch.zeros(32, 96, device="cuda")
    ws = torch.zeros(cz.cz_act_wgrad_workspace(dy, 96), dtype=torch.uint8, device="cuda")
    cz.cz_act_wgrad(dy, ck, g, workspace=ws)
    nan = torch.isnan(g).cpu()
    assert bool(nan[:, 32:64].all()) and not bool(nan[:, :32].any()) and not bool(nan[:, 64:].any())
