"""Token log probabilities on the GPU against the fp64 oracle.

d = (x - max) inv_temp log2(e) carries two roundings (2^-23 |d|) and 2^d another 2^-22; terms with large |d| are small, so
the sum of exponentials is good to 3e-6 and its logarithm to that; lse then rounds at its own size.  So lse, logp and
the alternatives are within 5e-6 (1 + |max inv_temp| + |value|), the entropy within 5e-6 (1 + ln vocab).  The gradient's p
inherits lse's error as a relative one: 2e-5 (1 + |max inv_temp|) of the terms' magnitudes, 2^-8 more in bf16.  Ids are
compared for equality."""

import numpy as np
import pytest
import torch

from oracle import train_ops as O
from zero_sharded_gb300 import cz

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _strided(t, pad, offset=0):
    wide = torch.full((t.shape[0] * (t.shape[1] + pad) + offset,), 77.0, dtype=t.dtype, device="cuda")
    v = wide[offset:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
    v.copy_(t)
    return v


def _forward(x, t, inv_temp, k):
    rows = x.shape[0]
    o = dict(logp=torch.zeros(rows, device="cuda"), entropy=torch.zeros(rows, device="cuda"), lse=torch.zeros(rows, device="cuda"),
             ids=torch.full((rows, k), -7, dtype=torch.int64, device="cuda"), top=torch.zeros(rows, k, device="cuda"))
    cz.cz_token_logp_fwd(x, t, o["logp"], entropy=o["entropy"], lse=o["lse"], top_ids=o["ids"], top_logp=o["top"], inv_temp=inv_temp)
    torch.cuda.synchronize()
    return o


def _near(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and np.isinf(got).sum() == inf.sum(), what
    fine = np.isfinite(want)
    err, tol = np.abs(got - np.where(fine, want, 0)), np.broadcast_to(tol, want.shape)
    assert (err[fine] <= tol[fine]).all(), (what, float((err[fine] / tol[fine]).max()))


def _check_forward(x, t, inv_temp, k):
    o = _forward(x, t, inv_temp, k)
    xn = x.double().cpu().numpy()
    f = O.logp_fwd(xn, t.cpu().numpy(), inv_temp, k)
    m = np.where(np.isfinite(f["lse"]), np.abs(np.where(np.isfinite(xn), xn, -np.inf).max(1)), 0) * inv_temp
    mag = lambda v: 5e-6 * (1 + m + np.where(np.isfinite(v), np.abs(v), 0))  # noqa: E731
    _near(o["lse"], f["lse"], mag(f["lse"]), "lse")
    _near(o["logp"], f["logp"], mag(f["logp"]), "logp")
    _near(o["entropy"], f["entropy"], 5e-6 * (1 + np.log(x.shape[1])), "entropy")
    assert np.array_equal(o["ids"].cpu().numpy(), f["ids"]), "ids"
    _near(o["top"], f["top"], 5e-6 * (1 + m[:, None] + np.where(np.isfinite(f["top"]), np.abs(f["top"]), 0)), "top")
    return o, f


def _logits(rows, vocab, seed, scale=4.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g) * scale * torch.rand(rows, 1, generator=g)
    return x, torch.randint(0, vocab, (rows,), generator=g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,k,inv_temp,pad,offset", [
    (1, 1, 1, 1.0, 0, 0), (2, 5, 5, 0.5, 0, 0), (3, 7, 0, 1.0, 2, 3), (40, 33, 32, 1.0, 0, 1), (300, 1001, 8, 2.0, 0, 0),
    (700, 128, 20, 1.0, 0, 0), (5, 4099, 20, 1.25, 5, 0), (3, 40000, 32, 1.0, 0, 2), (1, 131072, 20, 1.0, 0, 0), (2, 100003, 8, 1.0, 13, 0)])
def test_forward(rows, vocab, k, inv_temp, pad, offset, dtype):
    x, t = _logits(rows, vocab, vocab + rows)
    if rows > 1:
        t[0] = -1
    _check_forward(_strided(x.to(TYPES[dtype]), pad, offset), t.cuda(), inv_temp, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [3, 1000, 50000])
@pytest.mark.parametrize("inv_temp", [1.0, 1.5])
def test_masked_empty_and_special_rows(vocab, dtype, inv_temp):
    low = torch.finfo(TYPES[dtype]).min
    x, t = _logits(11, vocab, 5)
    x[1] = -float("inf")                                # nothing left
    x[2, 1:] = -float("inf")                            # one entry left
    x[3, ::2] = low                                     # masked by the lowest value
    x[4] = low                                          # nothing but masks
    x[5, vocab // 2] = float("nan")
    x[6, 0] = float("inf")
    x[7] = 0.25                                         # all ties
    x[8, :] = torch.where(torch.arange(vocab) % 2 == 0, 0.0, -0.0)
    x[9] += 500.0
    t[2], t[3], t[10] = 0, 1, vocab + 3
    x, t = x.to(TYPES[dtype]).cuda(), t.cuda()
    k = min(vocab, 20)
    _check_forward(x, t, inv_temp, k)
    fwd = _forward(x, t, inv_temp, 0)
    g, ge = torch.randn(11, device="cuda"), torch.randn(11, device="cuda")
    d = torch.full_like(x, 9.0)
    cz.cz_token_logp_bwd(x, t, fwd["lse"], d, entropy=fwd["entropy"], g_logp=g, g_entropy=ge, inv_temp=inv_temp)
    d = d.float().cpu()
    assert bool((d[1] == 0).all())
    assert torch.isnan(d).all(1).tolist() == [i in (5, 6, 10) for i in range(11)]
    assert bool((d[2, 1:] == 0).all()) and bool((d[3, ::2] == 0).all())
    assert bool((d[4] == 0).all())


@pytest.mark.parametrize("vocab,dtype,repeat", [(1000, "f32", 110), (1003, "bf16", 110), (20001, "f32", 55), (40000, "bf16", 55)])
def test_many_rows(vocab, dtype, repeat):
    """Rows enough for the smaller blocks: plain and special ones, repeated; copies at the same alignment (every eighth has
    it) give the same bits."""
    x, t = _logits(23, vocab, 17)
    x[1] = -float("inf")
    x[2, 1:] = -float("inf")
    x[3, ::2] = torch.finfo(TYPES[dtype]).min
    x[4] = 0.25
    x[5, vocab // 2] = float("nan")
    x[6] = torch.arange(vocab) * 2.0 ** -12             # ascending
    x[7] = torch.floor(torch.arange(vocab) / 512.0)
    x[8, 3] = float("inf")
    t[2], t[3], t[9], t[10] = 0, 1, -1, vocab
    x, t = x.to(TYPES[dtype]).cuda(), t.cuda()
    for k in (32, 5):
        _check_forward(x, t, 1.25, k)
        one = _forward(x.repeat(repeat, 1), t.repeat(repeat), 1.25, k)
        f = O.logp_fwd(x.double().cpu().numpy(), t.cpu().numpy(), 1.25, k)
        for name, v in one.items():
            v = v.view(repeat, 23, -1)
            bits = v if v.dtype == torch.int64 else v.view(torch.int32)
            assert bool((bits[8:] == bits[:-8]).all()), name
        m = np.where(np.isfinite(f["lse"]), np.abs(x.double().nan_to_num(0, 0, -1e300).max(1).values.cpu().numpy()), 0) * 1.25
        mag = lambda v: 5e-6 * (1 + m + np.where(np.isfinite(v), np.abs(v), 0))  # noqa: E731
        for c in range(8):
            own = {name: v[23 * c:23 * c + 23] for name, v in one.items()}
            for name in ("lse", "logp"):
                _near(own[name], f[name], mag(f[name]), name)
            _near(own["entropy"], f["entropy"], 5e-6 * (1 + np.log(vocab)), "entropy")
            assert np.array_equal(own["ids"].cpu().numpy(), f["ids"])
            _near(own["top"], f["top"], 5e-6 * (1 + m[:, None] + np.where(np.isfinite(f["top"]), np.abs(f["top"]), 0)), "top")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("at", [3e4, -3e4, 1e30, -1e30, 3e38])
def test_rows_of_large_values(at, dtype):
    """Rows whose values differ by less than their size: spacing of the type around a large maximum, with masked entries
    of both kinds and a part of nothing but masks."""
    vocab = 70001
    x, t = _logits(4, vocab, 12, 3.0)
    x = (x * abs(at) * 2.0 ** -7).clamp(-0.4 * abs(at), 0.0) + at
    x[1, ::3] = -float("inf")
    x[2, vocab // 3:] = torch.finfo(TYPES[dtype]).min
    x[2, vocab // 2::2] = -float("inf")
    x[3, 4096:] = -float("inf")
    t[2], t[3] = 0, 1
    t[1] = 1
    _check_forward(x.to(TYPES[dtype]).cuda(), t.cuda(), 1.0, 20)


@pytest.mark.parametrize("shape", ["ascending", "one thread's part", "sorted blocks"])
def test_alternatives_of_skewed_rows(shape):
    """Rows that put forward more candidates than the buffer holds."""
    vocab = 70000
    i = torch.arange(vocab, dtype=torch.float32)
    if shape == "ascending":
        x = i * 1e-4
    elif shape == "one thread's part":
        x = torch.where((i.long() // 4) % 512 < 40, 5.0, 0.0) + i * 1e-6
    else:
        x = torch.floor(i / 4096)
    x = torch.stack([x, x.flip(0)]).repeat(200, 1)[:400]
    _check_forward(x[:3].cuda(), torch.tensor([5, 0, vocab - 1]).cuda(), 1.0, 32)      # a cluster a row
    o = _forward(x.cuda(), torch.zeros(400, dtype=torch.int64, device="cuda"), 1.0, 32)  # a block a row
    f = O.logp_fwd(x[:2].numpy(), [0, 0], 1.0, 32)
    assert np.array_equal(o["ids"].cpu().numpy(), np.tile(f["ids"], (200, 1)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,inv_temp,pad,offset,entropy", [
    (1, 1, 1.0, 0, 0, True), (5, 7, 0.5, 1, 3, True), (33, 1000, 1.0, 0, 0, False), (3, 40001, 1.25, 0, 1, True), (200, 4096, 2.0, 8, 0, True),
    (2, 131072, 1.0, 0, 0, True)])
@pytest.mark.parametrize("place", ["own", "other alignment", "in place"])
def test_backward(rows, vocab, inv_temp, pad, offset, entropy, dtype, place):
    x, t = _logits(rows, vocab, vocab)
    if rows > 2:
        t[1] = -1
    x, t = _strided(x.to(TYPES[dtype]), pad, offset), t.cuda()
    fwd = _forward(x, t, inv_temp, 0)
    g, ge = torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda") if entropy else None
    xn = x.double().cpu().numpy()
    d = x if place == "in place" else _strided(torch.zeros(rows, vocab, dtype=TYPES[dtype]), pad + (place != "own"), offset + (place != "own"))
    cz.cz_token_logp_bwd(x, t, fwd["lse"], d, entropy=fwd["entropy"] if entropy else None, g_logp=g, g_entropy=ge, inv_temp=inv_temp)
    torch.cuda.synchronize()
    gn, gen = g.double().cpu().numpy(), None if ge is None else ge.double().cpu().numpy()
    want = O.logp_bwd(xn, t.cpu().numpy(), gn, gen, inv_temp)
    f = O.logp_fwd(xn, t.cpu().numpy(), inv_temp)
    lp = xn * inv_temp - f["lse"][:, None]
    live = (t.cpu().numpy() >= 0)[:, None]
    mag = np.exp(lp) * (live * np.abs(gn[:, None]) + (0 if gen is None else np.abs(gen[:, None]) * (np.abs(lp) + f["entropy"][:, None])))
    hot = np.zeros_like(xn)
    hot[np.arange(rows), np.maximum(t.cpu().numpy(), 0)] = 1
    mag += live * hot * np.abs(gn[:, None])
    m = np.abs(xn.max(1, keepdims=True)) * inv_temp
    tol = 2e-5 * (1 + m) * mag * inv_temp + 1e-30 + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
    err = np.abs(d.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())
    if pad and place == "own":
        assert bool((d.as_strided((rows, pad), (vocab + pad, 1), d.storage_offset() + vocab) == 77.0).all())


def test_gradient_against_differences_of_the_definition():
    """A random direction, step 1e-4 in fp64 (truncation 1e-8): the gradient's own bound holds."""
    x, t = _logits(4, 300, 8)
    t[2] = -1
    xc, tc = x.cuda(), t.cuda()
    f = _forward(xc, tc, 0.8, 0)
    g, ge = torch.randn(4, device="cuda"), torch.randn(4, device="cuda")
    d = torch.empty_like(xc)
    cz.cz_token_logp_bwd(xc, tc, f["lse"], d, entropy=f["entropy"], g_logp=g, g_entropy=ge, inv_temp=0.8)
    step = np.random.default_rng(0).standard_normal((4, 300))
    ends = []
    for e in (1e-4, -1e-4):
        o = O.logp_fwd(x.double().numpy() + e * step, t.numpy(), 0.8)
        ends.append((o["logp"] * g.cpu().numpy()).sum() + (o["entropy"] * ge.cpu().numpy()).sum())
    dn = d.double().cpu().numpy()
    assert abs((ends[0] - ends[1]) / 2e-4 - (dn * step).sum()) <= 2e-5 * 20 * np.abs(dn * step).sum()


def test_no_rows_graph_capture_and_repeats():
    e = torch.empty(0, 10, device="cuda")
    v, i = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    cz.cz_token_logp_fwd(e, i, v, lse=v)
    cz.cz_token_logp_bwd(e, i, v, e)
    x, t = _logits(5, 50000, 3)
    x, t = x.cuda(), t.cuda()
    want = _forward(x, t, 1.0, 8)
    o = {k: torch.zeros_like(w) for k, w in want.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cz.cz_token_logp_fwd(x, t, o["logp"], entropy=o["entropy"], lse=o["lse"], top_ids=o["ids"], top_logp=o["top"], stream=side)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], want[k]) for k in o)
