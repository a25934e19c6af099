"""Norms around a block with gate and residual scales on the GPU against the fp64 oracle.

Everything between loads and stores is fp32: sums of squares of up to 16384 terms in trees of depth < 60 (relative error
< 60 2^-24 = 3.6e-6, halved by the square root), about ten further roundings (6e-7) and the exponential of a gate
(2^-21 for |gate| < 8).  So an output is within 1e-5 of the sum of the magnitudes of its terms, and a gradient, which
goes through two such chains, within 3e-5; 2^-8 of the value more where it is stored as bf16."""

import numpy as np
import pytest
import torch

from oracle import train_ops as O
from zero_sharded_gb300 import cz

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
H, Y = 0.75, 1.25


def _strided(t, pad):
    wide = torch.full((t.shape[0], t.shape[1] + pad), 77.0, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _inputs(rows, cols, ht, yt, gate, pad, seed=0):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    s = dict(h=_strided((3 * rnd(rows, cols)).to(TYPES[ht]), pad), y=_strided((rnd(rows, cols) * torch.exp(rnd(rows, 1))).to(TYPES[yt]), pad),
             dx=_strided((0.1 * rnd(rows, cols)).to(TYPES[yt]), pad), dh=_strided((0.1 * rnd(rows, cols)).to(TYPES[ht]), pad),
             w_post=(1 + 0.2 * rnd(cols)).cuda(), w_pre=(1 + 0.2 * rnd(cols)).cuda())
    if rows > 2:
        s["y"][1] = 0                                    # a row of nothing
    s["gate"] = None if gate is None else rnd(cols).cuda() if gate == "channel" else _strided(rnd(rows, cols).to(TYPES[yt]), pad)
    return s


def _within(got, want, mag, dtype, tol, what):
    err = np.abs(_np(got) - want)
    bound = tol * mag + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0) + 1e-30
    assert np.isfinite(_np(got)).all(), what
    assert (err <= bound).all(), (what, float((err / bound).max()))


CASES = [(1, 1, "f32", "f32", None, "identity", 0), (1, 64, "bf16", "bf16", None, "identity", 0), (3, 33, "f32", "bf16", "token", "silu", 0),
         (19, 200, "bf16", "bf16", "channel", "sigmoid", 0), (130, 256, "f32", "f32", "token", "sigmoid", 8),
         (37, 1000, "bf16", "f32", "channel", "silu", 0), (700, 96, "f32", "bf16", None, "identity", 1),
         (65, 2047, "f32", "bf16", "token", "silu", 0), (40, 2048, "bf16", "bf16", "channel", "identity", 0),
         (9, 4104, "bf16", "bf16", "token", "sigmoid", 24), (401, 5120, "bf16", "bf16", "channel", "sigmoid", 0),
         (5, 8193, "f32", "f32", None, "identity", 0), (3, 16384, "bf16", "bf16", "channel", "silu", 0), (2, 16383, "f32", "bf16", None, "identity", 0)]


@pytest.mark.parametrize("norms", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("rows,cols,ht,yt,gate,act,pad", CASES)
def test_forward(rows, cols, ht, yt, gate, act, pad, norms):
    post, pre = norms
    s = _inputs(rows, cols, ht, yt, gate, pad, seed=cols)
    h_out, x = _strided(torch.zeros(rows, cols, dtype=TYPES[ht]), pad), _strided(torch.zeros(rows, cols, dtype=TYPES[yt]), pad)
    rp, rx = torch.zeros(rows, device="cuda"), torch.zeros(rows, device="cuda")
    cks = [torch.zeros(cz.cz_act_size(rows, cols), dtype=torch.uint8, device="cuda") for _ in range(3)]
    cz.cz_block_norm_fwd(s["h"], s["y"], h_out, x=x if pre else None, w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"],
                         gate_act=act, h_scale=H, y_scale=Y, post_norm=post, pre_norm=pre, rstd_post=rp, rstd_pre=rx,
                         h_ckpt=cks[0], y_ckpt=cks[1], x_ckpt=cks[2] if pre else None)
    f = O.norm_fwd(_np(s["h"]), _np(s["y"]), _np(s["w_post"]), _np(s["w_pre"]), _np(s["gate"]), act, H, Y, post=post, pre=pre)
    g = 1.0 if s["gate"] is None else np.abs(O.gate_act(_np(s["gate"]), act)[0])
    mag = H * np.abs(_np(s["h"])) + Y * g * np.abs(f["n"])
    _within(h_out, f["h"], mag, TYPES[ht], 1e-5, "h")
    if post:
        _within(rp, f["r_post"], f["r_post"], torch.float32, 1e-5, "r_post")
    if pre:
        mag = np.abs(_np(s["w_pre"])) * (f["r_pre"][:, None] * mag + np.abs(f["h"]) * f["r_pre"][:, None])
        _within(x, f["x"], mag, TYPES[yt], 1e-5, "x")
        _within(rx, f["r_pre"], f["r_pre"], torch.float32, 1e-5, "r_pre")
    if pad:
        assert bool((h_out.as_strided((rows, pad), (cols + pad, 1), cols) == 77.0).all()), "written past the row"
    # the checkpoints: y's to the bit; those of computed values within the format's error of them
    q, b = O.ckpt_encode(s["y"].float().cpu().numpy())
    gq, gb = O.ckpt_split(cks[1].cpu().numpy(), rows, cols)
    assert np.array_equal(gq, q) and np.array_equal(gb, b)
    for ck, want in ((cks[0], f["h"]), (cks[2], f["x"] if pre else None)):
        if want is None:
            continue
        gq, gb = O.ckpt_split(ck.cpu().numpy(), rows, cols)
        back = O.ckpt_decode(gq, gb, cols)
        for k in range(0, cols, 32):
            top = np.abs(want[:, k:k + 32]).max(1, keepdims=True)
            assert (np.abs(back[:, k:k + 32] - want[:, k:k + 32]) <= top * (1 / 127 + 1e-4)).all()


def _backward(s, rows, cols, act, post, pre, ckpt, accumulate=False, workspace=True):
    f = O.norm_fwd(_np(s["h"]), _np(s["y"]), _np(s["w_post"]), _np(s["w_pre"]), _np(s["gate"]), act, H, Y, post=post, pre=pre)
    pad = s["h"].stride(0) - cols if rows > 1 else 0
    h2 = _strided(torch.from_numpy(f["h"]).to(s["h"].dtype), pad)
    rp, rx = (torch.from_numpy(f[k]).float().cuda() for k in ("r_post", "r_pre"))
    out = dict(dh=_strided(torch.zeros(rows, cols, dtype=s["h"].dtype), pad), dy=_strided(torch.zeros(rows, cols, dtype=s["y"].dtype), pad))
    start = {}
    for k, on in (("dw_post", post), ("dw_pre", pre)):
        if on:
            start[k] = torch.randn(cols, device="cuda")
            out[k] = start[k].clone()
    if s["gate"] is not None:
        if s["gate"].dim() == 1:
            start["dgate"] = torch.randn(cols, device="cuda")
            out["dgate"] = start["dgate"].clone()
        else:
            out["dgate"] = _strided(torch.zeros(rows, cols, dtype=s["y"].dtype), pad)
    cks = {}
    hv, yv = h2, s["y"]
    if ckpt:
        for k, t in (("h_ckpt", h2), ("y_ckpt", s["y"])):
            cks[k] = torch.zeros(cz.cz_act_size(rows, cols), dtype=torch.uint8, device="cuda")
            cz.cz_act_encode(t, cks[k])
        hv, yv = (torch.empty(rows, cols, device="cuda") for _ in range(2))
        cz.cz_act_decode(cks["h_ckpt"], hv)
        cz.cz_act_decode(cks["y_ckpt"], yv)
    ws = torch.zeros(cz.cz_block_norm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    cz.cz_block_norm_bwd(None if ckpt else h2, None if ckpt else s["y"], s["dx"] if pre else None, s["dh"], w_post=s["w_post"],
                         w_pre=s["w_pre"], gate=s["gate"], gate_act=act, h_scale=H, y_scale=Y, post_norm=post, pre_norm=pre,
                         rstd_post=rp, rstd_pre=rx, accumulate=accumulate, workspace=ws, **out, **cks)
    torch.cuda.synchronize()
    a = dict(w_post=_np(s["w_post"]), w_pre=_np(s["w_pre"]), gate=_np(s["gate"]), act=act, h_scale=H, y_scale=Y, post=post, pre=pre)
    want = O.norm_bwd(_np(hv), _np(yv), _np(s["dx"]), _np(s["dh"]), _np(rp), _np(rx), **a)
    # magnitudes of the terms, stage by stage
    r_h, r_y = _np(rx)[:, None], _np(rp)[:, None]
    hh, yh = np.abs(_np(hv)) * r_h, np.abs(_np(yv)) * (r_y if post else 1.0)
    d = np.abs(_np(s["dh"]))
    mag = {}
    if pre:
        gx = np.abs(_np(s["dx"]) * a["w_pre"])
        d = d + r_h * (gx + hh * (gx * hh).mean(1, keepdims=True))
        mag["dw_pre"] = (np.abs(_np(s["dx"])) * hh).sum(0)
    value, slope = (1.0, 0.0) if a["gate"] is None else (np.abs(v) for v in O.gate_act(a["gate"], act))
    n = yh * (np.abs(a["w_post"]) if post else 1.0)
    dn = Y * value * d
    mag["dh"] = H * d
    # silu's slope is a sum of terms of both signs
    mag["dgate"] = Y * (slope + (0.5 if act == "silu" else 0.0)) * n * d
    if post:
        gy = dn * np.abs(a["w_post"])
        mag["dw_post"] = (dn * yh).sum(0)
        mag["dy"] = r_y * (gy + yh * (gy * yh).mean(1, keepdims=True))
    else:
        mag["dy"] = dn
    for k, t in out.items():
        w, m = want[k], mag[k]
        if k == "dgate" and s["gate"].dim() == 1:
            w, m = w.sum(0), m.sum(0)
        if accumulate and k in start:
            w, m = w + _np(start[k]), m + np.abs(_np(start[k]))
        _within(t, w, m, t.dtype, 3e-5, k)
        if pad and t.dim() == 2:
            assert bool((t.as_strided((rows, pad), (cols + pad, 1), cols) == 77.0).all()), "written past the row"
    return out


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("norms", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("rows,cols,ht,yt,gate,act,pad", CASES)
def test_backward(rows, cols, ht, yt, gate, act, pad, norms, ckpt):
    _backward(_inputs(rows, cols, ht, yt, gate, pad, seed=cols + 1), rows, cols, act, *norms, ckpt)


@pytest.mark.parametrize("rows,cols,ht,yt,gate,act,pad,ckpt", [
    (170300, 8, "bf16", "bf16", "channel", "sigmoid", 0, False),          # 70 rows a row group
    (400, 8456, "bf16", "bf16", "channel", "silu", 0, False),             # rows over the blocks of a cluster, several rows each
    (400, 8456, "f32", "bf16", "channel", "silu", 0, True), (311, 8193, "bf16", "bf16", None, "identity", 1, False),
    (170, 12299, "f32", "f32", "token", "sigmoid", 0, False), (170, 16384, "f32", "f32", "token", "silu", 0, False),
    (165, 16383, "bf16", "bf16", None, "identity", 0, True)])
def test_backward_walks_over_rows(rows, cols, ht, yt, gate, act, pad, ckpt):
    s = _inputs(rows, cols, ht, yt, gate, pad, seed=cols + 2)
    a = _backward(s, rows, cols, act, True, True, ckpt)
    b = _backward(s, rows, cols, act, True, True, ckpt)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_backward_accumulates_and_repeats_bit_for_bit():
    s = _inputs(1500, 320, "f32", "bf16", "channel", 0, seed=5)
    _backward(s, 1500, 320, "sigmoid", True, True, False, accumulate=True)
    a = _backward(s, 1500, 320, "sigmoid", True, True, False)
    b = _backward(s, 1500, 320, "sigmoid", True, True, False)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_in_place_stream_and_gradient():
    """h_out may be h, and dh may be dh_in: the same bits as with buffers of their own."""
    s = _inputs(50, 512, "bf16", "bf16", None, 0, seed=6)
    out, x, r = torch.empty_like(s["h"]), torch.empty_like(s["y"]), torch.empty(2, 50, device="cuda")
    cz.cz_block_norm_fwd(s["h"], s["y"], out, x=x, rstd_post=r[0], rstd_pre=r[1])
    h = s["h"].clone()
    cz.cz_block_norm_fwd(h, s["y"], h)
    assert torch.equal(h, out)
    dh, dy = torch.empty_like(out), torch.empty_like(x)
    kw = dict(rstd_post=r[0], rstd_pre=r[1])
    cz.cz_block_norm_bwd(out, s["y"], s["dx"], s["dh"], dh, dy, **kw)
    g = s["dh"].clone()
    cz.cz_block_norm_bwd(out, s["y"], s["dx"], g, g, dy, **kw)
    assert torch.equal(g, dh)


def test_no_rows():
    e = torch.empty(0, 64, device="cuda")
    cz.cz_block_norm_fwd(e, e.bfloat16(), e, x=e.bfloat16())
    w = torch.ones(64, device="cuda")
    ws = torch.zeros(cz.cz_block_norm_workspace(0, 64), dtype=torch.uint8, device="cuda")
    cz.cz_block_norm_bwd(e, e, e, e, e, e, rstd_post=torch.empty(0, device="cuda"), rstd_pre=torch.empty(0, device="cuda"),
                         dw_post=w, dw_pre=w.clone(), workspace=ws)
    assert bool((w == 0).all())


def test_a_nan_stays_in_its_row():
    s = _inputs(6, 512, "f32", "bf16", None, 0)
    s["y"][2, 100] = float("nan")
    out, x = torch.empty_like(s["h"]), torch.empty_like(s["y"])
    cz.cz_block_norm_fwd(s["h"], s["y"], out, x=x)
    rows = torch.isnan(out).any(1).cpu()
    assert rows.tolist() == [False, False, True, False, False, False]
    assert torch.isnan(x).any(1).cpu().tolist() == rows.tolist()


def test_gradient_against_differences_of_the_definition():
    """A direction through all inputs: the GPU's gradients against the central difference of the fp64 forward (step 1e-6:
    the row of zeros bends over sqrt(eps) = 1e-3, a truncation of 1e-6, so the gradients' own 3e-5 bounds it)."""
    rows, cols = 6, 96
    s = _inputs(rows, cols, "f32", "f32", "token", 0, seed=11)
    out = _backward(s, rows, cols, "silu", True, True, False)
    rng = np.random.default_rng(0)
    names = dict(h="dh", y="dy", gate="dgate", w_post="dw_post", w_pre="dw_pre")
    step = {k: rng.standard_normal(s[k].shape) for k in names}
    ends = []
    for e in (1e-6, -1e-6):
        a = {k: _np(s[k]) + e * step[k] for k in names}
        f = O.norm_fwd(a["h"], a["y"], a["w_post"], a["w_pre"], a["gate"], "silu", H, Y)
        ends.append((f["h"] * _np(s["dh"])).sum() + (f["x"] * _np(s["dx"])).sum())
    slope = sum((_np(out[g]) * step[k]).sum() for k, g in names.items())
    size = sum(np.abs(_np(out[g]) * step[k]).sum() for k, g in names.items())
    assert abs((ends[0] - ends[1]) / 2e-6 - slope) <= 3e-5 * size
