"""Pins of the fp64 oracle of the training-step operators (CPU): hand-worked values, bounds, and every gradient against
central differences of its forward (step 1e-5 in fp64: truncation ~1e-10, rounding ~1e-11 of values of order 1, so 1e-7
of the gradient's scale)."""

import numpy as np
import pytest

from oracle import train_ops as O


def test_checkpoint_hand_worked():
    x = np.zeros((1, 64))
    x[0, :4] = [127.0, -126.5, 0.5, 1.5]       # scale 1; ties to even
    x[0, 32:35] = [127.5, 1.0, -3.0]           # above 127: scale 2
    q, b = O.ckpt_encode(x)
    assert b.tolist() == [[127, 128]]
    assert q[0, :4].tolist() == [127, -126, 0, 2]
    assert q[0, 32:35].tolist() == [64, 0, -2]                        # 63.75, 0.5 and -1.5 (to even)
    assert O.ckpt_decode(q, b, 64)[0, 32:35].tolist() == [128.0, 0.0, -4.0]


def test_checkpoint_bounds_and_corners():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((40, 75)) * 10.0 ** rng.integers(-30, 30, (40, 1))).astype(np.float32).astype(np.float64)
    x[3] = 0
    x[4, 7] = np.inf
    x[5, 70] = np.nan
    x[6, 0] = np.finfo(np.float32).max
    q, b = O.ckpt_encode(x)
    xh = O.ckpt_decode(q, b, 75)
    assert np.isnan(xh[4, :32]).all() and not np.isnan(xh[4, 32:]).any()
    assert np.isnan(xh[5, 64:]).all() and (xh[3] == 0).all()
    fine = np.isfinite(xh)
    assert np.isfinite(xh.astype(np.float32)[fine]).all()
    for r in range(40):
        for k in range(3):
            s = slice(32 * k, min(75, 32 * k + 32))
            if fine[r, s].all() and r != 6:
                a = np.abs(x[r, s]).max()
                assert np.abs(xh[r, s] - x[r, s]).max() <= max(a / 127, 2.0 ** -127)
    # the values survive bf16 unchanged: 8 significant bits hold 7 bits and a sign
    v = xh[fine].astype(np.float32)
    assert np.array_equal((v.view(np.uint32) & 0xFFFF), np.zeros(v.size, np.uint32))


@pytest.mark.parametrize("post,pre,gate,act", [(True, True, None, "identity"), (True, True, "channel", "sigmoid"),
                                               (True, True, "token", "silu"), (False, True, "token", "identity"),
                                               (True, False, "channel", "silu")])
def test_norm_gradients_against_differences(post, pre, gate, act):
    rng = np.random.default_rng(1)
    rows, cols = 3, 5
    h, y = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    wp, wx = rng.standard_normal(cols), rng.standard_normal(cols)
    g = None if gate is None else rng.standard_normal(cols if gate == "channel" else (rows, cols))
    dx, dh = rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    kw = dict(act=act, h_scale=0.9, y_scale=0.7, post=post, pre=pre)

    def loss(h, y, wp, wx, g):
        f = O.norm_fwd(h, y, wp, wx, g, **kw)
        return (f["h"] * dh).sum() + ((f["x"] * dx).sum() if pre else 0.0)

    f = O.norm_fwd(h, y, wp, wx, g, **kw)
    got = O.norm_bwd(f["h"], y, dx, dh, f["r_post"], f["r_pre"], wp, wx, g, **kw)
    args = dict(h=h, y=y, wp=wp, wx=wx, g=g)
    names = dict(h="dh", y="dy", **({"wp": "dw_post"} if post else {}), **({"wx": "dw_pre"} if pre else {}),
                 **({"g": "dgate"} if gate else {}))
    for name, key in names.items():
        want = got[key].sum(0) if name == "g" and gate == "channel" else got[key]
        for i in np.ndindex(args[name].shape):
            ends = []
            for e in (1e-5, -1e-5):
                moved = args[name].copy()
                moved[i] += e
                ends.append(loss(**{**args, name: moved}))
            assert abs((ends[0] - ends[1]) / 2e-5 - want[i]) < 1e-7 * (1 + np.abs(want).max()), (name, i)


def test_logp_values():
    x = np.log(np.array([[0.5, 0.25, 0.125, 0.125], [1, 1, 1, 1]]))
    f = O.logp_fwd(x, [1, -1], 1.0, 3)
    assert np.allclose(f["logp"], [np.log(0.25), 0]) and np.allclose(f["lse"], [0, np.log(4)])
    assert np.allclose(f["entropy"], [1.75 * np.log(2), np.log(4)])
    assert f["ids"].tolist() == [[0, 1, 2], [0, 1, 2]]                # ties to the lowest index
    e = O.logp_fwd(np.full((1, 3), -np.inf), [2], 2.0, 2)
    assert e["lse"][0] == e["logp"][0] == -np.inf and e["entropy"][0] == 0 and e["ids"].tolist() == [[0, 1]]


def test_logp_gradients_against_differences():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 6)) * 2
    t, gl, ge = np.array([4, -1, 0]), rng.standard_normal(3), rng.standard_normal(3)
    d = O.logp_bwd(x, t, gl, ge, 1.3)
    for i in np.ndindex(x.shape):
        ends = []
        for e in (1e-5, -1e-5):
            z = x.copy()
            z[i] += e
            f = O.logp_fwd(z, t, 1.3)
            ends.append((f["logp"] * gl).sum() + (f["entropy"] * ge).sum())
        assert abs((ends[0] - ends[1]) / 2e-5 - d[i]) < 1e-7 * (1 + np.abs(d).max())
    x[0, 2] = -np.inf                                                  # a masked entry takes no gradient
    assert O.logp_bwd(x, t, gl, ge, 1.3)[0, 2] == 0
