"""Refusals of the training-step operators (CPU): invalid arguments are turned down on the host before any GPU work."""

import ctypes

import pytest
import torch

from oracle import train_ops as O
from zero_sharded_gb300 import cz

BF, F = torch.bfloat16, torch.float32


def _refused(call, *args, status=cz.CZ_ERR_INVALID, **kw):
    with pytest.raises(cz.CzError) as e:
        call(*args, **kw)
    assert e.value.status == status, e.value


def test_checkpoint_sizes_and_refusals():
    for rows, cols in ((0, 5), (1, 1), (7, 33), (33, 2048), (5, 513)):
        assert cz.cz_act_size(rows, cols) == O.ckpt_layout(rows, cols)[3]
    _refused(cz.cz_act_size, -1, 4)
    _refused(cz.cz_act_size, 4, 0)
    x, ck = torch.zeros(4, 64), torch.zeros(cz.cz_act_size(4, 64) + 16, dtype=torch.uint8)
    _refused(cz.cz_act_encode, x.double(), ck)
    _refused(cz.cz_act_encode, x.t(), ck)
    _refused(cz.cz_act_encode, x, None)
    _refused(cz.cz_act_encode, x, ck[:100], status=cz.CZ_ERR_NOMEM)
    _refused(cz.cz_act_decode, ck[1 + (-ck.data_ptr()) % 16:], x)                      # buffer not 16-byte aligned
    lib = cz.load()
    assert lib.cz_act_encode(x.data_ptr(), cz.CZ_F32, 63, 4, 64, ck.data_ptr(), None) == cz.CZ_ERR_INVALID   # stride below the row
    assert lib.cz_act_encode(x.data_ptr() + 2, cz.CZ_F32, 64, 3, 64, ck.data_ptr(), None) == cz.CZ_ERR_INVALID
    assert lib.cz_act_encode(x.data_ptr(), 7, 64, 4, 64, ck.data_ptr(), None) == cz.CZ_ERR_INVALID
    assert lib.cz_act_size(4, 4, None) == cz.CZ_ERR_INVALID


def test_wgrad_refusals():
    dy, ck, out = torch.zeros(8, 32, dtype=BF), torch.zeros(cz.cz_act_size(8, 64), dtype=torch.uint8), torch.zeros(32, 64)
    ws = torch.zeros(cz.cz_act_wgrad_workspace(dy, 64) + 512, dtype=torch.uint8)
    ws = ws[(-ws.data_ptr()) % 256:]
    _refused(cz.cz_act_wgrad, dy.float(), ck, out, workspace=ws)
    _refused(cz.cz_act_wgrad, dy, ck, out[:31], workspace=ws)
    _refused(cz.cz_act_wgrad, dy, ck, out.t().contiguous().t(), workspace=ws)
    _refused(cz.cz_act_wgrad, dy, ck, out, add=out.bfloat16(), workspace=ws)
    _refused(cz.cz_act_wgrad, dy, ck[:64], out, workspace=ws, status=cz.CZ_ERR_NOMEM)
    _refused(cz.cz_act_wgrad, dy, ck, out, status=cz.CZ_ERR_NOMEM)
    _refused(cz.cz_act_wgrad, dy, ck, out, workspace=ws[:64], status=cz.CZ_ERR_NOMEM)
    _refused(cz.cz_act_wgrad, dy, ck, out, workspace=ws[8:])
    _refused(cz.cz_act_wgrad_workspace, dy, 0)


def test_block_norm_refusals():
    h, y, r, w = torch.zeros(4, 64), torch.zeros(4, 64, dtype=BF), torch.zeros(4), torch.ones(64)
    _refused(cz.cz_block_norm_fwd, h, y[:, :32], h)
    _refused(cz.cz_block_norm_fwd, h.double(), y, h)
    _refused(cz.cz_block_norm_fwd, h, y, torch.zeros(4, 64, dtype=BF))
    _refused(cz.cz_block_norm_fwd, h, y, h, w_post=w[:63])
    _refused(cz.cz_block_norm_fwd, h, y, h, w_pre=w.double())
    _refused(cz.cz_block_norm_fwd, h, y, h, gate=w, gate_act="tanh")
    _refused(cz.cz_block_norm_fwd, h, y, h, gate=h)                                    # a token gate has the type of y
    _refused(cz.cz_block_norm_fwd, h, y, h, eps=-1.0)
    _refused(cz.cz_block_norm_fwd, h, y, h, y_scale=float("inf"))
    _refused(cz.cz_block_norm_fwd, h, y, h, x=torch.zeros_like(y), pre_norm=False)
    _refused(cz.cz_block_norm_fwd, h, y, h[:, :].flatten()[:0].view(0, 64))
    wide = torch.zeros(2, cz.CZ_NORM_MAX_COLS + 1)
    _refused(cz.cz_block_norm_fwd, wide, wide.bfloat16(), wide)
    big = torch.zeros(5, 64)
    _refused(cz.cz_block_norm_fwd, big[:4], y, big[1:])                                # overlaps its input by a row
    dh, dy, dx = torch.zeros_like(h), torch.zeros_like(y), torch.zeros_like(y)
    kw = dict(rstd_post=r, rstd_pre=r)
    _refused(cz.cz_block_norm_bwd, h, y, dx, None, dh, dy, rstd_post=r)
    _refused(cz.cz_block_norm_bwd, h, y, None, None, dh, dy, **kw)
    _refused(cz.cz_block_norm_bwd, None, y, dx, None, dh, dy, **kw)
    _refused(cz.cz_block_norm_bwd, h, None, dx, None, dh, dy, **kw)
    _refused(cz.cz_block_norm_bwd, h, y, dx, None, h, dy, **kw)                        # an output over an input it still reads
    _refused(cz.cz_block_norm_bwd, h, y, dx, None, dh, dy, dgate=w, **kw)
    _refused(cz.cz_block_norm_bwd, h, y, dx, None, dh, dy, dw_pre=w, status=cz.CZ_ERR_NOMEM, **kw)
    _refused(cz.cz_block_norm_bwd, h, y, dx, None, dh, dy, dw_pre=w, workspace=torch.zeros(8), status=cz.CZ_ERR_NOMEM, **kw)
    _refused(cz.cz_block_norm_bwd, None, None, None, None, None, None)
    _refused(cz.cz_block_norm_workspace, 4, 0)
    lib = cz.load()
    assert lib.cz_block_norm_fwd(None, None) == cz.CZ_ERR_INVALID
    a = cz.cz_norm_args_default()
    assert (a.post_norm, a.pre_norm, a.gate_kind, a.h_scale, a.y_scale) == (1, 1, 0, 1.0, 1.0)
    a.rows, a.cols, a.h, a.y, a.ld_h, a.ld_y, a.gate_kind = 4, 64, h.data_ptr(), y.data_ptr(), 64, 64, 3
    assert lib.cz_block_norm_fwd(ctypes.byref(a), None) == cz.CZ_ERR_INVALID


def test_token_logp_refusals():
    x, t, v = torch.zeros(4, 100), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    ids, top = torch.zeros(4, 33, dtype=torch.int64), torch.zeros(4, 33)
    _refused(cz.cz_token_logp_fwd, x.half(), t, v)
    _refused(cz.cz_token_logp_fwd, x, t.int(), v)
    _refused(cz.cz_token_logp_fwd, x, t[:3], v)
    _refused(cz.cz_token_logp_fwd, x, t, v.double())
    _refused(cz.cz_token_logp_fwd, x, t, None)
    _refused(cz.cz_token_logp_fwd, x, t, v, inv_temp=0.0)
    _refused(cz.cz_token_logp_fwd, x, t, v, inv_temp=float("nan"))
    _refused(cz.cz_token_logp_fwd, x, t, v, top_ids=ids, top_logp=top)                 # more than CZ_LOGP_MAX_TOP
    _refused(cz.cz_token_logp_fwd, x[:, :8], t, v, top_ids=ids[:, :9].contiguous(), top_logp=top[:, :9].contiguous())
    _refused(cz.cz_token_logp_fwd, x, t, v, top_ids=ids)
    _refused(cz.cz_token_logp_bwd, x, t, v, x[:, :99])
    _refused(cz.cz_token_logp_bwd, x, t, None, torch.zeros_like(x))
    _refused(cz.cz_token_logp_bwd, x, t, v, x.bfloat16())
    _refused(cz.cz_token_logp_bwd, x, t, v, torch.zeros_like(x), g_entropy=v)          # without the entropy
    big = torch.zeros(5, 100)
    _refused(cz.cz_token_logp_bwd, big[:4], t, v, big[1:])


def test_valid_arguments_without_a_device_are_unsupported_or_run():
    """On a machine without an sm_103 device a valid call says so; it does not fall back."""
    if torch.cuda.is_available():
        pytest.skip("has a GPU")
    x, ck = torch.zeros(4, 64), torch.zeros(cz.cz_act_size(4, 64), dtype=torch.uint8)
    with pytest.raises(cz.CzError) as e:
        cz.cz_act_encode(x, ck)
    assert e.value.status in (cz.CZ_ERR_UNSUPPORTED, cz.CZ_ERR_CUDA)


def test_norm_arguments_as_bytes_match_the_structure():
    """The binding packs cz_norm_args in one go: every field lands where the structure has it."""
    names = [n for n, _ in cz.cz_norm_args._fields_]
    packed = cz._NORM_ARGS.pack(*range(1, len(names) + 1))
    a = cz.cz_norm_args.from_buffer_copy(packed)
    assert len(packed) == ctypes.sizeof(cz.cz_norm_args)
    assert [int(getattr(a, n)) for n in names] == list(range(1, len(names) + 1))
