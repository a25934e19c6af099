"""Measured cases of the training-step operators: norms around a block with its gate and residual scale,
8-bit activation checkpoints with the weight gradient taken from them, and token log probabilities with
entropy and top alternatives; forward and backward.

`own = False` computes the plain form (elementary torch operations in 32 bits, rounded once at the end);
`own = True` makes the library's calls on the same state.  `exact` is the definition in 64 bits, written
apart from the plain form.
"""

from __future__ import annotations

import math

import torch

own = False

F32, BF16 = torch.float32, torch.bfloat16
TYPES = {"f32": F32, "bf16": BF16}
BLOCK = 32          # channels that share an exponent in an 8-bit checkpoint
EPS = 1e-6
H_SCALE, Y_SCALE = 1.0, 0.7071067690849304     # residual scales (the second is an fp32 value)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a prompt's handful of tokens at the 1.7B layer's width: latency
        dict(name="norm_fwd_small", op="norm_fwd", rows=16, cols=2048, stream="bf16", gate="none", keep=False, pad=0),
        # a micro-batch of 4 x 4096 tokens at the 32B layers' width, the next block's input also kept in 8 bits
        dict(name="norm_fwd_keep_large", op="norm_fwd", rows=16384, cols=5120, stream="bf16", gate="channel", keep=True,
             pad=0),
        # packed sequences of odd total length, an odd width, an fp32 residual stream and a gate for every token
        dict(name="norm_bwd_odd", op="norm_bwd", rows=4099, cols=2047, stream="f32", gate="token", ckpt=False, pad=0),
        # the backward of the large micro-batch, stream and block output read from their 8-bit checkpoints
        dict(name="norm_bwd_ckpt_large", op="norm_bwd", rows=16384, cols=5120, stream="bf16", gate="channel", ckpt=True,
             pad=0),
        # a short sequence's input kept and read back for recomputation
        dict(name="keep_small", op="keep", rows=33, cols=2048, dtype="f32", pad=0),
        # the widest activation of the 32B layers (input of the down projection)
        dict(name="keep_large", op="keep", rows=16384, cols=25600, dtype="bf16", pad=0),
        # gate projection of the 1.7B layer, one sequence and a token more, into an fp32 gradient buffer
        dict(name="wgrad_layer", op="wgrad", rows=4097, n_out=6144, n_in=2048, out="f32", add=False, pad=0),
        # up projection of the 32B layers, added to the gradient of the micro-batches before
        dict(name="wgrad_large", op="wgrad", rows=8192, n_out=25600, n_in=5120, out="f32", add=True, pad=0),
        # the last tokens of three answers, with twenty alternatives each
        dict(name="logp_fwd_small", op="logp_fwd", rows=3, vocab=131072, dtype="f32", top=20, masked=0, inv_temp=1.0,
             pad=0),
        # a training batch's logits, the vocabulary padded with masked entries, at a temperature
        dict(name="logp_fwd_large", op="logp_fwd", rows=8191, vocab=131072, dtype="bf16", top=8, masked=61,
             inv_temp=1.25, pad=0),
        # gradient for a few tokens
        dict(name="logp_bwd_small", op="logp_bwd", rows=5, vocab=32000, dtype="f32", masked=0, inv_temp=1.0, pad=0),
        # gradient of a training batch: an odd vocabulary in padded rows
        dict(name="logp_bwd_large", op="logp_bwd", rows=8192, vocab=100003, dtype="bf16", masked=0, inv_temp=1.0,
             pad=29),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _pad(rng, n):
    """No padding, rows padded to a multiple of 64 elements, or an odd stride."""
    kind = rng.randrange(3)
    return 0 if kind == 0 else (-n) % 64 + 64 if kind == 1 else 1 + 2 * rng.randrange(4)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "keep", "wgrad", "logp_fwd", "logp_bwd"])
    if op in ("norm_fwd", "norm_bwd", "keep"):
        cols = _log_int(rng, 64, 12288)
        cols = cols if rng.random() < 0.35 else max(64, cols // 32 * 32)
        cols = cols + 32 if cols == 3072 else cols
        rows = _log_int(rng, 1, min(32768, 16384 * 5120 // cols))
        case = dict(op=op, rows=rows, cols=cols, pad=_pad(rng, cols))
        if op == "keep":
            return dict(case, dtype=rng.choice(["f32", "bf16"]))
        case.update(stream=rng.choice(["f32", "bf16"]), gate=rng.choice(["none", "channel", "token"]))
        return dict(case, keep=rng.random() < 0.5) if op == "norm_fwd" else dict(case, ckpt=rng.random() < 0.5)
    if op == "wgrad":
        n_out = _log_int(rng, 32, 16384)
        n_in = _log_int(rng, 32, min(16384, 25600 * 5120 // n_out))
        if rng.random() < 0.65:
            n_out, n_in = max(32, n_out // 32 * 32), max(32, n_in // 32 * 32)
        n_out, n_in = (n + 32 if n == 3072 else n for n in (n_out, n_in))
        rows = _log_int(rng, 1, max(1, min(16384, 8192 * 25600 * 5120 // (n_out * n_in))))
        return dict(op=op, rows=rows, n_out=n_out, n_in=n_in, out=rng.choice(["f32", "bf16"]), add=rng.random() < 0.5,
                    pad=_pad(rng, n_out))
    vocab = _log_int(rng, 1000, 160000)
    rows = _log_int(rng, 1, min(8192, 8191 * 131072 // vocab))
    case = dict(op=op, rows=rows, vocab=vocab, dtype=rng.choice(["f32", "bf16"]), masked=rng.choice([0, 0, 77]),
                inv_temp=rng.choice([1.0, 0.5, 1.25]), pad=_pad(rng, vocab))
    return dict(case, top=rng.choice([0, 1, 5, 8, 20])) if op == "logp_fwd" else case


# ---------------------------------------------------------------- states
def _strided(t, pad):
    """The values of t in rows of cols + pad elements."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _activations(gen, rows, cols, scale):
    """Activations as a trained network has them: tokens of differing size, a few large channels."""
    dev = gen.device
    x = torch.randn(rows, cols, device=dev, generator=gen)
    x *= scale * torch.exp(0.5 * torch.randn(rows, 1, device=dev, generator=gen))
    x *= torch.where(torch.rand(cols, device=dev, generator=gen) < 0.01, 12.0, 1.0)
    return x


def _ckpt_bytes(rows, cols):
    ld_q = -(-cols // BLOCK) * BLOCK
    ld_e = -(-(ld_q // BLOCK) // 16) * 16
    at = -(-rows * ld_q // 128) * 128
    return ld_q, ld_e, at, at + rows * ld_e


def _ckpt_of(x):
    """A checkpoint buffer of x (fp32): int8 rows padded to whole blocks, then one biased exponent a block."""
    rows, cols = x.shape
    ld_q, ld_e, at, n = _ckpt_bytes(rows, cols)
    q, b = _quantised(x)
    buf = torch.zeros(n, dtype=torch.uint8, device=x.device)
    buf[:rows * ld_q].view(rows, ld_q).copy_(q.to(torch.int8).reshape(rows, ld_q).view(torch.uint8))
    buf[at:].view(rows, ld_e)[:, :ld_q // BLOCK].copy_(b.to(torch.uint8))
    return buf


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rand = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    op, rows, pad = case["op"], case["rows"], case["pad"]
    s = dict(case=dict(case))
    empty = lambda r, c, t: torch.empty(r, c + pad, dtype=t, device="cuda")[:, :c]  # noqa: E731
    if op in ("norm_fwd", "norm_bwd"):
        cols, st = case["cols"], TYPES[case["stream"]]
        h = _strided(_activations(gen, rows, cols, 4.0).to(st), pad)
        y = _strided(_activations(gen, rows, cols, 0.5).to(BF16), pad)
        s.update(w_post=1 + 0.1 * rand(cols), w_pre=1 + 0.2 * rand(cols), gate=None)
        if case["gate"] == "channel":
            s["gate"] = rand(cols)
        elif case["gate"] == "token":
            s["gate"] = _strided(rand(rows, cols).to(BF16), pad)
        s.update(h=h, y=y, r_post=torch.empty(rows, device="cuda"), r_pre=torch.empty(rows, device="cuda"))
        if op == "norm_fwd":
            s.update(h_out=empty(rows, cols, st), x=empty(rows, cols, BF16))
            if case["keep"]:
                s.update(ckpt=torch.empty(_ckpt_bytes(rows, cols)[3], dtype=torch.uint8, device="cuda"),
                         x8=empty(rows, cols, BF16))
            return s
        s.update(dx=_strided((1e-3 * rand(rows, cols)).to(BF16), pad), dh_in=_strided((1e-3 * rand(rows, cols)).to(st), pad))
        s["r_post"] = 1 / torch.sqrt(y.float().square().mean(1) + EPS)
        s["r_pre"] = 1 / torch.sqrt(h.float().square().mean(1) + EPS)
        s.update(dh=empty(rows, cols, st), dy=empty(rows, cols, BF16), dw_post=torch.empty(cols, device="cuda"),
                 dw_pre=torch.empty(cols, device="cuda"), dgate=None, h_ckpt=None, y_ckpt=None)
        if s["gate"] is not None:
            s["dgate"] = torch.empty(cols, device="cuda") if case["gate"] == "channel" else empty(rows, cols, BF16)
        if case["ckpt"]:
            s.update(h_ckpt=_ckpt_of(h.float()), y_ckpt=_ckpt_of(y.float()), h=None, y=None)
        # room for the partial sums of the column gradients
        s["workspace"] = torch.zeros(_norm_workspace(cols), dtype=torch.uint8, device="cuda")
        return s
    if op == "keep":
        cols, dt = case["cols"], TYPES[case["dtype"]]
        s.update(x=_strided(_activations(gen, rows, cols, 1.0).to(dt), pad), out=empty(rows, cols, dt),
                 ckpt=torch.empty(_ckpt_bytes(rows, cols)[3], dtype=torch.uint8, device="cuda"))
        return s
    if op == "wgrad":
        n_out, n_in, dt = case["n_out"], case["n_in"], TYPES[case["out"]]
        s["ckpt"] = _ckpt_of(_activations(gen, rows, n_in, 1.0))
        s["dy"] = _strided((1e-3 * rand(rows, n_out)).to(BF16), pad)
        s["out"] = torch.empty(n_out, n_in, dtype=dt, device="cuda")
        s["add"] = (1e-2 * rand(n_out, n_in)).to(dt) if case["add"] else None
        s["workspace"] = torch.zeros(_wgrad_workspace(rows, n_out, n_in), dtype=torch.uint8, device="cuda")
        return s
    vocab, dt = case["vocab"], TYPES[case["dtype"]]
    z = rand(rows, vocab)
    z *= 0.5 + 4 * torch.rand(rows, 1, device="cuda", generator=gen)
    t = torch.randint(0, vocab - case["masked"], (rows,), device="cuda", generator=gen)
    sure = 8.0 * (torch.rand(rows, device="cuda", generator=gen) < 0.5)
    z[torch.arange(rows, device="cuda"), t] += sure
    if case["masked"]:
        z[:, vocab - case["masked"]:] = -math.inf
    s["logits"] = _strided(z.to(dt), pad)
    del z
    t[torch.rand(rows, device="cuda", generator=gen) < 0.05] = -1          # padding tokens
    s["targets"] = t
    vec = lambda: torch.empty(rows, device="cuda")  # noqa: E731
    if op == "logp_fwd":
        k = case["top"]
        s.update(logp=vec(), entropy=vec(), lse=vec(), ids=torch.empty(rows, k, dtype=torch.int64, device="cuda"),
                 top=torch.empty(rows, k, device="cuda"))
        return s
    s["lse"], s["entropy"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    for r in range(0, rows, 1024):
        _, s["entropy"][r:r + 1024], s["lse"][r:r + 1024] = _logp_plain(s["logits"][r:r + 1024], t[r:r + 1024],
                                                                        case["inv_temp"])
    s.update(g_logp=rand(rows) / rows, g_entropy=0.01 * rand(rows) / rows, dlogits=empty(rows, vocab, dt))
    return s


def _norm_workspace(cols):
    return 256 + 4 * 3 * 608 * (-(-cols // 32) * 32)


def _wgrad_workspace(rows, n_out, n_in):
    """The status word, split sums of small products, and an aligned copy of rows whose stride is not."""
    tiles = lambda n: -(-n // 256) * 256  # noqa: E731
    return 256 + 4 * min(16 * tiles(n_out) * tiles(n_in), 152 * 2 * 256 * 256) + 2 * rows * (-(-n_out // 64) * 64) + 1024


# ---------------------------------------------------------------- plain forms (32 bits)
def _quantised(x):
    """Blocks of 32: the smallest power of two that holds the block in +-127, and the rounded values."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    a = x.abs().amax(2)
    m, e = torch.frexp(a)
    e = (torch.where(m <= 0.9921875, e - 7, e - 6)).clamp(min=-126)
    e = torch.where(a > 0, e, torch.full_like(e, -126))
    scale = ((127 - e) << 23).view(F32)
    q = torch.round(x * scale[:, :, None])
    return q, e + 127


def _of_quantised(q, b, cols):
    v = q * ((b.to(torch.int32) << 23).view(F32))[:, :, None]
    return v.view(q.shape[0], -1)[:, :cols]


def _of_ckpt(buf, rows, cols):
    ld_q, ld_e, at, _ = _ckpt_bytes(rows, cols)
    q = buf[:rows * ld_q].view(torch.int8).view(rows, -1, BLOCK).float()
    b = buf[at:].view(rows, ld_e)[:, :ld_q // BLOCK]
    return _of_quantised(q, b, cols)


def _gate_plain(gate):
    """The gate is a sigmoid of its input."""
    return 1.0 if gate is None else torch.sigmoid(gate.float())


def _norm_fwd_plain(s):
    h, y = s["h"].float(), s["y"].float()
    r_post = 1 / torch.sqrt(y.square().mean(1) + EPS)
    n = y * r_post[:, None] * s["w_post"]
    h = H_SCALE * h + Y_SCALE * _gate_plain(s["gate"]) * n
    r_pre = 1 / torch.sqrt(h.square().mean(1) + EPS)
    x = h * r_pre[:, None] * s["w_pre"]
    out = dict(h=h.to(s["h"].dtype), x=x.to(BF16), r_post=r_post, r_pre=r_pre)
    if s["case"]["keep"]:
        out["x8"] = _of_quantised(*_quantised(x), x.shape[1]).to(BF16)
    return out


def _norm_bwd_plain(s):
    c = s["case"]
    rows, cols = c["rows"], c["cols"]
    h = s["h"].float() if s["h"] is not None else _of_ckpt(s["h_ckpt"], rows, cols)
    y = s["y"].float() if s["y"] is not None else _of_ckpt(s["y_ckpt"], rows, cols)
    h = h * s["r_pre"][:, None]
    dx = s["dx"].float()
    g = dx * s["w_pre"]
    d = s["dh_in"].float() + s["r_pre"][:, None] * (g - h * (g * h).mean(1, keepdim=True))
    out = dict(dw_pre=(dx * h).sum(0), dh=(H_SCALE * d).to(s["dh"].dtype))
    del h, g, dx
    y = y * s["r_post"][:, None]
    gate = _gate_plain(s["gate"])
    dn = Y_SCALE * gate * d
    out["dw_post"] = (dn * y).sum(0)
    if s["gate"] is not None:
        dg = Y_SCALE * gate * (1 - gate) * y * s["w_post"] * d
        out["dgate"] = dg.sum(0) if c["gate"] == "channel" else dg.to(BF16)
    g = dn * s["w_post"]
    out["dy"] = (s["r_post"][:, None] * (g - y * (g * y).mean(1, keepdim=True))).to(BF16)
    return out


def _logp_plain(logits, targets, inv_temp):
    z = logits.float() * inv_temp
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    entropy = lse[:, 0] - torch.where(e > 0, e * z, 0.0).sum(1) / total[:, 0]
    logp = torch.where(targets >= 0, z.gather(1, targets.clamp(min=0)[:, None])[:, 0] - lse[:, 0], 0.0)
    return logp, entropy, lse[:, 0]


def _top_plain(logits, lse, k, inv_temp):
    """Largest first, ties to the lowest index: one 64-bit key of (value, index) an entry."""
    z = logits.float() + 0.0
    i = z.view(torch.int32)
    key = torch.where(i < 0, ~(i & 0x7fffffff), i).to(torch.int64) << 32
    key += torch.arange(z.shape[1] - 1, -1, -1, device=z.device)
    ids = z.shape[1] - 1 - (torch.topk(key, k, dim=1).values & 0xffffffff)
    return ids, z.gather(1, ids) * inv_temp - lse[:, None]


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm_fwd":
        return _norm_fwd_plain(s)
    if c["op"] == "norm_bwd":
        return _norm_bwd_plain(s)
    if c["op"] == "keep":
        return dict(out=_of_quantised(*_quantised(s["x"].float()), c["cols"]).to(s["x"].dtype))
    if c["op"] == "wgrad":
        dw = s["dy"].float().T @ _of_ckpt(s["ckpt"], c["rows"], c["n_in"])
        if s["add"] is not None:
            dw += s["add"].float()
        return dict(dw=dw.to(s["out"].dtype))
    if c["op"] == "logp_fwd":
        logp, entropy, lse = _logp_plain(s["logits"], s["targets"], c["inv_temp"])
        out = dict(logp=logp, entropy=entropy, lse=lse)
        if c["top"]:
            out["ids"], out["top"] = _top_plain(s["logits"], lse, c["top"], c["inv_temp"])
        return out
    lp = s["logits"].float() * c["inv_temp"] - s["lse"][:, None]
    p = torch.exp(lp)
    g = torch.where(s["targets"] >= 0, s["g_logp"], 0.0)
    d = torch.where(p > 0, -p * (g[:, None] + s["g_entropy"][:, None] * (lp + s["entropy"][:, None])), 0.0)
    d.scatter_add_(1, s["targets"].clamp(min=0)[:, None], g[:, None])
    return dict(dlogits=(d * c["inv_temp"]).to(s["logits"].dtype))


# ---------------------------------------------------------------- the library's calls
def _run_own(s):
    from zero_sharded_gb300 import cz

    c, stream = s["case"], torch.cuda.current_stream()
    if c["op"] == "norm_fwd":
        cz.cz_block_norm_fwd(s["h"], s["y"], s["h_out"], x=s["x"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"],
                             gate_act="sigmoid", h_scale=H_SCALE, y_scale=Y_SCALE, eps=EPS, rstd_post=s["r_post"],
                             rstd_pre=s["r_pre"], x_ckpt=s.get("ckpt"), stream=stream)
        out = dict(h=s["h_out"], x=s["x"], r_post=s["r_post"], r_pre=s["r_pre"])
        if c["keep"]:
            cz.cz_act_decode(s["ckpt"], s["x8"], stream=stream)
            out["x8"] = s["x8"]
        return out
    if c["op"] == "norm_bwd":
        cz.cz_block_norm_bwd(s["h"], s["y"], s["dx"], s["dh_in"], s["dh"], s["dy"], w_post=s["w_post"], w_pre=s["w_pre"],
                             gate=s["gate"], gate_act="sigmoid", h_scale=H_SCALE, y_scale=Y_SCALE, rstd_post=s["r_post"],
                             rstd_pre=s["r_pre"], h_ckpt=s["h_ckpt"], y_ckpt=s["y_ckpt"], dw_post=s["dw_post"],
                             dw_pre=s["dw_pre"], dgate=s["dgate"], workspace=s["workspace"], stream=stream)
        out = dict(dh=s["dh"], dy=s["dy"], dw_post=s["dw_post"], dw_pre=s["dw_pre"])
        if s["dgate"] is not None:
            out["dgate"] = s["dgate"]
        return out
    if c["op"] == "keep":
        cz.cz_act_encode(s["x"], s["ckpt"], stream=stream)
        cz.cz_act_decode(s["ckpt"], s["out"], stream=stream)
        return dict(out=s["out"])
    if c["op"] == "wgrad":
        cz.cz_act_wgrad(s["dy"], s["ckpt"], s["out"], add=s["add"], workspace=s["workspace"], stream=stream)
        return dict(dw=s["out"])
    if c["op"] == "logp_fwd":
        cz.cz_token_logp_fwd(s["logits"], s["targets"], s["logp"], entropy=s["entropy"], lse=s["lse"], top_ids=s["ids"],
                             top_logp=s["top"], inv_temp=c["inv_temp"], stream=stream)
        out = dict(logp=s["logp"], entropy=s["entropy"], lse=s["lse"])
        if c["top"]:
            out.update(ids=s["ids"], top=s["top"])
        return out
    cz.cz_token_logp_bwd(s["logits"], s["targets"], s["lse"], s["dlogits"], entropy=s["entropy"], g_logp=s["g_logp"],
                         g_entropy=s["g_entropy"], inv_temp=c["inv_temp"], stream=stream)
    return dict(dlogits=s["dlogits"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- work of one pass
def work(case):
    op, rows = case["op"], case["rows"]
    size = lambda t: {"f32": 4, "bf16": 2}[t]  # noqa: E731
    kept = 1 + 1 / BLOCK
    if op in ("norm_fwd", "norm_bwd"):
        n, st = rows * case["cols"], size(case["stream"])
        token = 2 if case["gate"] == "token" else 0
        vectors = 4 * case["cols"] * (3 if case["gate"] == "channel" else 2)
        if op == "norm_fwd":       # h, y, gate -> h', x (and the checkpoint, read back as values)
            per = 2 * st + 2 + 2 + token + (2 * kept + 2 if case["keep"] else 0)
            return dict(bytes=n * per + vectors + 8 * rows, flops=14 * n)
        read = 2 * kept if case["ckpt"] else st + 2      # h', y; then dx, dh' -> dh, dy (and the gate's)
        return dict(bytes=n * (read + 2 + st + st + 2 + 2 * token) + 2 * vectors + 8 * rows, flops=30 * n)
    if op == "keep":               # values -> checkpoint -> values
        n = rows * case["cols"]
        return dict(bytes=n * (2 * size(case["dtype"]) + 2 * kept), flops=4 * n)
    if op == "wgrad":
        n, k = case["n_out"], case["n_in"]
        return dict(bytes=rows * (2 * n + kept * k) + n * k * size(case["out"]) * (2 if case["add"] else 1),
                    flops=2 * rows * n * k)
    n = rows * case["vocab"]
    if op == "logp_fwd":
        return dict(bytes=n * size(case["dtype"]) + rows * (20 + 12 * case["top"]), flops=5 * n)
    return dict(bytes=2 * n * size(case["dtype"]) + 24 * rows, flops=8 * n)


# ---------------------------------------------------------------- the definitions in 64 bits
def _two_to(e):
    """2^e in 64 bits for whole e, without rounding."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_blocks(x):
    """x^ of a 64-bit x: q 2^E with the smallest E such that every |x| of the block is at most 127 * 2^E."""
    rows, cols = x.shape
    n = -(-cols // BLOCK) * BLOCK
    wide = x.new_zeros(rows, n)
    wide[:, :cols] = x
    wide = wide.view(rows, n // BLOCK, BLOCK)
    top = wide.abs().max(dim=2, keepdim=True).values
    e = torch.floor(torch.log2(top.clamp(min=1e-300))) - 7       # one or two too small; exact comparisons mend it
    e = torch.where(top > 127 * _two_to(e), e + 1, e)
    e = torch.where(top > 127 * _two_to(e), e + 1, e).clamp(min=-126)
    unit = _two_to(e)
    return (torch.round(wide / unit) * unit).view(rows, n)[:, :cols]


def _exact_decode(buf, rows, cols):
    ld_q, ld_e, at, _ = _ckpt_bytes(rows, cols)
    q = buf[:rows * ld_q].view(torch.int8).view(rows, ld_q).double()
    e = buf[at:at + rows * ld_e].view(rows, ld_e).double()[:, :ld_q // BLOCK] - 127
    return (q * _two_to(e).repeat_interleave(BLOCK, dim=1))[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    s.pop("workspace", None)
    f = lambda name: s[name].double()  # noqa: E731
    if op in ("norm_fwd", "norm_bwd"):
        a, b = 1.0, float(torch.tensor(Y_SCALE, dtype=F32))
        act = 1.0 if s["gate"] is None else 1 / (1 + torch.exp(-f("gate")))
    if op == "norm_fwd":
        y, h = f("y"), f("h")
        sq_y = (y * y).sum(1) / y.shape[1]
        h = a * h + b * act * (y / torch.sqrt(sq_y + EPS)[:, None] * f("w_post"))
        sq_h = (h * h).sum(1) / h.shape[1]
        x = h / torch.sqrt(sq_h + EPS)[:, None] * f("w_pre")
        out = dict(h=h, x=x, r_post=(sq_y + EPS) ** -0.5, r_pre=(sq_h + EPS) ** -0.5)
        if case["keep"]:
            out["x8"] = _exact_blocks(x)
        return out
    if op == "norm_bwd":
        rows, cols = case["rows"], case["cols"]
        y = _exact_decode(s["y_ckpt"], rows, cols) if case["ckpt"] else f("y")
        h = _exact_decode(s["h_ckpt"], rows, cols) if case["ckpt"] else f("h")
        r_h, r_y = f("r_pre")[:, None], f("r_post")[:, None]
        w_h, w_y, dx = f("w_pre"), f("w_post"), f("dx")
        # d of x_j = h_j r w_j with dr/dh_i = -r^3 h_i / n
        pull = (dx * w_h * h).sum(1, keepdim=True)
        d = f("dh_in") + r_h * w_h * dx - r_h ** 3 * h * pull / cols
        out = dict(dh=a * d, dw_pre=(dx * h * r_h).sum(0))
        dn = b * act * d
        out["dw_post"] = (dn * y * r_y).sum(0)
        pull = (dn * w_y * y).sum(1, keepdim=True)
        out["dy"] = r_y * w_y * dn - r_y ** 3 * y * pull / cols
        if s["gate"] is not None:
            dg = b * d * y * r_y * w_y * act * (1 - act)
            out["dgate"] = dg.sum(0) if case["gate"] == "channel" else dg
        return out
    if op == "keep":
        return dict(out=_exact_blocks(f("x")))
    if op == "wgrad":
        dw = torch.matmul(f("dy").t().contiguous(), _exact_decode(s["ckpt"], case["rows"], case["n_in"]))
        return dict(dw=dw if s["add"] is None else dw + f("add"))
    parts = []
    for r in range(0, case["rows"], 512):          # rows at a time: 64-bit rows of a large vocabulary are big
        z = s["logits"][r:r + 512].double() * case["inv_temp"]
        t = s["targets"][r:r + 512]
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        plogp = torch.where(torch.isinf(lp), 0.0, torch.exp(lp) * lp)
        entropy = -plogp.sum(1)
        at = torch.arange(len(t), device=t.device)
        if op == "logp_fwd":
            logp = torch.where(t < 0, 0.0, lp[at, t.clamp(min=0)])
            part = dict(logp=logp, entropy=entropy, lse=lse)
            if case["top"]:
                v, i = torch.sort(lp, dim=1, descending=True, stable=True)
                part.update(ids=i[:, :case["top"]].clone(), top=v[:, :case["top"]].clone())
        else:
            p = torch.exp(lp)
            g = torch.where(t < 0, 0.0, f("g_logp")[r:r + 512])
            hot = torch.zeros_like(p)
            hot[at, t.clamp(min=0)] = 1.0
            curve = torch.where(p > 0, p * (lp + entropy[:, None]), 0.0)
            part = dict(dlogits=(case["inv_temp"] * (g[:, None] * (hot - p) - f("g_entropy")[r:r + 512, None] * curve)).float())
        parts.append(part)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
