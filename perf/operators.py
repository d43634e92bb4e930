"""Measured work of the training operators around the block-sparse attention: the attention's
backward pass (on given block lists, as a whole call, and as a training step) and the RMS norm in
front of it with its gradient.

Where ``own`` is true, ``run`` makes the library's calls; otherwise it computes the same in elementary
torch operations in fp32.  ``exact`` states the definitions once more in 64 bits.
"""
import math

import torch

own = False

BF, F32 = torch.bfloat16, torch.float32
CUBE = (4, 4, 8)
MOST = 12 * 32760 * 32760 * 0.24 * 128  # head rows x kept keys x d of the largest listed case


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------
def listed():
    return [
        # the smallest call: two heads of a 4x8x8 grid in blocks of 64, where launches are all there is
        dict(name="lists 2x256 d64", op="lists", B=1, H=2, F=4, Hl=8, Wl=8, d=64, block=64, keep=0.5, empty=0),
        # a ragged grid with lists of every length, some query blocks keeping nothing (pruned regions)
        dict(name="lists 6x7007 d64", op="lists", B=2, H=3, F=11, Hl=13, Wl=49, d=64, block=128, keep=0.3, empty=3),
        # block 64 at head dimension 128: finer masks on an ordinary grid
        dict(name="lists 4x8190 b64", op="lists", B=1, H=4, F=21, Hl=15, Wl=26, d=128, block=64, keep=0.2, empty=0),
        # the Wan2.1-1.3B-shaped grid at the kept fraction of the default workload, the whole call
        dict(name="call 12x32760", op="call", B=1, H=12, F=21, Hl=30, Wl=52, d=128, block=128, kinds="half", w_s=2, w_t=140,
             topk=0),
        # local cubes and top-k cubes, whose key blocks are kept by very different numbers of query blocks
        dict(name="call cubes 6x14040", op="call", B=1, H=6, F=9, Hl=30, Wl=52, d=128, block=128, kinds="cube", w_s=0, w_t=0,
             topk=16),
        # a training step on a short clip: forward with its log-sum-exp, then the gradients
        dict(name="step 8x7800", op="step", B=1, H=8, F=5, Hl=30, Wl=52, d=128, block=128, kinds="half", w_s=1, w_t=200, topk=0),
        # Q's norm per head, from the projection's [B, N, H, d] to the attention's [B, H, N, d]
        dict(name="norm heads 12x32760", op="norm", B=1, H=12, N=32760, d=128, dtype="bf16", strided=True, residual=False, block=0),
        # the same rows straight to e4m3 codes with one scale per 128-row block, as the FP8 attention takes them
        dict(name="norm e4m3 blocks", op="norm", B=1, H=12, N=32760, d=128, dtype="bf16", strided=True, residual=False, block=128),
        # the hidden width with the residual's addition and a scale per row, for an 8-bit projection
        dict(name="norm residual e4m3", op="norm", B=1, H=1, N=32760, d=1536, dtype="bf16", strided=False, residual=True, block=1),
        # one ragged width in fp32, few rows
        dict(name="norm 77x1000 f32", op="norm", B=1, H=1, N=77, d=1000, dtype="f32", strided=False, residual=True, block=0),
        # gradient of the hidden-width norm with the residual stream's own gradient joining
        dict(name="norm bwd 32760x1536", op="norm_bwd", B=1, H=1, N=32760, d=1536, dtype="bf16", strided=False, residual=True),
        # gradient of Q's per-head norm: short rows, one weight shared by all heads
        dict(name="norm bwd heads", op="norm_bwd", B=1, H=12, N=32760, d=128, dtype="bf16", strided=True, residual=False),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_attention(rng, op):
    while True:
        d, block = rng.choice((64, 128)), rng.choice((64, 128))
        c = dict(op=op, B=rng.choice((1, 1, 2)), H=_logint(rng, 1, 12), F=_logint(rng, 1, 21), Hl=_logint(rng, 1, 30),
                 Wl=_logint(rng, 1, 52), d=d, block=block)
        n = c["F"] * c["Hl"] * c["Wl"]
        if op == "lists":
            c.update(keep=round(rng.uniform(0.05, 0.9), 3), empty=rng.choice((0, 0, 5)))
            kept = c["keep"] + block / n
        else:
            kinds = rng.choice(("half", "spatial", "temporal") + (("cube",) if block == 128 else ()))
            c.update(kinds=kinds, w_s=rng.randint(0, 3), w_t=_logint(rng, 1, 300), topk=rng.randint(0, 16) if kinds == "cube" else 0)
            kept = float(_keep(c).float().mean()) if kinds != "cube" else 1.0
        # the plain form gathers every list to the longest one's length
        if c["B"] * c["H"] * n * n * kept * d <= 0.5 * MOST and n >= 64:
            return c


def draw(rng):
    op = rng.choice(("lists", "call", "step", "norm", "norm_bwd"))
    if op not in ("norm", "norm_bwd"):
        return _draw_attention(rng, op)
    per_head = rng.random() < 0.5
    d = rng.choice((64, 128)) if per_head else rng.choice((_logint(rng, 8, 8192), 8 * _logint(rng, 1, 1024)))
    heads = rng.randint(1, 24) if per_head else 1
    n = _logint(rng, 1, min(32760, 32760 * 1536 // (d * heads)))
    c = dict(op=op, B=1, H=heads, N=n, d=d, dtype=rng.choice(("bf16", "bf16", "f32")), strided=per_head and rng.random() < 0.5,
             residual=rng.random() < 0.5)
    if op == "norm":
        c["block"] = rng.choice((0, 1, 64, 128)) if per_head else rng.choice((0, 1))
    return c


# ------------------------------------------------------------------------------------------
# layouts and masks
# ------------------------------------------------------------------------------------------
def _kinds(c):
    """0 spatial, 1 temporal, 2 cube, for each of the B*H heads."""
    one = {"spatial": [0], "temporal": [1], "cube": [2], "half": [0, 1]}[c["kinds"]]
    return [one[h % len(one)] for h in range(c["H"])] * c["B"]


def _tokens(c, kind):
    """Natural token of every slot of a head's layout, -1 where a slot holds none."""
    F, Hl, Wl = c["F"], c["Hl"], c["Wl"]
    t = torch.arange(F * Hl * Wl).view(F, Hl, Wl)
    if kind == 0:
        return t.reshape(-1)
    if kind == 1:
        return t.view(F, Hl * Wl).t().reshape(-1)
    cf, ch, cw = CUBE
    nf, nh, nw = -(-F // cf), -(-Hl // ch), -(-Wl // cw)
    p = torch.full((nf * cf, nh * ch, nw * cw), -1)
    p[:F, :Hl, :Wl] = t
    return p.view(nf, cf, nh, ch, nw, cw).permute(0, 2, 4, 1, 3, 5).reshape(-1)


def _pattern(c, kind):
    """Block pairs a spatial or temporal head keeps: their frame (position) intervals are near enough."""
    n, b = c["F"] * c["Hl"] * c["Wl"], c["block"]
    g, w = (c["Hl"] * c["Wl"], c["w_s"]) if kind == 0 else (c["F"], c["w_t"])
    i = torch.arange(-(-n // b))
    first, last = i * b // g, (torch.clamp((i + 1) * b, max=n) - 1) // g
    return (first[None, :] <= last[:, None] + w) & (last[None, :] >= first[:, None] - w)


def _cubes(c, q, k):
    """Own cube and the topk cubes of the pooled scores, per head; q, k [BH, C, 128, d] in the cube layout."""
    n = (_tokens(c, 2) >= 0).view(-1, 128).sum(1).double().to(q.device)
    s = (q.double().sum(2) / n[:, None]) @ (k.double().sum(2) / n[:, None]).transpose(1, 2)
    keep = torch.zeros_like(s, dtype=torch.bool)
    if c["topk"]:
        keep.scatter_(2, s.topk(min(c["topk"], s.shape[2]), dim=2).indices, True)
    return keep | torch.eye(s.shape[1], dtype=torch.bool, device=s.device)


def _keep(c):
    """Kept block pairs of the pattern heads, [B*H, nb, nb] on the CPU."""
    both = {k: _pattern(c, k) for k in set(_kinds(c))}
    return torch.stack([both[k] for k in _kinds(c)])


def _lists(keep):
    """Ascending key blocks of every query block, padded to the longest list, and their numbers."""
    cnt = keep.sum(2)
    most = max(1, int(cnt.max()))
    return (~keep).to(torch.uint8).argsort(dim=2, stable=True)[:, :, :most], cnt


# ------------------------------------------------------------------------------------------
# the plain forms
# ------------------------------------------------------------------------------------------
def _blocks(x, tok, block):
    """[BH, N, ...] rows in each head's layout, in blocks and in 32 bits; empty slots are zero."""
    pad = -tok.shape[1] % block
    tok = torch.nn.functional.pad(tok, (0, pad), value=-1)
    live = (tok >= 0).view(*tok.shape, *[1] * (x.dim() - 2))
    rows = x[torch.arange(x.shape[0], device=x.device)[:, None], tok.clamp(min=0)].float() * live
    return rows.view(x.shape[0], -1, block, *x.shape[2:]), (tok >= 0).view(x.shape[0], -1, block)


def _natural(x, tok, n):
    """Blocks of a layout back to [BH, n, ...] in natural order."""
    x = x.flatten(1, 2)[:, :tok.shape[1]]
    out = torch.zeros(x.shape[0], n + 1, *x.shape[2:], dtype=x.dtype, device=x.device)
    out[torch.arange(x.shape[0], device=x.device)[:, None], torch.where(tok < 0, n, tok)] = x
    return out[:, :n]


def _gathered(x, idx):
    """The listed blocks of every query block, [BH, nb, listed * block, ...]."""
    g = x[torch.arange(x.shape[0], device=x.device)[:, None, None], idx]
    return g.flatten(2, 3)


def _scores(c, qb, kb, live, idx, cnt):
    s = torch.matmul(qb, _gathered(kb, idx).transpose(2, 3)).mul_(1 / math.sqrt(c["d"]))
    ok = _gathered(live, idx) & (torch.arange(idx.shape[2], device=idx.device).repeat_interleave(c["block"]) < cnt[..., None])
    return s.masked_fill_(~ok[:, :, None, :], -math.inf)


def _plain_forward(c, q, k, v, tok, keep):
    qb, live = _blocks(q, tok, c["block"])
    kb, vb = _blocks(k, tok, c["block"])[0], _blocks(v, tok, c["block"])[0]
    idx, cnt = _lists(keep(qb, kb))
    s = _scores(c, qb, kb, live, idx, cnt)
    m = s.amax(3, keepdim=True)
    p = s.sub_(m.masked_fill(m.isinf(), 0.0)).exp_()
    total = p.sum(3, keepdim=True)
    o = torch.matmul(p, _gathered(vb, idx)) / total.clamp(min=1e-38)
    n = q.shape[1]
    return _natural(o, tok, n), _natural((m + total.log())[..., 0], tok, n)


def _plain_backward(c, q, k, v, o, lse, do, tok, keep):
    block, n = c["block"], q.shape[1]
    qb, live = _blocks(q, tok, block)
    kb, vb, dob = (_blocks(x, tok, block)[0] for x in (k, v, do))
    lseb = _blocks(torch.where(lse.isinf(), 0.0, lse), tok, block)[0]
    delta = (_blocks(o, tok, block)[0] * dob).sum(3, keepdim=True)
    idx, cnt = _lists(keep(qb, kb))
    p = _scores(c, qb, kb, live, idx, cnt).sub_(lseb[..., None]).exp_()
    p *= live[..., None]
    flat = (idx + torch.arange(idx.shape[0], device=idx.device)[:, None, None] * idx.shape[1]).reshape(-1)

    def onto_keys(a, b):
        g = torch.matmul(a.transpose(2, 3), b).view(-1, block, c["d"])
        return torch.zeros_like(kb).flatten(0, 1).index_add_(0, flat, g).view(kb.shape)

    dv = onto_keys(p, dob)
    ds = torch.matmul(dob, _gathered(vb, idx).transpose(2, 3)).sub_(delta).mul_(p)
    del p
    ds *= 1 / math.sqrt(c["d"])
    dk = onto_keys(ds, qb)
    dq = torch.matmul(ds, _gathered(kb, idx))
    return tuple(_natural(x, tok, n).to(BF) for x in (dq, dk, dv))


def _plain_keep(c, keep):
    """The mask as the call makes it: given, or chosen from the rows of the cube layout."""
    return (lambda qb, kb: _cubes(c, qb, kb)) if c.get("kinds") == "cube" else (lambda qb, kb: keep)


def _code(y, block):
    """e4m3 values with one power-of-two scale per `block` rows, as the values they stand for."""
    n = y.shape[2]
    rows = torch.nn.functional.pad(y, (0, 0, 0, -n % block)).unflatten(2, (-1, block))
    top = rows.abs().amax((3, 4), keepdim=True)
    m, e = torch.frexp(top)
    e = torch.where(top > 0, torch.where(m <= 0.875, e - 9, e - 8), 0)
    v = torch.ldexp(torch.ldexp(rows, -e).to(torch.float8_e4m3fn).to(y.dtype), e)
    return v.flatten(2, 3)[:, :, :n].to(BF)


def _plain_norm(c, s):
    dtype = s["x"].dtype
    x = s["x"].float()
    if c["residual"]:
        x = x + s["res"].float()
    rstd = (x.square().mean(3) + 1e-6).rsqrt()
    y = x * rstd[..., None] * s["w"].float()
    out = dict(rstd=rstd)
    if c["residual"]:
        out["sum"] = x.to(dtype)
    if c["block"]:
        out["codes"] = _code(y, c["block"])
    else:
        out["y"] = y.to(dtype)
    return out


def _plain_norm_backward(c, s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = x * s["rstd"][..., None]
    g = dy * s["w"].float()
    dx = s["rstd"][..., None] * (g - xh * (g * xh).mean(3, keepdim=True))
    if c["residual"]:
        dx = dx + s["dsum"].float()
    return dict(dx=dx.to(s["x"].dtype), dw=(dy * xh).sum((0, 1, 2)))


# ------------------------------------------------------------------------------------------
# the measured calls
# ------------------------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _inputs(c, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    if c["op"] in ("norm", "norm_bwd"):
        dtype = BF if c["dtype"] == "bf16" else F32
        B, H, N, d = c["B"], c["H"], c["N"], c["d"]

        def rows():  # activations with a few large channels, as projections give them
            scale = 1 + 4 * (torch.rand(d, generator=g, device="cuda") < 0.02)
            x = (_randn(g, B, N, H, d) * scale if c["strided"] else _randn(g, B, H, N, d) * scale).to(dtype)
            return x.transpose(1, 2) if c["strided"] else x

        s = dict(case=c, x=rows(), w=(1 + 0.1 * _randn(g, d)).to(dtype))
        if c["op"] == "norm":
            s["res"] = rows() if c["residual"] else None
        else:
            s["rstd"] = (s["x"].float().square().mean(3) + 1e-6).rsqrt()
            s["dy"] = _randn(g, B, H, N, d).to(dtype)
            s["dsum"] = _randn(g, B, H, N, d).to(dtype) if c["residual"] else None
        return s
    B, H, N, d, block = c["B"], c["H"], c["F"] * c["Hl"] * c["Wl"], c["d"], c["block"]
    q, k, v, do = (_randn(g, B * H, N, d) for _ in range(4))
    # half of the heads favour the own frame, half the own position
    f = torch.arange(N, device="cuda") // (c["Hl"] * c["Wl"])
    p = torch.arange(N, device="cuda") % (c["Hl"] * c["Wl"])
    u = torch.stack([_randn(g, c["F"], d)[f] if h % 2 == 0 else _randn(g, c["Hl"] * c["Wl"], d)[p] for h in range(B * H)])
    q, k = q + 2 * u, k + 2 * u
    q, k, v, do = (x.to(BF) for x in (q, k, v, do))
    if c["op"] == "lists":
        nb = -(-N // block)
        keep = (torch.rand(B * H, nb, nb, generator=g, device="cuda") < c["keep"]) | torch.eye(nb, dtype=torch.bool, device="cuda")
        if c["empty"]:
            keep[:, ::c["empty"]] = False
        tok = torch.arange(N, device="cuda").expand(B * H, N)
        kinds = [0] * (B * H)
    else:
        keep = _keep(c).cuda() if c["kinds"] != "cube" else None
        kinds = _kinds(c)
        both = {x: _tokens(c, x).cuda() for x in set(kinds)}
        tok = torch.stack([both[x] for x in kinds])
    s = dict(case=c, q=q, k=k, v=v, do=do, tok=tok, keep=keep, kinds=torch.tensor(kinds, dtype=torch.uint8, device="cuda"))
    if c["op"] != "step":
        o, s["lse"] = _plain_forward(c, q, k, v, tok, _plain_keep(c, keep))
        s["o"] = o.to(BF)
    if c["op"] == "lists":
        idx, cnt = _lists(keep)
        s["idx"] = torch.where(torch.arange(idx.shape[2], device="cuda") < cnt[..., None], idx, -1).to(torch.int32).contiguous()
        s["cnt"] = cnt.to(torch.int32)
    return s


def prepare(case, seed):
    c, s = case, _inputs(case, seed)
    if not own:
        return s
    import block_sparse_attention_31_b200 as vsa
    if c["op"] in ("norm", "norm_bwd"):
        s["norm"] = vsa.RMSNorm(c["B"], c["H"], c["N"], c["d"], dtype=s["x"].dtype, eps=1e-6, quantize=c.get("block", 0),
                                with_grad=c["op"] == "norm_bwd")
    elif c["op"] == "lists":
        s["shape"] = vsa.make_shape(c["B"], c["H"], c["F"], c["Hl"], c["Wl"], c["d"], c["block"])
        s["ws"] = torch.empty(vsa.vsa_sparse_attn_bwd_workspace_size(s["shape"]), dtype=torch.uint8, device="cuda")
        s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        cube = c["kinds"] == "cube"
        s["plan"] = vsa.SparseAttention(c["B"], c["H"], c["F"], c["Hl"], c["Wl"], c["d"], c["block"],
                                        select="cube" if cube else "given", w_s=c["w_s"], w_t=c["w_t"], topk=c["topk"],
                                        cube=CUBE if cube else None, with_grad=True)
    return s


def _own(c, s):
    import block_sparse_attention_31_b200 as vsa
    if c["op"] == "norm":
        r = s["norm"](s["x"], s["w"], residual=s["res"])
        out = dict(rstd=r.rstd)
        if c["residual"]:
            out["sum"] = r.sum
        if c["block"]:
            v = r.codes.view(torch.float8_e4m3fn).to(BF)
            scale = torch.exp2(r.exps.to(BF))
            if c["block"] > 1:
                scale = scale.repeat_interleave(c["block"], 2)[:, :, :c["N"]]
            out["codes"] = v.mul_(scale[..., None])
        else:
            out["y"] = r.y
        return out
    if c["op"] == "norm_bwd":
        dx, dw = s["norm"].backward(s["dy"], s["x"], s["rstd"], s["w"], dsum=s["dsum"])
        return dict(dx=dx, dw=dw)
    shape = (c["B"], c["H"], c["F"] * c["Hl"] * c["Wl"], c["d"])
    q, k, v, do = (s[x].view(shape) for x in ("q", "k", "v", "do"))
    flat = lambda xs: tuple(x.view(-1, *shape[2:]) for x in xs)  # noqa: E731
    if c["op"] == "lists":
        grads = [torch.empty_like(q) for _ in range(3)]
        vsa.vsa_sparse_attn_bwd(vsa.qkvo_grad(q, k, v, s["o"], do, s["lse"], *grads), None, s["kinds"], s["idx"], s["cnt"],
                                s["idx"].shape[2], s["shape"], 0.0, s["ws"], s["ws"].numel(), s["err"])
        return flat(grads)
    kinds = None if c["kinds"] == "cube" else s["kinds"]
    if c["op"] == "call":
        return flat(s["plan"].backward(do, q, k, v, s["o"].view(shape), s["lse"].view(shape[:3]), kinds=kinds))
    q, k, v = (x.detach().requires_grad_() for x in (q, k, v))
    o = s["plan"].attend(q, k, v, kinds=kinds)
    return flat((o.detach(),) + torch.autograd.grad(o, (q, k, v), do))


def run(state):
    c, s = state["case"], state
    if own:
        return _own(c, s)
    if c["op"] == "norm":
        return _plain_norm(c, s)
    if c["op"] == "norm_bwd":
        return _plain_norm_backward(c, s)
    keep = _plain_keep(c, s["keep"])
    if c["op"] != "step":
        return _plain_backward(c, s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["tok"], keep)
    o, lse = _plain_forward(c, s["q"], s["k"], s["v"], s["tok"], keep)
    return (o.to(BF),) + _plain_backward(c, s["q"], s["k"], s["v"], o, lse, s["do"], s["tok"], keep)


def work(case):
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        n, es = c["B"] * c["H"] * c["N"] * c["d"], 2 if c["dtype"] == "bf16" else 4
        rows = 4 * c["B"] * c["H"] * c["N"]
        if c["op"] == "norm":
            return dict(bytes=n * (es * (1 + 2 * c["residual"]) + (1 if c["block"] else es)) + rows, flops=5 * n)
        return dict(bytes=n * es * (3 + c["residual"]) + rows, flops=10 * n)
    heads, n = c["B"] * c["H"], c["F"] * c["Hl"] * c["Wl"]
    if c["op"] == "lists":
        pairs = c["keep"] * n * n * heads * (1 - (1 / c["empty"] if c["empty"] else 0))
    elif c["kinds"] == "cube":
        blocks = len(_tokens(c, 2)) // 128
        pairs = heads * n * n * min(1.0, (c["topk"] + 0.9) / blocks)
    else:
        pairs = float(_keep(c).double().mean()) * n * n * heads
    step = c["op"] == "step"  # reads q, k, v, do and writes o and three gradients: as many rows as the others
    return dict(bytes=heads * n * (c["d"] * 2 * 8 + 8), flops=pairs * c["d"] * (14 if step else 10))


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------
def _exact_allowed(c, kind, q, k, keep):
    """Which token may see which, [N, N] in natural order, for one head."""
    n, b = c["F"] * c["Hl"] * c["Wl"], c["block"]
    t = torch.arange(n, device="cuda")
    s = c["Hl"] * c["Wl"]
    f, p = t // s, t % s
    if kind == 2:
        h, w = p // c["Wl"], p % c["Wl"]
        nh, nw = -(-c["Hl"] // 4), -(-c["Wl"] // 8)
        cube = ((f // 4) * nh + h // 4) * nw + w // 8
        cubes = -(-c["F"] // 4) * nh * nw
        member = (cube[None, :] == torch.arange(cubes, device="cuda")[:, None]).double()
        member /= member.sum(1, keepdim=True)
        score = (member @ q.double()) @ (member @ k.double()).T
        kept = torch.eye(cubes, dtype=torch.bool, device="cuda")
        best = score.sort(dim=1, descending=True, stable=True).indices[:, :c["topk"]]
        return kept.scatter(1, best, True)[cube][:, cube]
    if c["op"] == "lists":
        return keep[t // b][:, t // b]
    slot, group, width = (t, f, c["w_s"]) if kind == 0 else (p * c["F"] + f, p, c["w_t"])
    block = slot // b
    nb = -(-n // b)
    low = torch.full((nb,), 1 << 30, device="cuda").scatter_reduce(0, block, group, "amin")
    high = torch.full((nb,), -1, device="cuda").scatter_reduce(0, block, group, "amax")
    gap = torch.maximum(low[None, :] - high[:, None], low[:, None] - high[None, :])
    return (gap <= width)[block][:, block]


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "norm":
        x = s["x"].double() + (s["res"].double() if c["residual"] else 0)
        rstd = 1 / torch.sqrt((x * x).sum(3) / c["d"] + 1e-6)
        y = torch.einsum("bhnd,bhn,d->bhnd", x, rstd, s["w"].double())
        out = dict(rstd=rstd, **({"sum": x} if c["residual"] else {}))
        if not c["block"]:
            return dict(out, y=y)
        return dict(out, codes=None)  # the nearest code is the definition: it has no value in 64 bits
    if c["op"] == "norm_bwd":
        x, w, r, dy = (s[k].double() for k in ("x", "w", "rstd", "dy"))
        xh = x * r[..., None]
        # d rstd / dx = -rstd^3 x / d
        dx = dy * w * r[..., None] - x * ((dy * w * x).sum(3) * r ** 3 / c["d"])[..., None]
        if c["residual"]:
            dx = dx + s["dsum"].double()
        return dict(dx=dx, dw=torch.einsum("bhnd,bhnd->d", dy, xh))
    n, scale = c["F"] * c["Hl"] * c["Wl"], 1 / math.sqrt(c["d"])
    outs = [[], [], [], []]
    for h, kind in enumerate(s["kinds"].tolist()):
        q, k, v, do = (s[x][h].double() for x in ("q", "k", "v", "do"))
        allowed = _exact_allowed(c, kind, s["q"][h], s["k"][h], s["keep"][h] if c["op"] == "lists" else None)
        p = (q @ k.T).mul_(scale).masked_fill_(~allowed, -math.inf)
        del allowed
        if c["op"] == "step":
            p = torch.softmax(p, dim=1)
            o = p @ v
        else:
            lse, o = s["lse"][h].double(), s["o"][h].double()
            p = p.sub_(torch.where(lse.isinf(), 0.0, lse)[:, None]).exp_()
        ds = (do @ v.T).sub_((do * o).sum(1, keepdim=True)).mul_(p)
        for to, x in zip(outs, (o, ds @ k * scale, ds.T @ q * scale, p.T @ do)):
            to.append(x)
        del p, ds
    outs = [torch.stack(x) for x in outs]
    return tuple(outs) if c["op"] == "step" else tuple(outs[1:])
