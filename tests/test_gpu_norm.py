"""GPU checks of the root-mean-square norm (vsa_rms_norm, vsa_rms_norm_bwd, RMSNorm) against 64 bits.

Tolerances.  An output of type t is rounded once, by at most eps(t) / 2 of its value.  In front of that the
arithmetic is fp32: the sum of squares adds up to 64 terms in a row per thread and joins the threads in a tree
(at most 64 + 12 roundings of 2^-24 each on a positive sum, halved by the square root), the root, the quotient and
two products add one or two more each: F = 2^-18 of the value covers them for d up to 16384.
"""
import numpy as np
import pytest
import torch

import oracle
import synthetic
from parity_util import cuda_err

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import block_sparse_attention_31_b200 as vsa
    from block_sparse_attention_31_b200 import _lib
else:
    vsa = _lib = None

BF, F32 = torch.bfloat16, torch.float32
F = 2.0 ** -18


def _half(t):
    return torch.finfo(t).eps / 2


def _rand(*shape, seed=0, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()


def _near(got, want, room, what):
    assert got.shape == want.shape
    over = (got.double() - want).abs() - room
    assert bool((over <= 0).all()), f"{what}: off by {float(((got.double() - want).abs()).max()):.3g}, {float(over.max()):.3g} too much"


def _reference(x, w, res, eps):
    s = x.double() + (res.double() if res is not None else 0.0)
    rstd = 1 / torch.sqrt((s * s).mean(3) + eps)
    return s, rstd, s * rstd[..., None] * (w.double() if w is not None else 1.0)


def _check_codes(codes, exps, y, block):
    """Each code is the nearest e4m3 value of y / 2^e, and e the smallest that holds the block."""
    N = y.shape[2]
    per_row = exps.repeat_interleave(block, 2)[:, :, :N].double()
    got = codes.view(torch.float8_e4m3fn).double()
    scaled = y / torch.exp2(per_row)[..., None]
    # nearest: half a step, 2^-4 of the value or half the subnormal step 2^-9
    assert bool(((got - scaled).abs() <= (scaled.abs() * 2.0 ** -4).clamp(min=2.0 ** -10) * (1 + 2.0 ** -14) +
                 F * scaled.abs()).all())
    rows = torch.nn.functional.pad(y, (0, 0, 0, -N % block)).unflatten(2, (-1, block))
    top = rows.abs().amax((3, 4))
    e = exps.double()
    assert bool((top <= 448 * torch.exp2(e) * (1 + F)).all())
    assert bool(((top > 224 * torch.exp2(e) * (1 - F)) | (top == 0)).all())
    assert bool((e[top == 0] == 0).all())


def _case(B, H, N, d, dtype, x, w, res, quantize=0, eps=1e-6):
    norm = vsa.RMSNorm(B, H, N, d, dtype=dtype, eps=eps, quantize=quantize, keep_y=True)
    r = norm(x, w, residual=res)
    s, rstd, y = _reference(x, w, res, eps)
    _near(r.rstd, rstd, rstd * F, "rstd")
    # a product below the smallest normal loses digits that count in absolute terms only
    tiny = torch.finfo(dtype).tiny
    _near(r.y, y, y.abs() * (F + _half(dtype)) + tiny, "y")
    if res is not None:
        _near(r.sum, s, s.abs() * (F + _half(dtype)) + tiny, "sum")
    if quantize:
        assert tuple(r.exps.shape) == (B, H, -(-N // quantize))
        _check_codes(r.codes, r.exps, y, quantize)
    return r


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [1, 7, 8, 32, 33, 64, 72, 100, 128, 129, 256, 500, 512, 513, 1000, 1024, 1536, 2048, 2049, 4096, 4104, 5120,
                               8192, 8200, 16384])
def test_widths(d, dtype):
    """Every way of holding a row, whole and ragged, with residual and codes per row."""
    N = 37 if d < 4096 else 5
    x, res, w = _rand(1, 1, N, d, seed=d, dtype=dtype), _rand(1, 1, N, d, seed=d + 1, dtype=dtype, scale=3.0), _rand(d, seed=2, dtype=dtype)
    _case(1, 1, N, d, dtype, x, w, res, quantize=1)
    _case(1, 1, N, d, dtype, x, None, None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("block", [64, 128])
@pytest.mark.parametrize("N", [1, 64, 127, 300])
def test_block_scales(N, block, d, dtype):
    """One exponent per block of rows of a head, the last one ragged; x as projection and contiguous."""
    w = _rand(d, seed=2, dtype=F32)
    x = _rand(2, N, 3, d, seed=N, dtype=dtype).transpose(1, 2)
    a = _case(2, 3, N, d, dtype, x, w, None, quantize=block)
    b = _case(2, 3, N, d, dtype, x.contiguous(), w, None, quantize=block)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.exps, b.exps) and torch.equal(a.y, b.y)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,d", [(64, 64), (128, 128)])
def test_more_blocks_than_fit_at_once(block, d, dtype):
    """CTAs that take several blocks each, some one more than others, heads of unlike sizes beside each other."""
    N = 1184 * 9 // 4 // 6 * block + 3      # 2664 blocks: 148 SMs hold at most 1184 of 64 rows at once
    x = _rand(2, N, 3, d, seed=9, dtype=dtype).transpose(1, 2) * torch.tensor([1.0, 1e-3, 1e3], device="cuda").to(dtype)[:, None, None]
    a = _case(2, 3, N, d, dtype, x, _rand(d, seed=2, dtype=dtype), None, quantize=block)
    # codes of a block do not depend on the others'
    b = vsa.RMSNorm(2, 3, block, d, dtype=dtype, quantize=block)(x[:, :, 77 * block:78 * block], _rand(d, seed=2, dtype=dtype))
    assert torch.equal(a.codes[:, :, 77 * block:78 * block], b.codes) and torch.equal(a.exps[:, :, 77:78], b.exps)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_and_unaligned_rows(dtype):
    """Views: projection, a slice of a fused projection, rows that start off 16 bytes, broadcast rows."""
    B, H, N, d = 2, 3, 45, 64
    w = _rand(d, seed=1, dtype=BF)
    fused = _rand(B, N, 3, H, d, seed=2, dtype=dtype)
    odd = _rand(B, H, N, d + 3, seed=3, dtype=dtype)[..., 1:1 + d]
    views = [fused[:, :, 1].transpose(1, 2), odd, _rand(B, H, 1, d, seed=4, dtype=dtype).expand(B, H, N, d),
             _rand(1, 1, 1, d, seed=5, dtype=dtype).expand(B, H, N, d), _rand(N, H, B, d, seed=6, dtype=dtype).permute(2, 1, 0, 3)]
    for x in views:
        for res in (None, views[0], views[1]):
            for quantize in (0, 1, 64):
                got = _case(B, H, N, d, dtype, x, w, res, quantize=quantize)
                want = _case(B, H, N, d, dtype, x.contiguous(), w, None if res is None else res.contiguous(), quantize=quantize)
                # threads of a row may be fewer or more: sums in another order
                _near(got.y, want.y.double(), want.y.double().abs() * (2 * F + 2 * _half(dtype)), "y")


def test_extremes():
    """Zero rows, huge and tiny rows, infinities and NaN: nothing spreads to another row."""
    d, N = 128, 130
    x = _rand(1, 1, N, d, seed=1, dtype=F32)
    x[0, 0, 3] = 0
    x[0, 0, 4] *= 1e18
    x[0, 0, 5] *= 1e-18
    _case(1, 1, N, d, F32, x, None, None, quantize=1)
    _case(1, 1, N, d, F32, x, None, None, quantize=128)
    clean = vsa.RMSNorm(1, 1, N, d, dtype=F32, quantize=1, keep_y=True)(x)
    bad = x.clone()
    bad[0, 0, 7, 2] = float("nan")
    bad[0, 0, 9, 2] = float("inf")
    r = vsa.RMSNorm(1, 1, N, d, dtype=F32, quantize=1, keep_y=True)(bad)
    keep = [i for i in range(N) if i not in (7, 9)]
    assert torch.equal(r.y[:, :, keep], clean.y[:, :, keep]) and torch.equal(r.codes[:, :, keep], clean.codes[:, :, keep])
    assert torch.isnan(r.y[0, 0, 7]).all() and torch.isnan(r.y[0, 0, 9, 2]) and (r.y[0, 0, 9, 3:] == 0).all()
    # an output beyond the floats saturates, with the exponent of the largest
    w = torch.full((d,), 3e38, device="cuda")
    r = vsa.RMSNorm(1, 1, N, d, dtype=F32, quantize=1)(x, w)
    v = r.codes.view(torch.float8_e4m3fn).float()
    assert torch.isfinite(v).all() and (r.exps[0, 0, :3] == 120).all() and (v[0, 0, :3].abs().amax(1) == 448).all()
    # zero eps and a zero row: 0 * inf, in that row only
    r = vsa.RMSNorm(1, 1, N, d, dtype=F32, eps=0.0)(x)
    assert torch.isnan(r.y[0, 0, 3]).all() and torch.isfinite(r.y[0, 0, :3]).all() and torch.isfinite(r.y[0, 0, 4:]).all()


def _backward_case(B, H, N, d, dtype, x, w, dy, d_sum):
    norm = vsa.RMSNorm(B, H, N, d, dtype=dtype, with_grad=True)
    s, rstd, _ = _reference(x, w, None, 1e-6)
    r32 = rstd.float()
    dx, dw = norm.backward(dy, x, r32, w, d_sum=d_sum)
    r = r32.double()[..., None]
    wd = w.double() if w is not None else 1.0
    xh, g = s * r, dy.double() * wd
    want = r * (g - xh * (g * xh).mean(3, keepdim=True)) + (d_sum.double() if d_sum is not None else 0.0)
    # the difference may cancel: fp32 errors count against its terms
    terms = r * (g.abs() + xh.abs() * (g * xh).abs().mean(3, keepdim=True)) + (d_sum.double().abs() if d_sum is not None else 0.0)
    _near(dx, want, terms * F + want.abs() * _half(dtype) + torch.finfo(dtype).tiny, "dx")
    if w is None:
        assert dw is None
    else:
        t = dy.double() * xh
        # a thread adds at most a few hundred rows in a row
        _near(dw, t.sum((0, 1, 2)), t.abs().sum((0, 1, 2)) * 2.0 ** -15 + 1e-30, "dw")
        again = norm.backward(dy, x, r32, w, d_sum=d_sum)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    return dx, dw


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [1, 8, 33, 64, 128, 129, 500, 513, 1000, 1536, 2048, 2056, 4104, 8192, 16384])
def test_backward_widths(d, dtype):
    N = 53 if d < 4096 else 5
    x, w, dy, ds = (_rand(*sh, seed=d + i, dtype=dtype) for i, sh in enumerate([(1, 1, N, d), (d,), (1, 1, N, d), (1, 1, N, d)]))
    _backward_case(1, 1, N, d, dtype, x, w, dy, ds)
    _backward_case(1, 1, N, d, dtype, x, None, dy, None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_backward_heads_and_strides(dtype):
    B, H, N, d = 2, 5, 1033, 128
    w, dy = _rand(d, seed=1, dtype=F32), _rand(B, H, N, d, seed=2, dtype=dtype)
    fused = _rand(B, N, 3, H, d, seed=3, dtype=dtype)
    # dx has x's order of dimensions only where x fills its memory
    for whole, x in ((True, _rand(B, N, H, d, seed=4, dtype=dtype).transpose(1, 2)), (False, fused[:, :, 2].transpose(1, 2)),
                     (False, _rand(B, H, N, d + 1, seed=5, dtype=dtype)[..., :d]),
                     (False, _rand(B, 1, N, d, seed=6, dtype=dtype).expand(B, H, N, d))):
        dx, _ = _backward_case(B, H, N, d, dtype, x, w, dy, None)
        assert (dx.stride() == x.stride()) == whole and (whole or dx.is_contiguous())
    # many rows a thread
    _backward_case(1, 1, 200000, 64, dtype, _rand(1, 1, 200000, 64, seed=7, dtype=dtype), w[:64].contiguous(),
                   _rand(1, 1, 200000, 64, seed=8, dtype=dtype), None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,N", [(256, 6007), (1000, 3001), (1536, 3001), (2056, 1301), (8200, 331), (16384, 331)])
def test_backward_many_rows_a_cta(d, N, dtype):
    """Every way of holding a row with more chunks than CTAs, some CTAs with one more, with and without d_sum."""
    x, w, dy, ds = (_rand(*sh, seed=d + i, dtype=dtype) for i, sh in enumerate([(1, 1, N, d), (d,), (1, 1, N, d), (1, 1, N, d)]))
    for d_sum in (None, ds):
        dx, _ = _backward_case(1, 1, N, d, dtype, x, w, dy, d_sum)
        few = vsa.RMSNorm(1, 1, 7, d, dtype=dtype, with_grad=True)
        rstd = _reference(x, w, None, 1e-6)[1].float()[:, :, -7:].clone()
        last = few.backward(dy[:, :, -7:].clone(), x[:, :, -7:].clone(), rstd, w,
                             d_sum=None if d_sum is None else d_sum[:, :, -7:].clone())[0]
        assert torch.equal(dx[:, :, -7:], last)  # a row's gradient does not depend on the others


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last rows come out as they do alone, and the first are not touched by them."""
    B, H, N, d = 1, 137, 122500, 128
    assert B * H * N * d > 1 << 31
    x = torch.zeros(B, N, H, d, dtype=BF, device="cuda")
    x[:, -300:] = _rand(B, 300, H, d, seed=1)
    w, dy = _rand(d, seed=2), torch.zeros(B, H, N, d, dtype=BF, device="cuda")
    dy[:, :, -300:] = _rand(B, H, 300, d, seed=3)
    tail = x[:, -300:].contiguous().transpose(1, 2)
    full, part = (vsa.RMSNorm(B, H, n, d, with_grad=True) for n in (N, 300))
    r, p = full(x.transpose(1, 2), w), part(tail, w)
    assert torch.equal(r.y[:, :, -300:], p.y) and torch.equal(r.rstd[:, :, -300:], p.rstd) and bool((r.y[:, :, :1000] == 0).all())
    rstd = r.rstd
    del r
    dx, dw = full.backward(dy, x.transpose(1, 2), rstd, w)
    px, pw = part.backward(dy[:, :, -300:].contiguous(), tail, p.rstd, w)
    assert torch.equal(dx[:, :, -300:], px) and bool((dx[:, :, :1000] == 0).all())
    # two fp32 sums of the same terms, each within 2^-15 of the sum of their sizes
    terms = (dy[:, :, -300:].double() * tail.double() * p.rstd.double()[..., None]).abs().sum((0, 1, 2))
    _near(dw, pw.double(), terms * 2.0 ** -14, "dw")


def test_normalise_is_differentiable():
    """autograd through x, weight and residual, one output or both, against torch's gradients in 64 bits."""
    B, H, N, d = 1, 2, 40, 128
    for dtype, wt in ((BF, BF), (F32, F32), (BF, F32)):
        norm = vsa.RMSNorm(B, H, N, d, dtype=dtype, with_grad=True)
        x = _rand(B, N, H, d, seed=1, dtype=dtype).transpose(1, 2).requires_grad_()
        w, res = _rand(d, seed=2, dtype=wt).requires_grad_(), _rand(B, H, N, d, seed=3, dtype=dtype).requires_grad_()
        u, v = _rand(B, H, N, d, seed=4, dtype=F32), _rand(B, H, N, d, seed=5, dtype=F32)
        for which in ("both", "y", "sum"):
            y, total = norm.normalise(x, w, res)
            loss = (y.float() * u).sum() * (which != "sum") + (total.float() * v).sum() * (which != "y")
            got = torch.autograd.grad(loss, (x, w, res), allow_unused=True)
            xd, wd, rd = (t.detach().double().requires_grad_() for t in (x, w, res))
            s = xd + rd
            yd = s / torch.sqrt((s * s).mean(3, keepdim=True) + 1e-6) * wd
            ref = (yd * u.double()).sum() * (which != "sum") + (s * v.double()).sum() * (which != "y")
            want = torch.autograd.grad(ref, (xd, wd, rd), allow_unused=True)
            for name, a, b in zip(("x", "w", "res"), got, want):
                if b is None or float(b.abs().max()) == 0.0:
                    continue
                # the sum the gradient starts from is rounded, and so are dy, d_sum and the result: four halves of a step
                # of the row's size
                room = 4 * _half(dtype) * b.abs().amax(-1, keepdim=True) + 4 * _half(wt) * b.abs().max()
                _near(a, b, room, f"{name} {which}")
        y = norm.normalise(x, None)
        (g,) = torch.autograd.grad(y.sum(), (x,))
        assert g.shape == x.shape and torch.isfinite(g).all()


def test_norm_codes_feed_the_fp8_attention():
    """Norm to codes -> vsa_sparse_attn_fwd_fp8qk, against the attention of the values the codes stand for."""
    H, N, d = 2, 300, 128
    shape = _lib.make_shape(1, H, 1, 1, N, d, 128)
    norm = vsa.RMSNorm(1, H, N, d, quantize=128)
    w = _rand(d, seed=1, dtype=F32)
    q, k = (norm(_rand(1, N, H, d, seed=s).transpose(1, 2), w) for s in (2, 3))
    v = _rand(1, H, N, d, seed=4)
    keep = np.tri(3, dtype=bool)
    idx, cnt = oracle.keep_to_lists(keep, 3)
    idx, cnt = (torch.from_numpy(np.stack([t] * H)[None].astype(np.int32)).cuda() for t in (idx, cnt))
    o, kinds, err = torch.empty_like(v), torch.zeros(H, dtype=torch.uint8, device="cuda"), cuda_err()
    _lib.vsa_sparse_attn_fwd_fp8qk(_lib.qkvo(v, v, v, o), None, q.codes, q.exps, k.codes, k.exps, kinds, idx, cnt, 3, shape, 0.0, err)
    assert _lib.vsa_get_device_error(err) == 0
    for h in range(H):
        rows = [oracle.dequantize_e4m3(t.codes[0, h].cpu().numpy(), t.exps[0, h].cpu().numpy(), 128) for t in (q, k)]
        want, _ = oracle.attention_rows(rows[0], rows[1], v[0, h].cpu().float().numpy(), np.arange(N), 128, keep, scale=d ** -0.5)
        got = o[0, h].cpu().double().numpy()
        assert np.abs(got - want).max() <= 2e-2 and np.linalg.norm(got - want) <= 1e-2 * np.linalg.norm(want)


def test_block_of_training():
    """Projection -> norm of Q and K -> sparse attention -> gradients of the projections and of the norm weights."""
    import math

    from grad_util import allowed_blocks
    from parity_util import keep_for_head
    wl = synthetic.Workload("t", 1, 2, 4, 6, 8, 64, 64, "bf16", "given")
    B, H, N, d = 1, 2, wl.N, 64
    kinds = torch.tensor([0, 1], dtype=torch.uint8, device="cuda")
    plan = vsa.SparseAttention(B, H, 4, 6, 8, d, 64, select="given", w_s=1, w_t=11, with_grad=True)
    norm = vsa.RMSNorm(B, H, N, d, with_grad=True)
    xq, xk = (_rand(B, N, H, d, seed=s).requires_grad_() for s in (1, 2))
    v, do = _rand(B, H, N, d, seed=3).requires_grad_(), _rand(B, H, N, d, seed=4)
    wq, wk = ((1 + 0.1 * _rand(d, seed=s, dtype=F32)).requires_grad_() for s in (5, 6))
    o = plan.attend(norm.normalise(xq.transpose(1, 2), wq), norm.normalise(xk.transpose(1, 2), wk), v, kinds=kinds)
    got = torch.autograd.grad(o, (xq, xk, v, wq, wk), do)
    assert plan.device_error() == 0
    ins = [t.detach().double().requires_grad_() for t in (xq, xk, v, wq, wk)]
    n64 = lambda x, w: x / torch.sqrt((x * x).mean(3, keepdim=True) + 1e-6) * w  # noqa: E731
    q, k = n64(ins[0].transpose(1, 2), ins[3]), n64(ins[1].transpose(1, 2), ins[4])
    loss = 0.0
    for h in range(H):
        al = allowed_blocks(keep_for_head(h, wl, 1, 11), oracle.layout_slots(h, 4, 6, 8), 64).cuda()
        p = torch.softmax((q[0, h] @ k[0, h].T / math.sqrt(d)).masked_fill(~al, -math.inf), 1)
        loss = loss + (p @ ins[2][0, h] * do[0, h].double()).sum()
    want = torch.autograd.grad(loss, ins)
    for name, a, b in zip(("xq", "xk", "v", "wq", "wk"), got, want):
        # q, k, o, P, dS, dq, dk, dx: eight roundings of at most 2^-8 on the way, none of which grows with the
        # sums that follow it
        rel = float((a.double() - b).norm() / b.norm())
        assert rel <= 8 * 2.0 ** -8, f"{name}: {rel:.3g}"


def test_captured_replayed_and_streams():
    B, H, N, d = 1, 3, 200, 128
    norm = vsa.RMSNorm(B, H, N, d, with_grad=True, quantize=128, keep_y=True)
    x, w, dy = _rand(B, N, H, d, seed=1).transpose(1, 2), _rand(d, seed=2), _rand(B, H, N, d, seed=3)
    first = norm(x, w)
    norm.backward(dy, x, first.rstd, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = norm(x, w)
        grads = norm.backward(dy, x, r.rstd, w)
        with pytest.raises(RuntimeError, match="cannot be captured"):
            norm.normalise(x.detach().requires_grad_(), w)
    x.copy_(_rand(B, N, H, d, seed=7).transpose(1, 2))
    graph.replay()
    want = norm(x, w)
    for a, b in zip((*r, *grads), (*want, *norm.backward(dy, x, want.rstd, w))):
        assert a is None and b is None or torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = norm(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got.codes, want.codes) and torch.equal(got.y, want.y)


def test_refusals():
    x, w = _rand(1, 2, 10, 64), _rand(64)
    for kw in (dict(quantize=3), dict(d=100, quantize=64), dict(dtype=torch.float16), dict(quantize=1, with_grad=True)):
        with pytest.raises(ValueError):
            vsa.RMSNorm(**{**dict(B=1, H=2, N=10, d=64), **kw})
    for bad in (dict(d=16385), dict(N=0), dict(eps=-1.0), dict(eps=float("inf"))):
        with pytest.raises(vsa.VsaError):
            vsa.RMSNorm(**{**dict(B=1, H=2, N=10, d=64), **bad})
    norm = vsa.RMSNorm(1, 2, 10, 64, with_grad=True)
    for args in ((x.float(), w), (x[:, :1], w), (x, w[:32]), (x, w.half()), (x.cpu(), w), (x.transpose(2, 3).contiguous().transpose(2, 3), w)):
        with pytest.raises(ValueError):
            norm(*args)
    with pytest.raises(ValueError):
        norm(x, w, residual=x.float())
    r = norm(x, w)
    with pytest.raises(ValueError, match="contiguous"):
        norm.backward(x.transpose(1, 2).contiguous().transpose(1, 2), x, r.rstd, w)
    with pytest.raises(ValueError, match="rstd"):
        norm.backward(x, x, r.rstd.double(), w)
    with pytest.raises(ValueError, match="with_grad"):
        vsa.RMSNorm(1, 2, 10, 64).backward(x, x, r.rstd, w)
    with pytest.raises(ValueError, match="with_grad"):
        vsa.RMSNorm(1, 2, 10, 64).normalise(x, w)
