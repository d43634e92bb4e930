"""GPU checks of how the gradient and the norm are called: strided and unaligned arguments, streams, threads, unknown
head kinds, heads of unlike layouts beside each other."""
import threading

import numpy as np
import pytest
import torch

import oracle
import synthetic
from grad_util import allowed_blocks, assert_grads, reference
from parity_util import cuda_err, keep_for_head

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import block_sparse_attention_31_b200 as vsa
    from block_sparse_attention_31_b200 import _lib
else:
    vsa = _lib = None

BF, F32 = torch.bfloat16, torch.float32
S_, T_, C_ = 0, 1, 2


def _rand(*shape, seed=0, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _small(select="given", dtype=BF, **kw):
    """A plan of two heads on a ragged grid, its inputs and the gradient of its output."""
    plan = vsa.SparseAttention(1, 2, 5, 6, 10, 64, 64, dtype=dtype, select=select, w_s=1, w_t=9, with_grad=True, **kw)
    return (plan, *(_rand(1, 2, 300, 64, seed=s, dtype=dtype) for s in range(4)))


def _in_longer_rows(t):
    """The same values in rows that are one element longer than they are read."""
    rows = torch.full((*t.shape[:-1], t.shape[-1] + 1), 1e3, device="cuda")
    rows[..., :-1] = t
    return rows[..., :-1]


def _off_16_bytes(t):
    flat = torch.empty(t.numel() + 1, device="cuda")
    flat[1:] = t.flatten()
    return flat[1:].view(t.shape)


def test_log_sum_exp_in_longer_rows():
    """lse and d_lse cut out of longer rows, flat or per batch, or off 16 bytes: the bits of whole rows."""
    B, H, N, d = 2, 3, 300, 64
    shape = _lib.make_shape(B, H, 1, 1, N, d, 64)
    nb = _lib.vsa_num_blocks(shape)
    idx = torch.arange(nb, dtype=torch.int32, device="cuda").expand(B, H, nb, nb).contiguous()
    cnt = torch.full((B, H, nb), nb, dtype=torch.int32, device="cuda")
    kinds, err = torch.zeros(B * H, dtype=torch.uint8, device="cuda"), cuda_err()
    q, k, v, do = (_rand(B, H, N, d, seed=s) for s in range(4))
    o, lse, d_lse = torch.empty_like(q), torch.empty(B, H, N, device="cuda"), _rand(B, H, N, seed=4, dtype=F32)
    _lib.vsa_sparse_attn_fwd(_lib.qkvo(q, k, v, o, lse), None, kinds, idx, cnt, nb, shape, 0.0, err)
    ws = torch.empty(_lib.vsa_sparse_attn_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")

    def run(lse, d_lse, stream=None):
        grads = [torch.empty_like(q) for _ in range(3)]
        _lib.vsa_sparse_attn_bwd(_lib.qkvo_grad(q, k, v, o, do, lse, *grads, d_lse=d_lse), None, kinds, idx, cnt, nb, shape, 0.0,
                                 ws, ws.numel(), err, stream)
        return grads

    want = run(lse, d_lse)
    # the whole rows are right, to the eye of the element bounds
    for h in range(H):
        _, _, ref, bounds = reference(q[1, h], k[1, h], v[1, h], do[1, h], torch.ones(N, N, dtype=torch.bool, device="cuda"), o=o[1, h],
                                      lse=lse[1, h], d_lse=d_lse[1, h])
        assert_grads([g[1, h] for g in want], ref, bounds, f"head {h}")
    flat = _in_longer_rows(lse.view(B * H, N))
    assert not flat.is_contiguous()
    for a, b in ((flat, d_lse), (_in_longer_rows(lse), _in_longer_rows(d_lse)), (_off_16_bytes(lse), _off_16_bytes(d_lse)),
                 (lse.transpose(0, 1).contiguous().transpose(0, 1), d_lse)):
        for x, y in zip(run(a, b), want):
            assert torch.equal(x, y)
    side = torch.cuda.Stream()
    late = torch.zeros(B * H, N + 1, device="cuda")[:, :-1]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):      # there when the call's own stream comes to it
        torch.cuda._sleep(100_000_000)
        late.copy_(flat)
    got = run(late, d_lse, side)
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert _lib.vsa_get_device_error(err) == 0


def test_call_takes_a_log_sum_exp_in_longer_rows():
    plan, q, k, v, do = _small()
    kinds = torch.tensor([S_, T_], dtype=torch.uint8, device="cuda")
    o, lse = plan(q, k, v, kinds=kinds)
    d_lse = _rand(*lse.shape, seed=5, dtype=F32)
    want = plan.backward(do, q, k, v, o, lse, kinds=kinds, d_lse=d_lse)
    for cut in (_in_longer_rows, _off_16_bytes):
        for x, y in zip(plan.backward(do, q, k, v, o, cut(lse), kinds=kinds, d_lse=cut(d_lse)), want):
            assert torch.equal(x, y)


def test_gradient_of_the_sum_under_either_name():
    norm = vsa.RMSNorm(1, 2, 50, 64, with_grad=True)
    x, w, dy, ds = _rand(1, 2, 50, 64, seed=1), _rand(64, seed=2), _rand(1, 2, 50, 64, seed=3), _rand(1, 2, 50, 64, seed=4)
    rstd = norm(x, w).rstd
    for a, b in zip(norm.backward(dy, x, rstd, w, dsum=ds), norm.backward(dy, x, rstd, w, d_sum=ds)):
        assert torch.equal(a, b)
    with pytest.raises(ValueError, match="d_sum"):
        norm.backward(dy, x, rstd, w, d_sum=ds, dsum=ds)


def test_outputs_over_inputs_are_refused():
    """O's rounding errors over an input of their call, gradients and workspace over a set's buffers, whole or in part."""
    plan, q, k, v, do = _small()
    kinds = torch.tensor([S_, T_], dtype=torch.uint8, device="cuda")
    o, lse, n = torch.empty_like(q), torch.empty(1, 2, 300, device="cuda"), q.numel()
    for t in (q, k, v, o, lse.view(BF)):
        both = torch.cat([t.flatten(), torch.zeros(2 * n, dtype=BF, device="cuda")])       # t, then room behind it
        mine = both[:t.numel()].view(t.shape)
        args = dict(q=q, k=k, v=v, out=o, lse=lse)
        name = next(x for x, y in args.items() if y.data_ptr() == t.data_ptr())
        args[name] = mine.view(F32).view(lse.shape) if name == "lse" else mine
        last = (t.numel() - 1) // 8 * 8                                                      # the last place on 16 bytes in t
        for at in (0, 8, last):
            with pytest.raises(vsa.VsaError) as e:
                plan(**args, kinds=kinds, o_lo=both[at:at + n].view(q.shape))
            assert e.value.status == _lib.VSA_ERR_INVALID_ARG
        behind = -(-t.numel() // 8) * 8
        plan(**args, kinds=kinds, o_lo=both[behind:behind + n].view(q.shape))
    plan(q, k, v, out=o, lse=lse, kinds=kinds)
    room = torch.zeros(8 * n, dtype=BF, device="cuda")
    part = lambda at: room[at:at + n].view(q.shape)  # noqa: E731
    part(0).copy_(q)
    for out in ((part(8), part(2 * n), part(3 * n)), (part(n), part(2 * n - 8), part(4 * n)), (part(n), part(2 * n), part(n - 8))):
        with pytest.raises(vsa.VsaError):
            plan.backward(do, part(0), k, v, o, lse, kinds=kinds, out=out)
    grads = plan.backward(do, part(0), k, v, o, lse, kinds=kinds, out=(part(n), part(2 * n), part(3 * n)))
    for a, b in zip(grads, plan.backward(do, q, k, v, o, lse, kinds=kinds)):
        assert torch.equal(a, b)
    shape, err = _lib.make_shape(1, 2, 1, 1, 300, 64, 64), cuda_err()
    idx, cnt = torch.zeros(1, 2, 5, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 2, 5, dtype=torch.int32, device="cuda")
    need = _lib.vsa_sparse_attn_bwd_workspace_size(shape)
    for dq, ws in ((part(8), torch.empty(need, dtype=torch.uint8, device="cuda")), (part(n), part(0).view(torch.uint8).flatten())):
        with pytest.raises(vsa.VsaError) as e:
            _lib.vsa_sparse_attn_bwd(_lib.qkvo_grad(part(0), k, v, o, do, lse, dq, part(2 * n), part(3 * n)), None, kinds, idx, cnt, 1,
                                     shape, 0.0, ws, need, err)
        assert e.value.status == _lib.VSA_ERR_INVALID_ARG


def test_the_default_stream_by_its_handle():
    """Stream 0 is the default stream, not one of torch's own."""
    norm = vsa.RMSNorm(1, 2, 50, 64, with_grad=True)
    x, w, dy = _rand(1, 2, 50, 64, seed=1), _rand(64, seed=2), _rand(1, 2, 50, 64, seed=3)
    want = norm(x, w)
    grads = norm.backward(dy, x, want.rstd, w)
    late, late_dy = torch.zeros_like(x), torch.zeros_like(dy)
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        with torch.cuda.stream(default):
            torch.cuda._sleep(100_000_000)
            late.copy_(x)
            late_dy.copy_(dy)
        got = norm(late, w, stream=0)
        got_grads = norm.backward(late_dy, late, want.rstd, w, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got.y, want.y) and torch.equal(got.rstd, want.rstd)
    for a, b in zip(got_grads, grads):
        assert torch.equal(a, b)


def test_forward_on_another_stream_with_its_own_kinds():
    """The kinds of a call on another stream are its own, however late the current stream is."""
    plan, q, k, v, _ = _small()
    first, other = (torch.tensor(x, dtype=torch.uint8, device="cuda") for x in ([S_, T_], [T_, S_]))
    want = [t.clone() for t in plan(q, k, v, kinds=other)]
    plan(q, k, v, kinds=first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(400_000_000)                # the current stream is busy for some 0.2 s
    for stream in (side, side.cuda_stream):
        got = plan(q, k, v, kinds=other, stream=stream)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    torch.cuda.synchronize()


@pytest.mark.parametrize("which", ["sparse", "semantic"])
def test_outputs_on_another_stream_are_that_streams(which):
    """What a call on another stream allocates is not memory that the current stream still writes."""
    if which == "sparse":
        plan, q, k, v, _ = _small()
        kinds = torch.tensor([S_, T_], dtype=torch.uint8, device="cuda")
        call = lambda **kw: plan(q, k, v, kinds=kinds, **kw)[0]  # noqa: E731
    else:
        sem = vsa.SemanticAttention(1, 2, 5, 6, 10, 64, 64, cq=4, ck=4, iters=2)
        q, k, v = (_rand(1, 2, 300, 64, seed=s) for s in range(3))
        call = lambda **kw: sem(q, k, v, **kw)  # noqa: E731
    want = call().clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    late = [torch.empty_like(q) for _ in range(8)]
    torch.cuda._sleep(200_000_000)
    for x in late:
        x.fill_(7.0)
    del x, late                                   # free for the current stream, which still has to write them
    got = call(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def _at_once(jobs, times):
    """Each job `times` times on a thread and a stream of its own; what they raised."""
    start, raised = threading.Barrier(len(jobs)), []

    def work(job):
        start.wait()
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(times):
                    job()
        except Exception as e:  # noqa: BLE001
            raised.append(f"{type(e).__name__}: {e}")

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return raised


def _attention(nb, gradient):
    N, d = nb * 64, 64
    shape = _lib.make_shape(1, 1, 1, 1, N, d, 64)
    idx = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, 1, nb, 1)
    cnt, kinds, err = torch.ones(1, 1, nb, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.uint8, device="cuda"), cuda_err()
    q, o, lse = _rand(1, 1, N, d), _rand(1, 1, N, d), torch.zeros(1, 1, N, device="cuda")
    if not gradient:
        return lambda: _lib.vsa_sparse_attn_fwd(_lib.qkvo(q, q, q, o, lse), None, kinds, idx, cnt, 1, shape, 0.0, err)
    ws = torch.empty(_lib.vsa_sparse_attn_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")
    grads = [torch.empty_like(q) for _ in range(3)]
    return lambda: _lib.vsa_sparse_attn_bwd(_lib.qkvo_grad(q, q, q, o, o, lse, *grads), None, kinds, idx, cnt, 1, shape, 0.0, ws,
                                            ws.numel(), err)


@pytest.mark.parametrize("gradient", [False, True])
def test_first_call_of_a_thread(gradient):
    """A thread whose first work on the device is the library's launch."""
    torch.cuda.synchronize()
    assert _at_once([_attention(2, gradient)], 1) == []


def _norm_gradient(d, with_sum):
    norm = vsa.RMSNorm(1, 1, 4, d, with_grad=True)
    x, dy, ds = (_rand(1, 1, 4, d, seed=s) for s in range(3))
    w = _rand(d, seed=4)
    rstd = norm(x, w).rstd
    return lambda: norm.backward(dy, x, rstd, w, d_sum=ds if with_sum else None)


def _norm_codes(block):
    norm, x = vsa.RMSNorm(1, 1, 200, 128, quantize=block), _rand(1, 1, 200, 128)
    return lambda: norm(x)


@pytest.mark.parametrize("what", ["norm gradient", "norm codes", "attention gradient", "attention"])
def test_threads_launch_one_kernel_in_unlike_sizes(what):
    """Launches of one kernel with more and with less shared memory, from two threads at a time, all start."""
    make = {"norm gradient": lambda: [_norm_gradient(1536, False), _norm_gradient(1536, True)],
            "norm codes": lambda: [_norm_codes(64), _norm_codes(128)],
            "attention gradient": lambda: [_attention(2, True), _attention(4000, True)],
            "attention": lambda: [_attention(2, False), _attention(4000, False)]}[what]
    assert _at_once(make() + make(), 3000) == []


@pytest.mark.parametrize("byte", [9, 2])
@pytest.mark.parametrize("dtype,layout", [(BF, False), (BF, True), (F32, False)])
def test_call_with_unknown_kinds(dtype, layout, byte):
    """A head of unknown kind (a cube head without cubes among them): the error bit, a zero output that sees nothing and
    zero gradients, and the other head as without it."""
    plan, q, k, v, do = _small(dtype=dtype, layout_in_kernel=layout)
    good, bad = (torch.tensor(x, dtype=torch.uint8, device="cuda") for x in ([T_, S_], [T_, byte]))
    o, lse = plan(q, k, v, kinds=good)
    want = plan.backward(do, q, k, v, o, lse, kinds=good)
    assert plan.device_error() == 0
    plan.ws.fill_(0x41)                            # rows of earlier calls are not zeros
    plan.ws_bwd.fill_(0x41)
    o2, lse2, o_lo = torch.full_like(o, 5.0), torch.full_like(lse, 5.0), torch.full_like(o, 5.0)
    for lo in (None, o_lo):
        plan(q, k, v, out=o2.fill_(5.0), lse=lse2.fill_(5.0), kinds=bad, o_lo=lo)
        assert plan.device_error() & _lib.VSA_DEVERR_KIND
        plan.clear_error()
        assert torch.equal(o2[:, 0], o[:, 0]) and torch.equal(lse2[:, 0], lse[:, 0])
        assert (o2[:, 1] == 0).all() and (lse2[:, 1] == -torch.inf).all() and (lo is None or (lo[:, 1] == 0).all())
    grads = plan.backward(do, q, k, v, o, lse, kinds=bad, out=[torch.full_like(q, 9.0) for _ in range(3)])
    assert plan.device_error() & _lib.VSA_DEVERR_KIND
    for a, b in zip(grads, want):
        assert (a[:, 1] == 0).all() and torch.equal(a[:, 0], b[:, 0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_arguments_off_16_bytes(dtype):
    """A gradient that is a slice (as behind torch.cat), a weight out of one flat buffer: the bits of copies."""
    B, H, N, d = 1, 1, 5, 7
    norm = vsa.RMSNorm(B, H, N, d, dtype=dtype, with_grad=True)
    x, res = (_rand(B, H, N, d, seed=s, dtype=dtype).requires_grad_() for s in (1, 2))
    flat, go = _rand(d + 1, seed=3, dtype=dtype).requires_grad_(), _rand(5 * B, H, N, d, seed=4, dtype=dtype)
    w = flat[1:]
    assert w.data_ptr() % 16
    y, s = norm.normalise(x, w, res)
    z = norm.normalise(x, w)
    got = torch.autograd.grad(torch.cat([z, y, s, y, y]), (x, flat, res), go)
    w2 = w.detach().clone().requires_grad_()
    y, s = norm.normalise(x, w2, res)
    z = norm.normalise(x, w2)
    loss = [(z, go[:1].clone()), (y, go[1:2] + go[3:4] + go[4:5]), (s, go[2:3].clone())]
    want = torch.autograd.grad([a for a, _ in loss], (x, w2, res), [b for _, b in loss])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1][1:], want[1]) and torch.equal(got[2], want[2])
    # the calls themselves
    odd = torch.cat([go.flatten()[:1], go.flatten()])[1:].view(go.shape)
    r = norm(x.detach(), w.detach(), residual=res.detach())
    rstd = torch.cat([r.rstd.flatten()[:1], r.rstd.flatten()])[1:].view(r.rstd.shape)
    dx, dw = norm.backward(odd[1:2], r.sum, rstd, w.detach(), d_sum=odd[2:3])
    want = norm.backward(go[1:2].clone(), r.sum, r.rstd, w2.detach(), d_sum=go[2:3].clone())
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])


def test_attention_gradient_off_16_bytes():
    """The gradient of an output that went into one flat tensor behind a single element."""
    plan, q, k, v, do = _small()
    kinds = torch.tensor([S_, T_], dtype=torch.uint8, device="cuda")
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    one = torch.zeros(1, dtype=BF, device="cuda", requires_grad=True)
    o = plan.attend(*leaves, kinds=kinds)
    got = torch.autograd.grad(torch.cat([one, o.flatten()]), leaves, torch.cat([one.detach(), do.flatten()]))
    want = torch.autograd.grad(plan.attend(*leaves, kinds=kinds), leaves, do)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_attend_keeps_nothing_where_no_gradient_is_recorded(monkeypatch):
    plan, q, k, v, _ = _small()
    kinds = torch.tensor([S_, T_], dtype=torch.uint8, device="cuda")
    want = plan(q, k, v, kinds=kinds)[0]
    leaf = q.clone().requires_grad_()

    def refuse(*a, **kw):
        raise AssertionError("the rounding errors were asked for")

    monkeypatch.setattr(vsa, "vsa_attention_train", refuse)
    assert torch.equal(plan.attend(q, k, v, kinds=kinds), want)
    with torch.no_grad():
        o = plan.attend(leaf, k, v, kinds=kinds)
    assert torch.equal(o, want) and not o.requires_grad
    with pytest.raises(AssertionError):
        plan.attend(leaf, k, v, kinds=kinds)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [128, 129, 1536, 16384])
def test_norm_gradient_of_tiny_rows(d, dtype):
    """Rows of 1e-18 without an eps: 1 / rms squared times the sums of a row is beyond the floats, the gradient is not."""
    norm = vsa.RMSNorm(1, 1, 4, d, dtype=dtype, eps=0.0, with_grad=True)
    x, w = (_rand(1, 1, 4, d, seed=1, dtype=F32) * 1e-18).to(dtype), _rand(d, seed=2, dtype=F32)
    dy, ds = (100 * _rand(1, 1, 4, d, seed=3, dtype=F32)).to(dtype), _rand(1, 1, 4, d, seed=4, dtype=dtype)
    dy[0, 0, 1] = 100 * (x[0, 0, 1].float() * 1e18).to(dtype)            # all of it along the row: it nearly cancels
    rstd = norm(x, w).rstd
    s, r, g = x.double(), rstd.double()[..., None], dy.double() * w.double()
    mean = (g * s * r).mean(3, keepdim=True)
    want = r * (g - s * r * mean) + ds.double()
    # as in the norm's own tests: fp32 errors of 2^-18 against the terms, and the rounding of the result
    terms = r * (g.abs() + (s * r).abs() * (g * s * r).abs().mean(3, keepdim=True)) + ds.double().abs()
    dx, _ = norm.backward(dy, x, rstd, w, d_sum=ds)
    assert bool(((dx.double() - want).abs() <= terms * 2.0 ** -18 + want.abs() * torch.finfo(dtype).eps / 2).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_call_of_heads_of_every_kind(dtype):
    """Spatial, temporal and cube heads in one call: heads of N and of R rows, blocks past a head's last."""
    H, F, Hl, Wl, d = 3, 5, 7, 9, 64 if dtype == F32 else 128
    wl = synthetic.Workload("m", 1, H, F, Hl, Wl, d, 128, "bf16" if dtype == BF else "f32", "given", topk=2)
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl))
    do, d_lse = _rand(*q.shape, seed=9, dtype=dtype), _rand(*q.shape[:3], seed=8, dtype=F32)
    kinds = torch.tensor([S_, T_, C_], dtype=torch.uint8, device="cuda")
    plan = vsa.SparseAttention(1, H, F, Hl, Wl, d, 128, dtype=dtype, select="given", w_s=0, w_t=13, topk=2, cube=wl.cube, with_grad=True)
    o_lo = torch.full_like(q, 7.0)
    o, lse = plan(q, k, v, kinds=kinds, o_lo=o_lo)
    grads = plan.backward(do, q, k, v, o, lse, kinds=kinds, d_lse=d_lse)
    exact = plan.backward(do, q, k, v, o, lse, kinds=kinds, d_lse=d_lse, o_lo=o_lo)
    assert plan.device_error() == 0
    for h, kind in enumerate([S_, T_, C_]):
        q16, k16, v16, do16, o16 = (x[0, h].to(BF) for x in (q, k, v, do, o))
        al = allowed_blocks(keep_for_head(kind, wl, 0, 13, q16.cpu(), k16.cpu()), oracle.layout_slots(kind, F, Hl, Wl, wl.cube), 128).cuda()
        assert not al.all()
        _, _, want, bounds = reference(q16, k16, v16, do16, al, o=o16, lse=lse[0, h], d_lse=d_lse[0, h])
        assert_grads([g[0, h] for g in grads], want, bounds, f"kind {kind}")
        _, _, want, bounds = reference(q16, k16, v16, do16, al, d_lse=d_lse[0, h], own_o=True)
        assert_grads([g[0, h] for g in exact], want, [1.1 * x for x in bounds], f"exact: kind {kind}")


@pytest.mark.parametrize("lo", [False, True])
def test_lists_with_a_set_for_each_layout(lo):
    """Spatial heads from the natural set, the others from the permuted one, each set with its own O, log-sum-exp, their
    gradients and O's rounding errors; what a head does not use is NaN and stays as it is."""
    H, F, Hl, Wl, d, nan = 3, 5, 7, 9, 128, float("nan")
    wl = synthetic.Workload("m", 1, H, F, Hl, Wl, d, 128, "bf16", "given", topk=2)
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl))
    do, d_lse = _rand(*q.shape, seed=9), _rand(*q.shape[:3], seed=8, dtype=F32)
    kinds_list = [T_, S_, C_]
    kinds, err = torch.tensor(kinds_list, dtype=torch.uint8, device="cuda"), cuda_err()
    shape = _lib.make_shape(1, H, F, Hl, Wl, d, 128, wl.cube)
    R, nblk = _lib.vsa_layout_rows(shape), _lib.vsa_num_blocks(shape)
    assert R > wl.N
    idx, cnt = np.full((1, H, nblk, nblk), -1, np.int32), np.zeros((1, H, nblk), np.int32)
    o, o_lo, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(1, H, wl.N, device="cuda")
    masks, slots = [], []
    for h, kind in enumerate(kinds_list):
        keep = keep_for_head(kind, wl, 0, 13, q[0, h].cpu(), k[0, h].cpu())
        i, c = oracle.keep_to_lists(keep, nblk)
        idx[0, h, :keep.shape[0]], cnt[0, h, :keep.shape[0]] = i, c
        slots.append(torch.as_tensor(oracle.layout_slots(kind, F, Hl, Wl, wl.cube)).long().cuda())
        masks.append(allowed_blocks(keep, slots[h].cpu(), 128).cuda())
        o64, l64, _, _ = reference(q[0, h], k[0, h], v[0, h], do[0, h], masks[h])
        o[0, h], lse[0, h] = o64.to(BF), l64.float()
        o_lo[0, h] = (o64 - o[0, h].double()).to(BF)
    idx, cnt = torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda()

    def sets(x):
        nat, perm = torch.full_like(x, nan), torch.full((1, H, R, *x.shape[3:]), nan, dtype=x.dtype, device="cuda")
        for h, kind in enumerate(kinds_list):
            if kind == S_:
                nat[0, h] = x[0, h]
            else:
                perm[0, h] = 0
                perm[0, h, slots[h]] = x[0, h]
        return nat, perm

    both = [sets(x) for x in (q, k, v, o, do, lse)]
    dl, rest = sets(d_lse), sets(o_lo)
    grads = [(torch.full_like(q, 9.0), torch.full((1, H, R, d), 9.0, dtype=BF, device="cuda")) for _ in range(3)]
    nat, perm = (_lib.qkvo_grad(*(x[i] for x in both), *(x[i] for x in grads), d_lse=dl[i], o_lo=rest[i] if lo else None) for i in (0, 1))
    ws = torch.full((_lib.vsa_sparse_attn_bwd_workspace_size(shape),), 0x7f, dtype=torch.uint8, device="cuda")
    _lib.vsa_sparse_attn_bwd(nat, perm, kinds, idx, cnt, nblk, shape, 0.0, ws, ws.numel(), err)
    assert _lib.vsa_get_device_error(err) == 0
    for h, kind in enumerate(kinds_list):
        used = kind != S_
        got = [g[used][0, h][slots[h]] if used else g[0][0, h] for g in grads]
        args = (q[0, h], k[0, h], v[0, h], do[0, h], masks[h])
        if lo:
            # o + o_lo is the exact O but for half a step of o_lo, far below P_REL of it
            _, _, want, bounds = reference(*args, d_lse=d_lse[0, h], own_o=True)
        else:
            _, _, want, bounds = reference(*args, o=o[0, h], lse=lse[0, h], d_lse=d_lse[0, h])
        assert_grads(got, want, [1.1 * x for x in bounds] if lo else bounds, f"kind {kind}")
        for g in grads:
            assert (g[not used][0, h] == 9).all()
            if kind == T_:                       # rows behind the head's last block are not its own
                assert (g[1][0, h, -(-wl.N // 128) * 128:] == 9).all() and (g[1][0, h, wl.N:-(-wl.N // 128) * 128] == 0).all()


def test_codes_of_blocks_with_infinities():
    """The exponent of the largest float and saturated codes for the infinities; the block's other values by it."""
    shape = _lib.make_shape(1, 1, 1, 1, 256, 128, 128)
    x = _rand(1, 1, 256, 128, seed=1)
    x[0, 0, 3, 5], x[0, 0, 4, 6], x[0, 0, 5, 7] = float("inf"), -float("inf"), 3e38
    codes, exps = torch.zeros(1, 1, 256, 128, dtype=torch.uint8, device="cuda"), torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    kinds, err = torch.zeros(1, dtype=torch.uint8, device="cuda"), cuda_err()
    _lib.vsa_quantize_fp8(x, None, kinds, shape, codes, exps, err)
    assert _lib.vsa_get_device_error(err) == 0 and exps[0, 0] == 120 and exps[0, 1] < 0
    v = codes.view(torch.float8_e4m3fn).float()
    # 3e38 = 225.7 * 2^120, and e4m3 steps by 16 there
    assert v[0, 0, 3, 5] == 448 and v[0, 0, 4, 6] == -448 and v[0, 0, 5, 7] == 224
    small = x[0, 0, :128].abs() < 1e30
    assert (v[0, 0, :128][small] == 0).all()      # all far below the smallest code


@pytest.mark.parametrize("which", ["sparse", "semantic"])
def test_given_outputs_are_checked(which):
    """An output or a log-sum-exp that is not whole rows of its type would be written over its neighbours."""
    if which == "sparse":
        plan, q, k, v, _ = _small()
        kw = dict(kinds=torch.tensor([S_, T_], dtype=torch.uint8, device="cuda"))
    else:
        plan, kw = vsa.SemanticAttention(1, 2, 5, 6, 10, 64, 64, cq=4, ck=4, iters=2, with_lse=True), {}
        q, k, v = (_rand(1, 2, 300, 64, seed=s) for s in range(3))
    longer, rows = torch.zeros(1, 2, 301, 64, dtype=BF, device="cuda"), torch.zeros(1, 2, 301, device="cuda")
    lse = torch.empty(1, 2, 300, device="cuda")
    for out in (longer[:, :, 1:], q.float(), longer, q.cpu()):
        with pytest.raises(ValueError, match="out"):
            plan(q, k, v, out=out, **kw)
    for bad in (rows[:, :, 1:], lse.double(), rows, lse.cpu()):
        with pytest.raises(ValueError, match="lse"):
            plan(q, k, v, lse=bad, **kw)
    o, _ = plan(q, k, v, **kw)
    out, l2 = plan(q, k, v, out=torch.empty_like(q), lse=lse, **kw)
    assert torch.equal(out, o) and l2 is lse
