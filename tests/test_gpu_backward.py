"""GPU checks of the attention's gradient (vsa_sparse_attn_bwd, vsa_attention_bwd, SparseAttention.backward
and attend) against 64-bit gradients of the same masks."""
import math

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

S_, T_, C_ = 0, 1, 2


def _rows(shape, seed, scale=1.0):
    return synthetic.make_random(shape, torch.bfloat16, seed=seed, scale=scale).cuda()


def _lists(keeps, nblk, max_kv=None):
    H = len(keeps)
    max_kv = max_kv or max(1, max(int(kp.sum(axis=1).max()) if kp.size else 0 for kp in keeps))
    idx = np.full((1, H, nblk, max_kv), -1, dtype=np.int32)
    cnt = np.zeros((1, H, nblk), dtype=np.int32)
    for h, kp in enumerate(keeps):
        i_, c_ = oracle.keep_to_lists(kp, max_kv)
        idx[0, h, :kp.shape[0]] = i_
        cnt[0, h, :kp.shape[0]] = c_
    return torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(), max_kv


def _run_lists(shape, q, k, v, do, o, lse, kinds, idx, cnt, max_kv, d_lse=None, scale=0.0):
    ws_bytes = _lib.vsa_sparse_attn_bwd_workspace_size(shape)
    ws = torch.full((ws_bytes,), 0x7f, dtype=torch.uint8, device="cuda")
    grads = [torch.full_like(q, 9.0) for _ in range(3)]
    err = cuda_err()
    _lib.vsa_sparse_attn_bwd(_lib.qkvo_grad(q, k, v, o, do, lse, *grads, d_lse=d_lse), None, kinds, idx, cnt, max_kv,
                             shape, scale, ws, ws_bytes, err)
    return grads, _lib.vsa_get_device_error(err)


def _case(N, H, d, block, keeps, q, k, v, do, d_lse=None, scale=0.0):
    """Natural-order heads on given block masks: O and LSE exact to their types."""
    shape = _lib.make_shape(1, H, 1, 1, N, d, block)
    nblk = _lib.vsa_num_blocks(shape)
    idx, cnt, max_kv = _lists(keeps, nblk)
    kinds = torch.zeros(H, dtype=torch.uint8, device="cuda")
    t = np.arange(N)
    o, lse = torch.empty_like(q), torch.empty(1, H, N, device="cuda")
    for h in range(H):
        al = allowed_blocks(keeps[h], t, block).cuda()
        o_, lse_, _, _ = reference(q[0, h], k[0, h], v[0, h], do[0, h], al, scale=scale or None)
        o[0, h], lse[0, h] = o_.to(torch.bfloat16), lse_.float()
    grads, err = _run_lists(shape, q, k, v, do, o, lse, kinds, idx, cnt, max_kv, d_lse, scale)
    assert err == 0
    for h in range(H):
        al = allowed_blocks(keeps[h], t, block).cuda()
        _, _, want, bounds = reference(q[0, h], k[0, h], v[0, h], do[0, h], al, scale=scale or None,
                                       d_lse=None if d_lse is None else d_lse[0, h], o=o[0, h], lse=lse[0, h])
        assert_grads([g[0, h] for g in grads], want, bounds, f"head {h}")
    return grads


def _qkvdo(N, H, d, seed=0, scale=1.0):
    return tuple(_rows((1, H, N, d), seed * 10 + i, scale if i < 2 else 1.0) for i in range(4))


@pytest.mark.parametrize("d,block", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("N", [1, 63, 64, 129, 300, 1111])
def test_dense_lengths(N, d, block):
    nb = -(-N // block)
    _case(N, 2, d, block, [np.ones((nb, nb), dtype=bool)] * 2, *_qkvdo(N, 2, d, seed=N))


@pytest.mark.parametrize("d,block", [(128, 128), (64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("share", [0.1, 0.6])
def test_random_lists(d, block, share):
    """Lists of every length: empty rows, key blocks that nothing keeps, a ragged last block."""
    N = 11 * block + 37
    nb = -(-N // block)
    rng = np.random.default_rng(3)
    keeps = [rng.random((nb, nb)) < share for _ in range(3)]
    keeps[0][2] = False
    keeps[0][:, 5] = False
    keeps[1][:] = False                       # a head that keeps nothing: zeros
    keeps[2][-1] = True
    grads = _case(N, 3, d, block, keeps, *_qkvdo(N, 3, d, seed=1))
    assert all((g[0, 1] == 0).all() for g in grads)
    assert (grads[0][0, 0, 2 * block:3 * block] == 0).all()
    assert (grads[1][0, 0, 5 * block:6 * block] == 0).all() and (grads[2][0, 0, 5 * block:6 * block] == 0).all()


def test_peaked_and_far_scores():
    """Scores of some hundreds: the probabilities underflow nearly everywhere; and rows whose every score
    is far below zero, with a ragged tail whose zero rows would score above all of them."""
    N, d = 200, 128
    keeps = [np.ones((2, 2), dtype=bool)]
    q, k, v, do = _qkvdo(N, 1, d, seed=2, scale=6.0)
    _case(N, 1, d, 128, keeps, q, k, v, do)
    q, k = q * 0 + 4, -(k.abs() * 0.02 + 4).to(torch.bfloat16)
    _case(N, 1, d, 128, keeps, q.contiguous(), k.contiguous(), v, do)


def test_lse_gradient_and_scale():
    N, d = 300, 64
    q, k, v, do = _qkvdo(N, 2, d, seed=4)
    d_lse = torch.randn(1, 2, N, generator=torch.Generator().manual_seed(1)).cuda()
    _case(N, 2, d, 64, [np.tri(5, dtype=bool)] * 2, q, k, v, do, d_lse=d_lse, scale=0.3)


def test_heads_of_many_blocks():
    """More than 32 and more than 64 blocks a head: several words of every bitset."""
    N, d = 70 * 64 - 5, 64
    rng = np.random.default_rng(0)
    _case(N, 1, d, 64, [rng.random((70, 70)) < 0.3], *_qkvdo(N, 1, d, seed=5))


def test_two_runs_give_the_same_bits():
    N, d = 2000, 128
    rng = np.random.default_rng(1)
    args = (N, 2, d, 128, [rng.random((16, 16)) < 0.7 for _ in range(2)], *_qkvdo(N, 2, d, seed=6))
    for a, b in zip(_case(*args), _case(*args)):
        assert torch.equal(a, b)


def test_bad_lists_and_kinds():
    N, d = 256, 64
    q, k, v, do = _qkvdo(N, 2, d, seed=7)
    shape = _lib.make_shape(1, 2, 1, 1, N, d, 64)
    o, lse = torch.zeros_like(q), torch.zeros(1, 2, N, device="cuda")
    kinds = torch.zeros(2, dtype=torch.uint8, device="cuda")
    good = [[0, 1], [1, 2], [2, -1], [3, -1]]
    for bad, cnt in (([[0, 1], [1, 9], [2, -1], [3, -1]], [2, 2, 1, 1]), ([[1, 0], [1, 2], [2, -1], [3, -1]], [2, 2, 1, 1]),
                     (good, [2, 3, 1, 1]), (good, [-1, 2, 1, 1]), ([[-2, 1], [1, 2], [2, 1], [3, -1]], [2, 2, 1, 1])):
        idx = torch.tensor([bad, good], dtype=torch.int32, device="cuda")
        c = torch.tensor([cnt, [2, 2, 1, 1]], dtype=torch.int32, device="cuda")
        grads, err = _run_lists(shape, q, k, v, do, o, lse, kinds, idx, c, 2)
        assert err & _lib.VSA_DEVERR_KV_RANGE
        first = 0 if bad[0] != good[0] or cnt[0] < 0 else 1
        assert (grads[0][0, 0, first * 64:(first + 1) * 64] == 0).all()
        assert all(torch.isfinite(g).all() for g in grads)
    idx = torch.tensor([good, good], dtype=torch.int32, device="cuda")
    c = torch.tensor([[2, 2, 1, 1]] * 2, dtype=torch.int32, device="cuda")
    for byte in (9, 2):
        kinds[1] = byte
        grads, err = _run_lists(shape, q, k, v, do, o, lse, kinds, idx, c, 2)
        assert err & _lib.VSA_DEVERR_KIND
        assert all((g[0, 1] == 0).all() and (g[0, 0] != 0).any() for g in grads)


# ------------------------------------------------------------------------------------
# the whole call
# ------------------------------------------------------------------------------------
def _plan_case(plan, wl, kinds_list, q, k, v, do, kinds=None, d_lse=None, lo=False):
    """plan(q, k, v), then its gradients against 64 bits: with the call's own O and LSE, or (lo) with what O's
    rounding left over against the gradient of the exact attention too."""
    o_lo = torch.full_like(q, 7.0) if lo else None
    o, lse = plan(q, k, v, kinds=kinds, o_lo=o_lo)
    plain = plan(q, k, v, kinds=kinds)
    assert torch.equal(o, plain[0]) and torch.equal(lse, plain[1])
    grads = plan.backward(do, q, k, v, o, lse, kinds=kinds if kinds is not None else plan.kinds, d_lse=d_lse, o_lo=o_lo)
    assert plan.device_error() == 0
    for b in range(wl.B):
        for h, kind in enumerate(kinds_list):
            slots = oracle.layout_slots(kind, wl.F, wl.Hl, wl.Wl, wl.cube)
            q16, k16, v16, do16, o16 = (x[b, h].to(torch.bfloat16) for x in (q, k, v, do, o))
            keep = keep_for_head(kind, wl, plan.w_s, plan.w_t, q16.cpu(), k16.cpu())
            al = allowed_blocks(keep, slots, wl.block).cuda()
            dl = None if d_lse is None else d_lse[b, h]
            o64 = o16.double() + (o_lo[b, h].double() if lo else 0.0)
            _, _, want, bounds = reference(q16, k16, v16, do16, al, o=o64, lse=lse[b, h], d_lse=dl)
            # with o_lo the kernel holds the rows' sums of dS to d_lse: dq is that of the exact delta, not of o + o_lo,
            # which still has the forward call's rounding of P in it
            first = 1 if lo else 0
            assert_grads([g[b, h] for g in grads[first:]], want[first:], bounds[first:], f"batch {b} head {h} kind {kind}",
                         ("dq", "dk", "dv")[first:])
            if lo:
                # the rest is smaller than half a step of what it was left over from
                assert bool((o_lo[b, h].double().abs() <= o16.double().abs() * 2.0 ** -8 + 2.0 ** -133).all())
                # lse is the kernel's: within 2^-12 + 2^-20 |lse| of the exact one, an error of P like that of its own
                _, _, want, bounds = reference(q16, k16, v16, do16, al, d_lse=dl, own_o=True)
                assert_grads([g[b, h] for g in grads], want, [1.1 * x for x in bounds], f"exact: batch {b} head {h} kind {kind}")
    return o, lse, grads


@pytest.mark.parametrize("F,Hl,Wl,d,block,dtype", [(6, 8, 16, 128, 128, torch.bfloat16), (5, 6, 10, 64, 64, torch.bfloat16),
                                                   (7, 5, 9, 128, 64, torch.bfloat16), (4, 8, 8, 64, 64, torch.float32),
                                                   (9, 7, 11, 64, 128, torch.float32)])
def test_call_pattern_heads(F, Hl, Wl, d, block, dtype):
    wl = synthetic.Workload("b", 2, 2, F, Hl, Wl, d, block, "bf16" if dtype == torch.bfloat16 else "f32", "given")
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl))
    do = synthetic.make_random(q.shape, dtype, seed=9).cuda()
    d_lse = synthetic.make_random(q.shape[:3], torch.float32, seed=8).cuda()
    kinds = torch.tensor([S_, T_, S_, T_], dtype=torch.uint8, device="cuda")
    for layout in (False, True):
        plan = vsa.SparseAttention(2, 2, F, Hl, Wl, d, block, dtype=dtype, select="given", w_s=1, w_t=9, with_grad=True,
                                   layout_in_kernel=layout)
        _plan_case(plan, wl, [S_, T_], q, k, v, do, kinds=kinds, d_lse=d_lse)
        _plan_case(plan, wl, [S_, T_], q, k, v, do, kinds=kinds, lo=True)
        _plan_case(plan, wl, [S_, T_], q, k, v, do, kinds=kinds, d_lse=d_lse, lo=True)


@pytest.mark.parametrize("F,Hl,Wl,topk", [(5, 5, 9, 3), (9, 9, 17, 4), (4, 4, 8, 2)])
def test_call_cube_heads(F, Hl, Wl, topk):
    wl = synthetic.Workload("c", 1, 2, F, Hl, Wl, 128, 128, "bf16", "cube", topk=topk)
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl))
    do = _rows(q.shape, 11)
    plan = vsa.SparseAttention(1, 2, F, Hl, Wl, 128, 128, select="cube", topk=topk, cube=(4, 4, 8), with_grad=True)
    _plan_case(plan, wl, [C_, C_], q, k, v, do)
    _plan_case(plan, wl, [C_, C_], q, k, v, do, lo=True)


def test_call_profiled_heads():
    wl = synthetic.Workload("p", 1, 4, 6, 8, 16, 128, 128, "bf16", "profiled")
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl))
    plan = vsa.SparseAttention(1, 4, 6, 8, 16, 128, 128, select="profile", target=0.4, profile_frac=0.05, with_grad=True)
    plan(q, k, v)
    _plan_case(plan, wl, plan.kinds.tolist(), q, k, v, _rows(q.shape, 12))


def test_attend_matches_backward_and_differences():
    """autograd's gradients are backward's, and agree with differences of a 64-bit forward."""
    wl = synthetic.Workload("a", 1, 2, 4, 6, 8, 64, 64, "bf16", "given")
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl.with_(structure_scale=0.3)))
    kinds = torch.tensor([S_, T_], dtype=torch.uint8, device="cuda")
    plan = vsa.SparseAttention(1, 2, 4, 6, 8, 64, 64, select="given", w_s=1, w_t=11, with_grad=True)
    do = _rows(q.shape, 13)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = plan.attend(*leaves, kinds=kinds)
    other = plan.attend(*(x * 0.5 for x in (q, k, v)), kinds=1 - kinds)     # another call comes between
    o.backward(do)
    o2, lse, grads = _plan_case(plan, wl, [S_, T_], q, k, v, do, kinds=kinds, lo=True)
    assert torch.equal(o.detach(), o2) and other.shape == o.shape
    for x, g in zip(leaves, grads):
        assert torch.equal(x.grad, g)
    # only what is asked for, and a gradient that comes expanded
    vv = v.clone().requires_grad_()
    plan.attend(q, k, vv, kinds=kinds).sum().backward()
    assert torch.equal(vv.grad, plan.backward(torch.ones_like(o2), q, k, v, o2, lse, kinds=kinds)[2])   # dv: no delta

    def loss(h, x, y, z):
        keep = keep_for_head([S_, T_][h], wl, 1, 11)
        al = allowed_blocks(keep, oracle.layout_slots(h, 4, 6, 8), 64).cuda()
        s = (x @ y.T / 8).masked_fill(~al, -math.inf)
        return float((torch.softmax(s, 1) @ z * do[0, h].double()).sum())

    g = torch.Generator("cuda").manual_seed(5)
    for h in range(2):
        x = [t[0, h].double() for t in (q, k, v)]
        for i in range(3):
            u = torch.randn(x[0].shape, generator=g, device="cuda", dtype=torch.float64)
            e = 1e-5
            up, down = [list(x), list(x)]
            up[i], down[i] = x[i] + e * u, x[i] - e * u
            slope = (loss(h, *up) - loss(h, *down)) / (2 * e)
            al = allowed_blocks(keep_for_head([S_, T_][h], wl, 1, 11), oracle.layout_slots(h, 4, 6, 8), 64).cuda()
            _, _, _, bounds = reference(q[0, h], k[0, h], v[0, h], do[0, h], al, own_o=True)
            room = 1.1 * float((bounds[i] * u.abs()).sum())
            assert abs(slope - float((grads[i][0, h].double() * u).sum())) <= room


def test_captured_and_replayed():
    """The call and its gradient in one graph, replayed on new inputs; autograd is refused there."""
    wl = synthetic.Workload("g", 1, 2, 5, 6, 10, 128, 128, "bf16", "given")
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl))
    do = _rows(q.shape, 14)
    kinds = torch.tensor([S_, T_], dtype=torch.uint8, device="cuda")
    plan = vsa.SparseAttention(1, 2, 5, 6, 10, 128, 128, select="given", w_s=1, w_t=9, with_grad=True)
    o, lse = plan(q, k, v, kinds=kinds)
    outs = tuple(torch.empty_like(q) for _ in range(3))
    plan.backward(do, q, k, v, o, lse, kinds=kinds, out=outs)
    leaf = q.clone().requires_grad_()
    eager = plan.attend(leaf, k, v, kinds=kinds)              # an eager graph of the leaf lives on
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan(q, k, v, out=o, lse=lse, kinds=kinds)
        plan.backward(do, q, k, v, o, lse, kinds=kinds, out=outs)
        with pytest.raises(RuntimeError, match="cannot be captured"):
            plan.attend(leaf, k, v, kinds=kinds)
    eager.sum().backward()
    for seed in (20, 21):
        q.copy_(_rows(q.shape, seed))
        do.copy_(_rows(q.shape, seed + 5))
        graph.replay()
        got = [x.clone() for x in (o, *outs)]
        want_o, want_lse = plan(q, k, v, kinds=kinds)
        want = plan.backward(do, q, k, v, want_o, want_lse, kinds=kinds)
        for a, b in zip(got, (want_o, *want)):
            assert torch.equal(a, b)


def test_on_another_stream():
    wl = synthetic.Workload("s", 1, 2, 5, 6, 10, 128, 128, "bf16", "given")
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl))
    do = _rows(q.shape, 15)
    kinds = torch.tensor([S_, T_], dtype=torch.uint8, device="cuda")
    plan = vsa.SparseAttention(1, 2, 5, 6, 10, 128, 128, select="given", w_s=1, w_t=9, with_grad=True)
    o, lse = plan(q, k, v, kinds=kinds)
    want = plan.backward(do, q, k, v, o, lse, kinds=kinds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        got = plan.backward(do, q, k, v, o, lse, kinds=kinds, stream=stream)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("d,block", [(128, 128), (64, 64)])
def test_very_long_head(d, block):
    """So many blocks that the bitset takes a ring stage's place; a few blocks a list, near and far."""
    nb = 5700
    N = nb * block - 13
    shape = _lib.make_shape(1, 1, 1, 1, N, d, block)
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v, do = (torch.randn(1, 1, N, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4))
    i = torch.arange(nb, device="cuda")
    idx = torch.stack([i, (i * 7 + 3) % nb, (nb - 1 - i)], 1).sort(1).values
    dup = torch.cat([torch.zeros(nb, 1, dtype=torch.bool, device="cuda"), idx[:, 1:] == idx[:, :-1]], 1)
    idx = torch.where(dup, nb + 1, idx).sort(1).values
    cnt = (idx < nb).sum(1).to(torch.int32).contiguous()
    idx = torch.where(idx < nb, idx, -1).to(torch.int32).contiguous()
    kinds = torch.zeros(1, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(1, 1, N, device="cuda")
    err = cuda_err()
    _lib.vsa_sparse_attn_fwd(_lib.qkvo(q, k, v, o, lse), None, kinds, idx, cnt, 3, shape, 0.0, err)
    grads, e = _run_lists(shape, q, k, v, do, o, lse, kinds, idx, cnt, 3)
    assert e == 0 and _lib.vsa_get_device_error(err) == 0
    lists = [x[x >= 0].tolist() for x in idx.cpu()]
    for b in (0, 1, 2849, 2850, 5631, 5632, 5698, 5699):
        # every query block that keeps b or is b, every key block that these keep
        rows = sorted({b} | {j for j, x in enumerate(lists) if b in x})
        keys = sorted({x for j in rows for x in lists[j]})
        at = lambda bs: torch.cat([torch.arange(x * block, min(N, (x + 1) * block)) for x in bs]).cuda()  # noqa: E731
        qi, ki = at(rows), at(keys)
        al = torch.tensor([[x in lists[j] for x in keys] for j in rows])
        al = al.cuda()[torch.searchsorted(torch.tensor(rows).cuda(), qi // block)][:, torch.searchsorted(torch.tensor(keys).cuda(), ki // block)]
        _, _, want, bounds = reference(q[0, 0, qi], k[0, 0, ki], v[0, 0, ki], do[0, 0, qi], al, o=o[0, 0, qi], lse=lse[0, 0, qi])
        mine, key = qi // block == b, ki // block == b
        pick = (mine, key, key)
        assert_grads([grads[0][0, 0, qi][mine], grads[1][0, 0, ki][key], grads[2][0, 0, ki][key]],
                     [w[m] for w, m in zip(want, pick)], [w[m] for w, m in zip(bounds, pick)], f"block {b}")


def test_offsets_past_32_bits():
    """More than 2^31 elements a tensor: the last head is computed as the same head alone."""
    H, N, d = 142, 118800, 128
    assert H * N * d > 1 << 31
    nb = -(-N // 128)
    shape, one = (_lib.make_shape(1, h, 1, 1, N, d, 128) for h in (H, 1))
    idx = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, 1, nb, 1).repeat(1, H, 1, 1)
    cnt = torch.ones(1, H, nb, dtype=torch.int32, device="cuda")
    kinds = torch.zeros(H, dtype=torch.uint8, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    full = [torch.zeros(1, H, N, d, dtype=torch.bfloat16, device="cuda") for _ in range(5)]
    last = [torch.randn(1, 1, N, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]
    lse = torch.zeros(1, H, N, device="cuda")
    o, l1 = torch.empty_like(last[0]), torch.empty(1, 1, N, device="cuda")
    err = cuda_err()
    _lib.vsa_sparse_attn_fwd(_lib.qkvo(*last[:3], o, l1), None, kinds[:1], idx[:, :1], cnt[:, :1], 1, one, 0.0, err)
    for t, x in zip(full, (*last, o)):
        t[:, -1:] = x
    lse[:, -1:] = l1
    q, k, v, do, ofull = full
    grads, e = _run_lists(shape, q, k, v, do, ofull, lse, kinds, idx, cnt, 1)
    want, e1 = _run_lists(one, *last, o, l1, kinds[:1], idx[:, :1].contiguous(), cnt[:, :1].contiguous(), 1)
    assert e == 0 and e1 == 0 and _lib.vsa_get_device_error(err) == 0
    for a, b in zip(grads, want):
        assert torch.equal(a[:, -1:], b) and bool((a[:, :3] == 0).all())


def test_semantic_layouts():
    """Query and key rows in orders of their own (the semantic permutation's steps): gather, lists, gradient, scatter."""
    H, N, d, C = 2, 700, 128, 12
    wl = synthetic.Workload("sem", 1, H, 5, 10, 14, d, 128, "bf16", "semantic")
    q, k, v = (x.cuda() for x in synthetic.make_qkv(wl))
    do = _rows(q.shape, 31)
    shape = _lib.make_shape(1, H, 5, 10, 14, d, 128)
    nblk, err = _lib.vsa_num_blocks(shape), cuda_err()
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.empty(max(_lib.vsa_kmeans_workspace_size(shape, C), _lib.vsa_semantic_mask_workspace_size(shape)), dtype=torch.uint8,
                     device="cuda")
    found = []
    for x in (q, k):
        f = (torch.empty(H, C, d, device="cuda"), i32(H, N), i32(H, C), i32(H, N))
        _lib.vsa_kmeans(x, shape, C, 3, *f, ws, ws.numel(), err)
        found.append(f)
    keep, bits, idx, cnt = i32(H, C, 1), i32(1, H, nblk, 1), i32(1, H, nblk, nblk), i32(1, H, nblk)
    (cq, lq, nq, pq), (ck, lk, nk, pk) = found
    _lib.vsa_semantic_mask(cq, nq, lq, pq, C, ck, nk, lk, pk, C, shape, 0.5, 0.0, keep, bits, idx, cnt, nblk, ws, ws.numel(), err)
    p = [torch.empty_like(q) for _ in range(8)]
    for src, perm, dst in ((q, pq, p[0]), (k, pk, p[1]), (v, pk, p[2]), (do, pq, p[3])):
        _lib.vsa_gather_rows(src, perm, dst, shape, err)
    lse = torch.empty(1, H, N, device="cuda")
    kinds = torch.ones(H, dtype=torch.uint8, device="cuda")
    _lib.vsa_sparse_attn_fwd(_lib.qkvo(*p[:3], p[4], lse), _lib.qkvo(*p[:3], p[4], lse), kinds, idx, cnt, nblk, shape, 0.0, err)
    bws = torch.empty(_lib.vsa_sparse_attn_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")
    s = _lib.qkvo_grad(p[0], p[1], p[2], p[4], p[3], lse, p[5], p[6], p[7])
    _lib.vsa_sparse_attn_bwd(s, s, kinds, idx, cnt, nblk, shape, 0.0, bws, bws.numel(), err)
    grads = [torch.empty_like(q) for _ in range(3)]
    for src, perm, dst in ((p[5], pq, grads[0]), (p[6], pk, grads[1]), (p[7], pk, grads[2])):
        _lib.vsa_scatter_rows(src, None, perm, dst, None, shape, err)
    assert _lib.vsa_get_device_error(err) == 0
    for h in range(H):
        slot_q, slot_k = pq[h].long().argsort(), pk[h].long().argsort()
        mask = torch.zeros(nblk, nblk, dtype=torch.bool, device="cuda")
        for i in range(nblk):
            mask[i, idx[0, h, i, :int(cnt[0, h, i])].long()] = True
        assert 0 < int(mask.sum()) < nblk * nblk
        al = allowed_blocks(mask, slot_q, 128, slot_k)
        _, _, want, bounds = reference(q[0, h], k[0, h], v[0, h], do[0, h], al, o=p[4][0, h][slot_q], lse=lse[0, h][slot_q])
        assert_grads([x[0, h] for x in grads], want, bounds, f"head {h}")


def test_refusals():
    q = torch.zeros(1, 2, 256, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(1, 2, 256, device="cuda")
    plan = vsa.SparseAttention(1, 2, 4, 8, 8, 64, 64, select="given", w_s=0, w_t=0, with_grad=True)
    kinds = torch.zeros(2, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="kinds"):
        plan.backward(q, q, q, q, q, lse)
    with pytest.raises(ValueError, match="2 kinds"):
        plan.backward(q, q, q, q, q, lse, kinds=kinds[:1])
    with pytest.raises(ValueError, match="contiguous"):
        plan.backward(q.transpose(1, 2).contiguous().transpose(1, 2), q, q, q, q, lse, kinds=kinds)
    with pytest.raises(ValueError, match="contiguous"):
        plan.backward(q.float(), q, q, q, q, lse, kinds=kinds)
    with pytest.raises(ValueError, match="lse"):
        plan.backward(q, q, q, q, q, lse.double(), kinds=kinds)
    with pytest.raises(ValueError, match="out"):
        plan.backward(q, q, q, q, q, lse, kinds=kinds, out=(q, q))
    with pytest.raises(vsa.VsaError):
        plan.backward(q, q, q, q, q, lse, kinds=kinds, out=(q, torch.empty_like(q), torch.empty_like(q)))
    with pytest.raises(ValueError, match="with_grad"):
        vsa.SparseAttention(1, 2, 4, 8, 8, 64, 64, select="given").backward(q, q, q, q, q, lse, kinds=kinds)
    with pytest.raises(ValueError, match="with_grad"):
        vsa.SparseAttention(1, 2, 4, 8, 8, 64, 64, select="given").attend(q, q, q, kinds=kinds)
    with pytest.raises(ValueError, match="o_lo"):
        vsa.SparseAttention(1, 2, 4, 8, 8, 64, 64, select="given")(q, q, q, kinds=kinds, o_lo=q)
    with pytest.raises(ValueError, match="contiguous"):
        plan.backward(q, q, q, q, q, lse, kinds=kinds, o_lo=q.float())
    with pytest.raises(ValueError, match="no gradient"):
        vsa.SparseAttention(1, 2, 4, 8, 8, 128, 128, select="given", qk_fp8=True, with_grad=True)
    # a host address is refused before any launch
    shape = _lib.make_shape(1, 2, 4, 8, 8, 64, 64)
    ws = torch.empty(_lib.vsa_sparse_attn_bwd_workspace_size(shape), dtype=torch.uint8, device="cuda")
    idx, cnt = torch.zeros(1, 2, 4, 1, dtype=torch.int32, device="cuda"), torch.ones(1, 2, 4, dtype=torch.int32, device="cuda")
    host = torch.zeros(1, 2, 256, 64, dtype=torch.bfloat16)
    with pytest.raises(vsa.VsaError) as ex:
        _lib.vsa_sparse_attn_bwd(_lib.qkvo_grad(q, q, q, q, q, lse, torch.empty_like(q), torch.empty_like(q), host), None, kinds, idx, cnt, 1, shape, 0.0, ws,
                                 ws.numel(), cuda_err())
    assert ex.value.status == _lib.VSA_ERR_INVALID_ARG
