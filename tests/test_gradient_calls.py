"""CPU checks of what the binding makes of the gradient's arguments.  No kernel runs: the library's entry point is
replaced by one that reads its arguments back."""
import ctypes
import weakref

import pytest
import torch

from block_sparse_attention_31_b200 import _lib

BF, F32 = torch.bfloat16, torch.float32


def _set(B=1, H=2, rows=256, d=64, dtype=BF, **kw):
    """Tensors of one gradient set, some of them replaced."""
    out = {n: torch.zeros(B, H, rows, d, dtype=dtype) for n in ("q", "k", "v", "o", "d_o", "dq", "dk", "dv")}
    out["lse"] = torch.arange(B * H * rows, dtype=F32).view(B, H, rows)
    return {**out, **kw}


def _at(address, n):
    return torch.tensor((ctypes.c_float * n).from_address(address)[:])


def _lists(monkeypatch, natural, permuted=None, shape=None, **kw):
    """vsa_sparse_attn_bwd on the sets; the log-sum-exps (and their gradients) as the library would read them."""
    shape = shape or _lib.make_shape(1, 2, 4, 8, 8, 64, 64)
    seen = []

    def entry(nat, perm, *rest):
        for s in (nat, perm):
            if s is not None:
                s = s._obj
                seen.append([None if p is None else _at(p, 512) for p in (s.lse, s.d_lse)])
        return _lib.VSA_OK

    monkeypatch.setattr(_lib.lib, "vsa_sparse_attn_bwd", entry)
    ws = torch.zeros(_lib.vsa_sparse_attn_bwd_workspace_size(shape), dtype=torch.uint8)
    args = dict(kinds=torch.zeros(2, dtype=torch.uint8), kv_idx=torch.zeros(1, 2, 4, 1, dtype=torch.int32),
                kv_cnt=torch.ones(1, 2, 4, dtype=torch.int32), max_kv=1, shape=shape, scale=0.0, ws=ws, ws_bytes=ws.numel(),
                err=torch.zeros(1, dtype=torch.int32), stream=0)
    _lib.vsa_sparse_attn_bwd(natural, permuted, **{**args, **kw})
    return seen


def test_log_sum_exp_is_read_in_whole_rows(monkeypatch):
    """Rows cut out of longer ones, in another order of dimensions, or off 16 bytes: the library sees whole rows."""
    t = _set()
    want, d_lse = t["lse"].flatten(), torch.randn(1, 2, 256)
    longer = torch.full((2, 257), -1.0)
    longer[:, :256] = t["lse"][0]
    other = t["lse"].transpose(1, 2).contiguous().transpose(1, 2)
    off = torch.cat([torch.zeros(1), want])[1:]
    for lse in (t["lse"], longer[:, :256], longer[None, :, :256], other, off):
        for both in (False, True):
            s = _lib.qkvo_grad(**{**t, "lse": lse}, d_lse=d_lse)
            for got in _lists(monkeypatch, s, s if both else None):
                assert torch.equal(got[0], want) and torch.equal(got[1], d_lse.flatten())
    # the set itself keeps the tensors it was made of
    assert s.lse == off.data_ptr()
    # addresses pass as they are
    s = _lib.qkvo_grad(**{**t, "lse": t["lse"].data_ptr()})
    assert torch.equal(_lists(monkeypatch, s)[0][0], want)


def _strided(t):
    return t.transpose(0, -1).contiguous().transpose(0, -1)


@pytest.mark.parametrize("name", ["q", "k", "v", "o", "d_o", "dq", "dk", "dv", "o_lo"])
def test_lists_refuse_what_would_be_read_as_something_else(monkeypatch, name):
    """Tensors of another type, size or order of elements, in either set."""
    good = {**_set(), "o_lo": torch.zeros(1, 2, 256, 64, dtype=BF)}
    for bad in (good[name].float(), good[name][:, :1], _strided(good[name]), torch.zeros(1, 2, 320, 64, dtype=BF)):
        with pytest.raises(ValueError, match="natural set"):
            _lists(monkeypatch, _lib.qkvo_grad(**{**good, name: bad}))
        with pytest.raises(ValueError, match="permuted set"):
            _lists(monkeypatch, _lib.qkvo_grad(**good), _lib.qkvo_grad(**{**good, name: bad}))
    _lists(monkeypatch, _lib.qkvo_grad(**good), _lib.qkvo_grad(**good))


def test_lists_refuse_masks_and_scratch_of_another_form(monkeypatch):
    s = _lib.qkvo_grad(**_set())
    ok = dict(kinds=torch.zeros(2, dtype=torch.uint8), kv_idx=torch.zeros(1, 2, 4, 1, dtype=torch.int32),
              kv_cnt=torch.ones(1, 2, 4, dtype=torch.int32), err=torch.zeros(1, dtype=torch.int32))
    for name, t in ok.items():
        for bad in (t.long(), t.repeat(*[1] * (t.dim() - 1), 2)[..., ::2] if name != "err" else t[:0]):
            with pytest.raises(ValueError):
                _lists(monkeypatch, s, **{name: bad})
    with pytest.raises(ValueError, match="kv_idx"):
        _lists(monkeypatch, s, max_kv=2)                          # lists of one block
    with pytest.raises(ValueError, match="workspace"):
        _lists(monkeypatch, s, ws=torch.zeros(100, dtype=torch.uint8), ws_bytes=1 << 20)
    for bad in (_set()["lse"].double(), torch.zeros(1, 2, 255), torch.zeros(1, 2, 256, dtype=BF)):
        with pytest.raises(ValueError, match="lse"):
            _lists(monkeypatch, _lib.qkvo_grad(**{**_set(), "lse": bad}))
        with pytest.raises(ValueError, match="lse"):
            _lists(monkeypatch, _lib.qkvo_grad(**_set(), d_lse=bad))
    # a set of its own rows for each layout: 2 cubes of 128 slots for 4 x 4 x 9 tokens
    shape = _lib.make_shape(1, 2, 4, 4, 9, 64, 128, (4, 4, 8))
    lists = dict(kv_idx=torch.zeros(1, 2, 2, 1, dtype=torch.int32), kv_cnt=torch.ones(1, 2, 2, dtype=torch.int32))
    nat, perm = (_lib.qkvo_grad(**{k: v.data_ptr() if k == "lse" else v for k, v in _set(rows=n).items()}) for n in (144, 256))
    _lists(monkeypatch, nat, perm, shape, **lists)
    _lists(monkeypatch, perm, None, shape, **lists)
    for a, b in ((perm, perm), (nat, nat), (nat, None)):
        with pytest.raises(ValueError, match="set"):
            _lists(monkeypatch, a, b, shape, **lists)


@pytest.mark.parametrize("dtype,code", [(BF, _lib.VSA_BF16), (F32, _lib.VSA_F32)])
def test_calls_refuse_what_would_be_read_as_something_else(monkeypatch, dtype, code):
    """vsa_attention_train and vsa_attention_bwd: natural rows in the call's type."""
    shape, params = _lib.make_shape(1, 2, 4, 8, 8, 64, 64), _lib.make_params(0, 0)
    for name in ("vsa_attention_train", "vsa_attention_bwd"):
        monkeypatch.setattr(_lib.lib, name, lambda *a: _lib.VSA_OK)
    t, o_lo = _set(dtype=dtype), torch.zeros(1, 2, 256, 64, dtype=dtype)
    kinds, ws, err = torch.zeros(2, dtype=torch.uint8), torch.zeros(1 << 10, dtype=torch.uint8), torch.zeros(1, dtype=torch.int32)

    def train(lo=o_lo, kinds=kinds, ws_bytes=1 << 10, **kw):
        io = _lib.qkvo(*({**t, **kw}[n] for n in ("q", "k", "v", "o", "lse")))
        _lib.vsa_attention_train(io, lo, code, shape, params, 1, kinds, None, ws, ws_bytes, err, 0)

    def bwd(kinds=kinds, ws_bytes=1 << 10, **kw):
        _lib.vsa_attention_bwd(_lib.qkvo_grad(**{**t, **kw}), code, shape, params, kinds, ws, ws_bytes, err, 0)

    other = torch.zeros(1, 2, 256, 64, dtype=F32 if dtype == BF else BF)
    train()
    bwd()
    for call in (train, bwd):
        for name in ("q", "k", "v", "o"):
            for bad in (other, o_lo[:, :1], _strided(o_lo)):
                with pytest.raises(ValueError):
                    call(**{name: bad})
        for bad in (t["lse"].double(), t["lse"][:, :1]):
            with pytest.raises(ValueError):
                call(lse=bad)
        with pytest.raises(ValueError):
            call(kinds=kinds.long())
        with pytest.raises(ValueError):
            call(ws_bytes=1 << 11)
    with pytest.raises(ValueError):
        train(lse=t["lse"].transpose(1, 2).contiguous().transpose(1, 2))        # written: it has to be whole
    for bad in (other, _strided(o_lo)):
        with pytest.raises(ValueError):
            train(lo=bad)
        with pytest.raises(ValueError):
            bwd(dv=bad)


def test_norm_refuses_what_would_be_read_as_something_else(monkeypatch):
    for name in ("vsa_rms_norm", "vsa_rms_norm_bwd"):
        monkeypatch.setattr(_lib.lib, name, lambda *a: _lib.VSA_OK)
    B, H, N, d = 1, 2, 10, 64
    whole, proj = torch.zeros(B, H, N, d, dtype=BF), torch.zeros(B, N, H, d, dtype=BF)
    shape, views = _lib.make_norm_shape(B, H, N, d), _lib.make_norm_shape(B, H, N, d, (N * H * d, d, H * d), (N * H * d, d, H * d), 64)
    rows, w = torch.zeros(B, H, N), torch.zeros(d)
    codes, exps = torch.zeros(B, H, N, d, dtype=torch.uint8), torch.zeros(B, H, 1, dtype=torch.int32)

    def fwd(x=whole, res=None, w=w, sh=shape, wt=_lib.VSA_F32, **kw):
        _lib.vsa_rms_norm(x, res, _lib.VSA_BF16, w, wt, sh, **{**dict(y=whole, rstd=rows), **kw}, stream=0)

    def bwd(dy=whole, ds=None, s=whole, rstd=rows, dx=whole, dw=w, sh=shape, ws=torch.zeros(100, dtype=torch.uint8), wsb=100):
        _lib.vsa_rms_norm_bwd(dy, ds, s, _lib.VSA_BF16, None, 0, rstd, sh, dx, dw, ws, wsb, 0)

    fwd()
    fwd(x=proj, res=proj, sum=whole, codes=codes, exps=exps, sh=views)
    fwd(codes=codes.view(torch.float8_e4m3fn), exps=torch.zeros(B, H, N, dtype=torch.int32))
    bwd()
    bwd(s=proj, dx=proj, sh=views)
    strided = whole.transpose(1, 2).contiguous().transpose(1, 2)
    for bad in (whole.float(), strided, whole[:, :1]):
        for name in ("x", "y", "sum"):
            with pytest.raises(ValueError, match=name):
                fwd(**{name: bad})
        for name in ("dy", "ds", "s", "dx"):
            with pytest.raises(ValueError):
                bwd(**{name: bad})
    for bad in (rows.double(), rows[:, :1], rows.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError, match="rstd"):
            fwd(rstd=bad)
        with pytest.raises(ValueError, match="rstd"):
            bwd(rstd=bad)
    for bad in (w.to(BF), w[:32], torch.zeros(2 * d)[::2]):
        with pytest.raises(ValueError, match="weight"):
            fwd(w=bad)
        with pytest.raises(ValueError, match="d_weight"):
            bwd(dw=bad)
    with pytest.raises(ValueError, match="codes"):
        fwd(codes=codes.int(), exps=exps, sh=views, x=proj)
    with pytest.raises(ValueError, match="exponents"):
        fwd(codes=codes, exps=exps, x=whole)                      # one for each row is wanted
    # rows that reach behind the tensor's memory
    for bad in (proj[:, :-1], proj.flatten()[1:], proj.float()):
        short = bad.clone()
        with pytest.raises(ValueError, match="x"):
            fwd(x=short, sh=views)
        with pytest.raises(ValueError, match="dx"):
            bwd(dx=short, s=proj, sh=views)
    with pytest.raises(ValueError, match="workspace"):
        bwd(wsb=101)


def test_tensors_of_a_set_live_until_the_launch(monkeypatch):
    """A set that nothing else holds, with a log-sum-exp that has to be copied."""
    shape, refs, alive = _lib.make_shape(1, 2, 4, 8, 8, 64, 64), [], []
    monkeypatch.setattr(_lib.lib, "vsa_sparse_attn_bwd", lambda *a: alive.extend(r() is not None for r in refs) or _lib.VSA_OK)

    def fresh():
        t = {**_set(), "lse": torch.zeros(2, 257)[:, :256]}
        refs.extend(weakref.ref(x) for x in t.values())
        return _lib.qkvo_grad(**t)

    ws = torch.zeros(_lib.vsa_sparse_attn_bwd_workspace_size(shape), dtype=torch.uint8)
    _lib.vsa_sparse_attn_bwd(fresh(), fresh(), torch.zeros(2, dtype=torch.uint8), torch.zeros(1, 2, 4, 1, dtype=torch.int32),
                             torch.ones(1, 2, 4, dtype=torch.int32), 1, shape, 0.0, ws, ws.numel(), torch.zeros(1, dtype=torch.int32), 0)
    assert len(alive) == 18 and all(alive)
