"""CPU checks of what the binding makes of the gradient's arguments.  No kernel runs: the library's entry point is
replaced by one that reads its arguments back."""
import ctypes

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
