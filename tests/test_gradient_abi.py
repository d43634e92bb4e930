"""CPU checks of the gradient's entry points (host validation, workspace sizes) and of the 64-bit gradients
that the GPU tests compare with.  No kernel runs."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from block_sparse_attention_31_b200 import _lib
from grad_util import allowed_blocks, reference

FAKE = 0x10000  # 16-byte-aligned non-null address; never dereferenced (validation fails first)
s = ctypes.c_void_p(0)


def _set(**kw):
    out = dict(dq=FAKE + 256, dk=FAKE + 512, dv=FAKE + 768)
    return _lib.QKVOGrad(**{**{n: FAKE for n, _ in _lib.QKVOGrad._fields_}, **out, "d_lse": None, "o_lo": None, **kw})


def _lists(nat, perm, shape, ws_bytes, max_kv=4, scale=0.0, ws=FAKE):
    return _lib.lib.vsa_sparse_attn_bwd(ctypes.byref(nat), ctypes.byref(perm) if perm else None, FAKE, FAKE, FAKE, max_kv,
                                        ctypes.byref(shape), scale, ws, ws_bytes, FAKE, s)


def test_lists_refused_before_launch():
    shape = _lib.make_shape(1, 2, 4, 8, 8, 64, 64)
    need = _lib.vsa_sparse_attn_bwd_workspace_size(shape)
    assert need == 256 + 2 * 4 * 64 * 12                   # bitsets (2*4 words, 256-aligned), three terms a row
    for name, _ in _lib.QKVOGrad._fields_:
        if name not in ("d_lse", "o_lo"):
            assert _lists(_set(**{name: None}), None, shape, need) == _lib.VSA_ERR_INVALID_ARG
            assert _lists(_set(), _set(**{name: None}), shape, need) == _lib.VSA_ERR_INVALID_ARG
            assert _lists(_set(**{name: FAKE + 4}), None, shape, need) == _lib.VSA_ERR_INVALID_ARG
    for kw in (dict(dq=FAKE), dict(dk=FAKE + 256), dict(o_lo=FAKE + 768)):      # gradients over inputs or each other
        assert _lists(_set(**kw), None, shape, need) == _lib.VSA_ERR_INVALID_ARG
    assert _lists(_set(), None, shape, need - 1) == _lib.VSA_ERR_WORKSPACE
    assert _lists(_set(), None, shape, need, max_kv=0) == _lib.VSA_ERR_INVALID_ARG
    assert _lists(_set(), None, shape, need, scale=-1.0) == _lib.VSA_ERR_INVALID_ARG
    assert _lists(_set(), None, shape, need, scale=float("nan")) == _lib.VSA_ERR_INVALID_ARG
    assert _lists(_set(), None, shape, need, ws=FAKE + 8) == _lib.VSA_ERR_INVALID_ARG
    assert _lists(_set(), None, _lib.make_shape(1, 2, 4, 8, 8, 96, 64), need) == _lib.VSA_ERR_UNSUPPORTED
    assert _lib.vsa_sparse_attn_bwd_workspace_size(_lib.make_shape(1, 2, 4, 8, 8, 96, 64)) == 0
    # more blocks than the kernel's shared memory holds bits for, more CTAs than a grid holds
    far = _lib.make_shape(1, 1, 1, 1 << 14, 1 << 14, 64, 64)
    many = _lib.make_shape(1 << 12, 1 << 10, 1, 64, 1024, 64, 64)
    for sh in (far, many):
        assert _lib.vsa_sparse_attn_bwd_workspace_size(sh) == 0
        assert _lists(_set(), None, sh, 1 << 62) == _lib.VSA_ERR_UNSUPPORTED
    if not torch.cuda.is_available():                      # no device: no address is device memory
        assert _lists(_set(), None, shape, need) == _lib.VSA_ERR_INVALID_ARG


def test_call_refused_before_launch():
    shape, params = _lib.make_shape(1, 2, 4, 8, 8, 128, 128), _lib.make_params(0, 0)

    def call(io, p=params, sh=shape, dtype=1, ws_bytes=1 << 40, kind=FAKE, ws=FAKE):
        return _lib.lib.vsa_attention_bwd(ctypes.byref(io), dtype, ctypes.byref(sh), ctypes.byref(p), kind, ws, ws_bytes, FAKE, s)

    need = _lib.vsa_attention_bwd_workspace_size(shape, params, 1)
    assert need >= 7 * 2 * 256 * 128 * 2
    assert call(_set(), ws_bytes=need - 1) == _lib.VSA_ERR_WORKSPACE
    assert call(_set(lse=None)) == _lib.VSA_ERR_INVALID_ARG
    assert call(_set(dk=FAKE + 2)) == _lib.VSA_ERR_INVALID_ARG
    assert call(_set(), kind=None) == _lib.VSA_ERR_INVALID_ARG
    assert call(_set(), ws=None) == _lib.VSA_ERR_INVALID_ARG
    assert call(_set(), dtype=7) == _lib.VSA_ERR_INVALID_ARG
    assert call(_set(), p=_lib.make_params(-1, 0)) == _lib.VSA_ERR_INVALID_ARG
    assert call(_set(), p=_lib.make_params(0, 0, qk_fp8=True)) == _lib.VSA_ERR_UNSUPPORTED
    assert _lib.vsa_attention_bwd_workspace_size(shape, _lib.make_params(0, 0, qk_fp8=True), 1) == 0
    assert _lib.vsa_attention_bwd_workspace_size(shape, params, 3) == 0
    assert _lib.vsa_attention_bwd_workspace_size(_lib.make_shape(1, 2, 4, 8, 8, 32, 64), params, 1) == 0


@pytest.mark.parametrize("seed", range(3))
def test_reference_gradient_matches_differences(seed):
    """The 64-bit gradient is the slope of the oracle's attention."""
    N, d, block = 20, 8, 4
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn(N, d, generator=g, dtype=torch.float64) for _ in range(4))
    d_lse = torch.randn(N, generator=g, dtype=torch.float64)
    keep = torch.rand(5, 5, generator=g) < 0.5
    keep[1] = False
    slots = np.random.default_rng(seed).permutation(N)
    d_lse[torch.from_numpy(slots) // block == 1] = 0.0          # rows that see nothing have no finite lse
    _, _, grads, _ = reference(q, k, v, do, allowed_blocks(keep, slots, block), d_lse=d_lse)

    def loss(x):
        o, lse = oracle.attention_rows(*x, slots, block, keep.numpy(), scale=1 / math.sqrt(d))
        return float((torch.from_numpy(o) * do).sum()) + float((torch.from_numpy(np.where(np.isfinite(lse), lse, 0.0)) * d_lse).sum())

    for i in range(3):
        u, e = torch.randn(N, d, generator=g, dtype=torch.float64), 1e-5
        up, down = [q, k, v], [q, k, v]
        up[i], down[i] = up[i] + e * u, down[i] - e * u
        # central differences: an error of order e^2 of third derivatives of order one, and 1e-16 * |loss| / e
        assert (loss(up) - loss(down)) / (2 * e) == pytest.approx(float((grads[i] * u).sum()), rel=1e-6, abs=1e-7)


def test_norm_refused_before_launch():
    lib, good = _lib.lib, dict(B=1, H=2, N=10, d=64)

    def fwd(shape=good, x=FAKE, res=None, dtype=1, w=FAKE, wt=1, sum=None, y=FAKE + 192, codes=None, exps=None, rstd=FAKE, **kw):
        sh = _lib.make_norm_shape(**{**shape, **kw})
        return lib.vsa_rms_norm(x, res, dtype, w, wt, ctypes.byref(sh), sum, y, codes, exps, rstd, s)

    def bwd(shape=good, dy=FAKE, d_sum=None, x=FAKE + 64, dtype=1, w=FAKE, wt=0, rstd=FAKE, dx=FAKE + 128, dw=FAKE, ws=FAKE, wsb=1 << 30,
            **kw):
        sh = _lib.make_norm_shape(**{**shape, **kw})
        return lib.vsa_rms_norm_bwd(dy, d_sum, x, dtype, w, wt, rstd, ctypes.byref(sh), dx, dw, ws, wsb, s)

    inv, uns = _lib.VSA_ERR_INVALID_ARG, _lib.VSA_ERR_UNSUPPORTED
    for bad in (dict(B=0), dict(H=-1), dict(N=0), dict(d=0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(x_stride=(1, -1, 1)), dict(res_stride=(1 << 50, 1, 1))):
        assert fwd(**bad) == inv and bwd(**bad) == inv
        assert _lib.vsa_rms_norm_bwd_workspace_size(_lib.make_norm_shape(**{**good, **bad}), 1) == 0
    for bad in (dict(d=16385), dict(B=1 << 20, H=1 << 20), dict(B=1 << 10, H=1 << 10, N=1 << 12)):
        assert fwd(**bad) == uns and bwd(**bad) == uns
    assert fwd(x=None) == inv and fwd(x=FAKE + 1) == inv and fwd(dtype=2) == inv and fwd(wt=5) == inv
    assert fwd(y=None) == inv                                       # nothing to write
    assert fwd(sum=FAKE + 64) == inv                                # a sum needs a residual
    assert fwd(codes=FAKE + 64) == inv and fwd(exps=FAKE) == inv    # codes and exponents go together
    assert fwd(y=FAKE + 2) == inv and fwd(w=FAKE + 4) == inv and fwd(rstd=FAKE + 4) == inv
    assert fwd(x=FAKE + 64, y=FAKE + 64) == inv                     # in place
    assert fwd(res=FAKE + 64, sum=FAKE + 64) == inv
    assert fwd(codes=FAKE + 64, exps=FAKE, block=32) == uns
    assert fwd(codes=FAKE + 64, exps=FAKE, block=64, d=96) == uns
    assert bwd(dy=None) == inv and bwd(x=None) == inv and bwd(rstd=None) == inv and bwd(dx=None) == inv
    assert bwd(dx=FAKE) == inv and bwd(dx=FAKE + 64) == inv         # in place
    assert bwd(ws=None) == inv and bwd(wsb=8) == _lib.VSA_ERR_WORKSPACE
    assert bwd(res_stride=(0, 64, 32)) == inv                       # rows of dx that overlap
    assert bwd(res_stride=(0, 0, 64)) == inv                        # heads of dx that coincide
    size = _lib.vsa_rms_norm_bwd_workspace_size
    assert size(_lib.make_norm_shape(**good), 1) == 20 * 64 * 4          # a row of partial sums for each row at most
    assert size(_lib.make_norm_shape(**good), 2) == 0
    for d in (1, 64, 100, 1536, 16384):                                  # and at most a few MB a kernel's width
        for dtype in (0, 1):
            assert 4 * d <= size(_lib.make_norm_shape(1, 1, 1 << 20, d), dtype) <= 148 * 512 * 32 * 4 + 256


def test_train_call_refused_before_launch():
    shape, params = _lib.make_shape(1, 2, 4, 8, 8, 128, 128), _lib.make_params(0, 0)

    def call(io=(FAKE, FAKE, FAKE, FAKE, FAKE), o_lo=FAKE + 64, p=params, ws_bytes=1 << 40):
        q = _lib.QKVO(*io)
        return _lib.lib.vsa_attention_train(ctypes.byref(q), o_lo, 1, ctypes.byref(shape), ctypes.byref(p), 1, FAKE, None, FAKE, ws_bytes,
                                            FAKE, s)

    need = _lib.vsa_attention_train_workspace_size(shape, params, 1, 1)
    assert need >= _lib.vsa_attention_workspace_size(shape, params, 1, 1) + 2 * 256 * 128 * 2
    assert _lib.vsa_attention_train_workspace_size(shape, _lib.make_params(0, 0, qk_fp8=True), 1, 1) == 0
    assert call(o_lo=None) == _lib.VSA_ERR_INVALID_ARG and call(o_lo=FAKE + 4) == _lib.VSA_ERR_INVALID_ARG
    assert call(o_lo=FAKE) == _lib.VSA_ERR_INVALID_ARG                              # o itself
    assert call(io=(FAKE, FAKE, FAKE, FAKE, None)) == _lib.VSA_ERR_INVALID_ARG      # no lse
    assert call(io=(FAKE, None, FAKE, FAKE, FAKE)) == _lib.VSA_ERR_INVALID_ARG
    assert call(p=_lib.make_params(0, 0, qk_fp8=True)) == _lib.VSA_ERR_UNSUPPORTED
    if torch.cuda.is_available():                                                   # the workspace is looked at after the pointer
        return
    assert call() == _lib.VSA_ERR_INVALID_ARG
