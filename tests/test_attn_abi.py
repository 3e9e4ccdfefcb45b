"""include/dq4_attn.h without a GPU: its functions are exported, its arguments checked on the
host before any CUDA call, and the 64-bit definitions that the GPU tests compare with agree with
independent forms of the same."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import attention as oracle_attn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 12  # a fake aligned pointer, never followed on these paths


@pytest.fixture(scope="module")
def lib():
    from quantized_weight_dequantization_gb300 import build
    build.build()
    from quantized_weight_dequantization_gb300 import _attention
    return _attention._lib()


def test_declared_functions_are_exported(lib):
    text = open(os.path.join(ROOT, "include", "dq4_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*\w+\s+(dq4\w*)\s*\(", text, flags=re.M))
    assert names == {"dq4_qk_norm_rope", "dq4_qk_norm_rope_backward",
                     "dq4_qk_norm_rope_backward_workspace_bytes", "dq4_kv8_append",
                     "dq4_kv8_attention", "dq4_kv8_attention_workspace_bytes"}
    for name in names:
        assert hasattr(lib, name)
    for code in range(12, 16):
        assert lib.dq4_status_string(code) != b"unknown status"


def _cache(**kw):
    from quantized_weight_dequantization_gb300._attention import _Cache
    d = dict(k=P, v=P, k_scale=P, v_scale=P, pages=4, kv_heads=2, page=16, head_dim=64)
    d.update(kw)
    return ctypes.byref(_Cache(*[d[n] for n in ("k", "v", "k_scale", "v_scale", "pages",
                                                "kv_heads", "page", "head_dim")]))


BAD_CACHES = [(dict(head_dim=96), 12), (dict(kv_heads=0), 12), (dict(page=48), 14),
              (dict(page=8), 14), (dict(page=512), 14), (dict(pages=-1), 2), (dict(k=None), 1),
              (dict(v_scale=None), 1), (dict(k=P + 8), 6), (dict(k_scale=P + 2), 6)]


def test_norm_arguments(lib):
    base = dict(q=P, qt=128, qh=64, k=P, kt=128, kh=64, dt=1, tokens=3, hq=2, hk=1, dim=64, qw=P,
                kw=P, eps=1e-6, cos=P, sin=P, rows=9, rotary=64, inter=0, pos=P, qo=P, ko=P,
                bad=None)

    def call(**kw):
        d = dict(base, **kw)
        return lib.dq4_qk_norm_rope(*d.values(), None)

    for kw, st in ((dict(dt=3), 5), (dict(dt=-1), 5), (dict(tokens=-1), 2), (dict(hq=0), 12),
                   (dict(hk=-1), 12), (dict(dim=63), 12), (dict(dim=1026), 12),
                   (dict(sin=None), 1), (dict(rotary=66), 13), (dict(rotary=7), 13),
                   (dict(rotary=0), 13), (dict(pos=None), 1), (dict(q=None), 1),
                   (dict(ko=None), 1), (dict(kw=None), 1), (dict(q=P + 1), 6),
                   (dict(dt=2, q=P + 2), 6), (dict(pos=P + 4), 6), (dict(bad=P + 1), 6)):
        assert call(**kw) == st, kw
    assert call(tokens=0, q=None, k=None, qo=None, ko=None) == 0

    back = dict(dqo=P, dko=P, **{k: base[k] for k in list(base)[:20]}, dq=P, dk=P, dqw=P, dkw=P,
                ws=P, wsb=1 << 30, bad=None)

    def call_back(**kw):
        return lib.dq4_qk_norm_rope_backward(*dict(back, **kw).values(), None)

    for kw, st in ((dict(dqo=None), 1), (dict(dko=P + 1), 6), (dict(dqw=None), 1),
                   (dict(ws=None), 15), (dict(wsb=300), 15), (dict(ws=P + 16), 6),
                   (dict(dim=0), 12)):
        assert call_back(**kw) == st, kw
    assert lib.dq4_qk_norm_rope_backward_workspace_bytes(0) == 0
    assert lib.dq4_qk_norm_rope_backward_workspace_bytes(128) > 1024


def test_append_arguments(lib):
    base = dict(cache=_cache(), k=P, kt=128, kh=64, v=P, vt=128, vh=64, dt=1, tokens=5, table=P,
                ts=3, width=3, lens=P, cu=P, seqs=2, cos=P, sin=P, rows=9, rotary=64, inter=0,
                bad=None)

    def call(**kw):
        return lib.dq4_kv8_append(*dict(base, **kw).values(), None)

    for kw, st in BAD_CACHES:
        assert call(cache=_cache(**kw)) == st, kw
    for kw, st in ((dict(cache=None), 1), (dict(dt=2), 5), (dict(tokens=-1), 2),
                   (dict(seqs=-1), 2), (dict(width=-1), 2), (dict(cu=None), 2),
                   (dict(lens=None), 1), (dict(table=None), 1), (dict(cos=None), 1),
                   (dict(rotary=4), 13), (dict(rotary=72), 13), (dict(rotary=12), 13),
                   (dict(k=None), 1), (dict(v=P + 4), 6), (dict(kt=126), 6), (dict(vh=66), 6),
                   (dict(cos=P + 8), 6), (dict(lens=P + 2), 6)):
        assert call(**kw) == st, kw
    assert call(tokens=0, k=None, v=None) == 0


def test_attention_arguments(lib):
    base = dict(cache=_cache(), q=P, qt=256, qh=64, dt=1, tokens=5, heads=4, table=P, ts=3,
                width=3, lens=P, cu=P, seqs=2, max_new=4, scale=0.1, causal=1, window=0, out=P,
                lse=None, ws=P, wsb=1 << 40, bad=None)

    def call(**kw):
        return lib.dq4_kv8_attention(*dict(base, **kw).values(), None)

    for kw, st in BAD_CACHES:
        assert call(cache=_cache(**kw)) == st, kw
    for kw, st in ((dict(dt=2), 5), (dict(heads=3), 12), (dict(heads=0), 12), (dict(cu=None), 2),
                   (dict(window=-1), 2), (dict(max_new=-1), 2), (dict(q=None), 1),
                   (dict(out=None), 1), (dict(q=P + 8), 6), (dict(qt=260), 6), (dict(qh=66), 6),
                   (dict(out=P + 8), 6), (dict(lse=P + 2), 6), (dict(ws=None), 15),
                   (dict(wsb=0), 15), (dict(ws=P + 128), 6)):
        assert call(**kw) == st, kw
    assert call(tokens=0, q=None, out=None, ws=None) == 0
    size = lib.dq4_kv8_attention_workspace_bytes
    assert size(0, 4, 8, 2, 64) == 0 and size(4, 4, 8, 2, 64) > 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device status")
def test_no_device_is_reported(lib):
    assert lib.dq4_kv8_append(_cache(), P, 128, 64, P, 128, 64, 1, 5, P, 3, 3, P, P, 2, None,
                              None, 0, 0, 0, None, None) == 7


# ----------------------------------------------------- the 64-bit definitions themselves
def test_e4m3_rounding_against_torch():
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.float16)
    x = x[x.isfinite() & (x.abs() <= 448)]
    assert np.array_equal(oracle_attn.e4m3(x.double().numpy()),
                          x.to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_gradients_against_autograd(interleaved):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 4, 3, 12))
    w = rng.standard_normal(12)
    angle = rng.uniform(0, 6, (7, 4))
    pos = np.array([3, 0, 6, 3])
    cos, sin = np.cos(angle), np.sin(angle)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    n = torch.nn.functional.rms_norm(tx, (12,), tw, 1e-5)
    z = torch.polar(torch.ones(4, 1, 4, dtype=torch.float64), torch.tensor(angle[pos])[:, None])
    if interleaved:
        y = torch.view_as_real(torch.view_as_complex(n[..., :8].reshape(4, 3, 4, 2)) * z)
        y = torch.cat([y.flatten(-2), n[..., 8:]], -1)
    else:
        y = torch.complex(n[..., :4], n[..., 4:8]) * z
        y = torch.cat([y.real, y.imag, n[..., 8:]], -1)
    (y * torch.tensor(dy)).sum().backward()
    got, size = oracle_attn.norm_rope(x, w, cos, sin, pos, 1e-5, interleaved)
    assert np.allclose(got, y.detach().numpy(), atol=1e-12) and (size >= np.abs(got) - 1e-12).all()
    dx, dxs, dw, dws = oracle_attn.norm_rope_backward(dy, x, w, cos, sin, pos, 1e-5, interleaved)
    assert np.allclose(dx, tx.grad.numpy(), atol=1e-12)
    assert np.allclose(dw, tw.grad.numpy(), atol=1e-12)
    assert (dxs >= np.abs(dx) - 1e-12).all() and (dws >= np.abs(dw) - 1e-12).all()


def test_attention_definition_against_torch():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 3, 2, 4, 8))
    ones = np.ones((3, 2), np.float32)
    q = rng.standard_normal((6, 4, 8))
    table = np.array([[2, 0, 1]])
    out, lse, size, reach = oracle_attn.attend(q, k, v, ones, ones, table, [10], [0, 6], 0.3, True,
                                               0)
    kk, vv = (torch.tensor(np.concatenate([x[i] for i in (2, 0, 1)], 1)[:, :10]) for x in (k, v))
    tq = torch.tensor(q).transpose(0, 1)
    mask = torch.arange(10)[None] <= torch.arange(4, 10)[:, None]
    s = torch.einsum("hid,hjd->hij", tq, kk.repeat_interleave(2, 0)) * 0.3
    s = s.masked_fill(~mask, float("-inf"))
    want = torch.softmax(s, -1) @ vv.repeat_interleave(2, 0)
    assert np.allclose(out, want.transpose(0, 1).numpy())
    assert np.allclose(lse, torch.logsumexp(s, -1).T.numpy())
    assert (size >= np.abs(out) - 1e-12).all() and (reach > 0).all()


def test_append_definition_by_hand():
    """Two tokens that fit at different scales: 3.0 and 1000.0 in one page of one head."""
    codes, scales = np.full((1, 1, 2, 2), np.nan), np.full((1, 1), np.nan, np.float32)
    x = np.array([[[3.0, -1.0]], [[1000.0, 0.3]]], np.float32)
    oracle_attn.append(codes, scales, x[:1], None, None, [[0]], [1], [0, 1], False)
    assert scales[0, 0] == 2.0 ** -7 and np.array_equal(codes[0, 0, 0], [384.0, -128.0])
    oracle_attn.append(codes, scales, x[1:], None, None, [[0]], [2], [0, 1], False)
    assert scales[0, 0] == 4.0  # 448 * 2 < 1000 <= 448 * 4
    assert np.array_equal(codes[0, 0], [[0.75, -0.25], [256.0, 0.078125]])  # 250 -> 256
