"""The paged calls answer bad arguments before any CUDA call (no GPU needed)."""

import ctypes

import pytest

P = ctypes.c_void_p
A16, A8, A4 = P(0x100000), P(0x100008), P(0x100004)   # never dereferenced
N = P(0)


def _err(lib):
    return lib.q8a_last_error().decode()


def test_rope_refusals(lib):
    from chunked_prefill_attention_gb300 import q8attn as Q

    def call(x=A16, out=A16, dtype=0, n=4, heads=2, D=64, xs=128, os=128, pos=A8, f=A8, rot=32, layout=0, ms=1.0):
        return lib.attn_rope(x, out, dtype, n, heads, D, xs, os, pos, f, rot, layout, ms, 0, N)

    bad = Q.Q8A_ERR_INVALID_ARG
    for kw in (dict(n=-1), dict(n=(1 << 31) + 1), dict(heads=0), dict(heads=65536, xs=1 << 30, os=1 << 30),
               dict(xs=127), dict(os=64), dict(xs=(1 << 32) + 2), dict(x=N), dict(out=N), dict(pos=N), dict(f=N),
               dict(rot=0), dict(rot=33), dict(rot=66), dict(rot=-2), dict(layout=2), dict(ms=float("nan")),
               dict(ms=0.0), dict(xs=256)):   # the last: in place with two strides
        assert call(**kw) == bad, kw
        assert "attn_rope" in _err(lib)
    assert call(D=96) == Q.Q8A_ERR_UNSUPPORTED
    assert call(dtype=3) == Q.Q8A_ERR_UNSUPPORTED
    assert call(x=P(0x100001)) == Q.Q8A_ERR_MISALIGNED
    assert call(pos=A4) == Q.Q8A_ERR_MISALIGNED
    assert call(x=P(0x100002), out=A16, dtype=2) == Q.Q8A_ERR_MISALIGNED
    assert call(n=0, x=N, out=N) == Q.Q8A_OK


def test_append_and_read_refusals(lib):
    from chunked_prefill_attention_gb300 import q8attn as Q

    def append(k=A16, v=A16, dtype=1, n=4, heads=2, D=128, ks=256, vs=256, slots=A8, kp=A16, vp=A16, pages=3, pt=16,
               stride=2 * 16 * 136, pos=N, f=N, rot=0, layout=0, ms=1.0):
        return lib.q8kv_append_paged(k, v, dtype, n, heads, D, ks, vs, slots, kp, vp, pages, pt, stride, pos, f, rot,
                                     layout, ms, N)

    def read(kp=A16, vp=A16, pages=3, pt=16, stride=2 * 16 * 136, slots=A8, n=4, heads=2, D=128, ko=A16, vo=A16,
             dtype=0):
        return lib.q8kv_read_paged(kp, vp, pages, pt, stride, slots, n, heads, D, ko, vo, dtype, N)

    bad, mis, uns = Q.Q8A_ERR_INVALID_ARG, Q.Q8A_ERR_MISALIGNED, Q.Q8A_ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(heads=0), dict(pages=0), dict(pages=1 << 31), dict(pt=8), dict(pt=24), dict(pt=8192),
               dict(stride=2 * 16 * 136 - 16), dict(kp=N), dict(vp=N), dict(slots=N)):
        assert append(**kw) == bad and read(**kw) == bad, kw
    for kw in (dict(k=N), dict(v=N), dict(ks=128), dict(vs=240), dict(pos=A8), dict(f=A8),
               dict(pos=A8, f=A8, rot=130), dict(pos=A8, f=A8, rot=64, layout=-1)):
        assert append(**kw) == bad, kw
    for kw in (dict(ko=N), dict(vo=N)):
        assert read(**kw) == bad
    for kw in (dict(kp=A8), dict(vp=A8), dict(stride=2 * 16 * 136 + 8), dict(slots=A4)):
        assert append(**kw) == mis and read(**kw) == mis, kw
    for kw in (dict(k=A8), dict(v=A8), dict(ks=260)):
        assert append(**kw) == mis, kw
    assert read(ko=A8) == mis
    for kw in (dict(D=32), dict(dtype=3)):
        assert append(**kw) == uns and read(**kw) == uns
    assert append(n=0, k=N, kp=N) == Q.Q8A_OK and read(n=0, ko=N, kp=N) == Q.Q8A_OK


def test_attention_refusals(lib):
    from chunked_prefill_attention_gb300 import q8attn as Q

    def call(q=P(0x200000), dtype=0, qs=512, total=10, heads=8, kv=2, D=64, kp=A16, vp=A16, pages=3, pt=16,
             stride=2 * 16 * 68, table=A4, ts=4, lens=A4, cu=A4, batch=2, mq=5, mkv=64, scale=0.125, out=A16, ws=A16,
             floats=1 << 30):
        return lib.attn_paged(q, dtype, qs, total, heads, kv, D, kp, vp, pages, pt, stride, table, ts, lens, cu, batch,
                              mq, mkv, scale, 1, out, ws, floats, N)

    bad, mis, uns = Q.Q8A_ERR_INVALID_ARG, Q.Q8A_ERR_MISALIGNED, Q.Q8A_ERR_UNSUPPORTED
    for kw in (dict(heads=0), dict(kv=0), dict(kv=3), dict(batch=-1), dict(batch=(1 << 20) + 1), dict(total=-1),
               dict(total=1 << 31), dict(mq=-1), dict(mkv=-1), dict(scale=0.0), dict(scale=float("inf")),
               dict(qs=511), dict(pages=0), dict(pt=17), dict(q=N), dict(out=N), dict(lens=N), dict(cu=N), dict(table=N), dict(q=A16),
               dict(ts=-1), dict(mkv=65), dict(kp=N), dict(ts=4096, mkv=65536, ws=N),
               dict(ts=4096, mkv=65536, floats=10)):
        assert call(**kw) == bad, kw
    for kw in (dict(q=A8), dict(out=A8), dict(ws=A8), dict(qs=516), dict(kp=A8), dict(lens=P(0x100002))):
        assert call(**kw) == mis, kw
    for kw in (dict(D=96), dict(dtype=2), dict(total=1 << 29)):
        assert call(**kw) == uns, kw
    for kw in (dict(batch=0, q=N), dict(total=0, q=N), dict(mq=0, q=N)):
        assert call(**kw) == Q.Q8A_OK
    assert lib.q8a_paged_workspace_floats(1, 1, 8, 3, 1, 1, 64) == -1
    assert lib.q8a_paged_workspace_floats(1, 1, 8, 2, 1, 1, 96) == -1
    assert lib.q8a_paged_workspace_floats(0, 1, 8, 2, 1, 1, 64) == 0
    assert lib.q8a_paged_workspace_floats(1, 1, 8, 2, 1, 1, 64) == 0        # a CTA per unit
    assert lib.q8a_paged_workspace_floats(1, 1, 8, 2, 1, 1 << 20, 64) > 0


def test_rope_frequencies():
    torch = pytest.importorskip("torch")
    from chunked_prefill_attention_gb300 import q8attn as Q
    f = Q.rope_inv_freq(8)
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    assert torch.allclose(Q.rope_inv_freq(8, factor=4.0), f / 4)
    base = Q.rope_inv_freq(8, factor=4.0, scaling="base")
    assert base[0] == 1.0 and torch.allclose(base[-1], f[-1] / 4)
    bands = Q.rope_inv_freq(8, factor=4.0, scaling="bands", original_len=1000, low=1.0, high=4.0)
    assert bands[0] == f[0] and bands[1] == f[1]                 # 159 and 16 turns: kept
    assert torch.allclose(bands[3], f[3] / 4)                    # 0.16 turns: divided
    keep = (1000 * 0.01 / (2 * 3.141592653589793) - 1) / 3       # 1.59 turns: blended
    assert torch.allclose(bands[2], f[2] * keep + f[2] / 4 * (1 - keep))
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, factor=0.0), dict(rot_dim=8, scaling="x"),
               dict(rot_dim=8, scaling="bands")):
        with pytest.raises(ValueError):
            Q.rope_inv_freq(**kw)


def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    from chunked_prefill_attention_gb300 import q8attn as Q
    x = torch.zeros((2, 1, 64))
    pages = torch.zeros((1, 1, 16, 68), dtype=torch.uint8)
    with pytest.raises(Q.Q8AttnError):
        Q.attn_rope(x, torch.zeros(2, dtype=torch.int64), Q.rope_inv_freq(64))
    with pytest.raises(Q.Q8AttnError):
        Q.q8kv_append_paged(x, x, pages, pages, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(Q.Q8AttnError):
        Q.q8kv_read_paged(pages, pages, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(Q.Q8AttnError):
        Q.attn_paged(x.half(), pages, pages, torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32),
                     torch.tensor([0, 2], dtype=torch.int32), 2, 2)
