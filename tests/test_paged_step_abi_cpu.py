"""q8kv_extend_paged and attn_norm_rope answer bad arguments before any CUDA call (no GPU needed)."""

import ctypes

P = ctypes.c_void_p
N = P(0)


def err(lib):
    return lib.q8a_last_error().decode()


def test_extend_refusals(lib):
    from chunked_prefill_attention_gb300 import q8attn as Q
    at = {n: P(0x100000 + 0x100000 * i) for i, n in enumerate(
        ("new", "kv", "table", "free", "n_free", "kv_out", "cu", "slots", "pos", "left"))}

    def call(batch=4, width=8, capacity=100, page=16, total=64, **kw):
        p = {**at, **kw}
        return lib.q8kv_extend_paged(p["new"], p["kv"], batch, p["table"], width, p["free"], capacity, p["n_free"], page,
                                     total, p["kv_out"], p["cu"], p["slots"], p["pos"], p["left"], N)

    bad, mis = Q.Q8A_ERR_INVALID_ARG, Q.Q8A_ERR_MISALIGNED
    for kw in (dict(batch=-1), dict(batch=(1 << 20) + 1), dict(total=-1), dict(total=1 << 31), dict(page=8), dict(page=24),
               dict(page=8192), dict(width=-1), dict(width=1 << 31), dict(capacity=-1), dict(capacity=1 << 31)):
        assert call(**kw) == bad, kw
        assert "q8kv_extend_paged" in err(lib)
    for name in at:
        assert call(**{name: N}) == bad, name
        assert call(**{name: P(at[name].value + 2)}) == mis, name
    assert call(slots=P(at["slots"].value + 4)) == mis
    # outputs on each other, and on inputs; the lengths and the free pages' number only onto themselves
    for a in ("kv_out", "cu", "slots", "pos", "left", "table"):
        for b in at:
            if a == b or (a, b) in (("kv_out", "kv"), ("left", "n_free")):
                continue
            assert call(**{a: at[b]}) == bad and "overlap" in err(lib), (a, b)
    assert call(kv_out=P(at["kv"].value + 4)) == bad
    assert call(cu=P(at["slots"].value - 16)) == bad            # its last value lies on the first slot
    assert call(batch=1, left=P(at["kv"].value)) == bad


def test_norm_rope_refusals(lib):
    from chunked_prefill_attention_gb300 import q8attn as Q
    q, k, qo, ko, w, pos, f, ax = (P(0x1000000 * (i + 1)) for i in range(8))

    def call(q=q, qo=qo, heads=4, qs=512, qos=512, k=k, ko=ko, kv=2, ks=256, kos=256, dtype=1, n=5, D=128, qw=w, kw=w, wd=1,
             eps=1e-6, pos=pos, axes=1, ax=N, f=f, rot=128, layout=0, ms=1.0):
        return lib.attn_norm_rope(q, qo, heads, qs, qos, k, ko, kv, ks, kos, dtype, n, D, qw, kw, wd, eps, pos, axes, ax, f,
                                  rot, layout, ms, N)

    bad, mis, uns = Q.Q8A_ERR_INVALID_ARG, Q.Q8A_ERR_MISALIGNED, Q.Q8A_ERR_UNSUPPORTED
    for kw in (dict(n=-1), dict(n=(1 << 31) + 1), dict(heads=0), dict(heads=65536, qs=1 << 30, qos=1 << 30), dict(kv=-1),
               dict(kv=65536, ks=1 << 30, kos=1 << 30), dict(qs=511), dict(qos=511), dict(ks=255), dict(kos=255),
               dict(qs=(1 << 32) + 1), dict(q=N), dict(qo=N), dict(k=N), dict(ko=N), dict(eps=-1e-6),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(pos=N), dict(f=N), dict(rot=0), dict(rot=130),
               dict(rot=7), dict(layout=2), dict(ms=0.0), dict(ms=float("inf")), dict(axes=0), dict(axes=-1), dict(axes=2),
               dict(axes=65536, ax=ax), dict(qw=N, kw=N, pos=N, f=N)):
        assert call(**kw) == bad, kw
        assert "attn_norm_rope" in err(lib)
    assert call(kv=0, k=N, ko=N, qw=N, pos=N, f=N) == bad       # k's weight alone, without k
    for kw in (dict(D=96), dict(dtype=3), dict(dtype=-1), dict(wd=3)):
        assert call(**kw) == uns, kw
    for name, p in (("q", q), ("qo", qo), ("k", k), ("ko", ko), ("qw", w), ("kw", w), ("pos", pos), ("f", f)):
        assert call(**{name: P(p.value + 1)}) == mis, name
    assert call(axes=2, ax=P(ax.value + 2)) == mis
    assert call(dtype=2, q=P(q.value + 2)) == mis
    assert call(wd=2, qw=P(w.value + 2)) == mis
    for kw in (dict(qo=k), dict(ko=q), dict(qo=ko), dict(qo=P(q.value + 2)), dict(ko=P(k.value - 2)),
               dict(qo=q, qos=520), dict(ko=k, kos=264)):
        assert call(**kw) == bad, kw
    # slices of one fused buffer lie between each other: the next slice's first byte is another's, one less is not
    assert call(k=P(q.value + 1022), qs=1024, ks=1024, qo=q, qos=1024, ko=P(q.value + 1022), kos=1024) == bad
    assert call(n=0, q=N, qo=N, k=N, ko=N) == Q.Q8A_OK


def test_helpers():
    from chunked_prefill_attention_gb300 import q8attn as Q
    assert Q.rope_axes((2, 0, 3)).tolist() == [0, 0, 2, 2, 2]
