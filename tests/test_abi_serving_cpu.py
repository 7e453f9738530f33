"""Refusals of the serving operators: host-side checks before any launch (no call here reaches
CUDA), and the binding's own checks of shapes and types."""
import pytest
import torch

P = 4096


@pytest.fixture(scope="module")
def L():
    from linear_attention_state_kda_gb300 import build as libbuild
    libbuild.build()
    from linear_attention_state_kda_gb300 import kda
    return kda.lib()


def _norm(L, dt=1, T=4, Hq=2, Hk=1, d=128, q=P, qs=256, k=P, ks=128, eps=1e-6, flags=0, cs=P,
          n_pos=8, rot=64, qo=P, qos=256, ko=P, kos=128, w=None):
    return L.kda_head_norm_rope(dt, T, Hq, Hk, d, q, qs, k, ks, w, w, eps, flags, cs, n_pos, rot,
                                None, qo, qos, ko, kos, None, None)


def test_head_norm_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    U, A = kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG
    assert _norm(L, dt=2) == U and _norm(L, d=96) == U
    assert _norm(L, rot=24) == U and _norm(L, rot=144) == U and _norm(L, rot=-16) == U
    assert _norm(L, T=-1) == A and _norm(L, Hq=-1) == A and _norm(L, flags=4) == A
    assert _norm(L, eps=-1.0) == A and _norm(L, eps=float("nan")) == A
    assert _norm(L, q=None) == A and _norm(L, ko=None) == A
    assert _norm(L, cs=None) == A and _norm(L, n_pos=0) == A
    assert _norm(L, qs=248) == A and _norm(L, qs=257) == A and _norm(L, kos=64) == A
    assert _norm(L, q=P + 8) == A and _norm(L, w=P + 4) == A and _norm(L, cs=P + 4) == A
    assert _norm(L, qs=512) == A  # in place at another stride
    assert "kda_head_norm_rope" in kda.last_error()
    assert _norm(L, T=0) == kda.KDA_OK and _norm(L, Hq=0, Hk=0) == kda.KDA_OK


def _write(L, dt=1, n=1, T=4, cu=P, start=P, H=2, d=128, k=P, ks=256, v=P, vs=256, table=P, cols=4,
           kc=P, ksc=P, vc=P, vsc=P, pages=8):
    return L.kda_cache_write(dt, n, T, cu, start, None, H, d, k, ks, v, vs, table, cols, kc, ksc,
                             vc, vsc, pages, None, None)


def test_cache_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    U, A = kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG
    assert _write(L, dt=7) == U and _write(L, d=256) == U
    for bad in (dict(n=-1), dict(T=-1), dict(H=0), dict(H=70000), dict(cols=0), dict(pages=0),
                dict(n=2, cu=None), dict(start=None), dict(table=None), dict(k=None),
                dict(vc=None), dict(ksc=None), dict(k=P + 8), dict(kc=P + 4), dict(ks=128),
                dict(vs=260), dict(cols=1 << 25)):
        assert _write(L, **bad) == A, bad
    assert "kda_cache_write" in kda.last_error()
    assert _write(L, n=0) == kda.KDA_OK and _write(L, T=0) == kda.KDA_OK

    def read(dt=1, n=1, T=4, cu=P, k=P, v=P, kc=P, ksc=P):
        return L.kda_cache_read(dt, n, T, cu, P, 2, 128, P, 4, kc, ksc, P, P, 8, k, v, None, None)
    assert read(dt=9) == U
    assert read(k=None, v=None) == A and read(kc=None) == A and read(ksc=None) == A
    assert read(k=P + 2) == A and read(n=3, cu=None) == A
    assert read(T=0) == kda.KDA_OK


def _attn(L, dt=1, B=2, W=1, Hq=8, Hkv=2, d=128, q=P, start=P, table=P, cols=4, kc=P, pages=8, o=P,
          ws=None, n=None):
    from linear_attention_state_kda_gb300 import kda
    need = kda.cache_attention_workspace(2, 1, 8, 2, 128) if n is None else n
    return L.kda_cache_attention(dt, B, W, Hq, Hkv, d, 1.0, q, start, None, table, cols, kc, P, P,
                                 P, pages, o, P if ws is None else ws, need, None, None)


def test_attention_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    U, A = kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG
    assert _attn(L, dt=3) == U and _attn(L, d=80) == U and _attn(L, W=65537) == U
    assert _attn(L, W=-1) == U
    for bad in (dict(B=-1), dict(Hq=7), dict(Hkv=0), dict(Hq=0), dict(q=None), dict(start=None),
                dict(table=None), dict(kc=None), dict(o=None), dict(pages=0), dict(cols=0),
                dict(q=P + 4), dict(o=P + 8), dict(kc=P + 1), dict(B=1 << 24)):
        assert _attn(L, **bad) == A, bad
    assert "kda_cache_attention" in kda.last_error()
    assert _attn(L, B=0) == kda.KDA_OK and _attn(L, W=0) == kda.KDA_OK
    if kda.cache_attention_workspace(2, 1, 8, 2, 128) > 0:
        assert _attn(L, n=0) == kda.KDA_ERR_WORKSPACE
        assert _attn(L, ws=P + 16) == kda.KDA_ERR_WORKSPACE
    assert kda.cache_attention_workspace(0, 1, 8, 2, 128) == 0
    assert kda.cache_attention_workspace(2, 1, 7, 2, 128) == 0


def test_verify_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    U, A = kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG

    def call(dt=0, B=2, W=3, V=100, t=P, ts=100, q=P, qs=100, x=P, ua=P, us=P, slots=P, out=P,
             n=P, r=P):
        return L.kda_draft_verify(dt, B, W, V, t, ts, q, qs, x, None, ua, us, slots, out, n, r,
                                  None, None)
    assert call(dt=5) == U and call(W=17) == U and call(V=0) == U and call(V=1 << 23) == U
    for bad in (dict(B=-1), dict(t=None), dict(x=None), dict(ua=None), dict(us=None),
                dict(out=None), dict(n=None), dict(slots=None), dict(ts=99), dict(qs=99),
                dict(t=P + 2), dict(us=P + 1)):
        assert call(**bad) == A, bad
    assert "kda_draft_verify" in kda.last_error()
    assert call(B=0) == kda.KDA_OK


def test_binding_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros(4, 2, 128)
    with pytest.raises(ValueError):
        kda.head_norm_rope(x.transpose(0, 1), None)
    with pytest.raises(ValueError):
        kda.head_norm_rope(x, torch.zeros(3, 2, 128))
    with pytest.raises(TypeError):
        kda.head_norm_rope(x, None, q_weight=torch.ones(128, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        kda.head_norm_rope(x.half(), None)
    pool = [torch.zeros(8, 2, 64, 128, dtype=torch.uint8), torch.ones(8, 2)] * 2
    with pytest.raises(ValueError):
        kda.cache_write(x, x, i32(2), i32(1, 4), *pool)
    with pytest.raises(ValueError):
        kda.cache_write(x[:, :1], x[:, :1], i32(1), i32(1, 4), *pool)
    with pytest.raises(TypeError):
        kda.cache_write(x, x, torch.zeros(1), i32(1, 4), *pool)
    with pytest.raises(TypeError):
        kda.cache_write(x, x, i32(1), i32(1, 4), pool[0].float(), pool[1], pool[2].float(), pool[3])
    with pytest.raises(ValueError):
        kda.cache_attention(torch.zeros(3, 4, 128), i32(2), i32(2, 4), *pool)
    with pytest.raises(ValueError):
        kda.cache_attention(torch.zeros(2, 4, 64), i32(2), i32(2, 4), *pool)
    with pytest.raises(ValueError):
        kda.cache_read(i32(1), i32(1, 4), *pool, 5, cu_seqlens=i32(3))
    t = torch.zeros(2, 4, 50)
    with pytest.raises(ValueError):
        kda.draft_verify(t, i32(2, 2), torch.zeros(2, 3), torch.zeros(2))
    with pytest.raises(TypeError):
        kda.draft_verify(t, torch.zeros(2, 3), torch.zeros(2, 3), torch.zeros(2))
    with pytest.raises(ValueError):
        kda.draft_verify(t[:, :, ::2], i32(2, 3), torch.zeros(2, 3), torch.zeros(2))


def test_attention_workspace_of_refused_sizes(L):
    """Sizes that the call refuses need no workspace: no overflow on the way to the answer."""
    from linear_attention_state_kda_gb300 import kda
    for B, W, Hq, Hkv in ((1, 65536, 65536, 1), (1, 65536, 1 << 30, 1), (1 << 24, 1, 2, 2),
                          (1 << 30, 65536, 1 << 30, 1 << 30), (1, 65536, 16385, 1),
                          (1 << 24, 65536, 1 << 30, 1)):
        assert kda.cache_attention_workspace(B, W, Hq, Hkv, 128) == 0, (B, W, Hq, Hkv)
        assert _attn(L, B=B, W=W, Hq=Hq, Hkv=Hkv, n=0) == kda.KDA_ERR_INVALID_ARG
    most = kda.cache_attention_workspace(1, 65536, 16384, 1, 128)
    assert 2 ** 29 < most < 2 ** 31
