"""Refusals of the calls for bounded memory (linear attention with one decay per head, eviction from
the cache): host-side checks before any launch (no call here reaches CUDA), and the binding's own
checks of shapes and types."""
import pytest
import torch

P = 4096


@pytest.fixture(scope="module")
def L():
    from linear_attention_state_kda_gb300 import build as libbuild
    libbuild.build()
    from linear_attention_state_kda_gb300 import kda
    return kda.lib()


def _prefill(L, dt=0, n=1, T=10, cu=None, H=2, Hk=2, d=64, q=P, qs=128, k=P, ks=128, v=P, vs=128,
             g=P, gs=2, init=None, o=P, fin=None, ws=None, ws_bytes=0):
    return L.kda_decay_prefill(dt, n, T, cu, H, Hk, d, 1.0, q, qs, k, ks, v, vs, g, gs, init, o, fin,
                               ws, ws_bytes, None, None)


def test_prefill_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    U, A, W = kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_WORKSPACE
    assert _prefill(L, dt=2) == U and _prefill(L, d=96) == U and _prefill(L, d=0) == U
    for bad in (dict(H=0), dict(Hk=0), dict(H=3, vs=192), dict(H=65536, Hk=1), dict(n=-1), dict(T=-1),
                dict(n=2), dict(n=(1 << 24) + 1, cu=P), dict(q=None), dict(k=None), dict(v=None),
                dict(g=None), dict(o=None), dict(qs=124), dict(ks=130), dict(vs=64), dict(gs=1),
                dict(gs=-2), dict(q=P + 4), dict(k=P + 8), dict(v=P + 4), dict(o=P + 8),
                dict(g=P + 2), dict(init=P + 4), dict(fin=P + 8), dict(cu=P + 1),
                dict(init=P, fin=P)):
        assert _prefill(L, **bad) == A, bad
    assert "kda_decay_prefill" in kda.last_error()
    assert _prefill(L, n=0) == kda.KDA_OK and _prefill(L, T=0) == kda.KDA_OK
    T = 1 << 16
    need = kda.decay_prefill_workspace(torch.float32, 1, T, 2, 64)
    assert need > 0
    assert _prefill(L, T=T) == W and _prefill(L, T=T, ws=P + 16, ws_bytes=need) == W
    assert _prefill(L, T=T, ws=P, ws_bytes=need - 1) == W
    for x in ((2, 1, T, 2, 64), (0, 0, T, 2, 64), (0, 1, 0, 2, 64), (0, 1, T, 0, 64),
              (0, 1, T, 1 << 20, 64), (0, 1, T, 2, 80)):
        assert L.kda_decay_prefill_workspace(*x) == 0


def _window(L, dt=1, B=2, W=2, H=2, Hk=1, d=128, q=P, qs=128, k=P, ks=128, v=P, vs=256, g=P, gs=2,
            rs=P, ws=P, pool=P, n_slots=8, o=P):
    return L.kda_decay_window(dt, B, W, H, Hk, d, 1.0, q, qs, k, ks, v, vs, g, gs, rs, ws, pool,
                              n_slots, o, None, None)


def test_window_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    U, A = kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG
    assert _window(L, dt=5) == U and _window(L, d=32) == U and _window(L, W=17) == U
    assert _window(L, W=-1) == U
    for bad in (dict(B=-1), dict(H=0), dict(Hk=3), dict(n_slots=0), dict(rs=None), dict(ws=None),
                dict(pool=None), dict(q=None), dict(o=None), dict(qs=64), dict(vs=252), dict(gs=1),
                dict(pool=P + 4), dict(rs=P + 2), dict(o=P + 8), dict(B=1 << 29)):
        assert _window(L, **bad) == A, bad
    assert "kda_decay_window" in kda.last_error()
    assert _window(L, B=0) == kda.KDA_OK and _window(L, W=0) == kda.KDA_OK


def _weigh(L, dt=1, B=2, W=1, Hq=8, Hkv=2, d=128, q=P, start=P, table=P, cols=4, kc=P, ks=P, w=P,
           pages=8, ws=None, ws_bytes=0):
    return L.kda_cache_weigh(dt, B, W, Hq, Hkv, d, 1.0, 1.0, q, start, None, table, cols, kc, ks, w,
                             pages, ws, ws_bytes, None, None)


def test_weigh_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    U, A = kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG
    assert _weigh(L, dt=3) == U and _weigh(L, d=80) == U and _weigh(L, W=65537) == U
    assert _weigh(L, W=-1) == U
    for bad in (dict(B=-1), dict(Hq=7), dict(Hkv=0), dict(Hq=0), dict(q=None), dict(start=None),
                dict(table=None), dict(kc=None), dict(ks=None), dict(w=None), dict(pages=0),
                dict(cols=0), dict(q=P + 4), dict(w=P + 4), dict(kc=P + 1), dict(B=1 << 24)):
        assert _weigh(L, **bad) == A, bad
    assert "kda_cache_weigh" in kda.last_error()
    need = kda.cache_weigh_workspace(torch.bfloat16, 2, 40, 8, 2, 128, 4)
    assert need > 0 and kda.cache_weigh_workspace(torch.bfloat16, 2, 16, 8, 2, 128, 4) == 0
    assert kda.cache_weigh_workspace(torch.float32, 2, 40, 8, 2, 128, 4) == 0
    assert kda.cache_weigh_workspace(torch.float32, 2, 1, 8, 2, 128, 4000) > 0
    for x in (dict(), dict(ws=P + 16, ws_bytes=need), dict(ws=P, ws_bytes=need - 1)):
        assert _weigh(L, W=40, **x) == kda.KDA_ERR_WORKSPACE
    assert _weigh(L, cols=4000) == kda.KDA_ERR_WORKSPACE
    for x in ((1, 0, 40, 8, 2, 128, 4), (1, 2, 70000, 8, 2, 128, 4), (1, 2, 40, 7, 2, 128, 4),
              (1, 2, 40, 8, 2, 96, 4), (3, 2, 40, 8, 2, 128, 4), (1, 2, 40, 8, 2, 128, 0),
              (1, 2, 40, 8, 2, 128, 1 << 25)):
        assert L.kda_cache_weigh_workspace(*x) == 0
    assert _weigh(L, B=0) == kda.KDA_OK and _weigh(L, W=0) == kda.KDA_OK


def _evict(L, B=2, H=2, d=128, length=P, table=P, cols=4, new=P, new_cols=2, kc=P, ks=P, vc=P, vs=P,
           w=P, pages=8, budget=100, sinks=4, recent=10, count=2 * P, kept=P):
    return L.kda_cache_evict(B, H, d, length, table, cols, new, new_cols, kc, ks, vc, vs, w, pages,
                             budget, sinks, recent, count, kept, None, None)


def test_evict_refusals(L):
    from linear_attention_state_kda_gb300 import kda
    U, A = kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_INVALID_ARG
    assert _evict(L, d=96) == U
    for bad in (dict(B=-1), dict(H=0), dict(cols=0), dict(pages=0), dict(length=None),
                dict(table=None), dict(new=None), dict(kc=None), dict(vc=None), dict(ks=None),
                dict(vs=None), dict(w=None), dict(count=None), dict(kept=None), dict(new_cols=1),
                dict(budget=-1), dict(budget=(1 << 24) + 1, new_cols=1 << 20), dict(sinks=-1),
                dict(recent=-1), dict(sinks=60, recent=41), dict(count=P), dict(w=P + 8),
                dict(kc=P + 4), dict(kept=P + 2), dict(B=1 << 24)):
        assert _evict(L, **bad) == A, bad
    assert "kda_cache_evict" in kda.last_error()
    assert _evict(L, B=0) == kda.KDA_OK


def test_binding_refuses_shapes_and_types():
    from linear_attention_state_kda_gb300 import kda
    bf, i32 = torch.bfloat16, torch.int32
    q, v, g = torch.zeros(6, 1, 64, dtype=bf), torch.zeros(6, 2, 64, dtype=bf), torch.zeros(6, 2)
    slots, write, pool = torch.zeros(3, dtype=i32), torch.zeros(3, 2, dtype=i32), \
        torch.zeros(4, 2, 64, 64)
    with pytest.raises(ValueError):  # not on a CUDA device
        kda.decay_prefill(q, q, v, g)
    with pytest.raises(ValueError):
        kda.decay_window(q, q, v, g, slots, write, pool)
    for args in ((q, q[:5], v, g), (q, q, v[:5], g), (q, q, v, g[:5]), (q, q, v, g[0, :1]),
                 (q[..., :32], q[..., :32], v, g), (q.transpose(0, 1), q, v, g)):
        with pytest.raises(ValueError):
            kda.decay_prefill(*args)
    for args in ((q.float(), q, v, g), (q, q, v, g.double()), (q, q, v.half(), g), (q, q, v, None)):
        with pytest.raises(TypeError):
            kda.decay_prefill(*args)
    with pytest.raises(TypeError):
        kda.decay_window(q, q, v, g, slots.long(), write, pool)
    with pytest.raises(ValueError):
        kda.decay_window(q, q, v, g, slots, write[:, :1], pool)
    with pytest.raises(ValueError):
        kda.decay_window(q, q, v, g, slots, write, pool[:, :1])
    kc, ks, w = torch.zeros(4, 2, 64, 64, dtype=torch.uint8), torch.ones(4, 2), torch.zeros(4, 2, 64)
    table, x = torch.zeros(3, 2, dtype=i32), torch.zeros(3, 4, 64, dtype=bf)
    with pytest.raises(ValueError):
        kda.cache_weigh(x, slots, table, kc, ks, w)
    with pytest.raises(ValueError):
        kda.cache_weigh(x, slots, table, kc, ks, w[:3])
    with pytest.raises(TypeError):
        kda.cache_weigh(x, slots, table, kc, ks, w.bfloat16())
    with pytest.raises(ValueError):
        kda.cache_evict(slots, table, table, kc, ks, kc, ks, w, 100)
    with pytest.raises(ValueError):
        kda.cache_evict(slots, table, table[:2], kc, ks, kc, ks, w, 100)
    with pytest.raises(ValueError):
        kda.cache_evict(slots, table, table, kc, ks, kc, ks, w, -1)
    with pytest.raises(TypeError):
        kda.cache_evict(slots, table, table, kc, ks, kc, ks, w, 1.5)
