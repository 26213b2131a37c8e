"""CPU tests: argument checks of kv_norm_rope_append, the int8 cache and the modified-score attention entry points
(nothing reaches a GPU), and pins of their oracle."""
import math

import numpy as np
import pytest

from oracle import score_mod as O
from paged_kv_cache_433_b200 import kvpaged as K

PTR = 1 << 20  # a 16-byte aligned address that is never read: every call below returns before any launch


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_433_b200 import build

    build.build()


NR = dict(k_pages=PTR, v_pages=PTR, q_out=PTR, k_out=None, q=PTR, k_new=PTR, v_new=PTR, q_stride=1024, k_stride=256,
          v_stride=256, q_weight=None, k_weight=None, eps=1e-6, slots=PTR, positions=PTR, cos_sin=PTR, max_pos=64, style=0,
          B=0, H_q=8, H_kv=2, Dh=128, P=16, num_pages=10, dtype=1, err=None, stream=None)


def norm_rope(**kw):
    return K.lib().kv_norm_rope_append(*{**NR, **kw}.values())


def test_norm_rope_refusals():
    assert norm_rope() == K.KV_OK  # B = 0
    for bad in (dict(B=-1), dict(H_kv=0), dict(Dh=0), dict(dtype=3), dict(dtype=4), dict(dtype=9), dict(max_pos=0),
                dict(style=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(q_out=None),
                dict(q=None), dict(H_q=0), dict(P=0), dict(num_pages=0)):
        assert norm_rope(**bad) == K.KV_ERR_ARG, bad
    for bad in (dict(Dh=96), dict(Dh=8), dict(Dh=1024), dict(Dh=512, dtype=0)):
        assert norm_rope(**bad) == K.KV_ERR_UNSUPPORTED, bad
    for bad in (dict(k_new=None), dict(positions=None), dict(cos_sin=None), dict(v_pages=None), dict(v_new=None),
                dict(slots=None), dict(k_pages=None), dict(k_new=PTR + 8), dict(q=PTR + 2), dict(cos_sin=PTR + 4),
                dict(k_out=PTR + 8), dict(q_stride=1020), dict(q_stride=1023), dict(q_stride=0), dict(k_stride=128),
                dict(k_stride=-256), dict(v_stride=255), dict(q_stride=2048),  # q_out = q in place needs the contiguous stride
                dict(k_out=PTR, k_stride=512),
                dict(k_pages=None, v_pages=None, v_new=None, slots=None)):  # nothing to write k to
        assert norm_rope(B=2, **bad) == K.KV_ERR_ARG, bad


def test_int8_cache_refusals():
    L = K.lib()
    base = dict(kp=PTR, vp=PTR, sc=PTR, k=PTR, v=PTR, ks=256, vs=256, dt=1, slots=PTR, B=0, H=2, Dh=128, P=16, n=10,
                err=None, st=None)

    def append(**kw):
        return L.kv_append_int8(*{**base, **kw}.values())

    assert append() == K.KV_OK
    for bad in (dict(B=-1), dict(H=0), dict(Dh=0), dict(P=0), dict(n=0), dict(dt=3), dict(dt=4)):
        assert append(**bad) == K.KV_ERR_ARG, bad
    for bad in (dict(Dh=120), dict(Dh=48), dict(Dh=1024)):
        assert append(**bad) == K.KV_ERR_UNSUPPORTED, bad
    for bad in (dict(kp=None), dict(sc=None), dict(sc=PTR + 4), dict(k=PTR + 2), dict(slots=None), dict(ks=128),
                dict(vs=257), dict(ks=0)):
        assert append(B=2, **bad) == K.KV_ERR_ARG, bad

    base_d = dict(ko=PTR, vo=PTR, dt=1, no=4, kp=PTR, vp=PTR, sc=PTR, src=PTR, dst=PTR, n=0, H=2, Dh=128, P=16, np=10,
                  err=None, st=None)

    def dequant(**kw):
        return L.kv_dequant_pages_int8(*{**base_d, **kw}.values())

    assert dequant() == K.KV_OK
    for bad in (dict(n=-1), dict(dt=3), dict(dt=4), dict(no=0), dict(H=0), dict(np=0)):
        assert dequant(**bad) == K.KV_ERR_ARG, bad
    assert dequant(Dh=72) == K.KV_ERR_UNSUPPORTED
    for bad in (dict(ko=None), dict(src=None), dict(kp=PTR + 8)):
        assert dequant(n=2, **bad) == K.KV_ERR_ARG, bad

    base_c = dict(kp=PTR, vp=PTR, sc=PTR, src=PTR, dst=PTR, n=0, H=2, Dh=128, P=16, np=10, err=None, st=None)

    def copy(**kw):
        return L.kv_copy_pages_int8(*{**base_c, **kw}.values())

    assert copy() == K.KV_OK
    assert copy(n=-1) == K.KV_ERR_ARG and copy(P=0) == K.KV_ERR_ARG
    assert copy(Dh=72) == K.KV_ERR_UNSUPPORTED and copy(H=1, P=15) == K.KV_ERR_UNSUPPORTED
    assert copy(n=1, sc=None) == K.KV_ERR_ARG

    base_a = dict(out=PTR, q=PTR, qd=1, kp=PTR, vp=PTR, sc=PTR, tab=PTR, mb=16, lens=PTR, B=0, Hq=8, H=2, Dh=128, P=16,
                  n=10, scale=0.1, S=1, ws=None, wb=0, err=None, st=None)

    def decode(**kw):
        return L.paged_decode_attention_int8(*{**base_a, **kw}.values())

    assert decode() == K.KV_OK
    for bad in (dict(qd=0), dict(qd=-1), dict(qd=4), dict(B=-1), dict(Hq=7), dict(mb=0), dict(S=-1), dict(n=0)):
        assert decode(**bad) == K.KV_ERR_ARG, bad
    for bad in (dict(Dh=96), dict(P=8), dict(Hq=130), dict(B=70000)):
        assert decode(**bad) == K.KV_ERR_UNSUPPORTED, bad
    for bad in (dict(sc=None), dict(sc=PTR + 4), dict(out=None), dict(q=PTR + 2), dict(tab=None)):
        assert decode(B=1, **bad) == K.KV_ERR_ARG, bad
    assert decode(B=1, n=1 << 27) == K.KV_ERR_UNSUPPORTED  # TMA rows
    # the plain entry points do not take the int8 pool type
    plain = [PTR, PTR, PTR, PTR, PTR, 16, PTR, 1, 8, 2, 128, 16, 10, 0.1, 4, 1, None, 0, None, None]
    assert L.paged_decode_attention(*plain) == K.KV_ERR_ARG
    assert L.kv_append(PTR, PTR, PTR, PTR, PTR, 1, 2, 128, 16, 10, 4, None, None) == K.KV_ERR_ARG


def test_modified_attention_refusals():
    L = K.lib()
    base = dict(out=PTR, q=PTR, kp=PTR, vp=PTR, tab=PTR, mb=16, lens=PTR, B=0, Hq=8, H=2, Dh=128, P=16, n=10, scale=0.1,
                dt=1, cap=0.0, slopes=None, window=0, ks=None, S=1, ws=None, wb=0, err=None, st=None)

    def decode(**kw):
        return L.paged_decode_attention_mod(*{**base, **kw}.values())

    base_p = dict(out=PTR, q=PTR, qs=PTR, mq=4, nr=4, kp=PTR, vp=PTR, tab=PTR, mb=16, lens=PTR, B=0, Hq=8, H=2, Dh=128, P=16,
                  n=10, scale=0.1, dt=1, cap=0.0, slopes=None, window=0, ks=None, pl=None, err=None, st=None)

    def prefill(**kw):
        return L.paged_prefill_attention_mod(*{**base_p, **kw}.values())

    for f in (decode, prefill):
        assert f() == K.KV_OK
        for bad in (dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(window=-1), dict(dt=3), dict(dt=4),
                    dict(B=-1), dict(Hq=7), dict(mb=0), dict(n=0)):
            assert f(**bad) == K.KV_ERR_ARG, bad
        for bad in (dict(dt=0), dict(Dh=96), dict(P=8), dict(Hq=130)):
            assert f(**bad) == K.KV_ERR_UNSUPPORTED, bad
        for bad in (dict(out=None), dict(q=PTR + 2), dict(tab=None), dict(lens=None)):
            assert f(B=1, **bad) == K.KV_ERR_ARG, bad
        assert f(B=1, n=1 << 27) == K.KV_ERR_UNSUPPORTED
    assert decode(S=-1) == K.KV_ERR_ARG
    assert prefill(mq=-1) == K.KV_ERR_ARG and prefill(B=1, mq=0) == K.KV_OK
    assert prefill(nr=-1) == K.KV_ERR_ARG and prefill(B=1, nr=0) == K.KV_OK
    K.paged_decode_set_kernel(K.KV_DECODE_KERNEL_SIMT)  # the selection does not limit the groups of these entry points
    try:
        assert decode(Hq=100, H=2) == K.KV_OK
    finally:
        K.paged_decode_set_kernel(K.KV_DECODE_KERNEL_AUTO)


def test_binding_checks_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    t = torch.zeros((1, 2), dtype=torch.int32)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # CPU tensors
        K.paged_decode_attention_mod(q.float(), q, x, x, t, t[0, :1], 0.1)
    with pytest.raises(ValueError):  # float pools
        K.paged_decode_attention_int8(q.float(), q, x, x, x, t, t[0, :1], 0.1)
    with pytest.raises(ValueError):
        K.kv_append_int8(x, x, x, q, q, t, 16)


# ------------------------------------------------------------------ oracle pins
def test_oracle_visible_interval():
    assert O.visible(9, 20) == (0, 10)
    assert O.visible(9, 20, window=4) == (6, 10) and O.visible(2, 20, window=4) == (0, 3)
    assert O.visible(9, 20, key_start=8) == (8, 10) and O.visible(9, 20, window=4, key_start=3) == (6, 10)
    assert O.visible(9, 20, prefix=15) == (0, 15) and O.visible(9, 12, prefix=15) == (0, 12)
    assert O.visible(9, 20, prefix=3) == (0, 10) and O.visible(9, 20, key_start=12) == (12, 10)  # empty


def test_oracle_attend_row_by_hand():
    q = np.array([[2.0]])
    k, v = np.array([[[1.0]], [[0.5]], [[-1.0]]]), np.array([[[10.0]], [[20.0]], [[np.nan]]])
    cap, slope = 3.0, 0.25
    s0 = cap * math.tanh(1.0 * 2.0 / cap) - slope * 1
    s1 = cap * math.tanh(0.5 * 2.0 / cap)
    want = (10 * math.exp(s0) + 20 * math.exp(s1)) / (math.exp(s0) + math.exp(s1))
    assert abs(O.attend_row(q, k, v, 1, 3, 1.0, cap, [slope])[0, 0] - want) < 1e-12
    assert O.attend_row(q, k, v, 1, 3, 1.0, window=1)[0, 0] == 20.0
    assert O.attend_row(q, k, v, 1, 3, 1.0, key_start=2)[0, 0] == 0.0  # sees nothing
    assert np.isnan(O.attend_row(q, k, v, 2, 3, 1.0)[0, 0])


def test_oracle_quantise_pins():
    c, s = O.quantise_int8(np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1e-31, 0, 0, 0], [1, np.inf, 0, 0]]))
    assert c[0].tolist() == [127, -64, 0, 2] and s[0] == 1.0  # ties to even
    assert c[1:].any() == False and s[1] == 0 and s[2] == 0 and np.isnan(s[3])  # noqa: E712


def test_oracle_norm_rope_by_hand():
    x = np.array([[[3.0, 4.0]]])
    tab = np.array([[1.0, 0.0], [0.0, 1.0]])  # position 1: a quarter turn
    y = O.norm_rope(x, np.array([1.0, 2.0]), 0.0, np.array([1]), tab, "half")
    r = math.sqrt(12.5)
    assert np.allclose(y[0, 0], [-8 / r, 3 / r])
